"""Attention of a training step, forward and backward, against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import layer_util as lu
from text_embedding_encoder_gb300 import binding
from train_util import assert_within, make_context, stream, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def inputs(lens, heads, seed, tail=0, spread=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, H = sum(lens) + tail, heads * lu.HD
    qkv = torch.randn(T, 3 * H, generator=g, device="cuda")
    qkv[:, :H] *= spread
    qkv[:, 2 * H:] += 0.5
    do = torch.randn(T, H, generator=g, device="cuda")
    return qkv.bfloat16(), do.bfloat16()


def check(enc, lens, heads, window, seed=0, spread=2.0, tail=0, poison=None):
    """`tail`: rows behind the last text, of NaN."""
    qkv, do = inputs(lens, heads, seed, tail, spread)
    n = sum(lens)
    cu = lu.offsets(lens)
    if tail:
        qkv[n:], do[n:] = float("nan"), float("nan")
    if poison is not None:
        qkv[poison], do[poison] = float("nan"), float("inf")
    o, lse, (ws, size) = lu.attention_forward(enc, qkv, cu, heads, window)
    assert bool((ws[size:] == 0xFF).all())
    dqkv = lu.attention_backward(enc, qkv, cu, o, lse, do, heads, window)
    assert enc.device_status() == binding.TEE_OK
    a = 0
    for m in lens:
        b = a + m
        hit = poison is not None and bool(((poison >= a) & (poison < b)).any())
        if m and not hit:
            att = lu.Attention(qkv[a:b], heads, window)
            want, off, want_lse, lse_off = att.forward()
            assert_within(o[a:b], lu.packed(want), lu.packed(off))
            assert_within(lse[:, a:b], want_lse, lse_off)
            grads, bounds = att.backward(o[a:b], lse[:, a:b], do[a:b])
            assert_within(dqkv[a:b], lu.packed(grads), lu.packed(bounds))
        a = b
    if tail:      # left as they were
        assert bool(torch.isnan(o[n:].float()).all()) and bool(torch.isnan(lse[:, n:]).all())
        assert bool(torch.isnan(dqkv[n:].float()).all())


LENS = [[1], [2], [127], [128], [129], [64, 64], [65, 64], [1] * 130, [8, 37, 64, 150], [256, 256], [300, 5, 1, 0, 200, 0],
        [0, 0, 3], [8, 24, 57, 110, 190, 280, 382], [513, 127, 129, 2, 1000]]


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v[:8])))
@pytest.mark.parametrize("window", [-1, 0, 1, 64, 5000])
def test_lengths(enc, lens, window):
    check(enc, lens, 2, window, seed=len(lens))


@pytest.mark.parametrize("heads", [1, 3, 5, 12, 33])
def test_heads(enc, heads):
    check(enc, [100, 300, 20], heads, -1)
    check(enc, [100, 300, 20], heads, 50)


@pytest.mark.parametrize("window", [127, 128, 129, 200, 333])
def test_wide_windows(enc, window):
    check(enc, [1000, 90, 130, 500], 2, window)


@pytest.mark.parametrize("window", [-1, 16, 64])
def test_rows_behind_the_last_text_are_left_alone(enc, window):
    """They hold NaN, and tiles of keys and of queries reach into them."""
    check(enc, [200, 70, 30, 260], 3, window, tail=150)
    check(enc, [5], 1, window, tail=3)


@pytest.mark.parametrize("window", [-1, 3, 64])
def test_a_text_of_nan_stays_alone(enc, window):
    """Texts that share tiles with it, or whose tiles reach into it, are as if it were not there."""
    rows = torch.arange(140, 152, device="cuda")
    check(enc, [40, 60, 40, 12, 30, 200, 129], 2, window, poison=rows)
    check(enc, [140, 12, 300], 2, window, poison=rows)


def test_nan_outside_the_window(enc):
    """Rows that see no NaN through their window have finite results, in one text."""
    qkv, do = inputs([400], 2, 3)
    clean = qkv.clone()
    qkv[200] = float("nan")
    cu = lu.offsets([400])
    keep = [i for i in range(400) if abs(i - 200) > 20]
    far = [i for i in range(400) if abs(i - 200) > 40]
    o, lse, _ = lu.attention_forward(enc, qkv, cu, 2, 20)
    o2, lse2, _ = lu.attention_forward(enc, clean, cu, 2, 20)
    assert torch.isfinite(o[keep].float()).all() and torch.isfinite(lse[:, keep]).all()
    assert torch.equal(lse[:, keep], lse2[:, keep])
    assert (o[keep].float() - o2[keep].float()).abs().max() < 0.05
    g = lu.attention_backward(enc, qkv, cu, o, lse, do, 2, 20)
    assert torch.isfinite(g[far].float()).all()
    assert torch.isnan(o[200].float()).all() and torch.isnan(g[200].float()).any()


def test_large_scores(enc):
    """Probabilities near 0 and 1, and scores of hundreds."""
    check(enc, [300, 40], 2, -1, spread=40.0)
    check(enc, [300, 40], 2, 64, spread=40.0)


def test_equal_scores(enc):
    """Queries of zero: every key counts the same, dk is zero."""
    qkv, do = inputs([300], 1, 1)
    qkv[:, :64] = 0
    cu = lu.offsets([300])
    o, lse, _ = lu.attention_forward(enc, qkv, cu, 1, -1)
    assert_within(lse, torch.full_like(lse, np.log(300)), torch.full_like(lse, 1e-6, dtype=torch.float64))
    g = lu.attention_backward(enc, qkv, cu, o, lse, do, 1, -1)
    assert bool((g[:, 64:128] == 0).all())
    want = do.double().mean(0)
    assert ((g[:, 128:].double() - want).abs().max()) < 2.0 ** -7 * do.double().abs().mean()


def test_same_bits_and_packing(enc):
    """The same bits again; and a text's results are the same alone and in a batch where its tiles start alike."""
    lens = [700, 150, 20, 40, 600]
    qkv, do = inputs(lens, 4, 9)
    cu = lu.offsets(lens)
    for window in (-1, 64):
        first = lu.attention_forward(enc, qkv, cu, 4, window)[:2]
        g = lu.attention_backward(enc, qkv, cu, *first, do, 4, window)
        for _ in range(3):
            again = lu.attention_forward(enc, qkv, cu, 4, window)[:2]
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
            assert torch.equal(g, lu.attention_backward(enc, qkv, cu, *first, do, 4, window))
    alone, lse, _ = lu.attention_forward(enc, qkv[:700].contiguous(), lu.offsets([700]), 4, -1)
    whole, all_lse, _ = lu.attention_forward(enc, qkv, cu, 4, -1)
    assert torch.equal(alone, whole[:700]) and torch.equal(lse, all_lse[:, :700])


def test_many_texts(enc):
    """More texts than the plan keeps in shared memory."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 12, 6000).tolist()
    lens[3000] = 700
    qkv, do = inputs(lens, 1, 4)
    cu = lu.offsets(lens)
    o, lse, _ = lu.attention_forward(enc, qkv, cu, 1, -1)
    g = lu.attention_backward(enc, qkv, cu, o, lse, do, 1, -1)
    assert enc.device_status() == binding.TEE_OK
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all() and torch.isfinite(g.float()).all()
    for j in (0, 17, 2999, 3000, 3001, 5999):
        a, b = int(cu[j]), int(cu[j + 1])
        if a == b:
            continue
        att = lu.Attention(qkv[a:b], 1, -1)
        want, off, want_lse, lse_off = att.forward()
        assert_within(o[a:b], lu.packed(want), lu.packed(off))
        grads, bounds = att.backward(o[a:b], lse[:, a:b], do[a:b])
        assert_within(g[a:b], lu.packed(grads), lu.packed(bounds))


def test_long_text(enc):
    check(enc, [8192 + 77, 40], 1, -1)


def test_gradients_against_differences(enc):
    """The gradient of sum(o do) by central differences of the operator's own definition in 64 bits."""
    lens, heads = [40, 23], 1
    for window in (-1, 5):
        qkv, do = inputs(lens, heads, 2, spread=1.0)
        cu = lu.offsets(lens)
        o, lse, _ = lu.attention_forward(enc, qkv, cu, heads, window)
        g = lu.attention_backward(enc, qkv, cu, o, lse, do, heads, window)
        x = qkv.double()

        def value(x):
            total, a = 0.0, 0
            for m in lens:
                att = lu.Attention(x[a:a + m], heads, window)
                p = torch.exp(att.s - att.lse[:, :, None])
                total += float((lu.packed(p @ att.v) * do[a:a + m].double()).sum())
                a += m
            return total

        rng = np.random.default_rng(1)
        for _ in range(3):
            way = torch.tensor(rng.standard_normal(x.shape), device="cuda")
            slope = (value(x + 1e-5 * way) - value(x - 1e-5 * way)) / 2e-5
            # every element of g off by at most 2^-6 of the largest of its kind
            assert abs(float((g.double() * way).sum()) - slope) < 2.0 ** -6 * float(g.double().norm()) + 1e-3


def test_bad_offsets_are_refused_on_the_device(enc):
    qkv, do = inputs([300], 1, 1)
    for bad in ([1, 300], [0, 301], [0, 200, 100, 300], [0, -5, 300], [-1, 300]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for window in (-1, 8):
            o, lse, _ = lu.attention_forward(enc, qkv, cu, 1, window)
            assert enc.device_status() == binding.TEE_EINVAL
            assert enc.device_status() == binding.TEE_OK
            assert torch.isnan(o.float()).all() and torch.isnan(lse).all()
            good = torch.zeros(1, 300, device="cuda")
            g = lu.attention_backward(enc, qkv, cu, torch.zeros_like(do), good, do, 1, window)
            assert enc.device_status() == binding.TEE_EINVAL
            assert torch.isnan(g.float()).all()


def test_refusals(enc):
    qkv, do = inputs([64], 1, 1)
    cu, H = lu.offsets([64]), 64
    o, lse = torch.zeros(64, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 64, device="cuda")
    ws, n = workspace("attention_backward", 64, 1, 1)
    st = stream()

    def refused(name, *args):
        with pytest.raises(binding.TeeError) as e:
            enc.op(name, *args)
        assert e.value.code == binding.TEE_EINVAL

    good_f = [qkv, cu, o, lse, 64, 1, 1, -1, ws, n, st]
    good_b = [qkv, cu, o, lse, do, qkv.clone(), 64, 1, 1, -1, ws, n, st]
    for name, good, at in (("tee_op_attention_forward", good_f, 4), ("tee_op_attention_backward", good_b, 6)):
        for i, v in [(0, None), (1, None), (2, None), (3, None), (0, qkv.data_ptr() + 2), (1, cu.data_ptr() + 2),
                     (at, -1), (at, (1 << 24) + 1), (at + 1, -1), (at + 1, (1 << 20) + 1), (at + 2, 0), (at + 2, 513),
                     (at + 4, None), (at + 4, ws.data_ptr() + 8), (at + 5, 16)]:
            args = list(good)
            args[i] = v
            refused(name, *args)
        for none in (at, at + 1):          # nothing to do
            args = list(good)
            args[none] = 0
            enc.op(name, *args)
    refused("tee_op_attention_backward", *good_b[:4], None, *good_b[5:])
    refused("tee_op_attention_backward", *good_b[:5], None, *good_b[6:])


def test_captured_first_replayed_for_other_texts(enc):
    """A graph serves any texts that fit its sizes: n_texts offsets, the last ones equal where there are fewer."""
    T, heads = 600, 2
    qkv, do = inputs([T], heads, 1)
    cu = lu.offsets([600] + [0] * 7)
    o = torch.full((T, heads * 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse, dqkv = torch.full((heads, T), float("nan"), device="cuda"), torch.full_like(qkv, float("nan"))
    wf, nf = workspace("attention_forward", T, 8, heads)
    wb, nb = workspace("attention_backward", T, 8, heads)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        enc.op("tee_op_attention_forward", qkv, cu, o, lse, T, 8, heads, -1, wf, nf, stream())
        enc.op("tee_op_attention_backward", qkv, cu, o, lse, do, dqkv, T, 8, heads, -1, wb, nb, stream())
    for lens in ([600] + [0] * 7, [100] * 6 + [0, 0], [1, 2, 3, 4, 5, 6, 7, 500], [128, 128, 129, 0, 0, 60, 0, 0]):
        cu.copy_(lu.offsets(lens))
        q2, d2 = inputs([T], heads, sum(lens[:2]))
        qkv.copy_(q2)
        do.copy_(d2)
        graph.replay()
        torch.cuda.synchronize()
        n = sum(lens)
        e_o, e_lse, _ = lu.attention_forward(enc, qkv, cu, heads, -1)
        e_g = lu.attention_backward(enc, qkv, cu, e_o, e_lse, do, heads, -1)
        assert torch.equal(o[:n], e_o[:n]) and torch.equal(lse[:, :n], e_lse[:, :n]) and torch.equal(dqkv[:n], e_g[:n])


def test_streams_at_once(enc):
    """Calls on several streams, a workspace each."""
    cases, want = [], []
    for i, (lens, window) in enumerate([([900, 40], -1), ([500, 600], 64), ([30] * 40, -1), ([1500], 100)]):
        qkv, do = inputs(lens, 3, i)
        cases.append((qkv, do, lu.offsets(lens), window))
        o, lse, _ = lu.attention_forward(enc, qkv, cases[-1][2], 3, window)
        want.append((o, lse, lu.attention_backward(enc, qkv, cases[-1][2], o, lse, do, 3, window)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for (qkv, do, cu, window), s in zip(cases, streams):
            with torch.cuda.stream(s):
                o, lse, keep = lu.attention_forward(enc, qkv, cu, 3, window)
                g = torch.full_like(qkv, float("nan"))
                ws, n = workspace("attention_backward", len(qkv), len(cu) - 1, 3)
                enc.op("tee_op_attention_backward", qkv, cu, o, lse, do, g, len(qkv), len(cu) - 1, 3, window, ws, n, stream())
                got.append((o, lse, g, keep, ws))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_same_as_the_encoder_s_step(enc):
    """The pass's own attention step on the same rows: the same kernel, so the same outputs."""
    from text_embedding_encoder_gb300 import synth
    lens = [90, 300, 20, 10, 150]
    e = binding.Encoder(synth.TINY, "bf16", max_tokens=600, max_texts=8)
    e.load_weights(synth.make_weights(synth.TINY, seed=0))
    qkv, _ = inputs(lens, 4, 1)
    cu = lu.offsets(lens)
    h_cu = cu.cpu().numpy()
    for layer, window in ((0, -1), (1, 64)):
        want = torch.empty(570, 256, dtype=torch.bfloat16, device="cuda")
        e.op("tee_op_attention", layer, qkv, cu, h_cu, len(lens), want, stream())
        o, _, _ = lu.attention_forward(e, qkv, cu, 4, window)
        torch.cuda.synchronize()
        assert torch.equal(o, want)
    e.close()
