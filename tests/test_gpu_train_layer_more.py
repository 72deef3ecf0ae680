"""A layer's training operators at their ends: the longest text, tensors past 2^31 elements, outputs inside larger
buffers, calls from two threads and on several streams at once."""
import threading

import numpy as np
import pytest
import torch

import layer_util as lu
from text_embedding_encoder_gb300 import binding
from train_util import assert_within, make_context, stream, workspace

pytestmark = pytest.mark.gpu

B = torch.bfloat16


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def rows(T, heads, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    H = heads * lu.HD
    return (torch.randn(T, 3 * H, generator=g, device="cuda", dtype=B), torch.randn(T, H, generator=g, device="cuda", dtype=B))


def test_the_longest_text(enc):
    """131072 tokens; one more is refused."""
    n = 131072
    qkv, do = rows(n + 1, 1, 1)
    o, lse, _ = lu.attention_forward(enc, qkv[:n], lu.offsets([n]), 1, -1)
    g = lu.attention_backward(enc, qkv[:n], lu.offsets([n]), o, lse, do[:n], 1, -1)
    assert enc.device_status() == binding.TEE_OK
    x = qkv[:n].double()
    q, k, v = x[:, :64], x[:, 64:128], x[:, 128:]
    d, od = do[:n].double(), o.double()
    delta = (d * od).sum(1)
    for i in (0, 1, 70000, n - 1):
        s = k @ q[i] / 8
        want = torch.logsumexp(s, 0)
        assert abs(float(lse[0, i]) - float(want)) < 2e-5
        p = torch.exp(s - lse[0, i].double())
        # P rounded to bf16 term by term, the sum in fp32 (2^-23 of it at each of n / 16 steps), the output rounded
        size = p @ v.abs()
        off = (lu.HALF + 2.0 ** -12) * size + lu.mma(n, size)
        assert_within(o[i], p @ v, off + lu.HALF * ((p @ v).abs() + off))
        ds = p * (v @ d[i] - delta[i])
        size = ds.abs() @ k.abs() / 8
        off = (lu.HALF + 2.0 ** -10) * size + lu.mma(n, size)
        assert_within(g[i, :64], ds @ k / 8, off + lu.HALF * ((ds @ k / 8).abs() + off))
        pc = torch.exp(q @ k[i] / 8 - lse[0].double())
        size = pc @ d.abs()
        off = (lu.HALF + 2.0 ** -12) * size + lu.mma(n, size)
        assert_within(g[i, 128:], pc @ d, off + lu.HALF * ((pc @ d).abs() + off))
    keep = torch.full_like(do, 3.0)
    lu.attention_forward(enc, qkv, lu.offsets([n + 1]), 1, -1, o=keep)
    assert enc.device_status() == binding.TEE_EINVAL
    assert bool((keep == 3).all())


def test_past_two_to_the_31_elements(enc):
    """The last texts of a batch of 3.2e9 elements, against the same texts alone."""
    heads, n, T = 12, 64, 1400000
    H = heads * lu.HD
    lens = [n] * (T // n)
    T = sum(lens)
    tail, dtail = rows(5 * n, heads, 2)
    qkv = torch.zeros(T, 3 * H, dtype=B, device="cuda")
    do = torch.zeros(T, H, dtype=B, device="cuda")
    qkv[-5 * n:], do[-5 * n:] = tail, dtail
    cu, small = lu.offsets(lens), lu.offsets([n] * 5)
    pos = lu.positions([n] * 5)
    for window in (-1, 16):
        o, lse, _ = lu.attention_forward(enc, qkv, cu, heads, window)
        g = lu.attention_backward(enc, qkv, cu, o, lse, do, heads, window)
        want_o, want_lse, _ = lu.attention_forward(enc, tail, small, heads, window)
        want_g = lu.attention_backward(enc, tail, small, want_o, want_lse, dtail, heads, window)
        # (texts may share tiles with others here than alone, so sums may be taken in another order)
        assert float((o[-5 * n:].float() - want_o.float()).abs().max()) <= 2.0 ** -6
        assert float((lse[:, -5 * n:] - want_lse).abs().max()) < 1e-5
        assert float((g[-5 * n:].float() - want_g.float()).abs().max()) <= 2.0 ** -5 * float(want_g.float().abs().max())
        assert bool((o[:1000] == 0).all()) and bool((g[:1000] == 0).all())
    y = lu.rope(enc, qkv, pos.repeat(T // (5 * n) + 1)[:T][torch.arange(T, device="cuda") - T].contiguous(), heads, 10000.0)
    assert torch.isfinite(y[-5 * n:].float()).all()
    place = torch.arange(T - 5 * n, T, device="cuda", dtype=torch.int32)
    assert torch.equal(lu.rope(enc, qkv, torch.arange(T, device="cuda", dtype=torch.int32), heads, 10000.0)[-5 * n:],
                       lu.rope(enc, tail, place, heads, 10000.0))
    del o, g, y, do
    flat = qkv.view(-1)
    norm = lu.clip(enc, [flat], 1e30, [flat])
    want = float(tail.double().square().sum()) ** 0.5
    assert abs(float(norm[0]) - want) < 2.0 ** -18 * want


def test_geglu_past_two_to_the_31_elements(enc):
    """The last rows of 2.2e9 elements of z, against the same rows alone."""
    T, H, I = 1050000, 64, 2104
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=B)
    wi = (torch.randn(2 * I, H, generator=g, device="cuda") / 8).to(B)
    z = lu.geglu_forward(enc, x, wi)
    assert torch.equal(z[-300:], lu.geglu_forward(enc, x[-300:].contiguous(), wi))
    dz = torch.zeros_like(z)
    dz[-300:] = z[-300:]
    dx, dwi = lu.geglu_backward(enc, x, wi, dz)
    ref = lu.Geglu(x[-300:], wi)
    (want, off), (want_w, off_w) = ref.backward(dz[-300:])
    assert_within(dx[-300:], want, off)
    assert bool((dx[:-300] == 0).all())
    # the rows before add nothing, but the sums pass through fp32 from part to part
    assert_within(dwi, want_w, off_w + 2.0 ** -20 * want_w.abs())


def test_guards(enc):
    """Outputs inside larger buffers: nothing around them is written."""
    lens, heads = [200, 70, 129, 3], 3
    T, H = sum(lens), heads * lu.HD
    qkv, do = rows(T, heads, 5)
    cu = lu.offsets(lens)
    for window in (-1, 20):
        big_o = torch.full((T + 400, H), 7.0, dtype=B, device="cuda")
        big_l = torch.full((heads * T + 64,), 7.0, device="cuda")
        big_g = torch.full((T + 400, 3 * H), 7.0, dtype=B, device="cuda")
        o, lse = big_o[200:200 + T], big_l[16:16 + heads * T].view(heads, T)
        lu.attention_forward(enc, qkv, cu, heads, window, o=o, lse=lse)
        lu.attention_backward(enc, qkv, cu, o, lse, do, heads, window, dqkv=big_g[200:200 + T])
        for big, n, a in ((big_o, T, 200), (big_g, T, 200), (big_l, heads * T, 16)):
            assert bool((big[:a] == 7).all()) and bool((big[a + n:] == 7).all())
            assert not bool((big[a:a + n] == 7).all())


def calls(enc, seed):
    """One call of each operator, and what it gives."""
    qkv, do = rows(700, 2, seed)
    cu, pos = lu.offsets([300, 100, 300]), lu.positions([300, 100, 300])
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x, dz = torch.randn(500, 72, generator=g, device="cuda", dtype=B), torch.randn(500, 136, generator=g, device="cuda", dtype=B)
    wi = torch.randn(272, 72, generator=g, device="cuda", dtype=B)
    grads = [torch.randn(5000, generator=g, device="cuda"), torch.randn(70000, generator=g, device="cuda", dtype=B)]
    torch.cuda.current_stream().synchronize()

    def run():
        y = lu.rope(enc, qkv, pos, 2, 10000.0, y=torch.empty_like(qkv))
        o, lse = torch.empty_like(do), torch.empty(2, 700, device="cuda")
        dq, outs = torch.empty_like(qkv), [torch.empty_like(t) for t in grads]
        keep = [workspace(n, 700, 3, 2) for n in ("attention_forward", "attention_backward")]
        enc.op("tee_op_attention_forward", y, cu, o, lse, 700, 3, 2, -1, *keep[0], stream())
        enc.op("tee_op_attention_backward", y, cu, o, lse, do, dq, 700, 3, 2, -1, *keep[1], stream())
        z, dx, dwi = torch.empty_like(dz), torch.empty_like(x), torch.empty_like(wi)
        keep.append(workspace("geglu_backward", 500, 72, 136))
        enc.op("tee_op_geglu_forward", x, wi, z, 500, 72, 136, stream())
        enc.op("tee_op_geglu_backward", x, wi, dz, dx, dwi, 500, 72, 136, *keep[2], stream())
        keep.append(workspace("clip_gradients", 2))
        norm = lu.clip(enc, grads, 1.0, outs, keep[3])
        return [y, o, lse, dq, z, dx, dwi, norm] + outs, keep
    return run


def test_threads_and_streams(enc):
    """Two threads with a stream and workspaces each, one context: the bits of one call after the other."""
    runs = [calls(enc, s) for s in range(4)]
    want = [r()[0] for r in runs]
    torch.cuda.synchronize()
    got, wrong = [None] * 4, []

    def work(ids):
        try:
            for k in ids:
                s = torch.cuda.Stream()
                with torch.cuda.stream(s):
                    for _ in range(5):
                        got[k] = runs[k]()
                    s.synchronize()
        except Exception as e:   # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(ids,)) for ids in ((0, 1), (2, 3))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g[0], w))


def test_clip_numbers_of_tensors_from_the_host(enc):
    """The lists are read before the call returns: they may change at once."""
    grads = [torch.full((1000,), 2.0, device="cuda"), torch.full((1000,), 1.0, device="cuda")]
    outs = [torch.zeros(1000, device="cuda") for _ in grads]
    ptr = np.array([t.data_ptr() for t in grads], np.uint64)
    to = np.array([t.data_ptr() for t in outs], np.uint64)
    types, counts = np.zeros(2, np.int32), np.full(2, 1000, np.int64)
    norm = torch.zeros(2, device="cuda")
    ws, n = workspace("clip_gradients", 2)
    enc.op("tee_op_clip_gradients", ptr, types, counts, to, 2, 1.0, norm, ws, n, stream())
    ptr[:], to[:], types[:], counts[:] = 0, 0, 9, -1
    torch.cuda.synchronize()
    assert abs(float(norm[0]) - 5000 ** 0.5) < 1e-3
    assert abs(float(outs[0][0]) - 2 / 5000 ** 0.5) < 1e-6
