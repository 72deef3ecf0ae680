"""Attention of a training step over values that are not finite: they stay where the definition has them, whatever shares a
tile with them, and a batch of nothing else takes about the time of any other.  And over neighbours that are finite."""
import pytest
import torch

import layer_util as lu
from text_embedding_encoder_gb300 import binding
from train_util import assert_within, make_context, stream, workspace

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def inputs(T, heads, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    H = heads * lu.HD
    qkv = torch.randn(T, 3 * H, generator=g, device="cuda")
    qkv[:, 2 * H:] += 0.5
    return qkv.bfloat16(), torch.randn(T, H, generator=g, device="cuda").bfloat16()


def micros(call):
    """The shortest of five calls on the GPU, after one."""
    call()
    times = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        b.synchronize()
        times.append(1000 * a.elapsed_time(b))
    return min(times)


def forward_call(enc, qkv, cu, heads, window):
    T, n = len(qkv), len(cu) - 1
    o, lse = torch.empty(T, heads * lu.HD, dtype=torch.bfloat16, device="cuda"), torch.empty(heads, T, device="cuda")
    ws, size = workspace("attention_forward", T, n, heads)
    return o, lse, lambda: enc.op("tee_op_attention_forward", qkv, cu, o, lse, T, n, heads, window, ws, size, stream())


def backward_call(enc, qkv, cu, o, lse, do, heads, window):
    T, n = len(qkv), len(cu) - 1
    g = torch.empty_like(qkv)
    ws, size = workspace("attention_backward", T, n, heads)
    return g, lambda: enc.op("tee_op_attention_backward", qkv, cu, o, lse, do, g, T, n, heads, window, ws, size, stream())


@pytest.mark.parametrize("lens,window", [([32768], 64), ([700, 1000, 31068], 40000), ([60] * 500 + [100] * 27, -1)],
                         ids=["window", "wide", "short"])
@pytest.mark.parametrize("what", ["all", "k", "v"])
def test_forward_of_nan_takes_no_longer(enc, lens, window, what):
    """At most five times a finite batch's time: rows whose own sums or values are NaN cannot have another output.  (It was 84
    times where each was computed again from its keys, as a row beside another text's NaN has to be.)"""
    heads = 4
    H, T = heads * lu.HD, sum(lens)
    qkv, _ = inputs(T, heads, 1)
    cu = lu.offsets(lens)
    normal = micros(forward_call(enc, qkv, cu, heads, window)[2])
    qkv[:, {"all": slice(None), "k": slice(H, 2 * H), "v": slice(2 * H, None)}[what]] = NAN
    o, lse, call = forward_call(enc, qkv, cu, heads, window)
    took = micros(call)
    assert enc.device_status() == binding.TEE_OK
    assert bool(torch.isnan(o.float()).all())
    assert bool((torch.isfinite(lse) if what == "v" else torch.isnan(lse)).all())
    assert took < 5 * normal, (took, normal)


LENS = [[40, 60, 40, 12, 30, 200, 129], [400], [1] * 70 + [130, 3]]


@pytest.mark.parametrize("lens", LENS, ids=["texts", "one", "ones"])
@pytest.mark.parametrize("window", [-1, 0, 20, 64])
@pytest.mark.parametrize("value", [NAN, INF])
def test_forward_of_scattered_values(enc, lens, window, value):
    """Single elements of V: column c of the rows that see them, and no other."""
    heads, T = 2, sum(lens)
    qkv, _ = inputs(T, heads, 3)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    bad = torch.rand(T, heads * lu.HD, generator=g, device="cuda") < 0.0005
    bad[5, 3] = bad[T - 1, 100] = True
    clean = qkv.clone()
    qkv[:, 2 * heads * lu.HD:][bad] = value
    o, lse, _ = lu.attention_forward(enc, qkv, lu.offsets(lens), heads, window)
    assert enc.device_status() == binding.TEE_OK
    a = 0
    for m in lens:
        att = lu.Attention(clean[a:a + m], heads, window)
        want, off, want_lse, lse_off = att.forward()
        sees = torch.isfinite(att.s[0]).double()
        want, hit = lu.packed(want), sees @ bad[a:a + m].double() > 0
        want[hit] = value
        assert_within(o[a:a + m], want, lu.packed(off))
        assert_within(lse[:, a:a + m], want_lse, lse_off)
        a += m


def row_of_forward(qkv, a, b, i):
    """Output and log sum of row i of the text [a, b) in 64 bits (one head, the whole text), and the output's bound: P rounded
    to bf16 term by term, or not and the sum in fp32 by four chains, the output rounded."""
    x = qkv[a:b].double()
    k, v = x[:, 64:128], x[:, 128:]
    s = k @ qkv[i, :64].double() / 8
    lse = torch.logsumexp(s, 0)
    p = torch.exp(s - lse)
    size, want = p @ v.abs(), p @ v
    off = (lu.HALF + 2.0 ** -12) * size + lu.mma(b - a, size)
    return want, off + lu.HALF * (want.abs() + off), lse


def test_forward_beside_nan_with_the_widest_window(enc):
    """Rows of the longest text that share a tile with texts of NaN are computed again from 131072 keys each: right, and far from
    the two seconds after which a wait gives up."""
    n = 131072
    lens = [1, n, 50]
    T = sum(lens)
    qkv, _ = inputs(T, 1, 5)
    qkv[0], qkv[1 + n:] = NAN, NAN
    o, lse, call = forward_call(enc, qkv, lu.offsets(lens), 1, n)
    took = micros(call)
    assert enc.device_status() == binding.TEE_OK
    assert bool(torch.isnan(o[0].float()).all()) and bool(torch.isnan(o[1 + n:].float()).all())
    assert bool(torch.isfinite(o[1:1 + n].float()).all())
    for i in (1, 40, 127, 128, 70000, n - 1, n):
        want, off, want_lse = row_of_forward(qkv, 1, 1 + n, i)
        assert abs(float(lse[0, i]) - float(want_lse)) < 2e-5
        assert_within(o[i], want, off)
    assert took < 1e6, took


@pytest.mark.parametrize("lens", LENS, ids=["texts", "one", "ones"])
@pytest.mark.parametrize("window", [-1, 0, 20, 64])
@pytest.mark.parametrize("what", ["do", "inf do", "k"])
def test_backward_of_scattered_values(enc, lens, window, what):
    """Single elements of do, or of k with what the forward pass makes of it: in the gradients that they reach, and no other.
    An element of do reaches its own dq, dk of the rows that see it, and column c of their dv; one of k makes every row that
    sees it NaN, and with it the dk and dv of what those see."""
    heads, T = 2, sum(lens)
    H = heads * lu.HD
    qkv, do = inputs(T, heads, 3)
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    bad = torch.rand(T, H, generator=g, device="cuda") < 0.0003
    bad[5, 3] = bad[T - 1, 100] = True
    cu = lu.offsets(lens)
    clean, clean_do = qkv.clone(), do.clone()
    o, lse, _ = lu.attention_forward(enc, qkv, cu, heads, window)
    clean_o, clean_lse = o, lse
    if what == "k":
        qkv[:, H:2 * H][bad] = NAN
        o, lse, _ = lu.attention_forward(enc, qkv, cu, heads, window)
    else:
        do[bad] = INF if what == "inf do" else NAN
    got = lu.attention_backward(enc, qkv, cu, o, lse, do, heads, window)
    assert enc.device_status() == binding.TEE_OK
    a = 0
    for m in lens:
        b = a + m
        att = lu.Attention(clean[a:b], heads, window)
        grads, bounds = att.backward(clean_o[a:b], clean_lse[:, a:b], clean_do[a:b])
        want = [lu.packed(x) for x in grads]
        sees = torch.isfinite(att.s[0]).double()
        by_head = bad[a:b].view(m, heads, lu.HD).any(2)                       # rows with a bad element, for each head
        reached = sees @ by_head.double() > 0                                 # rows that see one
        wide = lambda rows: rows.repeat_interleave(lu.HD, dim=1)              # noqa: E731
        if what == "k":
            want[0][wide(reached)] = NAN
            again = wide(sees @ reached.double() > 0)
            want[1][again] = want[2][again] = NAN
        else:
            want[0][wide(by_head)] = NAN
            want[1][wide(reached)] = NAN
            want[2][sees @ bad[a:b].double() > 0] = INF if what == "inf do" else NAN
        for third in range(3):
            part, off = got[a:b, third * H:(third + 1) * H], lu.packed(bounds[third])
            if what == "inf do" and third < 2:      # infinite or NaN, as their differences come out
                fine = ~torch.isnan(want[third])
                assert not bool(torch.isfinite(part[~fine].float()).any())
                part, off, want[third] = part[fine], off[fine], want[third][fine]
            assert_within(part, want[third], off)
        a = b


@pytest.mark.parametrize("lens,window", [([32768], 64), ([700, 1000, 31068], 40000), ([60] * 500 + [100] * 27, -1)],
                         ids=["window", "wide", "short"])
@pytest.mark.parametrize("what", ["all", "k", "v", "do"])
def test_backward_of_nan_takes_no_longer(enc, lens, window, what):
    heads = 4
    H, T = heads * lu.HD, sum(lens)
    qkv, do = inputs(T, heads, 1)
    cu = lu.offsets(lens)
    o, lse, call = forward_call(enc, qkv, cu, heads, window)
    call()
    g, call = backward_call(enc, qkv, cu, o, lse, do, heads, window)
    normal = micros(call)
    clean = g.clone()
    if what in ("all", "do"):
        do[:] = NAN
    if what != "do":
        qkv[:, {"all": slice(None), "k": slice(H, 2 * H), "v": slice(2 * H, None)}[what]] = NAN
        o, lse, call = forward_call(enc, qkv, cu, heads, window)
        call()
    g, call = backward_call(enc, qkv, cu, o, lse, do, heads, window)
    took = micros(call)
    assert enc.device_status() == binding.TEE_OK
    assert bool(torch.isnan(g[:, :2 * H].float()).all())
    if what == "v":      # dv needs none of v
        assert torch.equal(g[:, 2 * H:], clean[:, 2 * H:])
    else:
        assert bool(torch.isnan(g[:, 2 * H:].float()).all())
    assert took < 5 * normal, (took, normal)


def test_backward_beside_nan_with_the_widest_window(enc):
    """The longest text between two of NaN, with a window as wide: right, and far from the two seconds of a wait."""
    n = 131072
    lens = [1, n, 50]
    T = sum(lens)
    qkv, do = inputs(T, 1, 5)
    cu = lu.offsets(lens)
    o, lse, call = forward_call(enc, qkv, cu, 1, n)
    call()
    for x in (qkv, do, o):
        x[0], x[1 + n:] = NAN, NAN
    lse[:, 0], lse[:, 1 + n:] = NAN, NAN
    g, call = backward_call(enc, qkv, cu, o, lse, do, 1, n)
    took = micros(call)
    assert enc.device_status() == binding.TEE_OK
    assert bool(torch.isnan(g[0].float()).all()) and bool(torch.isnan(g[1 + n:].float()).all())
    assert bool(torch.isfinite(g[1:1 + n].float()).all())
    x, d = qkv[1:1 + n].double(), do[1:1 + n].double()
    q, k, v = x[:, :64], x[:, 64:128], x[:, 128:]
    delta, stat = (d * o[1:1 + n].double()).sum(1), lse[0, 1:1 + n].double()
    for i in (0, 39, 126, 127, 70000, n - 2, n - 1):
        p = torch.exp(k @ q[i] / 8 - stat[i])
        ds = p * (v @ d[i] - delta[i])
        pc = torch.exp(q @ k[i] / 8 - stat)
        dsc = pc * (d @ v[i] - delta)
        # P or dS rounded to bf16 term by term, or not and the sum in fp32 by four chains; dp and delta to 2^-10 of their size
        for part, w, other in ((g[1 + i, :64], ds / 8, k), (g[1 + i, 64:128], dsc / 8, q), (g[1 + i, 128:], pc, d)):
            want, size = w @ other, w.abs() @ other.abs()
            off = (lu.HALF + 2.0 ** -10) * size + lu.mma(n, size)
            assert_within(part, want, off + lu.HALF * (want.abs() + off))
    assert took < 1e6, took


@pytest.mark.parametrize("window", [-1, 16, 64])
def test_finite_neighbours_change_no_bit(enc, window):
    """Another text's values, and those of rows behind the last text, whatever finite ones they are."""
    lens, heads = [40, 200, 60, 30], 2
    n, a, b = sum(lens), 40, 240
    qkv, do = inputs(n + 100, heads, 9)
    cu = lu.offsets(lens)
    other, d_other = inputs(n + 100, heads, 10)
    keep = []
    for scale in (None, 1.0, 1000.0):
        q, d = qkv.clone(), do.clone()
        if scale:
            for rows in (slice(0, a), slice(b, None)):
                q[rows], d[rows] = other[rows] * scale, d_other[rows] * scale
        o, lse, _ = lu.attention_forward(enc, q, cu, heads, window)
        o[n:], lse[:, n:] = (0.0, 0.0) if scale is None else (scale, -scale)
        keep.append((o[a:b], lse[:, a:b], lu.attention_backward(enc, q, cu, o, lse, d, heads, window)[a:b]))
    for other in keep[1:]:
        assert all(torch.equal(x, y) for x, y in zip(keep[0], other))
