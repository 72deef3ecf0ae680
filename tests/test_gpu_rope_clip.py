"""Rotary positions and the clipping of gradients against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

import layer_util as lu
from text_embedding_encoder_gb300 import binding
from train_util import ROUND, assert_within, make_context, stream, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


# ---- rotary positions ----------------------------------------------------------

def turned(x, pos, heads, base, sign):
    T = len(x)
    angle = pos.double()[:, None] * float(base) ** (-torch.arange(32, device="cuda").double() / 32)
    c, s = angle.cos()[:, None], sign * angle.sin()[:, None]
    x = x.double().view(T, 3 * heads, 2, 32)
    u, v = x[:, :2 * heads, 0], x[:, :2 * heads, 1]
    y = torch.stack([u * c - v * s, v * c + u * s], dim=2)
    # cos and sin off by 2e-7 (an angle by 1e-7 of 2 pi at most, and their own roundings), two products and a sum
    size = (u.abs() + v.abs())[:, :, None].expand_as(y)
    off = torch.cat([size * 5e-7, torch.zeros_like(x[:, 2 * heads:])], dim=1).view(T, -1)
    return torch.cat([y, x[:, 2 * heads:]], dim=1).view(T, -1), off


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,heads", [(1, 1), (3, 12), (259, 4), (1051, 12), (10000, 3), (7, 512)])
def test_rope(enc, T, heads, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn(T, 192 * heads, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 131072, (T,), generator=g, device="cuda").int()
    pos[0] = 0
    for base in (10000.0, 160000.0, 1.0, 0.5):
        for backward in (False, True):
            y = lu.rope(enc, x, pos, heads, base, backward)
            want, off = turned(x, pos, heads, base, -1 if backward else 1)
            assert_within(y, want, off + ROUND[dtype] * (want.abs() + off))
            place = x.clone()
            lu.rope(enc, place, pos, heads, base, backward, y=place)
            assert torch.equal(place, y)
    assert torch.equal(y[0], x[0])          # position 0: no turn


def test_rope_there_and_back(enc):
    x = torch.randn(500, 192 * 2, device="cuda")
    pos = torch.arange(500, device="cuda", dtype=torch.int32)
    back = lu.rope(enc, lu.rope(enc, x, pos, 2, 10000.0), pos, 2, 10000.0, backward=True)
    assert float((back - x).abs().max()) < 2e-6 * float(x.abs().max())


def test_rope_positions_of_texts(enc):
    """The positions that the library's own step gives, and negative ones."""
    lens = [5, 300, 1]
    pos = torch.empty(306, dtype=torch.int32, device="cuda")
    cu = lu.offsets(lens)
    enc2 = binding.Encoder(enc.shape, "bf16", max_tokens=306, max_texts=4)
    enc2.op("tee_op_positions", cu, cu.cpu().numpy(), 3, pos, stream())
    assert torch.equal(pos, lu.positions(lens))
    x = torch.randn(306, 192, device="cuda")
    assert torch.equal(lu.rope(enc, x, -pos, 1, 10000.0), lu.rope(enc, x, pos, 1, 10000.0, backward=True))
    enc2.close()


def test_rope_refusals(enc):
    x, pos = torch.zeros(4, 192, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    good = [x, binding.TEE_F32, pos, x, 4, 1, 10000.0, stream()]
    for name in ("tee_op_rope_forward", "tee_op_rope_backward"):
        for i, v in [(0, None), (0, x.data_ptr() + 4), (1, 2), (2, None), (2, pos.data_ptr() + 1), (3, None), (4, -1),
                     (4, (1 << 24) + 1), (5, 0), (5, 513), (6, 0.0), (6, -1.0), (6, math.inf), (6, math.nan)]:
            args = list(good)
            args[i] = v
            with pytest.raises(binding.TeeError) as e:
                enc.op(name, *args)
            assert e.value.code == binding.TEE_EINVAL
        enc.op(name, None, binding.TEE_F32, None, None, 0, 1, 10000.0, stream())


# ---- clipping -------------------------------------------------------------------

def tensors(sizes, dtypes, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(d) for n, d in zip(sizes, dtypes)]


def check(enc, grads, max_norm, place=False):
    want = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    keep = [t.clone() for t in grads]
    outs = None if place else [torch.full_like(t, float("nan")) for t in grads]
    norm, factor = lu.clip(enc, grads, max_norm, outs).tolist()
    # at most 64 squares to an fp32 sum, the rest in 64 bits
    assert abs(norm - want) <= 2.0 ** -18 * want
    f = min(1.0, max_norm / want) if want else 1.0
    assert abs(factor - f) <= 2.0 ** -18 * f
    for t, o in zip(keep, grads if place else outs):
        exact = t.double() * factor
        assert_within(o, exact, ROUND[t.dtype] * exact.abs() + 2.0 ** -149)
    if not place:
        assert all(torch.equal(a, b) for a, b in zip(keep, grads))


B, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("place", [False, True])
@pytest.mark.parametrize("sizes", [[1], [7], [16384], [16385], [100, 0, 3, 768], [300000, 1, 5000, 17, 70001], [0]])
def test_clip_sizes(enc, sizes, place):
    for dtypes in ([F] * 9, [B] * 9, [B, F, B, F, B]):
        for max_norm in (0.0, 0.5, 1.0, 1e9):
            check(enc, tensors(sizes, dtypes, seed=len(sizes)), max_norm, place)


def test_clip_many_tensors(enc):
    """More than a launch takes, empty ones among them."""
    sizes = [(37 * i) % 3001 for i in range(700)]
    check(enc, tensors(sizes, [B, F] * 350), 3.0)
    check(enc, tensors(sizes, [F, B] * 350), 3.0, place=True)
    check(enc, tensors([0] * 600, [F] * 600), 1.0)


def test_clip_no_tensors(enc):
    norm = torch.full((2,), float("nan"), device="cuda")
    ws, n = workspace("clip_gradients", 0)
    enc.op("tee_op_clip_gradients", None, None, None, None, 0, 1.0, norm, ws, n, stream())
    assert norm.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e18, 1e25, 1e36])
def test_clip_far_magnitudes(enc, scale):
    """Squares that fp32 does not hold."""
    check(enc, tensors([5000, 16384], [F, B], scale=scale), 1.0 if scale > 1 else 1e-28)


def test_clip_zero_and_one_tiny(enc):
    grads = [torch.zeros(50000, device="cuda"), torch.zeros(50000, dtype=B, device="cuda")]
    assert lu.clip(enc, grads, 1.0).tolist() == [0.0, 1.0]
    grads[0][49999] = 1e-40
    norm, factor = lu.clip(enc, grads, 1.0).tolist()
    assert abs(norm - 1e-40) < 1e-44 and factor == 1.0


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_clip_not_finite(enc, value):
    """Passed on as they are; the norm tells."""
    grads = tensors([3000, 20000], [F, B])
    grads[1][777] = value
    keep = [t.clone() for t in grads]
    outs = [torch.zeros_like(t) for t in grads]
    norm, factor = lu.clip(enc, grads, 0.1, outs).tolist()
    assert factor == 1.0 and (math.isnan(norm) if math.isnan(value) else norm == math.inf)
    for a, b in zip(keep, outs):
        assert torch.equal(a.view(torch.int32 if a.dtype == F else torch.int16), b.view(torch.int32 if a.dtype == F else torch.int16))


def test_clip_infinite_max(enc):
    grads = tensors([3000], [F])
    assert lu.clip(enc, grads, math.inf).tolist()[1] == 1.0


def test_clip_views_off_alignment(enc):
    flat = torch.randn(100000, device="cuda")
    half = torch.randn(100000, device="cuda").to(B)
    check(enc, [flat[1:50001], flat[50003:], half[3:40004], half[40005:]], 2.0)
    grads = [flat[1:50001], flat[50003:], half[3:40004], half[40005:]]
    edge = flat[50001:50003].clone()
    check(enc, grads, 1.0, place=True)
    assert torch.equal(edge, flat[50001:50003])


def test_clip_same_bits(enc):
    grads = tensors([1000000, 777, 300001], [B, F, F])
    a = lu.clip(enc, grads, math.inf)
    for _ in range(3):
        assert torch.equal(a, lu.clip(enc, grads, math.inf))


def test_clip_refusals(enc):
    g = tensors([100, 100], [F, F])
    o = [torch.empty_like(t) for t in g]
    ptr = lambda ts: np.array([t.data_ptr() for t in ts], np.uint64)   # noqa: E731
    types, counts = np.zeros(2, np.int32), np.full(2, 100, np.int64)
    norm = torch.zeros(2, device="cuda")
    ws, n = workspace("clip_gradients", 2)
    good = [ptr(g), types, counts, ptr(o), 2, 1.0, norm, ws, n, stream()]
    off = ptr(o)
    off[1] = off[0] + 200
    odd = ptr(g)
    odd[0] += 2
    none = ptr(g)
    none[1] = 0
    for i, v in [(0, None), (0, odd), (0, none), (1, None), (1, np.full(2, 5, np.int32)), (2, None),
                 (2, np.array([-1, 3], np.int64)), (2, np.array([1 << 40, 3], np.int64)), (3, off), (3, ptr([g[1], g[0]])),
                 (3, ptr([o[0], o[0]])), (3, ptr([o[0], g[0]])), (4, -1), (4, 65537), (5, -1.0), (5, math.nan), (6, None),
                 (6, norm.data_ptr() + 2), (7, None), (8, 8)]:
        args = list(good)
        args[i] = v
        with pytest.raises(binding.TeeError) as e:
            enc.op("tee_op_clip_gradients", *args)
        assert e.value.code == binding.TEE_EINVAL, i
    with pytest.raises(binding.TeeError):      # one tensor twice, in place
        enc.op("tee_op_clip_gradients", ptr([g[0], g[0]]), types, counts, None, 2, 1.0, norm, ws, n, stream())


def test_clip_captured(enc):
    grads, outs = tensors([5000, 40000], [F, B]), tensors([5000, 40000], [F, B])
    ws = workspace("clip_gradients", 2)
    norm = None
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        norm = lu.clip(enc, grads, 1.0, outs, ws)
    for seed in (1, 2):
        for t, v in zip(grads, tensors([5000, 40000], [F, B], seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        again = [torch.zeros_like(t) for t in grads]
        assert torch.equal(norm, lu.clip(enc, grads, 1.0, again))
        assert all(torch.equal(a, b) for a, b in zip(outs, again))
