"""The training LayerNorm and token lookup, forward and backward, through the C ABI on the GPU, against their
formulas in 64 bits (include/tee_train.h), with error bounds counted from the roundings (train_util)."""
import math

import numpy as np
import pytest

from text_embedding_encoder_gb300 import binding

torch = pytest.importorskip("torch")
from train_util import (ROUND, ROW_CHAIN, U, assert_within, embed_backward, embed_forward, ln_backward,  # noqa: E402
                        ln_forward, make_context, rounded, stream, workspace, KIND)

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)]
WIDTHS = [1, 2, 7, 8, 31, 100, 255, 256, 257, 264, 512, 760, 768, 1000, 1001, 1024, 1032, 2047, 2048, 2056, 4096, 5003, 8192]


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# ---- LayerNorm ---------------------------------------------------------------

def _ln_ref(x, gamma, eps):
    x, gamma = x.double(), gamma.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    return (x - mean) * rstd * gamma, mean, rstd


def _check_ln_forward(y, st, x, gamma, eps):
    want, mean, rstd = _ln_ref(x, gamma, eps)
    mag = x.double().abs().mean(1, keepdim=True)
    e_mean = (ROW_CHAIN + 1) * U * mag                       # the mean's error
    # the variance: squares of differences (three roundings each) added up; the mean's error enters squared, and
    # the differences' error from the mean's as 2 e_mean mean|x - mean| -- the sum of (x - mean) is not exactly 0
    var = 1 / rstd ** 2 - eps
    dev = (x.double() - mean).abs().mean(1, keepdim=True)
    e_var = (ROW_CHAIN + 5) * U * var + e_mean ** 2 + 2 * e_mean * U * (ROW_CHAIN + 2) * dev + 2 * U * (var + eps)
    e_rstd = rstd * (0.5 * e_var * rstd ** 2 * 1.01 + 3 * U)
    d = (x.double() - mean).abs()
    bound = gamma.double().abs() * (rstd * (e_mean + U * d) + d * e_rstd) + 3 * U * want.abs()
    assert_within(y, want, rounded(bound, want, y.dtype))
    if st is not None:
        assert_within(st[:, :1], mean, e_mean + U * mean.abs())
        assert_within(st[:, 1:], rstd, e_rstd)


@pytest.mark.parametrize("H", WIDTHS)
def test_ln_forward_widths(enc, H):
    for seed, (tx, ty) in enumerate(TYPES):
        for T in (1, 9, 70):
            g = _gen(100 * H + seed + T)
            x = (_randn(g, T, H) * torch.exp(_randn(g, T, 1)) + 2 * _randn(g, T, 1)).to(tx)
            gamma = 1 + 0.3 * _randn(g, H)
            y, st = ln_forward(enc, x, gamma, ty)
            _check_ln_forward(y, st, x, gamma, 1e-5)


def test_ln_forward_many_rows_and_no_stats(enc):
    g = _gen(5)
    x, gamma = _randn(g, 65537, 96) + 1, 1 + 0.1 * _randn(g, 96)
    y, st = ln_forward(enc, x, gamma, BF16)
    _check_ln_forward(y, st, x, gamma, 1e-5)
    y2, _ = ln_forward(enc, x, gamma, BF16, stats=False)
    assert torch.equal(y, y2)


def test_ln_forward_odd_rows(enc):
    """Constant rows (variance 0), huge offsets, tiny and huge scales, and rows with NaN or an infinity, each for itself."""
    H = 768
    g = _gen(6)
    x = _randn(g, 8, H)
    x[1] = 3.25                         # variance 0: y = 0
    x[2] = x[2] * 1e-12
    x[3] = x[3] * 1e15
    x[4] = x[4] + 1000
    x[5, 17] = float("nan")
    x[6, 767] = float("inf")
    gamma = 1 + 0.1 * _randn(g, H)
    y, st = ln_forward(enc, x, gamma, F32)
    keep = [0, 1, 2, 3, 4, 7]
    _check_ln_forward(y[keep], st[keep], x[keep], gamma, 1e-5)
    assert torch.equal(y[1], torch.zeros_like(y[1]))
    assert bool(torch.isnan(y[5]).all()) and bool(torch.isnan(y[6]).all())


def test_ln_forward_in_place(enc):
    g = _gen(7)
    x, gamma = _randn(g, 300, 1001), 1 + 0.1 * _randn(g, 1001)
    want, _ = ln_forward(enc, x, gamma, F32)
    y, _ = ln_forward(enc, x, gamma, F32, y=x)
    assert torch.equal(y, want)


def _check_ln_backward(dx, dgamma, dy, x, gamma, st, res):
    T, H = x.shape
    mean, rstd = st[:, :1].double(), st[:, 1:].double()
    xh = (x.double() - mean) * rstd
    e_xh = 2 * U * xh.abs()                                 # a difference and a product
    u = dy.double() * gamma.double()
    mu, mux = u.mean(1, keepdim=True), (u * xh).mean(1, keepdim=True)
    want = rstd * (u - mu - xh * mux)
    e_mu = (ROW_CHAIN + 4) * U * u.abs().mean(1, keepdim=True)
    e_mux = (ROW_CHAIN + 7) * U * (u * xh).abs().mean(1, keepdim=True)
    bound = rstd * (e_mu + xh.abs() * e_mux + e_xh * mux.abs()
                    + 5 * U * (u.abs() + mu.abs() + (xh * mux).abs())) + U * want.abs()
    if res is not None:
        want = want + res.double()
        bound = bound + U * want.abs()
    assert_within(dx, want, rounded(bound, want, dx.dtype))
    # rows per lane: at most T / 256 for the grids of this device; then a block's groups and the blocks' partials
    chain = T / 256 + 64
    assert_within(dgamma, (dy.double() * xh).sum(0), (chain + 4) * U * (dy.double() * xh).abs().sum(0))


@pytest.mark.parametrize("H", WIDTHS)
def test_ln_backward_widths(enc, H):
    for seed, (tx, ty) in enumerate(TYPES):
        for T in (1, 9, 70):
            g = _gen(7000 + 100 * H + seed + T)
            x = (_randn(g, T, H) * torch.exp(_randn(g, T, 1)) + 2 * _randn(g, T, 1)).to(tx)
            gamma, dy = 1 + 0.3 * _randn(g, H), _randn(g, T, H).to(ty)
            _, st = ln_forward(enc, x, gamma, ty)
            for res in (None, _randn(g, T, H).to(tx)):
                dx, dgamma = ln_backward(enc, dy, x, gamma, st, res)
                _check_ln_backward(dx, dgamma, dy, x, gamma, st, res)


@pytest.mark.parametrize("T,H", [(5000, 768), (20001, 250), (2500, 1536), (700, 8192), (9000, 8)])
def test_ln_backward_many_rows(enc, T, H):
    g = _gen(T)
    x, gamma, dy = _randn(g, T, H), 1 + 0.3 * _randn(g, H), _randn(g, T, H).to(BF16)
    _, st = ln_forward(enc, x, gamma, BF16)
    dx, dgamma = ln_backward(enc, dy, x, gamma, st)
    _check_ln_backward(dx, dgamma, dy, x, gamma, st, None)
    dx2, dgamma2 = ln_backward(enc, dy, x, gamma, st)
    assert torch.equal(dx, dx2) and torch.equal(dgamma, dgamma2)        # the same bits again


def test_ln_backward_in_place_of_each_input(enc):
    g = _gen(9)
    x, gamma, dy, res = _randn(g, 333, 768), 1 + 0.1 * _randn(g, 768), _randn(g, 333, 768), _randn(g, 333, 768)
    _, st = ln_forward(enc, x, gamma, F32)
    want, dg = ln_backward(enc, dy, x, gamma, st, res)
    for name in ("res", "x", "dy"):
        a = {"x": x.clone(), "dy": dy.clone(), "res": res.clone()}
        dx, dg2 = ln_backward(enc, a["dy"], a["x"], gamma, st, a["res"], dx=a[name])
        assert torch.equal(dx, want) and torch.equal(dg, dg2)


def test_ln_backward_of_no_rows(enc):
    dgamma = torch.full((96,), 7.0, device="cuda")
    enc.op("tee_op_layernorm_backward", None, KIND[F32], None, KIND[F32], None, None, None, None, dgamma, 0, 96, None, 0,
           stream())
    assert float(dgamma.abs().max()) == 0.0


def test_ln_gradients_against_differences(enc):
    """dx and dgamma against central differences of sum(dy y) in 64 bits."""
    g = _gen(10)
    T, H, eps = 3, 40, 1e-5
    x, gamma, dy = _randn(g, T, H), 1 + 0.1 * _randn(g, H), _randn(g, T, H)
    _, st = ln_forward(enc, x, gamma, F32, eps=eps)
    dx, dgamma = ln_backward(enc, dy, x, gamma, st)

    def f(x, gamma):
        return float((dy.double() * _ln_ref(x, gamma, eps)[0]).sum())
    step = 1e-5
    for t, h in [(0, 0), (1, 17), (2, 39)]:
        d = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        d[t, h] = step
        num = (f(x.double() + d, gamma) - f(x.double() - d, gamma)) / (2 * step)
        # truncation ~ step^2 f''' and cancellation ~ 1e-16 / step are below 1e-8; the kernel's own error is fp32's
        assert abs(num - float(dx[t, h])) <= 1e-5 * (1 + abs(num))
        d = torch.zeros(H, dtype=torch.float64, device="cuda")
        d[h] = step
        num = (f(x, gamma.double() + d) - f(x, gamma.double() - d)) / (2 * step)
        assert abs(num - float(dgamma[h])) <= 1e-5 * (1 + abs(num))


# ---- token lookup -------------------------------------------------------------

@pytest.mark.parametrize("H", [1, 3, 8, 24, 62, 96, 250, 256, 264, 768, 1000, 2500])
def test_embed_forward(enc, H):
    for te, ty in TYPES:
        for T, V in ((1, 1), (37, 5), (1051, 777), (8193, 99)):
            g = _gen(H + T)
            table = _randn(g, V, H).to(te)
            ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
            got = embed_forward(enc, table, ids, ty, 27.7)
            # one fp32 product, rounded once more to a bf16 output: equal bits
            assert torch.equal(got, (table[ids.long()].float() * torch.tensor(27.7)).to(ty))
    assert enc.device_status() == 0


def test_embed_out_of_range_ids(enc):
    H, V = 96, 50
    g = _gen(1)
    table = _randn(g, V, H)
    ids = torch.tensor([3, -1, 49, 50, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32, device="cuda")
    got = embed_forward(enc, table, ids, F32, 1.0)
    assert enc.device_status() == binding.TEE_EINVAL and enc.device_status() == 0
    ok = torch.tensor([0, 2, 6], device="cuda")
    assert torch.equal(got[ok], table[ids[ok].long()])
    assert float(got[[1, 3, 4, 5]].abs().max()) == 0.0
    dy = _randn(g, 7, H)
    dy[1] = float("nan")                     # belongs to no row
    grad = embed_backward(enc, dy, ids, V, F32, 1.0)
    assert enc.device_status() == binding.TEE_EINVAL and enc.device_status() == 0
    want = torch.zeros(V, H, device="cuda")
    want[ids[ok].long()] = dy[ok]
    assert torch.equal(grad, want)


def _check_embed_backward(grad, dy, ids, V, scale, old=None):
    T, H = dy.shape
    want = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, ids.long(), dy.double())
    mag = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, ids.long(), dy.double().abs())
    # 8 tokens (T <= 16384) or 32 in a warp, 8 warps, the pieces of a run that crosses blocks in four slices, and their sum
    chain = 8 + 8 + T / 256 + 8 if T <= 16384 else 32 + 8 + T / 1024 + 8
    s = float(np.float32(scale))
    want, bound = want * s, (chain + 1) * U * mag * abs(s)
    if old is not None:
        want = want + old.double()
        bound = bound + U * want.abs()
    hit = torch.zeros(V, dtype=torch.bool, device="cuda")
    hit[ids.long()] = True
    assert_within(grad[hit], want[hit], rounded(bound, want, grad.dtype)[hit])
    rest = torch.zeros_like(grad) if old is None else old
    assert torch.equal(grad[~hit], rest[~hit])


def _ids(kind, T, V, g):
    if kind == "uniform":
        return torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    if kind == "one":                                   # every token the same id
        return torch.full((T,), V - 1, dtype=torch.int32, device="cuda")
    if kind == "descending":
        return (torch.arange(T - 1, -1, -1, device="cuda") % V).int()
    if kind == "runs":                                  # runs of every length around the blocks' 256 tokens
        n = torch.tensor([1, 255, 256, 257, 31, 32, 33, 511, 513, 1, 1, 2, 700], device="cuda")
        return torch.arange(len(n), device="cuda").repeat_interleave(n).repeat(-(-T // int(n.sum())))[:T].int() % V
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    return torch.where(torch.rand(T, generator=g, device="cuda") < 0.4, torch.full_like(ids, V // 2), ids)


@pytest.mark.parametrize("kind", ["uniform", "one", "descending", "runs", "heavy"])
@pytest.mark.parametrize("T,V,H", [(1, 1, 8), (1, 9, 5), (31, 2, 24), (33, 40, 257), (256, 511, 40), (257, 512, 264),
                                   (2561, 513, 96), (8193, 5000, 33), (20000, 300001, 8), (16385, 60000, 72)])
def test_embed_backward(enc, kind, T, V, H):
    for n, (te, ty) in enumerate(TYPES):
        g = _gen(T + H + n)
        ids, dy = _ids(kind, T, V, g), _randn(g, T, H).to(ty)
        grad = embed_backward(enc, dy, ids, V, te, 5.1)
        _check_embed_backward(grad, dy, ids, V, 5.1)
        old = _randn(g, V, H).to(te)
        into = old.clone()
        _check_embed_backward(embed_backward(enc, dy, ids, V, te, 5.1, into=into), dy, ids, V, 5.1, old)
    assert enc.device_status() == 0


@pytest.mark.parametrize("kind", ["uniform", "one", "heavy"])
def test_embed_backward_large(enc, kind):
    T, V, H = 70001, 102400, 768
    g = _gen(3)
    ids, dy = _ids(kind, T, V, g), _randn(g, T, H)
    grad = embed_backward(enc, dy, ids, V, BF16, 1.0)
    _check_embed_backward(grad, dy, ids, V, 1.0)
    assert torch.equal(grad, embed_backward(enc, dy, ids, V, BF16, 1.0))         # the same bits again


def test_embed_backward_passes_nan_to_its_own_row_only(enc):
    T, V, H = 600, 40, 96
    g = _gen(4)
    ids, dy = torch.arange(T, device="cuda").int() % V, _randn(g, T, H)
    dy[13, 5] = float("nan")
    dy[14, 7] = float("inf")
    grad = embed_backward(enc, dy, ids, V, F32, 2.0)
    bad = torch.zeros(V, H, dtype=torch.bool, device="cuda")
    bad[13, 5] = bad[14, 7] = True
    assert bool(torch.isnan(grad[13, 5])) and float(grad[14, 7]) == math.inf
    assert bool(torch.isfinite(grad[~bad]).all())


def test_embed_backward_of_no_tokens(enc):
    grad = torch.full((50, 24), 3.0, device="cuda")
    enc.op("tee_op_embed_backward", None, KIND[F32], None, grad, KIND[F32], 0, 50, 24, 1.0, 1, None, 0, stream())
    assert float(grad.min()) == 3.0
    enc.op("tee_op_embed_backward", None, KIND[F32], None, grad, KIND[F32], 0, 50, 24, 1.0, 0, None, 0, stream())
    assert float(grad.abs().max()) == 0.0


def test_embed_backward_is_the_forward_transposed(enc):
    """<forward(E), dy> = <E, backward(dy)>: the lookup is linear in the table."""
    T, V, H = 900, 300, 64
    g = _gen(8)
    table, dy = _randn(g, V, H), _randn(g, T, H)
    ids = _ids("heavy", T, V, g)
    a = (embed_forward(enc, table, ids, F32, 3.0).double() * dy.double())
    b = (table.double() * embed_backward(enc, dy, ids, V, F32, 3.0).double())
    assert abs(float(a.sum() - b.sum())) <= 64 * U * float(a.abs().sum() + b.abs().sum())


# ---- streams, graphs, refusals ----------------------------------------------------

def test_other_stream_and_graph_replay(enc):
    """The calls run on the stream they are given and can be captured; a replay works on what the buffers then hold."""
    T, V, H = 700, 300, 96
    g = _gen(11)
    table, gamma, ids = _randn(g, V, H), 1 + 0.1 * _randn(g, H), _ids("heavy", T, V, g)
    x, y = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    st, dx, dgamma = torch.empty(T, 2, device="cuda"), torch.empty(T, H, device="cuda"), torch.empty(H, device="cuda")
    grad, dy = torch.empty(V, H, device="cuda"), _randn(g, T, H)
    ws1, n1 = workspace("layernorm_backward", T, H)
    ws2, n2 = workspace("embed_backward", T, V, H)
    f = KIND[F32]

    def step():
        enc.op("tee_op_embed_forward", table, f, ids, x, f, T, V, H, 2.0, stream())
        enc.op("tee_op_layernorm_forward", x, f, gamma, y, f, st, T, H, 1e-5, stream())
        enc.op("tee_op_layernorm_backward", dy, f, x, f, gamma, st, None, dx, dgamma, T, H, ws1, n1, stream())
        enc.op("tee_op_embed_backward", dx, f, ids, grad, f, T, V, H, 2.0, 0, ws2, n2, stream())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    first = [a.clone() for a in (y, dx, dgamma, grad)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    for a, b in zip(first, (y, dx, dgamma, grad)):
        assert torch.equal(a, b)
    table.copy_(_randn(g, V, H))
    dy.copy_(_randn(g, T, H))
    graph.replay()
    got = [a.clone() for a in (y, dx, dgamma, grad)]
    step()
    for a, b, c in zip(got, (y, dx, dgamma, grad), first):
        assert torch.equal(a, b) and not torch.equal(a, c)


def test_refusals_launch_nothing(enc):
    T, V, H = 10, 12, 24
    out = torch.full((64, 64), 5.0, device="cuda")
    a, ids, st = torch.zeros(64, 64, device="cuda"), torch.zeros(64, dtype=torch.int32, device="cuda"), torch.zeros(64, 2, device="cuda")
    odd = a.view(-1)[1:]
    f, s = KIND[F32], stream()
    ws, _ = workspace("embed_backward", T, V, H)
    need_ln, need_e = binding.workspace_bytes("layernorm_backward", T, H), binding.workspace_bytes("embed_backward", T, V, H)
    good = {
        "tee_op_layernorm_forward": [a, f, a, out, f, st, T, H, 1e-5, s],
        "tee_op_layernorm_backward": [a, f, a, f, a, st, a, out, out, T, H, ws, need_ln, s],
        "tee_op_embed_forward": [a, f, ids, out, f, T, V, H, 1.0, s],
        "tee_op_embed_backward": [a, f, ids, out, f, T, V, H, 1.0, 0, ws, need_e, s],
    }
    bad = {
        "tee_op_layernorm_forward": {0: [None, odd], 1: [2, -1], 2: [None, odd], 3: [None, odd], 4: [7], 6: [-1, 2 ** 30 + 1],
                                     7: [0, -3, 8193], 8: [-1.0, float("nan")]},
        "tee_op_layernorm_backward": {0: [None, odd], 1: [2], 2: [None, odd], 3: [3], 4: [None, odd], 5: [None, odd], 6: [odd],
                                      7: [None, odd], 8: [None, odd], 9: [-1, 2 ** 30 + 1], 10: [0, 8193], 11: [None, ws[1:]],
                                      12: [need_ln - 1, 0]},
        "tee_op_embed_forward": {0: [None, odd], 1: [2], 2: [None], 3: [None, odd], 4: [9], 5: [-1, 2 ** 30 + 1], 6: [0, -1], 7: [0, 65537]},
        "tee_op_embed_backward": {0: [None, odd], 1: [2], 2: [None], 3: [None, odd], 4: [9], 5: [-1, 2 ** 30 + 1], 6: [0, -1],
                                  7: [0, 65537], 9: [2, -1], 10: [None, ws[1:]], 11: [need_e - 1, 0]},
    }
    for name, args in good.items():
        for i, values in bad[name].items():
            for v in values:
                call = list(args)
                call[i] = v
                with pytest.raises(binding.TeeError) as e:
                    enc.op(name, *call)
                assert e.value.code == binding.TEE_EINVAL and name[7:] in str(e.value), (name, i, v)
    torch.cuda.synchronize()
    assert float(out.min()) == 5.0 and float(out.max()) == 5.0
    assert enc.device_status() == 0


def test_empty_calls_check_no_device_pointer(enc):
    f, s = KIND[F32], stream()
    enc.op("tee_op_layernorm_forward", None, f, None, None, f, None, 0, 24, 1e-5, s)
    enc.op("tee_op_embed_forward", None, f, None, None, f, 0, 12, 24, 1.0, s)


# widths of each vector size (1, 2, 4, 8) on both sides of where the layout of a row changes
MORE_WIDTHS = [130, 258, 260, 259, 511, 510, 513, 514, 516, 767, 770, 772, 776, 1023, 1022, 1020, 1025, 1026, 1028, 1532, 1534,
               1538, 1540, 2049, 2050, 2052, 4095, 4094, 4092, 4097, 4098, 4100, 8190, 8191]


@pytest.mark.parametrize("H", MORE_WIDTHS)
def test_ln_layouts(enc, H):
    for seed, (tx, ty) in enumerate(TYPES):
        for T in (3, 61):
            g = _gen(90000 + 100 * H + seed + T)
            x = (_randn(g, T, H) * torch.exp(_randn(g, T, 1)) + 2 * _randn(g, T, 1)).to(tx)
            gamma, dy = 1 + 0.3 * _randn(g, H), _randn(g, T, H).to(ty)
            y, st = ln_forward(enc, x, gamma, ty)
            _check_ln_forward(y, st, x, gamma, 1e-5)
            res = _randn(g, T, H).to(tx) if T == 3 else None
            dx, dgamma = ln_backward(enc, dy, x, gamma, st, res, guard=4096)
            _check_ln_backward(dx, dgamma, dy, x, gamma, st, res)


@pytest.mark.parametrize("T,H", [(20001, 251), (5001, 511), (3001, 770), (2501, 1001), (2001, 1537), (1500, 2050), (1301, 4095)])
def test_ln_backward_many_rows_of_odd_widths(enc, T, H):
    for tx, ty in TYPES:
        g = _gen(T + H)
        x, gamma, dy = _randn(g, T, H).to(tx), 1 + 0.3 * _randn(g, H), _randn(g, T, H).to(ty)
        y, st = ln_forward(enc, x, gamma, ty)
        _check_ln_forward(y, st, x, gamma, 1e-5)
        dx, dgamma = ln_backward(enc, dy, x, gamma, st, guard=4096)
        _check_ln_backward(dx, dgamma, dy, x, gamma, st, None)


@pytest.mark.parametrize("H", [1, 2, 3, 5, 7, 8, 9, 17, 30, 33, 66, 130, 250, 258, 514, 999, 1001, 1030])
def test_embed_of_any_width(enc, H):
    """Vectors of every size, rows that begin anywhere in 16 bytes, chunks of many short rows; nothing behind the table."""
    V = 3001
    for seed, (ty, te) in enumerate(TYPES):
        for T in (5, 700, 5000):
            g = _gen(50000 + H + seed + T)
            ids = _ids("heavy", T, V, g)
            dy = _randn(g, T, H).to(ty)
            buf = torch.full((V * H + 64,), 7.0, dtype=te, device="cuda")
            grad = buf[:V * H].view(V, H)
            ws, n = workspace("embed_backward", T, V, H)
            enc.op("tee_op_embed_backward", dy, KIND[ty], ids, grad, KIND[te], T, V, H, 0.5, 0, ws, n, stream())
            _check_embed_backward(grad, dy, ids, V, 0.5)
            assert bool((buf[V * H:] == 7.0).all())
            old = grad.clone()
            embed_backward(enc, dy, ids, V, te, 0.5, into=grad)
            _check_embed_backward(grad, dy, ids, V, 0.5, old=old)
            table = _randn(g, V, H).to(te)
            y = embed_forward(enc, table, ids, ty, 1.5)
            assert torch.equal(y, (table[ids.long()].float() * 1.5).to(ty))
