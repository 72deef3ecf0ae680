"""The softmax cross entropy over the vocabulary and its gradients, through the C ABI on the GPU, against the
formulas in 64 bits (include/tee_train.h), with error bounds counted from the roundings.

Bounds.  A logit is a sum of H exact products in fp32, each addition off by at most 2^-23 of the magnitudes' sum
(the tensor cores may truncate): e_l = H 2^-23 sum |x w|.  exp2 on the special-function unit is off by 2^-22, its
argument by U times its size.  D is rounded to bf16 (2^-8); the sums over V or N are fp32 again."""
import math

import pytest

from text_embedding_encoder_gb300 import binding

torch = pytest.importorskip("torch")
from train_util import U, assert_within, loss_backward, loss_forward, make_context, stream, workspace  # noqa: E402

pytestmark = pytest.mark.gpu

IGNORE = -100
F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def _inputs(N, V, H, live="some", seed=0, spread=1.0):
    """States and table with an offset of their own, so that the sums over rows and over the vocabulary do not cancel
    and a missing tile shows."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * N + 1009 * V + H + seed)
    x = (0.4 + 0.8 * torch.randn(N, H, generator=g, device="cuda")).to(BF16)
    w = (0.3 + torch.randn(V, H, generator=g, device="cuda")).mul_(spread / math.sqrt(H)).to(BF16)
    t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    keep = torch.zeros(N, dtype=torch.bool, device="cuda")
    if live == "all":
        keep[:] = True
    elif live == "some":
        keep = torch.rand(N, generator=g, device="cuda") < 0.4
    elif live == "first":
        keep[0] = True
    elif live == "last":
        keep[-1] = True
    t = torch.where(keep, t, torch.full_like(t, IGNORE))
    gloss = torch.rand(N, generator=g, device="cuda") * 0.7 - 0.2
    return x, w, t, gloss


def _logits(x, w, t):
    live = (t != IGNORE).nonzero().squeeze(1)
    xs, ws = x[live].double(), w.double()
    z = xs @ ws.t()
    e = len(w[0]) * 2.0 ** -23 * (xs.abs() @ ws.abs().t())
    return live, z, e


def _check_forward(loss, lse, x, w, t):
    live, z, e = _logits(x, w, t)
    assert loss.dtype == lse.dtype == F32
    dead = t == IGNORE
    assert bool((loss[dead] == 0).all()) and bool((lse[dead] == 0).all())
    if not len(live):
        return
    want = torch.logsumexp(z, 1)
    # exponents: 2^-22 and the argument's rounding (p |log2 p| <= 0.54, and the reference exponent's share cancels);
    # sums: 16 per accumulator, 4 chunks of a tile, the tiles' slices and their join, each step with an exp2
    tiles = (len(w) + 255) // 256
    e_lse = e.max(1).values + 2.0 ** -22 + U * (4 * want.abs() + 80 + 8 * (tiles / 16 + 16))
    assert_within(lse[live], want, e_lse + U * want.abs())
    at = t[live].long()[:, None]
    target = z.gather(1, at).squeeze(1)
    assert_within(loss[live], want - target, e_lse + e.gather(1, at).squeeze(1) + U * ((want - target).abs() + target.abs()))


def _check_backward(dx, dw, x, w, t, lse, gloss):
    live, z, e = _logits(x, w, t)
    N, (V, H) = len(x), w.shape
    g = gloss[live].double()[:, None]
    p = torch.exp(z - lse[live].double()[:, None])
    hot = torch.zeros_like(p).scatter_(1, t[live].long()[:, None], 1.0)
    d = g * (p - hot)
    # (below 2^-126 the unit gives 0)
    e_p = p * torch.expm1(e + 2.0 ** -22 + U * (2 * z.abs() + 4 * lse[live].double().abs()[:, None] + 2)) + 2.0 ** -126
    e_d = (g.abs() * e_p + 3 * U * d.abs()) * (1 + 2.0 ** -8) + d.abs() * 2.0 ** -8
    if dx is not None:
        want = torch.zeros(N, H, dtype=F64, device="cuda")
        bound = torch.zeros_like(want)
        aw = w.double().abs()
        want[live] = d @ w.double()
        bound[live] = e_d @ aw + (V + 8) * 2.0 ** -23 * (d.abs() @ aw)
        assert_within(dx, want, bound + 2.0 ** -8 * (want.abs() + bound))
        if len(live) and float(want.norm()) > 0:
            # in the norm the roundings of D and of dx are independent: 2^-8 / sqrt 3 each of their parts, doubled
            part = (d.abs() ** 2 @ aw ** 2).sqrt().norm() + want.norm()
            assert float((dx.double() - want).norm()) <= 2 * 2.0 ** -8 / math.sqrt(3) * float(part) + float((g.abs() * e_p @ aw).norm())
    if dw is not None:
        ax = x[live].double().abs()
        want = d.t() @ x[live].double()
        bound = e_d.t() @ ax + (len(live) + 8) * 2.0 ** -23 * (d.abs().t() @ ax)
        assert_within(dw, want, bound + 2.0 ** -8 * (want.abs() + bound))


def _both(enc, x, w, t, gloss, shift=0.0):
    loss, lse = loss_forward(enc, x, w, t)
    _check_forward(loss, lse, x, w, t)
    # the backward formula holds for any lse; a shift keeps sum p - 1 from cancelling the common part of the rows
    lse = lse - shift
    dx, dw = loss_backward(enc, x, w, t, lse, gloss)
    _check_backward(dx, dw, x, w, t, lse, gloss)
    assert enc.device_status() == 0
    return loss, lse, dx, dw


@pytest.mark.parametrize("V", [1, 2, 63, 64, 65, 255, 256, 257, 1000, 4099])
@pytest.mark.parametrize("N", [1, 5, 127, 129, 256, 257])
def test_rows_and_vocabulary_sizes(enc, N, V):
    x, w, t, g = _inputs(N, V, 72, live="all")
    _both(enc, x, w, t, g, shift=1.0)


@pytest.mark.parametrize("H", [8, 16, 56, 64, 72, 128, 200, 256, 264, 320, 512, 768, 1000, 1024, 2056])
def test_widths(enc, H):
    for N, V in ((300, 700), (3, 5000)):
        x, w, t, g = _inputs(N, V, H)
        t[0] = V - 1
        _both(enc, x, w, t, g, shift=1.0)


@pytest.mark.parametrize("live", ["all", "none", "some", "first", "last"])
@pytest.mark.parametrize("N", [1, 40, 513, 3001])
def test_ignored_positions(enc, N, live):
    x, w, t, g = _inputs(N, 1500, 96, live=live)
    dead = t == IGNORE
    x[dead] = float("nan")                                  # not looked at
    g[dead] = float("inf")
    loss, lse, dx, dw = _both(enc, x, w, t, g)
    assert bool((dx[dead] == 0).all()) and bool(torch.isfinite(dw).all())
    if live == "none":
        assert float(dw.abs().max()) == 0.0


def test_few_rows_many_columns(enc):
    """The products of D are split over slices of the vocabulary where there are few rows."""
    for N, V, H in ((1, 102400, 768), (17, 50001, 768), (300, 30011, 256)):
        x, w, t, g = _inputs(N, V, H, live="all")
        _both(enc, x, w, t, g, shift=1.5)


def test_several_pieces(enc):
    """Enough rows for the vocabulary to be taken in three pieces, the last one ragged."""
    x, w, t, g = _inputs(30000, 9001, 64, live="all")
    assert binding.workspace_bytes("vocab_loss_backward", 30000, 9001, 64) < 2 * 30208 * 9001 * 2   # less than all of D
    _both(enc, x, w, t, g, shift=0.7)
    x, w, t, g = _inputs(40000, 5000, 136)
    a = _both(enc, x, w, t, g)
    b = _both(enc, x, w, t, g)
    assert all(torch.equal(p, q) for p, q in zip(a, b))     # the same bits again


def test_sharp_and_flat_distributions(enc):
    """Logits of several hundred (probabilities of exactly 0 and 1), and all alike."""
    for spread in (300.0, 0.0):
        x, w, t, g = _inputs(200, 3000, 128, live="all", spread=spread)
        _both(enc, x, w, t, g)
    x, w, t, g = _inputs(200, 3000, 128, live="all", spread=20.0)
    best = (x.float() @ w.float().t()).argmax(1).int()
    loss, _ = loss_forward(enc, x, w, best)
    assert bool((loss >= -1e-3).all())


def test_one_gradient_only(enc):
    x, w, t, g = _inputs(400, 2000, 256)
    loss, lse = loss_forward(enc, x, w, t)
    dx, dw = loss_backward(enc, x, w, t, lse, g)
    only_dx, none = loss_backward(enc, x, w, t, lse, g, want_dw=False)
    assert none is None and torch.equal(only_dx, dx)
    none, only_dw = loss_backward(enc, x, w, t, lse, g, want_dx=False)
    assert none is None and torch.equal(only_dw, dw)


def test_upstream_gradients(enc):
    """All zero, of widely different sizes, and tiny ones."""
    x, w, t, _ = _inputs(300, 900, 96, live="all")
    _, lse = loss_forward(enc, x, w, t)
    n = torch.arange(300, device="cuda")
    for g in (torch.zeros(300, device="cuda"), torch.where(n % 3 == 0, 1e3, 1e-3).float(), torch.full((300,), 1e-30, device="cuda"),
              torch.where(n == 7, -5.0, 0.0).float()):
        dx, dw = loss_backward(enc, x, w, t, lse, g)
        _check_backward(dx, dw, x, w, t, lse, g)


def test_nan_and_infinity_stay_in_their_row(enc):
    x, w, t, g = _inputs(50, 600, 64, live="all")
    clean, _ = loss_forward(enc, x, w, t)
    x[3, 5] = float("nan")
    loss, lse = loss_forward(enc, x, w, t)
    ok = torch.arange(50, device="cuda") != 3
    assert bool(torch.isnan(loss[3])) and bool(torch.isnan(lse[3])) and torch.equal(loss[ok], clean[ok])
    dx, dw = loss_backward(enc, x, w, t, lse, g)
    assert bool(torch.isnan(dx[3]).all()) and bool(torch.isfinite(dx[ok]).all()) and bool(torch.isnan(dw).all())


def test_minus_infinity_logits(enc):
    """A table row of -inf against positive states: its probability is 0 and it reaches no other row's loss."""
    x, w, t, _ = _inputs(40, 700, 64, live="all")
    x = x.abs()
    w[256:512] = -float("inf")                              # a whole tile
    w[5] = -float("inf")
    t = torch.where((t >= 256) & (t < 512) | (t == 5), torch.full_like(t, 9), t)
    loss, lse = loss_forward(enc, x, w, t)
    keep = torch.ones(700, dtype=torch.bool, device="cuda")
    keep[256:512] = keep[5] = False
    z = x.double() @ w[keep].double().t()
    assert_within(lse, torch.logsumexp(z, 1), torch.tensor(1e-4, dtype=F64, device="cuda"))
    assert bool(torch.isfinite(loss).all())


def test_infinite_logits(enc):
    """A logit of +inf makes its row's lse and loss infinite, whatever the other logits are and wherever it stands."""
    for v in (5, 70, 300, 699):
        x, w, t, _ = _inputs(40, 700, 64, live="all")
        x = x.abs() + 0.5
        w[v] = float("inf")
        w[(v + 64) % 700] = 30.0                            # logits past 1000 in another part of the row
        w[(v + 128) % 700] = 40.0
        t = torch.where(t == v, torch.full_like(t, (v + 1) % 700), t)
        loss, lse = loss_forward(enc, x, w, t)
        assert bool((lse == float("inf")).all()) and bool((loss == float("inf")).all())


def test_unbounded_table_row_reaches_no_other_row_of_dw(enc):
    """With a table row of -inf the padding behind the last counted position has no defined logits; it adds nothing."""
    x, w, t, g = _inputs(40, 700, 64, live="all")
    x = x.abs()
    w[5] = -float("inf")
    t = torch.where(t == 5, torch.full_like(t, 9), t)
    _, lse = loss_forward(enc, x, w, t)
    _, dw = loss_backward(enc, x, w, t, lse, g)
    keep = torch.arange(700, device="cuda") != 5
    small = torch.where(t > 5, t - 1, t)
    _, want = loss_backward(enc, x, w[keep].contiguous(), small, lse, g)
    assert bool(torch.isfinite(dw).all()) and torch.equal(dw[keep], want) and float(dw[5].abs().max()) == 0.0


@pytest.mark.parametrize("N", [3, 300])
@pytest.mark.parametrize("V", [65, 700, 4099])
def test_all_logits_far_below_zero(enc, N, V):
    """lse is near -150: behind the table's last row, where a tile's logits are 0, exp(0 - lse) would be infinite."""
    x, w, t, g = _inputs(N, V, 64, live="all")
    x, w = x.abs() + 0.5, -1.5 - w.abs()
    _, lse, _, _ = _both(enc, x, w, t, g)
    assert float(lse.max()) < -89.0


def test_out_of_range_targets(enc):
    x, w, t, g = _inputs(60, 500, 64, live="all")
    clean = t.clone()
    clean[[2, 30, 59]] = IGNORE
    want = loss_forward(enc, x, w, clean)
    want_back = loss_backward(enc, x, w, clean, want[1], g)
    assert enc.device_status() == 0
    t[2], t[30], t[59] = 500, -1, 2 ** 31 - 1
    got = loss_forward(enc, x, w, t)
    assert enc.device_status() == binding.TEE_EINVAL and enc.device_status() == 0
    back = loss_backward(enc, x, w, t, got[1], g)
    assert enc.device_status() == binding.TEE_EINVAL and enc.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want + want_back, got + back))


def test_ignore_id_may_be_a_token(enc):
    x, w, t, g = _inputs(300, 40, 64, live="all")
    loss, lse = loss_forward(enc, x, w, t, ignore=3)
    other, _ = loss_forward(enc, x, w, torch.where(t == 3, torch.full_like(t, IGNORE), t))
    assert int((t == 3).sum()) > 0 and torch.equal(loss, other)
    assert enc.device_status() == 0


def test_gradients_against_differences(enc):
    """Central differences of sum(g loss) in 64 bits along random directions."""
    x, w, t, g = _inputs(20, 300, 64, live="some")
    t[:4] = torch.tensor([1, 2, 3, 299], dtype=torch.int32, device="cuda")
    _, lse = loss_forward(enc, x, w, t)
    dx, dw = loss_backward(enc, x, w, t, lse, g)
    live = t != IGNORE

    def f(x, w):
        z = torch.log_softmax(x[live] @ w.t(), 1)
        return -float((g[live].double() * z.gather(1, t[live].long()[:, None]).squeeze(1)).sum())
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    for name, grad in (("x", dx), ("w", dw)):
        a, b = x.double(), w.double()
        u = torch.randn(grad.shape, generator=gen, device="cuda", dtype=F64)
        h = 1e-4
        num = (f(a + h * u, b) - f(a - h * u, b)) / (2 * h) if name == "x" else (f(a, b + h * u) - f(a, b - h * u)) / (2 * h)
        got = float((grad.double() * u).sum())
        # a random direction averages the roundings: six standard deviations of 2 x 2^-8 / sqrt 3 per element of the
        # gradient and of the parts it is made of, plus the differences' own h^2
        d = (torch.softmax(a[live] @ b.t(), 1) * g[live].double()[:, None]).abs()
        parts = (d ** 2 @ b ** 2).sum() + ((g[live].double()[:, None] * b[t[live].long()]) ** 2).sum() if name == "x" \
            else (d.t() ** 2 @ a[live] ** 2).sum() + ((g[live].double()[:, None] * a[live]) ** 2).sum()
        assert abs(num - got) <= 6 * 2 * 2.0 ** -8 / math.sqrt(3) * math.sqrt(float((grad.double() ** 2).sum() + parts)) + 1e-6


def test_no_positions(enc):
    dw = torch.full((100, 64), 3.0, dtype=BF16, device="cuda")
    enc.op("tee_op_vocab_loss_forward", None, None, None, None, None, 0, 100, 64, IGNORE, None, 0, stream())
    enc.op("tee_op_vocab_loss_backward", None, None, None, None, None, None, dw, 0, 100, 64, IGNORE, None, 0, stream())
    assert float(dw.abs().max()) == 0.0


def test_rows_behind_the_outputs_are_left_alone(enc):
    N, V, H = 130, 260, 72
    x, w, t, g = _inputs(N, V, H, live="all")
    want = loss_forward(enc, x, w, t)
    back = loss_backward(enc, x, w, t, want[1], g)
    loss, lse = (torch.full((N + 50,), 7.0, device="cuda") for _ in range(2))
    dx, dw = torch.full((N + 300, H), 7.0, dtype=BF16, device="cuda"), torch.full((V + 300, H), 7.0, dtype=BF16, device="cuda")
    ws, n = workspace("vocab_loss_forward", N, V, H, slack=4096)
    enc.op("tee_op_vocab_loss_forward", x, w, t, loss, lse, N, V, H, IGNORE, ws, n, stream())
    ws2, n2 = workspace("vocab_loss_backward", N, V, H, slack=4096)
    enc.op("tee_op_vocab_loss_backward", x, w, t, lse, g, dx, dw, N, V, H, IGNORE, ws2, n2, stream())
    for a, b in zip(want + back, (loss, lse, dx, dw)):
        assert torch.equal(a, b[:len(a)]) and bool((b[len(a):] == 7.0).all())
    assert bool((ws[n:] == 0xFF).all()) and bool((ws2[n2:] == 0xFF).all())


def test_graph_replay_on_new_inputs_and_counts(enc):
    N, V, H = 700, 1900, 128
    x, w, t, g = _inputs(N, V, H)
    loss, lse = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    dx, dw = torch.empty(N, H, dtype=BF16, device="cuda"), torch.empty(V, H, dtype=BF16, device="cuda")
    ws, n = workspace("vocab_loss_forward", N, V, H)
    ws2, n2 = workspace("vocab_loss_backward", N, V, H)

    def step():
        enc.op("tee_op_vocab_loss_forward", x, w, t, loss, lse, N, V, H, IGNORE, ws, n, stream())
        enc.op("tee_op_vocab_loss_backward", x, w, t, lse, g, dx, dw, N, V, H, IGNORE, ws2, n2, stream())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for live in ("all", "none", "some", "last"):
        x2, _, t2, g2 = _inputs(N, V, H, live=live, seed=5)
        x.copy_(x2), t.copy_(t2), g.copy_(g2)
        graph.replay()
        got = [a.clone() for a in (loss, lse, dx, dw)]
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (loss, lse, dx, dw)))
        _check_forward(loss, lse, x, w, t)
        _check_backward(dx, dw, x, w, t, lse, g)


def test_refusals_launch_nothing(enc):
    N, V, H = 10, 12, 24
    out = torch.full((64, 64), 5.0, device="cuda")
    a, ids = torch.zeros(64, 64, device="cuda"), torch.zeros(64, dtype=torch.int32, device="cuda")
    odd = a.view(-1)[1:]
    s = stream()
    ws, nf = workspace("vocab_loss_forward", N, V, H)
    ws2, nb = workspace("vocab_loss_backward", N, V, H)
    sizes = {"N": [-1, 2 ** 24 + 1], "V": [0, -5, 2 ** 24 + 1], "H": [0, 4, 12, 8200, -8]}
    fwd = [a, a, ids, out, out[32:], N, V, H, IGNORE, ws, nf, s]
    bwd = [a, a, ids, a, a, out, out[32:], N, V, H, IGNORE, ws2, nb, s]
    bad_f = {0: [None, odd], 1: [None, odd], 2: [None], 3: [None], 4: [None], 5: sizes["N"], 6: sizes["V"], 7: sizes["H"],
             9: [None, ws[4:]], 10: [nf - 1, 0]}
    bad_b = {0: [None, odd], 1: [None, odd], 2: [None], 3: [None], 4: [None], 5: [odd], 6: [odd], 7: sizes["N"], 8: sizes["V"],
             9: sizes["H"], 11: [None, ws2[4:]], 12: [nb - 1, 0]}
    for name, args, bad in (("tee_op_vocab_loss_forward", fwd, bad_f), ("tee_op_vocab_loss_backward", bwd, bad_b)):
        for i, values in bad.items():
            for v in values:
                call = list(args)
                call[i] = v
                with pytest.raises(binding.TeeError) as e:
                    enc.op(name, *call)
                assert e.value.code == binding.TEE_EINVAL and name[7:] in str(e.value), (name, i, v)
    call = list(bwd)
    call[5] = call[6] = None
    with pytest.raises(binding.TeeError):
        enc.op("tee_op_vocab_loss_backward", *call)
    torch.cuda.synchronize()
    assert float(out.min()) == 5.0 and float(out.max()) == 5.0
    assert enc.device_status() == 0


@pytest.mark.parametrize("n", [1, 2, 60, 127, 128])
def test_few_positions_are_as_exact_as_the_output_type(enc, n):
    """Up to 128 counted positions D keeps its second half of bits: the gradients' error is their own rounding."""
    x, w, t, _ = _inputs(700, 1500, 256, live="all")
    t[n:] = IGNORE
    t = t[torch.randperm(700, device="cuda")].contiguous()
    g = torch.full((700,), 1.0 / 3, device="cuda")
    _, lse = loss_forward(enc, x, w, t)
    dx, dw = loss_backward(enc, x, w, t, lse, g)
    _check_backward(dx, dw, x, w, t, lse, g)
    live = t != IGNORE
    d = torch.exp(x[live].double() @ w.double().t() - lse[live].double()[:, None])
    d.scatter_add_(1, t[live].long()[:, None], -torch.ones(n, 1, dtype=F64, device="cuda"))
    d = d * g[live].double()[:, None]
    # rounding alone is 2^-8 of the value at most, 2^-8 / sqrt 3 in the norm; 1.15 times that leaves 0.3 of it for D's
    for got, want in ((dx[live], d @ w.double()), (dw, d.t() @ x[live].double())):
        assert float((got.double() - want).norm()) <= 1.15 * 2.0 ** -8 / math.sqrt(3) * float(want.norm())
