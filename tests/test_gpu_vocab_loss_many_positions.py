"""The table's gradient as a sum over very many positions, none of which cancels another: the tensor cores drop up to
2^-24 of a sum at every step of 16 positions, so that a sum taken in one go is low by 2^-28 a position -- 0.7 % was
measured at 2^20 positions, 10 % at 2^24.

Bound.  At most 65536 positions are summed in one go, 4096 steps, each losing at most 17 last bits of 2^-23 of the sum
so far; the sum grows evenly, so half of that on average, and truncation drops half a bit on average: measured 4e-8 a
step, 2e-4 in all.  2^-11 (4.9e-4) is granted for it.  The mean over the entries' roundings to bf16 is left: 2^-8 of an
entry at most, 2^-8 / sqrt 3 in the root mean square; D's are averaged by the many positions."""
import math

import pytest

torch = pytest.importorskip("torch")
from text_embedding_encoder_gb300 import binding  # noqa: E402
from train_util import loss_backward, loss_forward, make_context, stream, workspace  # noqa: E402

pytestmark = pytest.mark.gpu

IGNORE = -100
F64, BF16 = torch.float64, torch.bfloat16


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def _positive(N, V, H, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(N + 7 * V + H + seed)
    x = torch.rand(N, H, generator=g, device="cuda").add_(0.5).to(BF16)
    w = (0.3 * torch.randn(V, H, generator=g, device="cuda")).to(BF16)
    return x, w, torch.zeros(N, dtype=torch.int32, device="cuda"), g


def _exact(x, w, t, lse, gloss):
    """dx in 64 bits by slices (as a function of the slice), and dw."""
    dw = torch.zeros(w.shape, dtype=F64, device="cuda")
    norms = [0.0, 0.0]
    for a in range(0, len(x), 1 << 20):
        s = slice(a, a + (1 << 20))
        live = t[s] != IGNORE
        d = torch.exp(x[s].double() @ w.double().t() - lse[s].double()[:, None])
        d.scatter_add_(1, t[s].long().clamp(min=0)[:, None], -torch.ones(len(d), 1, dtype=F64, device="cuda"))
        d = torch.where(live[:, None], d * gloss[s].double()[:, None], torch.zeros_like(d))
        dw += d.t() @ x[s].double().nan_to_num(0.0)
        yield s, d @ w.double()
    yield None, dw


def _compare(x, w, t, lse, gloss, dx, dw):
    off = size = 0.0
    for s, want in _exact(x, w, t, lse, gloss):
        if s is None:
            rel = (dw.double() - want) / want
            assert float(rel.abs().max()) <= 2.0 ** -8 + 2.0 ** -9      # one rounding, the sums, D's average
            # the mean of m independent roundings, six standard deviations of 2^-8 / sqrt 3 / sqrt m
            assert abs(float(rel.mean())) <= 2.0 ** -11 + 6 * 2.0 ** -8 / math.sqrt(3 * rel.numel())
        elif dx is not None:
            off += float(((dx[s].double() - want) ** 2).sum())
            size += float((want ** 2).sum())
    # D of five entries or so: rounded like dx itself
    assert dx is None or math.sqrt(off) <= math.sqrt(2) * 2.0 ** -8 / math.sqrt(3) * math.sqrt(size)


@pytest.mark.parametrize("N,V,H", [(65536, 5, 64), (65537, 7, 72), (1 << 18, 5, 64), ((1 << 20) + 77, 9, 64), (1 << 22, 5, 64),
                                   (1 << 24, 5, 8)])
def test_sums_over_many_positions(enc, N, V, H):
    x, w, t, _ = _positive(N, V, H)
    loss, lse = loss_forward(enc, x, w, t)
    gloss = torch.full((N,), 1.0 / N, device="cuda")
    dx, dw = loss_backward(enc, x, w, t, lse, gloss)
    _compare(x, w, t, lse, gloss, dx, dw)
    if N < 1 << 22:
        only_dx, _ = loss_backward(enc, x, w, t, lse, gloss, want_dw=False)
        _, only_dw = loss_backward(enc, x, w, t, lse, gloss, want_dx=False)
        assert torch.equal(only_dx, dx) and torch.equal(only_dw, dw)
    assert enc.device_status() == 0


@pytest.mark.parametrize("live", ["none", "first", "last", "second half", "few"])
def test_counted_positions_anywhere(enc, live):
    """Parts of the batch without any counted position, and parts with a few."""
    N, V, H = 200_001, 300, 64
    x, w, t, g = _positive(N, V, H, seed=1)
    n = torch.arange(N, device="cuda")
    t = (n % V).int()
    keep = {"none": n < 0, "first": n == 0, "last": n == N - 1, "second half": n >= N // 2, "few": n % 5000 == 3}[live]
    t = torch.where(keep, t, torch.full_like(t, IGNORE))
    x[~keep] = float("nan")                                 # not looked at
    _, lse = loss_forward(enc, x, w, t)
    gloss = torch.where(n < N // 2, 1.0, 1e-3).float()      # the parts' largest gradients differ
    dx, dw = loss_backward(enc, x, w, t, lse, gloss)
    assert bool((dx[~keep] == 0).all()) and bool(torch.isfinite(dw).all()) and enc.device_status() == 0
    # each counted position by itself, in 64 bits; at most one rounding of D and one of the output, 2^-8 each of the parts
    rows = keep.nonzero().squeeze(1)
    d = torch.exp(x[rows].double() @ w.double().t() - lse[rows].double()[:, None])
    d.scatter_add_(1, t[rows].long()[:, None], -torch.ones(len(rows), 1, dtype=F64, device="cuda"))
    d *= gloss[rows].double()[:, None]
    for got, want, parts in ((dx[rows], d @ w.double(), d.abs() @ w.double().abs()),
                             (dw, d.t() @ x[rows].double(), d.abs().t() @ x[rows].double().abs())):
        assert bool(((got.double() - want).abs() <= 2.0 ** -8 * (parts + want.abs()) + 2.0 ** -11 * parts).all())


def test_several_pieces_and_parts_give_the_same_bits_again(enc):
    N, V, H = 140_000, 5001, 72
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = torch.randn(N, H, generator=g, device="cuda").to(BF16)
    w = (torch.randn(V, H, generator=g, device="cuda") / 6).to(BF16)
    t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    t[torch.rand(N, generator=g, device="cuda") < 0.5] = IGNORE
    _, lse = loss_forward(enc, x, w, t)
    gloss = torch.rand(N, generator=g, device="cuda")
    a = loss_backward(enc, x, w, t, lse, gloss)
    b = loss_backward(enc, x, w, t, lse, gloss)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # against the same batch in two calls: dx where a part's largest gradient is the same, dw as a sum
    live = t != IGNORE
    d_norm = [loss_backward(enc, x[s].contiguous(), w, t[s].contiguous(), lse[s].contiguous(), gloss[s].contiguous())
              for s in (slice(0, 70_000), slice(70_000, N))]
    want = d_norm[0][1].double() + d_norm[1][1].double()
    # three roundings to bf16 and D's twice over
    assert float((a[1].double() - want).norm()) <= math.sqrt(5) * 2.0 ** -8 / math.sqrt(3) * float(
        (d_norm[0][1].double() ** 2 + d_norm[1][1].double() ** 2).sum().sqrt())
    both = torch.cat([d_norm[0][0], d_norm[1][0]]).double()
    assert float((a[0].double() - both)[live].norm()) <= 2 * 2.0 ** -8 / math.sqrt(3) * float(both.norm())
    # captured, on another workspace
    dx, dw = torch.empty_like(a[0]), torch.empty_like(a[1])
    ws, n = workspace("vocab_loss_backward", N, V, H, slack=4096)
    assert n == binding.workspace_bytes("vocab_loss_backward", N, V, H)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        enc.op("tee_op_vocab_loss_backward", x, w, t, lse, gloss, dx, dw, N, V, H, IGNORE, ws, n, stream())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, a[0]) and torch.equal(dw, a[1]) and bool((ws[n:] == 0xFF).all())
    assert enc.device_status() == 0
