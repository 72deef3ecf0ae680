"""Gradients of the vocabulary loss where the model is sure of the target: exp(logit - lse) is near 1 there, and the
target's entry of D, exp(logit - lse) - 1, is what is left after the cancellation.

The reference takes D from its definition in 64 bits, with the lse that the call is given.  Bounds, entry by entry:
  * target's entry: the logit counts as exact to 2^-40 of its terms (its products are exact, their sum keeps what its
    roundings lose); lse is subtracted and expm1 taken, a few fp32 roundings of the entry itself: 16 U |D|.
  * other entries: relative (H / 16 + 2) 2^-23 sum |x w| (products added by the tensor cores, 16 at a time, each
    addition possibly truncated), 2^-22 of the exponential, the roundings of its argument.
  * D is held in bf16: 2^-8 of each entry, 2^-16 up to 128 counted positions (two halves).
  * sums over V or n in fp32: (count + 8) 2^-23 of the sum of magnitudes; one rounding of the output, 2^-8."""
import math

import pytest

torch = pytest.importorskip("torch")
from train_util import U, assert_within, loss_backward, loss_forward, make_context  # noqa: E402

pytestmark = pytest.mark.gpu

IGNORE = -100
F64, BF16 = torch.float64, torch.bfloat16


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def _confident(N, n, V, H, seed=0):
    """n counted positions of N whose target has all but 1e-5 .. 1e-2 of the probability (up to a small factor)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7919 * n + 31 * V + H + seed)
    w = (torch.randn(V, H, generator=g, device="cuda") / math.sqrt(H)).to(BF16)
    t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    rest = 10.0 ** (-5 + 3 * torch.rand(N, generator=g, device="cuda", dtype=F64))
    noise = 0.5 * torch.randn(N, H, generator=g, device="cuda").double()
    wt = w[t.long()].double()
    others = torch.logsumexp(noise @ w.double().t(), 1)
    pull = (others - rest.log() - (noise * wt).sum(1)) / (wt * wt).sum(1)
    x = (noise + pull[:, None] * wt).to(BF16)
    keep = torch.randperm(N, generator=g, device="cuda")[:n]
    targets = torch.full_like(t, IGNORE)
    targets[keep] = t[keep]
    gloss = (0.2 + torch.rand(N, generator=g, device="cuda")) / n
    return x, w, targets, gloss


def _check(dx, dw, x, w, t, lse, gloss):
    live = (t != IGNORE).nonzero().squeeze(1)
    n, (V, H) = len(live), w.shape
    xs, ws, g, l = x[live].double(), w.double(), gloss[live].double()[:, None], lse[live].double()[:, None]
    at = t[live].long()[:, None]
    z = xs @ ws.t()
    left = -torch.expm1(z.gather(1, at) - l)
    assert 1e-6 < float(left.min()) and float(left.max()) < 0.5          # (of the inputs, not of the outputs)
    d = torch.exp(z - l).scatter_(1, at, -left)
    held = 2.0 ** -16 if n <= 128 else 2.0 ** -8
    e = (H / 16 + 2) * 2.0 ** -23 * (xs.abs() @ ws.abs().t()) + 2.0 ** -22 + U * (2 * z.abs() + 4 * l.abs() + 4)
    e_d = d * torch.expm1(e)
    e_d.scatter_(1, at, 16 * U * left)
    e_d = g * (e_d + held * (d.abs() + e_d))
    d = g * d
    for got, want, bound in ((dx[live], d @ ws, e_d @ ws.abs() + (V + 8) * 2.0 ** -23 * (d.abs() @ ws.abs())),
                             (dw, d.t() @ xs, e_d.t() @ xs.abs() + (n + 8) * 2.0 ** -23 * (d.abs().t() @ xs.abs()))):
        assert_within(got, want, bound + 2.0 ** -8 * (want.abs() + bound))


@pytest.mark.parametrize("H", [64, 256, 768])
@pytest.mark.parametrize("n", [1, 100, 128, 129, 700])
def test_gradients_where_the_target_is_nearly_certain(enc, n, H):
    x, w, t, gloss = _confident(701, n, 3001, H)
    live = t != IGNORE
    lse = torch.zeros(len(t), device="cuda")
    lse[live] = torch.logsumexp(x[live].double() @ w.double().t(), 1).float()
    dx, dw = loss_backward(enc, x, w, t, lse, gloss)
    _check(dx, dw, x, w, t, lse, gloss)
    only_dx, _ = loss_backward(enc, x, w, t, lse, gloss, want_dw=False)
    _, only_dw = loss_backward(enc, x, w, t, lse, gloss, want_dx=False)
    assert torch.equal(only_dx, dx) and torch.equal(only_dw, dw)
    assert enc.device_status() == 0


@pytest.mark.parametrize("n", [100, 700])
def test_with_the_forward_pass_s_own_lse(enc, n):
    x, w, t, gloss = _confident(701, n, 3001, 256, seed=1)
    _, lse = loss_forward(enc, x, w, t)
    dx, dw = loss_backward(enc, x, w, t, lse, gloss)
    _check(dx, dw, x, w, t, lse, gloss)


def test_several_pieces(enc):
    """Targets in every piece of the vocabulary and in its last, ragged one."""
    x, w, t, gloss = _confident(20000, 20000, 7001, 64)
    lse = torch.cat([torch.logsumexp(x[i:i + 4000].double() @ w.double().t(), 1) for i in range(0, 20000, 4000)]).float()
    dx, dw = loss_backward(enc, x, w, t, lse, gloss)
    assert int(t.max()) >= 6144 and int(t.min()) < 2048
    _check(dx, dw, x, w, t, lse, gloss)


@pytest.mark.parametrize("n", [40, 300])
def test_target_of_no_probability(enc, n):
    """A target whose logit is -inf: the loss is infinite, its entry of D is -1."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    x = torch.rand(n, 64, generator=g, device="cuda").add_(0.1).to(BF16)
    w = torch.randn(500, 64, generator=g, device="cuda").to(BF16)
    w[7] = -float("inf")
    t = torch.randint(8, 500, (n,), generator=g, device="cuda", dtype=torch.int32)
    t[3] = 7
    loss, lse = loss_forward(enc, x, w, t)
    ok = torch.arange(n, device="cuda") != 3
    assert float(loss[3]) == float("inf") and bool(torch.isfinite(loss[ok]).all()) and bool(torch.isfinite(lse).all())
    gloss = torch.full((n,), 0.25, device="cuda")
    _, dw = loss_backward(enc, x, w, t, lse, gloss)
    assert_within(dw[7], -0.25 * x[3].double(), 2.0 ** -8 * 0.25 * x[3].double())
    assert bool(torch.isfinite(dw).all())
