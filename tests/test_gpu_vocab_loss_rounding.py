"""What the vocabulary loss's gradients lose by D in bf16, measured against 64 bits in the norm and held to what the
roundings cost when they are made one by one in 64 bits: above 128 counted positions D = ratio (p - [target]) is
rounded once (its rows divided by the largest upstream gradient), the outputs once; in dx the target's entry counts
with what its rounding left over.

An fp32 value next to a border between two bf16 numbers may fall to the other side: its error is then the same up to
the fp32 error.  So the norms agree up to their own spread: n H or V H (at least 50000) independent roundings, and at
least 129 of the targets' entries of D where those count, which gives the square of the norm a spread of
sqrt(4/5 / 129) = 8 % at most (x^2 of a uniform x), the norm of 4 %.  Kernel and simulation make the same roundings,
so they share that spread; 5 % more than the simulated norm is granted."""
import math

import pytest

torch = pytest.importorskip("torch")
from train_util import loss_backward, loss_forward, make_context  # noqa: E402

pytestmark = pytest.mark.gpu

IGNORE = -100
F64, BF16 = torch.float64, torch.bfloat16


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def _case(N, n, V, H, pull, equal):
    g = torch.Generator(device="cuda")
    g.manual_seed(N + n + V + H)
    w = (torch.randn(V, H, generator=g, device="cuda") / math.sqrt(H)).to(BF16)
    t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn(N, H, generator=g, device="cuda") + pull * torch.rand(N, 1, generator=g, device="cuda") * w[t.long()].float()
    targets = torch.full_like(t, IGNORE)
    keep = torch.randperm(N, generator=g, device="cuda")[:n]
    targets[keep] = t[keep]
    gloss = torch.full((N,), 1.0 / n, device="cuda") if equal else torch.rand(N, generator=g, device="cuda") - 0.3
    return x.to(BF16), w, targets, gloss


@pytest.mark.parametrize("equal", [True, False])
@pytest.mark.parametrize("N,n,V,H,pull", [(600, 129, 3001, 768, 0.0), (600, 600, 3001, 768, 6.0), (1051, 315, 9999, 256, 8.0),
                                          (3000, 3000, 1000, 64, 3.0), (20000, 20000, 5000, 72, 4.0)])
def test_gradients_lose_no_more_than_the_roundings(enc, N, n, V, H, pull, equal):
    x, w, t, gloss = _case(N, n, V, H, pull, equal)
    _, lse = loss_forward(enc, x, w, t)
    dx, dw = loss_backward(enc, x, w, t, lse, gloss)
    live = (t != IGNORE).nonzero().squeeze(1)
    ws, gmax = w.double(), gloss[live].abs().max().double()
    dx_want, dx_sim = torch.empty(2, n, H, dtype=F64, device="cuda")
    dw_want, dw_sim = torch.zeros(2, V, H, dtype=F64, device="cuda")
    for a in range(0, n, 4000):
        rows = live[a:a + 4000]
        xs, at = x[rows].double(), t[rows].long()[:, None]
        d = torch.exp(xs @ ws.t() - lse[rows].double()[:, None])
        d.scatter_add_(1, at, -torch.ones(len(rows), 1, dtype=F64, device="cuda"))
        d *= gloss[rows].double()[:, None]
        held = (d / gmax).to(BF16).double() * gmax
        dx_want[a:a + 4000] = d @ ws
        dw_want += d.t() @ xs
        dw_sim += held.t() @ xs
        held.scatter_(1, at, d.gather(1, at))                   # dx has the target's entry whole
        dx_sim[a:a + 4000] = held @ ws
    for name, got, want, sim in (("dx", dx[live], dx_want, dx_sim), ("dw", dw, dw_want, dw_sim)):
        err = float((got.double() - want).norm())
        by_rounding = float((sim.to(BF16).double() - want).norm())
        print(name, "%.3e of the norm, the roundings %.3e, of the output alone %.3e" % (
            err / float(want.norm()), by_rounding / float(want.norm()), float((want.to(BF16).double() - want).norm() / want.norm())))
        # (fp32: sums of V or n terms, the exponent's argument; 2^-17 of the norm)
        assert err <= 1.05 * by_rounding + 2.0 ** -17 * float(want.norm()), name
    assert enc.device_status() == 0
