"""The whole masked-token step against autograd in 64 bits, with the two tensors that the step holds in bf16 between
its operators -- the normalised states and their gradient -- taken over as the operators rounded them.  What is left to
differ is each operator's own arithmetic, so the bounds are those of the outputs' roundings and of D's.

In the norm a rounding to bf16 costs at most 2^-8 / sqrt 3 of the values (the half step 2^-8 of a mantissa near 1,
uniform within it), and roundings of different values are independent: squares add.  5 % on top for the spread of the
sums over at least 800 roundings (4.4 standard deviations of 2.5 % / sqrt 5).  A logit out of the tensor cores was
measured up to 2^-20 of itself low; 2^-18 of the largest is granted, relative to each entry of D.  An exponential below
2^-126 is 0 in fp32.

Without the layers in between all masked positions have the same states; `context` adds to the looked-up rows what those
layers would, so that each has its own."""
import math

import pytest

torch = pytest.importorskip("torch")
from train_util import (U, assert_within, embed_backward, embed_forward, ln_backward, ln_forward, loss_backward,  # noqa: E402
                        loss_forward, make_context)

pytestmark = pytest.mark.gpu

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
IGNORE, MASK, EPS = -100, 4, 1e-5
ROUNDED = 2.0 ** -8 / math.sqrt(3) * 1.05


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


class Held(torch.autograd.Function):
    """The states as the step holds them on the way forward, their gradient likewise on the way back."""
    @staticmethod
    def forward(ctx, y, y_held, dy_held, seen):
        ctx.dy_held, ctx.seen = dy_held, seen
        return y_held

    @staticmethod
    def backward(ctx, dy):
        ctx.seen.append(dy)
        return ctx.dy_held, None, None, None


@pytest.mark.parametrize("context", [0.0, 1.0])
@pytest.mark.parametrize("T,V,H", [(259, 4096, 256), (700, 900, 64), (1051, 3001, 768), (2000, 20000, 384)])
def test_step(enc, T, V, H, context):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    table = (0.2 * torch.randn(V, H, generator=g, device="cuda")).to(BF16)
    gamma = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
    truth = torch.randint(5, V // 2, (T,), generator=g, device="cuda", dtype=torch.int32)   # the upper half: no token
    masked = torch.rand(T, generator=g, device="cuda") < 0.6
    ids = torch.where(masked, torch.full_like(truth, MASK), truth)
    targets = torch.where(masked, truth, torch.full_like(truth, IGNORE))
    n, scale = int(masked.sum()), 2.0
    assert n > 128                                              # D in one bf16 number

    around = context * torch.randn(T, H, generator=g, device="cuda")
    x = embed_forward(enc, table, ids, F32, scale) + around
    y, st = ln_forward(enc, x, gamma, BF16)
    loss, lse = loss_forward(enc, y, table, targets)
    gloss = torch.full((T,), 1.0 / n, device="cuda")
    dy, dtable = loss_backward(enc, y, table, targets, lse, gloss)
    dx, dgamma = ln_backward(enc, dy, x, gamma, st)
    embed_backward(enc, dx, ids, V, BF16, scale, into=dtable)
    assert enc.device_status() == 0

    # the same in 64 bits
    t64, g64, seen = table.double().requires_grad_(), gamma.double().requires_grad_(), []
    x64 = t64[ids.long()] * scale + around.double()
    mean = x64.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x64 - mean) ** 2).mean(1, keepdim=True) + EPS)
    xhat = (x64 - mean) * rstd
    y64 = xhat * g64
    held = Held.apply(y64, y.double(), dy.double(), seen)
    w64 = table.double().requires_grad_()                       # the table as the loss's weight, apart from the lookup
    live = masked.nonzero().squeeze(1)
    z = held[live] @ w64.t()
    at = targets[live].long()[:, None]
    lse64 = torch.logsumexp(z, 1)
    want = (lse64 - z.gather(1, at).squeeze(1)).mean()
    want.backward()

    with torch.no_grad():
        # fp32: 45 additions of a row's mean, as many of its variance, a few operations more
        assert_within(y, y64, 2.0 ** -8 * y64.abs() * (1 + 2.0 ** -8) + 120 * U * (y64.abs() + gamma.double().abs()))
        e = 2.0 ** -18 * float(z.abs().max())
        assert abs(float(loss.double().sum() / n) - float(want)) <= e + 64 * U * float(want)
        assert bool((loss[~masked] == 0).all())
        # (lse is given in fp32: U |lse| on every entry of D)
        d = (torch.exp(z - lse64[:, None]).scatter_add_(1, at, -torch.ones(n, 1, dtype=F64, device="cuda"))) / n
        e_d = e + 2 * U * float(lse64.abs().max())
        none = 2.0 ** -126 / n
        off = float((d.abs() @ w64.abs()).norm()) * e_d + none * math.sqrt(n) * float(w64.abs().sum(0).norm())
        # the states' gradient: its own rounding, and D's of all entries but the target's
        rest = d.clone().scatter_(1, at, 0.0)
        part = float((rest ** 2 @ w64 ** 2).sum())
        assert float((dy.double() - seen[0]).norm()) <= ROUNDED * math.sqrt(float(seen[0].norm()) ** 2 + part) + off
        assert float(dy[~masked].abs().max()) == 0.0
        # the gain's gradient from that gradient: fp32 alone, 120 U of xhat as above, up to 80 more additions
        terms = dy.double().abs().t() @ (xhat.abs() + 1)
        assert bool(((dgamma.double() - g64.grad).abs() <= 200 * U * torch.diagonal(terms)).all())
        # the table's: D's rounding, the loss's share rounded, the lookup's added and rounded again
        share, lookup = w64.grad, t64.grad
        total = share + lookup
        part = d.t() ** 2 @ held[live] ** 2
        off = (d.abs().t() @ held[live].abs()) * e_d + none * held[live].abs().sum(0)
        rows = torch.zeros(V, dtype=torch.bool, device="cuda")
        rows[MASK] = True
        upper = torch.arange(V, device="cuda") >= V // 2
        has_target = torch.zeros_like(rows)
        has_target[truth[masked].long()] = True
        has_token = torch.zeros_like(rows)
        has_token[truth[~masked].long()] = True
        for name, of in (("mask token", rows), ("no token, no target", upper), ("target only", has_target & ~has_token & ~rows),
                         ("token only", has_token & ~has_target), ("token and target", has_token & has_target)):
            if int(of.sum()) * H < 800 and name != "mask token":
                continue
            err = float((dtable.double() - total)[of].norm())
            twice = float((lookup[of] != 0).any()) * float(share[of].norm()) ** 2
            bound = ROUNDED * math.sqrt(float(part[of].sum()) + float(total[of].norm()) ** 2 + twice) + float(off[of].norm()) \
                + 200 * U * float(lookup[of].norm())
            assert err <= bound * (1.2 if name == "mask token" else 1.0), name   # (one row: H roundings, a wider spread)
