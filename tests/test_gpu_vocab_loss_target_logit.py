"""The loss takes the target's logit by a sum of its own and not out of the tensor cores, whose sums are low by 2^-20 of
a logit at 768 columns and 2^-18 at 2048.  Here the target's logit is far from zero and the others are near zero, so
that an error of it shows in the loss (far below zero) or in lse (far above), and the others' errors cannot."""
import math

import pytest

torch = pytest.importorskip("torch")
from train_util import U, assert_within, loss_forward, make_context  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("N,V,H", [(64, 2001, 768), (300, 700, 256), (40, 5000, 2048)])
def test_loss_of_targets_far_from_the_others(enc, N, V, H, sign):
    g = torch.Generator(device="cuda")
    g.manual_seed(N + V + H)
    half, targets_of = H // 2, 8
    # rows 0 .. 7 have columns of their own in the first half, the others all of the second
    w, own = torch.zeros(V, H, device="cuda"), half // targets_of
    for k in range(targets_of):
        w[k, k * own:(k + 1) * own] = torch.randn(own, generator=g, device="cuda") / math.sqrt(own)
    w[targets_of:, half:] = torch.randn(V - targets_of, half, generator=g, device="cuda") / math.sqrt(half)
    w = w.bfloat16()
    t = torch.randint(0, targets_of, (N,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.zeros(N, H, device="cuda")
    x[:, :half] = sign * 150 * w[t.long(), :half].float()       # the target's logit: near +-150
    x[:, half:] = 0.01 * torch.randn(N, half, generator=g, device="cuda")
    x = x.bfloat16()
    loss, lse = loss_forward(enc, x, w, t)
    z = x.double() @ w.double().t()
    at = t.long()[:, None]
    target, want_lse = z.gather(1, at).squeeze(1), torch.logsumexp(z, 1)
    assert float((sign * target).min()) > 60
    # An error of a logit v moves lse by p_v of it.  A tensor-core sum of 16 products and the sum so far drops at most
    # 17 times the last bit, 2^-23, of the largest of them, which is at most max_partial.
    steps = x.double().view(N, 1, H // 16, 16) * w.double().view(1, V, H // 16, 16) if N * V * H < 2 ** 28 else None
    if steps is None:
        products = [(x[i].double() * w.double()).view(V, H // 16, 16) for i in range(N)]
        largest = torch.stack([p.sum(2).cumsum(1).abs().amax(1) for p in products])
        product = torch.stack([p.abs().amax((1, 2)) for p in products])
    else:
        largest, product = steps.sum(3).cumsum(2).abs().amax(2), steps.abs().amax((2, 3))
    e = H / 16 * 17 * 2.0 ** -23 * torch.maximum(largest, product)
    p = torch.exp(z - want_lse[:, None])
    off = (p * e).scatter(1, at, 0.0).sum(1)                    # (the target's is put right)
    # exponentials 2^-22, their arguments and the sums of up to 64 parts in fp32: relative to the sum, as log takes it
    off = off + 2.0 ** -22 + 80 * U
    # with the target nearly certain only what the others add counts
    if sign > 0:
        off = torch.minimum(off, (1 - p.gather(1, at).squeeze(1)) * 0.5 + 2.0 ** -22 + 2 * U * want_lse.abs())
    assert_within(loss, want_lse - target, off + U * (want_lse - target).abs())
    assert_within(lse, want_lse, off + U * want_lse.abs())
