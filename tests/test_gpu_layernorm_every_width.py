"""LayerNorm backward at every width: the layout that the kernel takes and the workspace that the host asks for go by two
lists of widths, which have to name the same ones (a call whose layout has another number of warps a row is an error)."""
import pytest

torch = pytest.importorskip("torch")
from train_util import U, ln_backward, ln_forward, make_context  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
PAIRS = [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)]


@pytest.mark.parametrize("part", range(8))
def test_every_width(lib, part):
    enc = make_context()
    g = torch.Generator(device="cuda")
    g.manual_seed(part)
    T = 3
    for H in range(1 + 1024 * part, 1025 + 1024 * part):
        xt, yt = PAIRS[(H // 8) % 4]                        # (every remainder of 8 with every pair)
        x = torch.randn(T, H, generator=g, device="cuda").to(xt)
        dy = torch.randn(T, H, generator=g, device="cuda").to(yt)
        gamma = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
        st = ln_forward(enc, x, gamma, yt)[1]
        dx, dgamma = ln_backward(enc, dy, x, gamma, st, guard=64)
        mean, rstd = st.double().unbind(1)
        xhat = (x.double() - mean[:, None]) * rstd[:, None]
        terms = dy.double() * xhat
        # three terms a column, each three roundings off, and their sum: 8 U of the magnitudes
        assert bool(((dgamma.double() - terms.sum(0)).abs() <= 8 * U * (terms.abs().sum(0) + 1e-3)).all()), H
        u = dy.double() * gamma.double()
        want = rstd[:, None] * (u - u.mean(1, keepdim=True) - xhat * (u * xhat).mean(1, keepdim=True))
        # sums of at most 32 elements a lane, five shuffles and eight warps; 80 U of the terms, and dx's own rounding
        size = rstd[:, None] * (u.abs() + u.abs().mean(1, keepdim=True) + xhat.abs() * (u * xhat).abs().mean(1, keepdim=True))
        assert bool(((dx.double() - want).abs() <= 80 * U * size + (2.0 ** -8 if xt == BF16 else U) * want.abs()).all()), H
    enc.close()
