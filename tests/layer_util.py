"""Shared helpers of the tests of a layer's training operators: calls, 64-bit definitions, and error bounds.

As in train_util the bounds count roundings.  A tensor-core sum of n products may drop up to 2^-23 of what it holds at
each of its n / 16 steps, which mma() bounds; an operand rounded to bf16 is off by at most HALF of itself.
"""
import numpy as np
import torch

from train_util import KIND, stream, workspace

HALF = 2.0 ** -8
HD = 64


def mma(n, magnitudes):
    """Error of a tensor-core sum of n products whose magnitudes add up to `magnitudes`."""
    return (n / 16 + 2) * 2.0 ** -23 * magnitudes


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def positions(lens):
    return torch.tensor(np.concatenate([np.arange(n) for n in lens] + [[]]), dtype=torch.int32, device="cuda")


def attention_forward(enc, qkv, cu, heads, window, n_texts=None, o=None, lse=None, st=None):
    T = len(qkv)
    n_texts = len(cu) - 1 if n_texts is None else n_texts
    o = torch.full((T, heads * HD), float("nan"), dtype=torch.bfloat16, device="cuda") if o is None else o
    lse = torch.full((heads, T), float("nan"), device="cuda") if lse is None else lse
    ws, n = workspace("attention_forward", T, n_texts, heads, slack=64)
    enc.op("tee_op_attention_forward", qkv, cu, o, lse, T, n_texts, heads, window, ws, n, stream() if st is None else st)
    return o, lse, (ws, n)


def attention_backward(enc, qkv, cu, o, lse, do, heads, window, dqkv=None):
    T, n_texts = len(qkv), len(cu) - 1
    dqkv = torch.full_like(qkv, float("nan")) if dqkv is None else dqkv
    ws, n = workspace("attention_backward", T, n_texts, heads, slack=64)
    enc.op("tee_op_attention_backward", qkv, cu, o, lse, do, dqkv, T, n_texts, heads, window, ws, n, stream())
    assert bool((ws[n:] == 0xFF).all())
    return dqkv


class Attention:
    """One text's attention in 64 bits: q, k, v [heads, n, 64]."""

    def __init__(self, qkv, heads, window):
        n = len(qkv)
        self.q, self.k, self.v = qkv.double().view(n, 3, heads, HD).permute(1, 2, 0, 3)
        s = self.q @ self.k.transpose(1, 2) / 8
        i = torch.arange(n, device=qkv.device)
        if window >= 0:
            s = s.masked_fill((i[:, None] - i).abs() > window, -torch.inf)
        self.size = (self.q.abs() @ self.k.abs().transpose(1, 2)) / 8       # what a score's error goes by
        self.s, self.lse = s, torch.logsumexp(s, dim=2)

    def score_error(self):
        # the product, its scale and the exponent's fp32 roundings, ex2's 2^-22
        return mma(HD, self.size) + 2.0 ** -22 * (self.size + self.lse.abs()[:, :, None] + 1)

    def forward(self):
        p = torch.exp(self.s - self.lse[:, :, None])
        err = torch.where(p > 0, self.score_error(), 0)
        o = p @ self.v
        # scores, the sum's own error, P rounded, the product's sum
        off = (p * (2 * err + HALF + 2.0 ** -20)) @ self.v.abs() + mma(len(p[0]), p @ self.v.abs())
        lse_off = (p * err).sum(2) + 2.0 ** -20 * (1 + self.lse.abs())
        return o, off + HALF * (o.abs() + off), self.lse, lse_off

    def backward(self, o, lse, do):
        """Gradients [3, heads, n, 64] and their bounds, with o and lse as the operator is given them."""
        heads = len(self.q)
        o, do = (x.double().view(len(x), heads, HD).transpose(0, 1) for x in (o, do))
        p = torch.exp(self.s - lse.double()[:, :, None])
        err = torch.where(p > 0, self.score_error() + 2.0 ** -22 * lse.double().abs()[:, :, None], 0)
        dp, delta = do @ self.v.transpose(1, 2), (do * o).sum(2, keepdim=True)
        dp_size, delta_size = do.abs() @ self.v.abs().transpose(1, 2), (do * o).abs().sum(2, keepdim=True)
        ds = p * (dp - delta)
        ds_off = p * (mma(HD, dp_size) + 2.0 ** -20 * delta_size) + ds.abs() * err
        ds_off = ds_off * 1.01 + HALF * (ds.abs() + ds_off)
        p_off = p * err * 1.01 + HALF * p * 1.01
        n = len(p[0])
        grads, bounds = [], []
        for g, off, size in ((ds @ self.k / 8, ds_off @ self.k.abs() / 8, ds.abs() @ self.k.abs() / 8),
                             (ds.transpose(1, 2) @ self.q / 8, ds_off.transpose(1, 2) @ self.q.abs() / 8,
                              ds.abs().transpose(1, 2) @ self.q.abs() / 8),
                             (p.transpose(1, 2) @ do, p_off.transpose(1, 2) @ do.abs(), p.transpose(1, 2) @ do.abs())):
            off = off * 1.01 + mma(n, size)
            grads.append(g)
            bounds.append(off + HALF * (g.abs() + off))
        return torch.stack(grads), torch.stack(bounds)


def packed(x):
    """[parts, heads, n, 64] as packed rows."""
    return x.permute(2, 0, 1, 3).flatten(1) if x.dim() == 4 else x.transpose(0, 1).flatten(1)


def geglu_forward(enc, x, wi, z=None):
    T, H, I = len(x), x.shape[1], len(wi) // 2
    z = torch.full((T, I), float("nan"), dtype=torch.bfloat16, device="cuda") if z is None else z
    enc.op("tee_op_geglu_forward", x, wi, z, T, H, I, stream())
    return z


def geglu_backward(enc, x, wi, dz, want_dx=True, want_dwi=True):
    T, H, I = len(x), x.shape[1], len(wi) // 2
    dx = torch.full_like(x, float("nan")) if want_dx else None
    dwi = torch.full_like(wi, float("nan")) if want_dwi else None
    ws, n = workspace("geglu_backward", T, H, I, slack=64)
    enc.op("tee_op_geglu_backward", x, wi, dz, dx, dwi, T, H, I, ws, n, stream())
    assert bool((ws[n:] == 0xFF).all())
    return dx, dwi


GELU_OFF = 1e-6          # of GELU and GELU' (erf 1.5e-7, hardware reciprocal and exponential), times |a| where it counts


class Geglu:
    """The gated half in 64 bits, with bounds."""

    def __init__(self, x, wi):
        self.x, self.w = x.double(), wi.double()
        H, I = x.shape[1], len(wi) // 2
        u, size = self.x @ self.w.t(), self.x.abs() @ self.w.abs().t()
        self.a, self.g = u[:, :I], u[:, I:]
        self.a_off, self.g_off = mma(H, size[:, :I]), mma(H, size[:, I:])
        self.cdf = 0.5 * torch.special.erfc(-self.a / 2 ** 0.5)
        self.gelu = self.a * self.cdf
        self.slope = self.cdf + self.a * torch.exp(-self.a ** 2 / 2) / (2 * np.pi) ** 0.5
        self.gelu_off = 1.13 * self.a_off + GELU_OFF + 2.0 ** -21 * self.gelu.abs()

    def forward(self):
        z = self.gelu * self.g
        off = 1.01 * (self.gelu_off * self.g.abs() + self.gelu.abs() * self.g_off) + 2.0 ** -22 * z.abs()
        return z, off + HALF * (z.abs() + off)

    def backward(self, dz):
        dz = dz.double()
        da, dg = dz * self.g * self.slope, dz * self.gelu
        slope_off = 0.8 * self.a_off + GELU_OFF + 2.0 ** -21
        da_off = 1.01 * dz.abs() * (self.g_off * 1.13 + self.g.abs() * slope_off)
        dg_off = 1.01 * dz.abs() * self.gelu_off
        du, off = torch.cat([da, dg], 1), torch.cat([da_off, dg_off], 1)
        off = off + HALF * (du.abs() + off)
        dx, dw = du @ self.w, du.t() @ self.x
        dx_off = off @ self.w.abs() + mma(du.shape[1], du.abs() @ self.w.abs())
        dw_off = off.t() @ self.x.abs() + mma(len(du), du.abs().t() @ self.x.abs())
        return (dx, dx_off + HALF * (dx.abs() + dx_off)), (dw, dw_off + HALF * (dw.abs() + dw_off))


def rope(enc, x, pos, heads, base, backward=False, y=None):
    y = torch.full_like(x, float("nan")) if y is None else y
    enc.op("tee_op_rope_backward" if backward else "tee_op_rope_forward", x, KIND[x.dtype], pos, y, len(x), heads, base,
           stream())
    return y


def clip(enc, grads, max_norm, outs=None, ws=None):
    """`outs` None: in place.  Returns {norm, factor}."""
    n = len(grads)
    ptr = lambda ts: np.array([t.data_ptr() for t in ts], np.uint64)    # noqa: E731
    norm = torch.full((2,), float("nan"), device="cuda")
    ws, size = workspace("clip_gradients", n) if ws is None else ws
    enc.op("tee_op_clip_gradients", ptr(grads), np.array([KIND[t.dtype] for t in grads], np.int32),
           np.array([t.numel() for t in grads], np.int64), None if outs is None else ptr(outs), n, max_norm, norm, ws, size,
           stream())
    return norm
