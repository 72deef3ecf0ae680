"""Shared helpers of the training operators' tests: a context, typed calls, and error bounds.

The bounds count roundings: an fp32 operation is off by at most U = 2^-24 relative to its result, a sum of n terms
by at most (its longest chain of additions) U times the sum of the terms' magnitudes, and an output rounded to bf16
by 2^-8 of its value.
"""
import torch

from text_embedding_encoder_gb300 import binding, synth

U = 2.0 ** -24
KIND = {torch.float32: binding.TEE_F32, torch.bfloat16: binding.TEE_BF16}
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# longest chain of additions of a row sum: 32 elements per lane, five shuffles, eight warps
ROW_CHAIN = 45


def make_context():
    return binding.Encoder(synth.TINY, "bf16", max_tokens=64, max_texts=4)


def stream():
    return torch.cuda.current_stream().cuda_stream


def workspace(name, *sizes, slack=0):
    n = binding.workspace_bytes(name, *sizes)
    # a workspace holds no zeros and no numbers to begin with
    return torch.full((n + slack,), 0xFF, dtype=torch.uint8, device="cuda"), n


def rounded(bound, value, dtype):
    """`bound` on an fp32 result plus the rounding of `value` to the output's type."""
    return bound + ROUND[dtype] * (value.abs() + bound)


def assert_within(got, want, bound):
    """Element by element; NaN and infinities have to be in the same places."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    over = ((got - want).abs() - bound.expand_as(want))[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, (float(over.max()), float((got - want)[fine].abs().max()))


def ln_forward(enc, x, gamma, y_dtype, eps=1e-5, stats=True, y=None):
    T, H = x.shape
    y = torch.full((T, H), float("nan"), dtype=y_dtype, device="cuda") if y is None else y
    st = torch.full((T, 2), float("nan"), device="cuda") if stats else None
    enc.op("tee_op_layernorm_forward", x, KIND[x.dtype], gamma, y, KIND[y.dtype], st, T, H, eps, stream())
    return y, st


def ln_backward(enc, dy, x, gamma, stats, res=None, dx=None, guard=0):
    """`guard`: that many bytes behind the workspace are checked to be left alone."""
    T, H = x.shape
    dx = torch.full((T, H), float("nan"), dtype=x.dtype, device="cuda") if dx is None else dx
    dgamma = torch.full((H,), float("nan"), device="cuda")
    ws, n = workspace("layernorm_backward", T, H, slack=guard)
    enc.op("tee_op_layernorm_backward", dy, KIND[dy.dtype], x, KIND[x.dtype], gamma, stats, res, dx, dgamma, T, H,
           ws, n, stream())
    assert not guard or bool((ws[n:] == 0xFF).all())
    return dx, dgamma


def embed_forward(enc, table, ids, y_dtype, scale):
    (V, H), T = table.shape, len(ids)
    y = torch.full((T, H), float("nan"), dtype=y_dtype, device="cuda")
    enc.op("tee_op_embed_forward", table, KIND[table.dtype], ids, y, KIND[y_dtype], T, V, H, scale, stream())
    return y


def embed_backward(enc, dy, ids, V, e_dtype, scale, into=None):
    T, H = dy.shape
    grad = torch.full((V, H), float("nan"), dtype=e_dtype, device="cuda") if into is None else into
    ws, n = workspace("embed_backward", T, V, H)
    enc.op("tee_op_embed_backward", dy, KIND[dy.dtype], ids, grad, KIND[grad.dtype], T, V, H, scale,
           int(into is not None), ws, n, stream())
    return grad


def loss_forward(enc, x, w, targets, ignore=-100):
    (N, H), V = x.shape, len(w)
    loss, lse = (torch.full((N,), float("nan"), device="cuda") for _ in range(2))
    ws, n = workspace("vocab_loss_forward", N, V, H)
    enc.op("tee_op_vocab_loss_forward", x, w, targets, loss, lse, N, V, H, ignore, ws, n, stream())
    return loss, lse


def loss_backward(enc, x, w, targets, lse, gloss, ignore=-100, want_dx=True, want_dw=True):
    (N, H), V = x.shape, len(w)
    dx = torch.full((N, H), float("nan"), dtype=torch.bfloat16, device="cuda") if want_dx else None
    dw = torch.full((V, H), float("nan"), dtype=torch.bfloat16, device="cuda") if want_dw else None
    ws, n = workspace("vocab_loss_backward", N, V, H)
    enc.op("tee_op_vocab_loss_backward", x, w, targets, lse, gloss, dx, dw, N, V, H, ignore, ws, n, stream())
    return dx, dw
