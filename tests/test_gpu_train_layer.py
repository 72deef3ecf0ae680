"""A whole encoder layer trained with the library's operators, as a training program runs them: LayerNorm, the QKV
projection, rotary positions, attention, the output projection, LayerNorm, the gated feed-forward half, the down
projection, backward through all of it, and the gradients clipped by their common norm.  The four projections are plain
matrix products."""
import pytest
import torch

import layer_util as lu
from text_embedding_encoder_gb300 import binding
from train_util import assert_within, ln_backward, ln_forward, make_context, stream

pytestmark = pytest.mark.gpu

LENS = [8, 37, 0, 64, 150, 300]
HEADS, H, I = 4, 256, 512
B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def parameters(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    return {"ln1": 1 + 0.1 * normal(H), "wqkv": (normal(3 * H, H) * 0.09).to(B), "wo": (normal(H, H) * 0.06).to(B),
            "ln2": 1 + 0.1 * normal(H), "wi": (normal(2 * I, H) * 0.08).to(B), "wd": (normal(H, I) * 0.05).to(B)}


def forward(enc, p, x, pos, cu, window, base):
    s = {"x": x}
    s["y1"], s["st1"] = ln_forward(enc, x, p["ln1"], B)
    qkv = s["y1"] @ p["wqkv"].t()
    s["qkv"] = lu.rope(enc, qkv, pos, HEADS, base, y=qkv)            # in place
    s["o"], s["lse"], _ = lu.attention_forward(enc, s["qkv"], cu, HEADS, window)
    s["x1"] = x + (s["o"] @ p["wo"].t()).float()
    s["y2"], s["st2"] = ln_forward(enc, s["x1"], p["ln2"], B)
    s["z"] = lu.geglu_forward(enc, s["y2"], p["wi"])
    s["out"] = s["x1"] + (s["z"] @ p["wd"].t()).float()
    return s


def backward(enc, p, s, dout, pos, cu, window, base):
    g = {}
    d16 = dout.to(B)
    g["wd"], dz = d16.t() @ s["z"], d16 @ p["wd"]
    dy2, g["wi"] = lu.geglu_backward(enc, s["y2"], p["wi"], dz)
    dx1, g["ln2"] = ln_backward(enc, dy2, s["x1"], p["ln2"], s["st2"], res=dout)
    d16 = dx1.to(B)
    g["wo"], do = d16.t() @ s["o"], d16 @ p["wo"]
    dqkv = lu.attention_backward(enc, s["qkv"], cu, s["o"], s["lse"], do, HEADS, window)
    dqkv = lu.rope(enc, dqkv, pos, HEADS, base, backward=True, y=dqkv)
    g["wqkv"], dy1 = dqkv.t() @ s["y1"], dqkv @ p["wqkv"]
    dx, g["ln1"] = ln_backward(enc, dy1, s["x"], p["ln1"], s["st1"], res=dx1)
    return dx, g


def definition(p, x, lens, window, base):
    """The layer in 64 bits, by torch's own derivatives."""
    def norm(x, gain):
        return torch.nn.functional.layer_norm(x, (H,), eps=1e-5) * gain

    def text(qkv):
        n = len(qkv)
        q, k, v = qkv.view(n, 3, HEADS, 64).permute(1, 2, 0, 3)
        angle = torch.arange(n, device="cuda").double()[:, None] * base ** (-torch.arange(32, device="cuda").double() / 32)
        c, s = angle.cos(), angle.sin()

        def turn(u):
            a, b = u[..., :32], u[..., 32:]
            return torch.cat([a * c - b * s, b * c + a * s], dim=-1)

        z = turn(q) @ turn(k).transpose(1, 2) / 8
        if window >= 0:
            i = torch.arange(n, device="cuda")
            z = z.masked_fill((i[:, None] - i).abs() > window, -torch.inf)
        return (torch.softmax(z, 2) @ v).transpose(0, 1).reshape(n, H)

    qkv = norm(x, p["ln1"]) @ p["wqkv"].t()
    o = torch.cat([text(part) for part in qkv.split(lens) if len(part)])
    x1 = x + o @ p["wo"].t()
    u = norm(x1, p["ln2"]) @ p["wi"].t()
    return x1 + (torch.nn.functional.gelu(u[:, :I]) * u[:, I:]) @ p["wd"].t()


def batch(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T = sum(LENS)
    return torch.randn(T, H, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda") / T


@pytest.mark.parametrize("window,base", [(-1, 160000.0), (64, 10000.0)])
def test_layer(enc, window, base):
    p, (x, dout) = parameters(), batch(1)
    cu, pos = lu.offsets(LENS), lu.positions(LENS)
    s = forward(enc, p, x, pos, cu, window, base)
    dx, grads = backward(enc, p, s, dout, pos, cu, window, base)
    assert enc.device_status() == binding.TEE_OK

    p64 = {k: v.double().requires_grad_() for k, v in p.items()}
    x64 = x.double().requires_grad_()
    out = definition(p64, x64, LENS, window, base)
    out.backward(dout.double())
    # Every path takes at most eight tensors rounded to bf16 on its way forward (the norm's output, qkv before and after its
    # rotation, P, o, its projection, the second norm's output and z or its projection) and as many back; a rounding moves
    # a tensor by at most 2^-8 of its norm, and as roundings are without a sign their effects add up as squares.
    bound = 2.0 ** -8 * 16 ** 0.5

    def off(got, want):
        return float((got.double() - want).norm() / want.norm())

    assert off(s["out"], out.detach()) < bound
    assert off(dx, x64.grad) < bound
    for k in p:
        assert off(grads[k], p64[k].grad) < bound, k

    # clipped in place, by the norm of what the step made
    names = sorted(grads)
    keep = {k: grads[k].clone() for k in names}
    total = sum(float(grads[k].double().square().sum()) for k in names) ** 0.5
    norm, factor = lu.clip(enc, [grads[k] for k in names], 0.5 * total).tolist()
    assert abs(norm - total) <= 2.0 ** -18 * total and abs(factor - 0.5) <= 2.0 ** -18
    for k in names:
        want = keep[k].double() * factor
        assert_within(grads[k], want, 2.0 ** (-8 if keep[k].dtype == B else -23) * want.abs())


def test_layer_captured(enc):
    """The same step, captured before any eager one of these sizes and replayed for other texts, gives the eager step's bits."""
    p, T = parameters(2), sum(LENS)
    x, dout = batch(3)
    cu, pos = lu.offsets(LENS), lu.positions(LENS)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):            # (the library that runs the projections wants its first calls outside)
        for w in (p["wqkv"], p["wo"], p["wi"], p["wd"]):
            torch.empty(T, w.shape[1], dtype=B, device="cuda") @ w.t()
            torch.empty(T, w.shape[0], dtype=B, device="cuda") @ w
            torch.empty(T, w.shape[0], dtype=B, device="cuda").t() @ torch.empty(T, w.shape[1], dtype=B, device="cuda")
    torch.cuda.synchronize()
    names = ["ln1", "ln2", "wd", "wi", "wo", "wqkv"]
    ws = {}

    def step():
        # as forward() and backward(), without the tests' host-side checks, which a capture does not allow
        def empty(like, *shape):
            return torch.empty(shape, dtype=like.dtype, device="cuda")

        def space(name, *sizes):
            if (name, sizes) not in ws:
                n = binding.workspace_bytes(name, *sizes)
                ws[name, sizes] = torch.empty(n, dtype=torch.uint8, device="cuda"), n
            return ws[name, sizes]

        st = stream()
        y1, y2 = empty(p["wo"], T, H), empty(p["wo"], T, H)
        st1, st2 = empty(x, T, 2), empty(x, T, 2)
        enc.op("tee_op_layernorm_forward", x, binding.TEE_F32, p["ln1"], y1, binding.TEE_BF16, st1, T, H, 1e-5, st)
        qkv = y1 @ p["wqkv"].t()
        enc.op("tee_op_rope_forward", qkv, binding.TEE_BF16, pos, qkv, T, HEADS, 10000.0, st)
        o, lse = empty(y1, T, H), empty(x, HEADS, T)
        enc.op("tee_op_attention_forward", qkv, cu, o, lse, T, len(LENS), HEADS, -1,
               *space("attention_forward", T, len(LENS), HEADS), st)
        x1 = x + (o @ p["wo"].t()).float()
        enc.op("tee_op_layernorm_forward", x1, binding.TEE_F32, p["ln2"], y2, binding.TEE_BF16, st2, T, H, 1e-5, st)
        z = empty(y1, T, I)
        enc.op("tee_op_geglu_forward", y2, p["wi"], z, T, H, I, st)
        out = x1 + (z @ p["wd"].t()).float()
        d16 = dout.to(B)
        g = {"wd": d16.t() @ z, "wi": empty(p["wi"], 2 * I, H), "ln1": empty(x, H), "ln2": empty(x, H)}
        dy2, dx1, dx = empty(y1, T, H), empty(x, T, H), empty(x, T, H)
        enc.op("tee_op_geglu_backward", y2, p["wi"], d16 @ p["wd"], dy2, g["wi"], T, H, I, *space("geglu_backward", T, H, I), st)
        enc.op("tee_op_layernorm_backward", dy2, binding.TEE_BF16, x1, binding.TEE_F32, p["ln2"], st2, dout, dx1, g["ln2"],
               T, H, *space("layernorm_backward", T, H), st)
        d16 = dx1.to(B)
        g["wo"], dqkv = d16.t() @ o, empty(qkv, T, 3 * H)
        enc.op("tee_op_attention_backward", qkv, cu, o, lse, d16 @ p["wo"], dqkv, T, len(LENS), HEADS, -1,
               *space("attention_backward", T, len(LENS), HEADS), st)
        enc.op("tee_op_rope_backward", dqkv, binding.TEE_BF16, pos, dqkv, T, HEADS, 10000.0, st)
        g["wqkv"] = dqkv.t() @ y1
        enc.op("tee_op_layernorm_backward", dqkv @ p["wqkv"], binding.TEE_BF16, x, binding.TEE_F32, p["ln1"], st1, dx1, dx,
               g["ln1"], T, H, *space("layernorm_backward", T, H), st)
        norm = lu.clip(enc, [g[k] for k in names], 1e-3, None, space("clip_gradients", len(names)))
        return [out, dx, norm] + [g[k] for k in names]

    for k, sizes in (("attention_forward", (T, len(LENS), HEADS)), ("attention_backward", (T, len(LENS), HEADS)),
                     ("geglu_backward", (T, H, I)), ("layernorm_backward", (T, H)), ("clip_gradients", (len(names),))):
        n = binding.workspace_bytes(k, *sizes)
        ws[k, sizes] = torch.empty(n, dtype=torch.uint8, device="cuda"), n
    with torch.cuda.graph(graph):
        got = step()
    for seed, lens in ((4, LENS), (5, [300, 64, 37, 8, 150, 0]), (6, [559, 0, 0, 0, 0, 0])):
        nx, nd = batch(seed)
        x.copy_(nx)
        dout.copy_(nd)
        cu.copy_(lu.offsets(lens))
        pos.copy_(lu.positions(lens))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
        assert all(bool(torch.isfinite(t.float()).all()) for t in kept)
    assert enc.device_status() == binding.TEE_OK
