"""The training-side operators of the library (include/tee_train.h) as measurable cases.

A fine-tuning step of the encoder begins with the scaled token-embedding lookup, normalises rows with the bias-free
LayerNorm, and ends, for masked-token prediction, with the softmax cross entropy over the vocabulary, whose weight is
the token table itself.  Each of the three has its forward and its backward pass here.

Sizes: the tiny encoder (hidden 256, vocabulary 4096, 259 tokens), the accuracy batch (1051 tokens), the throughput
batches (2048 and 32768 tokens) and the long documents (65536 tokens) of the 310m shape (hidden 768, vocabulary 102400).
"""
import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}
IGNORE = -100
EPS = 1e-5


def listed():
    return [
        # LayerNorm over the rows of the smallest packed batch, fp32 as the fp32 path keeps it: launch latency
        {"name": "ln_fwd_tiny", "op": "ln_fwd", "T": 259, "H": 256, "x": "f32", "y": "f32"},
        # LayerNorm of eight long documents: fp32 residual stream in, bf16 activations out
        {"name": "ln_fwd_long", "op": "ln_fwd", "T": 65536, "H": 768, "x": "f32", "y": "bf16"},
        # its backward pass on the ragged accuracy batch, joined with the gradient of the residual branch
        {"name": "ln_bwd_ragged", "op": "ln_bwd", "T": 1051, "H": 768, "x": "f32", "y": "bf16", "res": True},
        # its backward pass on a full training batch
        {"name": "ln_bwd_32k", "op": "ln_bwd", "T": 32768, "H": 768, "x": "f32", "y": "bf16", "res": True},
        # token lookup of the smallest batch
        {"name": "embed_fwd_tiny", "op": "embed_fwd", "T": 259, "V": 4096, "H": 256, "e": "f32", "y": "f32", "ids": "zipf"},
        # token lookup of a full training batch into the fp32 residual stream
        {"name": "embed_fwd_32k", "op": "embed_fwd", "T": 32768, "V": 102400, "H": 768, "e": "bf16", "y": "f32", "ids": "mlm"},
        # the table's gradient for a short batch: nearly every id once, most of the table untouched
        {"name": "embed_bwd_2k", "op": "embed_bwd", "T": 2048, "V": 102400, "H": 768, "e": "bf16", "y": "f32", "ids": "uniform"},
        # the table's gradient for masked-token training: one id holds 30 % of the tokens, the rest fall off as 1/rank
        {"name": "embed_bwd_64k", "op": "embed_bwd", "T": 65536, "V": 102400, "H": 768, "e": "f32", "y": "f32", "ids": "mlm"},
        # the loss of the tiny encoder, every position counted
        {"name": "loss_fwd_tiny", "op": "loss_fwd", "T": 259, "V": 4096, "H": 256, "live": 1.0},
        # the loss of a full masked-token batch: 30 % of the positions are counted
        {"name": "loss_fwd_mlm", "op": "loss_fwd", "T": 32768, "V": 102400, "H": 768, "live": 0.3},
        # the loss's gradients for the ragged accuracy batch
        {"name": "loss_bwd_ragged", "op": "loss_bwd", "T": 1051, "V": 102400, "H": 768, "live": 0.3},
        # the loss's gradients for a full masked-token batch
        {"name": "loss_bwd_mlm", "op": "loss_bwd", "T": 32768, "V": 102400, "H": 768, "live": 0.3},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "embed_fwd", "embed_bwd", "loss_fwd", "loss_bwd"])
    T = _log_uniform(rng, 1, 65536)
    if op.startswith("ln"):
        H = _log_uniform(rng, 8, 2048)          # odd widths among them
        T = min(T, 65536 * 768 // H)
        c = {"op": op, "T": T, "H": H, "x": rng.choice(["f32", "f32", "bf16"]), "y": rng.choice(["f32", "bf16", "bf16"])}
        if op == "ln_bwd":
            c["T"] = min(T, 32768 * 768 // H)
            c["res"] = rng.random() < 0.5
        return c
    if op.startswith("embed"):
        return {"op": op, "T": min(T, 32768) if op == "embed_fwd" else T, "V": _log_uniform(rng, 500, 102400),
                "H": _log_uniform(rng, 32, 768), "e": rng.choice(["f32", "bf16"]), "y": rng.choice(["f32", "bf16"]),
                "ids": rng.choice(["uniform", "zipf", "mlm"])}
    live = rng.choice([0.15, 0.2, 0.3, 1.0])
    return {"op": op, "T": min(T, int(9830 / live)), "V": _log_uniform(rng, 500, 102400),
            "H": 8 * _log_uniform(rng, 4, 96), "live": live}


# ---- inputs ------------------------------------------------------------------

def _ids(kind, T, V, g):
    """Token ids: uniform, falling off as 1/rank, or the latter with 30 % of the tokens replaced by one mask id."""
    u = torch.rand(T, generator=g, device="cuda")
    if kind == "uniform":
        return (u * V).long().clamp_(max=V - 1).int()
    ids = (torch.exp(u.double() * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
    if kind == "mlm":
        ids = torch.where(torch.rand(T, generator=g, device="cuda") < 0.3, torch.full_like(ids, min(4, V - 1)), ids)
    return ids.int()


def _live(case):
    """Number of counted positions of a loss case."""
    return max(1, int(round(case["T"] * case["live"])))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, H = case["T"], case["H"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"].startswith("ln"):
        # residual rows: unlike scales from row to row, a mean of their own, and gains near 1
        s["x"] = (normal(T, H) * torch.exp(0.5 * normal(T, 1)) + 0.3 * normal(T, 1)).to(TYPES[case["x"]])
        s["gamma"] = 1 + 0.02 * normal(H)
        if case["op"] == "ln_bwd":
            s["dy"] = normal(T, H).to(TYPES[case["y"]])
            x = s["x"].double()
            var, mean = torch.var_mean(x, dim=1, correction=0)
            s["stats"] = torch.stack([mean, torch.rsqrt(var + EPS)], dim=1).float()
            s["res"] = normal(T, H).to(TYPES[case["x"]]) if case["res"] else None
    elif case["op"].startswith("embed"):
        s["ids"] = _ids(case["ids"], T, case["V"], g)
        s["scale"] = math.sqrt(H)
        if case["op"] == "embed_fwd":
            s["table"] = (0.02 * normal(case["V"], H)).to(TYPES[case["e"]])
        else:
            s["dy"] = normal(T, H).to(TYPES[case["y"]])
    else:
        V, n = case["V"], _live(case)
        s["w"] = (0.02 * normal(V, H)).bfloat16()
        at = torch.randperm(T, generator=g, device="cuda")[:n]
        s["targets"] = torch.full((T,), IGNORE, dtype=torch.int32, device="cuda")
        s["targets"][at] = _ids("zipf", n, V, g)
        # normalised states, drawn towards their target's row by as much as a model in training has learnt
        pull = 12 * torch.rand(T, 1, generator=g, device="cuda") / (0.0004 * H)
        x = normal(T, H) + pull * s["w"][s["targets"].long().clamp(min=0)].float()
        s["x"] = x.bfloat16()
        if case["op"] == "loss_bwd":
            live = s["targets"] >= 0
            s["lse"] = torch.zeros(T, device="cuda")
            s["lse"][live] = torch.logsumexp(s["x"][live].float() @ s["w"].float().t(), dim=1)
            s["gloss"] = torch.full((T,), 1.0 / n, device="cuda")     # the mean over the counted positions
    return s


# ---- the plain forms -----------------------------------------------------------

def _ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(dim=1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + EPS)
    y = d * rstd * s["gamma"]
    return y.to(TYPES[s["case"]["y"]]), torch.cat([mean, rstd], dim=1)


def _ln_bwd(s):
    x, dy, mean, rstd = s["x"].float(), s["dy"].float(), s["stats"][:, :1], s["stats"][:, 1:]
    xhat = (x - mean) * rstd
    gdy = dy * s["gamma"]
    dx = rstd * (gdy - gdy.mean(dim=1, keepdim=True) - xhat * (gdy * xhat).mean(dim=1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return dx.to(s["x"].dtype), (dy * xhat).sum(dim=0)


def _embed_fwd(s):
    return (s["table"][s["ids"].long()].float() * s["scale"]).to(TYPES[s["case"]["y"]])


def _embed_bwd(s):
    c = s["case"]
    grad = torch.zeros(c["V"], c["H"], device="cuda")
    grad.index_add_(0, s["ids"].long(), s["dy"].float())
    return (grad * s["scale"]).to(TYPES[c["e"]])


def _loss_fwd(s):
    live = (s["targets"] >= 0).nonzero().squeeze(1)
    t = s["targets"][live].long()
    logits = s["x"][live].float() @ s["w"].float().t()
    top = logits.max(dim=1, keepdim=True).values
    lse_live = top.squeeze(1) + (logits - top).exp().sum(dim=1).log()
    loss, lse = torch.zeros(2, len(s["targets"]), device="cuda")
    lse[live] = lse_live
    loss[live] = lse_live - logits.gather(1, t[:, None]).squeeze(1)
    return loss, lse


def _loss_bwd(s):
    live = (s["targets"] >= 0).nonzero().squeeze(1)
    t = s["targets"][live].long()
    x, w = s["x"][live].float(), s["w"].float()
    p = (x @ w.t() - s["lse"][live][:, None]).exp()
    p[torch.arange(len(t), device="cuda"), t] -= 1
    p *= s["gloss"][live][:, None]
    dx = torch.zeros(s["x"].shape, dtype=BF16, device="cuda")
    dx[live] = (p @ w).bfloat16()
    return dx, (p.t() @ x).bfloat16()


PLAIN = {"ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd, "embed_fwd": _embed_fwd, "embed_bwd": _embed_bwd,
         "loss_fwd": _loss_fwd, "loss_bwd": _loss_bwd}


# ---- the framework's calls -----------------------------------------------------

_encoder = None


def _context():
    """The library context such a program holds (the operators take its device and its status word)."""
    global _encoder
    if _encoder is None:
        from text_embedding_encoder_gb300 import binding, synth
        _encoder = binding.Encoder(synth.TINY, "bf16", max_tokens=64, max_texts=4)
    return _encoder


def _own(s):
    from text_embedding_encoder_gb300 import binding
    enc, c = _context(), s["case"]
    T, H, st = c["T"], c["H"], torch.cuda.current_stream().cuda_stream
    kinds = {F32: binding.TEE_F32, BF16: binding.TEE_BF16}

    def empty(shape, dtype=F32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def workspace(name, *sizes):
        n = binding.workspace_bytes(name, *sizes)
        return torch.empty(n, dtype=torch.uint8, device="cuda"), n

    if c["op"] == "ln_fwd":
        y, stats = empty((T, H), TYPES[c["y"]]), empty((T, 2))
        enc.op("tee_op_layernorm_forward", s["x"], kinds[s["x"].dtype], s["gamma"], y, kinds[y.dtype], stats, T, H, EPS, st)
        return y, stats
    if c["op"] == "ln_bwd":
        dx, dgamma = empty((T, H), s["x"].dtype), empty(H)
        ws, n = workspace("layernorm_backward", T, H)
        enc.op("tee_op_layernorm_backward", s["dy"], kinds[s["dy"].dtype], s["x"], kinds[s["x"].dtype], s["gamma"],
               s["stats"], s["res"], dx, dgamma, T, H, ws, n, st)
        return dx, dgamma
    V = c["V"]
    if c["op"] == "embed_fwd":
        y = empty((T, H), TYPES[c["y"]])
        enc.op("tee_op_embed_forward", s["table"], kinds[s["table"].dtype], s["ids"], y, kinds[y.dtype], T, V, H,
               s["scale"], st)
        return y
    if c["op"] == "embed_bwd":
        grad = empty((V, H), TYPES[c["e"]])
        ws, n = workspace("embed_backward", T, V, H)
        enc.op("tee_op_embed_backward", s["dy"], kinds[s["dy"].dtype], s["ids"], grad, kinds[grad.dtype], T, V, H,
               s["scale"], 0, ws, n, st)
        return grad
    if c["op"] == "loss_fwd":
        loss, lse = empty(T), empty(T)
        ws, n = workspace("vocab_loss_forward", T, V, H)
        enc.op("tee_op_vocab_loss_forward", s["x"], s["w"], s["targets"], loss, lse, T, V, H, IGNORE, ws, n, st)
        return loss, lse
    dx, dw = empty((T, H), BF16), empty((V, H), BF16)
    ws, n = workspace("vocab_loss_backward", T, V, H)
    enc.op("tee_op_vocab_loss_backward", s["x"], s["w"], s["targets"], s["lse"], s["gloss"], dx, dw, T, V, H, IGNORE,
           ws, n, st)
    return dx, dw


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------

def _size(kind):
    return 2 if kind == "bf16" else 4


def work(case):
    T, H = case["T"], case["H"]
    if case["op"] == "ln_fwd":
        return {"bytes": T * H * (_size(case["x"]) + _size(case["y"])) + 4 * H + 8 * T, "flops": 8 * T * H}
    if case["op"] == "ln_bwd":
        passes = 3 if case["res"] else 2
        return {"bytes": T * H * (passes * _size(case["x"]) + _size(case["y"])) + 8 * H + 8 * T, "flops": 15 * T * H}
    V = case["V"]
    if case["op"] == "embed_fwd":
        return {"bytes": min(T, V) * H * _size(case["e"]) + T * H * _size(case["y"]) + 4 * T, "flops": T * H}
    if case["op"] == "embed_bwd":
        return {"bytes": T * H * _size(case["y"]) + V * H * _size(case["e"]) + 4 * T, "flops": T * H}
    n = _live(case)
    if case["op"] == "loss_fwd":
        return {"bytes": 2 * (n + V) * H + 12 * T, "flops": 2 * n * V * H}
    return {"bytes": 2 * (n + V) * H + 2 * (T + V) * H + 12 * T, "flops": 6 * n * V * H}


# ---- the definitions in 64 bits --------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op == "ln_fwd":
        var, mean = torch.var_mean(c["x"], dim=1, correction=0)
        rstd = (var + EPS).rsqrt()
        return torch.einsum("th,t,h->th", c["x"] - mean[:, None], rstd, c["gamma"]), torch.stack([mean, rstd], dim=1)
    if op == "ln_bwd":
        # through the Jacobian: dx = r (I - 1 1^T / H - xhat xhat^T / H) (gamma dy)
        m, r = c["stats"].unbind(1)
        xhat = torch.einsum("th,t->th", c["x"] - m[:, None], r)
        u = torch.einsum("th,h->th", c["dy"], c["gamma"])
        along = torch.einsum("th,th->t", u, xhat) / case["H"]
        dx = torch.einsum("th,t->th", u - u.sum(1, keepdim=True) / case["H"] - torch.einsum("t,th->th", along, xhat), r)
        if c["res"] is not None:
            dx += c["res"]
        return dx, torch.einsum("th,th->h", c["dy"], xhat)
    if op == "embed_fwd":
        return torch.index_select(c["table"], 0, s["ids"].long()).mul_(c["scale"])
    if op == "embed_bwd":
        order = torch.argsort(s["ids"].long(), stable=True)
        upto = torch.cat([torch.zeros(1, case["H"], dtype=torch.float64, device="cuda"), c["dy"][order].cumsum(0)])
        count = torch.bincount(s["ids"].long(), minlength=case["V"])
        end = count.cumsum(0)
        return (upto[end] - upto[end - count]) * c["scale"]
    rows = [i for i, t in enumerate(s["targets"].tolist()) if t != IGNORE]
    rows = torch.tensor(rows, device="cuda")
    x, t = c["x"][rows], s["targets"].long()[rows]
    if op == "loss_fwd":
        loss, lse = (torch.zeros(case["T"], dtype=torch.float64, device="cuda") for _ in range(2))
        for a in range(0, len(rows), 2048):
            z = x[a:a + 2048] @ c["w"].t()
            lse[rows[a:a + 2048]] = torch.logsumexp(z, dim=1)
            loss[rows[a:a + 2048]] = -torch.log_softmax(z, dim=1).gather(1, t[a:a + 2048, None]).squeeze(1)
        return loss, lse
    dx, dw = torch.zeros_like(c["x"]), torch.zeros_like(c["w"])
    for a in range(0, len(rows), 2048):
        r, tt = rows[a:a + 2048], t[a:a + 2048]
        gl = c["gloss"][r]
        d = torch.exp(x[a:a + 2048] @ c["w"].t() - c["lse"][r][:, None]) * gl[:, None]
        d.scatter_add_(1, tt[:, None], -gl[:, None])
        dx[r] = d @ c["w"]
        dw += d.t() @ x[a:a + 2048]
    return dx, dw
