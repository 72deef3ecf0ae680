"""The training operators of an encoder layer's inside (include/tee_train.h) as measurable cases.

Between the LayerNorms and the vocabulary loss of perf/operators.py a fine-tuning step runs, in every layer, rotary
positions on the packed qkv rows, attention confined to each text (the whole text or a window), and the gated
feed-forward projections, each forward and backward; it ends with clipping all gradients by their common norm.

Sizes: the tiny encoder (hidden 256, 4 heads, GeGLU width 512, 259 tokens), the accuracy batch (1051 tokens), the
throughput batch (32768 tokens, text lengths log-uniform in 8 .. 1024) and the long documents (8 of 8192 tokens) of the
310m shape (hidden 768, 12 heads of 64, GeGLU width 3072, 25 layers, vocabulary 102400).
"""
import math
import random

import numpy as np
import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}
HEAD = 64
SCALE = 1 / math.sqrt(HEAD)


def listed():
    return [
        # attention of a window layer over a full training batch, whose texts share tiles
        {"name": "attn_fwd_window_32k", "op": "attn_fwd", "T": 32768, "heads": 12, "window": 64, "lens": "sweep"},
        # its backward pass on the smallest batch: launch latency
        {"name": "attn_bwd_tiny", "op": "attn_bwd", "T": 259, "heads": 4, "window": -1, "lens": "tiny"},
        # its backward pass on a window layer of a full training batch
        {"name": "attn_bwd_window_32k", "op": "attn_bwd", "T": 32768, "heads": 12, "window": 64, "lens": "sweep"},
        # its backward pass on a whole-text layer of eight long documents: the largest work
        {"name": "attn_bwd_long", "op": "attn_bwd", "T": 65536, "heads": 12, "window": -1, "lens": "long"},
        # the feed-forward block's gated half on the smallest batch
        {"name": "geglu_fwd_tiny", "op": "geglu_fwd", "T": 259, "H": 256, "I": 512},
        # the same on a full training batch
        {"name": "geglu_fwd_32k", "op": "geglu_fwd", "T": 32768, "H": 768, "I": 3072},
        # its backward pass on the ragged accuracy batch
        {"name": "geglu_bwd_ragged", "op": "geglu_bwd", "T": 1051, "H": 768, "I": 3072},
        # its backward pass on a full training batch
        {"name": "geglu_bwd_32k", "op": "geglu_bwd", "T": 32768, "H": 768, "I": 3072},
        # rotary positions of the ragged accuracy batch, fp32 rows as an fp32 program keeps them
        {"name": "rope_fwd_ragged", "op": "rope_fwd", "T": 1051, "heads": 12, "lens": "accuracy", "x": "f32", "base": 10000.0},
        # the rotation's gradient for the long documents: far positions, base of the whole-text layers
        {"name": "rope_bwd_long", "op": "rope_bwd", "T": 65536, "heads": 12, "lens": "long", "x": "bf16", "base": 160000.0},
        # clipping of the tiny encoder's gradients, fp32: few small tensors
        {"name": "clip_tiny", "op": "clip", "layers": 3, "V": 4096, "H": 256, "I": 512, "g": "f32", "max": 1.0},
        # clipping of all gradients of the 310m encoder: bf16, the norms' gains in fp32
        {"name": "clip_310m", "op": "clip", "layers": 25, "V": 102400, "H": 768, "I": 3072, "g": "bf16", "max": 1.0},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_bwd", "attn_bwd", "geglu_fwd", "geglu_bwd", "rope_fwd", "rope_bwd", "clip"])
    T = _log_uniform(rng, 1, 65536)
    if op.startswith("attn"):
        lens = rng.choice(["sweep", "sweep", "short", "long", "one"])
        return {"op": op, "T": min(T, 16384) if lens == "one" else T, "heads": rng.randint(1, 12),
                "window": rng.choice([-1, -1, 64, _log_uniform(rng, 1, 256)]), "lens": lens}
    if op.startswith("geglu"):
        H, I = 8 * _log_uniform(rng, 4, 128), 8 * _log_uniform(rng, 8, 384)      # odd multiples of 8 among them
        return {"op": op, "T": min(T, 32768 * 768 * 3072 // (H * I)), "H": H, "I": I}
    if op.startswith("rope"):
        return {"op": op, "T": T, "heads": rng.randint(1, 12), "lens": rng.choice(["sweep", "short", "long", "one"]),
                "x": rng.choice(["f32", "bf16", "bf16"]) if T <= 32768 else "bf16", "base": rng.choice([10000.0, 160000.0])}
    H = _log_uniform(rng, 64, 768)                                               # odd widths
    return {"op": op, "layers": rng.randint(1, 25), "V": _log_uniform(rng, 500, 102400), "H": H, "I": rng.randint(H, 4 * H),
            "g": rng.choice(["f32", "bf16", "bf16"]) if H < 400 else "bf16", "max": rng.choice([0.5, 1.0, 1e6])}


# ---- inputs ------------------------------------------------------------------

def _lengths(case):
    """Text lengths of a packed batch of exactly T tokens."""
    T, kind = case["T"], case["lens"]
    if kind == "tiny":
        return [8, 37, 64, 150]
    if kind == "accuracy":
        return [8, 24, 57, 110, 190, 280, 382]
    lo, hi = {"sweep": (8, 1024), "short": (1, 64), "long": (8192, 8192), "one": (T, T)}[kind]
    rng, lens, left = random.Random(T), [], T
    while left:
        lens.append(min(left, _log_uniform(rng, lo, hi)))
        left -= lens[-1]
    return lens


def _gradient_sizes(case):
    """Elements of an encoder's parameters: the table, and per layer four projections and two gains."""
    H, I = case["H"], case["I"]
    return [case["V"] * H] + case["layers"] * [3 * H * H, H * H, 2 * I * H, H * I], case["layers"] * [H, H]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    op, s = case["op"], {"case": case}
    if op == "clip":
        s["flat"], s["out"], s["at"] = {}, {}, {}
        for kind, sizes in zip((case["g"], "f32"), _gradient_sizes(case)):
            key = kind if kind not in s["flat"] else kind + "_gains"
            starts = np.concatenate([[0], np.cumsum([-(-n // 8) * 8 for n in sizes])])
            flat = torch.zeros(int(starts[-1]), dtype=TYPES[kind], device="cuda")
            for a, n in zip(starts, sizes):       # one scale for each tensor, as layers differ; nothing between them
                flat[int(a):int(a) + n] = (normal(n) * (0.003 * math.exp(0.3 * (n % 7)))).to(flat.dtype)
            s["flat"][key], s["out"][key] = flat, torch.zeros_like(flat)
            s["at"][key] = (starts[:-1].astype(np.int64), np.asarray(sizes, np.int64))
        # the lists that a training program makes once: addresses, where to, types and counts
        parts = [(s["flat"][k], s["out"][k], *s["at"][k]) for k in s["flat"]]
        s["from"] = np.concatenate([f.data_ptr() + a * f.element_size() for f, _, a, _ in parts]).astype(np.uint64)
        s["to"] = np.concatenate([o.data_ptr() + a * o.element_size() for _, o, a, _ in parts]).astype(np.uint64)
        s["types"] = np.concatenate([np.full(len(n), int(f.dtype == BF16), np.int32) for f, _, _, n in parts])
        s["counts"] = np.concatenate([n for _, _, _, n in parts])
        return s
    T = case["T"]
    if op.startswith("geglu"):
        H, I = case["H"], case["I"]
        s["x"] = normal(T, H).bfloat16()          # rows out of a LayerNorm
        s["wi"] = (normal(2 * I, H) * (1.2 / math.sqrt(H))).bfloat16()
        if op == "geglu_bwd":
            s["dz"] = (normal(T, I) * torch.exp(0.5 * normal(T, 1))).bfloat16()
        return s
    H, lens = case["heads"] * HEAD, _lengths(case)
    s["lens"] = lens
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    s["cu"] = torch.from_numpy(cu).cuda()
    s["pos"] = torch.from_numpy(np.concatenate([np.arange(n, dtype=np.int32) for n in lens])).cuda()
    if op.startswith("rope"):
        s["x"] = normal(T, 3 * H).to(TYPES[case["x"]])
        return s
    # scores of standard deviation 2, so that some keys stand out; values with a mean of their own in each column
    s["qkv"] = torch.cat([2 * normal(T, H), normal(T, H), normal(T, H) + 0.5 * normal(1, H)], dim=1).bfloat16()
    if op == "attn_bwd":
        s["o"], s["lse"] = _attn_fwd(s)
        s["do"] = normal(T, H).bfloat16()
    return s


# ---- the plain forms -----------------------------------------------------------

def _blocks(s):
    """The batch as blocks of (query rows [B, M], key rows [B, N], which keys a row sees [B, M, N]); rows that are none
    are T.  Whole-text layers: the texts of like length together, padded to the longest.  Window layers: 128 rows of the
    packed batch and the keys around them."""
    c, T = s["case"], s["case"]["T"]
    w, cu = c["window"], s["cu"].long()
    if w >= 0:
        start = s["cu"].new_zeros(T).long()
        start[cu[:-1]] = 1
        text = start.cumsum(0)
        first = torch.arange(0, T, 128, device="cuda")[:, None]
        rows, keys = first + torch.arange(128, device="cuda"), first - w + torch.arange(128 + 2 * w, device="cuda")
        there = (keys >= 0) & (keys < T)
        near = (rows[:, :, None] - keys[:, None, :]).abs() <= w
        see = near & there[:, None, :] & (text[rows.clamp(max=T - 1)][:, :, None] == text[keys.clamp(0, T - 1)][:, None, :])
        see &= (rows < T)[:, :, None]
        return [(rows.clamp(max=T), torch.where(there, keys, T), see)]
    by_size = {}
    for j, n in enumerate(s["lens"]):
        by_size.setdefault(max(n - 1, 0).bit_length(), []).append(j)
    blocks = []
    for texts in by_size.values():
        longest = max(s["lens"][j] for j in texts)
        j = torch.tensor(texts, device="cuda")
        at = torch.arange(longest, device="cuda")
        there = at < (cu[j + 1] - cu[j])[:, None]
        rows = torch.where(there, cu[j][:, None] + at, T)
        blocks.append((rows, rows, there[:, :, None] & there[:, None, :]))
    return blocks


def _heads(s, rows, keys):
    """Ranges of heads taken at once, as many as keep a block's scores within 2 GB."""
    n, most = s["case"]["heads"], max(1, (1 << 29) // (rows.shape[0] * rows.shape[1] * keys.shape[1]))
    return [range(a, min(a + most, n)) for a in range(0, n, most)]


def _part(s, x, third, hs, at):
    """fp32 [B, heads, rows, 64] of a [T, 3H] or [T, H] tensor, zeros for rows that are none."""
    a = (third * s["case"]["heads"] + hs.start) * HEAD
    x = torch.nn.functional.pad(x[:, a:a + len(hs) * HEAD].float(), (0, 0, 0, 1))
    return x[at].view(*at.shape, len(hs), HEAD).transpose(1, 2)


def _flat(x):
    """[B, heads, rows, 64] as the rows of a [T, H] tensor."""
    return x.transpose(1, 2).flatten(2).flatten(0, 1)


def _attn_fwd(s):
    T, heads = s["case"]["T"], s["case"]["heads"]
    o = torch.zeros(T + 1, heads * HEAD, dtype=BF16, device="cuda")
    lse = torch.zeros(T + 1, heads, device="cuda")
    for rows, keys, see in _blocks(s):
        for hs in _heads(s, rows, keys):
            q, k, v = _part(s, s["qkv"], 0, hs, rows), _part(s, s["qkv"], 1, hs, keys), _part(s, s["qkv"], 2, hs, keys)
            z = (q * SCALE) @ k.transpose(2, 3)
            z.masked_fill_(~see[:, None], -math.inf)
            top = z.max(dim=3, keepdim=True).values.clamp(min=-1e30)
            p = z.sub_(top).exp_()
            total = p.sum(dim=3, keepdim=True)
            o[rows.reshape(-1), hs.start * HEAD:hs.stop * HEAD] = _flat((p @ v) / total).bfloat16()
            lse[rows.reshape(-1), hs.start:hs.stop] = _flat(top + total.log())
    return o[:T].contiguous(), lse[:T].t().contiguous()


def _attn_bwd(s):
    T, heads = s["case"]["T"], s["case"]["heads"]
    grad = torch.zeros(T + 1, 3 * heads * HEAD, device="cuda")
    lse = torch.nn.functional.pad(s["lse"].t(), (0, 0, 0, 1))
    for rows, keys, see in _blocks(s):
        for hs in _heads(s, rows, keys):
            q, k, v = _part(s, s["qkv"], 0, hs, rows), _part(s, s["qkv"], 1, hs, keys), _part(s, s["qkv"], 2, hs, keys)
            o, do = _part(s, s["o"], 0, hs, rows), _part(s, s["do"], 0, hs, rows)
            p = ((q * SCALE) @ k.transpose(2, 3)).sub_(lse[rows, hs.start:hs.stop].transpose(1, 2)[..., None])
            p.masked_fill_(~see[:, None], -math.inf).exp_()
            dz = (do @ v.transpose(2, 3)).sub_((do * o).sum(dim=3, keepdim=True)).mul_(p).mul_(SCALE)
            for third, at, part in ((0, rows, dz @ k), (1, keys, dz.transpose(2, 3) @ q), (2, keys, p.transpose(2, 3) @ do)):
                a = third * heads + hs.start
                grad[:, a * HEAD:(a + len(hs)) * HEAD].index_add_(0, at.reshape(-1), _flat(part))
    return grad[:T].bfloat16()


def _geglu_parts(s):
    I = s["case"]["I"]
    u = s["x"].float() @ s["wi"].float().t()
    a, g = u[:, :I], u[:, I:]
    return a, g, 0.5 * (1 + torch.erf(a * math.sqrt(0.5)))


def _geglu_fwd(s):
    a, g, phi = _geglu_parts(s)
    return (a * phi * g).bfloat16()


def _geglu_bwd(s):
    a, g, phi = _geglu_parts(s)
    dz = s["dz"].float()
    density = torch.exp(-0.5 * a * a) * (1 / math.sqrt(2 * math.pi))
    du = torch.cat([dz * g * (phi + a * density), dz * a * phi], dim=1)
    return (du @ s["wi"].float()).bfloat16(), (du.t() @ s["x"].float()).bfloat16()


def _rope(s, sign):
    c = s["case"]
    heads = c["heads"]
    j = torch.arange(HEAD // 2, dtype=torch.float64, device="cuda")
    angle = s["pos"].double()[:, None] * c["base"] ** (-2 * j / HEAD)
    cos, sin = angle.cos().float()[:, None], sign * angle.sin().float()[:, None]
    x = s["x"].float().view(-1, 3 * heads, HEAD)
    u, v = x[:, :2 * heads, :HEAD // 2], x[:, :2 * heads, HEAD // 2:]
    turned = torch.cat([u * cos - v * sin, v * cos + u * sin], dim=2)
    return torch.cat([turned, x[:, 2 * heads:]], dim=1).view(-1, 3 * heads * HEAD).to(s["x"].dtype)


def _clip(s):
    total = sum(flat.float().square().sum(dtype=torch.float64) for flat in s["flat"].values())
    norm = total.sqrt().float()
    factor = (s["case"]["max"] / norm).clamp(max=1.0)
    return [norm, factor] + [(flat.float() * factor).to(flat.dtype) for flat in s["flat"].values()]


PLAIN = {"attn_fwd": _attn_fwd, "attn_bwd": _attn_bwd, "geglu_fwd": _geglu_fwd, "geglu_bwd": _geglu_bwd,
         "rope_fwd": lambda s: _rope(s, 1), "rope_bwd": lambda s: _rope(s, -1), "clip": _clip}


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
    enc, c, op = _context(), s["case"], s["case"]["op"]
    st = torch.cuda.current_stream().cuda_stream

    def empty(shape, dtype=F32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def workspace(name, *sizes):
        n = binding.workspace_bytes(name, *sizes)
        return torch.empty(n, dtype=torch.uint8, device="cuda"), n

    if op == "clip":
        norm = empty(2)
        ws, n = workspace("clip_gradients", len(s["counts"]))
        enc.op("tee_op_clip_gradients", s["from"], s["types"], s["counts"], s["to"], len(s["counts"]), c["max"], norm, ws, n, st)
        return [norm[0], norm[1]] + list(s["out"].values())
    T = c["T"]
    if op == "geglu_fwd":
        z = empty((T, c["I"]), BF16)
        enc.op("tee_op_geglu_forward", s["x"], s["wi"], z, T, c["H"], c["I"], st)
        return z
    if op == "geglu_bwd":
        dx, dwi = empty((T, c["H"]), BF16), empty((2 * c["I"], c["H"]), BF16)
        ws, n = workspace("geglu_backward", T, c["H"], c["I"])
        enc.op("tee_op_geglu_backward", s["x"], s["wi"], s["dz"], dx, dwi, T, c["H"], c["I"], ws, n, st)
        return dx, dwi
    heads = c["heads"]
    if op.startswith("rope"):
        y = empty((T, 3 * heads * HEAD), s["x"].dtype)
        enc.op("tee_op_rope_forward" if op == "rope_fwd" else "tee_op_rope_backward", s["x"],
               binding.TEE_BF16 if y.dtype == BF16 else binding.TEE_F32, s["pos"], y, T, heads, c["base"], st)
        return y
    texts = len(s["lens"])
    if op == "attn_fwd":
        o, lse = empty((T, heads * HEAD), BF16), empty((heads, T))
        ws, n = workspace("attention_forward", T, texts, heads)
        enc.op("tee_op_attention_forward", s["qkv"], s["cu"], o, lse, T, texts, heads, c["window"], ws, n, st)
        return o, lse
    dqkv = empty((T, 3 * heads * HEAD), BF16)
    ws, n = workspace("attention_backward", T, texts, heads)
    enc.op("tee_op_attention_backward", s["qkv"], s["cu"], s["o"], s["lse"], s["do"], dqkv, T, texts, heads, c["window"],
           ws, n, st)
    return dqkv


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ----------------------------------------------

def _pairs(case):
    """(query, key) pairs that see each other."""
    w = case["window"]
    if w < 0:
        return sum(n * n for n in _lengths(case))
    return sum(n * n if n <= w else n * (2 * w + 1) - w * (w + 1) if n > 2 * w else n + 2 * sum(n - d for d in range(1, w + 1))
               for n in _lengths(case))


def work(case):
    op = case["op"]
    if op == "clip":
        main, gains = (sum(n) for n in _gradient_sizes(case))
        return {"bytes": 2 * main * (2 if case["g"] == "bf16" else 4) + 8 * gains, "flops": 3 * (main + gains)}
    T = case["T"]
    if op.startswith("geglu"):
        H, I = case["H"], case["I"]
        if op == "geglu_fwd":
            return {"bytes": 2 * (T * H + 2 * I * H + T * I), "flops": 4 * T * I * H}
        return {"bytes": 2 * (2 * T * H + 4 * I * H + T * I), "flops": 12 * T * I * H}
    heads = case["heads"]
    H = heads * HEAD
    if op.startswith("rope"):
        return {"bytes": 6 * T * H * (2 if case["x"] == "bf16" else 4) + 4 * T, "flops": 6 * T * H}
    if op == "attn_fwd":
        return {"bytes": 8 * T * H + 4 * T * heads, "flops": 4 * HEAD * heads * _pairs(case)}
    return {"bytes": 16 * T * H + 4 * T * heads, "flops": 10 * HEAD * heads * _pairs(case)}


# ---- the definitions in 64 bits --------------------------------------------------

def _exact_attention(c, s, op):
    """Text by text, all heads at once, every score there is; a window is cut out of the whole matrix."""
    T, heads = c["T"], c["heads"]

    def by_head(x):
        return x.double().view(len(x), -1, heads, HEAD).permute(1, 2, 0, 3)     # [parts, heads, rows, 64]

    outs, stats, grads, a = [], [], [], 0
    for n in s["lens"]:
        q, k, v = by_head(s["qkv"][a:a + n])
        z = torch.einsum("hid,hjd->hij", q, k).div_(8.0)
        if c["window"] >= 0:
            i = torch.arange(n, device="cuda")
            z.masked_fill_((i[:, None] - i).abs() > c["window"], -math.inf)
        if op == "attn_fwd":
            stats.append(torch.logsumexp(z, dim=2))
            outs.append(torch.einsum("hij,hjd->ihd", torch.softmax(z, dim=2), v).reshape(n, -1))
        else:
            p = torch.exp(z.sub_(s["lse"][:, a:a + n].double()[:, :, None]))
            do, o = by_head(s["do"][a:a + n])[0], by_head(s["o"][a:a + n])[0]
            dv = torch.einsum("hij,hid->jhd", p, do)
            ds = p.mul_(torch.einsum("hid,hjd->hij", do, v) - torch.einsum("hid,hid->hi", do, o)[:, :, None]).div_(8.0)
            dq, dk = torch.einsum("hij,hjd->ihd", ds, k), torch.einsum("hij,hid->jhd", ds, q)
            grads.append(torch.cat([dq.reshape(n, -1), dk.reshape(n, -1), dv.reshape(n, -1)], dim=1))
        a += n
    return (torch.cat(outs), torch.cat(stats, dim=1)) if op == "attn_fwd" else torch.cat(grads)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("attn"):
        return _exact_attention(case, s, op)
    if op.startswith("rope"):
        heads = case["heads"]
        j = torch.arange(32, device="cuda").double()
        turn = torch.polar(torch.ones_like(j), s["pos"].double()[:, None] / torch.pow(case["base"], j / 32))
        x = s["x"].double().view(-1, 3 * heads, 2, 32)
        z = torch.complex(x[:, :2 * heads, 0], x[:, :2 * heads, 1])
        z = torch.einsum("thj,tj->thj", z, turn if op == "rope_fwd" else turn.conj())
        return torch.cat([torch.stack([z.real, z.imag], dim=2), x[:, 2 * heads:]], dim=1).reshape(len(x), -1)
    if op == "clip":
        flats = [flat.double() for flat in s["flat"].values()]
        norm = torch.sqrt(sum(torch.dot(f, f) for f in flats))
        factor = torch.minimum(torch.ones_like(norm), case["max"] / norm)
        return [norm, factor] + [f * factor for f in flats]
    x, w = s["x"].double(), s["wi"].double()
    a, g = torch.einsum("th,ih->ti", x, w).chunk(2, dim=1)
    half_erfc = torch.special.erfc(-a / math.sqrt(2.0)) / 2
    if op == "geglu_fwd":
        return torch.einsum("ti,ti,ti->ti", a, half_erfc, g)
    dz = s["dz"].double()
    slope = half_erfc + a * torch.exp(-a.square() / 2) / math.sqrt(2 * math.pi)
    da, dg = dz * g * slope, dz * a * half_erfc
    wa, wg = w.chunk(2)
    dx = torch.einsum("ti,ih->th", da, wa) + torch.einsum("ti,ih->th", dg, wg)
    return dx, torch.cat([torch.einsum("ti,th->ih", da, x), torch.einsum("ti,th->ih", dg, x)])
