"""What the profiling hook says of the training operators: never more work than they do."""
import math

import pytest

from text_embedding_encoder_gb300 import synth

torch = pytest.importorskip("torch")
from train_util import embed_backward, ln_backward, ln_forward, loss_backward, loss_forward, make_context  # noqa: E402

pytestmark = pytest.mark.gpu

IGNORE = -100
F32, BF16 = torch.float32, torch.bfloat16


def _loss_problem(N, V, H, counted):
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    x = torch.randn(N, H, generator=g, device="cuda").to(BF16)
    w = (torch.randn(V, H, generator=g, device="cuda") / math.sqrt(H)).to(BF16)
    t = torch.full((N,), IGNORE, dtype=torch.int32, device="cuda")
    t[:counted] = 3
    return x, w, t, torch.full((N,), 1.0 / counted, device="cuda")


def _profiled(enc, call):
    enc.profile_enable(True)
    call()
    stats = enc.profile_read()
    enc.profile_enable(False)
    return {k: v for k, v in stats.items() if v["launches"]}


def test_the_loss_claims_no_work_of_ignored_positions(lib):
    enc = make_context()
    N, V, H, n = 4000, 3000, 256, 200
    x, w, t, g = _loss_problem(N, V, H, n)
    lse = loss_forward(enc, x, w, t)[1]
    forward = _profiled(enc, lambda: loss_forward(enc, x, w, t))
    assert set(forward) == {"loss"}
    s = forward["loss"]
    assert s["launches"] == 1 and s["total_ms"] > 0
    assert s["flops"] <= 2 * n * V * H and s["bytes"] == 2 * V * H + 12 * N
    for dx, dw in ((True, True), (True, False), (False, True)):
        s = _profiled(enc, lambda: loss_backward(enc, x, w, t, lse, g, want_dx=dx, want_dw=dw))["loss"]
        assert s["flops"] <= (2 + 2 * dx + 2 * dw) * n * V * H
        assert s["bytes"] == 2 * V * H + 12 * N + dx * 2 * N * H + dw * 2 * V * H
    enc.close()


def test_the_projections_rate_is_their_own(lib):
    """A loss between two encodes on one context leaves the projections' launches, flops and bytes as they were."""
    from text_embedding_encoder_gb300 import binding
    enc = binding.Encoder(synth.TINY, "bf16", max_tokens=512, max_texts=16)
    enc.load_weights(synth.make_weights(synth.TINY, seed=0))
    ids, cu = synth.make_batch(synth.TINY_LENGTHS, synth.TINY.vocab, seed=0)
    x, w, t, _ = _loss_problem(500, 3000, 256, 100)
    alone = _profiled(enc, lambda: (enc.encode(ids, cu), enc.encode(ids, cu)))
    mixed = _profiled(enc, lambda: (enc.encode(ids, cu), loss_forward(enc, x, w, t), enc.encode(ids, cu)))
    for k in ("launches", "flops", "bytes"):
        assert mixed["gemm"][k] == alone["gemm"][k]
    assert set(mixed) - set(alone) == {"loss"}
    enc.close()


def test_bytes_of_the_memory_bound_operators(lib):
    enc = make_context()
    T, H, V = 300, 128, 700
    x, gamma = torch.randn(T, H, device="cuda"), torch.ones(H, device="cuda")
    y, st = ln_forward(enc, x, gamma, BF16)
    s = _profiled(enc, lambda: ln_forward(enc, x, gamma, BF16))["layernorm"]
    assert s["flops"] == 0 and s["bytes"] == T * H * 6
    s = _profiled(enc, lambda: ln_backward(enc, y, x, gamma, st))["layernorm"]
    assert s["flops"] == 0 and s["bytes"] == T * H * 10
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    s = _profiled(enc, lambda: embed_backward(enc, x, ids, V, F32, 1.0))["embed"]
    assert s["flops"] == 0 and s["bytes"] == T * H * 4 + V * H * 4
    enc.close()
