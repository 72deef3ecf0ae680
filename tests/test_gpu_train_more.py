"""The training operators where calls meet: a first call inside a capture, one context for encoding and training,
several streams at once, and buffers past 2^31 elements."""
import os
import subprocess
import sys

import numpy as np
import pytest

from text_embedding_encoder_gb300 import synth

torch = pytest.importorskip("torch")
from train_util import (KIND, embed_backward, embed_forward, ln_backward, ln_forward, loss_backward, loss_forward,  # noqa: E402
                        make_context, stream, workspace)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16 = torch.float32, torch.bfloat16

CAPTURE_FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from train_util import *
enc = make_context()
T, V, H = 300, 700, 96
g = torch.Generator(device="cuda"); g.manual_seed(0)
table = torch.randn(V, H, generator=g, device="cuda").bfloat16()
ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
targets = (ids + 1) % V
gamma = torch.ones(H, device="cuda")
x, st, dx = torch.empty(T, H, device="cuda"), torch.empty(T, 2, device="cuda"), torch.empty(T, H, device="cuda")
y, dy, dt = (torch.empty(n, H, device="cuda", dtype=torch.bfloat16) for n in (T, T, V))
loss, lse, gl, dg = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.ones(T, device="cuda"), torch.empty(H, device="cuda")
a, b = workspace("vocab_loss_forward", T, V, H), workspace("vocab_loss_backward", T, V, H)
c, d = workspace("layernorm_backward", T, H), workspace("embed_backward", T, V, H)
def step():
    s = stream()
    enc.op("tee_op_embed_forward", table, 1, ids, x, 0, T, V, H, 1.0, s)
    enc.op("tee_op_layernorm_forward", x, 0, gamma, y, 1, st, T, H, 1e-5, s)
    enc.op("tee_op_vocab_loss_forward", y, table, targets, loss, lse, T, V, H, -100, *a, s)
    enc.op("tee_op_vocab_loss_backward", y, table, targets, lse, gl, dy, dt, T, V, H, -100, *b, s)
    enc.op("tee_op_layernorm_backward", dy, 1, x, 0, gamma, st, None, dx, dg, T, H, *c, s)
    enc.op("tee_op_embed_backward", dx, 0, ids, dt, 1, T, V, H, 1.0, 1, *d, s)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (loss, dt, dg)]
step()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(got, (loss, dt, dg)))
assert bool(torch.isfinite(loss).all()) and float(loss.sum()) > 0
print("captured first")
"""


def test_first_call_inside_a_capture(lib):
    """Nothing has to be called before a capture: kernels are set up without touching the stream."""
    code = CAPTURE_FIRST.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_encoding_and_training_share_a_context(lib):
    from text_embedding_encoder_gb300 import binding
    enc = binding.Encoder(synth.TINY, "bf16", max_tokens=512, max_texts=16)
    enc.load_weights(synth.make_weights(synth.TINY, seed=0))
    ids, cu = synth.make_batch(synth.TINY_LENGTHS, synth.TINY.vocab, seed=0)
    before = enc.encode(ids, cu)
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x, w = torch.randn(500, 256, generator=g, device="cuda").bfloat16(), torch.randn(3000, 256, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, 3000, (500,), generator=g, device="cuda", dtype=torch.int32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss, lse = loss_forward(enc, x, w, t)
    during = enc.encode(ids, cu)
    with torch.cuda.stream(side):
        again, _ = loss_forward(enc, x, w, t)
    torch.cuda.synchronize()
    assert np.array_equal(before, during) and torch.equal(loss, again)
    assert enc.device_status() == 0
    enc.close()


def test_calls_at_once_on_several_streams(lib):
    """Every call has its buffers and its workspace; what runs beside it changes nothing."""
    enc = make_context()
    jobs = []
    for seed in range(4):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        N, V, H = 900 + 100 * seed, 2500, 128
        x, w = torch.randn(N, H, generator=g, device="cuda").bfloat16(), torch.randn(V, H, generator=g, device="cuda").bfloat16()
        t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
        jobs.append((x, w, t, torch.rand(N, generator=g, device="cuda")))

    def run(x, w, t, gl):
        loss, lse = loss_forward(enc, x, w, t)
        dx, dw = loss_backward(enc, x, w, t, lse, gl)
        st = ln_forward(enc, x, torch.ones(x.shape[1], device="cuda"), F32)[1]
        d, dg = ln_backward(enc, dx, x, torch.ones(x.shape[1], device="cuda"), st)
        return loss, dw, dg, embed_backward(enc, d, t, len(w), F32, 1.0)
    want = [run(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for j, s in zip(jobs, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(run(*j))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert enc.device_status() == 0
    enc.close()


def test_buffers_past_two_to_the_31(lib):
    enc = make_context()
    V, H = 2_900_001, 768                                    # 2.2e9 elements
    rows = torch.tensor([0, 1, 1_400_000, 2_796_202, 2_796_203, V - 2, V - 1], device="cuda")
    table = torch.zeros(V, H, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    table[rows] = torch.randn(len(rows), H, generator=g, device="cuda").bfloat16()
    ids = rows.int()
    assert torch.equal(embed_forward(enc, table, ids, BF16, 1.0), table[rows])
    dy = torch.randn(len(rows), H, generator=g, device="cuda")
    grad = embed_backward(enc, dy, ids, V, BF16, 1.0)
    assert torch.equal(grad[rows], dy.bfloat16())
    hit = grad.view(-1).view(torch.int16)
    assert int(torch.count_nonzero(hit)) == int(torch.count_nonzero(dy.bfloat16()))
    # LayerNorm over the table's rows: zero rows give zeros
    y, _ = ln_forward(enc, table, torch.ones(H, device="cuda"), BF16, y=grad)
    want, _ = ln_forward(enc, table[rows].contiguous(), torch.ones(H, device="cuda"), BF16)
    assert torch.equal(y[rows], want) and int(torch.count_nonzero(y.view(-1).view(torch.int16))) == int(torch.count_nonzero(want))
    # the loss against the whole table: the rows at its end take part
    x = (table[rows[4:]].float() / 100).bfloat16()           # target logits near 8, lse near 15
    t = ids[4:].contiguous()
    loss, lse = loss_forward(enc, x, table, t)
    z = x.double() @ table[rows].double().t()
    ref = torch.logsumexp(torch.cat([z, torch.full((3, 1), float(np.log(V - len(rows))), dtype=torch.float64, device="cuda")], 1), 1)
    # zero rows: exp 0 each.  2.9e6 terms in fp32, tile by tile
    assert float((lse.double() - ref).abs().max()) <= 1e-4 * float(ref.abs().max())
    dx, dw = loss_backward(enc, x, table, t, lse, torch.ones(3, device="cuda"))
    d = torch.exp(z - lse.double()[:, None])
    d[torch.arange(3), torch.arange(3) + 4] -= 1
    want_w = d.t() @ x.double()
    assert float((dw[rows].double() - want_w).norm()) <= 2.0 ** -7 * float(want_w.norm())
    want_x = d @ table[rows].double()
    assert float((dx.double() - want_x).norm()) <= 2.0 ** -7 * float(want_x.norm())
    assert enc.device_status() == 0
    enc.close()


def test_layernorm_past_two_to_the_31(lib):
    enc = make_context()
    T, H = 2_900_001, 768
    x = torch.ones(T, H, dtype=BF16, device="cuda")
    rows = torch.tensor([0, 2_796_203, T - 1], device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x[rows] = torch.randn(3, H, generator=g, device="cuda").bfloat16()
    gamma = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
    y, st = ln_forward(enc, x, gamma, BF16)
    want, want_st = ln_forward(enc, x[rows].contiguous(), gamma, BF16)
    assert torch.equal(y[rows], want) and torch.equal(st[rows], want_st)
    assert int(torch.count_nonzero(y.view(-1).view(torch.int16))) == int(torch.count_nonzero(want))   # constant rows give 0
    dx, dgamma = ln_backward(enc, y, x, gamma, st)
    small, small_g = ln_backward(enc, want, x[rows].contiguous(), gamma, want_st)
    assert torch.equal(dx[rows], small) and int(torch.count_nonzero(dx.view(-1).view(torch.int16))) == int(torch.count_nonzero(small))
    assert float((dgamma - small_g).abs().max()) <= 1e-5 * float(small_g.abs().max())
    enc.close()


def test_workspaces_at_any_sixteen_bytes(lib):
    """A workspace needs 16-byte alignment only; 16 bytes off a 256-byte boundary it gives the same bits, and nothing
    is written before or behind it."""
    enc = make_context()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def sizes():
        for N, V, H, T in ((300, 3001, 136, 700), (40, 9000, 64, 5000), (2000, 700, 264, 20000)):
            x, w = torch.randn(N, H, generator=g, device="cuda").bfloat16(), torch.randn(V, H, generator=g, device="cuda").bfloat16()
            t = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
            ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
            ids[: T // 3] = 3
            yield N, V, H, T, x, w, t, ids, torch.randn(T, H, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")

    for N, V, H, T, x, w, t, ids, dy, gl in sizes():
        gamma = torch.ones(H, device="cuda")
        st = ln_forward(enc, dy, gamma, BF16)[1]
        results = []
        for shift in (0, 16):
            kept = []

            def ws(name, *s):
                buf, n = workspace(name, *s, slack=512)
                kept.append((buf, n))
                return buf.data_ptr() + shift, n
            loss, lse = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
            dx, dw, dt = torch.empty_like(x), torch.empty_like(w), torch.empty(V, H, device="cuda")
            dn, dg = torch.empty_like(dy), torch.empty(H, device="cuda")
            s = stream()
            enc.op("tee_op_vocab_loss_forward", x, w, t, loss, lse, N, V, H, -100, *ws("vocab_loss_forward", N, V, H), s)
            enc.op("tee_op_vocab_loss_backward", x, w, t, lse, gl, dx, dw, N, V, H, -100, *ws("vocab_loss_backward", N, V, H), s)
            enc.op("tee_op_embed_backward", dy, KIND[F32], ids, dt, KIND[F32], T, V, H, 1.0, 0, *ws("embed_backward", T, V, H), s)
            enc.op("tee_op_layernorm_backward", dy, KIND[F32], dy, KIND[F32], gamma, st, None, dn, dg, T, H,
                   *ws("layernorm_backward", T, H), s)
            torch.cuda.synchronize()
            for buf, n in kept:
                assert bool((buf[:shift] == 0xFF).all()) and bool((buf[shift + n:] == 0xFF).all())
            results.append((loss, lse, dx, dw, dt, dn, dg))
        assert all(torch.equal(a, b) for a, b in zip(*results))
    assert enc.device_status() == 0
    enc.close()


def test_calls_from_two_threads(lib):
    """Each with its own context, stream and workspace."""
    import threading
    results, errors = {}, []

    def run(k):
        try:
            enc = make_context()
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                g = torch.Generator(device="cuda")
                g.manual_seed(7)
                x, w = torch.randn(700, 128, generator=g, device="cuda").bfloat16(), torch.randn(900, 128, generator=g, device="cuda").bfloat16()
                t = torch.randint(0, 900, (700,), generator=g, device="cuda", dtype=torch.int32)
                for _ in range(20):
                    loss, lse = loss_forward(enc, x, w, t)
                    dx, dw = loss_backward(enc, x, w, t, lse, torch.ones(700, device="cuda"))
                    table = embed_backward(enc, dx, t, 900, BF16, 1.0, into=dw)
            side.synchronize()
            assert enc.device_status() == 0
            results[k] = (loss, table)
            enc.close()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    [th.start() for th in threads]
    [th.join() for th in threads]
    assert not errors, errors
    assert all(torch.equal(a, b) for a, b in zip(results[0], results[1]))
