"""The gated half of the feed-forward block, forward and backward, against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import layer_util as lu
from text_embedding_encoder_gb300 import binding
from train_util import assert_within, make_context, stream, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def inputs(T, H, I, seed=0, spread=1.2):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    return normal(T, H).bfloat16(), (normal(2 * I, H) * spread / H ** 0.5).bfloat16(), normal(T, I).bfloat16()


def check(enc, T, H, I, seed=0, spread=1.2):
    x, wi, dz = inputs(T, H, I, seed, spread)
    ref = lu.Geglu(x, wi)
    z = lu.geglu_forward(enc, x, wi)
    assert_within(z, *ref.forward())
    dx, dwi = lu.geglu_backward(enc, x, wi, dz)
    want_dx, want_dwi = ref.backward(dz)
    assert_within(dx, *want_dx)
    assert_within(dwi, *want_dwi)
    assert enc.device_status() == binding.TEE_OK


SIZES = [(1, 8, 8), (1, 768, 64), (3, 64, 128), (127, 72, 136), (128, 64, 64), (129, 256, 512), (255, 8, 1000), (256, 256, 256),
         (257, 264, 8), (259, 256, 512), (512, 1000, 120), (513, 520, 392), (1051, 768, 640), (2000, 40, 24), (5000, 136, 72)]


@pytest.mark.parametrize("T,H,I", SIZES)
def test_sizes(enc, T, H, I):
    check(enc, T, H, I, seed=T)


def test_the_310m_block(enc):
    check(enc, 1051, 768, 3072)


def test_many_rows_few_columns(enc):
    """Sums over the rows that are split among the CTA pairs."""
    check(enc, 20000, 64, 64)
    check(enc, 9000, 512, 72)


def test_more_rows_than_one_part(enc):
    check(enc, 65536 + 300, 32, 40)
    check(enc, 131072 + 1, 8, 16)


def test_far_from_zero(enc):
    """Projections of tens, where the activation is the identity or nothing."""
    check(enc, 300, 128, 128, spread=30.0)


def test_one_gradient_alone(enc):
    x, wi, dz = inputs(300, 136, 200)
    dx, dwi = lu.geglu_backward(enc, x, wi, dz)
    assert torch.equal(dx, lu.geglu_backward(enc, x, wi, dz, want_dwi=False)[0])
    assert torch.equal(dwi, lu.geglu_backward(enc, x, wi, dz, want_dx=False)[1])


def test_no_rows(enc):
    _, wi, _ = inputs(1, 64, 64)
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert lu.geglu_forward(enc, empty, wi).numel() == 0
    dx, dwi = lu.geglu_backward(enc, empty, wi, empty)
    assert bool((dwi == 0).all())


def test_rows_of_nan_stay_alone(enc):
    """dx and z of other rows do not see them."""
    x, wi, dz = inputs(700, 64, 72)
    z, dx = lu.geglu_forward(enc, x, wi), lu.geglu_backward(enc, x, wi, dz)[0]
    x[300] = float("nan")
    z2, dx2 = lu.geglu_forward(enc, x, wi), lu.geglu_backward(enc, x, wi, dz)[0]
    keep = torch.arange(700, device="cuda") != 300
    assert torch.equal(z[keep], z2[keep]) and torch.equal(dx[keep], dx2[keep])
    assert torch.isnan(z2[300].float()).all() and torch.isnan(dx2[300].float()).all()


def test_guards(enc):
    """Outputs inside larger buffers: nothing around them is written."""
    T, H, I = 133, 72, 88
    x, wi, dz = inputs(T, H, I)
    big = torch.full((T + 300, I), 7.0, dtype=torch.bfloat16, device="cuda")
    lu.geglu_forward(enc, x, wi, z=big[100:])
    assert bool((big[:100] == 7).all()) and bool((big[100 + T:] == 7).all())
    bx = torch.full((T + 300, H), 7.0, dtype=torch.bfloat16, device="cuda")
    bw = torch.full((2 * I + 400, H), 7.0, dtype=torch.bfloat16, device="cuda")
    ws, n = workspace("geglu_backward", T, H, I, slack=4096)
    enc.op("tee_op_geglu_backward", x, wi, dz, bx[100:], bw[100:], T, H, I, ws, n, stream())
    torch.cuda.synchronize()
    assert bool((bx[:100] == 7).all()) and bool((bx[100 + T:] == 7).all())
    assert bool((bw[:100] == 7).all()) and bool((bw[100 + 2 * I:] == 7).all())
    assert bool((ws[n:] == 0xFF).all())


def test_same_as_the_encoder_s_step(enc):
    """The pass's own step with the same weights."""
    from text_embedding_encoder_gb300 import synth
    e = binding.Encoder(synth.TINY, "bf16", max_tokens=400, max_texts=8)
    w = synth.make_weights(synth.TINY, seed=0)
    e.load_weights(w)
    x = inputs(333, 256, 8)[0]
    wi = torch.from_numpy(np.ascontiguousarray(w.wi[1])).cuda().bfloat16()
    want = torch.empty(333, 512, dtype=torch.bfloat16, device="cuda")
    e.op("tee_op_ffn_in", 1, x, want, 333, stream())
    z = lu.geglu_forward(e, x, wi)
    torch.cuda.synchronize()
    assert torch.equal(z, want)
    e.close()


def test_gradients_against_differences(enc):
    x, wi, dz = inputs(50, 64, 48)
    dx, dwi = lu.geglu_backward(enc, x, wi, dz)
    rng = np.random.default_rng(0)

    def value(x, wi):
        r = lu.Geglu(x, wi)
        return float((r.gelu * r.g * dz.double()).sum())

    for t, grad in ((0, dx), (1, dwi)):
        args = [x.double(), wi.double()]
        way = torch.tensor(rng.standard_normal(args[t].shape), device="cuda")
        up, down = list(args), list(args)
        up[t], down[t] = args[t] + 1e-5 * way, args[t] - 1e-5 * way
        slope = (value(*up) - value(*down)) / 2e-5
        assert abs(float((grad.double() * way).sum()) - slope) < 2.0 ** -6 * float(grad.double().norm()) + 1e-3


def test_refusals(enc):
    x, wi, dz = inputs(64, 64, 64)
    z, dx, dwi = torch.empty_like(dz), torch.empty_like(x), torch.empty_like(wi)
    ws, n = workspace("geglu_backward", 64, 64, 64)
    st = stream()
    good_f, good_b = [x, wi, z, 64, 64, 64, st], [x, wi, dz, dx, dwi, 64, 64, 64, ws, n, st]

    def refused(name, args):
        with pytest.raises(binding.TeeError) as e:
            enc.op(name, *args)
        assert e.value.code == binding.TEE_EINVAL

    for name, good, at in (("tee_op_geglu_forward", good_f, 3), ("tee_op_geglu_backward", good_b, 5)):
        for i, v in [(0, None), (1, None), (2, None), (0, x.data_ptr() + 2), (2, dz.data_ptr() + 8), (at, -1),
                     (at, (1 << 24) + 1), (at + 1, 60), (at + 1, 0), (at + 1, 8200), (at + 2, 4), (at + 2, 32776)]:
            args = list(good)
            args[i] = v
            refused(name, args)
    for i, v in [(3, dx.data_ptr() + 4), (4, dwi.data_ptr() + 4), (8, None), (8, ws.data_ptr() + 8), (9, 16)]:
        args = list(good_b)
        args[i] = v
        refused("tee_op_geglu_backward", args)
    refused("tee_op_geglu_backward", [x, wi, dz, None, None, 64, 64, 64, ws, n, st])


def test_captured_first(enc):
    T, H, I = 700, 128, 200
    x, wi, dz = inputs(T, H, I)
    z, dx, dwi = (torch.full_like(t, float("nan")) for t in (dz, x, wi))
    ws, n = workspace("geglu_backward", T, H, I)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        enc.op("tee_op_geglu_forward", x, wi, z, T, H, I, stream())
        enc.op("tee_op_geglu_backward", x, wi, dz, dx, dwi, T, H, I, ws, n, stream())
    for seed in (1, 2):
        for t, v in zip((x, wi, dz), inputs(T, H, I, seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, lu.geglu_forward(enc, x, wi))
        ex, ew = lu.geglu_backward(enc, x, wi, dz)
        assert torch.equal(dx, ex) and torch.equal(dwi, ew)
