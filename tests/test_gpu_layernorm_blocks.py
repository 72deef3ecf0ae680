"""LayerNorm backward starts no more blocks than the SMs hold at once: a further block would run by itself behind the
others, and it adds a row of partial sums of the gain's gradient.  A block writes one such row into the workspace, which
shows how many ran."""
import pytest

torch = pytest.importorskip("torch")
from train_util import KIND, ln_forward, make_context, stream, workspace  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("H,resident", [(2049, 2), (3001, 2), (4095, 2), (255, 4), (1001, 4), (1024, 3), (4096, 3), (768, 2),
                                        (1536, 2), (4097, 2)])
def test_blocks_fit_the_gpu_at_once(enc, H, resident, xt, yt):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = 5000
    x, gamma = torch.randn(T, H, device="cuda").to(xt), torch.ones(H, device="cuda")
    y, st = ln_forward(enc, x, gamma, yt)
    dx, dgamma = torch.empty_like(x), torch.empty(H, device="cuda")
    ws, n = workspace("layernorm_backward", T, H)
    enc.op("tee_op_layernorm_backward", y, KIND[yt], x, KIND[xt], gamma, st, None, dx, dgamma, T, H, ws, n, stream())
    rows = n // (4 * H)
    written = (ws[:rows * 4 * H].view(torch.int32).view(rows, H) != -1).any(1)
    assert int(written.sum()) <= resident * sms
    assert bool(written[:int(written.sum())].all())
    # and the gain's gradient is the sum over what they wrote
    partial = ws[:rows * 4 * H].view(torch.float32).view(rows, H)[written].double()
    assert torch.allclose(dgamma.double(), partial.sum(0), rtol=0, atol=float(partial.abs().sum(0).max()) * rows * 2.0 ** -24)
