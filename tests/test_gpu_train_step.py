"""The training operators together, as a masked-token step over one token table runs them: lookup, LayerNorm, loss,
the gradients back through the loss and the norm, and the table's two gradients added into one."""
import math

import pytest

torch = pytest.importorskip("torch")
from train_util import (KIND, embed_forward, ln_backward, ln_forward, loss_backward, loss_forward, make_context,  # noqa: E402
                        embed_backward, stream, workspace)

pytestmark = pytest.mark.gpu

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
IGNORE = -100


@pytest.fixture(scope="module")
def enc(lib):
    e = make_context()
    yield e
    e.close()


def _problem(T, V, H, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    table = (0.3 * torch.randn(V, H, generator=g, device="cuda")).to(BF16)
    gamma = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
    truth = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    masked = torch.rand(T, generator=g, device="cuda") < 0.3
    masked[0] = True
    ids = torch.where(masked, torch.full_like(truth, 4), truth)       # the mask token
    targets = torch.where(masked, truth, torch.full_like(truth, IGNORE))
    return table, gamma, ids, targets


def _step(enc, table, gamma, ids, targets, scale):
    x = embed_forward(enc, table, ids, F32, scale)
    y, st = ln_forward(enc, x, gamma, BF16)
    loss, lse = loss_forward(enc, y, table, targets)
    n = (targets != IGNORE).sum()
    gloss = torch.ones_like(loss) / n
    dy, dtable = loss_backward(enc, y, table, targets, lse, gloss)
    dx, dgamma = ln_backward(enc, dy, x, gamma, st)
    embed_backward(enc, dx, ids, len(table), BF16, scale, into=dtable)
    return loss.sum() / n, dtable, dgamma, y


def _loss64(table, gamma, ids, targets, scale, eps=1e-5):
    x = table[ids.long()] * scale
    mean = x.mean(1, keepdim=True)
    y = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps) * gamma
    live = targets != IGNORE
    z = torch.log_softmax(y[live] @ table.t(), 1)
    return -z.gather(1, targets[live].long()[:, None]).mean()


@pytest.mark.parametrize("T,V,H", [(37, 50, 64), (259, 4096, 256), (1051, 3001, 768)])
def test_step_against_the_formulas_in_64_bits(enc, T, V, H):
    table, gamma, ids, targets = _problem(T, V, H, seed=T)
    scale = 2.0
    loss, dtable, dgamma, _ = _step(enc, table, gamma, ids, targets, scale)
    t64, g64 = table.double().requires_grad_(), gamma.double().requires_grad_()
    want = _loss64(t64, g64, ids, targets, scale)
    want.backward()
    # in the norm each rounding to bf16 is off by 2^-8 / sqrt 3 of its value: the states y on their way to the logits
    # (an error of a logit is at most |w| |dy|, here below 2^-8 |y| |w| / sqrt 3 = 1/8), D, dy, dtable twice
    rel = 2.0 ** -8 / math.sqrt(3)
    logit = rel * math.sqrt(H) * float(table.double().norm(dim=1).max()) / math.sqrt(H) * 1.2
    assert abs(float(loss) - float(want.detach())) <= 6 * logit
    assert float((dtable.double() - t64.grad).norm()) <= (logit + 5 * rel) * 2 * float(t64.grad.norm())
    assert float((dgamma.double() - g64.grad).norm()) <= (logit + 5 * rel) * 2 * float(g64.grad.norm()) + 1e-6
    assert enc.device_status() == 0


def test_gradient_along_itself_against_differences(enc):
    table, gamma, ids, targets = _problem(200, 500, 128, seed=3)
    _, dtable, _, _ = _step(enc, table, gamma, ids, targets, 2.0)
    u = dtable.double() / dtable.double().norm()
    h = 1e-4
    num = (_loss64(table.double() + h * u, gamma.double(), ids, targets, 2.0)
           - _loss64(table.double() - h * u, gamma.double(), ids, targets, 2.0)) / (2 * h)
    # the slope along the gradient is its norm, up to the gradient's own error (see above)
    assert abs(float(num) - float(dtable.double().norm())) <= 0.03 * float(num)


def test_step_in_a_graph_beside_another(enc):
    """Two captured steps with workspaces of their own, replayed on two streams at once, and an eager one between."""
    made = []
    for seed in (1, 2):
        table, gamma, ids, targets = _problem(500, 900, 128, seed)
        T, V, H = 500, 900, 128
        b = {"table": table, "gamma": gamma, "ids": ids, "t": targets,
             "x": torch.empty(T, H, device="cuda"), "y": torch.empty(T, H, dtype=BF16, device="cuda"),
             "st": torch.empty(T, 2, device="cuda"), "loss": torch.empty(T, device="cuda"), "lse": torch.empty(T, device="cuda"),
             "g": torch.full((T,), 0.01, device="cuda"), "dy": torch.empty(T, H, dtype=BF16, device="cuda"),
             "dt": torch.empty(V, H, dtype=BF16, device="cuda"), "dx": torch.empty(T, H, device="cuda"),
             "dg": torch.empty(H, device="cuda")}
        ws = {n: workspace(n, *a) for n, a in (("vocab_loss_forward", (T, V, H)), ("vocab_loss_backward", (T, V, H)),
                                               ("layernorm_backward", (T, H)), ("embed_backward", (T, V, H)))}

        def step(b=b, ws=ws):
            s, f, h = stream(), KIND[F32], KIND[BF16]
            enc.op("tee_op_embed_forward", b["table"], h, b["ids"], b["x"], f, T, V, H, 2.0, s)
            enc.op("tee_op_layernorm_forward", b["x"], f, b["gamma"], b["y"], h, b["st"], T, H, 1e-5, s)
            enc.op("tee_op_vocab_loss_forward", b["y"], b["table"], b["t"], b["loss"], b["lse"], T, V, H, IGNORE,
                   *ws["vocab_loss_forward"], s)
            enc.op("tee_op_vocab_loss_backward", b["y"], b["table"], b["t"], b["lse"], b["g"], b["dy"], b["dt"], T, V, H,
                   IGNORE, *ws["vocab_loss_backward"], s)
            enc.op("tee_op_layernorm_backward", b["dy"], h, b["x"], f, b["gamma"], b["st"], None, b["dx"], b["dg"], T, H,
                   *ws["layernorm_backward"], s)
            enc.op("tee_op_embed_backward", b["dx"], f, b["ids"], b["dt"], h, T, V, H, 2.0, 1, *ws["embed_backward"], s)
        step()
        torch.cuda.synchronize()
        want = [b[k].clone() for k in ("loss", "dt", "dg")]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        made.append((b, graph, want, torch.cuda.Stream(), ws))   # a graph's buffers live as long as it does
    for b, *_ in made:
        for k in ("loss", "dt", "dg"):
            b[k].fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        for _, graph, _, side, _ in made:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for b, _, want, *_ in made:
        assert all(torch.equal(b[k], a) for k, a in zip(("loss", "dt", "dg"), want))
