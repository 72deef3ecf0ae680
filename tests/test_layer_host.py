"""The host side of a layer's training operators, without a GPU: workspace sizes, and NULL contexts."""
import pytest

from test_abi import built_lib  # noqa: F401
from text_embedding_encoder_gb300 import binding

E = binding.TEE_EINVAL


@pytest.mark.parametrize("name,sizes", [
    *[(f"attention_{way}", s) for way in ("forward", "backward")
      for s in ((-1, 1, 1), ((1 << 24) + 1, 1, 1), (5, -1, 1), (5, (1 << 20) + 1, 1), (5, 1, 0), (5, 1, 513))],
    *[("geglu_backward", s) for s in ((-1, 64, 64), ((1 << 24) + 1, 64, 64), (5, 0, 64), (5, 60, 64), (5, 8200, 64),
                                      (5, 64, 0), (5, 64, 4), (5, 64, 32776))],
    ("clip_gradients", (-1,)), ("clip_gradients", (65537,)),
])
def test_workspace_refusals(built_lib, name, sizes):  # noqa: F811
    assert getattr(built_lib, f"tee_{name}_workspace")(*sizes) == E
    assert name in built_lib.tee_last_error(None).decode()


def test_workspace_sizes(built_lib):  # noqa: F811
    f, b = built_lib.tee_attention_forward_workspace, built_lib.tee_attention_backward_workspace
    assert f(0, 5, 2) == b(0, 5, 2) == f(5, 0, 2) == 0
    # per token its text's ends, and 16 bytes for each item; backward two floats for each token and head
    assert 8 * 32768 < f(32768, 150, 12) < 8 * 32768 + 16 * (32768 // 128 + 160) + 1024
    assert b(32768, 150, 12) == f(32768, 150, 12) + 2 * 4 * 12 * 32768
    assert b(1 << 24, 1, 512) > 1 << 35
    # texts of one token: items span up to 128 of them
    assert f(1 << 20, 1 << 20, 1) < (1 << 20) * (8 + 3 * 4) + 16 * (5 * (1 << 13) + 10) + 4096
    g = built_lib.tee_geglu_backward_workspace
    assert g(0, 64, 64) == 0
    assert g(32768, 768, 3072) >= 2 * 32768 * 2 * 3072
    assert g(1 << 24, 768, 3072) == g(1 << 23, 768, 3072)        # two parts' gradients at most
    assert built_lib.tee_clip_gradients_workspace(0) == built_lib.tee_clip_gradients_workspace(1) > 0


def test_null_context(built_lib):  # noqa: F811
    lib = built_lib
    assert lib.tee_op_rope_forward(None, None, 0, None, None, 0, 1, 1.0, None) == E
    assert lib.tee_op_rope_backward(None, None, 0, None, None, 0, 1, 1.0, None) == E
    assert lib.tee_op_attention_forward(None, None, None, None, None, 0, 0, 1, -1, None, 0, None) == E
    assert lib.tee_op_attention_backward(None, *[None] * 6, 0, 0, 1, -1, None, 0, None) == E
    assert lib.tee_op_geglu_forward(None, None, None, None, 0, 8, 8, None) == E
    assert lib.tee_op_geglu_backward(None, *[None] * 5, 0, 8, 8, None, 0, None) == E
    assert lib.tee_op_clip_gradients(None, None, None, None, None, 0, 1.0, None, None, 0, None) == E
