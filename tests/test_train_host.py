"""The training operators' host side, without a GPU: workspace sizes, and NULL contexts."""
import pytest

from test_abi import built_lib  # noqa: F401
from text_embedding_encoder_gb300 import binding


def test_workspace_sizes(built_lib):  # noqa: F811
    ln, em = built_lib.tee_layernorm_backward_workspace, built_lib.tee_embed_backward_workspace
    assert ln(0, 768) == 0
    assert ln(1, 768) == 768 * 4 and ln(8, 768) == 768 * 4 and ln(9, 768) == 2 * 768 * 4
    assert ln(1 << 30, 768) == ln(65536, 768) == 640 * 768 * 4        # the grid is bounded
    assert ln(1 << 30, 8192) == 640 * 8192 * 4
    assert em(0, 1, 1) == 0
    # two pair arrays, a state and two fp32 rows for each block of 64 tokens (256 past 16384 tokens), rounded up to
    # 256 bytes each
    assert em(257, 1000, 768) == 2 * 2304 + 256 + 2 * (5 * 768 * 4)
    assert em(16385, 1000, 768) == 2 * 131328 + 768 + 2 * (65 * 768 * 4)
    assert em(1 << 30, 1, 1) > 1 << 33                               # past 32 bits


@pytest.mark.parametrize("H,rows", [(251, 8), (257, 4), (510, 8), (511, 4), (513, 2), (770, 4), (772, 4), (1001, 2), (1025, 1),
                                    (1026, 2), (1536, 4), (1540, 2), (2050, 1), (4096, 1), (8191, 1)])
def test_layernorm_workspace_holds_a_row_for_each_block(built_lib, H, rows):  # noqa: F811
    """`rows` of the tensor to a block, as wide rows take several of its eight warps."""
    for T in (1, rows, rows + 1, 100):
        blocks = -(-T // rows)
        assert built_lib.tee_layernorm_backward_workspace(T, H) == -(-blocks * H * 4 // 256) * 256


@pytest.mark.parametrize("name,sizes", [
    ("layernorm_backward", (-1, 8)), ("layernorm_backward", (1, 0)), ("layernorm_backward", (1, 8193)),
    ("layernorm_backward", ((1 << 30) + 1, 8)), ("embed_backward", (-1, 5, 8)), ("embed_backward", (1, 0, 8)),
    ("embed_backward", (1, 5, 0)), ("embed_backward", (1, 5, 65537)),
])
def test_workspace_refusals(built_lib, name, sizes):  # noqa: F811
    assert getattr(built_lib, f"tee_{name}_workspace")(*sizes) == binding.TEE_EINVAL
    assert name in built_lib.tee_last_error(None).decode()


def test_null_context(built_lib):  # noqa: F811
    E = binding.TEE_EINVAL
    assert built_lib.tee_op_layernorm_forward(None, None, 0, None, None, 0, None, 0, 8, 1e-5, None) == E
    assert built_lib.tee_op_layernorm_backward(None, None, 0, None, 0, None, None, None, None, None, 0, 8, None, 0, None) == E
    assert built_lib.tee_op_embed_forward(None, None, 0, None, None, 0, 0, 1, 8, 1.0, None) == E
    assert built_lib.tee_op_embed_backward(None, None, 0, None, None, 0, 0, 1, 8, 1.0, 0, None, 0, None) == E


def test_vocab_loss_workspace(built_lib):  # noqa: F811
    f, b = built_lib.tee_vocab_loss_forward_workspace, built_lib.tee_vocab_loss_backward_workspace
    assert f(0, 100, 64) == 0 and b(0, 100, 64) == 0
    # far less than the logits, and D in pieces once all of it would be larger than 256 MB
    assert f(32768, 102400, 768) < 4 * 32768 * 102400 / 16
    assert b(32768, 102400, 768) < 2 * 32768 * 102400 / 4
    assert f(1 << 24, 16384, 8) > 1 << 32
    for bad in ((-1, 5, 8), (1 << 25, 5, 8), (5, 0, 8), (5, 1 << 25, 8), (5, 5, 0), (5, 5, 12), (5, 5, 8200)):
        for fn in (f, b):
            assert fn(*bad) == binding.TEE_EINVAL
            assert "vocab_loss" in built_lib.tee_last_error(None).decode()
    E = binding.TEE_EINVAL
    assert built_lib.tee_op_vocab_loss_forward(None, None, None, None, None, None, 1, 1, 8, -100, None, 0, None) == E
    assert built_lib.tee_op_vocab_loss_backward(None, *[None] * 7, 1, 1, 8, -100, None, 0, None) == E
