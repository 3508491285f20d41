"""Refusals of the block's operations for addresses that only a rare path
would use (no GPU needed)."""
import pytest

import neural_net_step_gb300 as nn
from tests.test_block_cpu import GB, GF, W8, P, _refused, lib  # noqa: F401


@pytest.mark.parametrize("f,good", [(nn.mlp_op_gated_linear, GF), (nn.mlp_op_gated_dgrad, GB), (nn.mlp_op_wgrad8, W8)])
@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_error_word_between_words(f, good, dtype, off):
    """err_dev is written by an atomic where a wait gives up: a word's address or none."""
    _refused(f, dict(good, dtype=dtype), err=P + off)


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("M,D", [(4, 65535 * 256 + 1), (4, 1 << 62), (1 << 62, 1 << 61), (1 << 31, 64), (0, 64), (4, -1)])
def test_no_workspace_size_for_refused_norms(dtype, M, D):
    """0 for shapes that the call refuses, not a product that wrapped around."""
    assert nn.mlp_op_layernorm_backward_workspace_bytes(dtype, M, D) == 0


def test_workspace_size_of_the_largest_norms():
    most = (1 << 31) - 1
    assert nn.mlp_op_layernorm_backward_workspace_bytes(nn.BF16, most, 65535 * 256) == 32 * 2 * 65535 * 256 * 4
    assert nn.mlp_op_layernorm_backward_workspace_bytes(nn.BF16, most, 8192) > 0
