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
