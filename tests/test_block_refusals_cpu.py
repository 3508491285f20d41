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


@pytest.mark.parametrize("f,good,rows", [
    (nn.mlp_op_wgrad8, dict(W8, dtype=nn.F32, K=1, lddw=1, ldq=1, lde=1, ws_bytes=1 << 40), "N"),
    (nn.mlp_op_wgrad, dict(dtype=nn.F32, N=4, K=1, B=1, dY=P, ldy=4, X=P, ldx=1, dW=P, lddw=1, db=P, ws=P, ws_bytes=1 << 40,
                           err=None, stream=None), "N"),
    (nn.mlp_op_dgrad, dict(dtype=nn.F32, act=0, M=4, N=4, K=4, dY=P, ldy=4, W=P, ldw=4, S=None, lds=0, dX=P, ldx=4,
                           err=None, stream=None), "M")])
def test_more_fp32_rows_than_a_grid_has(f, good, rows):
    """More rows of 64-row tiles than a grid takes: refused before the first of a call's kernels is enqueued."""
    pitch = dict(ldy=1 << 23) if rows == "N" else {}
    _refused(f, dict(good, **pitch), **{rows: 64 * 65535 + 1})


@pytest.mark.parametrize("f,good", [(nn.mlp_op_gated_linear, GF), (nn.mlp_op_gated_dgrad, GB)])
def test_gated_fp32_rows_beyond_the_stated_most(f, good):
    _refused(f, dict(good, dtype=nn.F32), M=65535 * 128 + 1)
