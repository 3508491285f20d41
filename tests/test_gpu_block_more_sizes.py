"""Sizes of the block's operations beyond their first tests: many rows wider
than 8192, fp32 weight gradients over long reductions."""
import pytest

import neural_net_step_gb300 as nn
from tests import test_gpu_ckpt8 as ckpt8
from tests import test_gpu_layernorm as ln

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("M,D,pad,off", [(300, 8200, 0, 0), (500, 12288, 0, 0), (200, 16384, 8, 8), (41, 40001, 1, 1)])
def test_wide_norm_of_many_rows(dtype, M, D, pad, off):
    ln.test_forward(dtype, M, D, pad, off)
    ln.test_backward(dtype, M, D, pad, off)


@pytest.mark.parametrize("N,K,B", [(100, 260, 5000), (520, 300, 2049), (33, 64, 20001), (1000, 784, 1003)])
def test_fp32_weight_gradient_of_many_rows(N, K, B):
    ckpt8.test_weight_gradient(nn.F32, N, K, B)
