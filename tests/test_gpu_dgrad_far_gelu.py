"""GELU's derivative in mlp_op_dgrad for pre-activations far out in both
tails: 1 and 0, not a clamped exponential times their cube."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import block_oracle as bo
from tests.block_util import DEV, HALF, TDT, U32, assert_within, stream
from tests.test_gpu_gated import TINY, _gate_exponent
from tests.test_gpu_gated_far_gates import GATES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,M,K", [(nn.F32, 60, 30), (nn.BF16, 60, 24), (nn.BF16, 130, 136), (nn.BF16, 40000, 264),
                                       (nn.BF16, 300, 520)])
def test_far_pre_activations(dtype, M, K):
    """dY W = 1, so that dX is act'(S)."""
    td, N = TDT[dtype], 8
    s = torch.from_numpy(np.resize(GATES, (M, K)).astype(np.float32)).to(td).to(DEV)
    dY, W = torch.ones(M, N, dtype=td, device=DEV), torch.full((N, K), 0.125, dtype=td, device=DEV)
    dX = torch.empty(M, K, dtype=td, device=DEV)
    nn.mlp_op_dgrad(dtype, nn.ACT_GELU_TANH, M, N, K, dY.data_ptr(), N, W.data_ptr(), K, s.data_ptr(), K,
                    dX.data_ptr(), K, None, stream())
    s = s.double().cpu().numpy()
    a, da = bo.act(s, bo.ACT_GELU_TANH), bo.act_grad(s, bo.ACT_GELU_TANH)
    t = (24 + 8 * _gate_exponent(s, bo.ACT_GELU_TANH)) * U32 * (np.abs(da) + np.minimum(np.abs(a), 1.2))
    assert_within(dX.double().cpu().numpy(), da, t + HALF[dtype] * (np.abs(da) + t) + TINY, "dX")


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
def test_nan_stays_nan(dtype):
    td, M, N, K = TDT[dtype], 20, 8, 136
    s = torch.zeros(M, K, dtype=td, device=DEV)
    s[3, 5] = float("nan")
    dY, W = torch.ones(M, N, dtype=td, device=DEV), torch.ones(N, K, dtype=td, device=DEV)
    dX = torch.empty(M, K, dtype=td, device=DEV)
    nn.mlp_op_dgrad(dtype, nn.ACT_GELU_TANH, M, N, K, dY.data_ptr(), N, W.data_ptr(), K, s.data_ptr(), K,
                    dX.data_ptr(), K, None, stream())
    assert torch.isnan(dX[3, 5]) and torch.isfinite(dX).sum().item() == M * K - 1
