"""What layer norm keeps of rows that hold NaN or an infinity."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import block_oracle as bo
from tests import test_gpu_layernorm as ln
from tests.block_util import DEV, TDT, assert_within, stream

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("D", [8, 96, 1000, 1001, 1024, 3002, 8192, 9001])
def test_kept_statistics_of_non_finite_rows(dtype, D):
    """A row that holds NaN or an infinity keeps no finite mean and rstd NaN,
    as the definition gives; its neighbours' are theirs."""
    td, M = TDT[dtype], 8
    rng = np.random.default_rng([11, dtype, D])
    x = ln._rows(rng, M, D, td)
    x[1, D // 2], x[3, 0], x[6, D - 1] = float("nan"), float("inf"), -float("inf")
    x = x.to(DEV)
    y, mean, rstd = torch.empty_like(x), torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    nn.mlp_op_layernorm(dtype, M, D, x.data_ptr(), D, None, None, ln.EPS, y.data_ptr(), D, mean.data_ptr(),
                        rstd.data_ptr(), stream())
    bad, good = [1, 3, 6], [0, 2, 4, 5, 7]
    assert torch.isnan(rstd[bad]).all() and not torch.isfinite(mean[bad]).any() and torch.isnan(y[bad]).all()
    x64 = x[good].double().cpu().numpy()
    want, mu, r = bo.layer_norm(x64, eps=ln.EPS)
    ty, tm, tr = ln._fwd_tol(x64, np.ones(D), want, mu, r, D, dtype)
    assert_within(mean[good].double().cpu().numpy(), mu, tm, "mean")
    assert_within(rstd[good].double().cpu().numpy(), r, tr, "rstd")
    assert_within(y[good].double().cpu().numpy(), want, ty, "y")
