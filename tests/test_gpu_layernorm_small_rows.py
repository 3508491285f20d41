"""Backward of layer norm over rows so small that rstd^2 passes fp32's range
(rstd itself does not): dx = rstd (w - mean(w) - xh mean(w xh)) is finite."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import block_oracle as bo
from tests.block_util import DEV, HALF, TDT, U32, Buf, assert_within, stream, sum_err

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("M,D", [(5, 64), (300, 1000), (40, 1001), (40, 1026), (9, 2048), (400, 5520), (5, 8192), (3, 9000)])
def test_rstd_squared_out_of_range(dtype, M, D):
    td = TDT[dtype]
    rng = np.random.default_rng([12, dtype, D])
    X = Buf(M, D, td, values=torch.from_numpy((rng.normal(size=(M, D)) * 2.0 ** -68).astype(np.float32)).to(td))
    dY = Buf(M, D, td, values=torch.from_numpy(rng.normal(size=(M, D)).astype(np.float32)).to(td))
    gamma = rng.normal(size=D).astype(np.float32)
    x, dy = X.np(), dY.np()
    _, mu, r = bo.layer_norm(x, eps=0.0)
    mu, r = mu.astype(np.float32), r.astype(np.float32)
    G, mean, rstd = (torch.from_numpy(a).to(DEV) for a in (gamma, mu, r))
    dX, dg, db = Buf(M, D, td), Buf(1, D, torch.float32), Buf(1, D, torch.float32)
    n = nn.mlp_op_layernorm_backward_workspace_bytes(dtype, M, D)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    nn.mlp_op_layernorm_backward(dtype, M, D, dY.ptr, D, X.ptr, D, G.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                 dX.ptr, D, dg.ptr, db.ptr, ws.data_ptr(), n, stream())
    mu, r, g = mu.astype(np.float64), r.astype(np.float64), gamma.astype(np.float64)
    want, wg, wb = bo.layer_norm_vjp(dy, x, mu, r, g)
    assert (r ** 2 > 3.5e38).all() and np.abs(want).max() < 1e30
    xh, w = (x - mu[:, None]) * r[:, None], dy * g
    c1, c2 = np.abs(w).mean(axis=1, keepdims=True), np.abs(w * xh).mean(axis=1, keepdims=True)
    t1, t2 = sum_err(c1, D) + 2 * U32 * c1, sum_err(c2, D) + 5 * U32 * c2
    t = r[:, None] * (t1 + np.abs(xh) * t2 + 2 * U32 * np.abs(xh) * c2 + 6 * U32 * (np.abs(w) + c1 + np.abs(xh) * c2))
    assert_within(dX.np(), want, t + HALF[dtype] * (np.abs(want) + t), "dx")
    absum = np.abs(dy * xh).sum(axis=0)
    assert_within(dg.np()[0], wg, sum_err(absum, M) + 4 * U32 * absum, "dgamma")
    assert_within(db.np()[0], wb, sum_err(np.abs(dy).sum(axis=0), M), "dbeta")
    dX.check_canary()
