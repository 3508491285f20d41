"""Scale byte 255 is NaN: every value of its row and 32 columns, and nothing
else, wherever a checkpoint is read."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import block_oracle as bo
from tests.block_util import DEV, TDT, Buf, stream

pytestmark = pytest.mark.gpu


def _checkpoint(rng, rows, cols, off=0):
    """Codes of moderate values, with three scales replaced by 255."""
    q, e = bo.q8_encode(rng.normal(size=(rows, cols)))
    for r in range(0, rows, 3):
        e[r, r % e.shape[1]] = 255
    Q, E = Buf(rows, cols, torch.uint8, off=off, values=torch.from_numpy(q)), Buf(rows, e.shape[1], torch.uint8, values=torch.from_numpy(e))
    return Q, E, bo.q8_decode(q, e)


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("rows,cols,off", [(7, 256, 0), (9, 100, 1), (5, 31, 0), (300, 1000, 0)])
def test_read_back(dtype, rows, cols, off):
    Q, E, want = _checkpoint(np.random.default_rng([31, dtype, cols]), rows, cols, off)
    Y = Buf(rows, cols, TDT[dtype])
    nn.mlp_op_dequant8(dtype, rows, cols, Q.ptr, Q.ld, E.ptr, E.ld, Y.ptr, Y.ld, stream())
    assert np.isnan(want).any() and np.isfinite(want).any()
    assert np.array_equal(Y.np(), want, equal_nan=True)


def test_every_code():
    Q = torch.arange(256, dtype=torch.uint8, device=DEV)[None].contiguous()
    E = torch.full((1, 8), 255, dtype=torch.uint8, device=DEV)
    Y = torch.zeros(1, 256, device=DEV)
    nn.mlp_op_dequant8(nn.F32, 1, 256, Q.data_ptr(), 256, E.data_ptr(), 8, Y.data_ptr(), 256, stream())
    assert torch.isnan(Y).all()


@pytest.mark.parametrize("dtype,M", [(nn.F32, 9), (nn.BF16, 9), (nn.BF16, 300)])
def test_gated_backward(dtype, M):
    td, F, N = TDT[dtype], 264, 64
    rng = np.random.default_rng([32, dtype, M])
    gq, ge, g = _checkpoint(rng, M, F)
    uq, ue, u = _checkpoint(rng, M, F)
    S, E = torch.cat([gq.t, uq.t], 1), torch.cat([ge.t, ue.t.flip(0)], 1)
    u = bo.q8_decode(uq.t.cpu().numpy(), ue.t.flip(0).cpu().numpy())
    dY, Wd = torch.ones(M, N, dtype=td, device=DEV), torch.ones(N, F, dtype=td, device=DEV)
    dS, H = torch.empty(M, 2 * F, dtype=td, device=DEV), torch.empty(M, F, dtype=td, device=DEV)
    nn.mlp_op_gated_dgrad(dtype, nn.ACT_SILU, M, N, F, dY.data_ptr(), N, Wd.data_ptr(), F, S.data_ptr(), 2 * F,
                          E.data_ptr(), E.shape[1], dS.data_ptr(), 2 * F, H.data_ptr(), F, None, stream())
    ds = dS.isnan().cpu().numpy()
    assert np.array_equal(ds[:, :F], np.isnan(g) | np.isnan(u)) and np.array_equal(ds[:, F:], np.isnan(g))
    assert np.array_equal(H.isnan().cpu().numpy(), np.isnan(g) | np.isnan(u))


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
def test_weight_gradient(dtype):
    B, N, K = 70, 64, 264
    Q, E, x = _checkpoint(np.random.default_rng([33, dtype]), B, K)
    dY, dW = torch.ones(B, N, dtype=TDT[dtype], device=DEV), torch.empty(N, K, device=DEV)
    n = nn.mlp_op_wgrad8_workspace_bytes(dtype, N, K, B)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    E.t[:, 4:] = 127                      # so that some columns hold no NaN
    x = bo.q8_decode(Q.t.cpu().numpy(), E.t.cpu().numpy())
    nn.mlp_op_wgrad8(dtype, N, K, B, dY.data_ptr(), N, Q.ptr, K, E.ptr, E.ld, dW.data_ptr(), K, None, ws.data_ptr(), n,
                     None, stream())
    bad = np.isnan(x).any(axis=0)
    assert bad.any() and not bad.all() and np.array_equal(dW.isnan().cpu().numpy(), np.tile(bad, (N, 1)))
