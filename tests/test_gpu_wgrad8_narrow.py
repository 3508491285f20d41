"""Weight gradients from 8-bit checkpoints with an output side below 256 and
many rows: as close to the product in 64 bits as the wide ones (no chain of
tensor-core products longer than 2048 rows)."""
import pytest
import torch

import neural_net_step_gb300 as nn
from tests.block_util import DEV, Buf, assert_within, stream, sum_err

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,B", [
    (200, 4096, 65536), (4096, 200, 30001), (24, 40, 70001), (128, 128, 131072), (1000, 136, 40000), (8, 2048, 50000),
    (264, 72, 20000), (130, 1032, 9000)])
def test_narrow_weight_gradient(N, K, B):
    g = torch.Generator(device=DEV)
    g.manual_seed(N + K + B)
    dY = Buf(B, N, torch.bfloat16, -(-N // 8) * 8, values=torch.randn((B, N), generator=g, device=DEV) * 1e-2)
    X = torch.randn((B, K), generator=g, device=DEV)
    Q, E = torch.empty(B, K, dtype=torch.uint8, device=DEV), torch.empty(B, -(-K // 32), dtype=torch.uint8, device=DEV)
    nn.mlp_op_quant8(nn.F32, B, K, X.data_ptr(), K, Q.data_ptr(), K, E.data_ptr(), E.shape[1], stream())
    nn.mlp_op_dequant8(nn.F32, B, K, Q.data_ptr(), K, E.data_ptr(), E.shape[1], X.data_ptr(), K, stream())
    dW, db = Buf(N, K, torch.float32), Buf(1, N, torch.float32)
    n = nn.mlp_op_wgrad8_workspace_bytes(nn.BF16, N, K, B)
    ws = Buf(1, n, torch.uint8)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = dY.t.double().T @ X.double()
    absum = dY.t.double().abs().sum(0).cpu().numpy()
    for d in (db.ptr, None):
        dW.t.fill_(float("nan"))
        nn.mlp_op_wgrad8(nn.BF16, N, K, B, dY.ptr, dY.ld, Q.data_ptr(), K, E.data_ptr(), E.shape[1], dW.ptr, K, d,
                         ws.ptr, n, err.data_ptr(), stream())
        assert err.item() == 0
        # the bound of the wide shapes: a chain of 2048 rows of 4-bit significands is 6e-7 off, one of 8192 3.6e-6
        off = ((dW.t.double() - want).norm() / want.norm()).item()
        assert off < 1e-6, off
    assert_within(db.np()[0], dY.t.double().sum(0).cpu().numpy(), sum_err(absum, B), "db")
    for b in (dW, db, ws):
        b.check_canary()
