"""The block's operations at the largest sizes they take in one direction:
rows, columns, reductions."""
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import block_oracle as bo
from tests import test_gpu_layernorm as ln
from tests.block_util import DEV, U32, stream

pytestmark = pytest.mark.gpu

MOST = (1 << 31) - 1


def test_gated_fp32_rows():
    """fp32: 65535 tiles of 128 rows.  Against products in 64 bits."""
    M, F, K = 65535 * 128, 8, 4
    gen = torch.Generator(DEV).manual_seed(1)
    x, w = torch.randn(M, K, generator=gen, device=DEV), torch.randn(2 * F, K, generator=gen, device=DEV)
    h, s = torch.empty(M, F, device=DEV), torch.empty(M, 2 * F, device=DEV)
    nn.mlp_op_gated_linear(nn.F32, nn.ACT_RELU, M, F, K, x.data_ptr(), K, w.data_ptr(), K, None, h.data_ptr(), F,
                           s.data_ptr(), 2 * F, None, 0, None, stream())
    want = x.double() @ w.double().T
    absum = x.double().abs() @ w.double().abs().T
    assert ((s.double() - want).abs() <= 2 * K * U32 * absum).all()
    s64 = s.double()
    want = s64[:, :F].clamp_min(0) * s64[:, F:]
    assert ((h.double() - want).abs() <= U32 * want.abs()).all()
    dy, wd, ds = torch.randn(M, K, generator=gen, device=DEV), torch.randn(K, F, generator=gen, device=DEV), torch.empty_like(s)
    nn.mlp_op_gated_dgrad(nn.F32, nn.ACT_RELU, M, K, F, dy.data_ptr(), K, wd.data_ptr(), F, s.data_ptr(), 2 * F, None, 0,
                          ds.data_ptr(), 2 * F, None, 0, None, stream())
    dh, adh = dy.double() @ wd.double(), dy.double().abs() @ wd.double().abs()
    on = (s64[:, :F] > 0).double()
    for got, f in ((ds[:, :F], s64[:, F:] * on), (ds[:, F:], s64[:, :F] * on)):
        assert ((got.double() - dh * f).abs() <= (2 * K + 4) * U32 * adh * f.abs()).all()


def test_norm_rows():
    """2^31 - 1 rows of one element: every one is its own mean, so y = beta."""
    x = torch.arange(1 << 16, dtype=torch.int32, device=DEV).to(torch.bfloat16).repeat(1 << 15)[:MOST]
    y = torch.zeros_like(x)
    g, b = torch.full((1,), 3.0, device=DEV), torch.full((1,), -1.5, device=DEV)
    nn.mlp_op_layernorm(nn.BF16, MOST, 1, x.data_ptr(), 1, g.data_ptr(), b.data_ptr(), 1e-5, y.data_ptr(), 1, None, None,
                        stream())
    assert (y == -1.5).all()


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
def test_norm_columns(dtype):
    ln.test_forward(dtype, 2, 65535 * 256, 0, 0)
    ln.test_backward(dtype, 2, 65535 * 256, 0, 0)


@pytest.mark.parametrize("rows,cols,off", [(MOST, 1, 0), (1, MOST - 64, 0), (1, MOST - 64, 1)])
def test_checkpoint(rows, cols, off):
    """Powers of two of one block's range read back as they are; a scale per block."""
    n, nb = rows * cols, -(-cols // 32)
    flat = torch.empty(n + off, dtype=torch.bfloat16, device=DEV)
    x = flat[off:]
    x.copy_(torch.tensor([1.0, -2.0, 0.5, 4.0, 0.25, -8.0, 16.0, 1.5], device=DEV).bfloat16().repeat(n // 8 + 1)[:n])
    q, e = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty(rows * nb, dtype=torch.uint8, device=DEV)
    nn.mlp_op_quant8(nn.BF16, rows, cols, x.data_ptr(), cols, q.data_ptr(), cols, e.data_ptr(), nb, stream())
    back = torch.empty(n + off, dtype=torch.bfloat16, device=DEV)
    nn.mlp_op_dequant8(nn.BF16, rows, cols, q.data_ptr(), cols, e.data_ptr(), nb, back[off:].data_ptr(), cols, stream())
    assert torch.equal(back[off:], x)
    _, want = bo.q8_encode(x[:32 * 8].double().cpu().numpy().reshape(-1, min(cols, 32)))
    assert e[:len(want)].cpu().numpy().tolist() == want[:, 0].tolist()


def test_weight_gradient_rows():
    """2^24 rows (several chunks to a split, every split used)."""
    N, K, B = 8, 32, 1 << 24
    gen = torch.Generator(DEV).manual_seed(2)
    dy, x = torch.randn(B, N, generator=gen, device=DEV).bfloat16(), torch.randn(B, K, generator=gen, device=DEV)
    q, e = torch.empty(B, K, dtype=torch.uint8, device=DEV), torch.empty(B, 1, dtype=torch.uint8, device=DEV)
    nn.mlp_op_quant8(nn.F32, B, K, x.data_ptr(), K, q.data_ptr(), K, e.data_ptr(), 1, stream())
    nn.mlp_op_dequant8(nn.F32, B, K, q.data_ptr(), K, e.data_ptr(), 1, x.data_ptr(), K, stream())
    n = nn.mlp_op_wgrad8_workspace_bytes(nn.BF16, N, K, B)
    ws, dw = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty(N, K, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    nn.mlp_op_wgrad8(nn.BF16, N, K, B, dy.data_ptr(), N, q.data_ptr(), K, e.data_ptr(), 1, dw.data_ptr(), K, None,
                     ws.data_ptr(), n, err.data_ptr(), stream())
    want = dy.double().T @ x.double()
    assert err.item() == 0 and ((dw.double() - want).norm() / want.norm()).item() < 1e-6
