"""8-bit activation checkpoints: codes and scales bit for bit against the
oracle, the values read back, and the weight gradient from a checkpoint."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import block_oracle as bo
from tests.block_util import DEV, TDT, U32, Buf, assert_within, stream, sum_err

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 0, 0), (1, 32, 0, 0), (2, 33, 0, 0), (3, 31, 1, 0), (5, 64, 0, 8), (7, 100, 0, 0), (7, 104, 0, 0),
          (4, 96, 3, 1), (65, 1000, 0, 0), (40, 1024, 16, 0), (130, 257, 7, 0), (600, 520, 0, 0)]


def _values(rng, rows, cols, td):
    x = rng.normal(size=(rows, cols)) * np.exp(3 * rng.normal(size=(rows, cols)))
    x *= 10.0 ** rng.integers(-30, 30, size=(rows, 1))
    x[rng.random(size=x.shape) < 0.05] = 0.0
    return torch.from_numpy(x.astype(np.float32)).to(td)


def _encode(dtype, X, Q, E):
    nn.mlp_op_quant8(dtype, X.rows, X.cols, X.ptr, X.ld, Q.ptr, Q.ld, E.ptr, E.ld, stream())


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("rows,cols,pad,off", SHAPES)
def test_codes_and_values(dtype, rows, cols, pad, off):
    td = TDT[dtype]
    rng = np.random.default_rng([1, dtype, rows, cols])
    X = Buf(rows, cols, td, cols + pad, off, _values(rng, rows, cols, td))
    Q = Buf(rows, cols, torch.uint8, cols + pad, off)
    E = Buf(rows, -(-cols // 32), torch.uint8, -(-cols // 32) + pad, off)
    Y = Buf(rows, cols, td, cols + pad, off)
    _encode(dtype, X, Q, E)
    q, e = bo.q8_encode(X.np())
    assert np.array_equal(Q.t.cpu().numpy(), q) and np.array_equal(E.t.cpu().numpy(), e)
    nn.mlp_op_dequant8(dtype, rows, cols, Q.ptr, Q.ld, E.ptr, E.ld, Y.ptr, Y.ld, stream())
    assert np.array_equal(Y.np(), bo.q8_decode(q, e))
    for b in (Q, E, Y):
        b.check_canary()


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("off", [0, 1])
def test_extremes(dtype, off):
    """Zeros of either sign, subnormals, the largest magnitudes, a value on
    the edge of its scale, infinities and NaN; a block of nothing but NaN."""
    td = TDT[dtype]
    x = torch.zeros(9, 64)
    x[1, :4] = torch.tensor([-0.0, 2.0 ** -133, -2.0 ** -130, 2.0 ** -126])
    x[2, 3], x[2, 40] = 2.0 ** 127, -1.875 * 2.0 ** 127
    x[3, :3] = torch.tensor([448.0, 1.0, 2.0 ** -9])
    x[4, :3] = torch.tensor([450.0, 1.0, 2.0 ** -9])
    x[5, 0], x[5, 1], x[5, 2] = float("inf"), -float("inf"), 3.0
    x[6, 5], x[6, 6] = float("nan"), -7.0
    x[7, :32] = float("nan")
    x[8] = torch.linspace(-448, 448, 64)
    X = Buf(9, 64, td, 64, off, x.to(td))
    Q, E, Y = Buf(9, 64, torch.uint8, 64, off), Buf(9, 2, torch.uint8), Buf(9, 64, td, 64, off)
    _encode(dtype, X, Q, E)
    nn.mlp_op_dequant8(dtype, 9, 64, Q.ptr, 64, E.ptr, 2, Y.ptr, 64, stream())
    q, e = bo.q8_encode(X.np())
    nan = np.isnan(bo.q8_decode(q, e))
    assert np.array_equal(E.t.cpu().numpy(), e)
    assert np.array_equal(Q.t.cpu().numpy()[~nan], q[~nan]) and np.all((Q.t.cpu().numpy()[nan] & 127) == 127)
    assert np.array_equal(Y.np(), bo.q8_decode(q, e), equal_nan=True)


def test_every_code_and_scale_reads_back():
    """All 256 codes under scales from the smallest to the largest, in fp32."""
    q = torch.arange(256, dtype=torch.uint8).repeat(255, 1)
    e = torch.arange(255, dtype=torch.uint8)[:, None].repeat(1, 8)
    Q, E = q.to(DEV), e.to(DEV)
    Y = torch.empty(255, 256, device=DEV)
    nn.mlp_op_dequant8(nn.F32, 255, 256, Q.data_ptr(), 256, E.data_ptr(), 8, Y.data_ptr(), 256, stream())
    with np.errstate(over="ignore"):
        want = bo.q8_decode(q.numpy(), e.numpy()).astype(np.float32)
    assert np.array_equal(Y.cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("dtype,N,K,B", [
    (nn.F32, 40, 33, 7), (nn.F32, 100, 128, 300), (nn.BF16, 64, 64, 1), (nn.BF16, 128, 200, 77),
    (nn.BF16, 1000, 264, 515), (nn.BF16, 512, 512, 4096), (nn.BF16, 24, 40, 2000)])
def test_weight_gradient(dtype, N, K, B):
    td = TDT[dtype]
    rng = np.random.default_rng([2, dtype, N, K, B])
    dY = Buf(B, N, td, N, 0, torch.from_numpy((rng.normal(size=(B, N)) * 1e-2).astype(np.float32)).to(td))
    q, e = bo.q8_encode(rng.normal(size=(B, K)).astype(np.float32).astype(np.float64))
    Q, E = torch.from_numpy(q).to(DEV), torch.from_numpy(e).to(DEV)
    dW, db = Buf(N, K, torch.float32, (K + 3) // 4 * 4), Buf(1, N, torch.float32)
    n = nn.mlp_op_wgrad8_workspace_bytes(dtype, N, K, B)
    ws = Buf(1, n, torch.uint8)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    nn.mlp_op_wgrad8(dtype, N, K, B, dY.ptr, N, Q.data_ptr(), K, E.data_ptr(), e.shape[1], dW.ptr, dW.ld, db.ptr,
                     ws.ptr, n, err.data_ptr(), stream())
    assert err.item() == 0
    dy, x = dY.np(), bo.q8_decode(q, e)
    absum = np.abs(dy).T @ np.abs(x)
    # the tensor cores' accumulator loses up to 2 steps of fp32 per 16 rows on top (not rounded to nearest)
    extra = 4 * U32 * (B / 16) * absum.max() if dtype == nn.BF16 else 0.0
    assert_within(dW.np(), dy.T @ x, sum_err(absum, B) + extra, "dW")
    assert_within(db.np()[0], dy.sum(axis=0), sum_err(np.abs(dy).sum(axis=0), B), "db")
    for b in (dW, db, ws):
        b.check_canary()
    # the same as mlp_op_wgrad on the values
    X = torch.from_numpy(x.astype(np.float32)).to(td).to(DEV)
    kp = (K + 7) // 8 * 8
    Xp = torch.zeros(B, kp, dtype=td, device=DEV)
    Xp[:, :K] = X
    m = nn.mlp_op_wgrad_workspace_bytes(dtype, N, K, B)
    w2, dW2 = torch.empty(max(m, 1), dtype=torch.uint8, device=DEV), Buf(N, K, torch.float32, dW.ld)
    nn.mlp_op_wgrad(dtype, N, K, B, dY.ptr, N, Xp.data_ptr(), kp, dW2.ptr, dW2.ld, None, w2.data_ptr(), m,
                    err.data_ptr(), stream())
    assert torch.equal(dW.t, dW2.t) or np.abs(dW.np() - dW2.np()).max() <= (sum_err(absum, B) + extra).max()


def test_captured():
    """Encode, decode and the weight gradient in one graph, replayed on new inputs."""
    B, N, K = 500, 128, 264
    rng = np.random.default_rng(5)
    x = torch.empty(B, K, dtype=torch.bfloat16, device=DEV)
    dy = torch.empty(B, N, dtype=torch.bfloat16, device=DEV)
    q, e = torch.empty(B, K, dtype=torch.uint8, device=DEV), torch.empty(B, 9, dtype=torch.uint8, device=DEV)
    y, dw = torch.empty_like(x), torch.empty(N, K, device=DEV)
    n = nn.mlp_op_wgrad8_workspace_bytes(nn.BF16, N, K, B)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def call():
        nn.mlp_op_quant8(nn.BF16, B, K, x.data_ptr(), K, q.data_ptr(), K, e.data_ptr(), 9, stream())
        nn.mlp_op_dequant8(nn.BF16, B, K, q.data_ptr(), K, e.data_ptr(), 9, y.data_ptr(), K, stream())
        nn.mlp_op_wgrad8(nn.BF16, N, K, B, dy.data_ptr(), N, q.data_ptr(), K, e.data_ptr(), 9, dw.data_ptr(), K, None,
                         ws.data_ptr(), n, None, stream())

    def fill():
        x.copy_(_values(rng, B, K, torch.bfloat16))
        dy.copy_(torch.from_numpy(rng.normal(size=(B, N)).astype(np.float32)).bfloat16())

    fill()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    fill()
    graph.replay()
    got = [t.clone() for t in (q, e, y, dw)]
    call()
    assert all(torch.equal(a, b) for a, b in zip(got, (q, e, y, dw)))


@pytest.mark.parametrize("N,K,B", [(5120, 1024, 4200), (2048, 4096, 2049), (256, 256, 6000), (1288, 520, 4096)])
def test_weight_gradient_of_many_units(N, K, B):
    """Several work units to a CTA pair, reductions of several chunks with a
    ragged last one, units with and without a part of the bias gradient:
    against the product in 64 bits, closer than one chain of MMAs would be."""
    g = torch.Generator(device=DEV)
    g.manual_seed(N + K + B)
    dY = (torch.randn((B, N), generator=g, device=DEV) * 1e-2).bfloat16()
    X = torch.randn((B, K), generator=g, device=DEV)
    Q, E = torch.empty(B, K, dtype=torch.uint8, device=DEV), torch.empty(B, -(-K // 32), dtype=torch.uint8, device=DEV)
    nn.mlp_op_quant8(nn.F32, B, K, X.data_ptr(), K, Q.data_ptr(), K, E.data_ptr(), E.shape[1], stream())
    nn.mlp_op_dequant8(nn.F32, B, K, Q.data_ptr(), K, E.data_ptr(), E.shape[1], X.data_ptr(), K, stream())
    dW, db = Buf(N, K, torch.float32), Buf(1, N, torch.float32)
    n = nn.mlp_op_wgrad8_workspace_bytes(nn.BF16, N, K, B)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for d in (db.ptr, None):
        dW.t.fill_(float("nan"))
        nn.mlp_op_wgrad8(nn.BF16, N, K, B, dY.data_ptr(), N, Q.data_ptr(), K, E.data_ptr(), E.shape[1], dW.ptr, K, d,
                         ws.data_ptr(), n, err.data_ptr(), stream())
        assert err.item() == 0
        want = dY.double().T @ X.double()
        off = (dW.t.double() - want).norm() / want.norm()
        # 1e-6: a chain of 2048 rows of 4-bit significands measured at 6e-7; one of 8192 is at 3e-6
        assert off < 1e-6, off.item()
    absum = dY.double().abs().sum(0).cpu().numpy()
    assert_within(db.np()[0], dY.double().sum(0).cpu().numpy(), sum_err(absum, B), "db")
    dW.check_canary()
    db.check_canary()
