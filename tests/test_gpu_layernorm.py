"""Layer norm, forward and backward, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import block_oracle as bo
from tests.block_util import DEV, HALF, TDT, U32, Buf, assert_within, stream, sum_err

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-5))


def _rows(rng, M, D, td):
    x = rng.normal(size=(M, D)) * np.exp(rng.normal(size=(M, 1))) + rng.normal(size=(M, 1)) * 3
    return torch.from_numpy(x.astype(np.float32)).to(td)


# dtype, M, D, row pitch beyond D, offset in elements
SHAPES = [(dt, M, D, pad, off) for dt in (nn.F32, nn.BF16) for M, D, pad, off in [
    (1, 1, 0, 0), (3, 2, 0, 0), (9, 7, 1, 1), (8, 8, 0, 0), (5, 31, 0, 0), (64, 64, 8, 8), (33, 250, 0, 0),
    (17, 256, 0, 0), (17, 257, 0, 3), (40, 512, 16, 0), (77, 784, 0, 0), (77, 1000, 0, 1), (1, 1024, 0, 0),
    (700, 1024, 0, 0), (12, 1025, 0, 0), (12, 1032, 0, 0), (30, 2048, 0, 0), (9, 4096, 8, 0), (9, 4100, 0, 0),
    (5, 8192, 0, 0), (5, 8191, 1, 0), (3, 8193, 0, 0), (2, 20000, 0, 8),
    # rows that start between 16-byte units, at whole words for bf16 too
    (21, 30, 2, 2), (21, 256, 2, 0), (41, 258, 0, 2), (41, 770, 2, 2), (1500, 2050, 0, 0), (7, 8190, 2, 2), (6, 8192, 0, 2),
    # several rows to a group of threads, the groups of one block at different counts
    (5003, 784, 0, 0), (1000, 5520, 0, 8), (2600, 1000, 24, 0), (3001, 1001, 0, 0), (3001, 2048, 0, 0), (20001, 96, 0, 0), (6001, 400, 0, 0),
    (7001, 280, 8, 8)]]


def _fwd_tol(x, gamma, y, mean, rstd, D, dtype):
    """Bounds of y, mean and rstd (each step's rounding carried along)."""
    d = x - mean[:, None]
    dm = sum_err(np.abs(x).mean(axis=1), D) + U32 * np.abs(mean)
    var = (d * d).mean(axis=1)
    # a squared difference carries 2 (dm + u |d|) |d|, the sum its own error
    dvar = (2 * (dm[:, None] + U32 * np.abs(d)) * np.abs(d)).mean(axis=1) + dm ** 2 + sum_err(var, D)
    dr = 0.5 * dvar / (var + EPS) * rstd + 6 * U32 * rstd
    dr = np.minimum(dr, rstd) * 1.01
    dxh = (dm[:, None] + U32 * np.abs(d)) * rstd[:, None] + np.abs(d) * dr[:, None] + 2 * U32 * np.abs(d) * rstd[:, None]
    ty = dxh * np.abs(gamma) + 2 * U32 * (np.abs(y) + np.abs(d * rstd[:, None] * gamma))
    return ty + HALF[dtype] * (np.abs(y) + ty), dm, dr + U32 * rstd


@pytest.mark.parametrize("dtype,M,D,pad,off", SHAPES)
def test_forward(dtype, M, D, pad, off):
    rng = np.random.default_rng([1, dtype, M, D])
    td = TDT[dtype]
    X = Buf(M, D, td, D + pad, off, _rows(rng, M, D, td))
    Y = Buf(M, D, td, D + pad, off)
    gamma, beta = rng.normal(size=D).astype(np.float32), rng.normal(size=D).astype(np.float32)
    G, B = torch.from_numpy(gamma).to(DEV), torch.from_numpy(beta).to(DEV)
    mean, rstd = Buf(1, M, torch.float32), Buf(1, M, torch.float32)
    nn.mlp_op_layernorm(dtype, M, D, X.ptr, X.ld, G.data_ptr(), B.data_ptr(), EPS, Y.ptr, Y.ld, mean.ptr, rstd.ptr,
                        stream())
    x = X.np()
    y, mu, r = bo.layer_norm(x, gamma.astype(np.float64), beta.astype(np.float64), EPS)
    ty, tm, tr = _fwd_tol(x, gamma, y, mu, r, D, dtype)
    assert_within(Y.np(), y, ty, "y")
    assert_within(mean.np()[0], mu, tm, "mean")
    assert_within(rstd.np()[0], r, tr, "rstd")
    for b in (Y, mean, rstd):
        b.check_canary()


@pytest.mark.parametrize("dtype,M,D,pad,off", SHAPES)
def test_backward(dtype, M, D, pad, off):
    rng = np.random.default_rng([2, dtype, M, D])
    td = TDT[dtype]
    X = Buf(M, D, td, D + pad, off, _rows(rng, M, D, td))
    dY = Buf(M, D, td, D + pad, off, torch.from_numpy(rng.normal(size=(M, D)).astype(np.float32)).to(td))
    dX = Buf(M, D, td, D + pad, off)
    gamma = rng.normal(size=D).astype(np.float32)
    x, dy = X.np(), dY.np()
    _, mu, r = bo.layer_norm(x, eps=EPS)
    mu, r = mu.astype(np.float32), r.astype(np.float32)
    G, mean, rstd = (torch.from_numpy(a).to(DEV) for a in (gamma, mu, r))
    dg, db = Buf(1, D, torch.float32), Buf(1, D, torch.float32)
    n = nn.mlp_op_layernorm_backward_workspace_bytes(dtype, M, D)
    ws = Buf(1, n // 4, torch.float32)
    nn.mlp_op_layernorm_backward(dtype, M, D, dY.ptr, dY.ld, X.ptr, X.ld, G.data_ptr(), mean.data_ptr(),
                                 rstd.data_ptr(), dX.ptr, dX.ld, dg.ptr, db.ptr, ws.ptr, n, stream())
    mu, r, g = mu.astype(np.float64), r.astype(np.float64), gamma.astype(np.float64)
    want, wg, wb = bo.layer_norm_vjp(dy, x, mu, r, g)
    xh = (x - mu[:, None]) * r[:, None]
    w = dy * g
    dxh = 2 * U32 * np.abs(xh)
    c1, c2 = np.abs(w).mean(axis=1, keepdims=True), np.abs(w * xh).mean(axis=1, keepdims=True)
    t1 = sum_err(c1, D) + 2 * U32 * c1
    t2 = sum_err(c2, D) + 5 * U32 * c2
    t = r[:, None] * (t1 + np.abs(xh) * t2 + dxh * c2 + 6 * U32 * (np.abs(w) + c1 + np.abs(xh) * c2))
    assert_within(dX.np(), want, t + HALF[dtype] * (np.abs(want) + t), "dx")
    assert_within(dg.np()[0], wg, sum_err(np.abs(dy * xh).sum(axis=0), M) + 4 * U32 * np.abs(dy * xh).sum(axis=0), "dgamma")
    assert_within(db.np()[0], wb, sum_err(np.abs(dy).sum(axis=0), M), "dbeta")
    for b in (dX, dg, db, ws):
        b.check_canary()


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("D", [64, 1000, 4096, 9000])
def test_optional_arguments_and_in_place(dtype, D):
    """No scale, no shift, no statistics; Y over X and dX over dY; one of the
    parameter gradients, or none and no workspace."""
    M, td = 13, TDT[dtype]
    rng = np.random.default_rng([3, dtype, D])
    x = _rows(rng, M, D, td).to(DEV)
    ones, zeros = torch.ones(D, device=DEV), torch.zeros(D, device=DEV)
    mean, rstd = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    full = torch.empty_like(x)
    nn.mlp_op_layernorm(dtype, M, D, x.data_ptr(), D, ones.data_ptr(), zeros.data_ptr(), EPS, full.data_ptr(), D,
                        mean.data_ptr(), rstd.data_ptr(), stream())
    y = x.clone()
    nn.mlp_op_layernorm(dtype, M, D, y.data_ptr(), D, None, None, EPS, y.data_ptr(), D, None, None, stream())
    assert torch.equal(y, full)
    dy = torch.from_numpy(rng.normal(size=(M, D)).astype(np.float32)).to(td).to(DEV)
    n = nn.mlp_op_layernorm_backward_workspace_bytes(dtype, M, D)
    ws = torch.empty(n // 4, device=DEV)
    dx, dg, db = torch.empty_like(x), torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    args = (x.data_ptr(), D)
    nn.mlp_op_layernorm_backward(dtype, M, D, dy.data_ptr(), D, *args, ones.data_ptr(), mean.data_ptr(),
                                 rstd.data_ptr(), dx.data_ptr(), D, dg.data_ptr(), db.data_ptr(), ws.data_ptr(), n,
                                 stream())
    dg2, db2, d2, d3 = torch.empty(D, device=DEV), torch.empty(D, device=DEV), dy.clone(), dy.clone()
    nn.mlp_op_layernorm_backward(dtype, M, D, d2.data_ptr(), D, *args, None, mean.data_ptr(), rstd.data_ptr(),
                                 d2.data_ptr(), D, dg2.data_ptr(), None, ws.data_ptr(), n, stream())
    nn.mlp_op_layernorm_backward(dtype, M, D, d3.data_ptr(), D, *args, None, mean.data_ptr(), rstd.data_ptr(),
                                 d3.data_ptr(), D, None, None, None, 0, stream())
    assert torch.equal(d2, dx) and torch.equal(d3, dx) and torch.equal(dg2, dg)
    nn.mlp_op_layernorm_backward(dtype, M, D, dy.data_ptr(), D, *args, None, mean.data_ptr(), rstd.data_ptr(),
                                 dx.data_ptr(), D, None, db2.data_ptr(), ws.data_ptr(), n, stream())
    assert torch.equal(db2, db)


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("D", [96, 1024, 3000, 9001])
def test_constant_rows_and_non_finite_rows(dtype, D):
    """A constant row has y = beta (variance exactly 0); a row holding NaN or
    infinity does not reach its neighbours."""
    td = TDT[dtype]
    x = torch.full((6, D), 2.5, dtype=td, device=DEV)
    x[1, D // 2], x[3, 0] = float("nan"), float("inf")
    beta = torch.linspace(-1, 1, D, device=DEV)
    y = torch.empty_like(x)
    rstd = torch.empty(6, device=DEV)
    nn.mlp_op_layernorm(dtype, 6, D, x.data_ptr(), D, None, beta.data_ptr(), EPS, y.data_ptr(), D, None,
                        rstd.data_ptr(), stream())
    for r in (0, 2, 4, 5):
        assert torch.equal(y[r], beta.to(td))
        assert abs(rstd[r].item() * EPS ** 0.5 - 1) < 4 * U32 * 2
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()


def test_large_offset_keeps_the_variance():
    """Rows far from zero: the variance is of the differences from the mean
    (a difference of squares would leave nothing of it)."""
    M, D = 5, 1024
    rng = np.random.default_rng(4)
    x = torch.from_numpy((rng.integers(-8, 9, size=(M, D)) / 8 + 4096.0).astype(np.float32)).to(DEV)
    y = torch.empty_like(x)
    nn.mlp_op_layernorm(nn.F32, M, D, x.data_ptr(), D, None, None, 0.0, y.data_ptr(), D, None, None, stream())
    want, mu, r = bo.layer_norm(x.double().cpu().numpy(), eps=0.0)
    # the mean's rounding to fp32 (half a step of 4097) would be U32 * 4097 * r; nothing above that is allowed
    assert np.abs(y.double().cpu().numpy() - want).max() < U32 * 4097 * r.max() + 8 * U32 * np.abs(want).max() + 1e-6 * 4


def test_gradients_against_differences():
    """dx, dgamma and dbeta of the fp32 kernels against central differences
    of the fp64 formula."""
    M, D = 4, 40
    rng = np.random.default_rng(6)
    x, dy = rng.normal(size=(M, D)).astype(np.float32), rng.normal(size=(M, D)).astype(np.float32)
    gamma = rng.normal(size=D).astype(np.float32)
    X, dY, G = (torch.from_numpy(a).to(DEV) for a in (x, dy, gamma))
    mean, rstd, Y = torch.empty(M, device=DEV), torch.empty(M, device=DEV), torch.empty_like(X)
    nn.mlp_op_layernorm(nn.F32, M, D, X.data_ptr(), D, G.data_ptr(), None, EPS, Y.data_ptr(), D, mean.data_ptr(),
                        rstd.data_ptr(), stream())
    n = nn.mlp_op_layernorm_backward_workspace_bytes(nn.F32, M, D)
    ws = torch.empty(n // 4, device=DEV)
    dX, dG, dB = torch.empty_like(X), torch.empty_like(G), torch.empty_like(G)
    nn.mlp_op_layernorm_backward(nn.F32, M, D, dY.data_ptr(), D, X.data_ptr(), D, G.data_ptr(), mean.data_ptr(),
                                 rstd.data_ptr(), dX.data_ptr(), D, dG.data_ptr(), dB.data_ptr(), ws.data_ptr(), n,
                                 stream())
    x64, g64 = x.astype(np.float64), gamma.astype(np.float64)
    f = lambda a, b, c: (bo.layer_norm(a, b, c, EPS)[0] * dy).sum()   # noqa: E731
    z, h = np.zeros(D), 1e-6
    for v, grad, at in ((x64, dX, 0), (g64, dG, 1), (z, dB, 2)):
        d = rng.normal(size=v.shape)
        a = [x64, g64, z]
        a[at] = v + h * d
        hi = f(*a)
        a[at] = v - h * d
        diff = (hi - f(*a)) / (2 * h)
        got = (grad.double().cpu().numpy() * d).sum()
        scale = np.abs(grad.double().cpu().numpy() * d).sum()
        assert abs(got - diff) < 64 * U32 * scale + 1e-7


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
def test_captured_and_on_another_stream(dtype):
    """Forward and backward captured in a graph and replayed on new inputs,
    and two streams at once with workspaces of their own: the eager results."""
    M, D, td = 300, 1024, TDT[dtype]
    rng = np.random.default_rng([7, dtype])
    n = nn.mlp_op_layernorm_backward_workspace_bytes(dtype, M, D)

    def state():
        return dict(x=torch.empty(M, D, dtype=td, device=DEV), dy=torch.empty(M, D, dtype=td, device=DEV),
                    y=torch.empty(M, D, dtype=td, device=DEV), dx=torch.empty(M, D, dtype=td, device=DEV),
                    g=torch.rand(D, device=DEV), mean=torch.empty(M, device=DEV), rstd=torch.empty(M, device=DEV),
                    dg=torch.empty(D, device=DEV), db=torch.empty(D, device=DEV), ws=torch.empty(n // 4, device=DEV))

    def call(s):
        p = {k: v.data_ptr() for k, v in s.items()}
        nn.mlp_op_layernorm(dtype, M, D, p["x"], D, p["g"], None, EPS, p["y"], D, p["mean"], p["rstd"], stream())
        nn.mlp_op_layernorm_backward(dtype, M, D, p["dy"], D, p["x"], D, p["g"], p["mean"], p["rstd"], p["dx"], D,
                                     p["dg"], p["db"], p["ws"], n, stream())

    def fill(s):
        s["x"].copy_(_rows(rng, M, D, td))
        s["dy"].copy_(_rows(rng, M, D, td))

    a, b = state(), state()
    fill(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a)
    for _ in range(2):
        fill(a)
        graph.replay()
        got = {k: a[k].clone() for k in ("y", "dx", "dg", "db")}
        call(a)
        assert all(torch.equal(got[k], a[k]) for k in got)
    fill(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            call(a)
        with torch.cuda.stream(s2):
            call(b)
    torch.cuda.synchronize()
    for s in (a, b):
        got = {k: s[k].clone() for k in ("y", "dx", "dg", "db")}
        call(s)
        assert all(torch.equal(got[k], s[k]) for k in got)
