"""Gates far out in both tails of the activations, each result held to its
own size: the derivative of GELU and SiLU is 1 and 0 there, not a product of
a clamped exponential with a power of the gate."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import block_oracle as bo
from tests.block_util import DEV, HALF, TDT, U32, assert_within, stream
from tests.test_gpu_gated import ACTS, GELU, SILU, TINY, _act_err, _gate_exponent

pytestmark = pytest.mark.gpu

FAR = np.array([1e12, 1e13, 1e15, 1.5e19, 1e20, 1e30, 3e38])
GATES = np.concatenate([FAR, -FAR, np.linspace(-200, 200, 161), np.linspace(-12, 12, 241), [0.0, 1e-30, -1e-30]])


def _gates(td, F):
    """[M, F]: every gate in some column, M rows."""
    rows = -(-len(GATES) // F)
    return torch.from_numpy(np.resize(GATES, (rows, F)).astype(np.float32)).to(td)


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [7, 300])
def test_backward_elementwise(dtype, act, M):
    """dh = 1 and u = 1: dS is [act'(g) | act(g)] and h is act(g)."""
    td, F, N = TDT[dtype], 64, 8
    g = _gates(td, F)
    g = g.repeat(-(-M // g.shape[0]), 1)[:M]
    S = torch.cat([g, torch.ones_like(g)], 1).to(DEV)
    dY, Wd = torch.ones(M, N, dtype=td, device=DEV), torch.full((N, F), 0.125, dtype=td, device=DEV)
    dS, H = torch.empty(M, 2 * F, dtype=td, device=DEV), torch.empty(M, F, dtype=td, device=DEV)
    nn.mlp_op_gated_dgrad(dtype, act, M, N, F, dY.data_ptr(), N, Wd.data_ptr(), F, S.data_ptr(), 2 * F, None, 0,
                          dS.data_ptr(), 2 * F, H.data_ptr(), F, None, stream())
    g = g.double().numpy()
    a, da = bo.act(g, act), bo.act_grad(g, act)
    ta = np.abs(a) * _act_err(g, act) + 3 * U32 * np.abs(a)
    td_ = (24 + 8 * _gate_exponent(g, act)) * U32 * (np.abs(da) + np.minimum(np.abs(a), 1.2)) if act in (GELU, SILU) else 0.0
    got = dS.double().cpu().numpy()
    assert_within(got[:, :F], da, td_ + HALF[dtype] * (np.abs(da) + td_) + TINY, "dg")
    assert_within(got[:, F:], a, ta + HALF[dtype] * (np.abs(a) + ta) + TINY, "du")
    assert_within(H.double().cpu().numpy(), a, ta + HALF[dtype] * (np.abs(a) + ta) + TINY, "h")


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 7, 40, 300])
def test_forward_elementwise(dtype, act, M):
    """u = 1: h is act(g), each to its own size; rows that hold NaN or an
    infinity are NaN and reach no other."""
    td, F, K = TDT[dtype], 64, 72
    g = np.resize(np.roll(GATES, M), M).astype(np.float32)
    x = torch.zeros(M, K, dtype=td)
    x[:, 0], x[:, 1] = torch.from_numpy(g).to(td), 1.0
    bad = {m: v for m, v in ((2, float("nan")), (5, float("inf")), (6, -float("inf"))) if m < M}
    for m, v in bad.items():
        x[m, 5] = v
    w = torch.zeros(2 * F, K, dtype=td)
    w[:F, 0], w[F:, 1] = 1.0, 1.0
    x, w = x.to(DEV), w.to(DEV)
    h, s = torch.empty(M, F, dtype=td, device=DEV), torch.empty(M, 2 * F, dtype=td, device=DEV)
    nn.mlp_op_gated_linear(dtype, act, M, F, K, x.data_ptr(), K, w.data_ptr(), K, None, h.data_ptr(), F, s.data_ptr(),
                           2 * F, None, 0, None, stream())
    rows = [m for m in range(M) if m not in bad]
    g = x[rows, 0].double().cpu().numpy()[:, None].repeat(F, 1)
    a = bo.act(g, act)
    t = np.abs(a) * _act_err(g, act) + U32 * np.abs(a)
    assert_within(h[rows].double().cpu().numpy(), a, t + HALF[dtype] * (np.abs(a) + t) + TINY, "h")
    assert torch.isnan(h[list(bad)]).all() and torch.isnan(s[list(bad)]).all()
