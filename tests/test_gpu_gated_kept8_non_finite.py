"""Pre-activations kept in 8 bits by the gated forward where some are NaN or
infinite: the codes that quantising them gives."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import block_oracle as bo
from tests.block_util import DEV, TDT, Buf, stream
from tests.test_gpu_gated import SILU

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("M,F", [(3, 64), (40, 72), (300, 264)])
def test_codes_of_non_finite_values(dtype, M, F):
    td, K, nb = TDT[dtype], 16, -(-F // 32)
    rng = np.random.default_rng([21, dtype, M])
    # s = x0 w0 + w1 with w1 of few bits: exact, and infinite where |x0 w0| passes fp32's range
    x = torch.zeros(M, K)
    x[:, 1] = 1.0
    x[0::3, 0] = 2.0 ** 127
    x[1, 7] = float("nan")
    x[M - 1, 7] = -float("inf")
    w = torch.zeros(2 * F, K)
    w[:, 1] = torch.from_numpy(rng.integers(-64, 65, size=2 * F) / 16.0)
    w[3::40, 0], w[5::50, 0] = 2.0, -2.0
    X, W = Buf(M, K, td, values=x.to(td)), Buf(2 * F, K, td, values=w.to(td))
    H, S, E = Buf(M, F, td), Buf(M, 2 * F, torch.uint8), Buf(M, 2 * nb, torch.uint8)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    nn.mlp_op_gated_linear(dtype, SILU, M, F, K, X.ptr, K, W.ptr, K, None, H.ptr, F, S.ptr, 2 * F, E.ptr, 2 * nb,
                           err.data_ptr(), stream())
    assert err.item() == 0
    s = X.np()[:, :1] * W.np()[:, 0] + W.np()[:, 1]
    s[s >= 2.0 ** 128], s[s <= -2.0 ** 128] = np.inf, -np.inf
    s[[1, M - 1]] = np.nan                       # 0 * NaN and 0 * inf in every column's sum
    assert np.isinf(s).any()
    for i in range(2):
        q, e = bo.q8_encode(s[:, i * F:(i + 1) * F])
        nan = (q & 127) == 127
        got = S.t.cpu().numpy()[:, i * F:(i + 1) * F]
        assert np.array_equal(E.t.cpu().numpy()[:, i * nb:(i + 1) * nb], e)
        assert np.array_equal(got[~nan], q[~nan]) and np.all((got[nan] & 127) == 127)
    # (a gate of -inf is NaN, as -inf / (1 + e^inf) is: the finite factors' results are finite)
    fin = np.isfinite(s[:, :F]) & np.isfinite(s[:, F:])
    assert np.array_equal(np.isfinite(H.np())[fin], np.ones(fin.sum(), bool))
    for b in (H, S, E):
        b.check_canary()
