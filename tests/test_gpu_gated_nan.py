"""A gate that is NaN makes its results NaN, whatever the activation: nothing
of a broken weight or row is hidden behind ReLU's maximum."""
import pytest
import torch

import neural_net_step_gb300 as nn
from tests.block_util import DEV, TDT, stream
from tests.test_gpu_gated import ACTS, NONE, RELU

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,M", [(nn.F32, 3), (nn.F32, 200), (nn.BF16, 1), (nn.BF16, 20), (nn.BF16, 300)])
@pytest.mark.parametrize("act", ACTS)
def test_nan_gate(dtype, M, act):
    td, F, K = TDT[dtype], 72, 64
    gen = torch.Generator(DEV).manual_seed(M)
    x, w = torch.randn(M, K, generator=gen, device=DEV).to(td), torch.randn(2 * F, K, generator=gen, device=DEV).to(td)
    w[9, 4] = float("nan")                     # one gate's weights; its up row is sound
    h, s = torch.empty(M, F, dtype=td, device=DEV), torch.empty(M, 2 * F, dtype=td, device=DEV)
    nn.mlp_op_gated_linear(dtype, act, M, F, K, x.data_ptr(), K, w.data_ptr(), K, None, h.data_ptr(), F, s.data_ptr(),
                           2 * F, None, 0, None, stream())
    others = [f for f in range(F) if f != 9]
    assert torch.isnan(s[:, 9]).all() and torch.isfinite(s[:, others]).all() and torch.isfinite(s[:, F:]).all()
    assert torch.isnan(h[:, 9]).all() and torch.isfinite(h[:, others]).all()
    dy, wd = torch.randn(M, 8, generator=gen, device=DEV).to(td), torch.randn(8, F, generator=gen, device=DEV).to(td)
    ds, h2 = torch.empty_like(s), torch.empty_like(h)
    nn.mlp_op_gated_dgrad(dtype, act, M, 8, F, dy.data_ptr(), 8, wd.data_ptr(), F, s.data_ptr(), 2 * F, None, 0,
                          ds.data_ptr(), 2 * F, h2.data_ptr(), F, None, stream())
    assert torch.isnan(h2[:, 9]).all() and torch.isnan(ds[:, F + 9]).all()
    if act not in (NONE, RELU):                # (none: act' = 1; ReLU: act' = (g > 0) = 0)
        assert torch.isnan(ds[:, 9]).all()
    assert torch.isfinite(ds[:, others]).all() and torch.isfinite(ds[:, [F + f for f in others]]).all()
    assert torch.isfinite(h2[:, others]).all()
