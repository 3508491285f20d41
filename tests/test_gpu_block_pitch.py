"""Rows whose offsets pass 2^31 elements: every matrix of the feed-forward
block's operations with a pitch of 2^26 and more, beside the others of its
element size in one allocation.  The results are those of compact matrices, bit for bit (the pitch
keeps the alignment, so the same kernels run)."""
import pytest
import torch

import neural_net_step_gb300 as nn
from tests.block_util import DEV, TDT, stream

pytestmark = pytest.mark.gpu

PITCH = (1 << 26) + 512          # elements of any type; 39 rows on: 2.6e9


class Field:
    """Matrices of up to 40 rows side by side in one allocation."""

    def __init__(self, es):
        self.raw = torch.empty(40 * PITCH * es, dtype=torch.uint8, device=DEV)
        self.at = 0

    def put(self, t):
        """A copy of t [rows, cols] in the field; its address is of row 0."""
        flat = self.raw.view(t.dtype)
        v = torch.as_strided(flat, t.shape, (PITCH, 1), self.at)
        v.copy_(t)
        self.at += -(-t.shape[1] // 64) * 64
        return v


def _both(make, call, outputs):
    """call(tensors, pitches) on compact matrices and in fields."""
    fields = {es: Field(es) for es in {v.element_size() for v in make.values()}}
    results = []
    for wide in (False, True):
        t = {k: (fields[v.element_size()].put(v) if wide else v.clone()) for k, v in make.items()}
        call(t, {k: v.stride(0) for k, v in t.items()})
        torch.cuda.synchronize()
        results.append({k: t[k].clone() for k in outputs})
    for k in outputs:
        assert torch.equal(results[0][k].view(torch.uint8), results[1][k].view(torch.uint8)), k


def _rand(gen, *shape, td=torch.float32):
    return torch.randn(*shape, generator=gen, device=DEV).to(td)


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
@pytest.mark.parametrize("D", [40, 1000, 8200])
def test_layernorm(dtype, D):
    gen, td, M = torch.Generator(DEV).manual_seed(1), TDT[dtype], 40
    g, b = _rand(gen, D), _rand(gen, D)
    mean, rstd = torch.empty(M, device=DEV), torch.empty(M, device=DEV)
    n = nn.mlp_op_layernorm_backward_workspace_bytes(dtype, M, D)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    dg, db = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    sums = []

    def call(t, ld):
        p = {k: v.data_ptr() for k, v in t.items()}
        nn.mlp_op_layernorm(dtype, M, D, p["x"], ld["x"], g.data_ptr(), b.data_ptr(), 1e-5, p["y"], ld["y"],
                            mean.data_ptr(), rstd.data_ptr(), stream())
        nn.mlp_op_layernorm_backward(dtype, M, D, p["dy"], ld["dy"], p["x"], ld["x"], g.data_ptr(), mean.data_ptr(),
                                     rstd.data_ptr(), p["dx"], ld["dx"], dg.data_ptr(), db.data_ptr(), ws.data_ptr(), n,
                                     stream())
        sums.append(torch.cat([dg, db, mean, rstd]))

    x, dy = _rand(gen, M, D, td=td), _rand(gen, M, D, td=td)
    _both(dict(x=x, dy=dy, y=torch.zeros_like(x), dx=torch.zeros_like(x)), call, ["y", "dx"])
    assert torch.equal(sums[0], sums[1])


@pytest.mark.parametrize("dtype", [nn.F32, nn.BF16])
def test_checkpoints(dtype):
    gen, td, M, K, N = torch.Generator(DEV).manual_seed(2), TDT[dtype], 40, 264, 256
    n = nn.mlp_op_wgrad8_workspace_bytes(dtype, N, K, M)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    dw, db = torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    sums = []

    def call(t, ld):
        p = {k: v.data_ptr() for k, v in t.items()}
        nn.mlp_op_quant8(dtype, M, K, p["x"], ld["x"], p["q"], ld["q"], p["e"], ld["e"], stream())
        nn.mlp_op_dequant8(dtype, M, K, p["q"], ld["q"], p["e"], ld["e"], p["y"], ld["y"], stream())
        nn.mlp_op_wgrad8(dtype, N, K, M, p["dy"], ld["dy"], p["q"], ld["q"], p["e"], ld["e"], dw.data_ptr(), K,
                         db.data_ptr(), ws.data_ptr(), n, None, stream())
        sums.append(torch.cat([dw.flatten(), db]))

    x = _rand(gen, M, K, td=td)
    _both(dict(x=x, y=torch.zeros_like(x), dy=_rand(gen, M, N, td=td), q=torch.zeros(M, K, dtype=torch.uint8, device=DEV),
               e=torch.zeros(M, 16, dtype=torch.uint8, device=DEV)), call, ["q", "e", "y"])
    assert torch.equal(sums[0], sums[1])


@pytest.mark.parametrize("dtype,M", [(nn.F32, 40), (nn.BF16, 16), (nn.BF16, 32), (nn.BF16, 40)])
@pytest.mark.parametrize("keep8", [False, True])
def test_gated(dtype, M, keep8):
    gen, td, F, K, N = torch.Generator(DEV).manual_seed(3), TDT[dtype], 256, 136, 72
    w, wd = _rand(gen, 2 * F, K, td=td), _rand(gen, N, F, td=td)
    pad = 40 - M                 # so that the last rows lie behind 2^31 elements: rows from pad on

    def call(t, ld):
        p = {k: v[pad:].data_ptr() for k, v in t.items()}
        e, le = (p["e"], ld["e"]) if keep8 else (None, 0)
        nn.mlp_op_gated_linear(dtype, nn.ACT_SILU, M, F, K, p["x"], ld["x"], w.data_ptr(), K, None, p["h"], ld["h"], p["s"],
                               ld["s"], e, le, None, stream())
        nn.mlp_op_gated_dgrad(dtype, nn.ACT_SILU, M, N, F, p["dy"], ld["dy"], wd.data_ptr(), F, p["s"], ld["s"], e, le,
                              p["ds"], ld["ds"], p["h2"], ld["h2"], None, stream())

    z = lambda c, d=td: torch.zeros(40, c, dtype=d, device=DEV)   # noqa: E731
    make = dict(x=_rand(gen, 40, K, td=td), dy=_rand(gen, 40, N, td=td), h=z(F), h2=z(F), ds=z(2 * F),
                s=z(2 * F, torch.uint8 if keep8 else td), e=z(16, torch.uint8))
    _both(make, call, ["h", "h2", "s", "e", "ds"])
