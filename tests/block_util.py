"""Helpers of the feed-forward block's GPU tests."""
import numpy as np
import torch

import neural_net_step_gb300 as nn

DEV = "cuda:0"
U32 = 2.0 ** -24                      # half a step of fp32, relative
HALF = {nn.F32: 2.0 ** -24, nn.BF16: 2.0 ** -8}
TDT = {nn.F32: torch.float32, nn.BF16: torch.bfloat16}


def stream():
    return torch.cuda.current_stream().cuda_stream


def sum_err(absum, n):
    """Error of an fp32 sum of n terms of absolute sum `absum`: 8x the rms
    growth of recursive summation (and at least 16 roundings)."""
    return (8.0 * np.sqrt(max(n, 1)) + 16.0) * U32 * absum


class Buf:
    """A [rows, cols] device matrix of row pitch ld, `off` elements past an
    aligned address, surrounded and padded by a canary."""

    def __init__(self, rows, cols, td, ld=None, off=0, values=None):
        self.rows, self.cols, self.ld, self.off = rows, cols, ld or cols, off
        self.flat = torch.full((off + rows * self.ld + 64,), 0x5A if td == torch.uint8 else float("nan"), dtype=td,
                               device=DEV)
        if td != torch.uint8:
            self.flat.fill_(-777.0)
        self.before = self.flat.clone()
        self.t = torch.as_strided(self.flat, (rows, cols), (self.ld, 1), off)
        if values is not None:
            self.t.copy_(values)

    @property
    def ptr(self):
        return self.flat.data_ptr() + self.off * self.flat.element_size()

    def check_canary(self):
        now = self.flat.clone()
        torch.as_strided(now, (self.rows, self.cols), (self.ld, 1), self.off).copy_(
            torch.as_strided(self.before, (self.rows, self.cols), (self.ld, 1), self.off))
        assert torch.equal(now, self.before), "written outside the matrix"

    def np(self):
        return self.t.detach().cpu().to(torch.float64).numpy()


def assert_within(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        r = np.where(bad, np.abs(got - want) / np.maximum(tol, 1e-300), 0.0)
        i = np.unravel_index(np.nanargmax(r), r.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} out of tolerance; worst at {i}: got {got[i]!r} "
                             f"want {want[i]!r} tol {np.broadcast_to(tol, got.shape)[i]!r}")
