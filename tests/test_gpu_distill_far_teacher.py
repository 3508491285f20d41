"""A teacher's logits count by their differences alone: rows far from zero (shifted, masked by the type's lowest value as a
whole, at fp32's ends over a T below 1) give what the same row near zero gives."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import logits_oracle as lo
from tests.block_util import HALF, TDT, assert_within
from tests.logits_util import distill_tol, logits, run_distill

pytestmark = pytest.mark.gpu

F, H = nn.F32, nn.BF16
LOW = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("T", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("C,k", [(50, 7), (3000, 40), (60000, 100)])
def test_a_shifted_teacher(dtype, T, C, k):
    rng = np.random.default_rng([1, C])
    shifts = [3e3, -5e4, 1e6, -2.0 ** 30, 3e38, LOW, -LOW, 20.0, -50.0, 700.0]
    B = len(shifts)
    z = logits(rng, B, C, TDT[dtype])
    ti = np.stack([rng.permutation(C)[:k] for _ in range(B)])
    # (what fp32 keeps of the shifted row is the row: at 2^30 and beyond its entries are equal or steps apart)
    tv = np.clip(rng.normal(size=(B, k)) * 2 + np.array(shifts)[:, None], LOW, -LOW).astype(np.float32)
    near = tv.astype(np.float64) - tv.max(1, keepdims=True)
    loss, dz, bits, x = run_distill(dtype, z, tv, ti, T=T, b=T * T)
    args = (x, near, ti, None, None, None, T, 0.0, T * T, 1.0)
    wl, wd, _ = lo.distill(*args)
    # (the oracle's own log-sums have 64 bits: at 1e6 still 2e-10 of one)
    assert np.allclose(wl[:3], lo.distill(x[:3], tv[:3].astype(np.float64), ti[:3], T=T, b=T * T)[0], rtol=1e-7)
    t1, t2 = distill_tol(*args, wl, wd, HALF[dtype])
    assert bits == 0 and np.isfinite(wl).all()
    assert_within(loss, wl, t1, "loss")
    assert_within(dz, wd, t2, "dz")


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("T", [0.5, 1.0])
def test_entries_of_the_lowest_value_beside_a_tail_have_no_weight(dtype, T):
    rng = np.random.default_rng(2)
    B, C, k = 4, 900, 9
    z = logits(rng, B, C, TDT[dtype])
    ti = np.stack([rng.permutation(C)[:k] for _ in range(B)])
    tv = np.full((B, k), LOW, np.float32)
    tail = rng.normal(size=B).astype(np.float32) * 3
    loss, dz, bits, x = run_distill(dtype, z, tv, ti, tail, T=T, b=T * T)
    args = (x, np.full((B, k), -np.inf), ti, tail, None, None, T, 0.0, T * T, 1.0)
    wl, wd, _ = lo.distill(*args)
    t1, t2 = distill_tol(x, np.full((B, k), -1e30), ti, tail, None, None, T, 0.0, T * T, 1.0, wl, wd, HALF[dtype])
    assert_within(loss, wl, 1e-5 * (1 + wl), "loss")
    assert_within(dz, wd, t2, "dz")


@pytest.mark.parametrize("dtype", [F, H])
def test_a_student_of_nothing_but_the_lowest_value(dtype):
    """A row masked as a whole is uniform."""
    rng = np.random.default_rng(3)
    B, C, k = 3, 700, 12
    low = torch.finfo(TDT[dtype]).min
    z = torch.full((B, C), low, dtype=TDT[dtype])
    ti = np.stack([rng.permutation(C)[:k] for _ in range(B)])
    tv = rng.normal(size=(B, k)).astype(np.float32) * 2
    for T in (0.5, 1.0, 2.0):
        loss, dz, bits, x = run_distill(dtype, z, tv, ti, T=T, b=T * T)
        args = (x - float(low), tv, ti, None, None, None, T, 0.0, T * T, 1.0)
        wl, wd, _ = lo.distill(*args)
        t1, t2 = distill_tol(*args, wl, wd, HALF[dtype])
        assert_within(loss, wl, t1, "loss")
        assert_within(dz, wd, t2, "dz")
