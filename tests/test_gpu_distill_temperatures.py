"""Distillation at high and low temperatures, soft and hard targets each alone, against bounds that are small next to what they
bound.

At a high T the teacher's and the student's shares of a column differ by about |z - t| / T of themselves, and each carries
the relative error of its exponential and its sum.  Those, not more, are what loss and gradient may be off by: the gradient by
its shares' errors, the loss (p times r^2 / 2 for r = log(p / q)) by p |r| times the error of r, and half that error's square."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import logits_oracle as lo
from tests.block_util import HALF, TDT, U32, assert_within
from tests.logits_util import EX2, run_distill

pytestmark = pytest.mark.gpu

F, H = nn.F32, nn.BF16
# a sum of at most 3000 terms: a thread's run of at most 48 in two lanes and two sums each, then trees of at most 16
# levels; each addition half a step
SUMS = (12 + 16) * U32


def _shares(x):
    p = np.exp(x - x.max())
    return p / p.sum()


def _bounds(z, tv, ti, tail, T):
    """(relative error of a share by row, its log-ratio r by class and for the rest, p, q, R)"""
    out = []
    for i in range(len(z)):
        x = z[i] / T
        q = _shares(x)
        t = np.append(tv[i].astype(np.float64) / T, -np.inf if tail is None else float(tail[i]))
        p = _shares(t)
        others = np.ones(z.shape[1], bool)
        others[ti[i]] = False
        R = q[others].sum()
        # exponent: factor, product and difference rounded at the size of (x - max) and of the reference that tail and the
        # largest share; expf and ex2; the two sums; two divisions
        far = max(np.ptp(x), np.ptp(t[np.isfinite(t)]))
        ref = abs(t[np.isfinite(t)]).max() if tail is not None else 0.0
        out.append((EX2 + 2 * U32 * (2 * far + ref) + SUMS + 6 * U32, p, q, R))
    return out


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("T", [3.0, 30.0, 300.0, 1000.0])
@pytest.mark.parametrize("C,k,tail", [(37, 37, False), (700, 9, False), (700, 9, True), (3000, 200, False), (3000, 200, True)])
def test_soft_targets_alone(dtype, T, C, k, tail):
    rng = np.random.default_rng([1, C])
    B = 5
    z = torch.from_numpy((rng.normal(size=(B, C)) * 2).astype(np.float32)).to(TDT[dtype])
    t = (z.double().numpy() + 2.0 * rng.normal(size=(B, C))).astype(np.float32).astype(np.float64)
    v, i, _, tl = lo.topk(t, k, T)
    v, tl = v.astype(np.float32), tl.astype(np.float32) if tail else None
    loss, dz, bits, x = run_distill(dtype, z, v, i, tl, T=T, b=T * T)
    wl, wd, _ = lo.distill(x, v, i, tl, T=T, b=T * T)
    td, tloss = np.zeros_like(wd), np.zeros(B)
    for n, (e, p, q, R) in enumerate(_bounds(x, v, i, tl, T)):
        share = q.copy()
        share[i[n]] += p[:-1]
        if p[-1] > 0:
            others = np.ones(C, bool)
            others[i[n]] = False
            share[others] *= 1 + p[-1] / R
        td[n] = T * 2 * e * share + (HALF[dtype] + 4 * U32) * np.abs(wd[n])
        ps, qs = p[p > 0], np.append(q[i[n]], R)[p > 0]
        r = np.abs(np.log(ps / qs))
        d = 2 * e + 4 * U32 * r
        tloss[n] = T * T * (np.abs(ps - qs) * d + np.maximum(ps, qs) * d * d).sum() + 8 * U32 * wl[n]
    assert bits == 0
    # the bounds say something: a loss or a gradient without its soft part is far outside them
    assert (tloss < 0.05 * wl).all() and (td.max(1) < 0.05 * np.abs(wd).max(1)).all()
    assert_within(loss, wl, tloss, "loss")
    assert_within(dz, wd, td, "dz")


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("T", [1e-6, 1e-3, 2.0, 30.0, 1e3, 1e6])
@pytest.mark.parametrize("C", [700, 3000])
def test_hard_labels_alone(dtype, T, C):
    """With kd_weight 0 the temperature changes nothing."""
    rng = np.random.default_rng([2, C])
    B, k = 5, 6
    z = torch.from_numpy((rng.normal(size=(B, C)) * 2).astype(np.float32)).to(TDT[dtype])
    x = z.double().numpy()
    v, i, _, tl = lo.topk(x + rng.normal(size=x.shape), k, 1.0)
    y = np.array([i[0, 0], i[1, 2], 5, 6, 7])
    loss, dz, bits, _ = run_distill(dtype, z, v, i, tl, y, None, T, 0.5, 0.0, 1.0)
    wl, wd, _ = lo.distill(x, v.astype(np.float32), i, tl.astype(np.float32), y, None, T, 0.5, 0.0, 1.0)
    e = np.array([EX2 * 2 + 4 * U32 * np.ptp(a) + SUMS * 2 + 6 * U32 for a in x])   # (T = 2: squares, twice the error)
    share = np.stack([_shares(a) for a in x])
    td = 0.5 * 2 * e[:, None] * share + (HALF[dtype] + 2 * U32) * np.abs(wd)
    td[np.arange(B), y] += 2 * U32
    tloss = 0.5 * (2 * e + 4 * U32 * (np.abs(x).max() + np.log(C)))
    assert bits == 0 and (td.max(1) < 0.02 * np.abs(wd).max(1)).all() and (tloss < 0.01 * wl).all()
    assert_within(loss, wl, tloss, "loss")
    assert_within(dz, wd, td, "dz")


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("T", [1e-6, 1e-4, 1e-2])
def test_soft_targets_alone_at_low_temperatures(dtype, T):
    """Logits that T brings to the usual size; loss and gradient relative to their own."""
    rng = np.random.default_rng(3)
    B, C, k = 5, 700, 9
    z = torch.from_numpy((rng.normal(size=(B, C)) * 2 * T).astype(np.float32)).to(TDT[dtype])
    T32 = float(np.float32(T))
    x = z.double().numpy()
    t = (x + T * rng.normal(size=x.shape)).astype(np.float32).astype(np.float64)
    v, i, _, tl = lo.topk(t, k, T32)
    v, tl = v.astype(np.float32), tl.astype(np.float32)
    b = float(np.float32(T))
    loss, dz, bits, _ = run_distill(dtype, z, v, i, tl, T=T, b=b)
    wl, wd, _ = lo.distill(x, v, i, tl, T=T32, b=b)
    td, tloss = np.zeros_like(wd), np.zeros(B)
    for n, (e, p, q, R) in enumerate(_bounds(x, v, i, tl, T32)):
        share = q.copy()
        share[i[n]] += p[:-1]
        others = np.ones(C, bool)
        others[i[n]] = False
        share[others] *= 1 + p[-1] / R
        td[n] = 2 * e * share + (HALF[dtype] + 6 * U32) * np.abs(wd[n])
        qs = np.append(q[i[n]], R)
        d = 2 * e + 4 * U32 * np.abs(np.log(p / qs))
        tloss[n] = b * (np.abs(p - qs) * d + np.maximum(p, qs) * d * d).sum() + 8 * U32 * wl[n]
    assert bits == 0 and (tloss < 0.01 * wl).all() and (td.max(1) < 0.02 * np.abs(wd).max(1)).all()
    assert_within(loss, wl, tloss, "loss")
    assert_within(dz, wd, td, "dz")
