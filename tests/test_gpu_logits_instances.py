"""Every instance of the top-k, selection and distillation kernels over many rounds of its threads, and rows shared by the blocks of
a cluster, on ordinary rows and on rows of equals, orders, masks, NaN and infinity, against the fp64 oracle.  A row's results are
the same bits whatever lies beside it in a call of the same size, and from one call to the next."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import logits_oracle as lo
from tests import logits_rows as lr
from tests.block_util import HALF, TDT, U32, assert_within
from tests.logits_util import distill_tol, logits, run_distill, run_topk, teacher
from tests.test_gpu_beam import run_select, scores_of

pytestmark = pytest.mark.gpu

F, H = lr.F, lr.H
BIG = float(np.finfo(np.float32).max)


def _same(got, want, tol, what):
    """A log-sum against its value; what leaves fp32 is infinite there."""
    if abs(want) > BIG:
        assert got == np.sign(want) * np.inf, (what, got, want)
    else:
        assert abs(got - want) <= tol, (what, got, want, tol)


def _check_row(kind, x, k, T, n, v, i, l, r, sums=True):
    wv, wi, wl, wr = (a[0] for a in lo.topk(x[None], k, T))
    assert np.array_equal(i, wi), kind
    assert np.array_equal(v, wv, equal_nan=True), kind
    if not sums:
        return
    left = np.ones(len(x), bool)
    left[wi] = False
    odd = lambda y: bool(np.isnan(y).any() or (y == np.inf).any())
    most = np.nanmax(x, initial=-np.inf) / T
    if odd(x):
        assert np.isnan(l), (kind, l)
    elif x.max() == -np.inf:
        assert l == -np.inf, (kind, l)
    else:
        _same(l, wl, lr.log_sum_tol(x / T, most, n), (kind, "lse"))
    if odd(x[left]):
        assert np.isnan(r) or r == np.inf, (kind, r)
    elif not left.any() or x[left].max() == -np.inf:
        assert r == -np.inf, (kind, r)
    else:
        _same(r, wr, lr.log_sum_tol(x[left] / T, most, n), (kind, "tail"))


@pytest.mark.parametrize("case", lr.TOPK, ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_topk(case):
    dtype, B, C, k, mode, threads, blocks, _ = case
    index = lr.TOPK.index(case)
    rng = np.random.default_rng([1, index])
    T, off, K = (1.0, 2.0, 0.5)[index % 3], (0, 3)[index % 2], len(lr.KINDS)
    rows = [lr.row(kind, rng, C, dtype, k) for kind in lr.KINDS]
    n = -(-C // (blocks * threads))
    pad = -C % 8   # (every row at the same address modulo 16: the same order of its sums)
    bits = {}
    for first in range(0, K, B):
        which = (first + np.arange(B)) % K
        z = torch.stack(rows)[torch.from_numpy(which)]
        a = run_topk(dtype, z, k, T, pad=pad, off=off)
        b = run_topk(dtype, z.flip(0), k, T, pad=pad, off=off)
        for j in range(B):
            got = [y[j] for y in a[:4]]
            for other in ([y[B - 1 - j] for y in b[:4]], bits.setdefault(int(which[j]), got)):
                assert all(np.array_equal(p, q, equal_nan=True) for p, q in zip(got, other)), lr.KINDS[which[j]]
    for w, kind in enumerate(lr.KINDS):
        _check_row(kind, rows[w].double().numpy(), k, T, n, *bits[w])


@pytest.mark.parametrize("lse,tail", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("dtype,B,C,k", [(F, 23, 70001, 40), (H, 23, 140001, 40), (H, 46, 140001, 200), (F, 9, 300001, 7)])
def test_topk_of_shared_rows_without_some_sums(dtype, B, C, k, lse, tail):
    rng = np.random.default_rng(2)
    kinds = [lr.KINDS[j % len(lr.KINDS)] for j in range(B)]
    z = torch.stack([lr.row(kind, rng, C, dtype, k) for kind in kinds])
    v, i, l, r, x = run_topk(dtype, z, k, 1.0, lse, tail)
    v2, i2, l2, r2, _ = run_topk(dtype, z, k, 1.0)
    assert np.array_equal(v, v2, equal_nan=True) and np.array_equal(i, i2)
    assert np.array_equal(l, l2, equal_nan=True) if lse else (l == -777).all()
    assert np.array_equal(r, r2, equal_nan=True) if tail else (r == -777).all()
    for j, kind in enumerate(kinds):
        _check_row(kind, x[j], k, 1.0, 1 << 10, v[j], i[j], l[j], r[j], sums=False)


def _check_entry(rows, s, m, done, eos, n, got):
    """One batch entry's selection.  Pairs of different beams whose totals are within the log-sums' errors may come in either
    order; everything else has one place."""
    ts, tp, tt, td = got
    W = len(rows)
    more = min(m + 16, rows.size)
    wt, wp, wc, wd = lo.beam_select(rows, s, more, done, eos)
    tot = lo.beam_totals(rows, s, done, eos)
    tol = np.zeros(W)
    for w in range(W):
        if not done[w] and np.isfinite(s[w]) and np.isfinite(tot[w]).any():
            tol[w] = lr.log_sum_tol(rows[w], rows[w].max(), n)
    fin = np.isfinite(wt)
    assert np.array_equal(np.isfinite(tot[tp, tt]), fin[:m]) and len(set(zip(tp, tt))) == m
    near = np.zeros(more, bool)
    a = np.where(fin, wt, 0.0)
    for j in np.flatnonzero(fin):
        near[j] = (fin & (wp != wp[j]) & (np.abs(a - a[j]) <= tol[wp] + tol[wp[j]])).any()
    sure = ~near[:m]
    assert sure.mean() > 0.5
    assert np.array_equal(tp[sure], wp[:m][sure]) and np.array_equal(tt[sure], wc[:m][sure]) and np.array_equal(td[sure], wd[:m][sure])
    assert np.array_equal(td, (tt == eos) | (done[tp] != 0))
    f = fin[:m]
    assert np.array_equal(ts[~f], wt[:m][~f], equal_nan=True)
    assert_within(ts[f], wt[:m][f], 2 * tol.max(initial=0.0) + U32 * np.abs(wt[:m][f]) + 1e-12, "scores")


@pytest.mark.parametrize("case", lr.SELECT, ids=lambda c: "-".join(str(x) for x in c[:5]))
def test_select(case):
    dtype, batch, W, C, m, mode, threads, blocks, _ = case
    index = lr.SELECT.index(case)
    rng = np.random.default_rng([3, index])
    D, K = min(batch, 6), len(lr.KINDS)
    kinds = [lr.KINDS[(7 * index + j) % K] for j in range(D * W)]
    rows = torch.stack([lr.row(kind, rng, C, dtype, m) for kind in kinds])
    s = scores_of(rng, D, W)
    done = (rng.uniform(size=(D, W)) < 0.15).astype(np.uint8)
    eos = C // 3
    e = np.arange(batch) % D
    z = rows.view(D, W, C)[torch.from_numpy(e)].reshape(batch * W, C)
    pad = -C % 8
    a = run_select(dtype, z, s[e], m, done[e], eos, pad=pad, off=5)
    b = run_select(dtype, z, s[e], m, done[e], eos, pad=pad, off=5)
    x = rows.double().numpy().reshape(D, W, C)
    n = -(-C // ((blocks if mode == lr.SLICES else 1) * threads))
    for j in range(batch):
        assert all(np.array_equal(p[j], q[j], equal_nan=True) and np.array_equal(p[j], p[e[j]], equal_nan=True)
                   for p, q in zip(a[:4], b[:4]))
    for j in range(D):
        _check_entry(x[j], s[j], m, done[j], eos, n, [y[j] for y in a[:4]])


@pytest.mark.parametrize("case", lr.DISTILL, ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_distill(case):
    dtype, B, C, k, blocks, threads, _ = case
    index = lr.DISTILL.index(case)
    rng = np.random.default_rng([4, index])
    D, T, off = 12, (1.0, 2.0, 4.0)[index % 3], (0, 3)[index % 2]
    z = logits(rng, D, C, TDT[dtype])
    tv, ti, tl = teacher(rng, z.double().numpy(), k, T)
    free = lambda i, n: torch.from_numpy(np.setdiff1d(rng.permutation(C)[:n], ti[i]))
    z[1, free(1, C // 3)] = -np.inf
    z[2, free(2, C // 3)] = torch.finfo(TDT[dtype]).min
    z[3, ti[3]] += 200.0
    ti[4, k // 3:] = -1
    ti[5], ti[6] = -1, -1
    tl[6] = -np.inf
    z[7, :], tl[7] = np.nan, np.nan
    z[8, torch.from_numpy(np.setdiff1d(np.arange(C // 2), ti[8]))] = -np.inf
    y = rng.integers(0, C, D)
    y[[1, 2, 8]], y[9] = ti[[1, 2, 8], 0], ti[9, k - 1]
    w = np.ones(D, np.float32)
    w[7], w[11], y[7] = 0.0, 0.5, -100
    e = np.arange(B) % D
    args = (tv[e], ti[e], tl[e], y[e], w[e], T, 0.4, 0.6 * T * T, 1.0 / D)
    pad = -C % 8
    loss, dz, bits, x = run_distill(dtype, z[torch.from_numpy(e)], *args, pad=pad, off=off, dpad=pad, doff=off)
    loss2, dz2, _, _ = run_distill(dtype, z[torch.from_numpy(e)], *args, pad=pad, off=off, in_place=True)
    alone, _, _, _ = run_distill(dtype, z[torch.from_numpy(e)], *args, pad=pad, off=off, grad=False)
    assert bits == 0
    assert np.array_equal(loss, loss[e]) and np.array_equal(dz, dz[e])
    assert np.array_equal(loss, loss2) and np.array_equal(dz, dz2) and np.array_equal(loss, alone)
    x, few = x[:D], np.arange(D) != 7
    f32 = lambda a: a.astype(np.float32)
    g = (x[few], f32(tv)[few], ti[few], f32(tl)[few], y[few], w[few], T, 0.4, 0.6 * T * T, 1.0 / D)
    wl, wd, _ = lo.distill(*g)
    t1, t2 = distill_tol(*g, wl, wd, HALF[dtype])
    assert loss[7] == 0 and not dz[7].any()
    assert_within(loss[:D][few], wl, t1, "loss")
    assert_within(dz[:D][few], wd, t2, "dz")


@pytest.mark.parametrize("dtype,B,C,k", [(H, 700, 16001, 20), (F, 160, 30001, 33), (H, 20, 300001, 64), (H, 1300, 4001, 8)])
def test_distill_with_a_gradient_at_another_address_modulo_16(dtype, B, C, k):
    """Written element by element: the same bits as by bulk copies."""
    rng = np.random.default_rng(5)
    D, T = 6, 2.0
    z = logits(rng, D, C, TDT[dtype])
    tv, ti, tl = teacher(rng, z.double().numpy(), k, T)
    y, e = rng.integers(0, C, D), np.arange(B) % D
    args = (dtype, z[torch.from_numpy(e)], tv[e], ti[e], tl[e], y[e], None, T, 0.4, 0.6 * T * T, 1.0)
    pad = -C % 8
    loss, dz, _, _ = run_distill(*args, pad=pad, dpad=pad)
    loss2, dz2, _, _ = run_distill(*args, pad=pad, dpad=pad + 1, doff=3)
    assert np.array_equal(loss, loss2) and np.array_equal(dz, dz2)
