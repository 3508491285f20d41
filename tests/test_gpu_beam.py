"""Beam search's selection and the reordering of states, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import logits_oracle as lo
from tests.block_util import DEV, TDT, U32, Buf, assert_within, stream
from tests.logits_util import EX2, SUM, IntBuf, logits

pytestmark = pytest.mark.gpu

F, H = nn.F32, nn.BF16


def run_select(dtype, z, scores, m, done=None, eos=-1, pad=0, off=0, in_place=False):
    batch, W = scores.shape
    C = z.shape[1]
    Z = Buf(batch * W, C, TDT[dtype], C + pad, off, z)
    S = Buf(batch, W, torch.float32, values=torch.as_tensor(scores))
    D = None if done is None else Buf(batch, W, torch.uint8, values=torch.as_tensor(done))
    SO = S if in_place else Buf(batch, m, torch.float32)
    DO = D if in_place and done is not None else Buf(batch, m, torch.uint8)
    P, T = IntBuf(batch, m), IntBuf(batch, m)
    n = nn.mlp_op_beam_select_workspace_bytes(dtype, batch, W, C, m)
    ws = Buf(1, n, torch.uint8, off=8)
    nn.mlp_op_beam_select(dtype, batch, W, C, m, Z.ptr, Z.ld, S.ptr, None if D is None else D.ptr, eos, SO.ptr, P.ptr, T.ptr,
                          DO.ptr, ws.ptr, n, stream())
    torch.cuda.synchronize()
    for b in (Z, S, SO, DO, P, T, ws):
        b.check_canary()
    return SO.np(), P.np().astype(int), T.np().astype(int), DO.np().astype(int), Z.np()


def check(dtype, z, scores, m, done=None, eos=-1, **kw):
    scores = np.asarray(scores, np.float32)
    s, p, t, d, x = run_select(dtype, z, scores, m, done, eos, **kw)
    batch, W = scores.shape
    for b in range(batch):
        rows = x[b * W:(b + 1) * W]
        wt, wp, wc, wd = lo.beam_select(rows, scores[b], min(m + 1, rows.size), None if done is None else done[b], eos)
        # what a row's log-sum may be off by; pairs of different beams further apart than that have one order
        fin = rows[np.isfinite(rows)]
        tol = 2 * (EX2 + SUM + 4 * U32 * (np.ptp(fin) if fin.size else 0))
        near = np.isfinite(wt[1:]) & np.isfinite(wt[:-1]) & (wt[:-1] - wt[1:] <= tol) & (wp[1:] != wp[:-1])
        if near.any():   # rounding may order these pairs of different beams either way: the totals are in order, all others are exact
            all_totals = lo.beam_totals(rows, scores[b], None if done is None else done[b], eos)
            got = all_totals[p[b], t[b]]
            assert len(set(zip(p[b], t[b]))) == m and np.abs(got - wt[:m])[np.isfinite(wt[:m])].max() <= tol
            free = np.zeros(m + 1, bool)
            free[:-1] |= near[:m]
            free[1:len(near) + 1] |= near[:m]
            sure = ~free[:m]
            assert near.mean() < 0.2
            assert np.array_equal(p[b][sure], wp[:m][sure]) and np.array_equal(t[b][sure], wc[:m][sure])
            assert np.array_equal(d[b], (t[b] == eos) | (False if done is None else done[b][p[b]] != 0))
        else:
            assert np.array_equal(p[b], wp[:m]) and np.array_equal(t[b], wc[:m]) and np.array_equal(d[b], wd[:m].astype(int))
        fine = np.isfinite(wt[:m])
        assert np.array_equal(s[b][~fine], wt[:m][~fine], equal_nan=True)
        assert_within(s[b][fine], wt[:m][fine], tol + U32 * np.abs(wt[:m][fine]), "scores")


def scores_of(rng, batch, W):
    return np.sort(-30 - 3 * rng.uniform(size=(batch, W)), axis=1)[:, ::-1].astype(np.float32)


# the coarse logits of bf16 are equal within a beam often, and never across beams (the scores and log-sums differ)
@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("batch,W,C,m,pad,off", [
    (1, 1, 1, 1, 0, 0), (2, 2, 3, 6, 1, 1), (3, 4, 5, 8, 0, 0), (1, 4, 100, 4, 0, 0), (2, 5, 1001, 10, 3, 5),
    (5, 3, 4096, 6, 0, 0), (1, 4, 32000, 8, 0, 0), (70, 8, 2000, 16, 0, 0), (2, 32, 500, 64, 0, 1), (1, 32, 9001, 32, 0, 0),
    (3, 6, 50001, 12, 0, 0), (40, 9, 12000, 9, 8, 0)])
def test_against_the_oracle(dtype, batch, W, C, m, pad, off):
    rng = np.random.default_rng([1, batch, W, C])
    done = (rng.uniform(size=(batch, W)) < 0.2).astype(np.uint8)
    check(dtype, logits(rng, batch * W, C, TDT[dtype]), scores_of(rng, batch, W), m, done, C // 2, pad=pad, off=off)


@pytest.mark.parametrize("dtype", [F, H])
def test_without_finished_beams_and_in_place(dtype):
    rng = np.random.default_rng(2)
    check(dtype, logits(rng, 12, 3000, TDT[dtype]), scores_of(rng, 3, 4), 4, in_place=True)
    check(dtype, logits(rng, 12, 3000, TDT[dtype]), scores_of(rng, 3, 4), 4, np.array([[0, 1, 0, 0]] * 3, np.uint8), 7,
          in_place=True)
    check(dtype, logits(rng, 12, 3000, TDT[dtype]), scores_of(rng, 3, 4), 8, None, 5)


@pytest.mark.parametrize("dtype", [F, H])
def test_first_step_masks_and_all_finished(dtype):
    rng = np.random.default_rng(3)
    W, C = 4, 2500
    s = np.full((5, W), -np.inf, np.float32)
    s[:, 0] = 0.0
    s[2] = -np.inf                         # nothing left at all
    s[4] = scores_of(rng, 1, W)[0]
    z = logits(rng, 5 * W, C, TDT[dtype])
    z[4, 10:] = -np.inf                    # fewer tokens allowed than taken, but for the first beam of entry 1
    z[12, :] = -np.inf                     # no token allowed
    z[17, 1:] = -np.inf                    # one token
    z[18, 3] = float("nan")
    z[19, 3] = float("inf")
    check(dtype, z, s, 16)
    done = np.ones((5, W), np.uint8)
    done[1] = [0, 1, 0, 0]
    check(dtype, z, s, 8, done, 0)
    s[0, 1] = float("nan")
    s[0, 2] = float("inf")
    check(dtype, z, s, 8)
    check(dtype, z, s, 64)


@pytest.mark.parametrize("W,C,m", [(4, 9, 20), (8, 3, 24), (16, 2, 30), (3, 40000, 12), (12, 5000, 24)])
def test_finished_beams_without_a_score(W, C, m):
    """A finished beam of score -infinity offers its tokens in order, one of NaN nothing; its flag stays."""
    rng = np.random.default_rng([9, W])
    s = scores_of(rng, 3, W)
    done = np.zeros((3, W), np.uint8)
    s[:, 1] = -np.inf
    done[:, :2] = 1
    s[1, 2], s[2, 0] = np.nan, -np.inf
    done[1, 2] = 1
    check(F, logits(rng, 3 * W, C, torch.float32), s, m, done, C - 1)


def test_totals_far_below_zero_are_compared_in_64_bits():
    """Scores of -1000: an fp32 total has a step of 6e-5, and beams 1e-5 apart keep their order."""
    rng = np.random.default_rng(4)
    z = logits(rng, 1, 4000, torch.float32, 0.5).repeat(4, 1)
    z[1] += 1.0                                      # (a shift leaves the row's log-probabilities)
    z = (z * 2 ** 10).round() / 2 ** 10              # exact in fp32 with the shift
    z[1] = z[0] + 1.0
    z[2:] = z[:2]
    s = np.array([[-1000.0, -1000.0001, -1000.0002, -1000.0003]], np.float32)   # fp32 neighbours 6.1e-5 apart
    check(F, z, s, 32)


def test_equal_beams_keep_their_order():
    """Beams of the same logits and score: every pair ties, the lower beam goes first, at any alignment."""
    rng = np.random.default_rng(5)
    for C, pad, off in ((3000, 0, 0), (33000, 0, 0), (40000, 8, 8)):
        z = logits(rng, 1, C, torch.bfloat16).repeat(6, 1)
        s, p, t, d, x = run_select(H, z, np.full((2, 3), -5.0, np.float32), 9, pad=pad, off=off)
        wt, wp, wc, _ = lo.beam_select(x[:3], [-5.0] * 3, 9)
        for b in range(2):
            assert np.array_equal(p[b], wp) and np.array_equal(t[b], wc)


def test_twice_gives_the_same_bits():
    rng = np.random.default_rng(6)
    z, s = logits(rng, 40, 20000, torch.bfloat16), scores_of(rng, 10, 4)
    a, b = run_select(H, z, s, 8), run_select(H, z, s, 8)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


# ---- reordering
def run_reorder(planes, batch, win, wout, n, td, pitch_pad=0, off=0, plane_pad=0, in_place=False, bad=False, ldp_pad=0):
    rng = np.random.default_rng([7, planes, batch, win, wout, n])
    gen = torch.Generator(device=DEV)
    gen.manual_seed(n)
    es = torch.empty(0, dtype=td).element_size()
    ld = n + pitch_pad

    def buf(w):
        rows = planes * (batch * w) + (planes - 1) * plane_pad
        flat = torch.randint(0, 100, (off + rows * ld + 8,), generator=gen, device=DEV).to(td)
        return flat, (batch * w + plane_pad) * ld

    src, sp = buf(win)
    dst, dp = (src, sp) if in_place else buf(wout)
    src0, dst0 = src.clone(), dst.clone()
    par = rng.integers(0, win, (batch, wout + ldp_pad))
    if bad:
        par[0, 0], par[-1, -1 - ldp_pad] = win, -1
    pt = torch.from_numpy(par.astype(np.int32)).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    nn.mlp_op_beam_reorder(planes, batch, win, wout, n * es, src.data_ptr() + off * es, ld * es, sp * es, pt.data_ptr(),
                           wout + ldp_pad, dst.data_ptr() + off * es, ld * es, dp * es, err.data_ptr(), stream())
    want = dst0.clone()
    for p in range(planes):
        for b in range(batch):
            for i in range(wout):
                f = int(par[b, i])
                if 0 <= f < win:
                    a = off + p * sp + (b * win + f) * ld
                    c = off + p * dp + (b * wout + i) * ld
                    want[c:c + n] = src0[a:a + n]
    torch.cuda.synchronize()
    assert torch.equal(dst, want)
    if not in_place:
        assert torch.equal(src, src0)
    assert err.item() == (1 if bad else 0)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("planes,batch,W,n,td,pitch_pad,off,plane_pad", [
    (1, 1, 1, 1, torch.uint8, 0, 0, 0), (1, 3, 4, 17, torch.uint8, 1, 1, 0), (2, 2, 3, 33, torch.bfloat16, 0, 0, 1),
    (2, 1, 4, 1024, torch.bfloat16, 0, 0, 0), (3, 5, 8, 520, torch.bfloat16, 8, 8, 2), (1, 2, 9, 1000, torch.float32, 0, 0, 0),
    (2, 3, 16, 770, torch.bfloat16, 2, 2, 0), (2, 2, 17, 300, torch.float32, 0, 0, 0), (1, 2, 32, 4097, torch.bfloat16, 1, 3, 0),
    (4, 2, 5, 20000, torch.float32, 0, 0, 0), (1, 70, 4, 64, torch.int32, 0, 0, 0), (2, 2, 12, 128, torch.uint8, 4, 4, 0)])
def test_reorder(planes, batch, W, n, td, pitch_pad, off, plane_pad, in_place):
    run_reorder(planes, batch, W, W, n, td, pitch_pad, off, plane_pad, in_place)


def test_reorder_other_counts_and_bad_parents():
    run_reorder(2, 3, 4, 8, 100, torch.bfloat16, ldp_pad=2)
    run_reorder(2, 3, 8, 2, 100, torch.bfloat16, ldp_pad=5)
    run_reorder(2, 3, 4, 4, 100, torch.bfloat16, bad=True)
    run_reorder(2, 3, 4, 4, 100, torch.bfloat16, in_place=True, bad=True)


def test_reorder_past_2_32_bytes():
    n = 1 << 30
    src = torch.empty(5 * n, dtype=torch.uint8, device=DEV)
    for i in range(5):
        src[i * n:(i + 1) * n] = i + 1
    par = torch.tensor([[4, 0, 1, 2, 3]], dtype=torch.int32, device=DEV)
    nn.mlp_op_beam_reorder(1, 1, 5, 5, n, src.data_ptr(), n, 0, par.data_ptr(), 5, src.data_ptr(), n, 0, None, stream())
    for i, v in enumerate([5, 1, 2, 3, 4]):
        assert (src[i * n:(i + 1) * n] == v).all()
