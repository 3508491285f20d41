"""The operations on logits at the ends of their ranges: temperatures, magnitudes, counts, and rows whose rest is far below."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import logits_oracle as lo
from tests.block_util import DEV, HALF, TDT, U32, assert_within, stream
from tests.logits_util import EX2, SUM, logits, run_distill, run_topk
from tests.test_gpu_beam import check as check_select, scores_of
from tests.test_gpu_distill import check as check_distill
from tests.test_gpu_topk import check as check_topk
from tests.logits_util import teacher

pytestmark = pytest.mark.gpu

F, H = nn.F32, nn.BF16


def _log_tol(x, T):
    """Of a log-sum at any temperature: exponents up to |x| / T are rounded at their own size."""
    return np.abs(x).max() / T * 4 * U32 + EX2 + SUM + 8 * U32


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("T", [1e-6, 1e-4, 1e-2, 1e2, 1e6])
def test_topk_at_every_temperature(dtype, T):
    rng = np.random.default_rng(1)
    for B, C, k in ((3, 3000, 7), (300, 9000, 40), (2, 150000, 5)):
        z = logits(rng, B, C, TDT[dtype])
        v, i, l, r, x = run_topk(dtype, z, k, T)
        wv, wi, wl, wr = lo.topk(x, k, float(np.float32(T)))
        assert np.array_equal(i, wi) and np.array_equal(v, wv)
        assert_within(l, wl, np.full(B, _log_tol(x, T)) + U32 * np.abs(wl), "lse")
        assert_within(r, wr, np.full(B, _log_tol(x, T)) + U32 * np.abs(wr), "tail")


def test_topk_of_huge_logits():
    """fp32 logits up to the type's ends: order and the largest entry's sum stay right."""
    rng = np.random.default_rng(2)
    for C in (2000, 70000):
        z = torch.from_numpy((rng.normal(size=(4, C)) * 1e38).clip(-3.4e38, 3.4e38).astype(np.float32))
        v, i, l, r, x = run_topk(F, z, 12, 1.0)
        wv, wi, wl, wr = lo.topk(x, 12, 1.0)
        assert np.array_equal(i, wi) and np.array_equal(v, wv)
        assert_within(l, wl, 4 * U32 * np.abs(wl), "lse")
        assert_within(r, wr, 4 * U32 * np.abs(wr), "tail")


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 200, 255, 256])
def test_topk_of_every_width(dtype, k):
    rng = np.random.default_rng([3, k])
    for B, C in ((2, 300), (400, 2600), (700, 700), (3, 33000), (1, 100001)):
        check_topk(dtype, logits(rng, B, C, TDT[dtype]), k)


@pytest.mark.parametrize("dtype", [F, H])
def test_topk_candidates_at_the_edges_of_a_row(dtype):
    """The largest elements lie before the first and behind the last whole 16 bytes."""
    rng = np.random.default_rng(4)
    for off in range(9):
        C = 1000 + off
        z = logits(rng, 5, C, torch.float32)
        z[:, :7] += 30.0
        z[:, -7:] += 30.0
        check_topk(dtype, z.to(TDT[dtype]), 20, off=off, pad=off % 3)


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("T", [1e-6, 1e-3, 2.0, 1e3, 1e6])
def test_distill_at_every_temperature(dtype, T):
    """Against the oracle on a student near its teacher in units of T (else every share is 0 or 1)."""
    rng = np.random.default_rng(5)
    T32 = float(np.float32(T))
    for C in (700, 70000):
        z = torch.from_numpy((rng.normal(size=(3, C)) * min(T, 1.0) * 2).astype(np.float32)).to(TDT[dtype])
        x = z.double().numpy()
        t = (x + min(T, 1.0) * rng.normal(size=x.shape)).astype(np.float32).astype(np.float64)
        v, i, _, tail = lo.topk(t, 9, T32)
        v, tail = v.astype(np.float32), tail.astype(np.float32)
        y = rng.integers(0, C, 3)
        loss, dz, bits, _ = run_distill(dtype, z, v, i, tail, y, None, T, 0.25, 0.5 * T, 1.0)
        wl, wd, _ = lo.distill(x, v, i, tail, y, None, T32, 0.25, float(np.float32(0.5 * T)), 1.0)
        assert bits == 0
        e = 64 * U32 * (1 + (np.abs(x).max() + np.abs(v).max()) / T) + 4 * (EX2 + SUM)
        assert_within(loss, wl, np.full(3, e) * (0.5 * T * (1 + np.log(C)) + 0.25 * (np.log(C) + np.abs(x).max() + 1)), "loss")
        assert_within(dz, wd, HALF[dtype] * np.abs(wd) + 2 * e * (np.abs(wd) + 0.75) * 1.5, "dz")


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("C", [900, 40000])
def test_distill_with_a_rest_far_below(dtype, C):
    """The student's other columns hold e^-150 and less, the teacher's half: the loss is that far, the gradient finite."""
    rng = np.random.default_rng(6)
    z = logits(rng, 4, C, torch.float32)
    k = 5
    ti = np.stack([rng.permutation(C)[:k] for _ in range(4)])
    for i in range(4):
        z[i, ti[i]] += 160.0 + 20.0 * i
    z = z.to(TDT[dtype])
    x = z.double().numpy()
    tv = rng.normal(size=(4, k)).astype(np.float32)
    tail = np.log(np.exp(tv).sum(1)).astype(np.float32)
    loss, dz, bits, _ = run_distill(dtype, z, tv, ti, tail)
    wl, wd, _ = lo.distill(x, tv, ti, tail)
    assert (wl > 60).all()
    assert_within(loss, wl, 2e-6 * wl, "loss")
    assert_within(dz, wd, HALF[dtype] * np.abs(wd) + 1e-5 * np.abs(wd) + 1e-6, "dz")


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("C", [20, 3000])
def test_distill_of_lowest_values_at_small_temperatures(dtype, C):
    """A teacher's weight of 1e-40 where the student's mask is the type's lowest value: a loss below one, not infinity."""
    rng = np.random.default_rng(8)
    T, k = 0.5, 20
    z = logits(rng, 3, C, torch.float32)
    tv, ti, _ = teacher(rng, z.double().numpy(), k, T)
    for i in range(3):
        top = tv[i].max()
        tv[i, 10:] = top - 46.0 - np.arange(10) * 0.1   # e^-92 and less
        z[i, ti[i, 10:]] = torch.finfo(torch.bfloat16).min
    z = z.to(TDT[dtype])
    loss, dz, bits, x = run_distill(dtype, z, tv, ti, T=T)
    wl, wd, _ = lo.distill(x, tv, ti, T=T)
    assert np.isfinite(wl).all() and (wl < 3).all()
    # weights of 1e-40 are multiples of 2^-149: 1e-5 of them, and of their share of the loss
    assert_within(loss, wl, 1e-4 * (1 + wl), "loss")
    assert_within(dz, wd, HALF[dtype] * np.abs(wd) + 1e-5, "dz")


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("T", [1.0, 2.0, 0.5])
def test_distill_of_every_width(dtype, T):
    rng = np.random.default_rng(7)
    for B, C, k in ((3, 256, 256), (2, 300, 129), (160, 1500, 128), (3, 24567, 32), (2, 24570, 33), (2, 51200, 1), (2, 131073, 17)):
        z = logits(rng, B, C, TDT[dtype])
        tv, ti, tl = teacher(rng, z.double().numpy(), k, T)
        check_distill(dtype, z, tv, ti, tl, ti[:, 0], None, T, 0.5, 0.5 * T * T, 1.0 / B)


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("W", [1, 2, 3, 7, 8, 9, 16, 31, 32])
def test_select_of_every_beam_count(dtype, W):
    rng = np.random.default_rng([8, W])
    for batch, C, m in ((1, 700, W), (3, 1234, min(64, 2 * W)), (2, 70000, W), (30, 64, 64), (2, 200001, min(64, W + 3))):
        done = (rng.uniform(size=(batch, W)) < 0.2).astype(np.uint8)
        check_select(dtype, logits(rng, batch * W, C, TDT[dtype]), scores_of(rng, batch, W), m, done, 3)


def test_on_a_stream_of_its_own_and_captured_twice():
    """A captured selection on a side stream, replayed with new logits in place."""
    rng = np.random.default_rng(9)
    batch, W, C, m = 3, 4, 5000, 8
    z = [logits(rng, batch * W, C, torch.bfloat16).to(DEV) for _ in range(3)]
    s0 = torch.from_numpy(scores_of(rng, batch, W)).to(DEV)
    buf = z[0].clone()
    outs = [torch.zeros(batch, m, device=DEV)] + [torch.zeros(batch, m, dtype=torch.int32, device=DEV) for _ in range(2)]
    n = nn.mlp_op_beam_select_workspace_bytes(H, batch, W, C, m)
    ws = [torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2)]

    def call(w):
        nn.mlp_op_beam_select(H, batch, W, C, m, buf.data_ptr(), C, s0.data_ptr(), None, -1, outs[0].data_ptr(),
                              outs[1].data_ptr(), outs[2].data_ptr(), None, w.data_ptr(), n, stream())

    side = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for w in ws:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call(w)
        graphs.append(g)
    for x in z[1:]:
        buf.copy_(x)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for b in range(batch):
            wt, wp, wc, _ = lo.beam_select(x[b * W:(b + 1) * W].double().cpu().numpy(), s0[b].cpu().numpy(), m)
            assert np.array_equal(outs[1][b].cpu().numpy(), wp) and np.array_equal(outs[2][b].cpu().numpy(), wc)
