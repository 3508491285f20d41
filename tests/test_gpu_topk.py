"""The k largest entries of a row with its log-sums, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import logits_oracle as lo
from tests.block_util import DEV, TDT, assert_within, stream
from tests.logits_util import logits, lse_tol, run_topk

pytestmark = pytest.mark.gpu

F, H = nn.F32, nn.BF16


def check(dtype, z, k, T=1.0, **kw):
    v, i, l, r, x = run_topk(dtype, z, k, T, **kw)
    wv, wi, wl, wr = lo.topk(x, k, T)
    assert np.array_equal(i, wi)
    assert np.array_equal(v, wv, equal_nan=True)
    taken = np.zeros(x.shape, bool)
    np.put_along_axis(taken, wi, True, 1)
    # the smallest normal term that fp32 keeps is 2^-126 of the reference: less is as good as nothing
    if kw.get("lse", True):
        assert_within(np.exp(l - wl), np.ones_like(l), np.maximum(lse_tol(x / T, np.ones_like(taken)), 1e-7), "lse")
    if kw.get("tail", True):
        none = wr == -np.inf
        assert (r[none] == -np.inf).all()
        assert_within(r[~none], wr[~none], lse_tol(x / T, ~taken)[~none], "tail")


# dtype, B, C, k, T, pitch beyond C, offset in elements
@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("B,C,k,T,pad,off", [
    (1, 1, 1, 1.0, 0, 0), (3, 2, 2, 1.0, 1, 1), (5, 7, 3, 2.0, 0, 0), (2, 8, 8, 1.0, 0, 0), (4, 33, 1, 0.7, 0, 3),
    (3, 100, 99, 1.0, 4, 0), (6, 255, 17, 1.0, 0, 1), (2, 256, 256, 1.0, 0, 0), (7, 1000, 50, 3.0, 0, 0),
    (3, 1001, 5, 1.0, 0, 5), (300, 1003, 31, 1.0, 2, 7), (9, 4096, 129, 1.0, 0, 0), (2, 8191, 64, 0.5, 1, 0),
    (700, 2000, 256, 1.0, 0, 0), (5, 12345, 33, 1.0, 0, 2), (1, 32000, 50, 1.0, 0, 0), (400, 32000, 64, 2.0, 0, 0),
    (310, 32001, 200, 1.0, 0, 0), (3, 50001, 100, 1.0, 7, 1)])
def test_against_the_oracle(dtype, B, C, k, T, pad, off):
    check(dtype, logits(np.random.default_rng([1, B, C, k]), B, C, TDT[dtype]), k, T, pad=pad, off=off)


@pytest.mark.parametrize("dtype,B,C,k", [(F, 2, 384000, 256), (H, 2, 384000, 256), (H, 160, 100003, 40), (F, 90, 140001, 7),
                                         (H, 1, 262144, 1)])
def test_wide_rows(dtype, B, C, k):
    check(dtype, logits(np.random.default_rng([2, C, k]), B, C, TDT[dtype]), k, 1.0)


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("B", [2, 400])
@pytest.mark.parametrize("kind", ["constant", "two_values", "rising", "falling", "few_left", "lowest", "one_left",
                                  "all_masked", "one_thread", "zeros"])
def test_rows_in_order_with_equals_and_masks(dtype, B, kind):
    """Rows that leave the threshold too many or too few candidates."""
    rng = np.random.default_rng(3)
    C = 20003
    z = logits(rng, B, C, torch.float32)
    if kind == "constant":
        z[:] = -3.25
    elif kind == "two_values":
        z = torch.from_numpy((rng.uniform(size=(B, C)) < 0.5).astype(np.float32))
    elif kind == "rising":
        z = torch.linspace(-30, 30, C).repeat(B, 1)
    elif kind == "falling":
        z = torch.linspace(30, -30, C).repeat(B, 1)
    elif kind == "few_left":
        z[:, torch.from_numpy(rng.permutation(C)[:C - 10])] = -np.inf
    elif kind == "lowest":
        z[:, torch.from_numpy(rng.permutation(C)[:C - 10])] = torch.finfo(TDT[dtype]).min
    elif kind == "one_left":
        z[:, 1:] = -np.inf
    elif kind == "all_masked":
        z[:] = -np.inf
    elif kind == "one_thread":   # the largest are all in a few threads' elements
        per = 16 // TDT[dtype].itemsize
        z[:, (torch.arange(C) // per) % 128 == 5] += 40
    else:
        z = torch.where(torch.from_numpy(rng.uniform(size=(B, C)) < 0.5), torch.tensor(0.0), torch.tensor(-0.0))
    if kind == "all_masked":
        v, i, l, r, x = run_topk(dtype, z, 33)
        assert (v == -np.inf).all() and (i == np.arange(33)).all() and (l == -np.inf).all() and (r == -np.inf).all()
        return
    check(dtype, z.to(TDT[dtype]), 33)


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("B,C,k,T", [(3, 3000, 1, 1.0), (3, 32000, 8, 0.05), (2, 100000, 5, 1.0), (2, 300000, 3, 0.1)])
def test_a_tail_far_below_what_is_taken(dtype, B, C, k, T):
    """The tail is the log of its own sum, however far the k entries stand out."""
    rng = np.random.default_rng(8)
    z = logits(rng, B, C, TDT[dtype])
    for b in range(B):
        z[b, torch.from_numpy(rng.permutation(C)[:k])] += 200.0
    check(dtype, z, k, T)
    z[:, 5] = 500.0                                # and one of the tail above the others
    z[:, 6] = 505.0
    check(dtype, z, k + 1, T)


@pytest.mark.parametrize("dtype", [F, H])
def test_nan_is_last_and_reaches_the_sums(dtype):
    rng = np.random.default_rng(4)
    z = logits(rng, 6, 3001, TDT[dtype])
    z[0, 100] = float("nan")
    z[1, :] = float("nan")
    z[2, 20:] = float("nan")
    z[3, 7] = float("inf")
    z[4, 50:] = -float("inf")
    z[4, 60] = float("nan")
    v, i, l, r, x = run_topk(dtype, z, 64)
    wv, wi, wl, wr = lo.topk(x, 64, 1.0)
    assert np.array_equal(i, wi) and np.array_equal(v, wv, equal_nan=True)
    assert np.isnan(l[[0, 1, 2, 3, 4]]).all() and np.isfinite(l[5])
    assert np.isnan(r[[0, 1, 2, 4]]).all() and np.isfinite(r[[3, 5]]).all()


def test_each_row_is_the_same_whatever_is_beside_it():
    """Places, counts and sums do not depend on the grid, and twice gives the same bits."""
    z = logits(np.random.default_rng(5), 500, 9000, torch.bfloat16)
    a = run_topk(H, z, 40)
    b = run_topk(H, z, 40)
    assert all(np.array_equal(x, y) for x, y in zip(a[:4], b[:4]))


@pytest.mark.parametrize("lse,tail", [(False, False), (True, False), (False, True)])
def test_without_the_sums(lse, tail):
    z = logits(np.random.default_rng(6), 30, 5000, torch.bfloat16)
    check(H, z, 20, lse=lse, tail=tail)
    check(H, z[:2].repeat(1, 5), 20, lse=lse, tail=tail)


def test_rows_past_2_31_elements():
    C, ld, B = 4099, (1 << 30) + 8, 3
    flat = torch.empty(2 * ld + C, dtype=torch.bfloat16, device=DEV)
    z = logits(np.random.default_rng(7), B, C, torch.bfloat16)
    for b in range(B):
        flat[b * ld:b * ld + C] = z[b].to(DEV)
    v = torch.empty(B, 9, device=DEV)
    i = torch.empty(B, 9, dtype=torch.int32, device=DEV)
    nn.mlp_op_topk(H, B, C, 9, flat.data_ptr(), ld, 1.0, v.data_ptr(), 9, i.data_ptr(), 9, None, None, stream())
    wv, wi, _, _ = lo.topk(z.double().numpy(), 9, 1.0)
    assert np.array_equal(i.cpu().numpy(), wi) and np.array_equal(v.cpu().numpy(), wv)
