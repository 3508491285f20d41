"""Distillation from a teacher's top logits, loss and gradient, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import neural_net_step_gb300 as nn
from oracle import logits_oracle as lo
from tests.block_util import DEV, HALF, TDT, U32, assert_within, stream
from tests.logits_util import distill_tol, logits, run_distill, teacher

pytestmark = pytest.mark.gpu

F, H = nn.F32, nn.BF16


def check(dtype, z, tv, ti, tail, labels, w, T, a, b, g, **kw):
    loss, dz, bits, x = run_distill(dtype, z, tv, ti, tail, labels, w, T, a, b, g, **kw)
    f32 = lambda v: None if v is None else np.asarray(v, np.float32)
    wl, wd, bad = lo.distill(x, f32(tv), np.asarray(ti), f32(tail), labels, f32(w), T, a, b, g)
    assert bits == (1 if bad.any() else 0)
    tl, td = distill_tol(x, f32(tv), np.where(bad[:, None], -1, np.asarray(ti)), None if tail is None else f32(tail),
                         None if labels is None else np.where(bad, 0, labels), w, T, a, b, g, wl, wd, HALF[dtype])
    assert_within(loss, wl, tl, "loss")
    if kw.get("grad", True):
        assert_within(dz, wd, td, "dz")
    return loss, dz


# B, C, k, T, tail, labels, weights, z pitch beyond C, offset, dz pitch beyond C, offset
SHAPES = [
    (1, 1, 1, 1.0, False, True, False, 0, 0, 0, 0), (2, 2, 1, 2.0, True, False, False, 1, 1, 1, 1),
    (3, 5, 5, 1.0, False, True, True, 0, 0, 0, 0), (4, 8, 3, 1.0, True, True, False, 0, 3, 0, 3),
    (3, 15, 4, 2.0, True, True, True, 1, 9, 1, 9), (5, 100, 7, 4.0, True, False, True, 0, 0, 4, 1),
    (3, 257, 20, 1.0, False, True, False, 7, 2, 7, 2), (2, 1000, 200, 0.7, True, True, False, 0, 0, 0, 0),
    (330, 1003, 31, 2.0, True, True, True, 0, 5, 0, 5), (4, 4096, 64, 1.0, True, False, False, 0, 0, 8, 0),
    (350, 2500, 16, 1.0, True, True, False, 3, 0, 3, 0), (2, 9999, 256, 3.0, True, True, True, 0, 1, 0, 2),
    (1, 32000, 64, 2.0, True, False, False, 0, 0, 0, 0), (330, 32000, 20, 2.0, True, True, True, 0, 0, 0, 0),
    (40, 50001, 100, 1.0, False, True, False, 0, 0, 0, 0), (2, 100002, 33, 2.0, True, True, False, 1, 6, 1, 6)]


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("B,C,k,T,tail,labels,weights,pad,off,dpad,doff", SHAPES)
def test_against_the_oracle(dtype, B, C, k, T, tail, labels, weights, pad, off, dpad, doff):
    rng = np.random.default_rng([1, B, C, k])
    z = logits(rng, B, C, TDT[dtype])
    tv, ti, tl = teacher(rng, z.double().numpy(), k, T)
    y = np.where(rng.uniform(size=B) < 0.5, ti[:, 0], rng.integers(0, C, B)) if labels else None
    w = rng.uniform(0.5, 2.0, B) * (rng.uniform(size=B) < 0.8) if weights else None
    w = None if w is None else w.astype(np.float32)
    check(dtype, z, tv, ti, tl if tail else None, y, w, T, 0.4 if labels else 0.0, 0.6 * T * T, 1.0 / B, pad=pad, off=off,
          dpad=dpad, doff=doff)


@pytest.mark.parametrize("dtype,C,k", [(F, 384000, 256), (H, 384000, 100)])
def test_widest_rows(dtype, C, k):
    rng = np.random.default_rng([2, C])
    z = logits(rng, 2, C, TDT[dtype])
    tv, ti, tl = teacher(rng, z.double().numpy(), k, 2.0)
    check(dtype, z, tv, ti, tl, ti[:, 3], None, 2.0, 0.5, 2.0, 0.5)


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("C", [777, 40000])
def test_loss_alone_and_in_place(dtype, C):
    rng = np.random.default_rng(3)
    z = logits(rng, 50, C, TDT[dtype])
    tv, ti, tl = teacher(rng, z.double().numpy(), 10, 2.0)
    y = rng.integers(0, C, 50)
    w = (rng.uniform(size=50) < 0.7).astype(np.float32)
    args = (dtype, z, tv, ti, tl, y, w, 2.0, 0.5, 2.0, 0.1)
    loss, dz = check(*args)
    alone, _ = check(*args, grad=False)
    there, dz2 = check(*args, in_place=True, pad=3, off=1, dpad=3, doff=1)
    assert np.array_equal(loss, alone)
    assert_within(there, loss, 1e-5 * np.abs(loss) + 1e-6, "in place")   # (another phase: another order of the sums)


@pytest.mark.parametrize("dtype", [F, H])
def test_rows_of_weight_zero_hold_anything(dtype):
    rng = np.random.default_rng(4)
    for C in (500, 33001):
        z = logits(rng, 8, C, TDT[dtype])
        tv, ti, tl = teacher(rng, z.double().numpy(), 6, 1.0)
        y = rng.integers(0, C, 8)
        w = np.ones(8, np.float32)
        w[[1, 4, 7]] = 0
        z[1] = float("nan")
        z[4] = float("inf")
        ti[7, :] = 1 << 30
        y[4] = -100
        tv[1] = np.nan
        tl[7] = np.nan
        loss, dz, bits, x = run_distill(dtype, z, tv, ti, tl, y, w, 1.0, 0.5, 0.5, 1.0)
        assert bits == 0 and not loss[[1, 4, 7]].any() and not dz[[1, 4, 7]].any()
        keep = [0, 2, 3, 5, 6]
        wl, wd, _ = lo.distill(x[keep], tv[keep], ti[keep], tl[keep], y[keep], None, 1.0, 0.5, 0.5, 1.0)
        t1, t2 = distill_tol(x[keep], tv[keep], ti[keep], tl[keep], y[keep], None, 1.0, 0.5, 0.5, 1.0, wl, wd, HALF[dtype])
        assert_within(loss[keep], wl, t1, "loss")
        assert_within(dz[keep], wd, t2, "dz")


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("C", [600, 60000])
def test_unused_entries_and_empty_teachers(dtype, C):
    rng = np.random.default_rng(5)
    z = logits(rng, 7, C, TDT[dtype])
    tv, ti, tl = teacher(rng, z.double().numpy(), 12, 2.0)
    ti[0, 5:] = -1
    ti[1, ::2] = -1          # anywhere in the row
    ti[2, :] = -1            # the tail alone
    ti[3, :] = -1
    tl[3] = -np.inf          # nothing at all
    tv[4, :] = -np.inf       # entries without weight: their columns stay out of the tail
    tv[5, 3] = -np.inf
    tv[ti == -1] = np.nan    # (not read)
    y = rng.integers(0, C, 7)
    w = None
    loss, dz, bits, x = run_distill(dtype, z, tv, ti, tl, y, w, 2.0, 0.25, 4.0, 1.0)
    tv0 = np.where(ti == -1, 0, tv)
    wl, wd, _ = lo.distill(x, tv0, ti, tl, y, w, 2.0, 0.25, 4.0, 1.0)
    t1, t2 = distill_tol(x, np.where(np.isinf(tv0), -1e30, tv0), ti, tl, y, w, 2.0, 0.25, 4.0, 1.0, wl, wd, HALF[dtype])
    # (an entry of -infinity has no size of its own in the bound)
    t1[[4, 5]] = 1e-5 * (1 + np.abs(wl[[4, 5]]))
    assert bits == 0
    assert_within(loss, wl, t1, "loss")
    assert_within(dz, wd, t2, "dz")


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("C", [400, 40000])
def test_bad_rows_set_the_error_bit_and_are_zero(dtype, C):
    rng = np.random.default_rng(6)
    for what in ("high", "low", "twice", "label", "label_low"):
        z = logits(rng, 5, C, TDT[dtype])
        tv, ti, tl = teacher(rng, z.double().numpy(), 9, 1.0)
        y = rng.integers(0, C, 5)
        if what == "high":
            ti[2, 4] = C
        elif what == "low":
            ti[2, 4] = -2
        elif what == "twice":
            ti[2, 4] = ti[2, 8]
        elif what == "label":
            y[2] = C
        else:
            y[2] = -1
        loss, dz, bits, x = run_distill(dtype, z, tv, ti, tl, y, None, 1.0, 0.5, 0.5, 1.0)
        assert bits == 1 and loss[2] == 0 and not dz[2].any() and (loss[[0, 1, 3, 4]] != 0).all()
        assert dz[[0, 1, 3, 4]].any(axis=1).all()
        # a label that carries no weight is not read
        if what.startswith("label"):
            assert run_distill(dtype, z, tv, ti, tl, y, None, 1.0, 0.0, 0.5, 1.0)[2] == 0


@pytest.mark.parametrize("dtype", [F, H])
def test_masked_columns(dtype):
    rng = np.random.default_rng(7)
    C = 3000
    z = logits(rng, 6, C, TDT[dtype])
    tv, ti, tl = teacher(rng, z.double().numpy(), 8, 2.0)
    for i in range(6):   # masked where the teacher gives no weight but in row 1 and 2
        z[i, torch.from_numpy(np.setdiff1d(rng.permutation(C)[:1000], ti[i]))] = -np.inf if i % 2 else torch.finfo(TDT[dtype]).min
    tl[5] = -np.inf
    z[5, torch.from_numpy(np.setdiff1d(np.arange(C), ti[5]))] = -np.inf   # nothing but the teacher's columns
    check(dtype, z, tv, ti, tl, ti[:, 1], None, 2.0, 0.5, 2.0, 1.0)
    # weight where the student has none: an infinite loss, a finite gradient
    z[0, ti[0, 2]] = -np.inf
    tl[1] = 0.0
    z[1, torch.from_numpy(np.setdiff1d(np.arange(C), ti[1]))] = -np.inf
    z[2, 5] = float("nan")
    z[3, 5] = float("inf")
    z[4, :] = -np.inf
    loss, dz, bits, x = run_distill(dtype, z, tv, ti, tl, None, None, 2.0, 0.0, 4.0, 1.0)
    assert bits == 0 and np.isposinf(loss[[0, 1]]).all() and np.isnan(loss[[2, 3, 4]]).all() and np.isfinite(loss[5])
    wl, wd, _ = lo.distill(x[[0, 1]], tv[[0, 1]], ti[[0, 1]], tl[[0, 1]], None, None, 2.0, 0.0, 4.0, 1.0)
    assert np.isposinf(wl).all()
    assert_within(dz[[0, 1]], wd, HALF[dtype] * np.abs(wd) + 1e-5, "dz")
    assert np.isnan(dz[2]).all() and np.isnan(dz[3]).any()


def test_a_student_near_its_teacher_has_a_small_exact_loss():
    rng = np.random.default_rng(8)
    z = logits(rng, 200, 20000, torch.float32, 3.0)
    x = z.double().numpy()
    v, i, _, tail = lo.topk(x + 1e-2 * rng.normal(size=x.shape), 50, 2.0)
    v, tail = v.astype(np.float32), tail.astype(np.float32)
    loss, dz, _, _ = run_distill(F, z, v, i, tail, T=2.0, b=4.0)
    wl, wd, _ = lo.distill(x, v, i, tail, T=2.0, b=4.0)
    # a loss of about 1e-4: the logarithms' errors are those of ratios near one
    assert np.abs(wl).max() < 1e-3
    assert_within(loss, wl, np.full(200, 4.0 * 4e-7), "loss")


def test_gradient_against_differences():
    """dz of the whole call in fp32 against central differences of its own loss (fp64 sums of fp32 losses)."""
    rng = np.random.default_rng(9)
    B, C, k = 2, 40, 6
    z = logits(rng, B, C, torch.float32)
    tv, ti, tl = teacher(rng, z.double().numpy(), k, 2.0)
    y, w = np.array([3, ti[1, 0]]), np.array([1.0, 0.5], np.float32)
    f = lambda q: run_distill(F, q, tv, ti, tl, y, w, 2.0, 0.5, 2.0, 1.0)
    _, dz, _, _ = f(z)
    h = 2.0 ** -5
    for c in range(C):
        e = torch.zeros(B, C)
        e[:, c] = h
        up, down = f(z + e)[0], f(z - e)[0]
        # the loss's own rounding (2e-6) over 2 h, and h^2 / 6 times a third derivative of at most 4
        assert np.abs((up - down) / (2 * h) - dz[:, c]).max() < 2 * 2e-6 / (2 * h) + h * h * 4 / 6


def test_rows_past_2_31_elements():
    C, ld, B, k = 4099, (1 << 30) + 8, 3, 5
    rng = np.random.default_rng(10)
    z = logits(rng, B, C, torch.bfloat16)
    tv, ti, tl = teacher(rng, z.double().numpy(), k, 1.0)
    flat = torch.zeros(2 * ld + C, dtype=torch.bfloat16, device=DEV)
    for b in range(B):
        flat[b * ld:b * ld + C] = z[b].to(DEV)
    t = [torch.from_numpy(a).to(DEV) for a in (tv, ti.astype(np.int32), tl)]
    loss = torch.empty(B, device=DEV)
    nn.mlp_op_distill(H, B, C, k, flat.data_ptr(), ld, t[0].data_ptr(), k, t[1].data_ptr(), k, t[2].data_ptr(), None, None,
                      1.0, 0.0, 1.0, 1.0, flat.data_ptr(), ld, loss.data_ptr(), None, stream())
    wl, wd, _ = lo.distill(z.double().numpy(), tv, ti, tl)
    got = np.stack([flat[b * ld:b * ld + C].double().cpu().numpy() for b in range(B)])
    assert_within(got, wd, HALF[H] * np.abs(wd) + 1e-5, "dz")
    assert_within(loss.cpu().numpy(), wl, 1e-5 * wl, "loss")


def test_twice_gives_the_same_bits():
    rng = np.random.default_rng(11)
    for C in (5000, 50000):
        z = logits(rng, 40, C, torch.bfloat16)
        tv, ti, tl = teacher(rng, z.double().numpy(), 30, 2.0)
        a, b = (run_distill(H, z, tv, ti, tl, ti[:, 0], None, 2.0, 0.5, 2.0, 1.0) for _ in range(2))
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
