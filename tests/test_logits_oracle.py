"""The fp64 definitions of the operations on logits, pinned to library functions, closed forms and differences."""
import numpy as np
import torch

from oracle import logits_oracle as lo


def test_topk_against_a_stable_sort():
    rng = np.random.default_rng(0)
    z = np.round(rng.normal(size=(20, 50)) * 2) / 2   # many equals
    v, i, l, tail = lo.topk(z, 7, 2.0)
    sv, si = torch.sort(torch.from_numpy(z), dim=1, descending=True, stable=True)
    assert np.array_equal(v, sv[:, :7].numpy()) and np.array_equal(i, si[:, :7].numpy())
    assert np.allclose(l, torch.logsumexp(torch.from_numpy(z) / 2, 1).numpy(), rtol=1e-14)
    assert np.allclose(tail, torch.logsumexp(sv[:, 7:] / 2, 1).numpy(), rtol=1e-14)
    assert np.allclose(np.exp(l), np.exp(tail) + np.exp(v / 2).sum(1))


def test_topk_orders_nan_last_and_takes_infinities():
    v, i, l, tail = lo.topk(np.array([[np.nan, -np.inf, 3.0, -np.inf, 3.0]]), 5, 1.0)
    assert i.tolist() == [[2, 4, 1, 3, 0]]
    v, i, l, tail = lo.topk(np.array([[1.0, 2.0]]), 2, 1.0)
    assert tail[0] == -np.inf and np.isclose(l[0], np.logaddexp(1, 2))


def test_distill_of_a_whole_vocabulary_is_the_divergence():
    rng = np.random.default_rng(1)
    z, t = rng.normal(size=(6, 9)), rng.normal(size=(6, 9))
    ti = np.stack([rng.permutation(9) for _ in range(6)])
    T = 2.0
    loss, dz, _ = lo.distill(z, np.take_along_axis(t, ti, 1), ti, T=T, b=T * T)
    zt = torch.from_numpy(z).requires_grad_()
    want = torch.nn.functional.kl_div(torch.log_softmax(zt / T, 1), torch.softmax(torch.from_numpy(t) / T, 1),
                                      reduction="none").sum(1) * T * T
    want.sum().backward()
    assert np.allclose(loss, want.detach().numpy(), rtol=1e-12) and np.allclose(dz, zt.grad.numpy(), atol=1e-13)


def test_distill_gradient_against_differences():
    rng = np.random.default_rng(2)
    B, C, k = 3, 11, 4
    z = rng.normal(size=(B, C))
    ti = np.stack([rng.permutation(C)[:k] for _ in range(B)])
    ti[1, 2:] = -1
    tv, tail = rng.normal(size=(B, k)), rng.normal(size=B)
    y, w = rng.integers(0, C, B), rng.uniform(0.5, 2, B)
    f = lambda z_: lo.distill(z_, tv, ti, tail, y, w, 1.7, 0.3, 1.9, 1.0)
    _, dz, _ = f(z)
    for i in range(B):
        for c in range(C):
            e = np.zeros_like(z)
            e[i, c] = 1e-5
            assert abs((f(z + e)[0].sum() - f(z - e)[0].sum()) / 2e-5 - dz[i, c]) < 1e-8


def test_distill_of_the_student_itself_is_zero():
    rng = np.random.default_rng(3)
    z = rng.normal(size=(4, 30)) * 3
    v, i, _, tail = lo.topk(z, 5, 2.0)
    loss, dz, _ = lo.distill(z, v, i, tail, T=2.0)
    assert np.abs(loss).max() < 1e-14 and np.abs(dz).max() < 1e-15


def test_distill_rows_that_do_not_count():
    z = np.full((3, 5), np.nan)
    z[2] = 1.0
    ti = np.array([[0, 9], [1, 1], [-1, -1]])
    loss, dz, bad = lo.distill(z, np.zeros((3, 2)), ti, weights=np.array([0.0, 1.0, 1.0]))
    assert not loss.any() and not dz.any() and bad.tolist() == [False, True, False]


def test_beam_select_against_a_sort_of_log_softmax():
    rng = np.random.default_rng(4)
    z, s = rng.normal(size=(3, 20)), np.array([-1.0, -1.5, -2.0])
    t, b, c, e = lo.beam_select(z, s, 8, done=[0, 1, 0], eos=4)
    lp = torch.log_softmax(torch.from_numpy(z), 1).numpy() + s[:, None]
    lp[1] = -np.inf
    lp[1, 4] = -1.5
    o = np.argsort(-lp.ravel(), kind="stable")[:8]
    assert np.array_equal(b, o // 20) and np.array_equal(c, o % 20) and np.allclose(t, lp.ravel()[o])
    assert np.array_equal(e, (b == 1) | (c == 4))


def test_beam_select_first_step_and_empty_rows():
    z = np.zeros((2, 3))
    t, b, c, _ = lo.beam_select(z, [0.0, -np.inf], 5)
    assert b.tolist() == [0, 0, 0, 1, 1] and c.tolist() == [0, 1, 2, 0, 1]
    assert np.allclose(t[:3], -np.log(3)) and (t[3:] == -np.inf).all()
    z[0] = np.nan
    z[1] = [-np.inf, 0.0, -np.inf]
    t, b, c, _ = lo.beam_select(z, [0.0, 0.0], 5)
    assert b.tolist() == [1, 1, 1, 0, 0] and c.tolist() == [1, 0, 2, 0, 1]
    assert t[0] == 0 and (t[1:3] == -np.inf).all() and np.isnan(t[3:]).all()
