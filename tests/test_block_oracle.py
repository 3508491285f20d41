"""The block oracle pinned: gradients against central differences, layer norm
against its invariants, e4m3 against its definition."""
import numpy as np
import pytest

from oracle import block_oracle as bo


def _diff(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_layer_norm_gradients_against_differences():
    rng = np.random.default_rng(1)
    x, gamma, beta = rng.normal(size=(5, 17)) * 3 + 1, rng.normal(size=17), rng.normal(size=17)
    dy = rng.normal(size=x.shape)
    _, mean, rstd = bo.layer_norm(x, gamma, beta)
    dx, dg, db = bo.layer_norm_vjp(dy, x, mean, rstd, gamma)
    for v, grad, f in ((x, dx, lambda t: (bo.layer_norm(t, gamma, beta)[0] * dy).sum()),
                       (gamma, dg, lambda t: (bo.layer_norm(x, t, beta)[0] * dy).sum()),
                       (beta, db, lambda t: (bo.layer_norm(x, gamma, t)[0] * dy).sum())):
        d = rng.normal(size=v.shape)
        # central differences: truncation h^2 = 1e-12, cancellation 2^-53 / h ~ 1e-10, values of order 10
        assert abs(_diff(f, v, d) - (grad * d).sum()) < 1e-7


def test_layer_norm_rows_have_mean_zero_and_unit_variance():
    x = np.random.default_rng(2).normal(size=(4, 33)) * 7 - 2
    y, _, _ = bo.layer_norm(x, eps=0.0)
    assert np.abs(y.mean(axis=1)).max() < 1e-14 and np.abs((y * y).mean(axis=1) - 1).max() < 1e-13


@pytest.mark.parametrize("kind", [bo.ACT_NONE, bo.ACT_RELU, bo.ACT_GELU_TANH, bo.ACT_SILU])
def test_gated_gradients_against_differences(kind):
    rng = np.random.default_rng(3 + kind)
    s, dh = rng.normal(size=(4, 22)), rng.normal(size=(4, 11))
    ds, h = bo.gated_vjp(dh, s, kind)
    f = lambda t: (bo.act(t[:, :11], kind) * t[:, 11:] * dh).sum()   # noqa: E731
    d = rng.normal(size=s.shape)
    assert abs(_diff(f, s, d) - (ds * d).sum()) < 1e-7
    assert np.array_equal(h, bo.act(s[:, :11], kind) * s[:, 11:])


def test_activations_are_the_textbook_ones():
    g = np.linspace(-5, 5, 101)
    gelu = 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
    assert np.abs(bo.act(g, bo.ACT_GELU_TANH) - gelu).max() < 1e-14
    assert np.abs(bo.act(g, bo.ACT_SILU) - g / (1 + np.exp(-g))).max() < 1e-14
    # far down the left tail: g e^{2c}, to first order in e^{2c} = 1e-17
    c = np.sqrt(2 / np.pi) * (-6.5 - 0.044715 * 6.5 ** 3)
    assert abs(bo.act(np.float64(-6.5), bo.ACT_GELU_TANH) / (-6.5 * np.exp(2 * c)) - 1) < 1e-13


def test_gated_linear_is_two_projections():
    rng = np.random.default_rng(9)
    x, w, b = rng.normal(size=(3, 5)), rng.normal(size=(8, 5)), rng.normal(size=8)
    h, s = bo.gated_linear(x, w, b, bo.ACT_NONE)
    assert np.allclose(h, (x @ w[:4].T + b[:4]) * (x @ w[4:].T + b[4:]), rtol=1e-14)
    assert s.shape == (3, 8)


def test_e4m3_codes():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)[None]
    e = np.full((1, 8), 127, np.uint8)
    want = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(bo.q8_decode(codes, e), want, equal_nan=True)
    # a code's own value encodes to it (the block's largest, 448, fixes the scale at 2^0)
    v = np.concatenate([bo.q8_decode(codes, e)[0][:127].repeat(1)])[:, None]
    x = np.concatenate([v, np.full((127, 1), 448.0)], axis=1)
    q, sc = bo.q8_encode(x)
    assert np.array_equal(q[:, 0], np.arange(127)) and np.all(sc == 127)


def test_8_bit_error_and_ties():
    rng = np.random.default_rng(5)
    x = rng.normal(size=(8, 70)) * np.exp(rng.normal(size=(8, 70)) * 3)
    q, e = bo.q8_encode(x)
    y = bo.q8_decode(q, e)
    k = np.repeat(e.astype(int) - 127, 32, axis=1)[:, :70].astype(float)
    assert np.all(np.abs(y - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (k - 10)))
    # halfway between 1 and 1.125 goes to the even code (1), between 1.125 and 1.25 to 1.25
    t = np.array([[448.0, 1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10]])
    assert np.array_equal(bo.q8_decode(*bo.q8_encode(t))[0], [448.0, 1.0, 1.25, -1.0, 0.0, 2.0 ** -8])


def test_8_bit_extremes():
    x = np.zeros((4, 33))
    x[1, 0] = 2.0 ** -149
    x[2, :3] = [np.inf, np.nan, 3.0]
    x[3, 32] = 2.0 ** 127
    q, e = bo.q8_encode(x)
    y = bo.q8_decode(q, e)
    assert np.all(y[0] == 0) and np.all(e[0] == 7) and y[1, 0] == 0
    assert np.isnan(y[2, 0]) and np.isnan(y[2, 1]) and y[2, 2] == 3.0
    assert y[3, 32] == 2.0 ** 127
