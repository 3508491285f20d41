"""What scale bytes stand for at both ends of their range, and how far a
checkpoint may be off its values (fp64 oracle)."""
import numpy as np

from oracle import block_oracle as bo


def test_scale_255_is_nan():
    codes = np.arange(256, dtype=np.uint8)[None]
    assert np.isnan(bo.q8_decode(codes, np.full((1, 8), 255, np.uint8))).all()
    e = np.array([[255, 254, 0, 127, 255, 127, 127, 127]], np.uint8)
    v = bo.q8_decode(np.full((1, 256), 56, np.uint8), e)[0].reshape(8, 32)     # code 56: 1.0
    assert np.isnan(v[[0, 4]]).all() and np.all(v[1] == 2.0 ** 127) and np.all(v[2] == 2.0 ** -127) and np.all(v[3] == 1)


def test_error_bound_down_to_the_smallest_blocks():
    """At most 2^-4 of the value, or 2^(k - 10) where that is more; that is
    2^-17.8 of the block's largest unless k stays at -120 (2^-130 then)."""
    rng = np.random.default_rng(8)
    x = rng.normal(size=(400, 32)) * np.exp(rng.normal(size=(400, 32))) * 2.0 ** np.linspace(-148, 119, 400)[:, None]
    x = x.astype(np.float32).astype(np.float64)
    q, e = bo.q8_encode(x)
    off, k = np.abs(bo.q8_decode(q, e) - x), e.astype(float) - 127
    assert np.all(off <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (k - 10)))
    amax = np.abs(x).max(axis=1, keepdims=True)
    small = amax < 224 * 2.0 ** -120
    assert np.all(k[small] == -120) and small.any() and not small.all()
    floor = np.where(small, 2.0 ** -130, amax * 2.0 ** -10 / 224)
    assert np.all(off <= np.maximum(2.0 ** -4 * np.abs(x), floor))
    # (2^-17.8 of the largest alone would not hold for them)
    assert np.any((off > np.maximum(2.0 ** -4 * np.abs(x), amax * 2.0 ** -10 / 224))[small[:, 0]])
