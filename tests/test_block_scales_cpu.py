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
