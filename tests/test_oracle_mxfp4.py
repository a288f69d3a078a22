"""Pins of the oracle's MXFP4 quantiser: the scale rule against a search over all exponents,
codes against ml_dtypes' float4_e2m1fn conversion of v / 2^e, values on the grid, the half-step
bound, and non-finite blocks."""

import ml_dtypes
import numpy as np

from oracle import mxfp4 as mx
from oracle.nvfp4 import e2m1_decode, unpack_nibbles


def test_scale_rule_against_a_search():
    rng = np.random.default_rng(1)
    edge = np.concatenate([np.float32(6.0) * np.exp2(np.arange(-120, 120, 7)).astype(np.float32)])
    amax = np.concatenate([edge, np.nextafter(edge, np.float32(0)), np.nextafter(edge, np.float32(np.inf)),
                           np.exp2(rng.uniform(-126, 127, 500)).astype(np.float32),
                           np.float32([0.0, 1e-45, 1e-40, 3.4028235e38])])
    got = mx.scale_exponent(amax)
    exps = np.arange(-127, 128)
    fits = amax.astype(np.float64)[:, None] <= 6.0 * np.exp2(exps.astype(np.float64))
    np.testing.assert_array_equal(got, exps[fits.argmax(1)])


def test_codes_against_the_library_conversion():
    rng = np.random.default_rng(2)
    v = (rng.standard_normal((64, 256)) * np.exp2(rng.integers(-20, 20, (64, 1)))).astype(np.float32)
    packed, s = mx.quantize_mxfp4(v)
    scaled = v.reshape(64, 8, 32) / np.exp2(s.astype(np.float64) - 127)[..., None]
    ref = scaled.astype(np.float32).astype(ml_dtypes.float4_e2m1fn).astype(np.float64)
    np.testing.assert_array_equal(e2m1_decode(unpack_nibbles(packed)).reshape(ref.shape), ref)
    # at most half of the largest step (2, between 4 and 6) of the block's scale
    back = mx.dequantize_mxfp4(packed, s).reshape(64, 8, 32)
    assert (np.abs(back - v.reshape(64, 8, 32)) <= np.exp2(s.astype(np.float64) - 127)[..., None]).all()


def test_values_on_the_grid_come_back():
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    rng = np.random.default_rng(3)
    v = rng.choice(np.concatenate([grid, -grid]), (16, 64))
    v[:, ::32] = 6.0
    v *= np.exp2(rng.integers(-30, 30, (16, 1)))
    packed, s = mx.quantize_mxfp4(v)
    np.testing.assert_array_equal(mx.dequantize_mxfp4(packed, s), v)


def test_zero_and_non_finite_blocks():
    v = np.zeros((3, 32))
    v[1, 5], v[2, 7] = np.nan, np.inf
    packed, s = mx.quantize_mxfp4(v)
    assert s.tolist() == [[0], [255], [255]] and not packed.any()
    back = mx.dequantize_mxfp4(packed, s)
    assert (back[0] == 0).all() and np.isnan(back[1:]).all()
