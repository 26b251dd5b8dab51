"""Pins of the MXFP4 oracle: the E2M1 grid, round to nearest even at every
midpoint, saturation, block exponents, NaN blocks, the packed layout and a
brute-force layer."""

import numpy as np
import pytest

from oracle import mxfp4 as o4


def test_e2m1_grid():
    assert list(o4.e2m1_decode(np.arange(8))) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert np.array_equal(o4.e2m1_decode(np.arange(8, 16)), -o4.e2m1_decode(np.arange(8)))
    assert np.array_equal(o4.e2m1_encode(o4.e2m1_decode(np.arange(16))), np.arange(16))  # -0 keeps its sign


def test_e2m1_midpoints_go_to_the_even_code():
    grid = o4.e2m1_decode(np.arange(8))
    for c in range(7):
        mid = (grid[c] + grid[c + 1]) / 2
        even = c if c % 2 == 0 else c + 1
        assert o4.e2m1_encode(mid) == even and o4.e2m1_encode(-mid) == even + 8
        assert o4.e2m1_encode(np.nextafter(mid, 0)) == c
        assert o4.e2m1_encode(np.nextafter(mid, 9)) == c + 1
    assert o4.e2m1_encode(7.9) == 7 and o4.e2m1_encode(-1e9) == 15


@pytest.mark.parametrize("amax,e", [(6.0, 0), (4.0, 0), (7.99, 0), (8.0, 1), (3.99, -1), (2.0 ** -125, -127),
                                    (2.0 ** -130, -127), (2.0 ** 127, 125)])
def test_block_exponent(amax, e):
    x = np.zeros((1, 32))
    x[0, 7] = -amax
    codes, s = o4.mx_quantize(x)
    assert s[0, 0] == e + 127
    assert codes[0, 0] == 0


def test_blocks_without_a_value_and_with_none_finite():
    x = np.zeros((3, 64))
    x[1, 40] = np.nan
    x[2, 3] = np.inf
    codes, s = o4.mx_quantize(x)
    assert (codes == 0).all()
    assert s.tolist() == [[0, 0], [0, 255], [255, 0]]
    v = o4.mx_dequantize(codes, s)
    assert np.isnan(v[1, 32:]).all() and np.isnan(v[2, :32]).all() and (v[0] == 0).all()


def test_error_bound():
    """Half a step below 6 (relative 1/4 of the value or 1/4 of the unit), a quarter above by saturation."""
    x = np.random.default_rng(0).standard_normal((64, 128))
    codes, s = o4.mx_quantize(x)
    unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, 1)
    err = np.abs(o4.mx_dequantize(codes, s) - x)
    assert (err <= np.where(np.abs(x) > 6 * unit, 2 * unit, np.maximum(np.abs(x) / 5, unit / 4)) + 1e-15).all()


def test_pack_low_nibble_first():
    assert o4.pack(np.array([[1, 2, 3, 15]], dtype=np.uint8)).tolist() == [[0x21, 0xF3]]


def test_layer_brute_force():
    rng = np.random.default_rng(1)
    x, W, A, B = rng.standard_normal((3, 64)), rng.standard_normal((2, 64)), rng.standard_normal((4, 64)), \
        rng.standard_normal((2, 4))
    xq, wq = o4.quantized(x), o4.quantized(W)
    want = np.zeros((3, 2))
    for m in range(3):
        h = [sum(x[m, k] * A[r, k] for k in range(64)) for r in range(4)]
        for n in range(2):
            want[m, n] = sum(xq[m, k] * wq[n, k] for k in range(64)) + sum(h[r] * B[n, r] for r in range(4))
    assert np.allclose(o4.lora_linear_mxfp4(x, W, A, B), want, rtol=1e-13, atol=1e-13)
