"""Pins of the 8-bit layer's and the block norms' oracle, from the definitions."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import block_oracle as bo


def test_e4m3_table_is_the_format():
    t = bo.e4m3_table()
    assert t[0x00] == 0 and t[0x01] == 2.0 ** -9 and t[0x08] == 2.0 ** -6
    assert t[0x38] == 1.0 and t[0x7E] == 448.0 and t[0xFE] == -448.0
    assert np.isnan(t[0x7F]) and np.isnan(t[0xFF])
    assert np.all(np.diff(t[:0x7F]) > 0)


def test_encode_takes_the_nearest_code_ties_to_even():
    t = bo.e4m3_table()
    codes = np.arange(0x7F)
    assert np.array_equal(bo.e4m3_encode(t[codes]), codes)
    assert np.array_equal(bo.e4m3_encode(-t[codes]), codes | 0x80)
    mid = (t[:0x7E] + t[1:0x7F]) / 2                      # exact in fp64
    even = np.where(codes[:-1] % 2 == 0, codes[:-1], codes[1:])
    assert np.array_equal(bo.e4m3_encode(mid), even)
    assert np.array_equal(bo.e4m3_encode(np.nextafter(mid, 0)), codes[:-1])
    assert np.array_equal(bo.e4m3_encode(np.nextafter(mid, 1e9)), codes[1:])


def test_scale_exponent_is_the_smallest_that_fits():
    rng = np.random.default_rng(0)
    a = np.concatenate([np.exp2(rng.uniform(-100, 127, 500)), 448 * np.exp2(np.arange(-90.0, 119)),
                        448 * np.exp2(np.arange(-90.0, 119)) * (1 + 2.0 ** -8)])
    for v, e in zip(a, bo.scale_exponent(a)):
        f, p = Fraction(float(v)), Fraction(2) ** int(e)
        assert f <= 448 * p and f > 448 * p / 2
    assert bo.scale_exponent(np.array([0.0, 2.0 ** -133, 448 * 2.0 ** -127])).tolist() == [0, -127, -127]


def test_quantize_blocks_and_storage():
    x = np.ones((3, 192))
    x[1, 128:] = 449.0
    x[2, :128] = 0.0
    x[2, 190] = np.inf
    codes, byte = bo.quantize(x)
    # 1 <= 448 * 2^-8 = 1.75, and 1 > 448 * 2^-9
    assert byte.tolist() == [[119, 119], [119, 128], [127, 255]]
    assert codes[0, 0] == bo.e4m3_encode(np.array(256.0)) and codes[2, 5] == 0
    st = bo.stored_scales(byte)
    assert st.shape == (1, 3, 4) and st[0, 1].tolist() == [119, 128, 127, 127]
    v = bo.values(codes, byte)
    assert v[0, 0] == 1.0 and v[2, 0] == 0.0 and np.isnan(v[2, 130])
    w = np.ones((130, 192))
    w[129, 0] = 1000.0
    codes, byte = bo.quantize_weight(w)
    assert byte.tolist() == [[119, 119], [129, 119]]
    assert bo.stored_weight_scales(byte)[1].tolist() == [129, 119, 127, 127]
    assert bo.values(codes, byte, 128)[127, 0] == 1.0 and bo.values(codes, byte, 128)[128, 0] == 1.0


def test_relative_error_of_a_quantised_value():
    """Half a step of 3 fraction bits is 2^-4 of the value; below the normal range 2^-10 of the scale."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 256)) * np.exp2(rng.integers(-12, 12, (50, 256)))
    codes, byte = bo.quantize(x)
    step = np.exp2(byte.astype(float) - 127).repeat(128, 1) * 2.0 ** -10
    assert np.all(np.abs(bo.values(codes, byte) - x) <= np.maximum(2.0 ** -4 * np.abs(x), step))


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_block_norm_formula(kind):
    rng = np.random.default_rng(2)
    x, y = rng.standard_normal((4, 16)), rng.standard_normal((4, 16))
    gate, scale, shift = rng.standard_normal((3, 2, 16))
    w, b = rng.standard_normal((2, 16))
    u, _, h, _ = bo.block_norm(x, y, gate, kind, w, b, 1e-3, 0.5, kind, b, w, scale, shift, 1e-2)
    for m in range(4):
        def norm(v, eps):
            c = v - (sum(v) / 16 if kind == "layer" else 0)
            return c / (sum(t * t for t in c) / 16 + eps) ** 0.5
        um = 0.5 * x[m] + gate[m // 2] * (norm(y[m], 1e-3) * w + b)
        assert np.allclose(u[m], um, rtol=1e-13, atol=1e-13)
        hm = (norm(um, 1e-2) * b + w) * (1 + scale[m // 2]) + shift[m // 2]
        assert np.allclose(h[m], hm, rtol=1e-12, atol=1e-12)
