"""Pins of the microscaled 4-bit oracle against the format's definition: the
sixteen element values, ties to the even code, saturation, the group exponent
and the byte layout."""
import itertools
from fractions import Fraction

import numpy as np

from oracle import codec, mx4


def test_element_values_follow_the_bit_fields():
    """e2m1: (-1)^s 2^(E-1) (1 + m/2) for E > 0, (-1)^s m/2 for E = 0."""
    for c in range(16):
        s, E, m = c >> 3, (c >> 1) & 3, c & 1
        want = (-1) ** s * (Fraction(m, 2) if E == 0 else Fraction(2) ** (E - 1) * (1 + Fraction(m, 2)))
        got = mx4.values(np.full((1, 32), c, np.uint8), np.full((1, 1), 127, np.uint8))[0, 0]
        assert Fraction(float(got)) == want


def test_rounding_is_nearest_with_ties_to_even():
    """Against an exhaustive search in exact fractions over a fine grid of [0, 8)."""
    a = np.arange(0, 8, 1 / 64)
    rows = np.zeros((a.size, 32))
    rows[:, 0], rows[:, 1] = a, 4.0          # the 4.0 holds the group's exponent at 0
    rows[a >= 4, 1] = 0.0
    code, byte, _ = mx4.quantize_rows(rows)
    assert (byte == 127).all()
    mags = [Fraction(float(m)) for m in mx4.MAGNITUDES]
    for x, c in zip(a, code[:, 0]):
        d = [abs(Fraction(float(x)) - m) for m in mags]
        best = [k for k in range(8) if d[k] == min(d)]
        want = best[0] if len(best) == 1 else next(k for k in best if k % 2 == 0)
        assert c == want, x


def test_group_exponent_and_special_groups():
    rows = np.zeros((7, 32))
    rows[1, 3] = 2.0 ** -149                 # the smallest fp32 value
    rows[2, 3] = 3.4e38
    rows[3, 5] = np.nan
    rows[4, 5] = -np.inf
    rows[5, 0] = -7.99                       # saturates at 6
    rows[6, 0], rows[6, 1] = 8.0, -0.5
    code, byte, _ = mx4.quantize_rows(rows)
    assert byte[:, 0].tolist() == [0, 0, 127 + 125, 255, 255, 127, 128]
    assert (code[0] == 0).all() and (code[3] == 0).all() and (code[4] == 0).all()
    assert code[5, 0] == 15 and code[6, 0] == 6 and code[6, 1] == 8   # -0.25 ties to (negative) zero
    v = mx4.values(code, byte)
    assert np.isnan(v[3]).all() and np.isnan(v[4]).all() and v[5, 0] == -6.0


def test_scale_tiles_follow_the_stated_byte_order():
    M, G = 200, 6
    byte = (np.arange(M * G) % 251).astype(np.uint8).reshape(M, G)
    t = mx4.tile_scales(byte)
    assert t.size == 2 * 2 * 512
    for r, g in itertools.product(range(0, M, 7), range(G)):
        tile = (r // 128) * 2 + g // 4
        assert t[512 * tile + (r % 128 % 32) * 16 + (r % 128 // 32) * 4 + g % 4] == byte[r, g]
    assert t.sum(dtype=np.int64) == byte.sum(dtype=np.int64)


def test_product_is_invariant_under_the_preparation():
    """x . w = y_x . y_w for rows scaled and rotated alike (no rounding)."""
    rng = np.random.default_rng(0)
    W, X, s = rng.standard_normal((5, 128)), rng.standard_normal((3, 128)), np.exp(rng.standard_normal(128))
    Yw, Yx = mx4.prepare_rows(W, s, False, 64, 9), mx4.prepare_rows(X, s, True, 64, 9)
    assert np.allclose(Yx @ Yw.T, X @ W.T, rtol=1e-12, atol=1e-12)


def test_decode_undoes_the_preparation():
    rng = np.random.default_rng(1)
    W, s = rng.standard_normal((4, 96)), np.exp(rng.standard_normal(96)).astype(np.float32)
    code, byte, _ = mx4.quantize_rows(mx4.prepare_rows(W, s, False, 32, 3))
    D = mx4.decode(code, byte, s, False, 32, 3)
    assert np.allclose(mx4.prepare_rows(D, s, False, 32, 3), mx4.values(code, byte), atol=1e-12)
    assert (codec.sign_mask(3, 96) != 1).any()
    assert np.array_equal(mx4.unpack_codes(mx4.pack_codes(code)), code)
