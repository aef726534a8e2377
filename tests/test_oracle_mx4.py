"""Pins of the 4-bit format's oracle: hand-worked blocks, brute force, and an independent bit-level construction."""

import numpy as np
import pytest

from oracle import mx4
from oracle.numerics import decode_bits
from workloads import random_bits


def test_code_values():
    assert mx4.MAGNITUDES.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def test_hand_worked_block():
    """Largest magnitude 13 = 1.625 * 2^3: scale 2^(3 - 2) = 2, so values are halved and rounded."""
    x = np.zeros((1, 32))
    x[0, :12] = [13, -13, 1, 0.5, 0.25, -0.5, 2.5, 3.5, 5, 7, 10, -9.9]
    c, s = mx4.quantize(x)
    assert s.tolist() == [[128]]
    # halves: 6.5 -> 6 (held), .5, .25 -> 0 (tie to even), .125 -> 0, -.25 -> -0, 1.25 -> 1 (tie), 1.75 -> 2 (tie),
    # 2.5 -> 2 (tie), 3.5 -> 4 (tie), 5 -> 4 (tie), -4.95 -> -4
    assert c[0, :12].tolist() == [7, 15, 1, 0, 0, 8, 2, 4, 4, 6, 6, 14]
    assert mx4.values(c, s)[0, :12].tolist() == [12, -12, 1, 0, 0, 0, 2, 4, 4, 8, 8, -8]


def test_special_blocks():
    x = np.zeros((1, 5 * 32))
    x[0, 32] = 2.0 ** -133            # the scale is held at 2^-127: 2^-133 / 2^-127 = 2^-6 -> 0
    x[0, 64] = np.inf
    x[0, 96] = np.nan
    x[0, 128] = 2.0 ** -125           # 2^-127 exactly: 4 * 2^-127
    c, s = mx4.quantize(x)
    assert s.tolist() == [[0, 0, 255, 255, 0]]
    assert not c[0, :128].any() and c[0, 128] == 6
    v = mx4.values(c, s)
    assert np.isnan(v[0, 64:128]).all() and v[0, 128] == 2.0 ** -125 and not v[0, :64].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_element_is_the_nearest_value(dtype):
    """Against brute force: no other code is nearer, and the scale makes the largest magnitude's exponent 2."""
    x = decode_bits(random_bits(5, 40 * 64, dtype), dtype).reshape(40, 64)
    x[:20] = np.ldexp(np.round(x[:20] / np.abs(x[:20]).max(1, keepdims=True) * 64), -3)   # many ties
    c, s = mx4.quantize(x)
    v = mx4.values(c, s)
    scale = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    grid = np.concatenate([mx4.MAGNITUDES, -mx4.MAGNITUDES])
    best = np.min(np.abs(x[..., None] - scale[..., None] * grid), axis=-1)
    assert np.array_equal(np.abs(x - v), best)
    top = np.abs(x).reshape(40, 2, 32).max(-1)
    ok = top >= 2.0 ** -125
    assert np.array_equal(np.frexp(top)[1][ok] - 1 - 2 + 127, s.astype(int)[ok])


def test_pack_layout_and_round_trip():
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 16, (5, 9 * 32)).astype(np.uint8)
    scales = rng.integers(0, 256, (5, 9)).astype(np.uint8)
    p, q = mx4.pack(codes, scales)
    assert p.shape == (5, 144) and q.shape == (2, 5, 8)
    assert p[3, 20] == codes[3, 40] | codes[3, 41] << 4
    assert q[0, 2, 7] == scales[2, 7] and q[1, 2, 0] == scales[2, 8] and not q[1, :, 1:].any()
    c, s = mx4.unpack(p, q)
    assert np.array_equal(c, codes) and np.array_equal(s, scales)


def test_gemm_of_stacked_problems():
    rng = np.random.default_rng(4)
    a, b = rng.integers(-3, 4, (6, 32)).astype(float), rng.integers(-3, 4, (3, 8, 32)).astype(float)
    out = mx4.gemm(a, b, [2, 2, 5])
    for m, p in ((0, 0), (1, 0), (2, 2), (4, 2)):
        assert np.array_equal(out[m], [sum(a[m, k] * b[p, n, k] for k in range(32)) for n in range(8)])
    assert np.isnan(out[5]).all()
