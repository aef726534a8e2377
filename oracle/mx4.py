"""The 4-bit (MX) format and products of 4-bit operands, in fp64 (test infrastructure only).

Written from the OCP Microscaling definition (MXFP4): blocks of 32 values of a
row, elements E2M1 (1 sign, 2 exponent, 1 mantissa bit, bias 1: 0, 0.5, 1, 1.5,
2, 3, 4, 6), one E8M0 scale per block (2^(byte - 127), 255 = NaN).

Readings: the shared exponent is floor(log2 max|x|) - 2 (2 is the exponent of
the largest element), held at -127 from below; elements round to nearest, ties
to the even code, and magnitudes past 6 are held as 6; a block with a NaN or an
infinity is a NaN block with zero codes; the last block of a row is filled up
with zeros.
"""

from __future__ import annotations

import numpy as np

BLOCK = 32
# magnitudes of the codes 0 .. 7: exponent field e = code >> 1, mantissa bit m = code & 1
MAGNITUDES = np.array([(m / 2.0 if e == 0 else (1 + m / 2.0) * 2.0 ** (e - 1)) for e in range(4) for m in range(2)])


def _code_of(y):
    """Code of one non-negative magnitude already divided by its scale."""
    if y >= MAGNITUDES[7]:
        return 7
    lo = int(np.searchsorted(MAGNITUDES, y, side="right")) - 1
    down, up = y - MAGNITUDES[lo], MAGNITUDES[lo + 1] - y
    if down == up:
        return lo if lo % 2 == 0 else lo + 1
    return lo if down < up else lo + 1


def quantize(x):
    """x [rows, cols] (fp64 values of a 16-bit type) -> (element codes uint8 [rows, 32 nb], scale bytes uint8 [rows, nb])."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    full = np.zeros((rows, nb * BLOCK))
    full[:, :cols] = x
    codes = np.zeros((rows, nb * BLOCK), np.uint8)
    scales = np.zeros((rows, nb), np.uint8)
    for r in range(rows):
        for b in range(nb):
            v = full[r, b * BLOCK:(b + 1) * BLOCK]
            if not np.all(np.isfinite(v)):
                scales[r, b] = 255
                continue
            top = np.max(np.abs(v))
            e = int(np.floor(np.log2(top))) - 2 if top > 0 else -127
            if top > 0:   # log2 in floating point: put right at the powers of two
                while 2.0 ** (e + 2) > top:
                    e -= 1
                while 2.0 ** (e + 3) <= top:
                    e += 1
            e = max(e, -127)
            scales[r, b] = e + 127
            codes[r, b * BLOCK:(b + 1) * BLOCK] = [_code_of(abs(t) / 2.0 ** e) | (8 if np.signbit(t) else 0) for t in v]
    return codes, scales


def pack(codes, scales):
    """Element codes and scale bytes in the library's layout: codes [rows, 16 nb], scales [ceil(nb / 8), rows, 8]."""
    rows, nb = scales.shape
    panels = -(-nb // 8)
    out = np.zeros((panels, rows, 8), np.uint8)
    for b in range(nb):
        out[b // 8, :, b % 8] = scales[:, b]
    return codes[:, 0::2] | (codes[:, 1::2] << 4), out


def unpack(packed, panels):
    """The inverse of ``pack``."""
    rows, nb = packed.shape[0], packed.shape[1] // 16
    codes = np.zeros((rows, nb * BLOCK), np.uint8)
    codes[:, 0::2] = packed & 15
    codes[:, 1::2] = packed >> 4
    return codes, np.stack([panels[b // 8, :, b % 8] for b in range(nb)], axis=1) if nb else np.zeros((rows, 0), np.uint8)


def values(codes, scales):
    """What element codes and scale bytes stand for, fp64 [rows, 32 nb]."""
    v = MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, BLOCK, axis=1)


def gemm(a, b, ends=None):
    """A [M, K] . B_p^T in fp64; b [problems, N, K]; problem p multiplies rows ends[p-1] .. ends[p] - 1 (default: all)."""
    ends = [a.shape[0]] if ends is None else ends
    out = np.full((a.shape[0], b.shape[1]), np.nan)
    begin = 0
    for p, end in enumerate(ends):
        out[begin:end] = a[begin:end] @ b[p].T
        begin = end
    return out
