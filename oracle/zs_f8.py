"""CPU oracle of the block-scaled 8-bit matrices, their products and the reduce's norm.

TEST INFRASTRUCTURE ONLY, as zs_oracle: plain numpy in float64, written from the
definitions in the library's header as numbers with exponents and mantissas. The codes
are the public e4m3 and e5m2; the blocks of 128 under a power of two are this library's
own (parity unpinned), pinned by brute force over every code.
"""
from __future__ import annotations

import numpy as np

F32, F64 = np.float32, np.float64
E4M3, E5M2 = 3, 4
MANT = {E4M3: 3, E5M2: 2}
BIAS = {E4M3: 7, E5M2: 15}
TOP = {E4M3: 8, E5M2: 15}       # the largest code is 1.75 * 2^TOP
BLOCK = 128


def ceil(a: int, b: int) -> int:
    return -(-a // b)


def code_values(kind: int) -> np.ndarray:
    """The 256 codes' values."""
    c = np.arange(256)
    m, bias = MANT[kind], BIAS[kind]
    field, part = (c & 127) >> m, (c & ((1 << m) - 1)) / (1 << m)
    v = np.where(field > 0, np.ldexp(1 + part, field - bias), np.ldexp(part, 1 - bias))
    if kind == E4M3:
        v = np.where((c & 127) == 127, np.nan, v)
    else:
        v = np.where((c & 127) > 124, np.nan, np.where((c & 127) == 124, np.inf, v))
    return np.where(c > 127, -v, v)


def block_scales(x, kind: int, block_rows: int) -> np.ndarray:
    """[ceil(rows / block_rows), ceil(cols / 128)] scale bytes: the smallest s >= 1 with
    the largest magnitude at most 1.75 * 2^(TOP + s - 127), 255 if it is not finite."""
    rows, cols = x.shape
    R, C = ceil(rows, block_rows), ceil(cols, BLOCK)
    a = np.zeros((R * block_rows, C * BLOCK))
    with np.errstate(invalid="ignore"):
        a[:rows, :cols] = np.abs(x.astype(F64))
    top = a.reshape(R, block_rows, C, BLOCK).max(axis=(1, 3))
    bad = ~np.isfinite(top)
    part, e = np.frexp(np.where(bad | (top == 0), 1.0, top) / 1.75)
    s = np.where(top == 0, 1, e - (part == 0.5) - TOP[kind] + 127)
    return np.where(bad, 255, np.maximum(s, 1)).astype(np.uint8)


def quantize(x, kind: int = E4M3, block_rows: int = 1):
    """(codes [rows, ld], scales [ceil(rows / block_rows), lds]) of a float32 matrix."""
    x = np.asarray(x, F32)
    rows, cols = x.shape
    s = block_scales(x, kind, block_rows)
    per = np.repeat(np.repeat(s.astype(np.int64), block_rows, 0)[:rows], BLOCK, 1)[:, :cols]
    with np.errstate(invalid="ignore"):
        y = np.where(per == 255, 0.0, np.abs(x.astype(F64)) * np.ldexp(1.0, 127 - np.where(per == 255, 127, per)))
    e = np.maximum(np.where(y > 0, np.frexp(y)[1] - 1, -200), 1 - BIAS[kind])
    q = np.rint(y / np.ldexp(1.0, e - MANT[kind])) * np.ldexp(1.0, e - MANT[kind])
    grid = code_values(kind)[: 127 if kind == E4M3 else 124]
    code = np.searchsorted(grid, q)
    assert np.array_equal(grid[code], q)
    code = np.where(per == 255, 0, code | (np.signbit(x) << 7))
    codes = np.zeros((rows, ceil(cols, BLOCK) * BLOCK), np.uint8)
    codes[:, :cols] = code
    scales = np.ones((s.shape[0], ceil(cols, 4 * BLOCK) * 4), np.uint8)
    scales[:, : s.shape[1]] = s
    return codes, scales


def values(codes, scales, rows: int, cols: int, kind: int = E4M3, block_rows: int = 1) -> np.ndarray:
    """What codes stand for, in float64."""
    s = np.repeat(np.repeat(scales.astype(np.int64), block_rows, 0)[:rows], BLOCK, 1)[:, :cols]
    v = code_values(kind)[codes[:, :cols]] * np.ldexp(1.0, s - 127)
    return np.where(s == 255, np.nan, v)


def quantized(x, kind: int = E4M3, block_rows: int = 1) -> np.ndarray:
    """Values of the 8-bit form of x, in float64."""
    x = np.asarray(x, F32)
    c, s = quantize(x, kind, block_rows)
    return values(c, s, x.shape[0], x.shape[1], kind, block_rows)


def product(a, b):
    """(a b^T, its terms' magnitudes' sums, the sums over groups of 8 along K of the largest
    term's magnitude), for values a [M, K], b [N, K] in float64."""
    M, K = a.shape
    N = b.shape[0]
    exact, mags, tops = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    for k in range(0, K, 8):
        t = a[:, None, k:k + 8] * b[None, :, k:k + 8]
        exact += t.sum(axis=2)
        t = np.abs(t)
        mags += t.sum(axis=2)
        tops += t.max(axis=2)
    return exact, mags, tops


def sum_of_squares(gs) -> float:
    """Of several float32 arrays: exact products, the float64 sum correctly rounded."""
    import math
    return math.fsum(float(v) for g in gs for v in np.asarray(g, F64).ravel() ** 2)
