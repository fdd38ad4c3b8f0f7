"""CPU oracle of the 8-bit moments, the microscaled 4-bit shards and the gradient norm.

TEST INFRASTRUCTURE ONLY, as zs_oracle: plain numpy, written from the definitions in
the library's header as numbers with exponents and mantissas in float64, not as bit
patterns, so that it shares nothing with the kernels' shifts. No outside source fixes
these formats' codes: parity unpinned; their values are pinned by brute force over
every code.
"""
from __future__ import annotations

import math
from typing import Sequence

import numpy as np

from . import zs_oracle as O

F32, F64 = np.float32, np.float64
M, V = 0, 1                 # kinds of 8-bit moments
BLOCK8, BLOCK4 = 256, 32
TOP = {M: 15, V: 31}        # exponent field of the largest code
MOST = {M: 127, V: 255}     # largest magnitude code
LEAST_SCALE = {M: 0, V: 11}


def _two(e):
    """2^e in float64, exact."""
    return np.ldexp(np.ones_like(np.asarray(e, F64)), np.asarray(e, np.int64))


def _per_element(scales, block, n):
    return np.repeat(np.asarray(scales, np.int64), block)[:n]


# ------------------------------------------------------------- 8-bit moments
def state8_values(codes, scales, kind: int) -> np.ndarray:
    """Values (float32) of codes: 3 bits of mantissa, then the exponent, subnormal
    at exponent 0, times 2^(s - K - 127); sign in bit 7 for m; NaN where s = 255."""
    c = np.asarray(codes, np.int64)
    s = _per_element(scales, BLOCK8, c.size)
    neg = (c > 127) if kind == M else np.zeros(c.shape, bool)
    mag = c & 127 if kind == M else c
    field, part = mag // 8, mag % 8
    x = np.where(field > 0, (1 + part / 8) * _two(field), part / 8 * 2.0)
    x = x * _two(s - TOP[kind] - 127)
    with np.errstate(over="ignore", under="ignore"):
        x = np.where(neg, -x, x).astype(F32)
    return np.where(s == 255, F32("nan"), x)


def state8_scales(x, kind: int) -> np.ndarray:
    """Smallest s for which a block's largest magnitude is at most the largest
    code's value 1.875 * 2^(s - 127); 255 if it is not finite. (For a magnitude that
    is subnormal in fp32, whose patterns all have exponent byte 0: 1 from 1.75 * 2^-127
    up.)"""
    x = np.abs(np.asarray(x, F32)).astype(F64)
    n = -(-x.size // BLOCK8)
    top = np.pad(x, (0, n * BLOCK8 - x.size)).reshape(n, BLOCK8).max(axis=1)
    bad = ~np.isfinite(top)
    part, e = np.frexp(np.where(bad, 1.0, top) / 1.875)
    s = np.where(top > 0, e + 127 - (part == 0.5), 0)
    s = np.where(top < 2.0**-126, top > 1.75 * 2.0**-127, s)
    s = np.clip(s, LEAST_SCALE[kind], 254)
    return np.where(bad, 255, s).astype(np.uint8)


def state8_encode(x, kind: int, rnd=None):
    """(codes, scales) of the float32 values x. rnd: one number in (0, 1) per
    element, the place at which its distance to the code below rounds up; None:
    to nearest, ties to the even code."""
    x = np.asarray(x, F32)
    scales = state8_scales(x, kind)
    s = _per_element(scales, BLOCK8, x.size)
    with np.errstate(invalid="ignore", over="ignore"):
        # a subnormal fp32 result of the scaling is rounded like any other
        y = np.abs((np.abs(x).astype(F64) * _two(TOP[kind] - np.where(s == 255, 0, s))).astype(F32))
    y = np.where(s == 255, 0, y).astype(F64)
    e = np.maximum(np.where(y > 0, np.frexp(y)[1] - 1, -126), -126)
    steps = y / _two(e - 3)                     # in eighths of the binade
    q = np.rint(steps) if rnd is None else np.floor(steps + np.asarray(rnd, F64))
    # the code of q eighths of binade e: q = 8..15 (16 is the next binade's 8),
    # q < 8 only in the subnormal range, where e = -126 is field 1's spacing
    c = np.minimum((e + 126) * 8 + q, MOST[kind]).astype(np.int64)
    if kind == M:
        c = np.where(np.signbit(x), c + 128, c)
    else:
        c = np.where(x > 0, np.maximum(c, 1), 0)
    return np.where(s == 255, 0, c).astype(np.uint8), scales


def _mix(x):
    x = x * np.uint64(0x6A09E667) & np.uint64(0xFFFFFFFF)
    x = x ^ (x >> np.uint64(15))
    x = x * np.uint64(0xBB67AE85) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def random_words(seed: int, tensor: int, n: int, first: int = 0) -> np.ndarray:
    """The 32 random bits of each of a tensor's n elements from `first` on."""
    u = np.uint64
    lo, hi = u(seed & 0xFFFFFFFF), u(seed >> 32)
    key = _mix(u((int(lo) + 0x9E3779B9 * (tensor + 1)) & 0xFFFFFFFF))
    key = _mix((key + hi) & u(0xFFFFFFFF))
    return _mix((np.arange(first, first + n, dtype=np.uint64) & u(0xFFFFFFFF)) ^ key)


def rounding_places(seed: int, tensor: int, n: int, first: int = 0):
    """rnd of state8_encode for m and for v."""
    r = random_words(seed, tensor, n, first)
    return (((r % 65536) * 16 + 8) / 2.0**20, ((r // 65536) * 16 + 8) / 2.0**20)


def adamw_step8(p, mc, ms, vc, vs, g, hp: O.AdamWHP, seed=None, tensor: int = 0, first: int = 0):
    """One AdamW step with 8-bit moments: the values of the codes, zs_oracle's fp32
    step, and the new moments encoded. Returns (p, mc, ms, vc, vs, w). `first`: the place
    in the tensor of the first element, a multiple of 256."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        p2, m1, v1, w = O.adamw_step(p, state8_values(mc, ms, M), state8_values(vc, vs, V), g, hp)
    rm, rv = (None, None) if seed is None else rounding_places(seed, tensor, len(m1), first)
    return (p2, *state8_encode(m1, M, rm), *state8_encode(v1, V, rv), w)


# ------------------------------------------------------------- the norm
def sumsq(grads: Sequence[np.ndarray]) -> float:
    """Sum of squares, correctly rounded (the products are exact in float64)."""
    return math.fsum(math.fsum((np.asarray(g, F64) ** 2).ravel()) for g in grads)


def clip_coef(total: float, max_norm: float):
    norm = math.sqrt(total)
    if math.isinf(max_norm):
        return F32(norm), F32(1)
    c = max_norm / (norm + 1e-6)
    return F32(norm), F32(1) if c >= 1 else F32(c)


# ------------------------------------------------------------- 4-bit shards
GRID4 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def mx4_values(codes, scales, S: int) -> np.ndarray:
    """float64 values of S elements (NaN where the scale byte is 255)."""
    b = np.asarray(codes, np.uint8)
    c = np.stack([b & 15, b >> 4], axis=1).reshape(-1)[:S].astype(np.int64)
    s = _per_element(scales, BLOCK4, S)
    x = np.where(c >= 8, -GRID4[c & 7], GRID4[c & 7]) * _two(s - 127)
    return np.where(s == 255, np.nan, x)


def mx4_quantize(x):
    """(codes, scales) of the float32 values x: the nearest of the grid, by its
    midpoints, ties to the even code."""
    x = np.asarray(x, F32)
    S, n = x.size, -(-x.size // BLOCK4)
    top = np.pad(np.abs(x), (0, n * BLOCK4 - S)).reshape(n, BLOCK4).max(axis=1).astype(F64)
    bad = ~np.isfinite(top)
    e = np.where(top > 0, np.frexp(np.where(bad, 1.0, top))[1] - 1, -200)
    scales = np.where(bad, 255, np.maximum(e - 2 + 127, 0)).astype(np.uint8)
    s = _per_element(scales, BLOCK4, S)
    with np.errstate(invalid="ignore"):
        a = np.abs(x).astype(F64) * _two(127 - np.where(s == 255, 127, s))
    mid = (GRID4[1:] + GRID4[:-1]) / 2
    k = np.searchsorted(mid, a, side="left")          # a tie: the code below
    odd = np.isin(a, mid) & (k % 2 == 1)              # which is odd: the one above
    c = np.minimum(k + odd, 7)
    c = np.where(np.signbit(x), c + 8, c)
    c = np.where(s == 255, 0, c)
    c = np.pad(c, (0, S % 2)).astype(np.uint8)
    return c[0::2] | (c[1::2] << 4), scales
