"""4-bit quantisation of blocks whose scale byte is 0 to 3: their scale, some or all of
their elements, or the halves between codes are subnormal numbers. Every code under every
one of these scales, ties and the neighbours of ties, bit for bit against the oracle."""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
from gpu_util import check_bits, device, to_np
from oracle import zs_formats as F
from oracle import zs_oracle as O
from test_gpu_mx4 import quantize

SCALES = (0, 1, 2, 3)


def neighbours(x, dtype):
    """x, the numbers of the type next to it, and all of them negated, as fp32."""
    x = np.asarray(x, np.float32)
    if dtype == "bf16":
        h = O.bf16_round(x).astype(np.int64)
        assert np.array_equal(O.bf16_widen(h.astype(np.uint16)), x)     # exact in the type
        y = np.concatenate([O.bf16_widen(np.maximum(h + d, 0).astype(np.uint16)) for d in (-1, 0, 1)])
    else:
        y = np.concatenate([np.nextafter(x, np.float32(-1)), x, np.nextafter(x, np.float32(np.inf))])
        y = np.maximum(y, 0)
    return np.concatenate([y, -y])


def blocks(dtype):
    """fp32 values, 32 a block: beside each of several largest magnitudes that give each
    scale, the grid's values, the midpoints between them, their neighbours, random numbers
    of every exponent below, the smallest numbers of the type and zeros of both signs."""
    rng = np.random.default_rng(4)
    smallest = 2.0**-149 if dtype == "f32" else 2.0**-133
    out = []
    for s in SCALES:
        unit = 2.0 ** (s - 127)
        mid = (F.GRID4[1:] + F.GRID4[:-1]) / 2
        x = neighbours(np.concatenate([F.GRID4, mid, [7.0]]) * unit, dtype)
        x = np.concatenate([x, [0.0, -0.0, smallest, -smallest],
                            rng.choice([-1, 1], 400) * rng.uniform(1, 2, 400)
                            * 2.0 ** rng.uniform(-149, s - 124, 400)]).astype(np.float32)
        for top in (4.0, 5.0, 6.0, 7.0, 7.96875):
            y = rng.permutation(x[np.abs(x) < 8 * unit])
            y = np.append(y, np.zeros(-y.size % 31, np.float32)).reshape(-1, 31)
            out.append(np.insert(y, rng.integers(0, 31), top * unit * rng.choice([-1, 1]), axis=1))
    for k in range(-149 if dtype == "f32" else -133, -124):   # blocks far below scale 0's largest
        y = (rng.choice([-1, 1], 32) * rng.uniform(0, 1, 32) * 2.0**k).astype(np.float32)
        y[rng.integers(0, 32)] = 2.0**k
        out.append(y[None])
    x = np.concatenate(out)[rng.permutation(sum(len(b) for b in out))].ravel()
    return O.bf16_round(x) if dtype == "bf16" else x


def oracle(x):
    return F.mx4_quantize(O.bf16_widen(x) if x.dtype == np.uint16 else x)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_the_inputs_reach_every_code_of_every_scale(dtype):
    codes, scales = oracle(blocks(dtype))
    c = np.stack([codes & 15, codes >> 4], axis=1).reshape(-1, 32)
    for s in SCALES:
        assert set(np.unique(c[scales == s])) == set(range(16)), s


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_quantize_small_scales(dtype):
    """In whole tiles of the kernel, and the first 1 to 40 blocks with a short last one in
    its element-by-element end."""
    x = blocks(dtype)
    assert x.size > 2 * 4096                          # elements of a tile with bf16
    for n in (x.size, *range(33, 40 * 32, 31)):
        codes, scales = quantize(x[:n], device())
        wc, ws = oracle(x[:n])
        check_bits(to_np(scales), ws, f"scales of {n}")
        check_bits(to_np(codes), wc, f"codes of {n}")


@pytest.mark.gpu
def test_quantize_every_small_bf16_value():
    """Every bf16 pattern of exponent byte 0 to 5, both signs, beside largest magnitudes
    of exponent byte 0 to 6."""
    h = np.arange(6 << 7, dtype=np.uint16)
    h = np.concatenate([h, h | 0x8000])
    for e in range(7):
        b = np.zeros((h.size, 32), np.uint16)
        b[:, 5] = h
        b[:, 30] = (e << 7) | 0x55
        codes, scales = quantize(b.ravel(), device())
        wc, ws = oracle(b.ravel())
        check_bits(to_np(scales), ws, f"scales, exponent byte {e}")
        check_bits(to_np(codes), wc, f"codes, exponent byte {e}")
