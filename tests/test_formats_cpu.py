"""The oracle of the 8-bit moments and 4-bit shards, pinned by brute force over every
code, and the host side of the calls over many tensors: layout, refusals, aliasing (no
GPU: every refused call ends before anything is enqueued)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
from fsdp_sharded_optimizer_zs_amd import _binding as B
from oracle import zs_formats as F
from oracle import zs_oracle as O

KINDS = (F.M, F.V)
INF, NAN = float("inf"), float("nan")


def all_values(kind, s):
    codes = np.arange(256, dtype=np.uint8)
    return F.state8_values(codes, [s], kind).astype(np.float64)


# ------------------------------------------------------------------ 8 bits
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("s", (11, 60, 127, 200, 254))
def test_codes_are_an_ordered_grid(kind, s):
    x = all_values(kind, s)[:F.MOST[kind] + 1]
    assert x[0] == 0 and np.all(np.diff(x) > 0)
    assert x[-1] == 1.875 * 2.0 ** (s - 127)
    normal = x[8:]
    assert np.all(np.diff(normal) / normal[:-1] <= 1 / 8)        # 3 bits of mantissa
    if kind == F.M:
        neg = all_values(kind, s)[128:]
        assert np.array_equal(neg, -x)


@pytest.mark.parametrize("kind", KINDS)
def test_encode_takes_the_nearest_code(kind):
    rng = np.random.default_rng(1)
    for k in range(20):
        x = (rng.standard_normal(256) * 10.0 ** rng.uniform(-6, 0, 256)
             * 2.0 ** int(rng.integers(-60, 60))).astype(np.float32)
        x = x if kind == F.M else np.abs(x)
        codes, scales = F.state8_encode(x, kind)
        grid = all_values(kind, scales[0])
        grid = grid if kind == F.M else grid[1:]                 # a positive v is never 0
        best = np.abs(x[:, None].astype(np.float64) - grid[None]).min(axis=1)
        got = np.abs(x.astype(np.float64) - F.state8_values(codes, scales, kind))
        assert np.array_equal(got, best)
        assert np.abs(x).max() <= 1.875 * 2.0 ** (int(scales[0]) - 127)
        assert np.abs(x).max() > 1.875 * 2.0 ** (int(scales[0]) - 128)


@pytest.mark.parametrize("kind", KINDS)
def test_ties_go_to_the_even_code(kind):
    s = 100
    g = all_values(kind, s)[:F.MOST[kind] + 1]
    mid = ((g[1:] + g[:-1]) / 2).astype(np.float32)[-120:-1]
    x = np.concatenate([mid, [np.float32(g[-1])]])
    codes, scales = F.state8_encode(x, kind)
    assert scales[0] == s and np.all(codes[:-1] % 2 == 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("s", (11, 12, 40, 127, 254))
def test_encoding_decoded_codes_keeps_every_value(kind, s):
    rng = np.random.default_rng(s)
    codes = rng.integers(0, 256, 256).astype(np.uint8)
    x = F.state8_values(codes, [s], kind)
    again = F.state8_values(*F.state8_encode(x, kind), kind)
    assert np.array_equal(x.view(np.uint32), again.view(np.uint32))


@pytest.mark.parametrize("kind", KINDS)
def test_a_block_with_a_nan_or_infinity_is_nan(kind):
    x = np.ones(512, np.float32)
    for bad in (np.nan, np.inf):
        x[300] = bad
        codes, scales = F.state8_encode(x, kind)
        y = F.state8_values(codes, scales, kind)
        assert scales[1] == 255 and np.isnan(y[256:]).all() and (y[:256] == 1).all()


def test_zeros_and_the_largest_numbers():
    for kind in KINDS:
        codes, scales = F.state8_encode(np.zeros(256, np.float32), kind)
        assert not codes.any() and not F.state8_values(codes, scales, kind).any()
        assert not F.state8_values(np.zeros(9, np.uint8), [0], kind).any()   # zeroed buffers
        top = np.full(256, np.finfo(np.float32).max, np.float32)
        y = F.state8_values(*F.state8_encode(top, kind), kind)
        assert np.isfinite(y).all() and np.all(y == np.float32(1.875 * 2.0**127))
    tiny = np.full(256, 1e-45, np.float32)
    assert (F.state8_values(*F.state8_encode(tiny, F.V), F.V) > 0).all()


def test_stochastic_rounding_keeps_the_mean():
    """4096 elements of one value: the mean is a sum of independent two-point
    variables of step d, so its standard deviation is at most d / 2 / 64; six of
    them, plus half of 2^-16 of a step for the 16 random bits."""
    n = 4096
    for kind, value in ((F.M, 1.3), (F.V, 1.57), (F.V, 1.001), (F.M, -1.06)):
        x = np.full(n, value, np.float32)
        x[::256] = 1.75 * np.sign(value)                          # the block's largest
        rm, rv = F.rounding_places(12345, 3, n)
        y = F.state8_values(*F.state8_encode(x, kind, rm if kind == F.M else rv), kind)
        keep = np.arange(n) % 256 != 0
        assert set(np.unique(y[keep])) <= {np.float32(np.floor(value * 8) / 8),
                                           np.float32(np.ceil(value * 8) / 8)}
        d = 0.125
        assert abs(y[keep].mean(dtype=np.float64) - np.float32(value)) <= 6 * d / 2 / 64 + d * 2**-17


def test_random_words_are_uniform_and_differ():
    """Each of 32 bits over 2^16 elements: mean 1/2 within 6 standard deviations
    (1/2 / 256); words of other seeds, tensors and the high seed half differ."""
    n = 1 << 16
    base = F.random_words(7, 0, n)
    bits = (base[:, None] >> np.arange(32, dtype=np.uint64)) & np.uint64(1)
    assert np.abs(bits.mean(axis=0) - 0.5).max() <= 6 * 0.5 / 256
    pairs = np.corrcoef(bits[:-1].T.astype(float), bits[1:].T.astype(float))[:32, 32:]
    assert np.abs(pairs).max() <= 6 / 256
    for other in (F.random_words(8, 0, n), F.random_words(7, 1, n), F.random_words(7 + 2**40, 0, n)):
        assert (base == other).mean() < 1e-3


def test_slow_second_moments_move_only_when_rounded_stochastically():
    """What the stochastic mode is for: with beta2 = 0.999 and no gradient, v shrinks
    by a thousandth a step. To nearest it never moves; stochastically its mean follows.
    After 200 steps the mean of 4096 elements is within 20% of 0.999^200 = 0.8186: one
    step's relative variance is at most frac (1 - frac) / 64 with frac = 0.016, 2.5e-4,
    so 200 add up to 0.05 and the mean's deviation to sqrt(0.05 / 4096) = 0.0035."""
    n = 4096
    hp = O.AdamWHP(1e-3, 0.9, 0.999, 1e-8, 0.0, 1)
    z = np.zeros(n, np.float32)
    x = np.full(n, 1.5, np.float32)
    for seed in (None, 1):
        mc, ms = np.zeros(n, np.uint8), np.zeros(n // 256, np.uint8)
        vc, vs = F.state8_encode(x, F.V)
        for t in range(200):
            _, mc, ms, vc, vs, _ = F.adamw_step8(z, mc, ms, vc, vs, z, hp,
                                                 None if seed is None else seed + t)
        mean = F.state8_values(vc, vs, F.V).mean(dtype=np.float64) / 1.5
        assert mean == 1.0 if seed is None else abs(mean - 0.8186) < 0.2 * 0.8186


# ------------------------------------------------------------------ 4 bits
def test_mx4_takes_the_nearest_value():
    rng = np.random.default_rng(2)
    grid = np.concatenate([F.GRID4, -F.GRID4])
    for k in range(50):
        x = (rng.standard_normal(32) * 2.0 ** int(rng.integers(-100, 100))).astype(np.float32)
        codes, scales = F.mx4_quantize(x)
        e = math.floor(math.log2(np.abs(x).max()))
        assert scales[0] == max(0, e - 2 + 127)
        best = np.abs(x.astype(np.float64)[:, None] - grid[None] * 2.0 ** (int(scales[0]) - 127))
        got = np.abs(F.mx4_values(codes, scales, 32) - x.astype(np.float64))
        assert np.array_equal(got, best.min(axis=1))


def test_mx4_ties_signs_and_specials():
    x = np.array([4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 7, -.25, -0.0, -7] + [0] * 20, np.float32)
    codes, scales = F.mx4_quantize(x)
    y = F.mx4_values(codes, scales, 32)
    assert scales[0] == 127
    assert y[:12].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 6, 0, 0, -6]
    assert np.signbit(y[9]) and np.signbit(y[10])
    odd = np.ones(33, np.float32)
    codes, scales = F.mx4_quantize(odd)
    assert codes.size == 17 and scales.size == 2 and codes[16] >> 4 == 0
    for bad in (np.nan, -np.inf):
        odd[32] = bad
        y = F.mx4_values(*F.mx4_quantize(odd), 33)
        assert np.isnan(y[32]) and (y[:32] == 1).all()
    assert not F.mx4_values(*F.mx4_quantize(np.zeros(5, np.float32)), 5).any()


# ------------------------------------------------------------------ host side
@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from fsdp_sharded_optimizer_zs_amd import build
        build.build()
    return zs.load()


def test_state8_layout(lib):
    rng = np.random.default_rng(0)
    for _ in range(50):
        numels = [int(n) for n in rng.integers(0, 5000, int(rng.integers(0, 9)))]
        off = zs.zs_state8_layout(numels)
        assert off[0] == 0 and len(off) == len(numels) + 1
        for t, n in enumerate(numels):
            assert off[t] % 1024 == 0 and 0 <= off[t + 1] - off[t] - n < 1024
    for bad, status in (([3, -1], zs.ZS_EINVAL), ([1 << 62, 1 << 62], zs.ZS_EUNSUPPORTED)):
        with pytest.raises(zs.ZsError) as e:
            zs.zs_state8_layout(bad)
        assert e.value.status == status


# Fake, never-dereferenced device addresses; skipped where a GPU is visible, so that a
# gap in the checks can never launch a kernel on them.
A = 0x7f0000000000
STEP = 0x1000000


@pytest.fixture
def no_gpu():
    if torch.cuda.device_count() > 0:
        pytest.skip("fake-address validation tests run only where no GPU is visible")


def entry(i=0, n=1000, state=zs.ZS_STATE_8BIT, **kw):
    at = A + i * 16 * STEP
    d = dict(p=at, m=at + STEP, v=at + 2 * STEP, w_out=at + 3 * STEP, g=at + 4 * STEP, numel=n)
    if state == zs.ZS_STATE_8BIT:
        d.update(m_scale=at + 5 * STEP, v_scale=at + 6 * STEP)
    d.update(kw)
    return B.zs_multi_tensor(**d)


def create(lib, entries, state=zs.ZS_STATE_8BIT, dtype=zs.ZS_BF16, T=None):
    arr = (B.zs_multi_tensor * max(1, len(entries)))(*entries)
    out = ctypes.c_void_p()
    st = lib.zs_multi_create(arr, len(entries) if T is None else T, state, dtype, ctypes.byref(out))
    return st, out


def make(lib, *args, **kw):
    st, h = create(lib, *args, **kw)
    assert st == zs.ZS_OK, zs.zs_last_error()
    return h


@pytest.mark.parametrize("state", (zs.ZS_STATE_NONE, zs.ZS_STATE_F32, zs.ZS_STATE_8BIT))
def test_image_holds_every_chunk(lib, no_gpu, state):
    """Each chunk's pointers, first element, tensor and length, tensors in order."""
    sizes = [0, 1, 4096, 4097, 0, 10000]
    es = [entry(i, n, state) if n else B.zs_multi_tensor() for i, n in enumerate(sizes)]
    es[3].w_out = None
    h = make(lib, es, state=state)
    img, nbytes = ctypes.c_void_p(), ctypes.c_int64()
    assert lib.zs_multi_image(h, ctypes.byref(img), ctypes.byref(nbytes)) == zs.ZS_OK
    raw = ctypes.string_at(img.value, nbytes.value)
    got = [(*np.frombuffer(c[:56], np.uint64).tolist(), *np.frombuffer(c[56:68], np.uint32).tolist())
           for c in (raw[k:k + 80] for k in range(0, len(raw), 80))]
    want = []
    for t, n in enumerate(sizes):
        for i in range(0, n, 4096):
            e, ms = es[t], 4 if state == zs.ZS_STATE_F32 else 1
            arrays = [0] * 6
            if state != zs.ZS_STATE_NONE:
                arrays = [e.p + 4 * i, e.m + ms * i, e.v + ms * i, 0, 0,
                          e.w_out + 2 * i if e.w_out else 0]
            if state == zs.ZS_STATE_8BIT:
                arrays[3:5] = [e.m_scale + i // 256, e.v_scale + i // 256]
            want.append((*arrays, e.g + 2 * i, i, t, min(4096, n - i)))
    assert got == want
    assert lib.zs_multi_destroy(h) == zs.ZS_OK
    assert lib.zs_multi_destroy(None) == zs.ZS_OK


@pytest.mark.parametrize("off", (0, 1, 31, 32, 63, 64, 65))
@pytest.mark.parametrize("n", (1, 63, 4032, 4033, 4095, 4096, 4097, 20_000))
def test_fp32_chunks_cover_a_tensor_and_start_on_lines(lib, no_gpu, n, off):
    """The chunks follow one another over the tensor, none over 4096 elements, and all
    but the first start where p is 256-byte aligned."""
    h = make(lib, [entry(0, n, zs.ZS_STATE_F32, p=A + 4 * off)], state=zs.ZS_STATE_F32)
    img, nbytes = ctypes.c_void_p(), ctypes.c_int64()
    lib.zs_multi_image(h, ctypes.byref(img), ctypes.byref(nbytes))
    raw = ctypes.string_at(img.value, nbytes.value)
    at = 0
    for k in range(0, len(raw), 80):
        p, m = np.frombuffer(raw[k:k + 16], np.uint64).tolist()
        first, _, live = np.frombuffer(raw[k + 56:k + 68], np.uint32).tolist()
        assert first == at and 1 <= live <= 4096
        assert p == A + 4 * off + 4 * at and m == A + STEP + 4 * at
        assert k == 0 or p % 256 == 0
        at += live
    assert at == n
    # gradients only: where g is at a multiple of 64 elements
    h = make(lib, [B.zs_multi_tensor(g=A + 2 * off, numel=n)], state=zs.ZS_STATE_NONE)
    lib.zs_multi_image(h, ctypes.byref(img), ctypes.byref(nbytes))
    raw = ctypes.string_at(img.value, nbytes.value)
    at = 0
    for k in range(0, len(raw), 80):
        g = np.frombuffer(raw[k + 48:k + 56], np.uint64).tolist()[0]
        first, _, live = np.frombuffer(raw[k + 56:k + 68], np.uint32).tolist()
        assert first == at and 1 <= live <= 4096 and g == A + 2 * off + 2 * at
        assert k == 0 or g % 128 == 0
        at += live
    assert at == n


@pytest.mark.parametrize("kw,status", [
    (dict(p=0), zs.ZS_EINVAL), (dict(m=0), zs.ZS_EINVAL), (dict(v=0), zs.ZS_EINVAL),
    (dict(g=0), zs.ZS_EINVAL), (dict(m_scale=0), zs.ZS_EINVAL), (dict(v_scale=0), zs.ZS_EINVAL),
    (dict(p=A + 2), zs.ZS_EINVAL), (dict(g=A + STEP * 4 + 1), zs.ZS_EINVAL),
    (dict(w_out=A + 3 * STEP + 1), zs.ZS_EINVAL), (dict(numel=-1), zs.ZS_EINVAL),
    (dict(numel=1 << 61), zs.ZS_EINVAL),
    (dict(m=A + 4 * 999), zs.ZS_EALIAS),                           # last byte of p
    (dict(v=A + STEP + 999), zs.ZS_EALIAS), (dict(w_out=A + 4 * 998), zs.ZS_EALIAS),
    (dict(m_scale=A + 2 * STEP + 5), zs.ZS_EALIAS), (dict(v_scale=A + 5 * STEP + 3), zs.ZS_EALIAS),
    (dict(g=A + 4 * 998), zs.ZS_EALIAS), (dict(g=A + 5 * STEP + 2), zs.ZS_EALIAS),
])
def test_multi_create_refuses(lib, no_gpu, kw, status):
    st, h = create(lib, [entry(0, **kw)])
    assert st == status and not h, zs.zs_last_error()


def test_multi_create_refuses_across_tensors(lib, no_gpu):
    assert create(lib, [entry(0), entry(0)])[0] == zs.ZS_EALIAS             # one tensor twice
    assert create(lib, [entry(0), entry(1, p=A + 4 * 999)])[0] == zs.ZS_EALIAS
    assert create(lib, [entry(0), entry(1, g=A + 2 * STEP)])[0] == zs.ZS_EALIAS
    # side by side is fine, and so is a gradient that two tensors share
    at = A + 4 * 1000
    make(lib, [entry(0), entry(1, p=at, g=A + 4 * STEP)])
    assert create(lib, [entry(0)], state=3)[0] == zs.ZS_EUNSUPPORTED
    assert create(lib, [entry(0)], dtype=5)[0] == zs.ZS_EUNSUPPORTED
    assert create(lib, [entry(0)], T=-1)[0] == zs.ZS_EINVAL
    assert create(lib, [entry(0)], state=zs.ZS_STATE_F32)[0] == zs.ZS_EINVAL  # scales given
    f32 = entry(0, state=zs.ZS_STATE_F32)
    assert create(lib, [f32])[0] == zs.ZS_EINVAL                              # scales missing
    make(lib, [f32], state=zs.ZS_STATE_F32)
    assert create(lib, [entry(0, state=zs.ZS_STATE_F32, m=A + STEP + 2)],
                  state=zs.ZS_STATE_F32)[0] == zs.ZS_EINVAL
    assert create(lib, [entry(0, state=zs.ZS_STATE_F32, v=A + STEP + 3996)],
                  state=zs.ZS_STATE_F32)[0] == zs.ZS_EALIAS
    # gradients only: nothing else is read
    make(lib, [B.zs_multi_tensor(g=A, numel=5)], state=zs.ZS_STATE_NONE)
    assert lib.zs_multi_create(None, 1, 0, zs.ZS_F32, ctypes.byref(ctypes.c_void_p())) == zs.ZS_EINVAL
    assert lib.zs_multi_create(None, 0, 0, zs.ZS_F32, None) == zs.ZS_EINVAL


def hp(**kw):
    d = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)
    d.update(kw)
    return B.zs_adamw_hp(*[d[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay", "step")])


def test_adamw_multi_refuses(lib, no_gpu):
    h = make(lib, [entry(0)])
    img = A + 15 * STEP

    def call(multi=h, image=img, h_=hp(), scale=None, opts=None):
        return lib.zs_adamw_multi(multi, image, ctypes.byref(h_) if h_ else None, scale,
                                  ctypes.byref(opts) if opts else None, None)

    junk = (ctypes.c_uint8 * 256)()
    assert call(multi=None) == zs.ZS_EINVAL
    assert call(multi=ctypes.addressof(junk)) == zs.ZS_EINVAL
    assert call(image=None) == zs.ZS_EINVAL
    assert call(image=img + 8) == zs.ZS_EINVAL
    assert call(h_=None) == zs.ZS_EINVAL
    for bad in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(lr=NAN), dict(eps=-1.0),
                dict(weight_decay=INF)):
        assert call(h_=hp(**bad)) == zs.ZS_EINVAL
    assert call(scale=A + 1) == zs.ZS_EINVAL
    for at in (A, A + 3996, A + STEP + 996, A + 2 * STEP, A + 3 * STEP + 1996, A + 5 * STEP):
        assert call(scale=at) == zs.ZS_EALIAS, at - A              # p, m, v, w_out, m_scale
    assert call(opts=B.zs_round_opts(2, 0, 0)) == zs.ZS_EINVAL
    assert call(opts=B.zs_round_opts(1, 1, 0)) == zs.ZS_EINVAL
    grads = make(lib, [B.zs_multi_tensor(g=A, numel=5)], state=zs.ZS_STATE_NONE)
    assert call(multi=grads) == zs.ZS_EINVAL and "gradients only" in zs.zs_last_error()
    for empty in (make(lib, []), make(lib, [B.zs_multi_tensor()] * 3)):
        assert call(multi=empty, image=None) == zs.ZS_OK                     # nothing to do


def test_grad_norm_refuses(lib, no_gpu):
    h = make(lib, [entry(0)])
    ok = dict(multi=h, image=A + 15 * STEP, max_norm=1.0, sumsq=A + 16 * STEP,
              nc=A + 17 * STEP, ws=A + 18 * STEP)

    def call(**kw):
        d = dict(ok, **kw)
        return lib.zs_grad_norm(d["multi"], d["image"], d["max_norm"], d["sumsq"], d["nc"],
                                d["ws"], None)

    for bad in (dict(multi=None), dict(image=None), dict(image=A + 4), dict(max_norm=0.0),
                dict(max_norm=-1.0), dict(max_norm=NAN), dict(sumsq=None), dict(nc=None),
                dict(ws=None), dict(sumsq=A + 16 * STEP + 4), dict(nc=A + 17 * STEP + 2),
                dict(ws=A + 18 * STEP + 8)):
        assert call(**bad) == zs.ZS_EINVAL, bad
    for bad in (dict(nc=A + 16 * STEP), dict(sumsq=A + 18 * STEP + 32760),
                dict(sumsq=A + 4 * STEP + 1992), dict(ws=A + 4 * STEP - 32768 + 16)):
        assert call(**bad) == zs.ZS_EALIAS, bad
    # several gradients, one of them inside another, one joined to another, one apart
    h = make(lib, [B.zs_multi_tensor(g=g, numel=n) for g, n in (
        (A, 1000), (A + 400, 10), (A + 2000, 1000), (A + 64000, 8))], state=zs.ZS_STATE_NONE)
    for at in (A, A + 1992, A + 2000, A + 3992, A + 64008):
        assert call(multi=h, sumsq=at) == zs.ZS_EALIAS, at - A
        assert call(multi=h, nc=at) == zs.ZS_EALIAS, at - A
    assert call(multi=h, ws=A + 64000 - 16000) == zs.ZS_EALIAS


def test_clip_coef_refuses(lib, no_gpu):
    arr = (ctypes.c_void_p * 2)(A, A + 8)
    assert lib.zs_clip_coef(arr, 0, 1.0, A + 64, None) == zs.ZS_EINVAL
    assert lib.zs_clip_coef(arr, 65, 1.0, A + 64, None) == zs.ZS_EINVAL
    assert lib.zs_clip_coef(arr, 2, 0.0, A + 64, None) == zs.ZS_EINVAL
    assert lib.zs_clip_coef(arr, 2, 1.0, None, None) == zs.ZS_EINVAL
    assert lib.zs_clip_coef(None, 2, 1.0, A + 64, None) == zs.ZS_EINVAL
    assert lib.zs_clip_coef(arr, 2, 1.0, A + 8, None) == zs.ZS_EALIAS
    assert lib.zs_clip_coef((ctypes.c_void_p * 1)(A + 4), 1, 1.0, A + 64, None) == zs.ZS_EINVAL


def test_state8_conversions_refuse(lib, no_gpu):
    x, c, s = A, A + STEP, A + 2 * STEP
    enc = lambda x=x, n=1000, k=0, c=c, s=s: lib.zs_state8_encode(x, n, k, c, s, None)
    dec = lambda c=c, s=s, n=1000, k=0, dt=zs.ZS_F32, o=x: lib.zs_state8_decode(c, s, n, k, dt, o, None)
    assert enc(k=2) == zs.ZS_EUNSUPPORTED and dec(k=-1) == zs.ZS_EUNSUPPORTED
    assert dec(dt=9) == zs.ZS_EUNSUPPORTED
    for f in (enc, dec):
        assert f(n=-1) == zs.ZS_EINVAL and f(c=None) == zs.ZS_EINVAL and f(s=None) == zs.ZS_EINVAL
        assert f(n=0) == zs.ZS_OK
    assert enc(x=None) == zs.ZS_EINVAL and enc(x=A + 2) == zs.ZS_EINVAL
    assert dec(o=None) == zs.ZS_EINVAL and dec(o=A + 2) == zs.ZS_EINVAL
    assert dec(dt=zs.ZS_BF16, o=A + 1) == zs.ZS_EINVAL
    assert enc(c=A + 3999) == zs.ZS_EALIAS and enc(s=A + 8) == zs.ZS_EALIAS
    assert enc(s=c + 999) == zs.ZS_EALIAS
    assert dec(c=A + 3999) == zs.ZS_EALIAS and dec(s=A - 3) == zs.ZS_EALIAS


def test_mx4_refuses(lib, no_gpu):
    q = lambda x=A, dt=zs.ZS_BF16, n=1000, c=A + STEP, s=A + 2 * STEP: lib.zs_quantize_mx4(
        x, dt, n, c, s, None)
    assert q(dt=0) == zs.ZS_EUNSUPPORTED and q(n=-1) == zs.ZS_EINVAL and q(n=0) == zs.ZS_OK
    assert q(x=None) == zs.ZS_EINVAL and q(c=None) == zs.ZS_EINVAL and q(s=None) == zs.ZS_EINVAL
    assert q(x=A + 1) == zs.ZS_EINVAL and q(dt=zs.ZS_F32, x=A + 2) == zs.ZS_EINVAL
    assert q(c=A + 1999) == zs.ZS_EALIAS and q(s=A) == zs.ZS_EALIAS
    assert q(s=A + STEP + 499) == zs.ZS_EALIAS

    def g(D=2, n=1000, dt=zs.ZS_BF16, out=A, c=(A + STEP, A + 2 * STEP), s=(A + 3 * STEP, A + 4 * STEP)):
        ca, sa = ((ctypes.c_void_p * 2)(*v) if v else None for v in (c, s))
        return lib.zs_gather_unit_mx4(ca, sa, D, n, dt, out, None)

    assert g(dt=3) == zs.ZS_EUNSUPPORTED and g(n=0) == zs.ZS_OK
    for bad in (dict(D=0), dict(D=65), dict(n=-1), dict(n=1 << 62), dict(out=None), dict(out=A + 1),
                dict(c=None), dict(s=None), dict(c=(A + STEP, 0)), dict(s=(0, A + STEP))):
        assert g(**bad) == zs.ZS_EINVAL, bad
    for bad in (dict(c=(A + 3999, A + STEP)), dict(s=(A + STEP, A + 5))):
        assert g(**bad) == zs.ZS_EALIAS, bad


def test_python_checks():
    cpu = torch.zeros(8)
    with pytest.raises(ValueError):
        zs.MultiTable(grads=[cpu])                                # not on the device
    with pytest.raises(ValueError):
        zs.MultiTable(p=[cpu], grads=[])
    for f in (lambda: zs.zs_quantize_mx4(cpu, cpu, cpu), lambda: zs.zs_gather_unit_mx4([], [], cpu),
              lambda: zs.zs_state8_encode(cpu, 0, cpu, cpu),
              lambda: zs.zs_state8_decode(cpu, cpu, 0, cpu),
              lambda: zs.zs_clip_coef([cpu], 1.0, cpu)):
        with pytest.raises(ValueError):
            f()


def test_clip_coefficient_of_the_oracle():
    assert F.clip_coef(4.0, 1.0) == (2, np.float32(1 / (2 + 1e-6)))
    assert F.clip_coef(0.25, 1.0) == (0.5, 1) and F.clip_coef(4.0, INF) == (2, 1)
