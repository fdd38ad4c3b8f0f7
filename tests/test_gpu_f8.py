"""Block-scaled 8-bit matrices on the GPU: codes bit for bit against the oracle, products
against sums in float64.

Scales are powers of two and a code is one rounding of an exact quotient, so codes, scale
bytes and decoded values have one right answer. Products are checked in two ways. Small
whole numbers under small powers of two give sums that every order and the instructions'
window hold exactly, so that C is the exact sum rounded once: any wrong index shows. For
values of all sizes the tolerance is the documented bound: for C in bf16 7 * 2^-13 of the
sum over groups of 8 along K of the largest product (Tops), plus 2^-8 of the value for the
rounding; for C in fp32 each step of 32 along K is rounded to fp32 (2^-23 of the running
sum, at most Mags, the magnitudes' sum; counted twice for its inside), plus 2^-24 of the
value. Adding up splits and the old C are a few fp32 additions more (32 * 2^-23 Mags)."""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
from gpu_util import check_bf16, check_bits, check_f32, device, to_np
from oracle import zs_f8 as F
from oracle import zs_oracle as O

pytestmark = pytest.mark.gpu

KINDS = (F.E4M3, F.E5M2)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def matrix(rows, cols, seed, wide=False, std=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * std
    if wide:
        x = x * 10.0 ** rng.uniform(-44, 37, (rows, 1)) * 10.0 ** rng.uniform(-5, 1, (rows, cols))
    return np.clip(x, -3.3e38, 3.3e38).astype(np.float32)


def on_device(x, dtype, pad=0, lead=0):
    """x as a matrix whose rows are `pad` elements apart, from element `lead` of an allocation;
    the float32 values that it holds."""
    rows, cols = x.shape
    x = O.bf16_widen(O.bf16_round(x)) if dtype == "bf16" else x
    store = torch.full((lead + rows * (cols + pad) + 1,), 55.0, dtype=DTYPES[dtype], device=device())
    view = store[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.from_numpy(x).to(device()))
    return view, x


class Guarded:
    """An F8Matrix whose codes and scales have sentinel bytes around them."""

    def __init__(self, rows, cols, kind, block_rows, fill=0xEE):
        self.parts, views = [], []
        for n in zs.zs_f8_layout(rows, cols, block_rows):
            a = torch.full((n + 512,), fill, dtype=torch.uint8, device=device())
            self.parts.append((a, n))
            views.append(a[256:256 + n])
        self.fill = fill
        self.m = zs.F8Matrix(*views, rows, cols, kind, block_rows)

    def check(self, codes, scales, what):
        for (a, n), want, name in zip(self.parts, (codes, scales), ("codes", "scales")):
            check_bits(to_np(a[256:256 + n]), want.ravel(), f"{what} {name}")
            assert bool((a[:256] == self.fill).all() and (a[256 + n:] == self.fill).all()), what


def f8(x, kind=F.E4M3, block_rows=1):
    """An F8Matrix made by the oracle from float32 values, and its values in float64."""
    c, s = F.quantize(x, kind, block_rows)
    t = [torch.from_numpy(np.ascontiguousarray(v).ravel()).to(device()) for v in (c, s)]
    return zs.F8Matrix(*t, *x.shape, kind, block_rows), F.values(c, s, *x.shape, kind, block_rows)


SHAPES = [(1, 1), (1, 7), (7, 1), (3, 8), (5, 127), (127, 5), (128, 128), (129, 129), (1, 512), (2, 513),
          (130, 1000), (300, 257), (256, 1024)]


@pytest.mark.parametrize("block_rows", (1, 128))
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(rows, cols, dtype, block_rows):
    for seed, (wide, pad, lead, kind, kind_t) in enumerate([
            (False, 0, 0, F.E4M3, F.E4M3), (True, 3, 1, F.E5M2, F.E4M3), (True, 0, 5, F.E4M3, F.E5M2)]):
        x, h = on_device(matrix(rows, cols, seed + rows * cols, wide), dtype, pad, lead)
        out, out_t = Guarded(rows, cols, kind, block_rows), Guarded(cols, rows, kind_t, block_rows)
        one, one_t = Guarded(rows, cols, kind, block_rows), Guarded(cols, rows, kind_t, block_rows)
        zs.zs_quantize_f8(x, out.m, out_t.m)
        zs.zs_quantize_f8(x, one.m)
        zs.zs_quantize_f8(x, out_t=one_t.m)
        for o in (out, one):
            o.check(*F.quantize(h, kind, block_rows), f"{rows}x{cols} {seed}")
        for o in (out_t, one_t):
            o.check(*F.quantize(h.T, kind_t, block_rows), f"{rows}x{cols} {seed} transposed")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_quantize_specials(dtype, kind):
    x = matrix(140, 300, 9)
    x[3, 7], x[4, 140], x[5, 299], x[130, 1] = np.nan, np.inf, -np.inf, -np.nan
    x[10] = 0
    x[11] = -0.0
    x[12] = 1e-45
    x[13, ::2] = -1e-39
    x[13, 1::2] = 3e-40
    x[14, :128] = 3.38e38
    x[15] = np.float32(2.0**-119) * np.linspace(-2, 2, 300)       # codes under the least scale
    for block_rows in (1, 128):
        t, h = on_device(x, dtype)
        out, out_t = Guarded(140, 300, kind, block_rows), Guarded(300, 140, kind, block_rows)
        zs.zs_quantize_f8(t, out.m, out_t.m)
        out.check(*F.quantize(h, kind, block_rows), "rows")
        out_t.check(*F.quantize(h.T, kind, block_rows), "columns")


@pytest.mark.parametrize("kind", KINDS)
def test_quantize_every_bf16_value(kind):
    """Every finite bf16 value beside a block's largest magnitude of its own and of larger
    exponents, so that every tie and subnormal code is met."""
    h = np.arange(1 << 16, dtype=np.uint16)
    v = O.bf16_widen(h[(h & 0x7F80) != 0x7F80])
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(v.astype(np.float64)), 2.0**-133)))
    for shift in (0, 4, 9, 16, 18):
        top = np.exp2(np.clip(e + shift, -133, 127))
        x = np.zeros((v.size // 64 + 1, 128), np.float32)
        flat = x[:, :64].reshape(-1)
        order = np.argsort(e, kind="stable")
        flat[: v.size] = v[order]
        x[:, :64] = flat.reshape(x.shape[0], 64)
        t = np.zeros(x.shape[0] * 64)
        t[: v.size] = top[order]
        x[:, 64] = t.reshape(-1, 64).max(axis=1)
        d, hx = on_device(x, "bf16")
        out = Guarded(*x.shape, kind, 1)
        zs.zs_quantize_f8(d, out.m)
        out.check(*F.quantize(hx, kind), f"shift {shift}")


@pytest.mark.parametrize("out", ("bf16", "f32"))
@pytest.mark.parametrize("kind", KINDS)
def test_dequantize_every_code_and_scale(kind, out):
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(1, 256), (256, 1))
    scales = np.ones((256, 4), np.uint8)
    scales[:, 0] = scales[:, 1] = np.arange(256)
    m = zs.F8Matrix(*(torch.from_numpy(x.ravel().copy()).to(device()) for x in (codes, scales)), 256, 256, kind)
    with np.errstate(over="ignore"):
        want = F.values(codes, scales, 256, 256, kind).astype(np.float32)
    got = torch.zeros(256, 256, dtype=DTYPES[out], device=device())
    zs.zs_dequantize_f8(m, got)
    if out == "bf16":
        check_bf16(to_np(got).ravel(), O.bf16_round(want).ravel(), "values", exact=True)
    else:
        check_f32(to_np(got).ravel(), want.ravel(), "values", exact=True)


@pytest.mark.parametrize("block_rows", (1, 128))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dequantize(rows, cols, block_rows):
    m, want = f8(matrix(rows, cols, 3 * rows + cols), F.E5M2, block_rows)
    for out, pad, lead in (("bf16", 0, 0), ("f32", 3, 1), ("bf16", 5, 3)):
        store = torch.full((lead + rows * (cols + pad),), 55.0, dtype=DTYPES[out], device=device())
        view = store[lead:].view(rows, cols + pad)
        zs.zs_dequantize_f8(m, view[:, :cols])
        assert np.array_equal(view[:, :cols].double().cpu().numpy(), want)
        assert bool((view[:, cols:] == 55).all()) and bool((store[:lead] == 55).all())


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("D,S,offset,rows,cols", [
    (1, 128 * 128, 0, 128, 128), (1, 70_000, 37, 130, 257), (2, 20_002, 3, 200, 200), (4, 9_999, 1_001, 129, 300),
    (64, 700, 130, 150, 290), (5, 3, 1, 2, 7), (64, 1, 0, 8, 8), (8, 5_000, 39_999, 1, 1), (3, 50_000, 0, 1, 150_000),
    (3, 50_000, 11, 149_000, 1), (7, 4_096, 0, 128, 224)])
def test_gather(D, S, offset, rows, cols, dtype):
    flat = matrix(1, D * S, D + S, std=0.02)[0]
    flat = O.bf16_widen(O.bf16_round(flat)) if dtype == "bf16" else flat
    shards = []
    for r in range(D):
        lead = r % 3                                  # shards start anywhere
        s = torch.full((S + lead,), 9.0, dtype=DTYPES[dtype], device=device())
        s[lead:].copy_(torch.from_numpy(flat[r * S:(r + 1) * S]).to(device()))
        shards.append(s[lead:])
    h = flat[offset:offset + rows * cols].reshape(rows, cols)
    for block_rows in (128, 1):
        out, out_t = Guarded(rows, cols, F.E4M3, block_rows), Guarded(cols, rows, F.E4M3, block_rows)
        zs.zs_gather_matrix_f8(shards, offset, out.m, out_t.m)
        out.check(*F.quantize(h, F.E4M3, block_rows), "gathered")
        out_t.check(*F.quantize(h.T, F.E4M3, block_rows), "gathered, transposed")


# ------------------------------------------------------------------- products
def whole(rows, cols, seed, kind=F.E4M3):
    """Whole numbers -3 .. 3 under a power of two a block (oracle codes; the largest magnitude
    fixes the scale, so each block holds a 3)."""
    rng = np.random.default_rng(seed)
    x = rng.integers(-3, 4, (rows, cols)).astype(np.float32)
    x[:, ::128] = 3
    return x * np.repeat(2.0 ** rng.integers(-1, 2, (1, F.ceil(cols, 128))), 128, 1)[:, :cols].astype(np.float32)


def workspace(M, N, K, f=None):
    return torch.zeros((f or zs.zs_matmul_f8_workspace)(M, N, K), dtype=torch.uint8, device=device())


def out_matrix(M, N, dtype, pad=0, lead=0):
    store = torch.full((lead + M * (N + pad),), 55.0, dtype=DTYPES[dtype], device=device())
    full = store[lead:].view(M, N + pad)
    return store, full, full[:, :N]


def check_beside(store, full, N, lead, what):
    assert bool((full[:, N:] == 55).all()) and bool((store[:lead] == 55).all()), f"{what}: written beside C"


def rounded(x, dtype):
    x = x.astype(np.float32)
    return O.bf16_widen(O.bf16_round(x)) if dtype == "bf16" else x


PRODUCTS = [(1, 1, 1), (1, 16, 128), (1, 40, 1000), (2, 100, 4096), (3, 1, 129), (15, 33, 640), (16, 64, 512),
            (17, 17, 513), (31, 1000, 300), (33, 31, 2000), (64, 64, 128), (65, 130, 1500), (100, 300, 127),
            (128, 128, 1024), (129, 257, 385), (200, 520, 4100), (300, 1030, 700), (513, 600, 896)]


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_exact_products(M, N, K, dtype):
    ws = workspace(M, N, K)
    for i, (ka, kb, br_a, br_b, pad, lead) in enumerate([
            (F.E4M3, F.E4M3, 1, 1, 0, 0), (F.E5M2, F.E4M3, 1, 128, 3, 1), (F.E4M3, F.E5M2, 128, 1, 0, 3),
            (F.E5M2, F.E5M2, 128, 128, 1, 0)]):
        a, va = f8(whole(M, K, i), ka, br_a)
        b, vb = f8(whole(N, K, 90 + i), kb, br_b)
        want = va @ vb.T
        store, full, c = out_matrix(M, N, dtype, pad, lead)
        zs.zs_matmul_f8(a, b, c, workspace=ws)
        assert np.array_equal(c.double().cpu().numpy(), rounded(want, dtype).astype(np.float64))
        check_beside(store, full, N, lead, f"{i}")
        old = c.double().cpu().numpy()
        zs.zs_matmul_f8(a, b, c, accumulate=True, workspace=ws)
        assert np.array_equal(c.double().cpu().numpy(), rounded(old + want, dtype).astype(np.float64))
        check_beside(store, full, N, lead, f"{i} accumulated")


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("M,N,K", [(3333, 4200, 300), (3841, 3585, 1), (4096, 4096, 128), (5000, 2561, 1700),
                                   (2600, 5003, 640), (1000, 13_000, 257), (500, 4001, 11_000)])
def test_exact_large_products(M, N, K, dtype):
    """Sizes that fill the chip with the largest tiles; the sum by torch in fp32, which holds
    these whole numbers exactly."""
    for i, (ka, kb, br_a, br_b, pad) in enumerate([(F.E4M3, F.E4M3, 1, 128, 0), (F.E5M2, F.E4M3, 1, 1, 5)]):
        a, va = f8(whole(M, K, i), ka, br_a)
        b, vb = f8(whole(N, K, 90 + i), kb, br_b)
        va, vb = (torch.from_numpy(v.astype(np.float32)).to(device()) for v in (va, vb))
        want = torch.mm(va, vb.t().contiguous()).to(DTYPES[dtype])
        store, full, c = out_matrix(M, N, dtype, pad, 3 * (pad > 0))
        zs.zs_matmul_f8(a, b, c, workspace=workspace(M, N, K))
        assert torch.equal(c, want)
        check_beside(store, full, N, 3 * (pad > 0), f"{i}")


def tolerance(a, b, dtype):
    exact, mags, tops = F.product(a, b)
    n = F.ceil(a.shape[1], 32)
    if dtype == "bf16":
        return exact, 7 * 2.0**-13 * tops + 32 * 2.0**-23 * mags + 2.0**-8 * np.abs(exact)
    return exact, (2 * n + 32) * 2.0**-23 * mags + 2.0**-24 * np.abs(exact)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("ka,kb", [(F.E4M3, F.E4M3), (F.E5M2, F.E4M3), (F.E4M3, F.E5M2), (F.E5M2, F.E5M2)])
@pytest.mark.parametrize("M,N,K", [(1, 70, 1100), (5, 40, 130), (40, 50, 3000), (130, 140, 1024)])
def test_products_of_all_sizes(M, N, K, ka, kb, dtype):
    rng = np.random.default_rng(M + N)
    x = matrix(M, K, 1) * np.exp(rng.standard_normal((M, K)) * 2)
    y = matrix(N, K, 2) * np.exp(rng.standard_normal((1, K)) * 2) * 0.02
    a, va = f8(x.astype(np.float32), ka)
    b, vb = f8(y.astype(np.float32), kb, 128)
    exact, tol = tolerance(va, vb, dtype)
    _, _, c = out_matrix(M, N, dtype)
    zs.zs_matmul_f8(a, b, c, workspace=workspace(M, N, K))
    assert (np.abs(c.double().cpu().numpy() - exact) <= tol).all()


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("M,N", [(1, 20), (40, 70), (150, 300)])
def test_blocks_of_nan(M, N, dtype):
    """A block that is not finite makes what reads it NaN, and nothing else."""
    x, y = whole(M, 400, 5), whole(N, 400, 6)
    x[M // 2, 130] = np.inf
    y[N - 1, 399] = np.nan
    a, _ = f8(x)
    b, _ = f8(y)
    _, _, c = out_matrix(M, N, dtype)
    zs.zs_matmul_f8(a, b, c, workspace=workspace(M, N, 400))
    x[M // 2] = 0
    y[N - 1] = 0
    want = rounded(x.astype(np.float64) @ y.T.astype(np.float64), dtype)
    want[M // 2] = np.nan
    want[:, N - 1] = np.nan
    assert np.array_equal(c.float().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_scales_at_the_ends(dtype):
    """Blocks of very large and very small values whose products are in the middle."""
    x, y = whole(40, 256, 1), whole(50, 256, 2)
    for e in (100, -100):
        a, _ = f8((x * 2.0**e).astype(np.float32))
        b, _ = f8((y * 2.0**-e).astype(np.float32), F.E5M2, 128)
        _, _, c = out_matrix(40, 50, dtype)
        zs.zs_matmul_f8(a, b, c, workspace=workspace(40, 50, 256))
        want = rounded(x.astype(np.float64) @ y.T.astype(np.float64), dtype)
        assert np.array_equal(c.float().cpu().numpy(), want), e


@pytest.mark.parametrize("M,N", [(4, 20), (40, 50)])
def test_subnormal_values_and_codes(M, N):
    """Values down to 2^-135 under products in the middle: the 8-bit instructions take every
    code and scale byte; for C in fp32 operands pass through bf16, exact down to 2^-133."""
    x, y = whole(M, 256, 1).astype(np.float64), whole(N, 256, 2).astype(np.float64)
    for ex, ey in ((-124, 120), (-128, 120), (-131, 120), (-135, 124), (125, -125)):
        for kind in KINDS:
            a, va = f8((x * 2.0**ex).astype(np.float32), kind)
            b, vb = f8((y * 2.0**ey).astype(np.float32), F.E4M3, 128)
            for dtype in DTYPES:
                if dtype == "f32" and ex == -135:
                    continue
                _, _, c = out_matrix(M, N, dtype)
                zs.zs_matmul_f8(a, b, c, workspace=workspace(M, N, 256))
                assert np.array_equal(c.float().cpu().numpy(), rounded(va @ vb.T, dtype)), (ex, kind, dtype)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("M,N", [(4, 20), (40, 50)])
def test_codes_that_are_not_finite(M, N, dtype):
    """Codes of infinity and NaN that a caller wrote go through products as such."""
    a, b = zs.F8Matrix.empty(M, 128, zs.ZS_E5M2), zs.F8Matrix.empty(N, 128)
    a.codes.zero_()
    b.codes.fill_(0x38)                               # 1
    for m in (a, b):
        m.scales.fill_(127)
    for r, code in enumerate((0x3C, 0x7C, 0xFC, 0x7F)):
        a.codes.view(M, 128)[r, 5 + r] = code
    _, _, c = out_matrix(M, N, dtype)
    zs.zs_matmul_f8(a, b, c, workspace=workspace(M, N, 128))
    want = np.zeros((M, N), np.float32)
    want[:4] = np.array([1, np.inf, -np.inf, np.nan])[:, None]
    assert np.array_equal(c.float().cpu().numpy(), want, equal_nan=True)


def test_empty_products():
    ws = workspace(64, 64, 0)
    for M, N, K in ((0, 8, 256), (8, 0, 256), (70, 80, 0), (1, 5, 0)):
        a, b = (zs.F8Matrix.empty(r, K) for r in (M, N))
        for dtype in DTYPES:
            _, _, c = out_matrix(M, N, dtype)
            zs.zs_matmul_f8(a, b, c, workspace=ws)
            assert bool((c == 0).all())
            c.fill_(3)
            zs.zs_matmul_f8(a, b, c, accumulate=True, workspace=ws)
            assert bool((c == 3).all())
    y = torch.full((4, 6), 5.0, device=device())
    w = zs.F8Matrix.empty(6, 0, block_rows=128)
    zs.zs_linear_f8(torch.zeros(4, 0, device=device()), w, y, workspace(4, 6, 0, zs.zs_linear_f8_workspace))
    assert bool((y == 0).all())


def test_one_workspace_for_products_of_all_sizes():
    """Counts are at 0 after every call whatever came before, and results do not depend on it."""
    sizes = [(64, 64, 4096), (20, 700, 8192), (300, 64, 2048), (64, 64, 4096), (256, 256, 1024)]
    ws = torch.zeros(max(zs.zs_matmul_f8_workspace(*s) for s in sizes), dtype=torch.uint8, device=device())
    assert ws.numel() > 0
    for rep in range(2):
        for i, (M, N, K) in enumerate(sizes):
            a, va = f8(whole(M, K, i))
            b, vb = f8(whole(N, K, 50 + i))
            for dtype in DTYPES:
                _, _, c = out_matrix(M, N, dtype)
                zs.zs_matmul_f8(a, b, c, workspace=ws)
                assert np.array_equal(c.double().cpu().numpy(), rounded(va @ vb.T, dtype).astype(np.float64))


def test_same_bits_every_time():
    a, _ = f8(matrix(70, 5000, 1))
    b, _ = f8(matrix(90, 5000, 2))
    for dtype in DTYPES:
        got = []
        for _ in range(5):
            _, _, c = out_matrix(70, 90, dtype)
            zs.zs_matmul_f8(a, b, c, workspace=workspace(70, 90, 5000))
            got.append(c)
        assert all(torch.equal(got[0], g) for g in got[1:])


# ---------------------------------------------------------------- linear layer
@pytest.mark.parametrize("y_dtype", ("bf16", "f32"))
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (1, 300, 1000), (1, 37, 5), (2, 64, 2048), (3, 129, 640), (4, 50, 4100),
                                   (7, 33, 777), (16, 256, 256), (17, 40, 3000), (33, 257, 129), (130, 300, 520),
                                   (1, 700, 11008)])
def test_linear(M, N, K, dtype, y_dtype):
    for kind, br, pad, lead in ((F.E4M3, 128, 0, 0), (F.E5M2, 1, 3, 1)):
        x, h = on_device(matrix(M, K, M + K) * np.exp(matrix(1, K, 7)), dtype, pad, lead)
        w, vw = f8(matrix(N, K, 8, std=0.02), F.E4M3, br)
        store, full, y = out_matrix(M, N, y_dtype, pad, lead)
        zs.zs_linear_f8(x, w, y, workspace(M, N, K, zs.zs_linear_f8_workspace), type=kind)
        exact, tol = tolerance(F.quantized(h, kind), vw, y_dtype)
        assert (np.abs(y.double().cpu().numpy() - exact) <= tol).all()
        check_beside(store, full, N, lead, "linear")


@pytest.mark.parametrize("y_dtype", ("bf16", "f32"))
@pytest.mark.parametrize("M,N,K", [(17, 1, 1), (17, 64, 127), (33, 100, 128), (64, 64, 2048), (64, 70, 2049), (65, 1000, 513),
                                   (100, 65, 640), (1000, 700, 900), (777, 1001, 1500), (2048, 256, 1024), (129, 4000, 2047),
                                   (16, 300, 2000), (5, 40, 700), (40, 3000, 5000), (300, 20_000, 200)])
def test_linear_is_its_two_calls(M, N, K, y_dtype):
    """Codes that are made on the way give the bits of the quantiser's codes, in every form."""
    for i, (dtype, kind, kind_w, br, pad, lead) in enumerate([
            ("bf16", F.E4M3, F.E4M3, 128, 0, 0), ("f32", F.E5M2, F.E4M3, 1, 3, 1), ("bf16", F.E5M2, F.E5M2, 128, 5, 3),
            ("f32", F.E4M3, F.E5M2, 128, 0, 0)]):
        x, _ = on_device(matrix(M, K, i) * np.exp(matrix(M, 1, i + 9)), dtype, pad, lead)
        if i == 1:
            x[M // 2, K // 2] = float("inf")
            x[M // 3] = 2.0**-140
        w, _ = f8(matrix(N, K, 50 + i), kind_w, br)
        _, _, want = out_matrix(M, N, y_dtype)
        store, full, y = out_matrix(M, N, y_dtype, pad, lead)
        codes = zs.F8Matrix.empty(M, K, kind)
        zs.zs_quantize_f8(x, codes)
        zs.zs_matmul_f8(codes, w, want, workspace=workspace(M, N, K))
        zs.zs_linear_f8(x, w, y, workspace(M, N, K, zs.zs_linear_f8_workspace), type=kind)
        assert torch.equal(y.view(torch.int16 if y_dtype == "bf16" else torch.int32),
                           want.view(torch.int16 if y_dtype == "bf16" else torch.int32)), i
        check_beside(store, full, N, lead, f"{i}")


@pytest.mark.parametrize("M", (1, 2, 5, 16, 40))
def test_linear_of_not_finite_rows(M):
    x, h = on_device(whole(M, 300, 3), "bf16")
    x[M // 2, 140] = float("nan")
    w, vw = f8(whole(50, 300, 4), block_rows=1)
    _, _, y = out_matrix(M, 50, "bf16")
    zs.zs_linear_f8(x, w, y, workspace(M, 50, 300, zs.zs_linear_f8_workspace))
    want = rounded(F.quantized(h) @ vw.T, "bf16")
    want[M // 2] = np.nan
    assert np.array_equal(y.float().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 50, 40), (130, 64, 200), (257, 300, 129), (1000, 70, 90)])
def test_backward(M, N, K, kind):
    dev = device()
    w, hw = matrix(N, K, 2, std=0.02), None
    w_t, vw_t = f8(np.ascontiguousarray(w.T), F.E4M3, 128)
    ws = workspace(M, N, K, zs.zs_linear_f8_backward_workspace)
    for dtype, dx_dtype, dw_dtype, pad in (("bf16", "bf16", "bf16", 0), ("f32", "f32", "f32", 3), ("bf16", "bf16", "f32", 1)):
        dy, hdy = on_device(matrix(M, N, 3, std=1e-4) * np.exp(matrix(M, 1, 4)), dtype, pad, pad)
        x, hx = on_device(matrix(M, K, 5), dtype, pad)
        s1, f1, dx = out_matrix(M, K, dx_dtype, pad)
        # the weight's gradient as a view into a unit's flat gradient, at an odd element
        flat = torch.full((N * K + 9,), 55.0, dtype=DTYPES[dw_dtype], device=dev)
        dw = flat[5:5 + N * K].view(N, K)
        zs.zs_linear_f8_backward(dy, x, w_t, dx, dw, ws, grad_type=kind)
        e, t = tolerance(F.quantized(hdy, kind), vw_t, dx_dtype)
        assert (np.abs(dx.double().cpu().numpy() - e) <= t).all()
        check_beside(s1, f1, K, 0, "dx")
        e, t = tolerance(F.quantized(hdy.T, kind), F.quantized(hx.T), dw_dtype)
        assert (np.abs(dw.double().cpu().numpy() - e) <= t).all()
        assert bool((flat[:5] == 55).all() and (flat[5 + N * K:] == 55).all())
        # one of the two alone, and a second micro-batch added up
        dx2, dw2 = torch.zeros_like(dx), torch.zeros_like(dw)
        zs.zs_linear_f8_backward(dy, None, w_t, dx2, None, ws, grad_type=kind)
        zs.zs_linear_f8_backward(dy, x, None, None, dw2, ws, grad_type=kind)
        assert torch.equal(dx2, dx.contiguous()) and torch.equal(dw2, dw)
        zs.zs_linear_f8_backward(dy, x, None, None, dw2, ws, grad_type=kind, accumulate=True)
        assert (np.abs(dw2.double().cpu().numpy() - 2 * e) <= 2 * t + 2.0**-7 * np.abs(e)).all()


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("M,N,K", [(3900, 4000, 3850), (2000, 1900, 2000), (4200, 300, 300), (700, 5000, 40), (11_000, 4000, 512)])
def test_exact_large_backward(M, N, K, dtype):
    """Both products in one launch by every tile, and by other tiles and types in two: whole
    numbers under small powers of two, which 8 bits and every order of the sum hold exactly
    (below 2^24 of their steps)."""
    dev = device()
    dy, x, w = (torch.from_numpy(whole(a, b, i)).to(dev) for i, (a, b) in enumerate(((M, N), (M, K), (N, K))))
    want = [torch.mm(dy, w), torch.mm(dy.t().contiguous(), x)]
    ws = workspace(M, N, K, zs.zs_linear_f8_backward_workspace)
    for kind_w, kind, other, pad in ((F.E4M3, F.E4M3, False, 0), (F.E4M3, F.E5M2, False, 3), (F.E5M2, F.E4M3, False, 0),
                                     (F.E4M3, F.E4M3, True, 1)):
        w_t = zs.F8Matrix.empty(K, N, kind_w)
        zs.zs_quantize_f8(w, None, w_t)
        dw_dtype = {"bf16": "f32", "f32": "bf16"}[dtype] if other else dtype
        s1, f1, dx = out_matrix(M, K, dtype, pad, pad)
        s2, f2, dw = out_matrix(N, K, dw_dtype, pad, pad)
        zs.zs_linear_f8_backward(dy, x, w_t, dx, dw, ws, grad_type=kind)
        assert torch.equal(dx, want[0].to(DTYPES[dtype])) and torch.equal(dw, want[1].to(DTYPES[dw_dtype]))
        check_beside(s1, f1, K, pad, "dx")
        check_beside(s2, f2, K, pad, "dw")
        old = dw.to(torch.float32, copy=True)     # dw itself is added to
        zs.zs_linear_f8_backward(dy, x, w_t, dx, dw, ws, grad_type=kind, accumulate=True)
        assert torch.equal(dx, want[0].to(DTYPES[dtype])) and torch.equal(dw, (old + want[1]).to(DTYPES[dw_dtype]))


def test_gradients_against_differences():
    """The backward pass is the derivative of y = x w^T: for values that 8 bits hold exactly, of
    the sum over y * dy by differences of a whole step of one element."""
    dev = device()
    M, N, K = 9, 12, 20
    x, w, dy = whole(M, K, 1), whole(N, K, 2), whole(M, N, 3)
    loss = lambda x, w: float(((x.astype(np.float64) @ w.T) * dy).sum())
    dx, dw = torch.zeros(M, K, device=dev), torch.zeros(N, K, device=dev)
    w_t, _ = f8(np.ascontiguousarray(w.T), F.E4M3, 128)
    zs.zs_linear_f8_backward(on_device(dy, "f32")[0], on_device(x, "f32")[0], w_t, dx, dw,
                             workspace(M, N, K, zs.zs_linear_f8_backward_workspace))
    for i, j in ((0, 0), (3, 7), (8, 19)):
        for g, at in ((dx, x), (dw, w)):
            up = at.copy()
            up[i, j] += 1
            diff = (loss(up, w) if at is x else loss(x, up)) - loss(x, w)
            assert g[i, j].item() == diff


def test_empty_batch_gives_zero_gradients():
    dev = device()
    dw = torch.full((5, 6), 3.0, device=dev)
    empty = lambda n: torch.zeros(0, n, device=dev)
    ws = workspace(0, 5, 6, zs.zs_linear_f8_backward_workspace)
    zs.zs_linear_f8_backward(empty(5), empty(6), None, None, dw, ws, accumulate=True)
    assert bool((dw == 3).all())
    zs.zs_linear_f8_backward(empty(5), empty(6), None, None, dw, ws)
    assert bool((dw == 0).all())


# ----------------------------------------------------------------- as it is used
class Layer:
    """A unit of one matrix between two vectors, spread over D ranks: gathered in 8 bits, a
    layer's forward and backward pass, each rank's gradient into a flat contribution, the reduce
    with its norm, the clipped step, and the new working shards."""

    def __init__(self, D=3, M=70, N=90, K=130):
        dev = device()
        self.D, self.M, self.N, self.K = D, M, N, K
        _, self.n, self.n_pad, self.S = zs.zs_unit_layout([K, N * K, N], D)
        t = lambda x: torch.from_numpy(x).to(dev)
        self.p = [t(matrix(1, self.S, 10 + r, std=0.02)[0]) for r in range(D)]
        self.m, self.v = ([torch.zeros(self.S, device=dev) for _ in range(D)] for _ in range(2))
        self.w = [p.bfloat16() for p in self.p]
        self.x = [t(matrix(M, K, 20 + r)).bfloat16() for r in range(D)]
        self.dy = [t(matrix(M, N, 30 + r, std=1e-3)).bfloat16() for r in range(D)]
        self.w8, self.w8_t = zs.F8Matrix.empty(N, K, block_rows=128), zs.F8Matrix.empty(K, N, block_rows=128)
        self.y = [torch.zeros(M, N, dtype=torch.bfloat16, device=dev) for _ in range(D)]
        self.dx = [torch.zeros(M, K, dtype=torch.bfloat16, device=dev) for _ in range(D)]
        self.flat = [torch.zeros(self.n_pad, dtype=torch.bfloat16, device=dev) for _ in range(D)]
        self.g = [torch.zeros(self.S, device=dev) for _ in range(D)]
        self.sumsq = torch.zeros(1, dtype=torch.float64, device=dev)
        self.norm_coef = torch.zeros(2, device=dev)
        need = max(zs.zs_linear_f8_workspace(M, N, K), zs.zs_linear_f8_backward_workspace(M, N, K))
        self.ws = torch.zeros(need, dtype=torch.uint8, device=dev)
        self.norm_ws = torch.zeros(zs.ZS_NORM_WORKSPACE, dtype=torch.uint8, device=dev)

    def step(self, hp):
        N, K = self.N, self.K
        zs.zs_gather_matrix_f8(self.w, K, self.w8, self.w8_t)
        for r in range(self.D):
            zs.zs_linear_f8(self.x[r], self.w8, self.y[r], self.ws)
            dw = self.flat[r][K:K + N * K].view(N, K)
            zs.zs_linear_f8_backward(self.dy[r], self.x[r], self.w8_t, self.dx[r], dw, self.ws)
        for r in range(self.D):
            part = [f[r * self.S:(r + 1) * self.S] for f in self.flat]
            zs.zs_reduce_shard_norm(part, self.g[r], 0.05, self.sumsq, self.norm_coef, self.norm_ws,
                                    accumulate=r > 0)
        for r in range(self.D):
            zs.zs_adamw_step_clip(self.p[r], self.m[r], self.v[r], self.w[r], [self.g[r]], hp,
                                  self.norm_coef[1:])

    def state(self):
        return [*self.p, *self.m, *self.v, *self.w, *self.y, *self.dx, *self.flat, *self.g, self.sumsq,
                self.norm_coef]


HP = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)


def test_a_units_step_from_gather_to_clipped_update():
    L = Layer()
    h = [to_np(p).copy() for p in L.p]
    w = np.concatenate([to_np(x.float()) for x in L.w])[L.K:L.K + L.N * L.K].reshape(L.N, L.K)
    L.step(HP)
    vw = F.quantized(w, F.E4M3, 128)
    flats = []
    for r in range(L.D):
        x, dy = (to_np(t[r].float()) for t in (L.x, L.dy))
        for got, a, b in ((L.y[r], F.quantized(x), vw), (L.dx[r], F.quantized(dy), vw.T),
                          (L.flat[r][L.K:L.K + L.N * L.K].view(L.N, L.K), F.quantized(dy.T), F.quantized(x.T))):
            e, tol = tolerance(a, b, "bf16")
            assert (np.abs(got.double().cpu().numpy() - e) <= tol).all()
        flats.append(to_np(L.flat[r]))
    g = [O.reduce_shard([f[r * L.S:(r + 1) * L.S] for f in flats], O.BF16) for r in range(L.D)]
    total = F.sum_of_squares(g)
    assert abs(L.sumsq.item() - total) <= L.n_pad * 2.0**-53 * total
    norm, coef = (float(c) for c in L.norm_coef)
    assert 0 < coef < 1 and abs(coef - 0.05 / norm) < 1e-5
    for r in range(L.D):
        check_f32(to_np(L.g[r]), g[r], "g", exact=True)
        z = np.zeros(L.S, np.float32)
        p, m, v, wk = O.adamw_step(h[r], z, z, g[r] * np.float32(coef), O.AdamWHP(**HP))
        check_f32(to_np(L.p[r]), p, "p", exact=True)
        check_f32(to_np(L.m[r]), m, "m", exact=True)
        check_f32(to_np(L.v[r]), v, "v", exact=True)
        check_bf16(to_np(L.w[r]), wk, "w", exact=True)


def test_the_step_from_a_graph():
    """Captured once and replayed, with eager work of the same kind between the replays."""
    a, b = Layer(), Layer()
    Layer().step(HP)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        a.step(HP)
    torch.cuda.synchronize()
    for rep in range(4):
        for L in (a, b):
            for t in L.x + L.dy:
                t.mul_(1.25 if rep % 2 else 0.5)
        graph.replay()
        b.step(HP)
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(a.state(), b.state())), rep


def test_no_call_waits_or_allocates():
    run, warm = Layer(), Layer()
    warm.step(HP)
    busy = torch.zeros(1 << 30, device=device()).add_(1.0)
    torch.cuda.synchronize()
    free, held = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()
    done = torch.cuda.Event()
    for _ in range(60):
        busy.add_(1.0)
    done.record()
    run.step(HP)
    assert not done.query()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free and torch.cuda.memory_allocated() == held
    assert all(torch.equal(s, t) for s, t in zip(run.state(), warm.state()))


def test_two_streams_at_once():
    """Two layers at the same time, each with its own workspaces."""
    one, two, alone = Layer(), Layer(), Layer()
    alone.step(HP)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for L, s in zip((one, two), streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            L.step(HP)
    torch.cuda.synchronize()
    for L in (one, two):
        assert all(torch.equal(s, t) for s, t in zip(L.state(), alone.state()))


class Products:
    """Calls that split K, take few rows and make their codes on the way, on one workspace."""
    SIZES = [(70, 100, 4200), (3, 300, 1000), (1, 40, 20_000), (500, 700, 9000), (16, 260, 512)]

    def __init__(self, seed=1):
        dev = device()
        gen = torch.Generator(device=dev).manual_seed(seed)
        rand = lambda *n: torch.randn(*n, generator=gen, device=dev)
        self.x, self.w, self.y, self.c = [], [], [], []
        for M, N, K in self.SIZES:
            self.x.append(rand(M, K))
            self.w.append(zs.F8Matrix.empty(N, K, block_rows=128))
            zs.zs_quantize_f8(rand(N, K), self.w[-1])
            self.y.append(torch.zeros(M, N, dtype=torch.bfloat16, device=dev))
            self.c.append(torch.zeros(M, N, device=dev))
        need = max(f(*n) for n in self.SIZES for f in (zs.zs_matmul_f8_workspace, zs.zs_linear_f8_workspace))
        assert need > zs.zs_linear_f8_workspace(70, 100, 4200) > 70 * 4200
        self.ws = torch.zeros(need, dtype=torch.uint8, device=dev)
        self.a = [zs.F8Matrix.empty(M, K, zs.ZS_E5M2) for M, _, K in self.SIZES]

    def run(self):
        for x, w, y, c, a in zip(self.x, self.w, self.y, self.c, self.a):
            zs.zs_linear_f8(x, w, y, self.ws)
            zs.zs_quantize_f8(x, a)
            zs.zs_matmul_f8(a, w, c, accumulate=True, workspace=self.ws)

    def same(self, other):
        return all(torch.equal(a, b) for a, b in zip(self.y + self.c, other.y + other.c))


def test_products_from_a_graph():
    run, eager = Products(), Products()
    Products(2).run()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        run.run()
    torch.cuda.synchronize()
    for rep in range(4):
        for r in (run, eager):
            for x in r.x:
                x.mul_(-1.5)
        graph.replay()
        eager.run()
        torch.cuda.synchronize()
        assert run.same(eager), rep


def test_products_on_two_streams():
    """At the same time, each with a workspace of its own, behind work of the stream."""
    one, two, alone = Products(), Products(), Products()
    for _ in range(3):
        alone.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for r, s in zip((one, two), streams):
            with torch.cuda.stream(s):
                r.run()
    torch.cuda.synchronize()
    assert one.same(alone) and two.same(alone)
    zs.zs_linear_f8(one.x[0], one.w[0], one.y[0], one.ws, stream=streams[0])
    streams[0].synchronize()
    assert one.same(alone)


def test_refusals_on_the_device():
    dev = device()
    x = torch.zeros(64, 256, device=dev)
    out, out_t = zs.F8Matrix.empty(64, 256), zs.F8Matrix.empty(256, 64)
    bad = [lambda: zs.zs_quantize_f8(x), lambda: zs.zs_quantize_f8(x, zs.F8Matrix.empty(64, 255)),
           lambda: zs.zs_quantize_f8(x.t(), out_t), lambda: zs.zs_quantize_f8(x.half(), out),
           lambda: zs.zs_quantize_f8(x.cpu(), out), lambda: zs.zs_quantize_f8(x[0], out),
           lambda: zs.F8Matrix(out.codes[1:], out.scales, 64, 256),
           lambda: zs.F8Matrix(out.codes, out.scales.float(), 64, 256),
           lambda: zs.F8Matrix(out.codes, out.scales[::2], 64, 256),
           lambda: zs.zs_gather_matrix_f8([], 0, out), lambda: zs.zs_gather_matrix_f8([x, x.view(-1)[1:]], 0, out),
           lambda: zs.zs_dequantize_f8(out, x[:, :255]), lambda: zs.zs_matmul_f8(out, out_t, x),
           lambda: zs.zs_matmul_f8(out, out, x), lambda: zs.zs_linear_f8(x, out, x[:, :64], None),
           lambda: zs.zs_linear_f8(x, out_t, x, out.codes[:0]),
           lambda: zs.zs_linear_f8(x, out, torch.zeros(64, 64, device=dev), out.codes[:100]),
           lambda: zs.zs_linear_f8_backward(x, x, None, None, None, out.codes)]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            print("call", i, "was not refused")
    ws = workspace(64, 64, 256, zs.zs_linear_f8_backward_workspace)
    dy, dw = torch.zeros(64, 64, device=dev), torch.zeros(64, 256, device=dev)
    for call in (lambda: zs.zs_linear_f8_backward(dy, None, None, None, dw, ws),
                 lambda: zs.zs_linear_f8_backward(dy, x, None, x.clone(), dw, ws),
                 lambda: zs.zs_linear_f8_backward(dy, x.bfloat16(), None, None, dw, ws)):
        with pytest.raises((ValueError, TypeError)):
            call()
    for name, value in (("codes", out_t.codes), ("scales", out_t.scales), ("rows", 3), ("type", zs.ZS_E5M2)):
        with pytest.raises(AttributeError):
            setattr(out, name, value)
    for call in (lambda: zs.zs_quantize_f8(x, zs.F8Matrix(out.codes, out.scales, 64, 256, 9)),
                 lambda: zs.zs_gather_matrix_f8([x.view(-1)], 1, out)):
        with pytest.raises(zs.ZsError):
            call()


def test_rows_past_32_bits_of_codes():
    """Operands of more than 2^32 bytes of codes: the first and last rows of a tall product."""
    dev = device()
    K, M = 1 << 20, 4200
    a = zs.F8Matrix.empty(M, K)
    a.codes.zero_()
    a.scales.fill_(127)
    rows = (0, 1, 4095, 4096, 4199)
    one = np.full((1, K), 0, np.float32)
    for i, r in enumerate(rows):
        line = a.codes.view(M, -1)[r]
        line[::1 << 17] = 0x38 + 8 * i                # 2^i, eight times
    b = zs.F8Matrix.empty(3, K)
    b.codes.fill_(0x38)                               # 1
    b.scales.fill_(128)                               # times 2
    for dtype in DTYPES:
        _, _, c = out_matrix(M, 3, dtype)
        zs.zs_matmul_f8(a, b, c, workspace=workspace(M, 3, K))
        want = torch.zeros(M, 3)
        for i, r in enumerate(rows):
            want[r] = 8 * 2.0 ** i * 2
        assert torch.equal(c.float().cpu(), want)
    v = torch.zeros(M, K, dtype=torch.bfloat16, device=dev)
    zs.zs_dequantize_f8(a, v)
    q, q_t = zs.F8Matrix.empty(M, K, block_rows=128), zs.F8Matrix.empty(K, M, block_rows=128)
    zs.zs_quantize_f8(v, q, q_t)
    back = torch.zeros_like(v)
    zs.zs_dequantize_f8(q, back)
    assert torch.equal(back, v)
    del back
    back_t = torch.zeros(K, M, dtype=torch.bfloat16, device=dev)
    zs.zs_dequantize_f8(q_t, back_t)
    assert torch.equal(back_t[::1 << 17].t(), v[:, ::1 << 17]) and back_t.count_nonzero() == v.count_nonzero()
