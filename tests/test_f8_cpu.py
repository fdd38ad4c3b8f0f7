"""Block-scaled 8-bit matrices and the clipped step on the host: the oracle's codes by brute
force, the layout, and every refusal before anything is enqueued."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import fsdp_sharded_optimizer_zs_amd as zs
from fsdp_sharded_optimizer_zs_amd import _binding as B
from fsdp_sharded_optimizer_zs_amd import build as BUILD
from oracle import zs_f8 as F

KINDS = (F.E4M3, F.E5M2)
A = 0x7f0000000000        # fake device addresses, never read: every call fails in validation


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        BUILD.build()
    return zs.load()


def no_gpu():
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("fake-address validation tests run only where no GPU is visible")


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("kind,top,least", [(F.E4M3, 448.0, 2.0**-9), (F.E5M2, 57344.0, 2.0**-16)])
def test_code_values(kind, top, least):
    v = F.code_values(kind)
    fin = v[np.isfinite(v)]
    assert fin.max() == top and fin[fin > 0].min() == least
    assert np.array_equal(v[:128][np.isfinite(v[:128])], np.sort(fin[~np.signbit(fin)]))
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(
        torch.float8_e4m3fn if kind == F.E4M3 else torch.float8_e5m2).double().numpy()
    assert np.array_equal(t, v, equal_nan=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("exp", (-140, -127, -118, -20, 0, 60, 127))
def test_quantize_picks_the_nearest_code(kind, exp):
    """Against a search over every code's value."""
    rng = np.random.default_rng(exp + 200)
    x = (rng.standard_normal((3, 128)) * 2.0**exp).astype(np.float32)
    x = np.clip(x, -3e38, 3e38)
    grid = F.code_values(kind)
    grid = np.unique(np.abs(grid[np.isfinite(grid)]))
    codes, scales = F.quantize(x, kind)
    v = F.values(codes, scales, 3, 128, kind)
    for r in range(3):
        top = np.abs(x[r].astype(np.float64)).max()
        fits = [s for s in range(1, 255) if top <= grid[-1] * 2.0**(s - 127)]
        assert scales[r, 0] == fits[0]
        near = grid * 2.0**(int(scales[r, 0]) - 127)
        d = np.abs(np.abs(x[r].astype(np.float64))[:, None] - near)
        assert np.array_equal(np.abs(np.abs(x[r].astype(np.float64)) - np.abs(v[r])), d.min(axis=1))
        tie = np.isclose(np.sort(d, axis=1)[:, 0], np.sort(d, axis=1)[:, 1], rtol=0, atol=0)
        assert (codes[r, :128][tie] & 1 == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_quantizing_values_again_changes_nothing(kind):
    x = np.random.default_rng(3).standard_normal((5, 300)).astype(np.float32)
    v = F.quantized(x, kind).astype(np.float32)
    assert np.array_equal(F.quantized(v, kind), v.astype(np.float64))


def test_square_blocks_are_the_transposes_blocks():
    x = np.random.default_rng(4).standard_normal((200, 300)).astype(np.float32)
    assert np.array_equal(F.quantized(x, F.E4M3, 128), F.quantized(x.T, F.E4M3, 128).T)


def test_specials():
    x = np.zeros((4, 256), np.float32)
    x[0, 5], x[1, 200], x[2, 3] = np.nan, np.inf, -0.0
    codes, scales = F.quantize(x, F.E4M3)
    assert scales[:, :2].tolist() == [[255, 1], [1, 255], [1, 1], [1, 1]]
    assert codes[2, 3] == 0x80 and not codes[0].any()


def test_product_by_hand():
    a, b = np.array([[1.0, -2, 3]]), np.array([[4.0, 5, 6], [0, 1, 0]])
    e, m, t = F.product(a, b)
    assert e.tolist() == [[12, -2]] and m.tolist() == [[32, 2]] and t.tolist() == [[18, 2]]


# ------------------------------------------------------------------- the host
def test_layout(lib):
    for rows, cols, br in ((0, 0, 1), (1, 1, 1), (3, 128, 1), (129, 129, 128), (1000, 513, 1),
                           (1000, 512, 128), (2**31 - 1, 2**22, 1)):
        want = rows * F.ceil(cols, 128) * 128, F.ceil(rows, br) * 4 * F.ceil(cols, 512)
        assert zs.zs_f8_layout(rows, cols, br) == want
    for bad in ((-1, 1, 1), (1, -1, 1), (2**31, 1, 1), (1, 2**22 + 1, 1), (1, 1, 2), (1, 1, 64)):
        with pytest.raises(zs.ZsError) as e:
            zs.zs_f8_layout(*bad)
        assert e.value.status == zs.ZS_EINVAL


def test_workspace_sizes(lib):
    for f in (zs.zs_matmul_f8_workspace, zs.zs_linear_f8_workspace, zs.zs_linear_f8_backward_workspace):
        for M, N, K in ((0, 0, 0), (1, 1, 1), (1, 4096, 11008), (256, 256, 2**22), (4096, 11008, 4096)):
            assert 0 <= f(M, N, K) < 2**34
        with pytest.raises(zs.ZsError):
            f(1, 1, 2**22 + 1 if f is not zs.zs_linear_f8_backward_workspace else 2**31)
        with pytest.raises(zs.ZsError):
            f(-1, 1, 1)


def mat(codes=A, scales=A + 0x10000000, rows=64, cols=256, type=zs.ZS_E4M3, block_rows=1):
    return B.zs_f8_matrix(codes, scales, rows, cols, type, block_rows)


def ref(x):
    return None if x is None else ctypes.byref(x)


X, OUT, OUTT = A + 0x20000000, mat(), mat(A + 0x40000000, A + 0x50000000, 256, 64)


def quantize(lib, x=X, dtype=zs.ZS_BF16, ldx=256, out=OUT, out_t=OUTT):
    return lib.zs_quantize_f8(x, dtype, ldx, ref(out), ref(out_t), None)


def test_quantize_refusals(lib):
    no_gpu()
    assert quantize(lib, dtype=7) == zs.ZS_EUNSUPPORTED
    assert quantize(lib, out=mat(type=zs.ZS_BF16)) == zs.ZS_EUNSUPPORTED
    for kw in (dict(out=None, out_t=None), dict(x=None), dict(x=X + 1), dict(ldx=255), dict(ldx=2**62),
               dict(out=mat(codes=None)), dict(out=mat(scales=None)), dict(out=mat(codes=A + 8)),
               dict(out=mat(scales=A + 0x10000001)), dict(out=mat(rows=-1)), dict(out=mat(cols=2**22 + 1)),
               dict(out=mat(rows=2**31)), dict(out=mat(block_rows=2)), dict(out=mat(block_rows=128)),
               dict(out_t=mat(A + 0x40000000, A + 0x50000000, 256, 65))):
        assert quantize(lib, **kw) == zs.ZS_EINVAL, kw
        assert "zs_quantize_f8" in zs.zs_last_error()
    for kw in (dict(x=A), dict(x=A + 0x10000000), dict(out=mat(scales=A + 64)),
               dict(out_t=mat(A + 1024, A + 0x50000000, 256, 64)),
               dict(out_t=mat(A + 0x40000000, A + 0x10000004, 256, 64)), dict(x=A + 0x50000000 - 256)):
        assert quantize(lib, **kw) == zs.ZS_EALIAS, kw
    assert quantize(lib, x=None, out=mat(rows=0, codes=None, scales=None), out_t=None) == zs.ZS_OK
    assert quantize(lib, x=None, out=None, out_t=mat(cols=0, codes=None, scales=None)) == zs.ZS_OK


def gather(lib, shards=(X, X + 0x100000), S=10_000, dtype=zs.ZS_BF16, offset=5, out=OUT, out_t=None, D=None):
    arr = (ctypes.c_void_p * max(1, len(shards)))(*shards)
    return lib.zs_gather_matrix_f8(arr, len(shards) if D is None else D, S, dtype, offset, ref(out),
                                   ref(out_t), None)


def test_gather_refusals(lib):
    no_gpu()
    assert gather(lib, dtype=0) == zs.ZS_EUNSUPPORTED
    for kw in (dict(D=0), dict(D=65), dict(S=-1), dict(S=2**53), dict(offset=-1), dict(offset=20_000 - 64 * 256 + 1),
               dict(offset=2**62), dict(out=None), dict(shards=(X, None)), dict(shards=(X, X + 1)),
               dict(S=8191)):
        assert gather(lib, **kw) == zs.ZS_EINVAL, kw
    assert gather(lib, shards=(X, A + 100)) == zs.ZS_EALIAS
    assert gather(lib, S=0, offset=0, shards=(), D=1, out=mat(rows=0, codes=None)) == zs.ZS_OK


def test_dequantize_refusals(lib):
    no_gpu()
    f = lambda x=OUT, dtype=zs.ZS_F32, out=X, ld=256: lib.zs_dequantize_f8(ref(x), dtype, out, ld, None)
    assert f(dtype=3) == zs.ZS_EUNSUPPORTED
    for kw in (dict(x=None), dict(out=None), dict(out=X + 2), dict(ld=255)):
        assert f(**kw) == zs.ZS_EINVAL, kw
    assert f(out=A) == zs.ZS_EALIAS and f(x=mat(cols=0), out=None) == zs.ZS_OK


BM = mat(A + 0x40000000, A + 0x50000000, 32, 256)


def matmul(lib, a=OUT, b=BM, dtype=zs.ZS_BF16, c=X, ldc=32, acc=0, ws=A + 0x60000000):
    return lib.zs_matmul_f8(ref(a), ref(b), dtype, c, ldc, acc, ws, None)


def test_matmul_refusals(lib):
    no_gpu()
    assert matmul(lib, dtype=3) == zs.ZS_EUNSUPPORTED
    assert matmul(lib, b=mat(type=9)) == zs.ZS_EUNSUPPORTED
    big = mat(rows=1 << 26), mat(A + 0x40000000, A + 0x50000000, 1 << 26, 256)
    for kw in (dict(a=None), dict(b=mat(cols=128)), dict(c=None), dict(c=X + 1), dict(ldc=31), dict(acc=2),
               dict(a=mat(codes=A + 1)), dict(ws=A + 0x60000008, a=mat(rows=20, cols=2**20),
                                              b=mat(A + 0x40000000, A + 0x50000000, 1, 2**20)),
               dict(a=big[0], b=big[1], ldc=1 << 26)):
        assert matmul(lib, **kw) == zs.ZS_EINVAL, kw
    for kw in (dict(c=A), dict(c=A + 0x50000000)):
        assert matmul(lib, **kw) == zs.ZS_EALIAS, kw
    long = mat(rows=64, cols=2**16), mat(A + 0x40000000, A + 0x50000000, 32, 2**16)
    assert zs.zs_matmul_f8_workspace(64, 32, 2**16) > 0
    for ws in (X, A, A + 0x50000000):
        assert matmul(lib, *long, ws=ws) == zs.ZS_EALIAS, hex(ws)
    assert matmul(lib, *long, ws=None) == zs.ZS_EINVAL
    assert matmul(lib, a=mat(rows=0, codes=None), c=None) == zs.ZS_OK
    assert matmul(lib, b=mat(rows=0, codes=None), c=None) == zs.ZS_OK


def linear(lib, x=X, dtype=zs.ZS_BF16, M=40, ldx=256, type=zs.ZS_E4M3, w=OUT, yt=zs.ZS_BF16,
           y=A + 0x40000000, ldy=64, ws=A + 0x60000000):
    return lib.zs_linear_f8(x, dtype, M, ldx, type, ref(w), yt, y, ldy, ws, None)


def test_linear_refusals(lib):
    no_gpu()
    for kw in (dict(dtype=0), dict(yt=5), dict(type=1)):
        assert linear(lib, **kw) == zs.ZS_EUNSUPPORTED, kw
    for kw in (dict(x=None), dict(M=-1), dict(M=2**31), dict(ldx=255), dict(w=None), dict(y=None), dict(ldy=63),
               dict(ws=None), dict(ws=A + 0x60000001), dict(w=mat(block_rows=3))):
        assert linear(lib, **kw) == zs.ZS_EINVAL, kw
    for kw in (dict(y=X), dict(y=A), dict(ws=X), dict(ws=A + 0x40000000), dict(ws=A + 0x10000000)):
        assert linear(lib, **kw) == zs.ZS_EALIAS, kw
    assert linear(lib, M=0, x=None, y=None) == zs.ZS_OK
    # few rows need no workspace, and are refused what others are
    assert zs.zs_linear_f8_workspace(16, 64, 256) == 0 < zs.zs_linear_f8_workspace(17, 64, 256)
    for kw in (dict(x=None), dict(ldx=255), dict(y=None), dict(w=None)):
        assert linear(lib, M=16, ws=None, **kw) == zs.ZS_EINVAL, kw
    for y in (X, A, A + 0x10000000):
        assert linear(lib, M=16, ws=None, y=y) == zs.ZS_EALIAS


WT = mat(rows=256, cols=64)       # K x N of dy 8 x 64, x 8 x 256


def backward(lib, dy=X, lddy=64, x=X + 0x10000, ldx=256, dtype=zs.ZS_BF16, M=8, N=64, K=256, kind=zs.ZS_E5M2,
             w_t=WT, dxt=zs.ZS_BF16, dx=A + 0x40000000, lddx=256, dwt=zs.ZS_F32, dw=A + 0x41000000, lddw=256,
             acc=0, ws=A + 0x60000000):
    return lib.zs_linear_f8_backward(dy, lddy, x, ldx, dtype, M, N, K, kind, ref(w_t), dxt, dx, lddx, dwt, dw,
                                     lddw, acc, ws, None)


def test_backward_refusals(lib):
    no_gpu()
    for kw in (dict(dtype=0), dict(dxt=0), dict(dwt=9), dict(kind=2)):
        assert backward(lib, **kw) == zs.ZS_EUNSUPPORTED, kw
    for kw in (dict(dy=None), dict(x=None), dict(lddy=63), dict(ldx=255), dict(lddx=255), dict(lddw=255),
               dict(dx=None, dw=None), dict(w_t=None), dict(w_t=mat(rows=64, cols=256)), dict(acc=-1),
               dict(ws=None), dict(M=-1), dict(dw=A + 0x41000002), dict(M=2**23), dict(N=2**31)):
        assert backward(lib, **kw) == zs.ZS_EINVAL, kw
    for kw in (dict(dx=X), dict(dw=X + 0x10000), dict(dw=A), dict(dx=A + 0x10000000), dict(ws=X),
               dict(dw=A + 0x40000000), dict(ws=A), dict(ws=A + 0x41000000)):
        assert backward(lib, **kw) == zs.ZS_EALIAS, kw


HP = B.zs_adamw_hp(1e-3, 0.9, 0.95, 1e-8, 0.1, 1)


def test_reduce_norm_refusals(lib):
    no_gpu()
    S, g, sq, nc, ws = 1024, A, A + 0x10000, A + 0x10100, A + 0x20000
    c = (ctypes.c_void_p * 2)(A + 0x30000, A + 0x40000)

    def f(D=2, opts=None, dtype=zs.ZS_F32, S=S, g=g, mx=1.0, sq=sq, nc=nc, acc=0, ws=ws, c=c):
        return lib.zs_reduce_shard_norm(c, D, opts, dtype, S, g, mx, sq, nc, acc, ws, None)

    assert f(dtype=3) == zs.ZS_EUNSUPPORTED
    for kw in (dict(D=0), dict(S=-1), dict(g=None), dict(g=A + 2), dict(mx=0.0), dict(mx=float("nan")),
               dict(sq=None), dict(sq=A + 0x10004), dict(nc=A + 0x10102), dict(acc=2), dict(ws=None),
               dict(ws=A + 0x20008), dict(c=None)):
        assert f(**kw) == zs.ZS_EINVAL, kw
    for kw in (dict(sq=A), dict(nc=A + 4), dict(ws=A), dict(sq=A + 0x30008), dict(nc=A + 0x30008),
               dict(ws=A + 0x40000), dict(nc=sq), dict(sq=ws + 8), dict(nc=ws), dict(g=A + 0x30000)):
        assert f(**kw) == zs.ZS_EALIAS, kw


def test_clip_step_refusals(lib):
    no_gpu()
    p, m, v, w, S = A, A + 0x10000, A + 0x20000, A + 0x30000, 1024
    c = (ctypes.c_void_p * 1)(A + 0x40000)

    def f(scale=A + 0x50000, p=p, hp=HP, D=1, S=S):
        return lib.zs_adamw_step_clip(p, m, v, w, S, c, D, None, zs.ZS_F32, ref(hp), scale, None)

    for kw in (dict(scale=None), dict(scale=A + 0x50001), dict(p=None), dict(hp=None), dict(D=65), dict(S=-1)):
        assert f(**kw) == zs.ZS_EINVAL, kw
    for s in (p, m + 4, v + 4092, w + 2044):
        assert f(scale=s) == zs.ZS_EALIAS, hex(s)
    assert f(p=m) == zs.ZS_EALIAS and f(S=0, p=None) == zs.ZS_OK


# -------------------------------------------------------------------- geometry
DRIVER = r"""
#include <cstdio>
#include "zs_f8_grid.h"
#include "zs_multi_grid.h"
using namespace zs;
int main() {
    long long M, N, K;
    while (std::scanf("%lld %lld %lld", &M, &N, &K) == 3) {
        const F8Plan p = f8_plan(M, N, K);
        std::printf("%d %d %d %lld %lld %lld ", p.tm, p.tn, p.splits, (long long)p.tiles_m,
                    (long long)p.tiles_n, (long long)f8_partial_bytes(p));
        std::printf("%lld %lld %lld %lld %lld\n", (long long)f8_matmul_workspace(M, N, K), (long long)kF8Counts,
                    (long long)kF8CountBytes, (long long)reduce_norm_grid(M * K, 2),
                    (long long)reduce_norm_grid(M * K, 0));
    }
    return 0;
}
"""


def test_plans_cover_the_work_and_fit_the_workspace(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    (tmp_path / "d.cpp").write_text(DRIVER)
    subprocess.run([cxx, "-std=c++17", "-I", BUILD.CSRC, str(tmp_path / "d.cpp"), "-o", str(tmp_path / "d")],
                   check=True)
    sizes = (0, 1, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 256, 1000, 1024, 4096, 11008, 65536)
    cases = [(m, n, k) for m in sizes for n in sizes for k in (0, 1, 128, 129, 1024, 4096, 11008, 2**22)]
    cases += [(2**31 - 1, 1, 1), (1, 2**31 - 1, 128), (2**20, 2**20, 4096)]
    out = subprocess.run([str(tmp_path / "d")], input="".join("%d %d %d\n" % c for c in cases),
                         capture_output=True, text=True, check=True).stdout.split("\n")
    for (M, N, K), line in zip(cases, out):
        v = [int(x) for x in line.split()]
        tm, tn, splits, tiles_m, tiles_n, partial, need, counts, count_bytes, aligned, scalar = v
        assert tiles_m * tm >= M and tiles_n * tn >= N and (tiles_m - 1) * tm < max(M, 1)
        assert 1 <= splits <= max(1, -(-K // 128))
        if tm == 16:
            assert M <= 16 and need == partial == 0 and splits in (1, 2, 4, 8) and tiles_n <= 256
        elif splits > 1:
            assert tiles_m * tiles_n <= counts
            assert partial == tiles_m * tiles_n * splits * tm * tn * 4 and need >= count_bytes + partial
        assert count_bytes >= 2 * counts * 4 and need < 2**31
        for grid in (aligned, scalar):
            assert 1 <= grid <= 512
