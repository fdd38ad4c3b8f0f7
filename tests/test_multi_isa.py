"""Properties of the gfx950 code that zs_multi.hip and zs_mx4.hip compile to (hipcc's
assembly output with the library's own flags; CPU only), and their launch geometry.

- No packed fp32 VALU instruction, no spill to scratch, no flat load or store (the
  tables' pointers are global memory), no warning about alignment.
- The step kernels issue their loads in long runs before a wait: with 8-bit moments a
  wavefront's 16 wide loads, between the 2 scale bytes' loads and the wait for those;
  with fp32 moments (where forcing all 16 first measured slower) at least 8.
- Tensors at odd element offsets use the same wide instructions (an access split into
  elements would show as byte and short loads outnumbering the tails').
"""
import os
import re
import shutil
import subprocess

import pytest

from fsdp_sharded_optimizer_zs_amd import build as B

HIPCC = next((c for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc"))
              if c and os.path.exists(c)), None)
SOURCES = ("zs_multi.hip", "zs_mx4.hip")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if HIPCC is None:
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("isa")
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    out = {}
    for src in SOURCES:
        dst = d / (src + ".s")
        r = subprocess.run([HIPCC] + flags + ["--cuda-device-only", "-S", "-x", "hip",
                                              os.path.join(B.CSRC, src), "-o", str(dst)],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        out[src] = (dst.read_text(), r.stderr)
    return out


def kernels(text):
    return [(m.group(1), text[m.end():text.find(".Lfunc_end", m.end())])
            for m in re.finditer(r"^(_Z\S+):\s*(?:;.*)?$", text, re.M)]


@pytest.mark.slow
def test_no_packed_fp32_scratch_or_flat_access(asm):
    for src, (text, warnings) in asm.items():
        assert not re.findall(r"^\s*(v_pk_(?:add|mul|fma)_f32)\b", text, re.M), src
        sizes = re.findall(r"\.private_segment_fixed_size:\s*(\d+)", text)
        assert sizes and all(int(x) == 0 for x in sizes), src
        assert not re.findall(r"^\s*(flat_(?:load|store|atomic)\w*)", text, re.M), src
        assert "align-mismatch" not in warnings, src


@pytest.mark.slow
def test_step_kernels_load_in_long_runs(asm):
    text = asm["zs_multi.hip"][0]
    for pat, want in ((r"multi32_kernelILi[12]E", 8), (r"multi8_kernelILi[12]ELb[01]ELb0E", 16)):
        found = [(n, b) for n, b in kernels(text) if re.search(pat, n)]
        assert len(found) == 4, [n for n, _ in found]
        for n, body in found:
            longest = run = 0
            for op in re.findall(r"^\s*(global_load_dword\w*|s_waitcnt\s+vmcnt|s_cbranch)", body, re.M):
                run = run + 1 if op.startswith("global_load") else 0
                longest = max(longest, run)
            assert longest >= want, f"{n}: {longest} loads before a wait"


@pytest.mark.slow
def test_four_bit_conversions_are_the_hardwares(asm):
    text = asm["zs_mx4.hip"][0]
    for op, n in (("v_cvt_scalef32_pk_fp4_bf16", 4), ("v_cvt_scalef32_pk_fp4_f32", 4),
                  ("v_cvt_scalef32_pk_bf16_fp4", 4), ("v_cvt_scalef32_pk_f32_fp4", 4)):
        assert len(re.findall(r"^\s*%s\b" % op, text, re.M)) >= n, op


# ------------------------------------------------------------------ geometry
DRIVER = r"""
#include <cstdio>
#include "zs_multi_grid.h"
using namespace zs;
int main() {
    long long a, b;
    while (std::scanf("%lld %lld", &a, &b) == 2)
        std::printf("%lld %lld %lld %lld %lld %lld %lld\n", (long long)state8_grid(a, 4),
                    (long long)state8_grid(a, 2),
                    (long long)norm_grid(a), (long long)quantize_mx4_grid(a, 2),
                    (long long)quantize_mx4_grid(a, 4), (long long)gather_mx4_grid(a, 2, int(b)),
                    (long long)gather_mx4_grid(a, 4, int(b)));
    return 0;
}
"""
MAXG = (2**32 - 1) // 256


def test_grids_are_legal_and_cover_the_work(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    (tmp_path / "d.cpp").write_text(DRIVER)
    subprocess.run([cxx, "-std=c++17", "-I", B.CSRC, str(tmp_path / "d.cpp"), "-o",
                    str(tmp_path / "d")], check=True)
    sizes = [0, 1, 7, 255, 1023, 1024, 1025, 8191, 8192, 8193, 2**24, 2**31 - 1, 2**31, 2**32,
             2**36, 2**45, (2**63 - 1) // 64]
    cases = [(s, D) for s in sizes for D in (1, 3, 8, 64)]
    out = subprocess.run([str(tmp_path / "d")], input="".join("%d %d\n" % c for c in cases),
                         capture_output=True, text=True, check=True).stdout.split("\n")
    for (s, D), line in zip(cases, out):
        wide, narrow, norm, *mx4 = (int(x) for x in line.split())
        for blocks, units, per in ((wide, s, 4096), (narrow, s, 2048), (mx4[0], s, 4096), (mx4[1], s, 2048)):
            assert 1 <= blocks <= MAXG and (blocks == MAXG or blocks * per >= units)
        assert 1 <= norm <= 512 and (norm == 512 or norm * 4 >= s)
        for gather, per in ((mx4[2], 4096), (mx4[3], 2048)):     # the grid is gather x D
            assert 1 <= gather and gather * D <= MAXG
            assert gather == MAXG // D or gather * per >= s
