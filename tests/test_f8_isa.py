"""Properties of the gfx950 code that the 8-bit matrices' kernels compile to (hipcc's assembly
output with the library's own flags; CPU only).

- No packed fp32 VALU instruction, no spill to scratch, no flat load or store.
- Loads from memory to LDS are hand-written: the register that holds their LDS address is
  written by them alone, one wait state ahead of the load, so that no code of the compiler's
  finds it changed.
- The products' loops wait for a counted number of loads, never for all, and hold their
  matrix instructions: 8-bit ones for C in bf16, bf16 ones for C in fp32.
"""
import os
import re
import subprocess

import pytest

from fsdp_sharded_optimizer_zs_amd import build as B
from test_multi_isa import HIPCC, kernels

SOURCES = ("zs_f8_quant.hip", "zs_f8_gemm.hip", "zs_f8_few.hip")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if HIPCC is None:
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("isa8")
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    runs = {src: subprocess.Popen([HIPCC] + flags + ["--cuda-device-only", "-S", "-x", "hip", os.path.join(B.CSRC, src),
                                                     "-o", str(d / (src + ".s"))], stderr=subprocess.PIPE, text=True)
            for src in SOURCES}
    out = {}
    for src, p in runs.items():
        err = p.communicate()[1]
        assert p.returncode == 0, err[-2000:]
        out[src] = ((d / (src + ".s")).read_text(), err)
    return out


@pytest.mark.slow
def test_no_packed_fp32_scratch_or_flat_access(asm):
    for src, (text, warnings) in asm.items():
        assert not re.findall(r"^\s*(v_pk_(?:add|mul|fma)_f32)\b", text, re.M), src
        sizes = re.findall(r"\.private_segment_fixed_size:\s*(\d+)", text)
        assert sizes and all(int(x) == 0 for x in sizes), src
        assert not re.findall(r"^\s*(flat_(?:load|store|atomic)\w*)", text, re.M), src
        assert "align-mismatch" not in warnings, src


@pytest.mark.slow
def test_loads_to_lds_own_their_address_register(asm):
    for src in ("zs_f8_gemm.hip", "zs_f8_few.hip"):
        ops = [line.split(";")[0].strip() for line in asm[src][0].split("\n")]
        ops = [o for o in ops if re.match(r"[a-z]\w*(\s|$)", o)]
        loads = [i for i, o in enumerate(ops) if o.startswith("global_load_lds")]
        assert len(loads) > 100
        for i in loads:
            assert re.match(r"s_mov_b32 m0, s\d+$", ops[i - 2]) and re.match(r"s_nop 0", ops[i - 1]), ops[i - 2:i + 1]
        assert sum(bool(re.search(r"\bm0\b", o)) for o in ops) == len(loads), src


@pytest.mark.slow
def test_products_use_their_matrix_instructions(asm):
    found = [(n, b) for n, b in kernels(asm["zs_f8_gemm.hip"][0]) if "matmul" in n]
    assert len(found) == 2 * 3 * 4 * 2
    eights = 0
    for n, body in found:
        eight = len(re.findall(r"^\s*v_mfma_scale_f32_32x32x64_f8f6f4", body, re.M))
        wide = len(re.findall(r"^\s*v_mfma_f32_32x32x16_bf16", body, re.M))
        assert (eight > 0) != (wide > 0), n
        eights += eight > 0
        # the wait before the barrier that opens a half step leaves loads under way
        for m in re.finditer(r"^\s*v_mfma", body, re.M):
            before = body[:body.rfind("s_barrier", 0, m.start())]
            assert int(re.findall(r"s_waitcnt[^\n]*vmcnt\((\d+)\)", before)[-1]) > 0, n
    assert eights == len(found) // 2
    few = [(n, b) for n, b in kernels(asm["zs_f8_few.hip"][0]) if "few_kernel" in n]
    assert len(few) == 2 * 3 * 4 * 2
    assert sum("v_mfma_scale_f32_16x16x128_f8f6f4" in b for _, b in few) == len(few) // 2
    assert sum("v_mfma_f32_16x16x32_bf16" in b for _, b in few) == len(few) // 2


@pytest.mark.slow
def test_conversions_are_the_hardwares(asm):
    text = asm["zs_f8_quant.hip"][0]
    for op in ("v_cvt_scalef32_pk_fp8_bf16", "v_cvt_scalef32_pk_bf8_bf16", "v_cvt_scalef32_pk_fp8_f32",
               "v_cvt_scalef32_pk_bf8_f32", "v_cvt_pk_f32_fp8", "v_cvt_pk_f32_bf8"):
        assert len(re.findall(r"^\s*%s(?:_e32|_sdwa)?\b" % op, text, re.M)) >= 4, op
