"""Build libzs.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libzs.so")
SOURCES = ("zs_api.cpp", "zs_pipeline.cpp", "zs_ckpt.cpp", "zs_host.cpp", "zs_step.hip",
           "zs_move.hip", "zs_diag.hip", "zs_static.hip", "zs_multi.cpp", "zs_multi.hip",
           "zs_mx4.hip", "zs_f8.cpp", "zs_f8_quant.hip", "zs_f8_gemm.hip",
           "zs_f8_few.hip")

# -ffp-contract=off: no fused multiply-add in the step's arithmetic;
# correctly rounded fp32 divide and sqrt (the HIP default, stated);
# packed fp32 VALU ops disabled; symbols hidden except the C ABI.
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fvisibility=hidden", "-Wall", "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found: the HIP toolchain is required to build libzs")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.run(cmd, capture_output=True, text=True)


def build(out: str = LIB, defines: tuple = (), verbose: bool = False) -> str:
    """Compile every source, a few at a time, and link them."""
    tmp = out + ".tmp%d" % os.getpid()
    flags = [f for f in FLAGS if f != "-shared"] + ["-D" + d for d in defines]
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, s + ".o") for s in SOURCES]
        cmds = [[hipcc()] + flags + ["-c", "-x", "hip", os.path.join(CSRC, s), "-o", o]
                for s, o in zip(SOURCES, objects)]
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            runs = list(pool.map(lambda c: _run(c, verbose), cmds))
        if all(r.returncode == 0 for r in runs):
            runs.append(_run([hipcc()] + FLAGS + objects + ["-o", tmp], verbose))
    for r in runs:
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("hipcc failed building %s" % out)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
