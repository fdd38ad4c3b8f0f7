"""Launch geometry of the kernels that quantise and decode 8-bit matrices, on the host.

The grids come from the launchers' own header, compiled for the host; the workgroup sizes from
the launches that it feeds.
"""
import os
import re
import shutil
import subprocess

import pytest

from fsdp_sharded_optimizer_zs_amd import build as BUILD

DRIVER = r"""
#include <cstdio>
#include "zs_f8_grid.h"
using namespace zs;
int main() {
    long long rows, cols;
    while (std::scanf("%lld %lld", &rows, &cols) == 2)
        std::printf("%lld %lld\n", (long long)f8_quant_grid(f8_tiles(rows, cols)),
                    (long long)f8_values_grid(rows, cols));
    return 0;
}
"""
SIZES = ((1, 1), (128, 128), (129, 128), (4096, 11008), (2**30 - 128, 32), (2**30, 32), (2**30, 129),
         (2**31 - 1, 128), (2**31 - 1, 1), (2**24 - 128, 2**21), (2**23 - 128, 2**22), (2**25 - 128, 2**20))


def test_tile_grids_are_legal_launches(tmp_path):
    """512 threads to a tile that is quantised, 256 to one that is decoded: both launches stay
    under 2^32 threads, from one tile to the 2^31 - 1 that the entry points let through, and
    cover their work where they are not capped (the kernels loop past a capped grid)."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    with open(os.path.join(BUILD.CSRC, "zs_f8_quant.hip")) as f:
        source = f.read()
    # every launch of the two kernels that take a tile has the grid's number of threads
    launches = re.findall(r"hipLaunchKernelGGL\((.*?)stream", source, re.S)
    threads = [re.findall(r"dim3\((k\w+)\)", x)[-1] for x in launches]
    assert sorted(set(threads)) == ["kThreads", "kTileThreads"] and threads.count("kThreads") == 1
    assert "kTileThreads = kF8TileThreads" in source
    (tmp_path / "d.cpp").write_text(DRIVER)
    subprocess.run([cxx, "-std=c++17", "-I", BUILD.CSRC, str(tmp_path / "d.cpp"), "-o", str(tmp_path / "d")],
                   check=True)
    out = subprocess.run([str(tmp_path / "d")], input="".join("%d %d\n" % s for s in SIZES), capture_output=True,
                         text=True, check=True).stdout.split("\n")
    for (rows, cols), line in zip(SIZES, out):
        quant, values = (int(x) for x in line.split())
        tiles = -(-rows // 128) * -(-cols // 128)
        assert 1 <= quant and quant * 512 < 2**32 and 1 <= values and values * 256 < 2**32, (rows, cols)
        assert quant == min(tiles, (2**32 - 1) // 512) and tiles < 2**31, (rows, cols)
        # a workgroup's next tile, one grid further, is counted in 32 bits
        assert tiles + quant < 2**32
        if tiles <= 2**30:                        # what is decoded has no more
            assert 2 * tiles + values < 2**32
