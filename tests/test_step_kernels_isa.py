"""The step's and reduce's kernels that zs_step.hip compiles to (hipcc's assembly output with the
library's own flags; CPU only): those that some call launches, and no others.

- A clipped reduce is launched by the step alone, and not by the timed one.
- A fold of a number of contributions that is fixed at compile time is launched on aligned
  buffers only.
"""
import os
import re
import subprocess

import pytest

from fsdp_sharded_optimizer_zs_amd import build as B
from test_multi_isa import HIPCC

pytestmark = pytest.mark.slow


@pytest.fixture(scope="module")
def names(tmp_path_factory):
    if HIPCC is None:
        pytest.skip("hipcc not available")
    dst = tmp_path_factory.mktemp("isa") / "step.s"
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    r = subprocess.run([HIPCC] + flags + ["--cuda-device-only", "-S", "-x", "hip", os.path.join(B.CSRC, "zs_step.hip"),
                                          "-o", str(dst)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    found = re.findall(r"^\s*\.amdhsa_kernel (\S+)", dst.read_text(), re.M)
    assert found
    return found


def shape(name):
    """(kernel, clipped, sum, element type, fold length) of a kernel of this source."""
    kernel = re.search(r"\d+((?:adamw|reduce|reduce_norm)_(?:vec|scalar)?_?kernel)", name).group(1)
    what, dt, n = re.search(r"\d((?:Flat|Hybrid)Sum)ILi(\d)ELi(\d+)E", name).groups()
    tiles = re.search(r"EEELi(\d+)EEE?v", name)
    return kernel, "7Clipped" in name, what, int(dt), int(n), int(tiles.group(1)) if tiles else 0


def test_only_steps_are_clipped(names):
    got = sorted(shape(n) for n in names if "Clipped" in n)
    assert {k for k, *_ in got} == {"adamw_vec_kernel", "adamw_scalar_kernel"}
    want = [("adamw_vec_kernel", s, dt, n) for dt in (1, 2) for s, n in (("FlatSum", 0), ("FlatSum", 1), ("HybridSum", 0))]
    want += [("adamw_scalar_kernel", s, dt, 0) for dt in (1, 2) for s in ("FlatSum", "HybridSum")]
    assert sorted((k, s, dt, n) for k, _, s, dt, n, _ in got) == sorted(want)


def test_element_at_a_time_kernels_fold_at_run_time(names):
    got = [shape(n) for n in names if "Clipped" not in n]
    folds = {0, 1, 2, 4, 8, 16, 32}
    for kernel, element in (("adamw_vec_kernel", False), ("adamw_scalar_kernel", True), ("reduce_vec_kernel", False),
                            ("reduce_scalar_kernel", True), ("reduce_norm_kernel", False), ("reduce_norm_kernel", True)):
        mine = sorted((s, dt, n) for k, _, s, dt, n, tiles in got if k == kernel and (tiles == 0) == element)
        want = sorted((s, dt, n) for s in ("FlatSum", "HybridSum") for dt in (1, 2) for n in ({0} if element else folds))
        assert mine == want, (kernel, element)
