"""The reduce with its norm and the clipped step on views that start off a 16-byte boundary, as into a
flat gradient or a flat state, while the other buffers are aligned: the bits of the calls without them,
and nothing written beside a view."""
import math

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
import workloads as W
from gpu_util import check_bf16, check_f32, device, to_np
from oracle import zs_f8 as F
from oracle import zs_oracle as O

pytestmark = pytest.mark.gpu

SIZES = (1, 3, 512, 1023, 1024, 1025, 8193, 100_003, (1 << 20) + 4)
PAD = 8


def view(S, at, fill, dtype=torch.float32):
    """A view of S elements from element `at` of an aligned buffer on, and the whole buffer."""
    whole = torch.full((S + 2 * PAD,), fill, dtype=dtype, device=device())
    assert whole.data_ptr() % 256 == 0
    return whole[at:at + S], whole


def beside(whole, at, S, fill):
    return bool((whole[:at] == fill).all() and (whole[at + S:] == fill).all())


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("at", (0, 1, 2, 3, 4, 5))
def test_reduce_norm_into_a_view(at, dtype):
    for S in SIZES:
        for D in (1, 3, 8):
            c = [W.normal_f32(S, W.GRAD_SCALE, 10 * D + k, device()).to(dtype) for k in range(D)]
            assert all(x.data_ptr() % 16 == 0 for x in c)
            want = torch.zeros(S, device=device())
            zs.zs_reduce_shard_ex(c, want)
            got, whole = view(S, at, 7.0)
            sumsq = torch.zeros(1, dtype=torch.float64, device=device())
            nc = torch.zeros(2, device=device())
            ws = torch.zeros(zs.ZS_NORM_WORKSPACE, dtype=torch.uint8, device=device())
            for _ in range(2):
                zs.zs_reduce_shard_norm(c, got, 1.0, sumsq, nc, ws)
                assert torch.equal(got, want) and beside(whole, at, S, 7.0), (S, D)
                # n exact squares of one sign, n + 1 additions in fp64 in some order
                x = to_np(want)
                total = F.sum_of_squares([x]) if S < 10_000 else float(np.square(x.astype(np.float64)).sum())
                assert abs(sumsq.item() - total) <= 2 * (S + 2) * 2.0**-53 * total, (S, D)
                norm = math.sqrt(sumsq.item())
                assert abs(nc[0].item() - norm) <= 2.0**-24 * norm * (1 + 2.0**-20)


@pytest.mark.parametrize("which", ("p", "m", "v", "w", "pmvw"))
def test_clipped_step_of_views(which):
    for S in SIZES:
        for D, at in ((1, 1), (1, 4), (4, 3)):
            dev = device()
            c = [W.normal_f32(S, 1e-3, 7 * D + k, dev) for k in range(D)]
            g = torch.zeros(S, device=dev)
            zs.zs_reduce_shard_ex(c, g)
            start = dict(p=W.normal_f32(S, 0.02, 1, dev), m=W.normal_f32(S, 1e-3, 2, dev),
                         v=W.normal_f32(S, 1e-3, 3, dev).square(), w=torch.zeros(S, dtype=torch.int16, device=dev))
            want = O.adamw_step(*(to_np(start[k]) for k in "pmv"), to_np(g) * np.float32(0.37),
                                O.AdamWHP(step=3, **W.ADAMW_HP))
            views, wholes = {}, {}
            for k, x in start.items():
                views[k], wholes[k] = view(S, at if k in which else 0, 5, x.dtype)
                views[k].copy_(x)
            zs.zs_adamw_step_clip(*(views[k] for k in "pmvw"), c, dict(step=3, **W.ADAMW_HP),
                                  torch.full((1,), 0.37, device=dev))
            for k, exp in zip("pmv", want):
                check_f32(to_np(views[k]), exp, f"{k} D={D} S={S}", exact=True)
            check_bf16(to_np(views["w"]), want[3], f"w D={D} S={S}", exact=True)
            for k in "pmvw":
                assert beside(wholes[k], at if k in which else 0, S, 5), (k, S)
