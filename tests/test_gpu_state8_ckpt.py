"""8-bit moments through checkpoints and another sharding: decoded to fp32, saved or
re-sharded with p and w as 32-bit moments are, and encoded again. Same blocks: the same
values. Blocks that shift: each value is rounded once more, to nearest in its new block, by
at most half a code: 2^-4 of the value or half a subnormal step, 2^(s - K - 130) under scale
byte s (v, which never becomes 0, by a whole one)."""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
import workloads as W
from gpu_util import check_bits, check_f32, device, to_np
from oracle import zs_formats as F

pytestmark = pytest.mark.gpu

HP = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
KINDS = ((zs.ZS_STATE8_M, "m"), (zs.ZS_STATE8_V, "v"))


class Rank:
    """One rank's shard with 8-bit moments."""

    def __init__(self, S, seed):
        dev = device()
        byte = lambda n: torch.zeros(n, dtype=torch.uint8, device=dev)
        self.S, nb = S, -(-S // 256)
        self.p = W.normal_f32(S, 0.02, seed, dev)
        self.w = torch.zeros(S, dtype=torch.bfloat16, device=dev)
        self.g = W.normal_f32(S, 1e-3, seed + 1, dev)
        # blocks of very different magnitudes
        self.g *= torch.exp2(torch.arange(S, device=dev).div(200, rounding_mode="floor") % 24 - 12)
        self.codes, self.scales = {"m": byte(S), "v": byte(S)}, {"m": byte(nb), "v": byte(nb)}
        self.table = zs.MultiTable([self.p], [self.codes["m"]], [self.codes["v"]], [self.g], [self.w],
                                   [self.scales["m"]], [self.scales["v"]])

    def step(self, t):
        zs.zs_adamw_multi(self.table, dict(step=t, **HP), seed=t)

    def decoded(self):
        out = {k: torch.zeros(self.S, device=self.p.device) for _, k in KINDS}
        for kind, k in KINDS:
            zs.zs_state8_decode(self.codes[k], self.scales[k], kind, out[k])
        return out

    def encode(self, moments):
        for kind, k in KINDS:
            zs.zs_state8_encode(moments[k], kind, self.codes[k], self.scales[k])


def test_saved_and_loaded_moments_are_the_same(tmp_path):
    N, S = 5003, 5003
    a, b = Rank(S, 1), Rank(S, 1)
    for t in (1, 2, 3):
        a.step(t)
    x = a.decoded()
    zs.zs_shard_save(str(tmp_path / "s"), 0, 1, N, 3, a.p, x["m"], x["v"], a.w)
    y = {k: torch.zeros(S, device=a.p.device) for k in "mv"}
    zs.zs_shard_load(str(tmp_path / "s"), b.p, y["m"], y["v"], b.w)
    b.encode(y)
    z = b.decoded()
    for k in "mv":
        check_f32(to_np(z[k]), to_np(x[k]), k, exact=True)
    for r in (a, b):                               # and the run goes on alike
        r.step(4)
    torch.cuda.synchronize()
    check_f32(to_np(a.p), to_np(b.p), "p", exact=True)
    for k in "mv":
        check_f32(to_np(a.decoded()[k]), to_np(b.decoded()[k]), k, exact=True)


@pytest.mark.parametrize("D,D2,N", [(4, 3, 20_003), (2, 5, 4099), (3, 1, 1000)])
def test_resharded_moments_are_within_half_a_code(D, D2, N):
    dev = device()
    S, S2 = -(-N // D), -(-N // D2)
    ranks = [Rank(S, 10 + 2 * r) for r in range(D)]
    for r in ranks:
        r.step(1)
        r.step(2)
    src = [r.decoded() for r in ranks]
    new = [Rank(S2, 30) for _ in range(D2)]
    for kind, k in KINDS:
        dst = [torch.zeros(S2, device=dev) for _ in range(D2)]
        zs.zs_reshard([x[k] for x in src], N, dst)
        for r, x in zip(new, dst):
            zs.zs_state8_encode(x, kind, r.codes[k], r.scales[k])
        torch.cuda.synchronize()
        K = F.TOP[kind]
        for r, x in zip(new, dst):
            want = to_np(x).astype(np.float64)
            codes, scales = F.state8_encode(to_np(x), kind)
            check_bits(to_np(r.codes[k]), codes, f"{k} codes")
            check_bits(to_np(r.scales[k]), scales, f"{k} scales")
            got = to_np(r.decoded()[k]).astype(np.float64)
            s = np.repeat(scales.astype(int), 256)[:S2]
            step = np.ldexp(1.0, s - K - (130 if k == "m" else 129))
            assert np.all(np.abs(got - want) <= np.maximum(2.0**-4 * np.abs(want), step)), k
            assert np.array_equal(got == 0, want == 0) or k == "m"
