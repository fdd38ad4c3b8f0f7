"""The reduce with its norm and the step with a factor on the device: the bits of the calls
without them (elementwise, a fixed operation order), and the sum of squares within n * 2^-53
of the correctly rounded one (exact products of one sign, n fp64 additions in any order)."""
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

SIZES = (1, 2, 7, 511, 512, 1023, 1024, 1025, 4096, 8191, 8192, 8193, 100_003, 1 << 20, 4_300_001)


def contributions(D, S, dtype, seed, lead=0):
    dev = device()
    out = []
    for k in range(D):
        x = W.normal_f32(S + lead, W.GRAD_SCALE, seed * 100 + k, dev)
        out.append((x.bfloat16() if dtype == "bf16" else x)[lead:])
    return out


def buffers():
    dev = device()
    return (torch.full((1,), 5.0, dtype=torch.float64, device=dev), torch.full((2,), 5.0, device=dev),
            torch.zeros(zs.ZS_NORM_WORKSPACE, dtype=torch.uint8, device=dev))


def check_norm(sumsq, norm_coef, gs, max_norm, start=0.0):
    n = sum(g.size for g in gs)
    total = math.fsum([start, F.sum_of_squares(gs)]) if n < 300_000 else \
        start + sum(float(np.dot(g.astype(np.float64), g.astype(np.float64))) for g in gs)
    bound = 2 * (n + 2) * 2.0**-53 * total
    assert abs(sumsq.item() - total) <= bound
    s = sumsq.item()
    norm = math.sqrt(s)
    coef = 1.0 if math.isinf(max_norm) else min(1.0, max_norm / (norm + 1e-6))
    assert abs(norm_coef[0].item() - norm) <= 2.0**-23 * norm
    assert abs(norm_coef[1].item() - coef) <= 2.0**-23 * coef


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("S", SIZES)
def test_reduce_norm(S, dtype):
    for D, lead, opts in ((1, 0, {}), (4, 0, {}), (8, 1, {}), (3, 0, dict(scale=0.5)), (11, 0, {}),
                          (6, 0, dict(replicas=2, round_to_reduce_dtype=True)), (16, 0, {})):
        if D * S > 40_000_000:
            continue
        c = contributions(D, S, dtype, S % 97 + D, lead)
        want = torch.zeros(S, device=device())
        zs.zs_reduce_shard_ex(c, want, **opts)
        got = torch.full((S + 8,), 7.0, device=device())
        sumsq, nc, ws = buffers()
        for max_norm in (1e-3, math.inf):
            zs.zs_reduce_shard_norm(c, got[4:4 + S] if S % 4 == 0 else got[4:4 + S], max_norm, sumsq, nc, ws, **opts)
            assert torch.equal(got[4:4 + S], want)
            assert bool((got[:4] == 7).all() and (got[4 + S:] == 7).all())
            check_norm(sumsq, nc, [to_np(want)], max_norm)


def test_buckets_add_up():
    dev = device()
    sumsq, nc, ws = buffers()
    gs = []
    for k, (S, D, dtype) in enumerate([(100_000, 4, "bf16"), (0, 4, "bf16"), (33, 2, "f32"), (1 << 18, 1, "f32")]):
        c = contributions(D, S, dtype, k) if S else [torch.zeros(0, dtype=torch.bfloat16, device=dev)] * D
        g = torch.zeros(S, device=dev)
        zs.zs_reduce_shard_norm(c, g, 0.5, sumsq, nc, ws, accumulate=k > 0)
        gs.append(to_np(g))
        check_norm(sumsq, nc, gs, 0.5)
    joined = torch.zeros(2, device=dev)
    zs.zs_clip_coef([sumsq], 0.5, joined)
    assert torch.equal(joined, nc)


def test_empty_first_bucket_and_no_coefficient():
    sumsq, nc, ws = buffers()
    dev = device()
    zs.zs_reduce_shard_norm([torch.zeros(0, device=dev)], torch.zeros(0, device=dev), 1.0, sumsq, nc, ws)
    assert sumsq.item() == 0 and nc.tolist() == [0.0, 1.0]
    g = torch.zeros(100, device=dev)
    zs.zs_reduce_shard_norm([torch.ones(100, device=dev)], g, 1.0, sumsq, None, ws, accumulate=True)
    assert sumsq.item() == 100 and nc.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("value,norm,coef", [(float("nan"), "nan", "nan"), (float("inf"), "inf", 0.0),
                                             (1e30, 1e30, 1e-30)])
def test_gradients_that_are_not_finite(value, norm, coef):
    dev = device()
    c = torch.zeros(5000, device=dev)
    c[4321] = value
    sumsq, nc, ws = buffers()
    zs.zs_reduce_shard_norm([c], torch.zeros(5000, device=dev), 1.0, sumsq, nc, ws)
    got = [float(x) for x in nc]
    for g, w in zip(got, (norm, coef)):
        assert str(g) == str(w) or g == pytest.approx(float(w), rel=1e-6)


def test_same_sum_every_time_and_with_the_other_norms_workspace():
    c = contributions(4, 2_000_000, "bf16", 3)
    g = torch.zeros(2_000_000, device=device())
    sumsq, nc, ws = buffers()
    got = set()
    table = zs.MultiTable(grads=[g])
    for k in range(6):
        zs.zs_reduce_shard_norm(c, g, 1.0, sumsq, nc, ws)
        got.add(sumsq.item())
        zs.zs_grad_norm(table, 1.0, torch.zeros(1, dtype=torch.float64, device=device()), torch.zeros(2, device=device()), ws)
    assert len(got) == 1


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("S", (1, 5, 511, 1024, 1025, 5372, 100_003, 1 << 20))
def test_clipped_step(S, dtype):
    dev = device()
    for D, lead, factor, opts in ((1, 0, 0.37, {}), (1, 1, 1.0, {}), (4, 0, 1e-3, {}), (8, 0, 2.0**-10, dict(scale=1.0)),
                                  (6, 0, 0.9, dict(replicas=2, round_to_reduce_dtype=True)), (3, 0, 0.0, {}),
                                  (16, 0, 0.5, dict(keep_working_shard=True))):
        c = contributions(D, S, dtype, S % 89 + D, lead)
        reduce = {k: v for k, v in opts.items() if k != "keep_working_shard"}
        g = torch.zeros(S, device=dev)
        zs.zs_reduce_shard_ex(c, g, **reduce)
        p, m = W.normal_f32(S, 0.02, 1, dev), W.normal_f32(S, 1e-3, 2, dev)
        v = W.normal_f32(S, 1e-3, 3, dev).square()
        w = torch.zeros(S, dtype=torch.int16, device=dev)
        want = O.adamw_step(to_np(p), to_np(m), to_np(v), to_np(g) * np.float32(factor),
                            O.AdamWHP(step=3, **W.ADAMW_HP))
        zs.zs_adamw_step_clip(p, m, v, w, c, dict(step=3, **W.ADAMW_HP), torch.full((1,), factor, device=dev), **opts)
        for got, exp, name in zip((p, m, v), want, "pmv"):
            check_f32(to_np(got), exp, f"{name} D={D}", exact=True)
        check_bf16(to_np(w), want[3], f"w D={D}", exact=True)


def test_clipped_step_is_the_table_step():
    dev = device()
    S = 50_021
    g = W.normal_f32(S, 1e-3, 4, dev)
    factor = torch.full((1,), 0.123, device=dev)
    state = [[W.normal_f32(S, 0.02, 1, dev), W.normal_f32(S, 1e-3, 2, dev), W.normal_f32(S, 1e-3, 3, dev).square(),
              torch.zeros(S, dtype=torch.int16, device=dev)] for _ in range(2)]
    hp = dict(step=5, **W.ADAMW_HP)
    zs.zs_adamw_step_clip(*state[0], [g], hp, factor)
    p, m, v, w = state[1]
    zs.zs_adamw_multi(zs.MultiTable([p], [m], [v], [g], [w]), hp, grad_scale=factor)
    assert all(torch.equal(a, b) for a, b in zip(*state))


def test_refusals_on_the_device():
    dev = device()
    c, g = [torch.zeros(100, device=dev)], torch.zeros(100, device=dev)
    sumsq, nc, ws = buffers()
    for bad in (dict(grad_out=g[:99]), dict(grad_out=g.double()), dict(sumsq=nc), dict(norm_coef=nc[:1]),
                dict(workspace=ws[:100]), dict(replicas=2), dict(contribs=[c[0].half()])):
        kw = dict(contribs=c, grad_out=g, max_norm=1.0, sumsq=sumsq, norm_coef=nc, workspace=ws, **{})
        kw.update(bad)
        with pytest.raises((ValueError, TypeError)):
            zs.zs_reduce_shard_norm(**kw)
    p, m, v = (torch.zeros(100, device=dev) for _ in range(3))
    w = torch.zeros(100, dtype=torch.int16, device=dev)
    hp = dict(step=1, **W.ADAMW_HP)
    for scale in (nc, nc[1:].double(), torch.ones(1)):
        with pytest.raises((ValueError, TypeError)):
            zs.zs_adamw_step_clip(p, m, v, w, c, hp, scale)
    with pytest.raises(zs.ZsError) as e:
        zs.zs_adamw_step_clip(p, m, v, w, c, hp, p[3:4])
    assert e.value.status == zs.ZS_EALIAS
