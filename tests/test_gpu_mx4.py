"""Microscaled 4-bit shards against the oracle, bit for bit: the scale is the block's
exponent and the nearest value is chosen on exact products with powers of two, so
there is nothing to round differently."""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
import workloads as W
from gpu_util import check_bf16, check_bits, check_f32, device, to_np
from oracle import zs_formats as F
from oracle import zs_oracle as O
from test_gpu_multi import Arena, bits16

pytestmark = pytest.mark.gpu

SIZES = (1, 2, 3, 7, 8, 9, 31, 32, 33, 255, 256, 257, 2047, 2048, 4099, 100_003, 1 << 20)


def values(S, seed, wide):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal(S) * (10.0 ** rng.uniform(-45, 38, S) if wide else 0.02)).astype(np.float32)
    if S > 200 and wide:
        x[32:64] = 0
        x[70] = np.nan
        x[100] = np.inf
        x[150] = -0.0
        x[160:192] = np.float32(1e-45)
    return x


def quantize(x, dev, guards=True):
    """zs_quantize_mx4 of numpy values (uint16: bf16 bits) in guarded buffers."""
    S = x.size
    src = Arena([bits16(x)], torch.int16 if x.dtype == np.uint16 else torch.float32, dev)
    codes = Arena([np.zeros(-(-S // 2), np.uint8)], torch.uint8, dev)
    scales = Arena([np.zeros(-(-S // 32), np.uint8)], torch.uint8, dev)
    zs.zs_quantize_mx4(src.views[0], codes.views[0], scales.views[0])
    for a in (src, codes, scales):
        a.check_guards("quantize")
    return codes.views[0], scales.views[0]


@pytest.mark.parametrize("wide", (False, True))
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("S", SIZES)
def test_quantize(S, dtype, wide):
    x = values(S, S, wide)
    x = O.bf16_round(x) if dtype == "bf16" else x
    codes, scales = quantize(x, device())
    wc, ws = F.mx4_quantize(O.bf16_widen(x) if dtype == "bf16" else x)
    check_bits(to_np(scales), ws, "scales")
    check_bits(to_np(codes), wc, "codes")


def test_quantize_every_bf16_value():
    """Every finite bf16 bit pattern beside a block's largest value of each of its
    exponents: 128 blocks' worth of magnitudes a power of two."""
    h = np.arange(1 << 16, dtype=np.uint16)
    h = h[(h & 0x7F80) != 0x7F80]
    x = O.bf16_widen(h)
    for shift in (0, 1, 2, 5):
        top = np.float32(2.0) ** np.clip(np.floor(np.log2(np.maximum(np.abs(x), 1e-37))) + shift, -126, 127)
        blocks = np.zeros((x.size, 32), np.float32)
        blocks[:, 3] = x
        blocks[:, 17] = top
        b = O.bf16_round(blocks.ravel())
        codes, scales = quantize(b, device())
        wc, ws = F.mx4_quantize(O.bf16_widen(b))
        check_bits(to_np(scales), ws, f"scales, shift {shift}")
        check_bits(to_np(codes), wc, f"codes, shift {shift}")


@pytest.mark.parametrize("out", ("bf16", "f32"))
@pytest.mark.parametrize("D,S", [(1, 1), (1, 33), (2, 3), (3, 255), (4, 256), (4, 5372), (8, 4099),
                                 (16, 1024), (64, 1001), (5, 100_003), (2, 1 << 20)])
def test_gather(D, S, out):
    dev = device()
    rng = np.random.default_rng(D * 7 + S)
    codes = [rng.integers(0, 256, -(-S // 2)).astype(np.uint8) for _ in range(D)]
    scales = [rng.integers(0, 256, -(-S // 32)).astype(np.uint8) for _ in range(D)]
    with np.errstate(over="ignore"):
        want = np.concatenate([F.mx4_values(c, s, S) for c, s in zip(codes, scales)]).astype(np.float32)
    dc, ds = Arena(codes, torch.uint8, dev, 3), Arena(scales, torch.uint8, dev, 1)
    flat = Arena([np.zeros(D * S, np.int16 if out == "bf16" else np.float32)],
                 torch.int16 if out == "bf16" else torch.float32, dev)
    zs.zs_gather_unit_mx4(dc.views, ds.views, flat.views[0])
    if out == "bf16":
        check_bf16(to_np(flat.views[0]), O.bf16_round(want), "unit", exact=True)
    else:
        check_f32(to_np(flat.views[0]), want, "unit", exact=True)
    flat.check_guards("gather")


@pytest.mark.parametrize("out", ("bf16", "f32"))
def test_gather_every_code_and_scale(out):
    dev = device()
    codes = np.tile(np.arange(256, dtype=np.uint8), 16)          # 32 elements a block, 256 blocks
    scales = np.arange(256, dtype=np.uint8)
    S = 8192
    codes = codes[:S // 2]
    with np.errstate(over="ignore"):
        want = F.mx4_values(codes, scales, S).astype(np.float32)
    flat = torch.zeros(S, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device=dev)
    zs.zs_gather_unit_mx4([torch.from_numpy(codes).to(dev)], [torch.from_numpy(scales).to(dev)], flat)
    if out == "bf16":
        check_bf16(to_np(flat), O.bf16_round(want), "unit", exact=True)
    else:
        check_f32(to_np(flat), want, "unit", exact=True)


def test_gather_past_32_bits():
    """A unit of 2^31 + 64 * 37 elements (over 4 GiB of bf16): each shard's ends and random
    places against the oracle."""
    dev = device()
    D, S = 64, (1 << 25) + 37
    codes = [torch.randint(0, 256, (-(-S // 2),), dtype=torch.uint8, device=dev) for _ in range(D)]
    scales = [torch.randint(100, 140, (-(-S // 32),), dtype=torch.uint8, device=dev) for _ in range(D)]
    flat = torch.zeros(D * S, dtype=torch.bfloat16, device=dev)
    zs.zs_gather_unit_mx4(codes, scales, flat)
    torch.cuda.synchronize()
    for r in (0, 1, 31, 62, 63):
        c, s = to_np(codes[r]), to_np(scales[r])
        want = F.mx4_values(c, s, S).astype(np.float32)
        check_bf16(to_np(flat[r * S:(r + 1) * S]), O.bf16_round(want), f"shard {r}", exact=True)


def test_quantize_past_32_bits():
    """A shard of 2^32 + 37 bf16 elements: windows at its start, around element 2^31 and
    2^32 and at its end, quantised and gathered again."""
    dev = device()
    S = (1 << 32) + 37
    block = W.as_bf16_bits(W.normal_f32(1 << 20, 0.02, 78, dev))
    x = torch.empty(S, dtype=torch.int16, device=dev)
    x[:S - 37].view(-1, 1 << 20).copy_(block)
    x[S - 37:].copy_(block[5:42])
    codes = torch.zeros(-(-S // 2), dtype=torch.uint8, device=dev)
    scales = torch.zeros(-(-S // 32), dtype=torch.uint8, device=dev)
    zs.zs_quantize_mx4(x, codes, scales)
    flat = torch.zeros(S, dtype=torch.int16, device=dev)
    zs.zs_gather_unit_mx4([codes], [scales], flat)
    torch.cuda.synchronize()
    for a, k in ((0, 4096), (1 << 31, 4096), ((1 << 32) - 2048, 2048 + 37)):
        wc, ws = F.mx4_quantize(O.bf16_widen(to_np(x[a:a + k])))
        check_bits(to_np(codes[a // 2:a // 2 + wc.size]), wc, f"codes at {a}")
        check_bits(to_np(scales[a // 32:a // 32 + ws.size]), ws, f"scales at {a}")
        want = F.mx4_values(wc, ws, k).astype(np.float32)
        check_bf16(to_np(flat[a:a + k]), O.bf16_round(want), f"values at {a}", exact=True)


def test_step_quantize_gather_together():
    """A rank's working shards as a run uses them: each rank steps its shard, its bf16
    working shard is quantised, and the unit is gathered from the 4-bit shards; then the
    quantiser and the gather again from a graph."""
    dev = device()
    D, S = 4, 5003
    p = [W.normal_f32(S, 0.02, 90 + r, dev) for r in range(D)]
    g = [W.as_bf16_bits(W.normal_f32(S, 1e-3, 95 + r, dev)) for r in range(D)]
    m, v = ([torch.zeros(S, device=dev) for _ in range(D)] for _ in range(2))
    w = [torch.zeros(S, dtype=torch.int16, device=dev) for _ in range(D)]
    codes = [torch.zeros(-(-S // 2), dtype=torch.uint8, device=dev) for _ in range(D)]
    scales = [torch.zeros(-(-S // 32), dtype=torch.uint8, device=dev) for _ in range(D)]
    flat = torch.zeros(D * S, dtype=torch.bfloat16, device=dev)
    table = zs.MultiTable(p, m, v, g, w)

    def gather():
        for r in range(D):
            zs.zs_quantize_mx4(w[r], codes[r], scales[r])
        zs.zs_gather_unit_mx4(codes, scales, flat)

    def check(what):
        torch.cuda.synchronize()
        want = []
        for r in range(D):
            c, s = F.mx4_quantize(O.bf16_widen(to_np(w[r])))
            want.append(F.mx4_values(c, s, S).astype(np.float32))
        check_bf16(to_np(flat), O.bf16_round(np.concatenate(want)), what, exact=True)

    zs.zs_adamw_multi(table, dict(step=1, **W.ADAMW_HP))
    gather()
    check("eager")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        gather()
    for t in (2, 3, 4):
        zs.zs_adamw_multi(table, dict(step=t, **W.ADAMW_HP))
        graph.replay()
        check(f"replay after step {t}")


def test_refusals_on_the_device():
    dev = device()
    x = torch.zeros(100, device=dev)
    c, s = (torch.zeros(n, dtype=torch.uint8, device=dev) for n in (50, 4))
    for bad in ((x, c[:49], s), (x, c, s[:3]), (x.double(), c, s), (x[::2], c, s), (x, x, s)):
        with pytest.raises((ValueError, TypeError)):
            zs.zs_quantize_mx4(*bad)
    for bad in (([c], [], x), ([c, c], [s, s], x[:99]), ([c], [s], x.half()), ([c], [s[:1]], x)):
        with pytest.raises((ValueError, TypeError)):
            zs.zs_gather_unit_mx4(*bad)
    with pytest.raises(zs.ZsError) as e:
        zs.zs_gather_unit_mx4([x.view(torch.uint8)[:50]], [s], x)
    assert e.value.status == zs.ZS_EALIAS
