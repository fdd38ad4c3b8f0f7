"""The calls over many tensors, of the 8-bit moments and of the 4-bit shards enqueue and
return: they wait for nothing on the device and allocate nothing, so they run behind other
work and are captured into graphs."""
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
from gpu_util import device

pytestmark = pytest.mark.gpu

HP = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=2)
SIZES = [40_000, 1, 777, 5000]


class Run:
    """One of each call, on buffers made from a seed."""

    def __init__(self, seed=5):
        dev = device()
        gen = torch.Generator(device=dev).manual_seed(seed)
        rand = lambda n, s: torch.randn(n, generator=gen, device=dev) * s
        zero = lambda n, t=torch.uint8: torch.zeros(n, dtype=t, device=dev)
        off = zs.zs_state8_layout(SIZES)
        cut = [(a, a + n) for a, n in zip(off, SIZES)]
        blk = [(a // 256, a // 256 - (-n // 256)) for a, n in zip(off, SIZES)]
        n = sum(SIZES)
        self.b = dict(p=rand(n, 0.02), p8=rand(n, 0.02), g=rand(n, 1e-2), m=rand(n, 1e-4),
                      v=rand(n, 1e-3).square(), m32=rand(off[-1], 1e-4), v32=rand(off[-1], 1e-3).square(),
                      w=zero(n, torch.bfloat16), w8=zero(n, torch.bfloat16),
                      mc=zero(off[-1]), vc=zero(off[-1]), ms=zero(off[-1] // 256), vs=zero(off[-1] // 256),
                      mo=zero(off[-1], torch.float32), vo=zero(off[-1], torch.bfloat16),
                      sumsq=zero(1, torch.float64), nc=zero(2, torch.float32),
                      codes=zero(-(-n // 2)), scales=zero(-(-n // 32)), flat=zero(n, torch.float32))
        b, parts = self.b, lambda k: self.b[k].split(SIZES)
        self.ws = zero(zs.ZS_NORM_WORKSPACE)
        self.t32 = zs.MultiTable(parts("p"), parts("m"), parts("v"), parts("g"), parts("w"))
        self.t8 = zs.MultiTable(parts("p8"), [b["mc"][x:y] for x, y in cut], [b["vc"][x:y] for x, y in cut],
                                parts("g"), parts("w8"), [b["ms"][x:y] for x, y in blk],
                                [b["vs"][x:y] for x, y in blk])

    def calls(self):
        b = self.b
        return [
            lambda: zs.zs_state8_encode(b["m32"], zs.ZS_STATE8_M, b["mc"], b["ms"]),
            lambda: zs.zs_state8_encode(b["v32"], zs.ZS_STATE8_V, b["vc"], b["vs"]),
            lambda: zs.zs_grad_norm(self.t32, 0.5, b["sumsq"], b["nc"], self.ws),
            lambda: zs.zs_clip_coef([b["sumsq"]] * 3, 0.5, b["nc"]),
            lambda: zs.zs_adamw_multi(self.t32, HP, grad_scale=b["nc"][1:]),
            lambda: zs.zs_adamw_multi(self.t8, HP, grad_scale=b["nc"][1:], seed=9),
            lambda: zs.zs_state8_decode(b["mc"], b["ms"], zs.ZS_STATE8_M, b["mo"]),
            lambda: zs.zs_state8_decode(b["vc"], b["vs"], zs.ZS_STATE8_V, b["vo"]),
            lambda: zs.zs_quantize_mx4(b["w"], b["codes"], b["scales"]),
            lambda: zs.zs_gather_unit_mx4([b["codes"]], [b["scales"]], b["flat"]),
        ]

    def all(self):
        for call in self.calls():
            call()

    def same(self, other):
        return [k for k in self.b if not torch.equal(self.b[k], other.b[k])]


def test_no_call_waits_or_allocates():
    """Behind some 0.1 s of work on the stream every call returns while that is still
    running; neither torch's allocator nor the device's free memory changes."""
    run, warm = Run(), Run()
    warm.all()                                        # code is loaded on the first call
    busy = torch.zeros(1 << 30, device=device()).add_(1.0)     # 4 GiB read and written: over 1 ms
    torch.cuda.synchronize()
    free, held = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()
    for call in run.calls():
        done = torch.cuda.Event()
        for _ in range(30):
            busy.add_(1.0)
        done.record()
        call()
        assert not done.query()
        torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free and torch.cuda.memory_allocated() == held
    assert run.same(warm) == []


def test_every_call_is_captured_and_replayed():
    run, eager = Run(), Run()
    Run(6).all()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):        # an allocation or a wait would fail it
        run.all()
    torch.cuda.synchronize()
    assert run.same(Run()) == []                      # capturing runs nothing
    for rep in range(4):
        for r in (run, eager):
            r.b["g"].mul_(1.25)
            r.b["m32"].mul_(0.5)
        graph.replay()
        eager.all()
        torch.cuda.synchronize()
        assert run.same(eager) == [], rep
