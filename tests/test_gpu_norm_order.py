"""What the order of the norm's additions depends on: the tensors' sizes, and with gradients
only or fp32 moments the place of each tensor over 4,096 elements (its g, or its p) modulo 64
elements. With these alike the bits are the same, wherever the arrays lie; otherwise the
sums, of n terms of one sign in fp64, are within n * 2^-53 of the exact one."""
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
from gpu_util import device, to_np
from oracle import zs_formats as F

pytestmark = pytest.mark.gpu

SIZES = [4097, 1, 70_000, 0, 4096, 4033, 20_000, 8193, 300_001] + [5000] * 40


def norm(table):
    dev = device()
    s, nc = torch.zeros(1, dtype=torch.float64, device=dev), torch.zeros(2, device=dev)
    zs.zs_grad_norm(table, 0.1, s, nc, torch.zeros(zs.ZS_NORM_WORKSPACE, dtype=torch.uint8, device=dev))
    return float(s), to_np(nc).tolist()


def views(dtype, off, values=None):
    """The tensors end to end from element `off` of an allocation of their own."""
    flat, out = torch.zeros(sum(SIZES) + off, dtype=dtype, device=device()), []
    for i, n in enumerate(SIZES):
        out.append(flat[off:off + n])
        off += n
        if values is not None:
            out[-1].copy_(values[i])
    return out


@pytest.mark.parametrize("dtype", (torch.bfloat16, torch.float32))
def test_equal_places_give_equal_bits(dtype):
    dev = device()
    gen = torch.Generator(device=dev).manual_seed(3)
    # of very different sizes, so that another order of additions shows in the last bits
    g = [(torch.randn(n, generator=gen, device=dev) * torch.rand(n, generator=gen, device=dev).mul(8).exp())
         .to(dtype) for n in SIZES]
    f32, u8 = torch.float32, torch.uint8
    blocks = lambda: [torch.zeros(-(-n // 256), dtype=u8, device=dev) for n in SIZES]

    def tables(off):
        """Each kind of table, its deciding array from element `off` on, the others elsewhere."""
        return [zs.MultiTable(grads=views(dtype, off, g)),
                zs.MultiTable(views(f32, off), views(f32, 5), views(f32, 0), views(dtype, 3 * off, g)),
                zs.MultiTable(views(f32, off), views(u8, off), views(u8, 0), views(dtype, 2 * off, g),
                              m_scale=blocks(), v_scale=blocks())]

    total = F.sumsq([to_np(x.float()) for x in g])
    want = [norm(t) for t in tables(0)]
    assert want[0] == want[1]                     # g and p at the same places
    for off in (64, 64 * 37, 1, 31, 63):
        for k, table in enumerate(tables(off)):
            got = norm(table)
            if off % 64 == 0 or k == 2:           # 8-bit moments: the sizes alone
                assert got == want[k], (off, k)
            assert abs(got[0] - total) <= sum(SIZES) * 2.0**-53 * total
