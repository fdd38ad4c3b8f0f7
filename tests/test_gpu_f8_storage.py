"""8-bit matrices whose storage is freed between a unit's passes and taken again for the next gather."""
import pytest
import torch

import fsdp_sharded_optimizer_zs_amd as zs
from gpu_util import device

pytestmark = pytest.mark.gpu


def test_a_matrix_gathered_again_into_new_storage():
    dev = device()
    M, N, K, D = 40, 300, 500, 4
    gen = torch.Generator(device=dev).manual_seed(5)
    x = torch.randn(M, K, generator=gen, device=dev).bfloat16()
    S = -(-N * K // D)
    shards = [torch.randn(S, generator=gen, device=dev).bfloat16() for _ in range(D)]
    ws = torch.zeros(zs.zs_linear_f8_workspace(M, N, K), dtype=torch.uint8, device=dev)
    w = zs.F8Matrix.empty(N, K, block_rows=128)
    want = None
    for _ in range(4):
        zs.zs_gather_matrix_f8(shards, 0, w)
        y = torch.zeros(M, N, dtype=torch.bfloat16, device=dev)
        zs.zs_linear_f8(x, w, y, ws)
        want = y.clone() if want is None else want
        assert torch.equal(y, want)
        sizes = [t.untyped_storage().nbytes() for t in (w.codes, w.scales)]
        for t in (w.codes, w.scales):
            t.untyped_storage().resize_(0)
        with pytest.raises(ValueError):
            zs.zs_linear_f8(x, w, y, ws)
        # what takes the freed bytes is not written by the next gather
        others = [torch.full((n,), 77, dtype=torch.uint8, device=dev) for n in sizes]
        for t, n in zip((w.codes, w.scales), sizes):
            t.untyped_storage().resize_(n)
        zs.zs_gather_matrix_f8(shards, 0, w)
        assert all(bool((o == 77).all()) for o in others)
        del others
