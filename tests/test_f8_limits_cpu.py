"""Limits of the 8-bit matrices' entry points on the host: sizes that the kernels do not count."""
import pytest

import fsdp_sharded_optimizer_zs_amd as zs
from test_f8_cpu import A, lib, linear, mat, no_gpu  # noqa: F401

FAR = 1 << 60                  # behind every other range of a call


def test_linear_refuses_more_tiles_of_x_than_a_launch_counts(lib):  # noqa: F811
    """x is quantised by tiles of 128 x 128, counted in 32 bits: 2^31 of them and more are refused
    before anything is enqueued."""
    no_gpu()
    w = mat(A, A + (1 << 40), rows=1, cols=2**22)
    call = lambda M: linear(lib, x=FAR, M=M, ldx=2**22, w=w, y=1 << 59, ldy=1, ws=1 << 61)
    for M in (2**23 + 1, 2**24, 2**30 - 64):
        assert call(M) == zs.ZS_EINVAL, M
        assert "x has too many elements" in zs.zs_last_error()
