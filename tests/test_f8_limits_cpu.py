"""Sizes at the 8-bit matrices' entry points on the host: what the kernels do not count, and the
workspaces that layers ask for."""
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


def test_few_rows_without_a_workspace_are_those_of_the_header(lib):  # noqa: F811
    """M <= 16 and M * (129 * ceil(K / 128) + 16) <= 79872."""
    for M in range(0, 19):
        for K in (0, 1, 128, 640, 4096, 4864, 4865, 9856, 9857, 11_008, 19_712, 19_713, 79_232, 79_233, 2**22):
            few = M <= 16 and M * (129 * -(-K // 128) + 16) <= 79872
            for N in (1, 64, 4096):
                assert (zs.zs_linear_f8_workspace(M, N, K) == 0) == few, (M, N, K)
    for M, K in ((16, 4864), (8, 9856), (4, 19_712), (1, 79_232)):
        assert zs.zs_linear_f8_workspace(M, 4096, K) == 0 < zs.zs_linear_f8_workspace(M, 4096, K + 1)


def test_layers_that_place_no_codes_ask_for_none(lib):  # noqa: F811
    """Layers of one 64 x 64 tile a CU at most and K up to 1,024 (of more than 16 rows) make their codes on
    the way: their workspace does not grow with M x K. Others place M rows of codes and scales."""
    least = zs.zs_linear_f8_workspace(17, 64, 256)
    assert 0 < least <= 1 << 14
    for M, N, K in ((40, 64, 256), (512, 512, 256), (1000, 1000, 512), (2048, 256, 1024), (777, 1001, 1024),
                    (16384, 64, 1024)):
        assert zs.zs_linear_f8_workspace(M, N, K) == least, (M, N, K)
    for M, N, K in ((777, 1001, 1025), (777, 1001, 1500), (512, 512, 4096), (4096, 4096, 1024)):
        assert zs.zs_linear_f8_workspace(M, N, K) >= least + M * K, (M, N, K)
