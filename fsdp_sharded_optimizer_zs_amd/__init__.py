"""ZeRO-3 / FSDP shard step for AMD MI355X (gfx950).

One data-parallel rank's shard step, with D ranks simulated in one GPU's
memory: pack a unit into D shards, reduce-scatter arithmetic, fused
mixed-precision AdamW on the shard, and the all-gather's local rebuild.
The work runs in the HIP kernels of libzs.so; this package is its binding.
"""
from ._binding import (  # noqa: F401
    AdamWHP, LIB_PATH, ZS_BF16, ZS_EALIAS, ZS_EHIP, ZS_EINVAL, ZS_EUNSUPPORTED, ZS_F32,
    ZS_MAX_D, ZS_OK, ZsError, load, raw_adamw_step, zs_abi_version, zs_adamw_step,
    zs_adamw_step_ex, zs_reduce_shard_ex,
    zs_gather_unit, zs_last_error, zs_pack_flat, zs_reduce_shard, zs_step_pipelined,
    zs_unit_layout, zs_reshard, zs_shard_save, zs_shard_info_read, zs_shard_load,
    zs_shard_load_resharded, ZS_EIO, zs_adamw_step_host, zs_offload_step, zs_stream_ceiling,
    zs_hbm_probe, ZS_PROBE_READ, ZS_PROBE_WRITE, ZS_PROBE_COPY, ZS_PROBE_TRIAD, PackTable,
    zs_step_pipelined_static, ZS_W_STREAM, ZS_W_KEEP, zs_adamw_step_timed,
    zs_stream_ceiling_timed, MultiTable, zs_adamw_multi, zs_grad_norm, zs_clip_coef,
    zs_state8_layout, zs_state8_encode, zs_state8_decode, zs_quantize_mx4, zs_gather_unit_mx4,
    ZS_STATE_NONE, ZS_STATE_F32, ZS_STATE_8BIT, ZS_STATE8_M, ZS_STATE8_V, ZS_NORM_WORKSPACE,
    zs_reduce_shard_norm, zs_adamw_step_clip, F8Matrix, zs_f8_layout, zs_quantize_f8,
    zs_gather_matrix_f8, zs_dequantize_f8, zs_matmul_f8, zs_matmul_f8_workspace,
    zs_linear_f8, zs_linear_f8_workspace, zs_linear_f8_backward,
    zs_linear_f8_backward_workspace, ZS_E4M3, ZS_E5M2,
)

__all__ = [
    "zs_unit_layout", "zs_pack_flat", "zs_reduce_shard", "zs_adamw_step",
    "zs_reduce_shard_ex", "zs_adamw_step_ex", "zs_adamw_step_timed", "zs_reshard",
    "zs_shard_save", "zs_shard_info_read", "zs_shard_load", "zs_shard_load_resharded", "zs_adamw_step_host",
    "zs_offload_step", "zs_stream_ceiling", "zs_stream_ceiling_timed", "zs_hbm_probe",
    "ZS_PROBE_READ", "ZS_PROBE_WRITE", "ZS_PROBE_COPY", "ZS_PROBE_TRIAD",
    "zs_gather_unit", "zs_step_pipelined", "zs_last_error", "zs_abi_version", "AdamWHP", "ZsError",
    "ZS_BF16", "ZS_F32", "ZS_MAX_D", "load", "PackTable", "zs_step_pipelined_static",
    "MultiTable", "zs_adamw_multi", "zs_grad_norm", "zs_clip_coef", "zs_state8_layout",
    "zs_state8_encode", "zs_state8_decode", "zs_quantize_mx4", "zs_gather_unit_mx4",
    "ZS_STATE_NONE", "ZS_STATE_F32", "ZS_STATE_8BIT", "ZS_STATE8_M", "ZS_STATE8_V",
    "ZS_NORM_WORKSPACE",
    "zs_reduce_shard_norm", "zs_adamw_step_clip", "F8Matrix", "zs_f8_layout",
    "zs_quantize_f8", "zs_gather_matrix_f8", "zs_dequantize_f8", "zs_matmul_f8",
    "zs_matmul_f8_workspace", "zs_linear_f8", "zs_linear_f8_workspace",
    "zs_linear_f8_backward", "zs_linear_f8_backward_workspace", "ZS_E4M3", "ZS_E5M2",
]
