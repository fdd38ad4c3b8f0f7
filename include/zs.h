/*
 * zs.h -- C ABI of the ZeRO-3 shard-step library (libzs.so) for MI355X (gfx950).
 *
 * One data-parallel rank's ZeRO-3 / FSDP shard step, with the D ranks of a
 * data-parallel group simulated as D buffers in one GPU's memory:
 *
 *   zs_unit_layout   flat layout of one FSDP unit (host arithmetic only)
 *   zs_pack_flat     pack a unit's tensors into D contiguous shards
 *   zs_reduce_shard  reduce-scatter arithmetic for one shard
 *   zs_adamw_step    fused reduce + mixed-precision AdamW on one shard
 *   zs_reduce_shard_ex, zs_adamw_step_ex  the same under HYBRID_SHARD's
 *                    two-level reduce and/or reduce-dtype rounding
 *   zs_adamw_step_timed  zs_adamw_step_ex with the kernel's own start and
 *                    end recorded in two events (a measurement aid)
 *   zs_gather_unit   all-gather's local rebuild of a unit from its shards
 *   zs_step_pipelined  the step over a sequence of buckets, each bucket's
 *                    contribution transfer overlapped with the previous step
 *   zs_step_pipelined_static  the same with library-owned staging, for
 *                    callers that cannot allocate device memory
 *   zs_reshard       re-shard a unit from D to D2 shards on the device
 *   zs_shard_save, zs_shard_load, zs_shard_load_resharded, zs_shard_info_read
 *                    per-rank shard checkpoints, resumable at any D2
 *   zs_adamw_step_host, zs_offload_step
 *                    the step's AdamW on host cores (ZeRO-Offload)
 *   zs_multi_create, zs_adamw_multi
 *                    AdamW over many tensors in one launch, moments in 32 or
 *                    in 8 bits; zs_state8_layout, zs_state8_encode and
 *                    zs_state8_decode lay out and convert the 8-bit moments
 *   zs_quantize_f8, zs_gather_matrix_f8, zs_dequantize_f8
 *                    matrices in 8-bit floating point with a scale for each
 *                    block of 128 elements, also straight from a unit's shards
 *   zs_matmul_f8, zs_linear_f8, zs_linear_f8_backward
 *                    their products, and a linear layer's forward and backward
 *                    pass over a unit's 8-bit weights
 *   zs_grad_norm, zs_clip_coef
 *                    the L2 norm over many gradient tensors and the factor
 *                    that clips it, left on the device for zs_adamw_multi
 *   zs_reduce_shard_norm, zs_adamw_step_clip
 *                    the shard's reduce with the norm of its result, and the
 *                    step with the gradient multiplied by a clip factor that
 *                    is on the device
 *   zs_quantize_mx4, zs_gather_unit_mx4
 *                    a shard in microscaled 4-bit floating point, and the
 *                    all-gather's rebuild of a unit from such shards
 *   zs_stream_ceiling, zs_stream_ceiling_timed, zs_hbm_probe
 *                    measurement aids: the step's memory streams without its
 *                    arithmetic, and HBM's rate for one direction alone
 *
 * Sources (web pages, by title and section):
 *   [ZT]   "7.10 -- Fully-sharded data parallel (FSDP / ZeRO-3)", AI / ML
 *          Theory, chapter 7.
 *   [GPT8] "Building GPT from Scratch -- Part 8: FSDP -- When the Model
 *          Won't Fit".
 *   [RP]   "Distributed LLM Fine-Tuning at Scale: FSDP, ZeRO-3, and
 *          Multi-GPU Orchestration".
 *
 * Conventions shared by every entry point:
 *   - All data buffers are device memory owned by the caller. The library
 *     never allocates, frees or synchronizes; kernels are enqueued on the
 *     caller's stream (which must belong to the current HIP device) and the
 *     call returns as soon as they are enqueued.
 *   - Arrays of D pointers (shards, contributions) are HOST arrays of DEVICE
 *     pointers; they are copied into kernel arguments, so D <= ZS_MAX_D.
 *   - bf16 values are raw IEEE binary32 high halves stored as uint16.
 *   - Every argument is validated on the host before anything is enqueued.
 *     A failing call returns a nonzero status, enqueues nothing, and leaves
 *     a message for zs_last_error(). A launch failure reported by the HIP
 *     runtime returns ZS_EHIP. Faults of enqueued kernels surface at the
 *     caller's next synchronization, as for any HIP kernel.
 *   - Zero-length work (S == 0, T == 0) returns ZS_OK and enqueues nothing.
 *   - Calls are thread-safe; the error message is per calling thread.
 *   - Full-speed paths need 16-byte-aligned buffers; any other alignment
 *     allowed by the element size is correct but slower.
 */
#ifndef ZS_H_
#define ZS_H_

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t zs_status;
#define ZS_OK            0  /* success                                       */
#define ZS_EINVAL        1  /* an argument is out of range or inconsistent   */
#define ZS_EALIAS        2  /* an output overlaps an input it may not        */
#define ZS_EHIP          3  /* the HIP runtime reported an error             */
#define ZS_EUNSUPPORTED  4  /* unknown dtype or a size beyond the limits     */
#define ZS_EIO           5  /* a checkpoint file could not be read or written,
                               or failed its format or checksum checks    */

/* Element types. */
#define ZS_BF16 1  /* bf16 as uint16 bit patterns (2 bytes)                   */
#define ZS_F32  2  /* IEEE binary32 (4 bytes)                                 */

#define ZS_MAX_D 64  /* most ranks (or contributions) one call handles       */

/* One tensor of an FSDP unit: its data and where it lands in the flat unit. */
typedef struct {
    const void* ptr;      /* device pointer to numel contiguous elements      */
    int64_t numel;        /* >= 0                                             */
    int64_t flat_offset;  /* start in the flat unit: prefix sum of numels     */
} zs_tensor_ref;

/* AdamW hyperparameters, in double; the library rounds each derived
 * constant to fp32 once (see zs_adamw_step). */
typedef struct {
    double lr;            /* >= 0                                             */
    double beta1;         /* in [0, 1)                                        */
    double beta2;         /* in [0, 1)                                        */
    double eps;           /* >= 0                                             */
    double weight_decay;  /* >= 0, decoupled, multiplied by lr               */
    int64_t step;         /* t >= 1, the step being taken                     */
} zs_adamw_hp;

/*
 * zs_unit_layout -- flat layout of one FSDP unit (host only, no GPU work).
 *
 * [ZT] section 3 gives each rank r a partition P_r of about 1/D of the
 * parameters; [ZT] section 6 and [GPT8] "PyTorch FSDP Implementation" make
 * each transformer block one unit. Layout: the T tensors end to end in the
 * given order, no per-tensor alignment, the flat length N padded up to
 * N_pad = D * ceil(N / D); rank r owns flat[r*S, (r+1)*S) with S = N_pad / D.
 *
 *   numels      host, T entries, each >= 0 (may be NULL when T == 0)
 *   T           number of tensors, >= 0
 *   D           ranks, 1..ZS_MAX_D
 *   offsets_out host, T + 1 entries: offsets_out[j] = start of tensor j,
 *               offsets_out[T] = N
 *   n_out, n_pad_out, shard_len_out  host scalars: N, N_pad, S
 * Errors: ZS_EINVAL for a negative count, a NULL output or D out of range;
 * ZS_EUNSUPPORTED if N_pad overflows int64.
 */
zs_status zs_unit_layout(const int64_t* numels, int32_t T, int32_t D,
                         int64_t* offsets_out, int64_t* n_out,
                         int64_t* n_pad_out, int64_t* shard_len_out);

/*
 * zs_pack_flat -- pack a unit's tensors into its D shards (bit copy).
 *
 * The flat unit (layout of zs_unit_layout) is split into D contiguous
 * shards, the rank-ordered blocks of the all-gather diagram in [GPT8]
 * "AllGather vs AllReduce" and the local shards of [ZT] section 5.1:
 * shards[r][i] = flat[r*S + i], with flat[N, N_pad) = +0 (all-zero bits).
 * Bytes are copied unchanged whatever they hold.
 *
 *   h_table  host array of T tensor refs, checked by the library: numel >= 0,
 *            ptr non-NULL when numel > 0 and aligned to the element size,
 *            flat_offset equal to the prefix sum of the numels
 *   d_table  device array holding the same T refs byte for byte (the kernel
 *            reads this copy; the caller keeps it alive until the work is done)
 *   T        tensors, >= 0
 *   dtype    ZS_BF16 or ZS_F32 (element size of every tensor and shard)
 *   D        ranks, 1..ZS_MAX_D
 *   shards   host array of D device pointers, each to S elements
 *   S        shard length; must equal ceil(N / D) for N = sum of numels
 * Errors: ZS_EINVAL (inconsistent table, S, NULLs, alignment), ZS_EALIAS
 * (a shard overlaps a tensor or another shard), ZS_EUNSUPPORTED (dtype).
 */
zs_status zs_pack_flat(const zs_tensor_ref* h_table, const zs_tensor_ref* d_table,
                       int32_t T, int32_t dtype, int32_t D,
                       void* const* shards, int64_t S, hipStream_t stream);

/*
 * zs_reduce_shard -- reduce-scatter arithmetic for one rank's shard.
 *
 * [GPT8] "AllGather vs AllReduce": rank r receives the sum over ranks of
 * their gradients restricted to its shard; [ZT] section 4: this is the
 * all-reduce's result, scattered; DDP's all-reduce averages. For i < S:
 *   grad_out[i] = (((c_0[i] + c_1[i]) + ...) + c_{D-1}[i]) * float(1/D)
 * in fp32, contributions widened exactly from the reduce dtype (bf16 as in
 * [RP] section 2, or fp32 as in [GPT8] "Mixed Precision"), folded left to
 * right in rank order starting from c_0, one rounding per add, then one
 * multiply by 1/D rounded to fp32. The result stays fp32.
 *
 *   contribs  host array of D device pointers, each to S elements of dtype
 *   D         contributions, 1..ZS_MAX_D
 *   dtype     ZS_BF16 or ZS_F32
 *   S         >= 0
 *   grad_out  device, S floats
 * Errors: ZS_EINVAL, ZS_EALIAS (grad_out overlaps a contribution),
 * ZS_EUNSUPPORTED.
 */
zs_status zs_reduce_shard(const void* const* contribs, int32_t D, int32_t dtype,
                          int64_t S, float* grad_out, hipStream_t stream);

/*
 * zs_adamw_step -- fused reduce + mixed-precision AdamW on one shard.
 *
 * [ZT] section 3: a rank updates only its partition, from its fp32 master
 * copy, its m and v and its slice of the gradient; [ZT] section 6 and
 * [GPT8] "Mixed Precision": master and moments stay fp32, the working
 * weights are bf16. Per element, g is the zs_reduce_shard value of the
 * n_contrib contributions (their mean, folded in order), never stored; then
 * in fp32, each operation rounded on its own, no fused multiply-add:
 *   p1  = p * DEC
 *   m'  = B1 * m + B1c * g
 *   v'  = B2 * v + B2c * (g * g)
 *   den = sqrt(v') / BC2S + EPS
 *   p'  = p1 - SS * (m' / den)
 *   w   = bf16 round-to-nearest-even of p'
 * with constants rounded to fp32 once from double: B1 = beta1,
 * B1c = 1 - beta1, B2 = beta2, B2c = 1 - beta2, SS = lr / (1 - beta1^t),
 * BC2S = sqrt(1 - beta2^t), DEC = 1 - lr * weight_decay, EPS = eps, where
 * beta^t is t successive double multiplications starting from 1.0.
 * An unfused step (zs_reduce_shard, then this call with its output as the
 * single fp32 contribution) gives the same bits.
 *
 *   p, m, v   device, S floats each, updated in place (pairwise disjoint)
 *   w_out     device, S uint16 (bf16 working shard), written
 *   S         >= 0
 *   contribs  host array of n_contrib device pointers, S elements of dtype
 *   n_contrib 1..ZS_MAX_D
 *   dtype     ZS_BF16 or ZS_F32
 *   hp        host pointer to the hyperparameters
 * Errors: ZS_EINVAL (NULLs, alignment, hyperparameters out of range),
 * ZS_EALIAS (p, m, v, w_out overlap each other or a contribution),
 * ZS_EUNSUPPORTED.
 */
zs_status zs_adamw_step(float* p, float* m, float* v, uint16_t* w_out, int64_t S,
                        const void* const* contribs, int32_t n_contrib, int32_t dtype,
                        const zs_adamw_hp* hp, hipStream_t stream);

/* How the contributions of one shard are reduced (zs_reduce_shard_ex,
 * zs_adamw_step_ex), and how the step's bf16 working shard is stored.
 * All fields 0 except replicas = 1 is the flat reduce of zs_reduce_shard /
 * zs_adamw_step, which always multiply by 1/D (the averaged gradient); a
 * caller that wants another multiplier (1 for the plain sum of the
 * reduce-scatter diagram in [GPT8] "AllGather vs AllReduce", or a
 * loss-scale factor) sets scale here.
 *
 * working_shard_hint (zs_adamw_step_ex only; zs_reduce_shard_ex ignores it):
 *   ZS_W_STREAM  non-temporal stores, as every other stream of the step: the
 *                default, for a working shard read much later;
 *   ZS_W_KEEP    ordinary stores that allocate in the caches (L2 and the
 *                memory-side Infinity Cache), for a caller that reads the
 *                working shard right after -- the all-gather of the same unit,
 *                [ZT] section 5.1 / [GPT8] "The Lifecycle of a Parameter".
 *                The gather then reads it from the cache, so the shard crosses
 *                HBM once (written back later) instead of twice (written, then
 *                read). The values are the same bits either way. */
#define ZS_W_STREAM 0
#define ZS_W_KEEP   1
typedef struct {
    int32_t replicas;               /* R >= 1 replica groups (HYBRID_SHARD nodes) */
    int32_t round_to_reduce_dtype;  /* 0 or 1: each collective's output is held
                                       in the reduce dtype                        */
    double scale;                   /* finite, and finite once rounded to fp32;
                                       the one multiplier of the reduced sum,
                                       rounded to fp32 once; 0 means 1 / (R * D)  */
    int32_t working_shard_hint;     /* ZS_W_STREAM or ZS_W_KEEP                   */
    int32_t reserved;               /* must be 0                                  */
} zs_reduce_opts;

/*
 * zs_reduce_shard_ex -- reduce-scatter arithmetic under HYBRID_SHARD and/or
 * with the collectives' outputs rounded to the reduce dtype.
 *
 * [GPT8] "Sharding Strategies" and "HYBRID_SHARD: The Multi-Node Strategy":
 * parameters are fully sharded over the D GPUs of a node and replicated
 * over R nodes; each node reduce-scatters over its local ranks, then the
 * nodes all-reduce their shards. [RP] section 2 (reduce_dtype bf16) and
 * [GPT8] "Mixed Precision" (reduce_dtype fp32) give the dtype the
 * collectives communicate in. For i < S, with contributions replica-major
 * (contribs[j*D + k] = local rank k of node j):
 *   s_j = ((c_{j,0} + c_{j,1}) + ...) + c_{j,D-1}      fp32, per node j
 *   s_j = round_to_reduce_dtype(s_j)                   if opts->round...
 *   t   = ((s_0 + s_1) + ...) + s_{R-1}                fp32
 *   t   = round_to_reduce_dtype(t)                     if opts->round...
 *   grad_out[i] = t * float(1 / (R * D))
 * where round_to_reduce_dtype is bf16 round-to-nearest-even widened back
 * (exact identity for fp32); with opts->scale != 0 the last line multiplies
 * by float(opts->scale) instead. opts == NULL means R = 1, no rounding,
 * scale 1 / D.
 *
 *   contribs  host array of R * D device pointers (R * D <= ZS_MAX_D), each
 *             to S elements of dtype
 *   D         contributions per node, >= 1
 *   opts      host pointer or NULL
 * Other arguments and errors as zs_reduce_shard; ZS_EINVAL also for
 * replicas < 1, round_to_reduce_dtype not 0/1, R * D > ZS_MAX_D, a scale
 * that is not finite, an unknown working_shard_hint or reserved != 0.
 */
zs_status zs_reduce_shard_ex(const void* const* contribs, int32_t D, const zs_reduce_opts* opts,
                             int32_t dtype, int64_t S, float* grad_out, hipStream_t stream);

/*
 * zs_adamw_step_ex -- zs_adamw_step with the reduce of zs_reduce_shard_ex:
 * the gradient is the grad_out value of zs_reduce_shard_ex for these
 * contributions and opts (never stored, scale included), then the AdamW
 * update of zs_adamw_step; the working shard is stored as
 * opts->working_shard_hint asks.
 * Arguments and errors as zs_adamw_step and zs_reduce_shard_ex.
 */
zs_status zs_adamw_step_ex(float* p, float* m, float* v, uint16_t* w_out, int64_t S,
                           const void* const* contribs, int32_t D, const zs_reduce_opts* opts,
                           int32_t dtype, const zs_adamw_hp* hp, hipStream_t stream);

/*
 * zs_adamw_step_timed -- zs_adamw_step_ex whose kernel carries two timing
 * events: a measurement aid for benchmarks and profilers, same arithmetic,
 * same results bit for bit.
 *
 * A step with S > 0 is exactly one kernel launch. This call makes it with
 * hipExtLaunchKernel, which has the runtime record `start` at that kernel's
 * start and `stop` at its end, with no marker packets enqueued around it, so
 * hipEventElapsedTime(start, stop) times the kernel itself. (On MI355X, over
 * the 70B shard's 0.7 ms launches, these events read 0.7% above a kernel
 * trace's durations; events recorded with hipEventRecord before and after
 * each launch read 0.9% above.)
 *
 *   start, stop  distinct events created by the caller on the current device
 *                with timing enabled (hipEventCreate); each is re-recorded by
 *                this call, as by hipEventRecord, and stays the caller's
 * Other arguments and errors as zs_adamw_step_ex; ZS_EINVAL also when start
 * or stop is NULL or they are the same event. With S == 0 nothing is
 * launched and the events are not touched.
 */
zs_status zs_adamw_step_timed(float* p, float* m, float* v, uint16_t* w_out, int64_t S,
                              const void* const* contribs, int32_t D, const zs_reduce_opts* opts,
                              int32_t dtype, const zs_adamw_hp* hp, hipEvent_t start,
                              hipEvent_t stop, hipStream_t stream);

/*
 * zs_gather_unit -- the local data movement of all-gather.
 *
 * [GPT8] "AllGather vs AllReduce": afterwards every rank holds all blocks in
 * rank order; [ZT] section 5.1 gathers a block's shards into its full
 * parameters before each forward and backward. For r < D, i < S:
 *   flat_out[r*S + i] = shards[r][i]   (bit copy, padding included)
 * Tensor j of the unit is then the view flat_out[off_j, off_j + numel_j).
 *
 *   shards    host array of D device pointers, each to S elements
 *   D         1..ZS_MAX_D
 *   S         >= 0
 *   dtype     ZS_BF16 or ZS_F32
 *   flat_out  device, D * S elements
 * In place: a shard whose pointer is exactly flat_out + r * S (its own slot,
 * as in an in-place all-gather, where each rank's shard lives inside the
 * unit buffer) is already where it belongs and is not copied.
 * Errors: ZS_EINVAL, ZS_EALIAS (a shard overlaps flat_out anywhere but
 * exactly in its own slot), ZS_EUNSUPPORTED.
 */
zs_status zs_gather_unit(const void* const* shards, int32_t D, int64_t S,
                         int32_t dtype, void* flat_out, hipStream_t stream);

/* One bucket of a rank's shard (one FSDP unit's slice) for the pipelined step. */
typedef struct {
    float* p;                    /* device, S floats: fp32 master, updated in place */
    float* m;                    /* device, S floats: first moment, in place        */
    float* v;                    /* device, S floats: second moment, in place       */
    uint16_t* w_out;             /* device, S bf16: working shard, written          */
    int64_t S;                   /* >= 0; 0 skips the bucket                        */
    const void* const* sources;  /* host array of n_contrib pointers, each to S
                                    elements of the reduce dtype, in device memory
                                    or pinned host memory; read only            */
} zs_bucket;

/*
 * zs_step_pipelined -- the shard step over a sequence of buckets, with the
 * arrival of each bucket's contributions overlapped with the previous
 * bucket's fused step.
 *
 * [ZT] section 5.4 and [GPT8] "Prefetching: Hiding the Cost": FSDP issues
 * the collective of the next block while the current block computes, so
 * communication hides behind compute. Here the reduce-scatter's transfer is
 * stood in for by copies of the n_contrib contributions of bucket b from
 * `sources` into a device staging slot (slots alternate between staging0
 * and staging1), enqueued on `transfer`; the fused step of bucket b (the
 * exact arithmetic of zs_adamw_step with these contributions) runs on
 * `compute` once its copies have landed, and the copies of the bucket after
 * next wait until that step has released the slot. The first copies wait
 * for all work already enqueued on `compute`. Results are bit-identical to
 * calling zs_adamw_step on every bucket in order.
 *
 *   buckets      host array of n_buckets bucket descriptors
 *   n_buckets    >= 0
 *   n_contrib    1..ZS_MAX_D contributions per bucket
 *   dtype        ZS_BF16 or ZS_F32: element type of sources and staging
 *   staging0/1   device, n_contrib * staging_len elements each; contribution
 *                q of a bucket lands at element q * staging_len of its slot
 *   staging_len  >= every bucket's S (a multiple of 8 keeps the full-speed
 *                kernel)
 *   hp           host pointer to the hyperparameters (one step for all buckets)
 *   compute      stream that runs the steps; when all work enqueued on it by
 *                this call has completed, every copy has completed too
 *   transfer     stream that runs the copies (may equal compute: no overlap)
 * Returns after enqueuing; nothing is synchronized and no device memory is
 * allocated. The five events that order the two streams come from a
 * per-device pool in the library (created on first use, reused by later
 * calls), so a call creates no runtime object once the pool holds them.
 * Errors: ZS_EINVAL (NULLs, misalignment, a bucket larger than staging_len,
 * hyperparameters), ZS_EALIAS (any two of the buckets' p, m, v, w_out and the
 * staging slots overlap, or a source overlaps one of them), ZS_EUNSUPPORTED,
 * ZS_EHIP (a runtime call failed; buckets before the failing one may already
 * be enqueued).
 */
zs_status zs_step_pipelined(const zs_bucket* buckets, int32_t n_buckets, int32_t n_contrib,
                            int32_t dtype, void* staging0, void* staging1, int64_t staging_len,
                            const zs_adamw_hp* hp, hipStream_t compute, hipStream_t transfer);

/*
 * zs_step_pipelined_static -- zs_step_pipelined for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc. The caller passes the buckets (inputs and
 * outputs) only; the staging slots live in a device array of the library
 * (two slots of 64 MiB, 128 MiB in all on each device that runs this call,
 * held until the process ends). A bucket whose n_contrib contributions do
 * not fit one slot is staged and stepped in pieces of at most
 * P = floor(64 MiB / (n_contrib * element size) / 1024) * 1024 elements
 * (P >= 262,144), so there is no limit on a bucket's size; the results are
 * bit-identical to zs_step_pipelined (and to zs_adamw_step on every bucket),
 * the step being elementwise. Sources may be device or pinned host memory.
 *
 * The first call on a device sets up that device's staging array address and
 * five events; no call allocates device memory or calls an allocating
 * library routine. Every call on one device shares the same staging array:
 * calls whose work overlaps in time on one device (enqueued on different
 * compute streams, or from several threads) race on it and on its events;
 * calls enqueued one after another on the same compute stream are ordered
 * (each call's first copies wait for all work already on `compute`).
 *
 *   buckets, n_buckets, n_contrib, dtype, hp, compute, transfer
 *                as zs_step_pipelined (no staging arguments)
 * Errors: as zs_step_pipelined; ZS_EHIP also when the staging array's
 * set-up fails.
 */
zs_status zs_step_pipelined_static(const zs_bucket* buckets, int32_t n_buckets,
                                   int32_t n_contrib, int32_t dtype, const zs_adamw_hp* hp,
                                   hipStream_t compute, hipStream_t transfer);

/*
 * zs_reshard -- re-shard one unit from D shards to D2 shards, on the device.
 *
 * [GPT8] "Checkpointing with FSDP": a sharded state dict resumes only on
 * the same GPU count, while the full (gathered) state dict loads on any
 * count. This is the full state dict's gather followed by a fresh split,
 * in one pass with no flat buffer: for new rank r2 and j < S2, with
 * i = r2 * S2 + j,
 *   dst[r2][j] = src[i / S][i % S]   if i < N   (bit copy)
 *   dst[r2][j] = +0                  if i >= N  (the new padding)
 *
 *   src   host array of D device pointers, each to S = ceil(N / D) elements
 *   dst   host array of D2 device pointers, each to S2 = ceil(N / D2)
 *   N     real (unpadded) elements of the unit, >= 0
 *   dtype ZS_BF16 or ZS_F32 (2- or 4-byte elements; p, m, v and w are
 *         re-sharded one array at a time)
 * Errors: ZS_EINVAL (counts out of range, S or S2 not the layout's, NULLs,
 * misalignment), ZS_EALIAS (a dst shard overlaps another dst or any src),
 * ZS_EUNSUPPORTED.
 */
zs_status zs_reshard(const void* const* src, int32_t D, int64_t S, int64_t N, int32_t dtype,
                     void* const* dst, int32_t D2, int64_t S2, hipStream_t stream);

/* Layout and step of one rank's shard checkpoint. S = ceil(N / D). */
typedef struct {
    int32_t rank;   /* 0 <= rank < D                      */
    int32_t D;      /* ranks the state was sharded over   */
    int64_t N;      /* real elements of the sharded state */
    int64_t S;      /* elements per rank shard            */
    int64_t step;   /* optimizer steps taken, >= 0        */
} zs_shard_info;

/*
 * Shard checkpoints: each rank saves its own shard (p, m, v fp32 and w
 * bf16, S elements each) to its own file -- [GPT8] "Checkpointing with
 * FSDP", sharded state dict, and "Shared Storage for Checkpoints": every
 * rank writes its own shard file concurrently. A checkpoint taken at D
 * ranks loads back at D (zs_shard_load) or at any D2
 * (zs_shard_load_resharded), each new rank reading only the byte ranges it
 * owns from the old files.
 *
 * File format (little-endian). Header page, bytes [0, 4096):
 *   0 char[8] "ZSSHARD1"   8 uint32 version (1)   12 uint32 header bytes (4096)
 *   16 int32 rank   20 int32 D   24 int64 N   32 int64 S   40 int64 step
 *   48 int64 CRC block bytes (16 MiB)
 *   56 + 48 i, i = 0..3 (p, m, v, w): char[8] name, int32 dtype (ZS_F32 or
 *      ZS_BF16), uint32 0, uint64 data offset, uint64 data bytes, uint64 CRC
 *      table offset, uint64 CRC blocks
 *   4092 uint32 CRC-32C of bytes [0, 4092)
 * then the four arrays at 4096-aligned offsets, then per array one uint32
 * CRC-32C (Castagnoli: reflected polynomial 0x82F63B78, initial value and
 * final xor 0xFFFFFFFF) per 16 MiB block of its data. A file is written as
 * path + ".tmp" and
 * renamed into place when complete.
 *
 * Unlike the kernel entry points these calls SYNCHRONIZE `stream` (the
 * state must be final before it is saved, and loaded data is complete
 * when they return), move data through a 64 MiB pinned host buffer they
 * allocate and free, and do file IO. The state pointers are device memory.
 * Errors: ZS_EINVAL (arguments), ZS_EALIAS (state arrays overlap), ZS_EIO
 * (open/read/write failure, bad magic, version or header, a checksum
 * mismatch, files that are not ranks 0..D-1 of one checkpoint), ZS_EHIP.
 */
zs_status zs_shard_save(const char* path, const zs_shard_info* info, const float* p,
                        const float* m, const float* v, const uint16_t* w, hipStream_t stream);
zs_status zs_shard_info_read(const char* path, zs_shard_info* info);
zs_status zs_shard_load(const char* path, float* p, float* m, float* v, uint16_t* w, int64_t S,
                        zs_shard_info* info_out, hipStream_t stream);
/* paths: host array of D file names, paths[r] = rank r's file of one
 * checkpoint; fills rank `rank` of a D2-way sharding (S2 = ceil(N / D2)),
 * the new padding +0; info_out (may be NULL) gets rank, D2, N, S2, step. */
zs_status zs_shard_load_resharded(const char* const* paths, int32_t D, int32_t rank, int32_t D2,
                                  float* p, float* m, float* v, uint16_t* w, int64_t S2,
                                  zs_shard_info* info_out, hipStream_t stream);

/*
 * zs_adamw_step_host -- the AdamW update of zs_adamw_step on HOST memory,
 * on host cores (ZeRO-Offload's optimizer step).
 *
 * [ZT] section 8: the Adam optimizer state moves to CPU memory; each step
 * the gradients go to the CPU and the updated weights come back. This is
 * that CPU step: for i < S, with g = grad[i] (the reduced fp32 gradient, as
 * zs_reduce_shard writes it), exactly the operations of zs_adamw_step with
 * one fp32 contribution, in the same order and rounding, so the results are
 * bit-identical to the device step. Runs synchronously on `threads` host
 * threads (the calling thread is one of them), vectorized with AVX2 where
 * the CPU has it; denormals are kept whatever the caller's MXCSR.
 *
 *   p, m, v  host, S floats, updated in place;  w_out host, S bf16, written
 *   grad     host, S floats, read
 *   threads  1..1024
 * Errors: ZS_EINVAL (NULLs, misalignment, threads, hyperparameters),
 * ZS_EALIAS (any two of p, m, v, w_out, grad overlap).
 */
zs_status zs_adamw_step_host(float* p, float* m, float* v, uint16_t* w_out, int64_t S,
                             const float* grad, const zs_adamw_hp* hp, int32_t threads);

/*
 * zs_offload_step -- one ZeRO-Offload shard step: reduce on the device,
 * gradient down, AdamW on host cores, working shard up.
 *
 * [ZT] section 8 (cost: gradients to the CPU and weights back over PCIe
 * every step). Enqueues the zs_reduce_shard reduce of the D device
 * contributions into grad_dev on `stream`, then copies grad_dev to
 * grad_host in chunks of `chunk` elements on `stream`; as each chunk lands
 * the host steps it (zs_adamw_step_host arithmetic on p, m, v, w_host) and
 * enqueues its copy w_host -> w_dev on `h2d_stream`. Returns when the host
 * work is done; the last working-shard copies may still be in flight on
 * h2d_stream (synchronize it before reading w_dev or rewriting w_host).
 * Results are bit-identical to zs_adamw_step on the same contributions.
 *
 *   contribs   host array of D device pointers, S elements of dtype each
 *   grad_dev   device, S floats (scratch, written)
 *   grad_host  host, S floats (written; pinned memory makes the copies async)
 *   p, m, v    host, S floats, updated in place
 *   w_host     host, S bf16 (written; pinned for async copies)
 *   w_dev      device, S bf16 (written by the copies)
 *   threads    1..1024 host threads;  chunk  >= 1 elements per pipeline chunk
 * Errors: as zs_reduce_shard and zs_adamw_step_host; ZS_EALIAS also when
 * grad_dev and w_dev overlap each other or a contribution.
 */
zs_status zs_offload_step(const void* const* contribs, int32_t D, int32_t dtype, int64_t S,
                          float* grad_dev, float* grad_host, float* p, float* m, float* v,
                          uint16_t* w_host, uint16_t* w_dev, const zs_adamw_hp* hp,
                          int32_t threads, int64_t chunk, hipStream_t stream,
                          hipStream_t h2d_stream);

/*
 * zs_stream_ceiling -- a measurement aid, not part of the step: moves the
 * fused step's exact memory streams with none of its arithmetic (reads n
 * contributions and p, m, v; writes p, m, v and w), with the fused kernel's
 * launch shape, lane map and cache hints, so that the step kernel can be
 * read against what HBM delivers for its own mix of streams. The values it
 * writes are placeholders: p, m, v and w are garbage afterwards. Processes
 * the first 1024 * floor(S / 1024) elements; every buffer 16-byte aligned.
 * Errors: ZS_EINVAL, ZS_EALIAS, ZS_EUNSUPPORTED as zs_adamw_step.
 */
zs_status zs_stream_ceiling(float* p, float* m, float* v, uint16_t* w, int64_t S,
                            const void* const* contribs, int32_t n, int32_t dtype,
                            hipStream_t stream);

/*
 * zs_stream_ceiling_timed -- zs_stream_ceiling whose one kernel launch records
 * `start` and `stop` at its own start and end, as zs_adamw_step_timed does
 * for the step, so that the two are timed alike.
 *   start, stop  as zs_adamw_step_timed
 * Errors: as zs_stream_ceiling; ZS_EINVAL also when start or stop is NULL or
 * they are the same event. With S < 1024 nothing is launched and the events
 * are not touched.
 */
zs_status zs_stream_ceiling_timed(float* p, float* m, float* v, uint16_t* w, int64_t S,
                                  const void* const* contribs, int32_t n, int32_t dtype,
                                  hipEvent_t start, hipEvent_t stop, hipStream_t stream);

/*
 * zs_hbm_probe -- a measurement aid, not part of the step: the memory
 * system's own rate for one stream direction, a copy or a triad, so that the
 * step kernel's mix of reads and writes can be read against what HBM gives
 * each direction alone and a plain mix with the same ratio. Non-temporal 16-byte vector accesses in grid-stride order, on a
 * grid of 256-thread workgroups that covers the buffer (blocks_per_cu = 0)
 * or on a persistent grid of blocks_per_cu workgroups per CU:
 *
 *   ZS_PROBE_READ   reads bytes of buf (two vectors per lane in flight); may
 *                   write 16 bytes at buf2 (a sink that keeps the loads)
 *   ZS_PROBE_WRITE  writes bytes of buf (element i of each 16-byte vector v:
 *                   {v mod 2^32, v >> 32, 0x5a5a5a5a, 0} as uint32 words)
 *   ZS_PROBE_COPY   copies bytes of buf to buf2
 *   ZS_PROBE_TRIAD  two reads per write, the fused step's ratio in three
 *                   streams: buf holds 2 * bytes, buf2[i] = buf[i] ^
 *                   buf[bytes + i] for the bytes of buf2 (XOR of 32-bit words)
 *
 *   bytes           a multiple of 16 (per stream); 0 returns ZS_OK with no launch
 *   buf, buf2       16-byte aligned device pointers; buf2 unused for WRITE;
 *                   for READ, COPY and TRIAD buf2 must not overlap buf
 *   blocks_per_cu   0..16
 * Errors: ZS_EINVAL (kind, sizes, alignment, NULL), ZS_EALIAS, ZS_EHIP.
 */
enum { ZS_PROBE_READ = 0, ZS_PROBE_WRITE = 1, ZS_PROBE_COPY = 2, ZS_PROBE_TRIAD = 3 };
zs_status zs_hbm_probe(int32_t kind, void* buf, void* buf2, int64_t bytes,
                       int32_t blocks_per_cu, hipStream_t stream);

/*
 * Many tensors at once. A zs_multi is a host object that describes T tensors
 * (their gradients, and for the step their parameters and moments): it is
 * checked once, when it is made, and every later call reads the checked
 * description. Its image -- 80 bytes for each chunk of at most ZS_MULTI_CHUNK
 * elements of a tensor, one chunk a workgroup -- is copied by the caller to
 * device memory once and read there by the kernels.
 */
#define ZS_MULTI_CHUNK 4096

#define ZS_STATE_NONE 0  /* gradients only (zs_grad_norm)                       */
#define ZS_STATE_F32  1  /* m and v are fp32                                    */
#define ZS_STATE_8BIT 2  /* m and v are 8-bit codes with one scale byte per 256 */

typedef struct {
    float* p;          /* device, numel floats: fp32 master, updated in place       */
    void* m;           /* device, first moment: numel floats, or numel code bytes   */
    void* v;           /* device, second moment, likewise                           */
    uint8_t* m_scale;  /* device, ceil(numel / 256) scale bytes (ZS_STATE_8BIT),
                          else NULL                                                 */
    uint8_t* v_scale;  /* likewise                                                  */
    uint16_t* w_out;   /* device, numel bf16, written; NULL: no working copy        */
    const void* g;     /* device, numel gradient elements of the table's dtype      */
    int64_t numel;     /* >= 0                                                      */
} zs_multi_tensor;

typedef struct zs_multi zs_multi;

/*
 * zs_multi_create -- check a table of T tensors and make its zs_multi (host
 * memory of the library; no GPU work). The tensors may be of any sizes and
 * start at any address that their element types allow (views into a flat unit,
 * end to end). The table itself is copied.
 *
 *   tensors  host array of T descriptors (may be NULL when T == 0); with
 *            ZS_STATE_NONE only g and numel are read
 *   state    ZS_STATE_NONE, ZS_STATE_F32 or ZS_STATE_8BIT
 *   dtype    ZS_BF16 or ZS_F32: element type of every gradient
 *   out      receives the object
 * Errors: ZS_EINVAL (NULLs, misalignment, sizes), ZS_EALIAS (a written array
 * -- p, m, v, their scales, w_out -- overlaps another written array or a
 * gradient, of the same tensor or another: so a tensor listed twice),
 * ZS_EUNSUPPORTED (state, dtype).
 */
zs_status zs_multi_create(const zs_multi_tensor* tensors, int32_t T, int32_t state,
                          int32_t dtype, zs_multi** out);

/* zs_multi_image -- the host bytes that the caller copies, unchanged, to a
 * 16-byte aligned device buffer of its own and passes as `image` below. *bytes
 * is 0 when no tensor has an element. The pointer lives as long as the object. */
zs_status zs_multi_image(const zs_multi* multi, const void** image, int64_t* bytes);

/* zs_multi_destroy -- free the host object (NULL is allowed). Work already
 * enqueued does not read it; that work reads the device image. */
zs_status zs_multi_destroy(zs_multi* multi);

/* How 8-bit moments are rounded (zs_adamw_multi; ignored for ZS_STATE_F32). */
typedef struct {
    int32_t stochastic;  /* 0: to nearest, ties to even; 1: stochastically  */
    int32_t reserved;    /* must be 0                                       */
    uint64_t seed;       /* of the random numbers; a new one for each step  */
} zs_round_opts;

/*
 * zs_adamw_multi -- AdamW over every tensor of a table, in one launch.
 *
 * Per element, with g = widen(gradient) * *grad_scale (one fp32 product; no
 * product when grad_scale is NULL), the update of zs_adamw_step, operation by
 * operation: with ZS_STATE_F32 the results are the bits that zs_adamw_step gives
 * for each tensor and the single fp32 contribution g.
 *
 * With ZS_STATE_8BIT the moments are held as codes, and the update reads their
 * values, computes m' and v' as above and encodes them again (p' and w use m' and
 * v' before they are encoded). There p' = p * DEC - SS * (m' / den) is held to a bound
 * instead of an operation order, since roots and divisions rounded to the last bit
 * would cost more than the memory traffic: within 2^-21 |SS * (m' / den)| +
 * 2^-24 (|p * DEC| + |p'|) + (1 + SS / 2) 2^-149 of the formula's value for these m' and
 * v' wherever m' / den and p' are in fp32's range, the same in every run. With EPS * BC2S <
 * 2^-38, EPS > 2^125 or a beta in (0, 2^-60), p' is the fp32 step's, bit for bit; BC2S grows
 * with the step, so with a very small EPS early steps may be of that kind and later ones not
 * (none is with EPS = 1e-8 and 1 - beta2 > 1.4e-7).
 *
 * The codes: blocks of 256 elements, counted from the tensor's first element, share a
 * scale byte s, and a code c stands for
 *   m:  +-float_of_bits((c & 127) << 20) * 2^(s - 15)     (sign in bit 7)
 *   v:    float_of_bits(c << 20)         * 2^(s - 31)
 * -- a float with 3 bits of mantissa and 4 (m) or 5 (v) of exponent, whose
 * smallest values are subnormal. s = 255 marks a block that holds an infinity
 * or NaN: all its values are NaN. Zeroed codes and scales stand for 0. To
 * encode a block, with u the fp32 bits of its largest magnitude:
 *   s = 255 if u >= 0x7f800000 (all codes 0), else
 *       min(254, (u + 0xfffff) >> 23), for v at least 11
 * (the largest magnitude is at most the top code's value), and per element, with
 * b the fp32 bits of |x| * 2^(15 - s) (v: 2^(31 - s)):
 *   c = min(127 (v: 255), (b + a) >> 20), a = 0x7ffff + ((b >> 20) & 1) to nearest;
 * for v at least 1 when x > 0, so that a positive v never becomes 0. Stochastic
 * rounding takes a = (r16 << 4) | 8 with 16 random bits r16: it rounds up with
 * the probability that keeps the mean, so that slow changes of v (1 - beta2 of
 * it a step, less than half a code) are not lost. The random bits of element i of
 * tensor t, the low 16 of r for m and the high 16 for v, are, in 32-bit
 * arithmetic,
 *   mix(x): x *= 0x6a09e667; x ^= x >> 15; x *= 0xbb67ae85; x ^= x >> 16
 *   key = mix(mix(seed_lo + 0x9e3779b9 * (t + 1)) + seed_hi),  r = mix(i ^ key)
 * -- a cheap hash: each element's bits are uniform, so that no rounding is biased, but
 * those of elements 2^27 to 2^31 apart in one tensor are correlated, by up to 0.22.
 *
 *   multi       a table with ZS_STATE_F32 or ZS_STATE_8BIT
 *   image       device, 16-byte aligned: the copy of the table's image
 *   hp          host pointer to the hyperparameters (parameter groups with
 *               others are tables and calls of their own)
 *   grad_scale  device pointer to one float, or NULL; read when the kernel runs
 *               (zs_grad_norm's clip factor, a loss scale's inverse)
 *   round       host pointer, or NULL: to nearest
 * Errors: ZS_EINVAL, ZS_EALIAS (grad_scale or image lies in an array that the
 * step writes). Tables without elements enqueue nothing.
 */
zs_status zs_adamw_multi(const zs_multi* multi, const void* image, const zs_adamw_hp* hp,
                         const float* grad_scale, const zs_round_opts* round, hipStream_t stream);

/*
 * zs_state8_layout -- where T tensors' 8-bit moments start in one buffer (host
 * only): offsets_out[t] is a multiple of 1024, tensor after tensor;
 * offsets_out[T] is the buffer's length in codes. The scale bytes of tensor t
 * start at offsets_out[t] / 256 of a buffer of offsets_out[T] / 256 bytes, so the
 * whole buffer can be decoded in one call. A convenience: zs_multi_create takes
 * any other placement too.
 * Errors: ZS_EINVAL, ZS_EUNSUPPORTED as zs_unit_layout.
 */
zs_status zs_state8_layout(const int64_t* numels, int32_t T, int64_t* offsets_out);

#define ZS_STATE8_M 0  /* signed codes   */
#define ZS_STATE8_V 1  /* unsigned codes */

/*
 * zs_state8_encode, zs_state8_decode -- fp32 moments to 8-bit codes, rounded to
 * nearest (starting 8-bit moments from a 32-bit run or a checkpoint), and codes to
 * the values they stand for (checkpoints through zs_shard_save, re-sharding).
 * Encoding what was decoded gives the same values where the blocks of 256 hold the
 * same elements (but for blocks whose largest magnitude is below 2^-126). Shards of
 * other lengths have other blocks, whose values are rounded once more: by at most half
 * a code, 2^-4 of the value or half of the new block's smallest step (v: all of it).
 *
 *   x       device, S floats; for ZS_STATE8_V a negative one counts as NaN
 *   kind    ZS_STATE8_M or ZS_STATE8_V
 *   codes   device, S bytes;  scales  device, ceil(S / 256) bytes
 *   dtype   ZS_F32 (every value exact) or ZS_BF16 (exact down to 2^-133)
 *   out     device, S elements of dtype
 * Errors: ZS_EINVAL, ZS_EALIAS (x overlaps codes or scales, or these each other;
 * out overlaps codes or scales), ZS_EUNSUPPORTED.
 */
zs_status zs_state8_encode(const float* x, int64_t S, int32_t kind, uint8_t* codes,
                           uint8_t* scales, hipStream_t stream);
zs_status zs_state8_decode(const uint8_t* codes, const uint8_t* scales, int64_t S, int32_t kind,
                           int32_t dtype, void* out, hipStream_t stream);

#define ZS_NORM_WORKSPACE 32768  /* bytes of workspace zs_grad_norm needs */

/*
 * zs_grad_norm -- the L2 norm over the gradients of a table, and the factor that
 * brings it down to max_norm.
 *
 *   sumsq[0]     = sum of g * g over every element, in fp64 (exact products;
 *                  the order of the sum depends on the table alone: on
 *                  the tensors' sizes and, for each of more than
 *                  ZS_MULTI_CHUNK elements, on the place of g
 *                  (ZS_STATE_NONE) or p (ZS_STATE_F32) modulo 64 elements.
 *                  Equal gradients at other places, or in a table of another
 *                  state, may give other last bits)
 *   norm_coef[0] = float(sqrt(sumsq))
 *   norm_coef[1] = float(c) for c = max_norm / (sqrt(sumsq) + 1e-6) < 1, else 1
 *                  (NaN if the sum is NaN; 0 if it is infinite; always 1 when
 *                  max_norm is infinite)
 * norm_coef + 1 is what zs_adamw_multi takes as grad_scale. When the ranks of a
 * data-parallel group hold parts of the gradients, zs_clip_coef joins their sums.
 *
 *   multi, image  as zs_adamw_multi, with any state
 *   max_norm      > 0, or infinity: never clip
 *   sumsq         device, one double, 8-byte aligned
 *   norm_coef     device, two floats
 *   workspace     device, ZS_NORM_WORKSPACE bytes, 16-byte aligned, zeroed by the
 *                 caller before its first use; each call leaves it ready for the
 *                 next one. Calls that may run at the same time (other streams,
 *                 graphs) need one each
 * A table without elements gives 0, 0 and 1.
 * Errors: ZS_EINVAL, ZS_EALIAS (outputs and workspace overlap, or one of them a
 * gradient or the image).
 */
zs_status zs_grad_norm(const zs_multi* multi, const void* image, double max_norm, double* sumsq,
                       float* norm_coef, void* workspace, hipStream_t stream);

/*
 * zs_clip_coef -- norm_coef of zs_grad_norm for the sum, in rank order and fp64,
 * of D ranks' sums of squares.
 *   sumsq     host array of D device pointers, each to one double
 *   D         1..ZS_MAX_D
 * Errors: ZS_EINVAL, ZS_EALIAS (norm_coef overlaps a sum).
 */
zs_status zs_clip_coef(const double* const* sumsq, int32_t D, double max_norm, float* norm_coef,
                       hipStream_t stream);

/*
 * Microscaled 4-bit floating point: blocks of 32 elements share a power of two
 * 2^(s - 127) with s one byte, and each element is +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}
 * of it in 4 bits (sign in bit 3, the values in order in bits 0-2), element 2k in
 * the low and 2k + 1 in the high half of byte k. s = 255 marks a block of NaN.
 * A working shard takes 4.25 bits an element on the way to the gather.
 *
 * zs_quantize_mx4 -- a shard to that form. s = max(0, e - 2) with e the fp32
 * exponent byte of the block's largest magnitude (255 with all codes 0 if that is
 * not finite); |x| * 2^(127 - s) is rounded to the nearest value, ties to the even
 * code, and what is over 6 becomes 6. Signs are kept, of zeros too. The last block
 * may be short, and the last half byte of an odd shard is 0.
 *
 *   src     device, S elements of dtype (ZS_BF16 or ZS_F32)
 *   codes   device, ceil(S / 2) bytes;  scales  device, ceil(S / 32) bytes
 * Errors: ZS_EINVAL, ZS_EALIAS, ZS_EUNSUPPORTED.
 */
zs_status zs_quantize_mx4(const void* src, int32_t dtype, int64_t S, uint8_t* codes,
                          uint8_t* scales, hipStream_t stream);

/*
 * zs_gather_unit_mx4 -- zs_gather_unit from shards in that form:
 *   flat_out[r*S + i] = value of element i of shard r, for r < D, i < S,
 * rounded to dtype (to nearest even; every value that zs_quantize_mx4 writes is
 * exact in bf16 and fp32).
 *
 *   codes, scales  host arrays of D device pointers
 *   dtype          ZS_BF16 or ZS_F32;  flat_out  device, D * S elements
 * Errors: ZS_EINVAL, ZS_EALIAS (flat_out overlaps codes or scales),
 * ZS_EUNSUPPORTED.
 */
zs_status zs_gather_unit_mx4(const uint8_t* const* codes, const uint8_t* const* scales, int32_t D,
                             int64_t S, int32_t dtype, void* flat_out, hipStream_t stream);

/*
 * zs_reduce_shard_norm -- zs_reduce_shard_ex that also takes the sum of the
 * squares of what it writes, in the same pass: the clipped step of a rank whose
 * gradient is spread over the buckets of several units. Each bucket is reduced
 * when its contributions are there; after the last one norm_coef is that of the
 * whole gradient (one rank holding all of it: the D simulated ranks' shards; where
 * several ranks hold parts, zs_clip_coef joins their sums).
 *
 *   grad_out[i]  = the bits of zs_reduce_shard_ex
 *   sumsq[0]     = (accumulate ? sumsq[0] : 0) + sum of grad_out[i]^2, in fp64
 *                  (exact products; the order of the sum depends on S and on whether
 *                  every buffer is 16-byte aligned, on nothing else)
 *   norm_coef[0], norm_coef[1] = of sumsq[0], as zs_grad_norm
 *
 *   contribs, D, opts, dtype, S, grad_out  as zs_reduce_shard_ex
 *   max_norm     > 0, or infinity
 *   sumsq        device, one double;  norm_coef  device, two floats, or NULL
 *   accumulate   0 or 1: calls on one stream in turn add up
 *   workspace    device, ZS_NORM_WORKSPACE bytes, as zs_grad_norm (and shared with
 *                it, by calls that do not run at the same time)
 * With S == 0 and accumulate == 0 the sum is 0 and is written.
 * Errors: as zs_reduce_shard_ex and zs_grad_norm; ZS_EINVAL also when accumulate is
 * not 0 or 1.
 */
zs_status zs_reduce_shard_norm(const void* const* contribs, int32_t D, const zs_reduce_opts* opts,
                               int32_t dtype, int64_t S, float* grad_out, double max_norm,
                               double* sumsq, float* norm_coef, int32_t accumulate,
                               void* workspace, hipStream_t stream);

/*
 * zs_adamw_step_clip -- zs_adamw_step_ex whose gradient, the grad_out value of
 * zs_reduce_shard_ex, is multiplied by *grad_scale (one fp32 product, rounded) before
 * the update: bit for bit what zs_adamw_multi gives for the gradient grad_out.
 * With one fp32 contribution, zs_reduce_shard_norm's grad_out, and norm_coef + 1 this
 * is the clipped shard step; with the D contributions and the inverse of a loss scale
 * no reduced gradient is stored.
 *
 *   grad_scale  device, one float, read when the kernel runs
 * Other arguments and errors as zs_adamw_step_ex; ZS_EINVAL also when grad_scale is
 * NULL or misaligned, ZS_EALIAS when it lies in p, m, v or w_out.
 */
zs_status zs_adamw_step_clip(float* p, float* m, float* v, uint16_t* w_out, int64_t S,
                             const void* const* contribs, int32_t D, const zs_reduce_opts* opts,
                             int32_t dtype, const zs_adamw_hp* hp, const float* grad_scale,
                             hipStream_t stream);

/*
 * Block-scaled 8-bit floating point, in which a unit's matrices are multiplied.
 * A matrix's element is a code of 8 bits times 2^(s - 127) with one scale byte s for
 * each block of block_rows x 128 elements: 1 x 128 for activations and gradients
 * (128 elements of a row, along what a product sums over), 128 x 128 for weights, whose
 * transpose then has the same codes. Codes are e4m3 (sign, 4 bits of exponent, bias 7,
 * 3 of mantissa; largest 448, no infinity) or e5m2 (5 bits, bias 15, 2; largest finite
 * 57344). s = 255 marks a block of NaN. With u the fp32 bits of a block's largest
 * magnitude,
 *   s = 255 and all codes 0 if u >= 0x7f800000, else
 *       max(1, ((u + 0x1fffff) >> 23) - 8 (e5m2: 15)),
 * the smallest power of two under which the largest code holds that magnitude, and a
 * code is x * 2^(127 - s) rounded to nearest, ties to even (signs are kept, of zeros
 * too). Scales are powers of two, so that nothing but that one rounding is lost and the
 * matrix cores apply them.
 *
 * Layout: row r's codes are bytes [r * ld, r * ld + cols), ld = 128 * ceil(cols / 128),
 * followed by codes 0; the scale byte of its block c / 128 is byte
 * (r / block_rows) * lds + c / 128, lds = 4 * ceil(cols / 512), and what fills a row of
 * scale bytes is 1. Products read whole blocks: codes written by others must have the
 * zeros too.
 */
#define ZS_E4M3 3
#define ZS_E5M2 4

typedef struct {
    uint8_t* codes;      /* device, rows * ld bytes, 16-byte aligned                */
    uint8_t* scales;     /* device, ceil(rows / block_rows) * lds bytes, 4-byte aligned */
    int64_t rows;        /* 0 .. 2^31 - 1                                           */
    int64_t cols;        /* 0 .. 2^22                                               */
    int32_t type;        /* ZS_E4M3 or ZS_E5M2                                      */
    int32_t block_rows;  /* 1 or 128                                                */
} zs_f8_matrix;

/* zs_f8_layout -- bytes of codes and of scales of a rows x cols matrix (host only). */
zs_status zs_f8_layout(int64_t rows, int64_t cols, int32_t block_rows, int64_t* code_bytes,
                       int64_t* scale_bytes);

/*
 * zs_quantize_f8 -- a matrix to that form, as it is, transposed, or both from one read.
 *
 *   x      device, rows x cols elements of dtype (ZS_BF16 or ZS_F32), row r from element
 *          r * ldx on; ldx >= cols
 *   out    host pointer, rows x cols, or NULL
 *   out_t  host pointer, cols x rows, or NULL: the transpose, whose blocks run along x's
 *          columns. At least one of both; they share block_rows, not the type
 * Errors: ZS_EINVAL, ZS_EALIAS (x and the outputs overlap), ZS_EUNSUPPORTED.
 */
zs_status zs_quantize_f8(const void* x, int32_t dtype, int64_t ldx, const zs_f8_matrix* out,
                         const zs_f8_matrix* out_t, hipStream_t stream);

/*
 * zs_gather_matrix_f8 -- one matrix of a unit, from the unit's D shards straight to that
 * form: zs_gather_unit's elements [offset, offset + rows * cols) as a rows x cols matrix,
 * and zs_quantize_f8 of it, without the flat unit in between.
 *
 *   shards  host array of D device pointers, each to S elements of dtype
 *   offset  the matrix's first element in the flat unit (zs_unit_layout); the matrix ends
 *           within the D * S elements
 *   out, out_t  as zs_quantize_f8
 * Errors: ZS_EINVAL, ZS_EALIAS, ZS_EUNSUPPORTED.
 */
zs_status zs_gather_matrix_f8(const void* const* shards, int32_t D, int64_t S, int32_t dtype,
                              int64_t offset, const zs_f8_matrix* out, const zs_f8_matrix* out_t,
                              hipStream_t stream);

/*
 * zs_dequantize_f8 -- the values that a matrix in that form stands for, rounded to dtype
 * (to nearest even; exact but below 2^-126 and beyond the type's range).
 *   out  device, rows x cols elements of dtype, row r from element r * ldo on
 * Errors: ZS_EINVAL, ZS_EALIAS, ZS_EUNSUPPORTED.
 */
zs_status zs_dequantize_f8(const zs_f8_matrix* x, int32_t dtype, void* out, int64_t ldo,
                           hipStream_t stream);

/*
 * zs_matmul_f8 -- C = A B^T, or C += A B^T, over the values of two matrices in that form:
 *   c[m, n] = sum over k of a[m, k] * b[n, k]   (+ c[m, n] with accumulate)
 * for a of M x K, b of N x K. Blocks of NaN make every element that reads them NaN.
 *
 * The sum is rounded to C's type once (with accumulate after adding C's old value, in
 * fp32). For C in fp32 it is held in fp32 throughout, and the operands' values pass
 * through bf16: exact but beyond its range, at 2^128 and below 2^-133. For C in bf16 the 8-bit matrix
 * instructions form it: of 8 neighbouring products along K they drop what is below 2^-13
 * of the largest one's leading power of two, and hold the rest in fp32. It is then off by
 * at most 7 * 2^-13 of the sum of these largest products' magnitudes before the rounding to
 * bf16 (measured, of the results' norm: 2^-16 on normal data, 2^-14.5 where a few columns of
 * a are much larger than the others; to either side alike). The order of the sum depends on
 * M, N, K and the types alone.
 *
 *   c          device, M x N elements of dtype, row m from element m * ldc on; what lies
 *              between the rows is not written
 *   accumulate 0 or 1
 *   workspace  device, 16-byte aligned, zs_matmul_f8_workspace(M, N, K) bytes (NULL where
 *              that is 0), zeroed by the caller before its first use; each call leaves it
 *              ready for the next one, of any size it is large enough for. Calls that may
 *              run at the same time (other streams, graphs) need one each
 * With K = 0 the sum is 0. Errors: ZS_EINVAL (also when C has more than (2^32 - 1) / 256
 * tiles of 64 x 64), ZS_EALIAS (C or the workspace overlap an operand or each other),
 * ZS_EUNSUPPORTED.
 */
zs_status zs_matmul_f8(const zs_f8_matrix* a, const zs_f8_matrix* b, int32_t dtype, void* c,
                       int64_t ldc, int32_t accumulate, void* workspace, hipStream_t stream);
zs_status zs_matmul_f8_workspace(int64_t M, int64_t N, int64_t K, int64_t* bytes);

/*
 * zs_linear_f8 -- a linear layer over 8-bit weights: y = Q(x) w^T with Q the quantiser of
 * zs_quantize_f8 with 1 x 128 blocks, then zs_matmul_f8, with the same results. Two
 * launches, but one
 *   - with few rows (serving: one new token): M <= 16 whose codes fit a workgroup,
 *     M * (129 * ceil(K / 128) + 16) <= 79872: 16 rows up to K = 4864, 8 up to 9856, 4 up to
 *     19712, 1 up to 79232;
 *   - for other small layers: 0 < K <= 1024 and at most 256 tiles of 64 x 64 of y.
 *
 *   x     device, M x K elements of dtype, row stride ldx;  type  of its codes
 *   w     N x K, block_rows 1 or 128 (a gathered matrix)
 *   y     device, M x N elements of y_dtype, row stride ldy
 *   workspace  as zs_matmul_f8, of zs_linear_f8_workspace(M, N, K) bytes: 0 for those few
 *              rows, a fixed 8 KiB for those small layers (checked, not used), and x's codes
 *              and scales beside zs_matmul_f8's else
 * Errors: as zs_quantize_f8 and zs_matmul_f8.
 */
zs_status zs_linear_f8(const void* x, int32_t dtype, int64_t M, int64_t ldx, int32_t type,
                       const zs_f8_matrix* w, int32_t y_dtype, void* y, int64_t ldy,
                       void* workspace, hipStream_t stream);
zs_status zs_linear_f8_workspace(int64_t M, int64_t N, int64_t K, int64_t* bytes);

/*
 * zs_linear_f8_backward -- that layer's gradients from the output's gradient dy (M x N):
 *   dx = Q(dy) w             (M x K), w given transposed: w_t, K x N
 *   dw = Q(dy^T) Q(x^T)^T    (N x K), with accumulate dw += that
 * Q quantises along what each product sums over: dy by rows for dx, dy and x by columns
 * for dw. dw is usually a view into the unit's flat gradient, a contribution of
 * zs_reduce_shard.
 *
 *   dy, x      device, elements of dtype, row strides lddy, ldx
 *   dy_type    ZS_E4M3 or ZS_E5M2: of dy's codes (x's are e4m3)
 *   w_t        NULL when dx is NULL
 *   dx         device, elements of dx_dtype, row stride lddx; NULL: not computed
 *   dw         device, elements of dw_dtype, row stride lddw; NULL: not computed (x may
 *              then be NULL)
 *   workspace  as zs_matmul_f8, of zs_linear_f8_backward_workspace(M, N, K) bytes
 * Errors: as zs_quantize_f8 and zs_matmul_f8; ZS_EINVAL also when dx and dw are both NULL.
 */
zs_status zs_linear_f8_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                int32_t dtype, int64_t M, int64_t N, int64_t K, int32_t dy_type,
                                const zs_f8_matrix* w_t, int32_t dx_dtype, void* dx, int64_t lddx,
                                int32_t dw_dtype, void* dw, int64_t lddw, int32_t accumulate,
                                void* workspace, hipStream_t stream);
zs_status zs_linear_f8_backward_workspace(int64_t M, int64_t N, int64_t K, int64_t* bytes);

/* Text of the calling thread's most recent failure ("" if none). The pointer
 * stays valid until the thread's next call into the library. */
const char* zs_last_error(void);

/* ABI version of this header (major * 100 + minor). */
int32_t zs_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ZS_H_ */
