/*
 * zero_gb300.h -- C ABI of the partitioned mixed-precision ZeRO step on one
 * GB300 (sm_103a).  N data-parallel ranks are simulated inside one GPU's
 * HBM: every rank's 16-bit gradient buffer and parameter replica are
 * separate device buffers, and the owner shards of the fp32 optimizer state
 * are laid out back to back in one flat buffer.  The collectives of the
 * method (reduce-scatter, all-gather, per-bucket broadcast, the scalar
 * all-reduce of norm and overflow flag) are HBM streams fused into the
 * update kernels.
 *
 * Sources (web pages on ZeRO, cited by title and section):
 *  - "ZeRO: Memory Optimizations Toward Training Trillion Parameter Models"
 *    (summary), Sec. 3.1 mixed-precision Adam state (2+2+12 bytes/param),
 *    Sec. 5 stages P_os / P_os+g / P_os+g+p, Sec. 7 communication volume,
 *    residual states (gradient norm over the flattened buffer).
 *  - "zero-stages-simulation" README: flat contiguous partition, rank r owns
 *    chunk r; per-stage schedule table; byte-accurate accounting.
 *  - "CMU 11-868 L18: How ZeRO Cuts Data-Parallel Memory": ZeRO-1 call
 *    sequence (reduce-scatter into an FP32 shard, update, copy to 16-bit,
 *    all-gather); ZeRO-3 broadcast from owner before forward and backward.
 *
 * General conventions
 *  - Every call returns a zero_status_t.  Nothing aborts, throws or traps;
 *    on error the call launches nothing and zero_last_error() says why.
 *  - All tensor arguments are caller-owned DEVICE pointers (the caller
 *    allocates them, e.g. with PyTorch) unless a comment says "host".  The
 *    library owns only its workspace (status word, norm partials, chunk
 *    counters, and for some modes an fp32 gradient buffer of psi_pad floats).
 *  - Device pointers must be 16-byte aligned.  The 128-bit vector path runs
 *    when psi_pad (or a bucket's bounds) are multiples of 8, and for a bucket
 *    of double-buffered state also psi_pad (the second slot's offset);
 *    otherwise an element-wise path runs with the same arithmetic.
 *  - Calls are asynchronous on the given CUDA stream (a cudaStream_t passed
 *    as void*, NULL = legacy default stream).  One host thread per handle.
 *    The reduce-scatters and steps of one handle share its status word and
 *    norm partials, so they must run in order (one stream, or ordered by
 *    events); gathers may overlap them on another stream.  At most 64
 *    launches of one handle may be in flight at once: each takes the next
 *    of 64 work counters, round-robin.
 *  - The streaming kernels are launched with programmatic stream
 *    serialisation: the next one may be scheduled while the previous one
 *    drains, and waits in its first instruction until that one has
 *    completed.  Stream order is unchanged for the caller; a caller's own
 *    kernel or copy on the same stream runs after the library's work as
 *    usual, and the calls can be captured into a CUDA graph.
 *  - Elements [psi, psi_pad) are padding: gradients there are ignored, and
 *    master/m/v/params there are written as 0.
 *  - The loss scale, the count t of applied Adam steps and the live slot of
 *    double-buffered state are DEVICE-side handle state, so a step never
 *    waits for the host: an overflowing step halves the scale (floor 1.0)
 *    and leaves t unchanged without a host round trip.
 */
#ifndef ZERO_GB300_H
#define ZERO_GB300_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define ZERO_API __attribute__((visibility("default")))
#else
#define ZERO_API
#endif

typedef enum {
    ZERO_OK = 0,
    ZERO_EINVAL = 1,    /* bad argument: null/misaligned pointer, range, stage/mode mismatch */
    ZERO_ENOMEM = 2,    /* workspace allocation failed */
    ZERO_ECUDA = 3,     /* a CUDA runtime call or kernel launch failed */
    ZERO_ETIMEOUT = 4,  /* zero_get_status: a bounded wait inside a kernel gave up (staged step) */
    ZERO_ESTATE = 5     /* call sequence wrong (e.g. stage-3 step before every bucket was reduced) */
} zero_status_t;

typedef enum { ZERO_FP16 = 0, ZERO_BF16 = 1 } zero_dtype_t;

typedef enum {
    ZERO_MODE_AUTO = 0,            /* SPECULATIVE if possible, else TWO_PASS_WS for N > 4, else REREAD */
    ZERO_MODE_TWO_PASS_WS = 1,     /* pass 1 writes fp32 g_hat to workspace; pass 2 reads it */
    ZERO_MODE_TWO_PASS_REREAD = 2, /* pass 2 reduces the N gradient buffers again */
    ZERO_MODE_SPECULATIVE = 3,     /* one pass writing the shadow state slot; commit, roll back, or
                                      (one-shot step whose norm needs clipping) redo from the old slot */
    ZERO_MODE_SPECULATIVE_STAGED = 4 /* SPECULATIVE, inputs staged through shared memory by bulk
                                        async copies (stages 1/2 one-shot step; N <= 19, i.e. two
                                        stages of N*4 KiB + 24 KiB fit in 200 KiB of shared
                                        memory; psi_pad a multiple of 8; fp32 state 32-byte
                                        aligned; grads and master/m/v in device memory,
                                        not host memory; otherwise ZERO_EINVAL) */
} zero_mode_t;

/* zero_init_partition flags */
#define ZERO_F_DOUBLE_BUFFER 1u    /* master/m/v hold two slots of psi_pad floats (stages 1-3) */

#define ZERO_MAX_RANKS 64

typedef struct zero_handle* zero_handle_t;   /* opaque, library-owned */

typedef struct {
    float lr, beta1, beta2, eps, weight_decay;
    float max_norm;   /* global-norm clip threshold; <= 0 disables clipping */
    int32_t mode;     /* zero_mode_t */
} zero_hyper_t;

typedef struct {
    int32_t overflow;       /* last step skipped: a non-finite averaged gradient, or (error != 0)
                               a kernel wait that gave up */
    int32_t applied;        /* last step updated the state */
    int32_t state_slot;     /* live slot (0/1) of double-buffered master/m/v; 0 otherwise */
    int32_t error;          /* device-side error word, 0 = none; 1 = a bounded wait of the staged
                               step gave up.  Stays set until zero_set_scaler. */
    double grad_norm;       /* L2 norm of the averaged unscaled gradient of the last step; not
                               meaningful when overflow = 1 (a one-pass step stops at the
                               first non-finite value it finds) */
    double clip_coef;       /* fp32 factor applied to the gradient (1.0 when not clipping) */
    float loss_scale;       /* current loss scale, after any halving */
    float reserved;
    int64_t steps_applied;  /* t: Adam steps applied so far */
    int64_t steps_skipped;  /* steps skipped on overflow so far */
} zero_result_t;

typedef struct {
    uint64_t psi, psi_pad, shard, n_ranks, stage;
    uint64_t model_state_bytes_per_rank;  /* 16/4+12/N/2+14/N/16/N bytes x psi_pad, exact
                                             (stage 3 with a resident region: see
                                             zero_set_persistent) */
    uint64_t comm_elems_paper;            /* 2 psi_pad (stages 0-2), 3 psi_pad (stage 3) */
    uint64_t comm_elems_ring;             /* 2(N-1)/N psi_pad, 3(N-1)/N psi_pad for stage 3 */
    uint64_t hbm_read_bytes, hbm_write_bytes;   /* algorithmic HBM bytes of the last call */
    uint64_t hbm_read_total, hbm_write_total;   /* cumulative since init */
} zero_bytes_t;

/*
 * zero_init_partition -- a1: partition a flat buffer of psi parameters over
 * n_ranks simulated ranks and allocate the handle's workspace.
 *   ("zero-stages-simulation" README, flat partitioning: N near-equal
 *    contiguous chunks, rank r owns chunk r; ZeRO summary Sec. 5, P_os: N_d
 *    equal partitions.)
 * psi_pad = smallest multiple of n_ranks*align >= psi; shard = psi_pad/N;
 * offset_r = r*shard; real_r = clamp(psi - offset_r, 0, shard).
 *   psi      >= 0 (0 gives an empty step)
 *   n_ranks  1..ZERO_MAX_RANKS
 *   stage    0..3 (ZeRO-0 plain DP, P_os, P_os+g, P_os+g+p)
 *   dtype    zero_dtype_t of gradients and parameters
 *   align    >= 1 elements (8 keeps every shard 16-byte aligned)
 *   flags    ZERO_F_DOUBLE_BUFFER or 0 (stage 0 rejects it)
 *   out      host pointer receiving the handle
 * Uses the current CUDA device.  Errors: EINVAL, ENOMEM, ECUDA.
 */
ZERO_API int zero_init_partition(uint64_t psi, int n_ranks, int stage, int dtype, int align,
                        unsigned flags, zero_handle_t* out);

/*
 * zero_partition_info -- the partition (host values, exact).  offsets and
 * real are host arrays of n_ranks entries, or NULL.  Any output may be NULL.
 */
ZERO_API int zero_partition_info(zero_handle_t h, uint64_t* psi_pad, uint64_t* shard,
                        uint64_t* offsets, uint64_t* real);

/*
 * zero_set_scaler -- set the device-side loss scale, applied-step count t
 * and live state slot (0/1; must be 0 without ZERO_F_DOUBLE_BUFFER).  Used
 * before the first step and to resume from a checkpoint.  Stream-ordered.
 * The loss scale must be finite and > 0.  Errors: EINVAL, ECUDA.
 */
ZERO_API int zero_set_scaler(zero_handle_t h, float loss_scale, int64_t steps_applied,
                    int32_t state_slot, void* stream);

/*
 * zero_step -- one mixed-precision ZeRO step (a2..a8, a11).
 *   Stages 0-2: reduce the N ranks' 16-bit gradients in fixed order 0..N-1
 *   in fp32, divide by N*loss_scale (CMU notes, ZeRO-1 step 3: sum and
 *   average into an FP32 shard), test for inf/nan, form the global L2 norm
 *   (ZeRO summary, residual states: norm over the flattened gradient), clip
 *   if max_norm > 0, run AdamW on the owners' fp32 master/m/v (ZeRO summary
 *   Sec. 3.1 and Sec. 5), round to 16 bits and write every rank's replica
 *   (the all-gather; CMU notes steps 5-6).  Stage 0 all-reduces and updates
 *   N full replicas of the state (ZeRO summary Sec. 7, baseline DP).
 *   Stage 3: grads must be NULL; the N gradients were already consumed by
 *   zero_reduce_scatter_bucket calls covering [0, psi_pad) exactly once
 *   since the last step.  Stage 2 with grads NULL: the same, after
 *   zero_reduce_scatter_bucket_replicas calls.  This call finishes the norm/overflow/clip and
 *   (two-pass modes) applies Adam and writes the 16-bit shard.
 * On overflow nothing of master/m/v/params changes, the scale halves and t
 * is not advanced.
 * Speculative mode (ZERO_F_DOUBLE_BUFFER; AUTO picks it for stages 1/2):
 * one pass updates the shadow slot and the replicas assuming no clipping.
 * If the norm then calls for clipping, a second pass redoes the update
 * from the untouched old slot with the clip factor, so only clipped steps
 * pay for two passes.  Bucketed steps (stage 3, and stage 2 with NULL grads)
 * cannot re-read their gradients and use the two-pass mode when clipping.
 *   grads   host array of N device pointers, psi_pad 16-bit elements each
 *           (stages 0-2); NULL for stage 3
 *   params  host array of N device pointers to psi_pad 16-bit replicas
 *           (stages 0-2), or of 1 pointer to the psi_pad 16-bit
 *           concatenation of the owner shards (stage 3).  Replicas must
 *           equal the RNE cast of the live master on entry.
 *   master, m, v  fp32 device buffers.  Stages 1-3: psi_pad floats (the N
 *           owner shards back to back), or 2*psi_pad with
 *           ZERO_F_DOUBLE_BUFFER (slot s at offset s*psi_pad).  Stage 0:
 *           N*psi_pad floats, replica r at offset r*psi_pad.
 *   hyper   host pointer, read during the call only
 * Errors: EINVAL, ESTATE, ECUDA, ENOMEM (first two-pass call allocates the
 * fp32 workspace; make it before any stream capture).
 */
ZERO_API int zero_step(zero_handle_t h, const void* const* grads, void* const* params,
              float* master, float* m, float* v, const zero_hyper_t* hyper, void* stream);

/*
 * zero_gather_bucket -- a9: ZeRO-3 parameter gather of bucket [a, b): every
 * rank receives the owners' 16-bit values, out[r][j] = shard16[a + j].
 *   (ZeRO summary Sec. 5, P_os+g+p: the owner broadcasts a layer's
 *    parameters before its forward and again before its backward; CMU
 *    notes, ZeRO-3: ncclBroadcast from the owning GPU.)
 *   0 <= a <= b <= psi_pad.  shard16: device, psi_pad 16-bit elements.
 *   out: host array of N device pointers, b - a elements each.
 * Stage 3 only.  Errors: EINVAL, ECUDA.
 */
ZERO_API int zero_gather_bucket(zero_handle_t h, uint64_t a, uint64_t b, const void* shard16,
                       void* const* out, void* stream);

/*
 * zero_reduce_scatter_bucket -- a10: ZeRO-3 gradient reduce-scatter of
 * bucket [a, b) into the owners' shards: the a2..a5 steps restricted to the
 * bucket.  (ZeRO summary Sec. 5, P_os+g / P_os+g+p: reduce-scatter as the
 * gradients of each layer appear in backward; CMU notes, ZeRO-2/3: each
 * segment's gradients are reduced to its owner.)
 * With ZERO_F_DOUBLE_BUFFER and no clipping (mode AUTO or SPECULATIVE) the
 * bucket's AdamW update is fused here: new master/m/v go to the shadow slot
 * and the new 16-bit values straight into shard16[a, b); zero_step then
 * commits, or on overflow restores shard16 from the old master.  Otherwise
 * the averaged gradient is written to the fp32 workspace and zero_step
 * applies Adam.
 *   grads: host array of N device pointers, b - a 16-bit elements each.
 *   master, m, v, shard16: as for zero_step of stage 3 (may be NULL in
 *   two-pass modes).  Every call of one step must pass the same hyper.
 *   Buckets of one step must not overlap.  At most 4096 per step.
 * Stage 3 only.  Errors: EINVAL, ESTATE, ECUDA, ENOMEM.
 */
ZERO_API int zero_reduce_scatter_bucket(zero_handle_t h, uint64_t a, uint64_t b,
                               const void* const* grads, float* master, float* m, float* v,
                               void* shard16, const zero_hyper_t* hyper, void* stream);

/*
 * zero_reduce_scatter_gather_bucket -- zero_reduce_scatter_bucket of bucket
 * [a, b) and zero_gather_bucket of bucket [ga, gb) in one call: the
 * reduce-scatter of one layer's gradients in backward together with the
 * gather of the next layer's parameters, fetched one layer ahead.
 *   (ZeRO summary Sec. 5, P_os+g+p: in backward the parameters are gathered
 *    again in reverse order, a layer's gradients are reduce-scattered as they
 *    appear, and the next layer can be fetched while the current one is
 *    processed; "ZeRO Stage 1/2/3" guide, ZeRO-3 config: prefetch_bucket_size.)
 * The result is that of the two calls one after the other.  When both parts
 * are 8-wide (a, b - a, ga and gb - ga multiples of 8) they run as one launch
 * whose work counter hands out the reduce-scatter's chunks first and then
 * the gather's, so that the gather fills the end of the reduce-scatter;
 * otherwise the two calls are made in turn.  Either part may be empty.
 *   The two buckets must not overlap, and no out[r] may share memory with
 *   the 16-bit shard, master, m, v or a gradient row of [a, b) (ZERO_EINVAL).
 *   Arguments: those of zero_reduce_scatter_bucket, then ga, gb and out
 *   (host array of N device pointers, gb - ga elements each) as for
 *   zero_gather_bucket.  zero_bytes_moved counts both parts as this call.
 * Stage 3 only.  Errors: EINVAL, ESTATE, ECUDA, ENOMEM.
 */
ZERO_API int zero_reduce_scatter_gather_bucket(zero_handle_t h, uint64_t a, uint64_t b,
                                               const void* const* grads, float* master, float* m, float* v,
                                               void* shard16, const zero_hyper_t* hyper, uint64_t ga,
                                               uint64_t gb, void* const* out, void* stream);

/*
 * zero_reduce_scatter_bucket_replicas -- ZeRO-2 with the gradients reduced
 * during backward: the reduce-scatter of bucket [a, b) as its gradients
 * appear, after which the ranks may release or reuse their gradient
 * buffers for the next bucket (a constant-size buffer per rank).
 *   (ZeRO summary Sec. 5, P_os+g: reduce-scatter during backward, bucketized
 *    per partition, gradient memory freed; Sec. 6 CB: constant-size fused
 *    buffers; CMU notes, ZeRO-2: reduce each segment to its owner, delete.)
 * With ZERO_F_DOUBLE_BUFFER and no clipping the bucket's AdamW update and
 * its all-gather into every replica are fused here (shadow slot; replicas
 * written at once); zero_step(h, NULL grads, params, ...) then commits, or
 * on overflow restores the replicas from the old master.  Otherwise g_hat
 * goes to the fp32 workspace and that zero_step applies AdamW and writes
 * the replicas.  The buckets of one step must tile [0, psi_pad) without
 * overlap (at most 4096) and pass the same hyper.
 *   grads: host array of N device pointers, b - a 16-bit elements each
 *   params: host array of N device pointers to the psi_pad replicas
 *   master, m, v: as for zero_step (may be NULL in two-pass modes)
 * Stage 2 only.  Errors: EINVAL, ESTATE, ECUDA, ENOMEM.
 */
ZERO_API int zero_reduce_scatter_bucket_replicas(zero_handle_t h, uint64_t a, uint64_t b,
                                        const void* const* grads, float* master, float* m, float* v,
                                        void* const* params, const zero_hyper_t* hyper, void* stream);

/*
 * ZeRO++ block-quantized exchanges.  ("CMU 11-868 L18" notes, other memory
 * optimizations: ZeRO++ block-quantizes parameters from 16 bits to INT8 with
 * zero-point quantization for the forward gather, and quantizes the
 * backward reduce-scatter to INT8 or INT4.)
 * Format: blocks of ZERO_Q_BLOCK elements counted from the start of the
 * buffer (or bucket); per block lo = min and hi = max (a NaN makes both NaN),
 * scale = (hi - lo) / (2^bits - 1) in fp32, code = rint((x - lo) / scale)
 * with the subtraction and the division each rounded once, clamped to
 * [0, 2^bits - 1] (0 when scale == 0; 0 for a NaN); dequantized
 * x' = lo + code * scale (fp32 multiply, then add).  Codes: one byte per
 * element (bits = 8) or two per byte with the even element in the low nibble
 * (bits = 4); `scales` holds one {scale, lo} float pair per block.  Code
 * buffers and 16-bit buffers must be 16-byte aligned, scales 8-byte aligned.
 */
#define ZERO_Q_BLOCK 256

/* Quantize count 16-bit values (a rank's bucket gradient before the
 * reduce-scatter, qgZ).  Needs no handle: errors via zero_last_error(NULL). */
ZERO_API int zero_quantize_blocks(int dtype, int bits, const void* src16, uint64_t count, void* codes,
                         float* scales, void* stream);

/* Dequantize count values to 16 bits (RNE): what a rank computes with after
 * a quantized gather.  Needs no handle. */
ZERO_API int zero_dequantize_blocks(int dtype, int bits, const void* codes, const float* scales, uint64_t count,
                           void* out16, void* stream);

/* a9 with qwZ: the owners' 16-bit values of bucket [a, b) are quantized to
 * INT8 once and every rank r receives the codes (codes_out[r], b - a bytes)
 * and scales (scales_out[r], 2*ceil((b-a)/256) floats).  Stage 3 only.
 * Errors: EINVAL, ECUDA. */
ZERO_API int zero_gather_bucket_q8(zero_handle_t h, uint64_t a, uint64_t b, const void* shard16,
                          void* const* codes_out, float* const* scales_out, void* stream);

/* a10 with qgZ: zero_reduce_scatter_bucket whose inputs are the N ranks'
 * quantized bucket gradients (codes[r], scales[r], as zero_quantize_blocks
 * writes them for the bucket's b - a elements).  The owner sums the
 * dequantized values in rank order; everything after is as for
 * zero_reduce_scatter_bucket, and zero_step finishes the step.  Stage 3. */
ZERO_API int zero_reduce_scatter_bucket_q(zero_handle_t h, uint64_t a, uint64_t b, int bits,
                                 const void* const* codes, const float* const* scales, float* master,
                                 float* m, float* v, void* shard16, const zero_hyper_t* hyper, void* stream);

/*
 * zero_get_status -- a11: copy the device status of the last step to the
 * host struct *out (host pointer).  Synchronises the given stream.
 * Errors: EINVAL, ECUDA; ETIMEOUT (with *out filled) while the device error
 * word is set, i.e. after a staged step whose bounded wait gave up.
 */
ZERO_API int zero_get_status(zero_handle_t h, void* stream, zero_result_t* out);

/*
 * zero_debug_hold_staged -- test hook for the failure path of
 * ZERO_MODE_SPECULATIVE_STAGED.  In the next staged zero_step on this handle
 * (one-shot), CTA 0 stops issuing its bulk copies at its tile `tile` (its
 * tiles counted from 0), so its compute warps' bounded waits run out (about
 * 2 s) instead of receiving data.  No access leaves its buffers and every
 * wait ends.  That step is then skipped (overflow = 1, master/m/v and the
 * replicas unchanged, loss scale kept), the error word is set and
 * zero_get_status returns ZERO_ETIMEOUT until zero_set_scaler clears it.
 * tile < 0 clears a pending hold; a tile past CTA 0's last has no effect.
 * Errors: EINVAL (NULL handle).
 */
ZERO_API int zero_debug_hold_staged(zero_handle_t h, int64_t tile);

/*
 * zero_set_persistent -- tell a stage-3 handle that the flat region
 * [p0, psi_pad) stays replicated: every rank keeps a resident 16-bit copy of
 * it, refreshed by one gather after each update, and its buckets are not
 * gathered before forward or backward.
 *   ("ZeRO Stage 1/2/3" guide, ZeRO-3 config: param_persistence_threshold,
 *    parameters below it stay replicated; ZeRO summary Sec. 5 and Sec. 7 for
 *    the P_os+g+p memory and communication it changes.)
 * Host-only bookkeeping: it changes what zero_bytes_moved reports and
 * nothing that runs on the device (the caller makes the gathers; see the
 * package's ZeRO-3 schedule).  With psi_pers = psi_pad - p0:
 *   model_state_bytes_per_rank = 16 psi_pad / N + 2 psi_pers
 *   comm_elems_paper           = 3 psi_pad - psi_pers
 *   comm_elems_ring            = floor((N - 1)(3 psi_pad - psi_pers) / N)
 * p0 = psi_pad (the default) means no resident region.
 * Errors: EINVAL (NULL handle, stage != 3, p0 > psi_pad).
 */
ZERO_API int zero_set_persistent(zero_handle_t h, uint64_t p0);

/*
 * zero_bytes_moved -- D4/D5 accounting and algorithmic HBM bytes.
 *   (ZeRO summary Sec. 5 memory equations and Sec. 7 communication volume;
 *    "zero-stages-simulation" README: byte-accurate memory tracker and a
 *    counting interconnect.)  Host-only, exact integers.  The HBM counters
 *   count the bytes the method must move for the calls made, assuming
 *   each step applied (an overflow's rollback pass is not counted).
 */
ZERO_API int zero_bytes_moved(zero_handle_t h, zero_bytes_t* out);

/*
 * zero_step_noalloc -- the two-pass step of stages 1/2 for callers that
 * cannot allocate device memory.  The ZeRO pages have no counterpart: this
 * is a packaging of zero_step for such callers.
 * Some callers may not call cudaMalloc: code in a framework whose caching
 * allocator owns the device memory (a foreign cudaMalloc also synchronises
 * the whole device), or code under a memory budget fixed before training
 * starts.  zero_init_partition allocates a workspace, so those callers use
 * this call instead.  It takes no handle and calls no cudaMalloc, cudaFree
 * or other allocating routine.
 *   Its scratch -- the status word, the norm partials, the chunk counters
 *   and the fp32 averaged gradient -- lives in one static device array of
 *   ZERO_NOALLOC_MAX_PSI_PAD floats plus 324,960 bytes (about 16.3 MiB),
 *   which every GPU that loads the library holds until the
 *   process exits.  psi_pad above ZERO_NOALLOC_MAX_PSI_PAD is rejected
 *   with ZERO_EINVAL.
 *   The first call on a device looks up that array's device address
 *   (cudaGetSymbolAddress) and, like any first launch of a kernel, may have
 *   the driver load the library's kernels onto the device; make that first
 *   call before any stream capture.  Later calls leave the device's free
 *   memory unchanged.
 *   Every call shares the one array and overwrites what the last call left
 *   there (it clears the status word first): calls that overlap on the GPU,
 *   from any thread or stream, race and give wrong results.  Order them.
 * Arguments are those of zero_init_partition and zero_step (stages 1/2,
 * one state slot, updated in place), plus:
 *   loss_scale, steps_applied  host values of the loss scale and of t
 *           before this step.  The caller keeps them between calls: it
 *           passes what the previous call's result reported, so it reads
 *           that result back (after synchronising the stream) first.
 *   result  pointer the GPU can write (device, managed or pinned host
 *           memory; pageable host memory is refused), 8-byte aligned,
 *           receiving the step's
 *           zero_result_t, stream-ordered: overflow, applied, norm, clip
 *           factor, the loss scale after this step (halved on overflow,
 *           floor 1.0), t after this step, and steps_skipped = 1 if this
 *           call skipped its update (0 otherwise)
 *   hyper->mode must be ZERO_MODE_AUTO or ZERO_MODE_TWO_PASS_WS.
 * Errors: EINVAL (read zero_last_error(NULL)), ECUDA.
 */
#define ZERO_NOALLOC_MAX_PSI_PAD (1ull << 22)

/*
 * zero_noalloc_scratch_bytes -- bytes of the static device array that
 * zero_step_noalloc uses, per GPU that loads the library:
 * 4 * ZERO_NOALLOC_MAX_PSI_PAD + 324,960.  A host query: no CUDA call, no
 * GPU needed, no error.
 */
ZERO_API uint64_t zero_noalloc_scratch_bytes(void);

ZERO_API int zero_step_noalloc(uint64_t psi, int n_ranks, int stage, int dtype, int align,
                      const void* const* grads, void* const* params,
                      float* master, float* m, float* v, const zero_hyper_t* hyper,
                      float loss_scale, int64_t steps_applied, zero_result_t* result,
                      void* stream);

/*
 * Orthogonalised momentum (the Muon optimiser) for the matrices of a
 * partitioned model.  None of the ZeRO pages has a counterpart: the step
 * keeps their structure (the ranks' gradients averaged into fp32 state, the
 * new values rounded into every rank's replica) with another update rule.
 * A step over matrices that lie back to back in flat buffers of `count`
 * elements is three calls on one stream:
 *   1. zero_muon_momentum   gradients of all ranks -> momentum, update
 *   2. zero_muon_orthogonalize  once for each shape among the matrices
 *   3. zero_muon_apply      orthogonalised update -> master, all replicas
 * They take no handle, allocate nothing, can be captured into a CUDA graph
 * (after one call of each outside a capture, which loads the kernels) and
 * keep what a step carries to the next in a device struct of the caller's.
 * Errors: read zero_last_error(NULL).
 */
typedef struct {
    float lr, momentum, weight_decay;
    int32_t nesterov;      /* 1: update = g + momentum * m', 0: m' */
} zero_muon_hyper_t;

/* DEVICE memory of the caller's, 8-byte aligned; set by zero_muon_set_state.
 * `pending` holds the reasons to skip the step that is under way: */
#define ZERO_MUON_NONFINITE 1   /* zero_muon_momentum saw a non-finite averaged gradient */
#define ZERO_MUON_GAVE_UP 2     /* a bounded wait inside zero_muon_orthogonalize gave up */
typedef struct {
    float loss_scale;      /* halved (floor 1.0) after a step whose gradients overflowed */
    int32_t slot;          /* live slot (0/1) of the momentum */
    int32_t pending;       /* ZERO_MUON_* bits */
    int32_t overflow;      /* last finished step was skipped */
    int32_t applied;       /* last finished step updated the state */
    uint32_t ticket;       /* 0 between calls */
    int64_t steps_applied, steps_skipped;
    int32_t aborted;       /* last finished step was skipped for ZERO_MUON_GAVE_UP */
    int32_t reserved0;
    int64_t reserved[2];
} zero_muon_state_t;

/* Set the state: before the first step, or to resume.  Stream-ordered.  The
 * loss scale must be finite and > 0.  Errors: EINVAL, ECUDA. */
ZERO_API int zero_muon_set_state(zero_muon_state_t* state, float loss_scale, int64_t steps_applied, int32_t slot,
                                 void* stream);

/* Copy the state to the host struct *out.  Synchronises the stream. */
ZERO_API int zero_muon_get_state(const zero_muon_state_t* state, void* stream, zero_muon_state_t* out);

/*
 * zero_muon_momentum -- average, unscale, momentum, update:
 *   g = (sum over ranks, in rank order from +0, of f32(g_r)) / (N * loss_scale)
 *   m' = momentum * m + g;   update = nesterov ? g + momentum * m' : m'
 * each fp32 operation rounded once, the update rounded to bf16 for both
 * gradient types (an unscaled gradient can lie below fp16's range).
 *   dtype     zero_dtype_t of the gradients
 *   grads     host array of n_ranks device pointers, count elements each
 *   momentum  fp32, two slots of ceil(count/8)*8 floats: read from the live
 *             slot, written to the other
 *   update    count bf16 values
 * A non-finite averaged gradient is noted in the state; the step is then
 * skipped by zero_muon_apply, with the momentum as it was.
 * Pointers 16-byte aligned.  count 0 is an empty call.  Errors: EINVAL, ECUDA.
 */
ZERO_API int zero_muon_momentum(int dtype, int n_ranks, uint64_t count, const void* const* grads, float* momentum,
                                void* update, const zero_muon_hyper_t* hyper, zero_muon_state_t* state, void* stream);

/*
 * zero_muon_apply -- master = (1 - lr * weight_decay) * master - lr * ortho,
 * every replica = the 16-bit rounding of it; then the step is finished in
 * the state (the momentum's new slot becomes live).  When `pending` holds a
 * reason to skip it, master and replicas keep their values and the
 * momentum's live slot stays; the loss scale halves for a non-finite
 * gradient and is kept for a wait that gave up, which sets `aborted`.
 *   dtype   zero_dtype_t of the replicas
 *   ortho   count bf16 values;  master: count floats
 *   params  host array of n_ranks device pointers, count elements each
 * Pointers 16-byte aligned.  count 0 only finishes the step.  Errors: EINVAL, ECUDA.
 */
ZERO_API int zero_muon_apply(int dtype, int n_ranks, uint64_t count, const void* ortho, float* master,
                             void* const* params, const zero_muon_hyper_t* hyper, zero_muon_state_t* state,
                             void* stream);

/*
 * zero_orthogonalize -- a batch of rows x cols matrices of 16-bit values by
 * `steps` Newton-Schulz steps, rounded to bf16:
 *   X = G / ||G||_F;   X <- (a I + b A + c A^2) X with A = X X^T;
 *   dst = scale * X
 * (A is formed over the shorter side; the result is the same.)  A zero
 * matrix gives zeros; one that holds an infinity or a NaN gives NaN.
 *   dtype   zero_dtype_t of src; dst is bf16 for both
 *   batch   0..ZERO_MAX_MATRICES; sides 0..ZERO_MAX_SIDE
 *   src, dst  host arrays of `batch` device pointers (2-byte aligned; rows
 *           that start on 16 bytes are read and written faster), with
 *           ld_src and ld_dst elements between rows.  dst[i] may be src[i]
 *           when the leading dimensions agree; matrices may not overlap
 *           otherwise.
 *   coeffs  host array of 3 * steps floats, {a, b, c} of each step, or NULL
 *           for {3.4445, -4.7750, 2.0315} throughout
 *   steps   1..ZERO_MAX_NS_STEPS
 *   workspace  device memory, 256-byte aligned, at least
 *           zero_orthogonalize_workspace_bytes(batch, rows, cols) bytes; its
 *           contents need not be kept between calls
 * Intermediate matrices are held in fp16 with fixed scales, products
 * accumulate in fp32.  The coefficients must keep the singular values of
 * every X below 3 and those of a I + b A + c A^2 (and of the first two
 * steps' product of it) below 500, or fp16 overflows and the result is not
 * finite (the calls do not check that).  Against 64 bits the result is off
 * by about 2e-3 of its 2-norm, most of it the rounding to bf16 (1.7e-3); by
 * up to 3.3e-3 where the shorter side is 16 to 48, and below 16 by 2e-3 to
 * 5e-3 in the mean and up to 2e-2 for single matrices.
 * For a shorter side above 128 (or a longer one above 8192) the products run
 * as one cooperative launch that takes the whole GPU.
 * Errors: EINVAL, ECUDA; see zero_matrix_status for a wait that gave up.
 */
#define ZERO_MAX_MATRICES 128
#define ZERO_MAX_SIDE (1ull << 18)
#define ZERO_MAX_NS_STEPS 32
ZERO_API int zero_orthogonalize(int dtype, int batch, uint64_t rows, uint64_t cols, const void* const* src,
                                uint64_t ld_src, void* const* dst, uint64_t ld_dst, int steps, const float* coeffs,
                                float scale, void* workspace, uint64_t workspace_bytes, void* stream);

/* zero_orthogonalize for the matrices of a step: a wait inside its kernels
 * that gives up leaves an incomplete result, which is noted in the step's
 * state (ZERO_MUON_GAVE_UP), so that zero_muon_apply does not apply it.
 * Errors: EINVAL, ECUDA. */
ZERO_API int zero_muon_orthogonalize(int dtype, int batch, uint64_t rows, uint64_t cols, const void* const* src,
                                     uint64_t ld_src, void* const* dst, uint64_t ld_dst, int steps,
                                     const float* coeffs, float scale, void* workspace, uint64_t workspace_bytes,
                                     zero_muon_state_t* state, void* stream);

/* Bytes of zero_orthogonalize's workspace (a host query); 0 for sizes that it refuses or that are empty. */
ZERO_API uint64_t zero_orthogonalize_workspace_bytes(int batch, uint64_t rows, uint64_t cols);

/*
 * Microscaled 4-bit floats (the OCP MX format with e2m1 elements): a form of
 * a quarter of 16 bits whose codes the tensor cores multiply as they are, next
 * to the zero-point formats of zero_quantize_blocks, which must be dequantized
 * first.  These calls quantize, read back and multiply; none moves codes
 * between ranks, as zero_gather_bucket_q8 does for INT8.
 * A block is ZERO_MX_BLOCK consecutive values of a row.  Its scale is
 * 2^(floor(log2(largest magnitude)) - 2), not below 2^-127, one byte with a
 * bias of 127; a value's code is x / scale rounded to the nearest of +-{0,
 * 0.5, 1, 1.5, 2, 3, 4, 6}, ties to the even code, larger ones to 6.  A block
 * with an infinity or a NaN has the scale byte 255 and stands for NaN.
 * Layout of a rows x cols matrix:
 *   codes   rows of ceil(cols/32)*16 bytes, two codes a byte, the even one
 *           low, zeros after cols
 *   scales  tiles of 128 rows x 4 blocks, 512 bytes each, row-major over
 *           the matrix; byte 16 (r mod 32) + 4 (r div 32) + b of a tile;
 *           0 where the matrix has no row or block
 * Both 16-byte aligned.  16-bit matrices are row-major with `ld` elements
 * between rows, 2-byte aligned (faster when rows start on 16 bytes).
 * Errors of these calls: EINVAL, ECUDA (zero_last_error(NULL)).
 */
#define ZERO_MX_BLOCK 32
ZERO_API uint64_t zero_mx4_codes_bytes(uint64_t rows, uint64_t cols);
ZERO_API uint64_t zero_mx4_scales_bytes(uint64_t rows, uint64_t cols);

/* Quantize src16 (rows x cols) along its rows, or with transpose != 0 along
 * its columns: then codes and scales are those of the cols x rows transpose,
 * as the products of a backward pass take them. */
ZERO_API int zero_mx4_quantize(int dtype, uint64_t rows, uint64_t cols, const void* src16, uint64_t ld, int transpose,
                               void* codes, void* scales, void* stream);

/* The values of a rows x cols matrix of codes, rounded to 16 bits. */
ZERO_API int zero_mx4_dequantize(int dtype, uint64_t rows, uint64_t cols, const void* codes, const void* scales,
                                 void* out16, uint64_t ld, void* stream);

/* out16[m][n] = sum over k of A[m][k] * B[n][k], both quantized along k, fp32
 * accumulation, rounded to 16 bits.  Y = X W^T of a linear layer whose weight
 * is W [n][k]; its backward pass is the same call on transposed operands
 * (dX: dY and W along their shared outer dimension; dW: dY and X along the
 * tokens).  k = 0 gives zeros.  See zero_matrix_status. */
ZERO_API int zero_mx4_matmul(int dtype, uint64_t m, uint64_t n, uint64_t k, const void* a_codes, const void* a_scales,
                             const void* b_codes, const void* b_scales, void* out16, uint64_t ld, void* stream);

/*
 * Microscaled 8-bit floats: the same format with e4m3 elements, for linear
 * layers that 4 bits are too coarse for.  A block's scale is
 * 2^(floor(log2(largest magnitude)) - 8), not below 2^-127; a value's code is
 * x / scale rounded to the nearest e4m3 value (3 bits after the leading one,
 * down to 2^-9), ties to the even code, those above 448 to 448.  Blocks with
 * an infinity or a NaN, the scales' layout, alignment, transposition and
 * products are as for 4 bits; codes are one a byte, rows of ceil(cols/32)*32
 * bytes with zeros after cols.  Both operands of a product have 8 bits.
 */
ZERO_API uint64_t zero_mx8_codes_bytes(uint64_t rows, uint64_t cols);
ZERO_API uint64_t zero_mx8_scales_bytes(uint64_t rows, uint64_t cols);
ZERO_API int zero_mx8_quantize(int dtype, uint64_t rows, uint64_t cols, const void* src16, uint64_t ld, int transpose,
                               void* codes, void* scales, void* stream);
ZERO_API int zero_mx8_dequantize(int dtype, uint64_t rows, uint64_t cols, const void* codes, const void* scales,
                                 void* out16, uint64_t ld, void* stream);
ZERO_API int zero_mx8_matmul(int dtype, uint64_t m, uint64_t n, uint64_t k, const void* a_codes, const void* a_scales,
                             const void* b_codes, const void* b_scales, void* out16, uint64_t ld, void* stream);

/* Whether a bounded wait inside a kernel of zero_orthogonalize (or
 * zero_muon_orthogonalize), zero_mx4_matmul or zero_mx8_matmul has given up on this device
 * since the last call: ZERO_OK or ZERO_ETIMEOUT (that kernel's output is
 * incomplete).  Synchronises the stream.  The answer is the device's, for
 * all streams and callers together, and the first to ask gets it. */
ZERO_API int zero_matrix_status(void* stream);

/*
 * zero_debug_hold_matrix -- test hook for the failure path of the matrix
 * kernels.  In the next zero_orthogonalize, zero_muon_orthogonalize,
 * zero_mx4_matmul or zero_mx8_matmul of the process that launches a kernel with bounded waits
 * (one-shot), the barrier for stage `stage` of block 0's ring expects an
 * arrival that never comes (in the orthogonalisation of short sides every
 * block's barrier for its products, whatever the stage), so that the waits for it
 * run out (about 2 s).  No access leaves its buffers and every wait ends.
 * The call's output is incomplete, and zero_matrix_status returns
 * ZERO_ETIMEOUT once.  stage < 0 clears a pending hold; one that block 0
 * does not use has no effect.  Returns ZERO_OK.
 */
ZERO_API int zero_debug_hold_matrix(int64_t stage);

/*
 * The residual stream of a training step: what lies between its linear
 * layers.  Like the matrix calls these take no handle, allocate nothing and
 * can be captured into a CUDA graph (after one call of each outside a
 * capture).  Matrices are row-major with `ld` elements between rows, 2-byte
 * aligned; rows may not share memory.  Calls are faster, up to twice, when the
 * rows of all their matrices start on 16 bytes and are whole eights, and
 * weight16 starts on 16 bytes too.
 * Results are rounded once to 16 bits and repeat bit for bit.  An empty
 * matrix is an empty call.  A workspace's contents need not be kept between
 * calls; calls that share one (replays of captured ones too) must run in
 * order.  Errors: EINVAL, ECUDA (zero_last_error(NULL)).
 */

/*
 * Dropout by a counter-based generator: the numbers are a function of seed,
 * stream and place, so no mask is stored and the backward pass makes the same
 * call.  Each element gets 16 bits of Philox4x32-10 (Salmon et al., "Parallel
 * random numbers: as easy as 1, 2, 3", SC 2011):
 *   key      seed, low word first
 *   counter  its low 64 bits row * ceil(cols / 8) + floor(col / 8), its high
 *            64 bits the stream, offset + (step ? *step : 0)
 *   bits     of column c: word (c mod 8) / 2, its low half for an even c
 * With k = p * 65536 rounded to the nearest whole number (at most 65535), an
 * element is 0 where its bits are below k, whatever it was, and else its
 * value times 65536 / (65536 - k).  Give every layer and step a stream of its
 * own.
 */
typedef struct {
    double p;                /* share to drop, in [0, 1) */
    uint64_t seed, offset;
    const uint64_t* step;    /* DEVICE memory, 8-byte aligned, or NULL: read when the kernel runs, so that
                                replays of a captured graph can be given other numbers */
} zero_dropout_t;

/* out16 = dropout(src16), rows x cols; dropout NULL copies.  out16 may be
 * src16 when the leading dimensions agree; they may not overlap otherwise.
 * rows <= 2^30; cols <= 2^34, or 2^40 values in all without gaps, aligned and
 * in whole eights. */
ZERO_API int zero_dropout(int dtype, uint64_t rows, uint64_t cols, const void* src16, uint64_t ld_src, void* out16,
                          uint64_t ld_out, const zero_dropout_t* dropout, void* stream);

/*
 * zero_rms_norm -- the stream with a branch added to it, and its
 * root-mean-square norm:
 *   h = round16(residual + dropout(x))
 *   y = h / sqrt(mean over the row of h^2 + eps) * weight
 *   residual16  or NULL (0);  dropout: or NULL (none)
 *   weight16    cols values
 *   h16         h, or NULL
 *   out16       y in 16 bits, or NULL
 *   bits        4 or 8: y in that microscaled format, into codes and scales
 *               (one rounding, from fp32; zero_mx4_matmul and zero_mx8_matmul
 *               read them), or 0
 * Something must be written.  The statistics are those of h as it is stored,
 * in fp32, of scaled values where their squares would leave it (with eps = 0 a
 * row below 2^-127 gives infinities, one of zeros NaN).  h16 may be
 * x16 or residual16, and out16 x16 or residual16 (not both the same one),
 * where the leading dimensions agree; nothing may overlap otherwise.
 * cols <= ZERO_MAX_NORM_COLS, rows <= 2^30.
 */
#define ZERO_MAX_NORM_COLS 16384
ZERO_API int zero_rms_norm(int dtype, uint64_t rows, uint64_t cols, const void* x16, uint64_t ld_x, const void* residual16,
                           uint64_t ld_residual, const void* weight16, float eps, const zero_dropout_t* dropout, void* h16,
                           uint64_t ld_h, void* out16, uint64_t ld_out, int bits, void* codes, void* scales, void* stream);

/*
 * zero_rms_norm_backward -- with g = dy * weight and r = 1 / sqrt(mean(h^2) + eps):
 *   dh = r * (g - h * r^2 * mean(g * h)) + dh_in      the residual's gradient
 *   dx = dropout(dh)                                  the branch's
 *   dweight = sum over the rows of dy * h * r
 *   dy16        gradient of y;  h16: the forward call's h
 *   dh_in16     gradient of h from elsewhere (the stream goes on past the norm), or NULL (0)
 *   dx16        or NULL;  dweight16: cols values, or NULL
 *   dropout     the forward call's, or NULL
 *   workspace   for dweight16 (else NULL): 16-byte aligned, at least
 *               zero_rms_norm_backward_workspace_bytes(rows, cols) bytes
 * Any gradient of y through its 4 or 8 bits is that of the 16-bit y.  dh16 and
 * dx16 may each be dy16 or dh_in16 (not both the same one) where the leading
 * dimensions agree; nothing may overlap otherwise.  rows = 0 gives a dweight
 * of zeros.
 */
ZERO_API int zero_rms_norm_backward(int dtype, uint64_t rows, uint64_t cols, const void* dy16, uint64_t ld_dy, const void* h16,
                                    uint64_t ld_h, const void* weight16, float eps, const void* dh_in16, uint64_t ld_in,
                                    void* dh16, uint64_t ld_dh, const zero_dropout_t* dropout, void* dx16, uint64_t ld_dx,
                                    void* dweight16, void* workspace, uint64_t workspace_bytes, void* stream);

/* Bytes of that workspace (a host query); 0 for sizes that the call refuses or that are empty. */
ZERO_API uint64_t zero_rms_norm_backward_workspace_bytes(uint64_t rows, uint64_t cols);

/*
 * zero_embedding -- out16[t] = scale * table16[ids[t]], tokens x dim from a
 * vocab x dim table.  ids: device array of id_bytes (4 or 8) each, signed; one
 * outside [0, vocab) is padding and gives a row of zeros.
 * vocab 1..2^31, dim <= 2^20, tokens <= 2^31.
 */
ZERO_API int zero_embedding(int dtype, uint64_t vocab, uint64_t dim, const void* table16, uint64_t ld_table, uint64_t tokens,
                            const void* ids, int id_bytes, float scale, void* out16, uint64_t ld_out, void* stream);

/*
 * zero_embedding_backward -- dtable16[v] = scale * (sum of dout16[t] over the
 * tokens t with ids[t] = v), every row of the table (0 where no token names
 * it); with accumulate != 0 what the rows held is added before the rounding
 * (rows that no token names keep their values), as a table that is also the
 * output layer's weight needs.  Sums are fp32, in an order that the ids and
 * the sizes fix: up to 512 tokens, those of every eighth token, then these
 * eight sums; beyond, within pieces of 8 places of a stable sort by id, then
 * the pieces' sums (of more than 9 pieces every eighth one's, then these).
 * Padding adds nothing.  Nothing may overlap.
 *   workspace   256-byte aligned, at least
 *               zero_embedding_backward_workspace_bytes(vocab, dim, tokens) bytes
 * tokens = 0 gives zeros.
 */
ZERO_API int zero_embedding_backward(int dtype, uint64_t vocab, uint64_t dim, const void* dout16, uint64_t ld_dout,
                                     uint64_t tokens, const void* ids, int id_bytes, float scale, int accumulate,
                                     void* dtable16, uint64_t ld_dtable, void* workspace, uint64_t workspace_bytes,
                                     void* stream);

/* Bytes of that workspace (a host query); 0 for sizes that the call refuses or that are empty. */
ZERO_API uint64_t zero_embedding_backward_workspace_bytes(uint64_t vocab, uint64_t dim, uint64_t tokens);

/* Last error message of this handle (or of the last failed init when h is
 * NULL).  The string is owned by the library and valid until the next call. */
ZERO_API const char* zero_last_error(zero_handle_t h);

/* Free the handle and its workspace.  Synchronises the device first.  NULL is a no-op. */
ZERO_API void zero_destroy(zero_handle_t h);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_GB300_H */
