/*
 * bf16opt.h -- C ABI of the BF16 mixed-precision optimizer step for one GPU.
 *
 * What the library computes, per optimizer step over one rank's parameter
 * shard (the BF16Optimizer of BLOOM-176B training):
 *   1. the bf16 gradients of the GAS micro-batches are summed into an FP32
 *      accumulator, in micro-batch order, stored as FP32 after every add
 *      ("BLOOM 176B 训练技术概览", section "BF16 优化器": all accumulation in
 *      FP32, gradients accumulated in FP32 across pipeline micro-batches);
 *   2. the global L2 norm of the accumulated gradient is reduced
 *      deterministically and the gradient is clipped to max_grad_norm
 *      ("企业官网建设流程全解析" (cf-1.com), section 4.3: global-norm threshold 1.0;
 *      "单机多卡实战：Megatron-DeepSpeed训练类BLOOM模型全流程解析", section 3: clip_grad 1.0);
 *   3. AdamW with decoupled, lr-scaled weight decay and bias correction
 *      updates the FP32 master weights and the FP32 first/second moments
 *      ("企业官网建设流程全解析", section 1: FP32 master, momentum and variance;
 *      section 3.3: AdamW lr 6e-5, weight_decay 0.01) and the bf16 working
 *      parameters are written as the round-to-nearest-even bf16 of the FP32
 *      master, all in one pass.
 *
 * Conventions.
 *   - Every buffer is caller-owned device memory (e.g. from PyTorch) that must
 *     outlive the handle; buffers must not overlap.  The library owns only
 *     its scratch (segment/chunk tables, norm partials, norm scalars, the
 *     step counter and the per-step scalars).
 *   - FP32 buffers must be 4-byte aligned and bf16 buffers 2-byte aligned
 *     (BF16OPT_ERR_ALIGNMENT otherwise).  Any offset modulo 16 bytes works;
 *     full speed needs every buffer of a tensor to share the same element
 *     offset modulo 16 bytes, and the last few percent the same offset
 *     modulo 128 bytes (any such offset runs as fast as an aligned one).
 *   - Elements are counted in uint64_t; a tensor or shard may exceed 2^32.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  All device work is enqueued on it; no call synchronises
 *     except bf16opt_grad_norm with a non-NULL host_norm.
 *   - Every call returns 0 on success, a positive warning, or a negative
 *     error code; no C++ exception crosses the ABI.  On an error nothing is
 *     enqueued and the handle's sequence state is unchanged.
 *     bf16opt_last_error() gives a one-line message.
 *   - A handle is bound to the device that was current at bf16opt_create and
 *     is not thread-safe: use one handle from one host thread at a time.
 *     The library keeps a registry of live handles: a pointer that
 *     bf16opt_create did not return, or a handle already destroyed, is
 *     rejected with BF16OPT_ERR_INVALID_ARG by every call (bf16opt_destroy
 *     included) and never dereferenced.  bf16opt_destroy frees all the
 *     handle's memory but a small host record, so no later handle ever
 *     receives a destroyed handle's address.
 *   - Results are deterministic and do not depend on the launch grid (the
 *     environment variable BF16OPT_MAX_GRID, read at create, caps the CTAs
 *     per launch; it exists to test exactly that).
 *
 * Sequence per optimizer step (checked on the host; BF16OPT_ERR_SEQUENCE):
 *   accumulate(FIRST) ... accumulate(LAST) -> grad_norm -> step
 *   FIRST marks the first micro-batch (the accumulator is overwritten, not
 *   added to); LAST marks the last one (the norm's partial sums are fused
 *   into that pass).  FIRST|LAST is a single micro-batch.  grad_norm (or
 *   grad_norm_local) needs the LAST micro-batch: after FIRST without LAST it
 *   returns BF16OPT_ERR_SEQUENCE.  Any micro-batch may carry BF16OPT_DEFER (see
 *   there); LAST|DEFER is the plain "fuse the last micro-batch into the step"
 *   case.
 */
#ifndef BF16OPT_H
#define BF16OPT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------- */
#define BF16OPT_OK 0
#define BF16OPT_WARN_NONFINITE 1       /* grad_norm: the norm is Inf or NaN */
#define BF16OPT_ERR_INVALID_ARG (-1)   /* NULL handle/pointer, bad size, bad hyper-parameter, overlap */
#define BF16OPT_ERR_ALIGNMENT (-2)     /* FP32 pointer not 4-B aligned or bf16 pointer not 2-B aligned */
#define BF16OPT_ERR_SEQUENCE (-3)      /* call out of the accumulate -> grad_norm -> step order */
#define BF16OPT_ERR_OOM (-4)           /* the library's scratch could not be allocated */
#define BF16OPT_ERR_CUDA (-5)          /* a CUDA runtime call or kernel launch failed */
#define BF16OPT_ERR_UNSUPPORTED (-6)   /* e.g. no usable CUDA device */

/* ---- ABI version -------------------------------------------------------
 * Raised whenever a declaration, a constant or a struct layout of this header
 * changes.  bf16opt_abi_version() returns the value the library was built
 * with; code compiled against a header with another value must not use it.
 * No CUDA call; never fails. */
#define BF16OPT_ABI_VERSION 4
int bf16opt_abi_version(void);

/* ---- modes and flags --------------------------------------------------- */
#define BF16OPT_FLAT 0   /* one contiguous shard: five flat buffers + group ranges */
#define BF16OPT_LIST 1   /* ragged list: five buffers per tensor (separate allocations) */

#define BF16OPT_FIRST 1u /* first micro-batch of the step: acc = fp32(g) */
#define BF16OPT_LAST 2u  /* last micro-batch: fuse the norm's partial sums into this pass */
#define BF16OPT_DEFER 4u /* keep this micro-batch's gradient instead of folding it into the
                            FP32 accumulator now: it is folded (in micro-batch order) by
                            the next pass that reads gradients -- the next accumulate
                            without DEFER, or, if none follows before LAST, the norm and
                            the step kernels, so the accumulator is never stored for it.
                            The buffer must stay valid and unchanged until that pass has
                            run on the stream (until bf16opt_step for deferred micro-
                            batches of the last run).  At most BF16OPT_MAX_DEFERRED may be
                            pending.  Same FP32 adds in the same order: bit-identical to
                            not deferring; it trades 2 bytes/element of gradient memory
                            per pending micro-batch for 8 bytes/element of HBM traffic */

#define BF16OPT_MAX_DEFERRED 8

#define BF16OPT_MAX_GROUPS 16

/* ---- descriptors (host memory; copied by bf16opt_create) ---------------- */

/* FLAT mode: elements [begin, end) of the shard belong to parameter group `group`. */
typedef struct {
    uint64_t begin, end;
    uint32_t group;
    uint32_t reserved;     /* must be 0 */
} bf16opt_range_t;

/* LIST mode: one tensor; every pointer is device memory of `numel` elements. */
typedef struct {
    float *master;         /* FP32 master weights */
    float *exp_avg;        /* FP32 first moment m */
    float *exp_avg_sq;     /* FP32 second moment v */
    float *grad_accum;     /* FP32 gradient accumulator */
    uint16_t *param_bf16;  /* bf16 working parameters (bit patterns) */
    uint64_t numel;
    uint32_t group;
    uint32_t reserved;     /* must be 0 */
} bf16opt_tensor_t;

/* AdamW hyper-parameters of one parameter group. */
typedef struct {
    float lr;              /* >= 0 */
    float beta1, beta2;    /* in [0, 1) */
    float eps;             /* > 0 */
    float weight_decay;    /* >= 0; decoupled: p -= lr * weight_decay * p */
} bf16opt_group_t;

typedef struct {
    int32_t mode;                    /* BF16OPT_FLAT or BF16OPT_LIST */
    uint32_t n_groups;               /* 1 .. BF16OPT_MAX_GROUPS */
    const bf16opt_group_t *groups;   /* n_groups entries */
    /* FLAT */
    uint64_t n;                      /* shard elements (0 allowed) */
    float *master, *exp_avg, *exp_avg_sq, *grad_accum;
    uint16_t *param_bf16;
    const bf16opt_range_t *ranges;   /* must tile [0, n) in order; NULL/0 = one range, group 0 */
    uint32_t n_ranges;
    /* LIST */
    uint32_t n_tensors;
    const bf16opt_tensor_t *tensors;
    /* clipping */
    float max_grad_norm;             /* global L2 clip threshold; <= 0 disables clipping */
    float grad_scale;                /* multiplies the accumulated gradient before norm and
                                        update (rounded to FP32); 1 = none; finite, != 0 */
} bf16opt_desc_t;

typedef struct bf16opt bf16opt_t;    /* opaque handle */

/* ---- entry points ------------------------------------------------------- */

/* One handle per rank's parameter shard ("BLOOM 176B 训练技术概览", section
 * 并行细节 / ZeRO: each GPU holds only its part of the parameters, gradients
 * and optimizer states).  Validates `d` before any CUDA call, copies its host
 * arrays (the caller may free them on return), builds the segment and chunk
 * tables on the device and allocates the library's scratch; the device
 * buffers stay the caller's.  *out receives the handle (NULL on error).  The
 * step counter starts at 0.  Errors: INVALID_ARG (NULL d or out, bad mode,
 * 0 or more than BF16OPT_MAX_GROUPS groups, a hyper-parameter out of range,
 * non-finite max_grad_norm, zero or non-finite grad_scale, NULL buffers,
 * ranges that do not tile [0, n) in order, overlapping buffers, more than
 * 2^32 - 1 chunks), ALIGNMENT, UNSUPPORTED (no CUDA device), OOM, CUDA;
 * bf16opt_last_error(NULL) has the message. */
int bf16opt_create(const bf16opt_desc_t *d, bf16opt_t **out);

/* ZeRO-Offload variant ("企业官网建设流程全解析" (cf-1.com), section 3.3: the
 * DeepSpeed configuration with offload_optimizer on the CPU; "单机多卡实战：
 * Megatron-DeepSpeed训练类BLOOM模型全流程解析", section 6: offloading optimizer
 * state to host memory to fit larger models).  Explicitly selected, never a
 * fallback: a FLAT handle whose FP32 master, exp_avg and exp_avg_sq are HOST
 * memory (12 bytes per element off the device), while grad_accum and
 * param_bf16 are memory of the current device.  accumulate, grad_norm (and the
 * multi-rank calls), get/set_step, the LR schedule and skipping work as for
 * bf16opt_create.  bf16opt_step then: completes the accumulator if
 * micro-batches are still deferred; computes the step's scalars, advances the
 * step counter and takes the skip decision on the device (the same kernel as
 * the device step); copies the accumulator to the host in blocks of 2^24
 * elements, updates master and moments with the same FP32 operations as the
 * device step on n_threads host threads (<= 0: one per core) while the next
 * block is copied, and enqueues the copy of each block's bf16 parameters back
 * to param_bf16 on `stream`.  It returns when the host arrays hold the new
 * state; the bf16 parameters are on the device when `stream` reaches those
 * copies.  Results: the same bits as a device handle over the same values.
 * The library allocates 192 MiB of page-locked staging (less for a smaller
 * shard) and the threads.  Not during a stream capture.  Errors: as
 * bf16opt_create, and INVALID_ARG (not FLAT; master/moments not host memory;
 * grad_accum/param_bf16 not memory of the current device), OOM. */
int bf16opt_create_offload(const bf16opt_desc_t *d, int n_threads, bf16opt_t **out);

/* Adds one micro-batch of bf16 gradients into the FP32 accumulator
 * ("BLOOM 176B 训练技术概览", "BF16 优化器").
 *   FLAT: grad_flat = device bf16 buffer of n elements, grad_list = NULL.
 *   LIST: grad_flat = NULL, grad_list = HOST array of n_tensors device
 *         pointers (read during the call only).
 *   flags: BF16OPT_FIRST / BF16OPT_LAST / BF16OPT_DEFER (see above).
 * The gradient buffer is read on `stream`; it may be reused after the work
 * on `stream` is done, except under BF16OPT_DEFER (until the pass that folds
 * it).  Errors: SEQUENCE (no FIRST outside an accumulation), INVALID_ARG
 * (not a live handle, unknown flag, a NULL or wrong-mode gradient pointer, a
 * DEFER beyond BF16OPT_MAX_DEFERRED pending), ALIGNMENT (a gradient pointer
 * not 2-byte aligned), CUDA. */
int bf16opt_accumulate(bf16opt_t *h, const uint16_t *grad_flat, const uint16_t *const *grad_list,
                       unsigned flags, void *stream);

/* Finishes the deterministic global L2 norm of the accumulated gradient
 * (times grad_scale) and the clip coefficient c = max_grad_norm / norm if
 * norm > max_grad_norm, else 1 ("企业官网建设流程全解析", section 4.3).  Both stay
 * on the device for bf16opt_step.  host_norm == NULL: fully asynchronous.
 * host_norm != NULL: waits for `stream` and stores the norm (FP64); returns
 * BF16OPT_WARN_NONFINITE if it is Inf or NaN (the caller decides whether to
 * call bf16opt_step; the library skips nothing unless bf16opt_set_skip_nonfinite
 * asked it to).  Errors: SEQUENCE (no completed accumulation FIRST ... LAST
 * since the last step), INVALID_ARG (not a live handle), CUDA. */
int bf16opt_grad_norm(bf16opt_t *h, void *stream, double *host_norm);

/* Multi-rank use.  Under ZeRO every rank owns one partition of the parameters
 * and the clipping norm is global over all of them ("BLOOM 176B 训练技术概览",
 * section 并行细节 / ZeRO: each GPU holds only its part; "企业官网建设流程全解析",
 * section 4.3: the global norm).  The exchange is one FP64 scalar per rank;
 * moving it belongs to the caller's communication library, the arithmetic to
 * this one:
 *   1. bf16opt_grad_norm_local: in place of bf16opt_grad_norm, finishes this
 *      rank's sum of squares, waits for `stream` and stores it in *local_sumsq;
 *   2. the caller gathers every rank's value into an array in rank order
 *      (an all-gather);
 *   3. bf16opt_set_rank_sumsqs: sums that array in rank order (FP64, rank 0
 *      first: every rank gets the same bits, so every rank clips alike) and
 *      turns the sum into the norm and clip coefficient on the device
 *      (enqueued on `stream`); bf16opt_step follows.
 * Sequence: local needs a completed accumulation (as grad_norm); set_rank
 * and set_global need local.  A non-finite local or global sum is passed
 * through unchanged and reported as BF16OPT_WARN_NONFINITE (the caller decides
 * whether to step). */
int bf16opt_grad_norm_local(bf16opt_t *h, void *stream, double *local_sumsq);

/* per_rank: HOST array of the n_ranks gathered local sums, in rank order;
 * rank: this handle's rank, whose entry must equal, bit for bit, the value
 * bf16opt_grad_norm_local returned (a gather that put the values out of order
 * is refused).  global_norm: NULL, or receives sqrt of the rank-ordered sum
 * (no synchronisation).  Errors: INVALID_ARG (not a live handle, NULL
 * per_rank, n_ranks == 0, rank >= n_ranks, per_rank[rank] not this rank's
 * value), SEQUENCE (no grad_norm_local since the accumulation), CUDA. */
int bf16opt_set_rank_sumsqs(bf16opt_t *h, const double *per_rank, uint32_t n_ranks, uint32_t rank, void *stream,
                            double *global_norm);

/* The rank-ordered sum that bf16opt_set_rank_sumsqs uses:
 * *global_sumsq = ((per_rank[0] + per_rank[1]) + ...) + per_rank[n_ranks-1]
 * in FP64.  Host-only; needs no device or handle.  Errors: INVALID_ARG (NULL
 * pointer, n_ranks == 0). */
int bf16opt_sum_rank_sumsqs(const double *per_rank, uint32_t n_ranks, double *global_sumsq);

/* For callers that reduce the sums themselves: sets the norm and clip
 * coefficient from an already summed global_sumsq (enqueued on `stream`).
 * Every rank must pass the same bits.  Errors as bf16opt_set_rank_sumsqs. */
int bf16opt_set_global_sumsq(bf16opt_t *h, double global_sumsq, void *stream);

/* CUDA graphs.  The step counter, the hyper-parameters and the LR schedule
 * live on the device and bf16opt_step computes its scalars there, so the
 * sequence accumulate ... -> grad_norm (host_norm = NULL) -> step, captured
 * once on a stream, replays as later steps (same gradient buffers; lr_override
 * values are frozen into the capture).  Calls that synchronise (grad_norm with
 * host_norm, grad_norm_local, get/set_step, set_lr_schedule,
 * set_skip_nonfinite, debug_faults, create, create_offload, destroy, and step
 * on an offload handle) must stay outside a capture. */

/* One fused pass: clip, AdamW (t = t + 1, bias-corrected, decoupled
 * weight decay), FP32 master/moment update and bf16 parameter write
 * ("企业官网建设流程全解析", sections 1 and 3.3).
 * lr_override: NULL, or a HOST array of n_groups learning rates that
 * replaces the groups' lr for this step only (for an LR schedule; read during
 * the call only).  Errors: SEQUENCE (no grad_norm or set_global_sumsq since
 * the accumulation), INVALID_ARG (not a live handle, a negative or non-finite
 * lr_override entry), CUDA. */
int bf16opt_step(bf16opt_t *h, const float *lr_override, void *stream);

/* Learning-rate schedule of the training configuration ("单机多卡实战：
 * Megatron-DeepSpeed训练类BLOOM模型全流程解析", section 3: lr 6e-5, min_lr 1e-6,
 * lr_decay_style cosine, warmup_iters 500): linear warmup from 0 to the group's
 * lr over warmup_steps, then cosine decay to min_lr_ratio * lr at decay_steps,
 * then constant.  For the step number t >= 1 the factor on every group's lr is
 *   t <= warmup_steps:                f = t / warmup_steps
 *   warmup_steps < t <= decay_steps:  f = r + (1 - r) (1 + cos(pi (t - warmup_steps)
 *                                              / (decay_steps - warmup_steps))) / 2
 *   t > decay_steps:                  f = r                      (r = min_lr_ratio)
 * evaluated in FP64. */
typedef struct {
    int64_t warmup_steps;  /* >= 0 */
    int64_t decay_steps;   /* >= warmup_steps */
    float min_lr_ratio;    /* in [0, 1] */
    uint32_t reserved;     /* must be 0 */
} bf16opt_lr_schedule_t;

/* f(t) of the schedule above into *factor.  Host-only; needs no device or handle.
 * Errors: INVALID_ARG for NULL pointers, t < 1 or an invalid schedule. */
int bf16opt_lr_factor(const bf16opt_lr_schedule_t *s, int64_t t, double *factor);

/* Attaches a copy of schedule `s` to the handle (NULL detaches it).  Every later
 * bf16opt_step then uses lr = (lr_override[g] or the group's lr) * f(t) with t
 * the step number of that step (the step counter plus one, so a resumed run
 * that restored its counter with bf16opt_set_step continues the schedule).
 * Waits for all work on the handle's device first, so steps already enqueued
 * keep the old schedule; not during a stream capture.  Errors: INVALID_ARG
 * (not a live handle, an invalid schedule as for bf16opt_lr_factor), CUDA. */
int bf16opt_set_lr_schedule(bf16opt_t *h, const bf16opt_lr_schedule_t *s);

/* Opt-in guard for steps whose global norm is Inf or NaN (enable != 0): the
 * decision is taken on the device by bf16opt_step's first kernel, which then
 * leaves the step counter unchanged, and the fused kernel returns without
 * touching master, moments or bf16 parameters -- so it also holds inside a
 * captured CUDA graph, where the host cannot read the norm before the step.
 * Off by default: the method has no skip logic (bf16 does not overflow the
 * way fp16 does; "企业官网建设流程全解析", section 4.1) and grad_norm reports
 * BF16OPT_WARN_NONFINITE for the caller to act on.  Waits for all work on the
 * handle's device first, so steps already enqueued keep the old setting; not
 * during a stream capture.  Errors: INVALID_ARG (NULL handle), CUDA. */
int bf16opt_set_skip_nonfinite(bf16opt_t *h, int enable);

/* Frees the library's scratch (waits for the device); the caller's buffers
 * are untouched.  NULL is accepted.  A pointer that is not a live handle
 * (never created, or already destroyed) gives BF16OPT_ERR_INVALID_ARG. */
int bf16opt_destroy(bf16opt_t *h);

/* Step counter t (number of completed steps, kept on the device), for
 * checkpoint and resume: restore the caller's buffers and set_step(t) to
 * continue.  Both calls first wait for all work on the handle's device
 * (cudaDeviceSynchronize), so they are ordered after every step already
 * enqueued, on any stream (non-blocking ones included); not during a stream
 * capture.  Errors: INVALID_ARG (NULL, t < 0), CUDA. */
int bf16opt_get_step(const bf16opt_t *h, int64_t *t);
int bf16opt_set_step(bf16opt_t *h, int64_t t);

/* ---- allocation-free one-shot norm -----------------------------------------
 * No counterpart in the paper: a service entry point for callers that cannot
 * call cudaMalloc -- code inside another framework's launch path that is given
 * only a stream and a pre-planned workspace (plugins, custom-op launchers),
 * processes whose device memory is held by a caching allocator (a raw
 * cudaMalloc can then fail), and latency-sensitive loops that cannot take the
 * device synchronisation cudaMalloc/cudaFree imply.
 *
 * Computes, without a handle and without allocating anything, the global L2
 * norm of a flat FP32 gradient accumulator `grad_accum` of n elements (each
 * element times grad_scale, rounded to FP32), with the same deterministic
 * chunked reduction as bf16opt_grad_norm on a one-range FLAT shard over an
 * accumulator with the same offset modulo 128 bytes, and the
 * clip coefficient c = max_grad_norm / norm if norm > max_grad_norm (> 0),
 * else 1.  `out` is owned by the caller; the result is written there on
 * `stream` (nothing is synchronised).  `out` and `grad_accum` must be memory
 * the current device can use: its own device memory, managed memory, or
 * page-locked host memory (cudaMallocHost / cudaHostRegister, used through
 * its mapped device address); anything else (pageable host memory, another
 * device's memory) is refused with BF16OPT_ERR_INVALID_ARG before any work is
 * enqueued.
 *
 * Scratch: one FP64 partial per chunk of up to 32,768 elements, kept in a file-scope
 * device array of 65,536 entries (512 KiB) that every GPU loading this
 * library holds until the process exits; hence n is limited to
 * BF16OPT_STATIC_NORM_MAX_ELEMS (2^30) elements and larger n is rejected with
 * BF16OPT_ERR_INVALID_ARG before any work is enqueued.  Every call writes the
 * partials it later reads, so nothing has to start at zero.  All calls on a
 * device share that one array: calls whose work overlaps on the GPU (e.g. on
 * two streams without ordering between them) race and give wrong results.
 * The array's device address belongs to the context that loaded the library's
 * kernels: the first call on each device, and the first call after that
 * device's context was reset (cudaDeviceReset), looks it up
 * (cudaGetSymbolAddress) with the device current; make those calls before any
 * stream capture.  Errors: INVALID_ARG (NULL pointers, n too large,
 * non-finite or zero grad_scale, non-finite max_grad_norm, memory the device
 * cannot use), ALIGNMENT (grad_accum not 4-B aligned, out not 8-B aligned),
 * UNSUPPORTED (no device), CUDA (symbol lookup or launch failed);
 * bf16opt_last_error(NULL) has the message. */
#define BF16OPT_STATIC_NORM_MAX_ELEMS (((uint64_t)1) << 30)

typedef struct {
    double sumsq;      /* sum of squares of the (scaled) accumulated gradient */
    double norm;       /* sqrt(sumsq) */
    double clip_coef;  /* max_grad_norm / norm if norm > max_grad_norm, else 1 */
} bf16opt_norm_result_t;

int bf16opt_grad_norm_static(const float *grad_accum, uint64_t n, float grad_scale, float max_grad_norm,
                             bf16opt_norm_result_t *out, void *stream);

/* ---- data path of the step -------------------------------------------------
 * No counterpart in the paper.  Which kernel the handle's most recent
 * bf16opt_step ran (enqueued): NONE (no step yet, or the shard is empty),
 * VECTOR (per-thread 16-byte vector loads and stores), PIPELINE (bulk
 * asynchronous copies through shared memory; see below), HOST (an offload
 * handle: the host cores update the master and moments).  Errors: INVALID_ARG
 * (not a live handle, path NULL). */
#define BF16OPT_PATH_NONE 0
#define BF16OPT_PATH_VECTOR 1
#define BF16OPT_PATH_PIPELINE 2
#define BF16OPT_PATH_HOST 3
int bf16opt_step_path(const bf16opt_t *h, int *path);

/* ---- pipeline health ----------------------------------------------------
 * No counterpart in the paper: a health check of the copy pipeline.  On
 * shards of 2^25 elements and more whose buffers are aligned alike (per
 * segment: the FP32 streams at one element index modulo 4, the bf16 streams
 * at one modulo 8, agreeing modulo 4), bf16opt_step and the accumulate passes
 * after FIRST that store the accumulator move their traffic with bulk
 * asynchronous copies through a ring of shared-memory stages.  The
 * environment variable BF16OPT_PIPE=1 / 0, read when a handle is created,
 * forces this on / off.  Every wait on a stage is bounded (2 s; a stage
 * normally turns over in microseconds).  A wait that gives up is counted in
 * a device word and its CTA stops, leaving the rest of its units of that
 * pass not updated.  This call waits for the current device, stores that
 * device's count into *count (0 = every pass completed) and clears it.
 * Errors: INVALID_ARG (count NULL), UNSUPPORTED (no device), CUDA. */
int bf16opt_pipeline_timeouts(uint32_t *count);

/* ---- training operators ------------------------------------------------------
 * The memory-bound operators of a training step whose bf16 gradients the
 * accumulate passes take: a distillation loss at the head, the norms, gate and
 * residual scale around a block, a router's balance loss, policy and preference losses of
 * given tokens, a feed-forward block's activation with its inputs kept in 8 bits, and rotary
 * positions, each with its gradient.  No counterpart in the paper.
 *
 * They need no handle.  A call enqueues its kernels on `stream`, on the
 * current device, and neither allocates nor synchronises, so it can be captured
 * in a CUDA graph.  Every pointer is device memory unless stated otherwise, aligned to its
 * element; rows may start anywhere (a row stride counts elements and is at
 * least the row's length).  16-byte aligned rows run fastest.  An output may
 * not overlap an input or another output except where stated (what counts is the
 * span from the first row's start to the last row's end).  Descriptors are
 * read during the call.  Results are deterministic: the same inputs give the
 * same bits, whatever runs beside them.  Errors are reported as by the calls
 * without a handle: INVALID_ARG, ALIGNMENT, UNSUPPORTED (no CUDA device) or
 * CUDA, with the message in bf16opt_last_error(NULL); nothing is enqueued after
 * INVALID_ARG or ALIGNMENT.  A call over 0 rows does nothing (weight gradients
 * and losses of no rows are written as 0). */
#define BF16OPT_TYPE_BF16 0
#define BF16OPT_TYPE_F32 1
#define BF16OPT_INDEX_I32 0
#define BF16OPT_INDEX_I64 1

/* Distillation from a teacher's top logits.  z: the student's logits of a row;
 * (id_i, t_i), i < k: the teacher's kept entries; T: temperature.
 *   p_i = softmax over the row's entries of t / T, or, with teacher_lse,
 *         exp(t_i / T - teacher_lse[row]) (the teacher's own probabilities, whose
 *         sum P may be below 1); q = softmax(z / T); s = softmax(z);
 *   loss = w [ kl_weight T^2 (sum_i p_i (log p_i - log q[id_i]))
 *              + ce_weight (-log s[label]) ],           w = row_weight[row] or 1
 *   dz_j = w dloss [ kl_weight T (P q_j - sum_{i: id_i = j} p_i)
 *              + ce_weight (s_j - [j = label]) ].
 * An entry whose id is outside [0, vocab) or whose t is -inf does not exist; a
 * row without entries has no first term; a label outside [0, vocab) gives no
 * second term.  Entries may repeat an id.  A row whose w is 0 is not read: its
 * loss, log-sum-exps and gradient are 0.  Logits of -inf are masked
 * vocabulary: q = s = 0 there (a teacher's entry or label on one makes the loss
 * +inf; in a row with no other logit q = s = 0 everywhere).  NaN and +inf in
 * a row give NaN in that row alone. */
#define BF16OPT_DISTILL_MAX_K 1024

typedef struct {
    uint64_t rows;               /* tokens */
    uint32_t vocab;              /* 1 .. 2^30 */
    uint32_t k;                  /* teacher's entries per row, 0 .. BF16OPT_DISTILL_MAX_K */
    int32_t logits_type;         /* BF16OPT_TYPE_* of logits and dlogits */
    int32_t teacher_type;        /* BF16OPT_TYPE_* of teacher_logits */
    int32_t ids_type;            /* BF16OPT_INDEX_* of teacher_ids */
    int32_t labels_type;         /* BF16OPT_INDEX_* of labels */
    const void *logits;          /* [rows, vocab] */
    uint64_t logits_stride;
    const void *teacher_ids;     /* [rows, k] */
    uint64_t ids_stride;
    const void *teacher_logits;  /* [rows, k] */
    uint64_t teacher_stride;
    const float *teacher_lse;    /* NULL, or [rows]: log-sum-exp of the teacher's whole row at T */
    const void *labels;          /* NULL, or [rows] */
    const float *row_weight;     /* NULL, or [rows] */
    float temperature;           /* finite, > 0 */
    float kl_weight, ce_weight;  /* finite, >= 0; without labels there is no second term */
} bf16opt_distill_t;

/* loss: [rows] FP32.  lse: NULL, or [rows, 2] FP32: the log-sum-exp of z / T
 * and of z (the second repeats the first where ce_weight is 0 or labels is
 * NULL, and both are at T = 1 where kl_weight is 0), for bf16opt_distill_backward. */
int bf16opt_distill_forward(const bf16opt_distill_t *d, float *loss, float *lse, void *stream);

/* dlogits [rows, vocab], rounded once from FP32; it may be d->logits itself
 * with the same stride (the logits are then overwritten).  lse: as the forward
 * call with the same descriptor left it (a row for which one of them is 128 or
 * more in magnitude is read twice: one FP32 number does not hold the sum of a row
 * that lies far from 0).  dloss: NULL (1), or [rows] FP32: the gradient of the
 * row's loss. */
int bf16opt_distill_backward(const bf16opt_distill_t *d, const float *lse, const float *dloss, void *dlogits,
                             uint64_t dlogits_stride, void *stream);

/* Loss and gradient (for a gradient of dloss, or 1, of each row's loss) in one
 * pass: every logit is read once.  lse may be NULL. */
int bf16opt_distill_loss_grad(const bf16opt_distill_t *d, const float *dloss, float *loss, float *lse, void *dlogits,
                              uint64_t dlogits_stride, void *stream);

/* A block's output joined to the residual stream, with the norm behind the
 * block and the one before the next:
 *   u = N_post(y);  r = residual_scale x + branch_scale act(gate) u;  h = N_pre(r)
 * N is, for a row v of `hidden` elements,
 *   BF16OPT_NORM_NONE   v,
 *   BF16OPT_NORM_RMS    v / sqrt(mean(v^2) + eps) * weight + bias,
 *   BF16OPT_NORM_LAYER  (v - mean) / sqrt(var + eps) * weight + bias,
 * (a NULL weight is 1, a NULL bias 0); act is the identity or the sigmoid.  The gate
 * (NULL: 1) has gate_rows rows: rows / gate_rows consecutive rows share one, so
 * it is one learned vector (1), one for each sequence, or one for each token.
 * Statistics, products and sums are FP32; r and h are each rounded once (h is
 * computed from the unrounded r).  stats [rows, 4] FP32 keeps mean and
 * 1/sqrt(.. + eps) of r and of y (mean 0 for RMS, both 0 for NONE).
 *   backward: dr, dh (gradients of r by other readers and of h; either may be
 *   NULL: 0), r, y, stats as the forward call left them:
 *     g = dr + N_pre'(dh);  dx = residual_scale g;  du = branch_scale act(gate) g;
 *     dgate = branch_scale act'(gate) sum over the rows that share it of g u;
 *     dy = N_post'(du); the norms' weights' and biases' gradients over all rows.
 *   Row sums are FP32 in a fixed order.  NaN stays in its row, but for the
 *   weights' and shared gates' gradients. */
#define BF16OPT_NORM_NONE 0
#define BF16OPT_NORM_RMS 1
#define BF16OPT_NORM_LAYER 2
#define BF16OPT_GATE_IDENTITY 0
#define BF16OPT_GATE_SIGMOID 1
#define BF16OPT_NORM_MAX_HIDDEN 16384

typedef struct {
    uint64_t rows;
    uint32_t hidden;             /* 1 .. BF16OPT_NORM_MAX_HIDDEN */
    int32_t branch_type;         /* BF16OPT_TYPE_* of y, h, gate and their gradients */
    int32_t stream_type;         /* BF16OPT_TYPE_* of x, r and their gradients; F32 if branch_type is F32 */
    int32_t weight_type;         /* BF16OPT_TYPE_* of the norms' weights and biases and of their gradients */
    int32_t pre, post;           /* BF16OPT_NORM_* of N_pre and N_post */
    int32_t gate_act;            /* BF16OPT_GATE_* */
    uint32_t reserved;           /* must be 0 */
    uint64_t gate_rows;          /* 0 without a gate; divides rows */
    const void *gate;            /* NULL, or [gate_rows, hidden] */
    const void *pre_weight, *pre_bias, *post_weight, *post_bias;   /* each NULL or [hidden] */
    float residual_scale, branch_scale;   /* finite */
    float eps;                   /* finite, > 0 */
} bf16opt_norm_gate_t;

/* All rows are contiguous ([rows, hidden]).  h: NULL if pre is NONE.  stats may
 * be NULL (no backward).  r may be x (the stream updated in place), h may be y. */
int bf16opt_norm_gate_forward(const bf16opt_norm_gate_t *d, const void *x, const void *y, void *r, void *h,
                              float *stats, void *stream);

/* Bytes of scratch that the backward call of this descriptor needs (device
 * memory, 16-byte aligned, used on `stream` during the call only).  No CUDA
 * kernel; errors: INVALID_ARG, UNSUPPORTED. */
int bf16opt_norm_gate_workspace(const bf16opt_norm_gate_t *d, uint64_t *bytes);

/* The outputs of weights that d does not have are NULL; any other may be NULL
 * too, and is then not computed, except dx and dy. dx may be dr, dy may be dh. */
int bf16opt_norm_gate_backward(const bf16opt_norm_gate_t *d, const void *dr, const void *dh, const void *r,
                               const void *y, const float *stats, void *dx, void *dy, void *dgate, void *dpre_weight,
                               void *dpre_bias, void *dpost_weight, void *dpost_bias, void *workspace,
                               uint64_t workspace_bytes, void *stream);

/* A router's choice and its balance.  z: a token's logits over the experts,
 * p = softmax(z).  Chosen: the k largest logits, ties to the lowest expert,
 * in descending order; weights: their p, divided by their sum if renormalise.
 * The tokens form `groups` runs of tokens / groups (1: one batch; one for each
 * sequence: each sequence balanced for itself).  Over the n live tokens of a
 * group (mask NULL or nonzero), with counts_e tokens sent to expert e:
 *   f_e = counts_e experts / (k n),  P_e = mean p_e,
 *   loss = 1/groups sum over groups [ balance_weight sum_e f_e P_e
 *                                     + z_weight mean (log sum exp z)^2 ],
 * a group without live tokens adding 0.  Backward, with f constant, dloss the
 * gradient of the loss and dweights that of the weights:
 *   dz_j = dloss / (groups n) [ balance_weight p_j (f_j - sum_e f_e p_e)
 *          + 2 z_weight lse p_j ] + the gradient of the weights.
 * A masked token has ids -1, weights and gradient 0.  An expert whose logit
 * is -inf is never chosen (missing choices: id -1, weight 0, not counted); a token whose logits
 * all are is as if masked.  A NaN is chosen after every number but before -inf;
 * it makes the token's weights and gradient and the loss NaN (the other tokens'
 * gradients depend on it through the counts alone). */
#define BF16OPT_BALANCE_MAX_EXPERTS 1024
#define BF16OPT_BALANCE_MAX_K 32

typedef struct {
    uint64_t tokens;
    uint32_t experts;            /* 1 .. BF16OPT_BALANCE_MAX_EXPERTS */
    uint32_t k;                  /* 1 .. min(experts, BF16OPT_BALANCE_MAX_K) */
    uint64_t groups;             /* >= 1, divides tokens */
    int32_t logits_type;         /* BF16OPT_TYPE_* of logits and dlogits */
    int32_t renormalise;         /* 0 or 1 */
    const void *logits;          /* [tokens, experts] */
    uint64_t logits_stride;
    const uint8_t *mask;         /* NULL, or [tokens]: 0 = masked */
    float balance_weight, z_weight;   /* finite, >= 0 */
} bf16opt_balance_t;

/* ids [tokens, k] int32, weights [tokens, k] FP32, counts [groups, experts]
 * int32, loss [1] FP32, saved [tokens + groups] FP32 (each token's log-sum-exp,
 * then each group's n, for the backward call).  workspace: as for
 * bf16opt_norm_gate_workspace. */
int bf16opt_balance_workspace(const bf16opt_balance_t *d, uint64_t *bytes);
int bf16opt_balance_forward(const bf16opt_balance_t *d, int32_t *ids, float *weights, int32_t *counts, float *loss,
                            float *saved, void *workspace, uint64_t workspace_bytes, void *stream);

/* ids, counts, saved: as the forward call with the same descriptor left them.
 * dweights: NULL (0) or [tokens, k] FP32.  dloss: NULL (1) or [1] FP32.
 * dlogits [tokens, experts] with its stride; it may be d->logits itself. */
int bf16opt_balance_backward(const bf16opt_balance_t *d, const int32_t *ids, const int32_t *counts, const float *saved,
                             const float *dweights, const float *dloss, void *dlogits, uint64_t dlogits_stride,
                             void *stream);

/* Log-probabilities of given tokens, and two losses of them.  z: a row's logits, l its
 * label, T the temperature, s = softmax(z / T):
 *   logp = log s_l.
 * A row whose row_weight is 0, or whose label is outside [0, vocab), does not count: what stands in
 * it has no effect, and its loss, log-probability, saved numbers and gradient are 0.  Logits of
 * -inf are masked vocabulary (s = 0; a label on one, or a row with no other logit, has
 * logp -inf; in the latter s = 0 everywhere).  NaN and +inf in a row give NaN in that row
 * (and in what is summed over it) alone.
 *
 * saved [rows, 4] FP32 (16-byte aligned), which the forward calls leave for
 * bf16opt_token_logp_backward: the row's largest logit m, the sum of exp((z_j - m) / T), the
 * derivative c of the loss by logp, and the index (int32 bits) of the loss that it belongs
 * to, -1 for none. */
#define BF16OPT_TOKENS_MAX_ROWS 0x7fffffff

typedef struct {
    uint64_t rows;               /* tokens, at most BF16OPT_TOKENS_MAX_ROWS */
    uint32_t vocab;              /* 1 .. 2^30 */
    int32_t logits_type;         /* BF16OPT_TYPE_* of logits and dlogits */
    int32_t labels_type;         /* BF16OPT_INDEX_* of labels */
    float temperature;           /* finite, > 0, with a finite reciprocal */
    const void *logits;          /* [rows, vocab] */
    uint64_t logits_stride;
    const void *labels;          /* [rows] */
    const float *row_weight;     /* NULL (1), or [rows] */
} bf16opt_tokens_t;

/* logp [rows] FP32 (a weight other than 0 changes nothing here); saved may be NULL; c = 1. */
int bf16opt_token_logp_forward(const bf16opt_tokens_t *d, float *logp, float *saved, void *stream);

/* The backward call of all three: dz_j = c dloss[index] / T ([j = l] - s_j), rounded once.
 * saved: as a forward call with the same logits, labels and temperature left it (the
 * weights are in it).  dloss: NULL (1), or [losses] FP32 (an index outside counts as
 * none).  Rows whose c dloss is 0 are not read.  dlogits may be d->logits itself with the same stride. */
int bf16opt_token_logp_backward(const bf16opt_tokens_t *d, const float *saved, const float *dloss, uint64_t losses,
                                void *dlogits, uint64_t dlogits_stride, void *stream);

/* Clipped policy loss with a KL term.  A: advantage, w: row_weight,
 *   r = exp(logp - old_logp)  (old_logp NULL: it is logp itself, a constant: r = 1),
 *   k = exp(ref_logp - logp) - 1 - (ref_logp - logp)  (ref_logp NULL: 0),
 *   loss = w [ -min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A) + kl_weight k ],
 *   c = w [ -(r A where the minimum is r A, else 0) + kl_weight (1 - exp(ref_logp - logp)) ]. */
typedef struct {
    const float *advantage;      /* [rows] */
    const float *old_logp;       /* NULL, or [rows] */
    const float *ref_logp;       /* NULL, or [rows] */
    float clip_low, clip_high;   /* >= 0, clip_low <= 1; clip_high may be +inf */
    float kl_weight;             /* finite, >= 0 */
    uint32_t reserved;           /* must be 0 */
} bf16opt_policy_t;

/* loss, logp: [rows] FP32.  saved may be NULL. */
int bf16opt_policy_forward(const bf16opt_tokens_t *d, const bf16opt_policy_t *p, float *loss, float *logp, float *saved,
                           void *stream);

/* Loss and gradient (for a gradient of dloss [rows], or 1, of each row's loss) in one
 * pass over the logits.  dlogits as above; logp may be NULL. */
int bf16opt_policy_loss_grad(const bf16opt_tokens_t *d, const bf16opt_policy_t *p, const float *dloss, float *loss,
                             float *logp, void *dlogits, uint64_t dlogits_stride, void *stream);

/* Preference loss of pairs of sequences.  offsets [2 pairs + 1]: sequence i is rows
 * [offsets[i], offsets[i + 1]); sequence i < pairs is preferred to sequence pairs + i.
 * L_i: the sum of logp over the sequence's rows that count (row_weight is NULL here), divided by their
 * number if length_normalise (a sequence without any: 0).  ref_logp NULL: 0.
 *   h = (L_i - ref_i) - (L_j - ref_j), j = pairs + i;
 *   BF16OPT_PREFER_SIGMOID  m = beta h - margin;  loss = -(1 - e) log sigmoid(m) - e log sigmoid(-m),  e = label_smoothing,
 *   BF16OPT_PREFER_HINGE    m = beta h - margin;  loss = max(0, 1 - m),
 *   BF16OPT_PREFER_IPO      loss = (h - margin - 1 / (2 beta))^2.
 * Sums over a sequence are pairs of FP32 numbers (an addition is off by 2^-47 of the sum at
 * most).  Rows outside the sequences do not count.  Offsets that descend or lie outside
 * [0, rows] are taken to the nearest that do not (the sequence is then shorter or empty);
 * nothing outside the tensors is touched. */
#define BF16OPT_PREFER_SIGMOID 0
#define BF16OPT_PREFER_HINGE 1
#define BF16OPT_PREFER_IPO 2
#define BF16OPT_PREFER_MAX_PAIRS 65536

typedef struct {
    uint64_t pairs;              /* 0 .. BF16OPT_PREFER_MAX_PAIRS */
    int32_t offsets_type;        /* BF16OPT_INDEX_* */
    int32_t kind;                /* BF16OPT_PREFER_* */
    const void *offsets;         /* [2 pairs + 1] */
    const float *ref_logp;       /* NULL, or [2 pairs] */
    float beta;                  /* finite, > 0 */
    float label_smoothing;       /* 0 .. 0.5; SIGMOID alone uses it */
    float margin;                /* finite */
    int32_t length_normalise;    /* 0 or 1 */
} bf16opt_preference_t;

/* loss [pairs], logp [2 pairs] (L): FP32.  saved must be given. */
int bf16opt_preference_forward(const bf16opt_tokens_t *d, const bf16opt_preference_t *p, float *loss, float *logp,
                               float *saved, void *stream);

/* Activations kept in 8 bits, and the activation of a feed-forward block that keeps its inputs so.
 * A row's columns form runs of 32 (the last one may be shorter).  A run's scale is
 * 2^(b - 127), b the smallest byte for which its largest finite magnitude is at most 448
 * scales; each element is divided by it and rounded to the nearest e4m3 number, ties to even
 * (bias 7, largest 448, no infinities; one that would be 2^128 is kept as 1.875 2^127).  Inf and NaN are kept as NaN.
 * codes [rows, 32 runs], scales [rows, runs], runs = ceil(columns / 32); codes behind a
 * row's end are 0.  A row's elements are contiguous; its stride counts elements. */
#define BF16OPT_PACK_RUN 32

typedef struct {
    uint64_t rows;
    uint32_t columns;            /* 1 .. 2^30 */
    int32_t type;                /* BF16OPT_TYPE_* of everything that is not kept */
} bf16opt_pack_t;

/* codes: 16-byte aligned. */
int bf16opt_pack(const bf16opt_pack_t *d, const void *x, uint64_t x_stride, uint8_t *codes, uint8_t *scales, void *stream);
int bf16opt_unpack(const bf16opt_pack_t *d, const uint8_t *codes, const uint8_t *scales, void *x, uint64_t x_stride, void *stream);

/* h = act(gate) up  (up NULL: h = act(gate)), act one of
 *   BF16OPT_GLU_SILU  g sigmoid(g),
 *   BF16OPT_GLU_GELU  g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2 = g sigmoid(2 sqrt(2 / pi) (g + 0.044715 g^3))
 * (a sigmoid below 2^-128 counts as 0).
 * The forward call keeps gate and up in 8 bits (codes [parts, rows, 32 runs], scales
 * [parts, rows, runs]: gate's, then up's); the backward call works on what was kept, g' and u':
 *   dgate = dh u' act'(g'),  dup = dh act(g'),  and, if wanted, h' = act(g') u'
 * (which the gradient of the weights behind h needs, where h itself is not kept). */
#define BF16OPT_GLU_SILU 0
#define BF16OPT_GLU_GELU 1

typedef struct {
    uint64_t rows;
    uint32_t columns;            /* 1 .. 2^30 */
    int32_t type;                /* BF16OPT_TYPE_* of everything that is not kept */
    int32_t act;                 /* BF16OPT_GLU_* */
    int32_t gated;               /* 1: gate and up; 0: gate alone (up, dup: NULL) */
} bf16opt_glu_t;

/* codes and scales both NULL: nothing is kept.  h may be gate or up with the same stride. */
int bf16opt_glu_forward(const bf16opt_glu_t *d, const void *gate, uint64_t gate_stride, const void *up, uint64_t up_stride,
                        void *h, uint64_t h_stride, uint8_t *codes, uint8_t *scales, void *stream);

/* h may be NULL.  One of dgate, dup and h may be dh with the same stride.  Outputs may
 * be column ranges of one matrix (the same stride, no element twice). */
int bf16opt_glu_backward(const bf16opt_glu_t *d, const void *dh, uint64_t dh_stride, const uint8_t *codes, const uint8_t *scales,
                         void *dgate, uint64_t dgate_stride, void *dup, uint64_t dup_stride, void *h, uint64_t h_stride,
                         void *stream);

/* Rotary positions.  A head's first rotary_dim elements are pairs (x_i, x_{i + rotary_dim / 2})
 * (BF16OPT_ROTARY_HALF) or (x_{2i}, x_{2i + 1}) (BF16OPT_ROTARY_INTERLEAVED), i < rotary_dim / 2;
 * at position p each is turned by the angle p frequencies[i]:
 *   (a, b) -> scale (a cos - b sin, b cos + a sin)   (inverse: -sin),
 * the other elements are copied.  inverse gives the gradient of the inputs from that of the outputs.
 * The angle's whole turns are taken off in 64-bit whole numbers: p times the frequency to the nearest
 * 2^-64 turns, so up to |p| = 2^36 an angle is as exact as a near one (its FP32 number's 2^-24;
 * 2^-22 at 2^40).  Results are rounded once. */
#define BF16OPT_ROTARY_HALF 0
#define BF16OPT_ROTARY_INTERLEAVED 1
#define BF16OPT_ROTARY_MAX_DIM 256

typedef struct {
    uint64_t batch, seq;
    uint32_t heads, kv_heads;    /* of q and of k (0: no k) */
    uint32_t dim;                /* elements of a head, 1 .. 65536 */
    uint32_t rotary_dim;         /* even, 2 .. min(dim, BF16OPT_ROTARY_MAX_DIM) */
    int32_t type;                /* BF16OPT_TYPE_* of all four */
    int32_t layout;              /* BF16OPT_ROTARY_* */
    int32_t positions_type;      /* BF16OPT_INDEX_* */
    int32_t inverse;             /* 0 or 1 */
    const void *positions;       /* NULL (0, 1, ..), or [seq], or [batch, seq] */
    uint64_t positions_stride;   /* between batches: 0 or seq */
    int64_t offset;              /* added to every position */
    const double *frequencies;   /* host memory, [rotary_dim / 2]: radians per position, finite; read during the call */
    float scale;                 /* finite */
    uint32_t reserved;           /* must be 0 */
    uint64_t q_stride[3], k_stride[3], out_q_stride[3], out_k_stride[3];   /* elements between batches, tokens, heads */
} bf16opt_rotary_t;

/* A head's elements are contiguous; inputs may have any strides, outputs no element twice.  out_q
 * may be q and out_k k (with the same strides): then what is not turned is not touched.
 * Outputs may lie in one matrix with one another or with the inputs where every token's
 * (or every batch's) elements are apart. */
int bf16opt_rotary(const bf16opt_rotary_t *d, const void *q, const void *k, void *out_q, void *out_k, void *stream);

/* ---- checked build -------------------------------------------------------
 * No counterpart in the paper: a debugging aid standing in for a memory
 * checker.  In a build compiled with -DBF16K_CHECKS the kernels test, before
 * each chunk's accesses, that the chunk lies inside its segment, that its
 * scalar head and vector body stay inside the chunk and that every vector
 * pointer is 16-byte (FP32) / 8-byte (bf16) aligned; a violation sets a bit in
 * a device word (1 = chunk outside its segment, 2 = body outside the chunk,
 * 4 = misaligned vector pointer) and the chunk is skipped instead of accessed.
 * This call waits for the device, stores the word into *bits and clears it.
 * Release builds: *bits = 0 and BF16OPT_ERR_UNSUPPORTED.
 * Errors: INVALID_ARG (bits NULL), UNSUPPORTED, CUDA. */
int bf16opt_debug_faults(uint32_t *bits);

/* Static message of a status code; one-line message of the handle's last error. */
const char *bf16opt_error_string(int code);
const char *bf16opt_last_error(const bf16opt_t *h);

#ifdef __cplusplus
}
#endif
#endif /* BF16OPT_H */
