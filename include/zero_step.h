/*
 * zero_step.h -- C ABI of the fused per-rank ZeRO-1 shard step for MI355X
 * (gfx950).
 *
 * The operation ("CS336 Lecture 7: Parallelism 1", section "ZeRO Stage 1：
 * 优化器状态分片", the four-step workflow; "第2章 软件程序与专用硬件的结合",
 * section 2.3.4, Stage 1): every data-parallel rank holds a full bf16
 * gradient; a reduce-scatter gives rank i the *sum* over ranks of shard i;
 * rank i updates shard i with the optimizer state it alone keeps (fp32
 * master weights, fp32 first and second moments: the 16-bytes-per-parameter
 * table of section "训练内存的详细分析"); an all-gather then broadcasts the
 * updated bf16 parameters. This library performs the part of that step that
 * runs at one rank, on one GPU: the M gradient replicas of the shard are M
 * buffers in this GPU's memory.
 *
 *   g[i]  = (((g_0[i] + g_1[i]) + g_2[i]) + ... + g_{M-1}[i]) * grad_scale
 *           in binary32, ranks in ascending order, from the rank-0 value;
 *   found_inf = any g[i] is inf or NaN;
 *   norm  = sqrt(sum of g[i]^2 + external_sumsq)        (binary64 partials)
 *   coef  = min(1, max_grad_norm / (norm + 1e-6)) if max_grad_norm > 0 else 1
 *   skip  = found_inf && skip_on_nonfinite      (a skipped step writes nothing)
 *   AdamW (bias-corrected, eps outside the root, decay scaled by lr),
 *   evaluated in binary64 from the fp32 state and rounded once on store:
 *     m   = b1*m + (1-b1)*(coef*g);   v = b2*v + (1-b2)*(coef*g)^2
 *     w   = w*(1 - lr*wd) - lr * (m/(1-b1^t)) / (sqrt(v/(1-b2^t)) + eps)
 *   out   = bf16 round-to-nearest-even of the new fp32 w (the all-gather payload)
 *
 * AMP unscaling (grad_scale = 1/S) and the inf/NaN skip follow the
 * loss-scaling behaviour described in gsyq.cn/news/457874, section 3.2 trap 3;
 * the AdamW knob names follow its section 4.2 optimizer block. Clipping by the
 * global L2 norm is not on the pages; the coefficient is the common framework
 * convention above.
 *
 * Conventions for every entry point:
 *  - Pointers named *_dev, and every tensor pointer, are device pointers on the
 *    current HIP device. Arrays of pointers (grads) are HOST arrays holding
 *    device pointers. Structs passed by pointer (hparams, tensors) are host
 *    memory, read during the call only.
 *  - bf16 data are raw 16-bit codes (uint16). fp32 data are IEEE binary32.
 *  - The caller owns all memory. The library allocates no device memory; it
 *    keeps a small host-side cache of workspace plans. (The one exception is
 *    zero_step_noalloc's static scratch, a device array that is part of the
 *    library's code and is loaded with it.)
 *  - Every call is asynchronous on `stream` (0 = the null stream) and returns
 *    after enqueueing. Results are device-resident.
 *  - Errors: an int status (ZERO_OK or ZERO_ERR_*). On any error nothing is
 *    launched and no memory is written. n == 0 is a valid no-op. No C++
 *    exception crosses the ABI.
 *  - Any alignment is accepted; when all pointers of a tensor share their
 *    alignment modulo 16 bytes the kernels use 16-byte vector accesses.
 *  - The fused forms launch one workgroup per tile of a pass, at most
 *    2^31 - 1 tiles (an update pass's tiles hold 2048 elements: about 4.4e12
 *    elements per call); a larger call is ZERO_ERR_INVALID_ARGUMENT.
 *  - Outputs must not alias inputs or each other, except the in-place
 *    master/exp_avg/exp_avg_sq and what an entry point allows. The library
 *    never advances `step`: the caller increments it when the result record
 *    says `skipped == 0`.
 */
#ifndef ZERO_STEP_H
#define ZERO_STEP_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define ZERO_OK 0
#define ZERO_ERR_INVALID_ARGUMENT 1    /* null pointer, bad size or hyperparameter */
#define ZERO_ERR_WORKSPACE_TOO_SMALL 2 /* ws_bytes below the size query's answer */
#define ZERO_ERR_HIP 3                 /* a HIP runtime call failed (launch, copy) */
#define ZERO_ERR_STALE_WORKSPACE 4     /* set in zero_result.status by the device when a
                                          workspace no longer holds the plan of this call;
                                          the step then wrote nothing */
#define ZERO_ERR_BUCKET_PARTIALS 5     /* set in zero_result.status by zero_step_accumulated
                                          when a bucket partial was not written by a final
                                          zero_bucket_reduce with this stamp and grad_scale;
                                          the step then wrote nothing */
#define ZERO_ERR_SCRATCH_TOO_SMALL 6   /* zero_step_noalloc: the call's workspace would exceed
                                          ZERO_NOALLOC_SCRATCH_BYTES; nothing was launched */

/* Largest M accepted (ranks, i.e. gradient replicas per shard). */
#define ZERO_MAX_RANKS 65536

/* AdamW hyperparameters of one step (names as in a deepspeed_config.json
 * optimizer block, gsyq.cn/news/457874 section 4.2). Host memory. */
typedef struct zero_adamw_hparams {
    double lr;                 /* learning rate, finite, >= 0 */
    double beta1;              /* first-moment decay, in [0, 1) */
    double beta2;              /* second-moment decay, in [0, 1) */
    double eps;                /* added to sqrt of the bias-corrected v, finite, >= 0 */
    double weight_decay;       /* decoupled: w *= (1 - lr*weight_decay); finite */
    int64_t step;              /* t >= 1: index of this update (bias corrections) */
    double max_grad_norm;      /* > 0: clip g to this global L2 norm; <= 0: off */
    double grad_scale;         /* multiplies the fp32 sum, rounded to fp32 once: 1,
                                  1/S for an AMP loss scale S, 1/M for a mean; finite, > 0 */
    int32_t skip_on_nonfinite; /* nonzero: any inf/NaN in g skips the whole update */
    int32_t reserved;          /* must be 0 */
} zero_adamw_hparams;

/* One tensor's shard in a zero_step bucket list. Host memory. */
typedef struct zero_tensor {
    int64_t n;                /* elements in this shard, >= 0 */
    const void* const* grads; /* HOST array of M device pointers, n bf16 each (read only) */
    float* master;            /* device, n fp32 master weights, updated in place */
    float* exp_avg;           /* device, n fp32 first moments, updated in place */
    float* exp_avg_sq;        /* device, n fp32 second moments, updated in place */
    void* param_out;          /* device, n bf16 codes, written (the all-gather payload) */
} zero_tensor;

/* Device-resident result record of a step, 32 bytes, written by the library. */
typedef struct zero_result {
    double sumsq;      /* sum of g^2 over every element of the call, plus external_sumsq */
    double clip_coef;  /* coefficient applied to g, binary64 (1 when clipping is off) */
    float grad_norm;   /* sqrt(sumsq) rounded to fp32 (inf/NaN when found_inf) */
    int32_t found_inf; /* 1 when any unscaled reduced gradient is inf or NaN */
    int32_t skipped;   /* 1 when the update was not applied */
    int32_t status;    /* ZERO_OK, or ZERO_ERR_STALE_WORKSPACE */
} zero_result;

/*
 * zero_shard_reduce -- the reduce-scatter arithmetic at one rank
 * ("CS336 Lecture 7", section "五种基本集合通信操作", Reduce-Scatter; section
 * "ZeRO Stage 1", step 2: GPU i receives the summed gradient of shard i).
 *   g_out[i] = fl32(fold_{r=0..M-1} bf16->fp32(grads[r][i])) * fl32(grad_scale)
 * grads: host array of M device pointers to n bf16 codes. g_out: device, n
 * fp32, must not overlap any replica. 1 <= M <= ZERO_MAX_RANKS, n >= 0,
 * grad_scale finite and > 0. Bit-exact: the fold order is fixed.
 */
int zero_shard_reduce(const void* const* grads, int32_t M, int64_t n, double grad_scale, float* g_out,
                      hipStream_t stream);

/*
 * zero_grad_check_norm_workspace_bytes -- workspace size for
 * zero_grad_check_norm over n elements (0 when n == 0).
 */
size_t zero_grad_check_norm_workspace_bytes(int64_t n);

/*
 * zero_grad_check_norm -- non-finite check, global L2 norm, clip coefficient
 * and skip decision over an fp32 gradient g (device, n elements), written to
 * the device record res_dev. The check and the skip follow the loss-scaling
 * cycle of gsyq.cn/news/457874 section 3.2 trap 3 (a step whose unscaled
 * gradient holds inf or NaN is not applied); the norm is global because each
 * rank holds one shard of the summed gradient ("CS336 Lecture 7", "ZeRO
 * Stage 1" step 2), so the other ranks' share enters as external_sumsq.
 * Clipping by that norm is not on the pages: the coefficient is the common
 * framework rule stated at the top of this header. hp may be NULL (no clipping, no skip); only its
 * max_grad_norm and skip_on_nonfinite are read. external_sumsq is the other
 * ranks' sum of squares for a multi-GPU caller, 0 on one GPU: NaN and +inf
 * propagate into the norm, a negative value is ZERO_ERR_INVALID_ARGUMENT (as
 * in every call that takes it). ws: device workspace of at least
 * zero_grad_check_norm_workspace_bytes(n) bytes, contents irrelevant on entry.
 * The sum of squares uses exact binary64 squares and a fixed reduction tree
 * (bitwise repeatable on one device).
 */
int zero_grad_check_norm(const float* g, int64_t n, const zero_adamw_hparams* hp, double external_sumsq,
                         void* ws, size_t ws_bytes, zero_result* res_dev, hipStream_t stream);

/*
 * zero_adamw_step -- AdamW on fp32 master/exp_avg/exp_avg_sq (device, n each,
 * in place) from the fp32 gradient g (device, n), plus the bf16 emit into
 * param_out (device, n bf16 codes): the local update of "CS336 Lecture 7",
 * "ZeRO Stage 1" step 3 (rank i updates shard i with the optimizer state it
 * alone keeps: the fp32 master copy and both moments of the table in section
 * "训练内存的详细分析") and the bf16 payload of the all-gather in step 4; the
 * knobs are those of the AdamW optimizer block in gsyq.cn/news/457874
 * section 4.2, and the formula is the one stated at the top of this header. hp is required (max_grad_norm and
 * skip_on_nonfinite are ignored here). res_dev (device, may be NULL) supplies
 * clip_coef and skipped from zero_grad_check_norm: when skipped is set the
 * kernel writes nothing; when res_dev is NULL the coefficient is 1.
 */
int zero_adamw_step(float* master, float* exp_avg, float* exp_avg_sq, const float* g, void* param_out, int64_t n,
                    const zero_adamw_hparams* hp, const zero_result* res_dev, hipStream_t stream);

/*
 * zero_step_workspace_bytes -- workspace size for zero_step over this tensor
 * list and hyperparameters (pointers inside `tensors` are not read). Returns 0
 * on invalid arguments.
 */
size_t zero_step_workspace_bytes(const zero_tensor* tensors, int32_t T, int32_t M, const zero_adamw_hparams* hp);

/*
 * zero_step -- the fused step over a bucket list of T tensor shards, each with
 * M bf16 replicas ("CS336 Lecture 7", "ZeRO Stage 1" steps 2-3 and the
 * payload of step 4; per-layer buckets as in its section "ZeRO Stage 2").
 * The norm and found_inf are global over all T tensors. Without clipping and
 * skipping it is one streaming pass; with either, a first pass writes the fp32
 * reduced gradient to the workspace and a second pass applies the update.
 * Above ZERO_STREAM_STORES_MIN_PARAMS parameters in all the call's tensors
 * together, the state stores of the updating pass stream out to memory (see
 * ZERO_BUCKET_STREAM_STORES); the results do not depend on it.
 * ws: device workspace of zero_step_workspace_bytes(...) bytes, 256-byte
 * aligned. The workspace caches the tensor table of the call; it belongs to
 * the library from this call until the caller reuses it for anything else,
 * and two calls that share a workspace must not run concurrently. res_dev:
 * device result record. external_sumsq as for zero_grad_check_norm. Returns
 * ZERO_ERR_WORKSPACE_TOO_SMALL if ws_bytes is short.
 */
int zero_step(const zero_tensor* tensors, int32_t T, int32_t M, const zero_adamw_hparams* hp,
              double external_sumsq, void* ws, size_t ws_bytes, zero_result* res_dev, hipStream_t stream);

/* Bytes of the static device workspace of zero_step_noalloc (64 MiB per GPU). */
#define ZERO_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)

/*
 * zero_step_noalloc -- zero_step for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): the workspace is a static device array inside the
 * library, ZERO_NOALLOC_SCRATCH_BYTES bytes on each GPU, taken when the
 * library's code is loaded on that GPU and held until the process ends. The
 * call itself allocates nothing (no hipMalloc, no hipFree, no allocating
 * library routine); the caller still passes the tensors and res_dev.
 * Arguments, results and errors as for zero_step, plus
 * ZERO_ERR_SCRATCH_TOO_SMALL, returned before anything is launched, when
 * zero_step_workspace_bytes(tensors, T, M, hp) exceeds the scratch: the
 * single-pass plan takes about 12 bytes per 1024 elements plus 112 + 8*M
 * bytes per tensor (every workload up to billions of elements fits), a
 * two-pass plan (clipping or skipping) also holds the fp32 gradient, 4 bytes
 * per element (up to about 16 million elements).
 * Every call on one GPU shares that GPU's scratch, which keeps the last
 * call's plan and re-arms its own counters: calls on one GPU must be ordered
 * (one stream, or events); calls that overlap on one GPU race and corrupt
 * each other's results. A HIP graph that captures a call holds the scratch's
 * address, so a replay is valid only while no other call with a different
 * tensor list has used the scratch since the capture.
 */
int zero_step_noalloc(const zero_tensor* tensors, int32_t T, int32_t M, const zero_adamw_hparams* hp,
                      double external_sumsq, zero_result* res_dev, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Dynamic loss scale (AMP).
 *
 * gsyq.cn/news/457874 configures the fp16 loss scale with the fp16 block of
 * its section 4.2 listing (loss_scale 0 = dynamic, initial_scale_power,
 * loss_scale_window, hysteresis, min_loss_scale) and describes the scaler's
 * cycle in section 3.2 trap 3 (scale the loss, step on unscaled gradients,
 * update the scale). The pages name the knobs, not the rule; the rule read
 * from them:
 *   - S starts at 2^initial_scale_power;
 *   - a step whose unscaled reduced gradient holds inf/NaN is skipped and is
 *     an overflow; the hysteresis-th overflow in a row (counted since the last
 *     clean step or halving) halves S, never below min_scale, and restarts the
 *     count;
 *   - a clean step clears the overflow count; the window-th clean step in a
 *     row (counted since the last overflow or doubling) doubles S unless 2S is
 *     not a finite binary32 value, and restarts the count;
 *   - inv_scale = 1/S rounded to binary32 (exact while S is a power of two).
 * The state stays in device memory: a training loop moves it without a host
 * synchronisation.
 * ------------------------------------------------------------------------ */

/* Loss-scale state, 16 bytes, device memory, written by the library. */
typedef struct zero_loss_scale {
    float scale;        /* S: the factor the loss was multiplied by */
    float inv_scale;    /* 1/S rounded to binary32 */
    int32_t good_steps; /* clean steps in a row since the last overflow or doubling */
    int32_t overflows;  /* overflowing steps in a row since the last clean step or halving */
} zero_loss_scale;

/* Loss-scale knobs (host memory, read during the call). */
typedef struct zero_loss_scale_config {
    int32_t initial_scale_power; /* S starts at 2^power; -126 <= power <= 127 */
    int32_t window;              /* loss_scale_window: clean steps per doubling, >= 1 */
    int32_t hysteresis;          /* overflows in a row per halving, >= 1 */
    float min_scale;             /* min_loss_scale: finite, > 0 */
} zero_loss_scale_config;

/*
 * zero_loss_scale_init -- write the initial state (S = 2^initial_scale_power,
 * counts 0) to ls_dev (device, 16 bytes).
 */
int zero_loss_scale_init(const zero_loss_scale_config* cfg, zero_loss_scale* ls_dev, hipStream_t stream);

/*
 * zero_loss_scale_update -- move the state ls_dev on the found_inf flag of
 * the result record res_dev (device) of a step that used it, e.g. after
 * zero_shard_reduce with grad_scale = inv_scale and zero_grad_check_norm.
 * A record whose status is not ZERO_OK leaves the state unchanged.
 */
int zero_loss_scale_update(const zero_loss_scale_config* cfg, const zero_result* res_dev, zero_loss_scale* ls_dev,
                           hipStream_t stream);

/*
 * zero_step_amp_workspace_bytes -- workspace size for zero_step_amp (always
 * the two-pass plan). Returns 0 on invalid arguments.
 */
size_t zero_step_amp_workspace_bytes(const zero_tensor* tensors, int32_t T, int32_t M, const zero_adamw_hparams* hp);

/*
 * zero_step_amp -- zero_step with the dynamic loss scale in ls_dev: the fp32
 * sum is multiplied by fl32(grad_scale) * inv_scale (a binary32 product read
 * from ls_dev by the device, so the host never needs S); a step with any
 * inf/NaN in the unscaled gradient is always skipped (skip_on_nonfinite is
 * ignored); after the fold, the state moves on the step's found_inf. No
 * extra launch: the workgroup that writes the result record also updates
 * ls_dev. ls_dev must not change while the call runs, and two calls that share
 * ls_dev must be ordered (one stream). Other arguments and errors as for
 * zero_step; the workspace size is zero_step_amp_workspace_bytes(...).
 */
int zero_step_amp(const zero_tensor* tensors, int32_t T, int32_t M, const zero_adamw_hparams* hp,
                  const zero_loss_scale_config* cfg, zero_loss_scale* ls_dev, double external_sumsq, void* ws,
                  size_t ws_bytes, zero_result* res_dev, hipStream_t stream);

/* ------------------------------------------------------------------------
 * ZeRO-2, streaming.
 *
 * "CS336 Lecture 7: Parallelism 1", section "ZeRO Stage 2": as backward
 * produces each layer's gradient, it is reduced at once to the rank that owns
 * its shard, and the local copy is freed, so no rank holds a whole gradient.
 * gsyq.cn/news/457874 section 4.2 sends gradients in buckets
 * (reduce_bucket_size) and accumulates gradient_accumulation_steps
 * micro-batches per step. At one rank, on one GPU:
 *   - zero_bucket_reduce, once per bucket and micro-batch, as the bucket's M
 *     replicas arrive: acc[i] = fold(replicas) for the first micro-batch, or
 *     acc[i] = acc[i] + fold(replicas) (one binary32 add) for later ones. The
 *     fold is zero_shard_reduce's, without the scale: acc is the running sum
 *     of the reduce-scatter results. On the last micro-batch (FINAL) the call
 *     also writes the bucket's sum of squares and non-finite flag of
 *     g = acc * fl32(grad_scale) to a 32-byte bucket partial, stamped;
 *   - zero_step_accumulated, once per step: combines the bucket partials in
 *     index order into the result record (norm, clip coefficient, skip), then
 *     applies AdamW and the bf16 emit from g = acc * fl32(grad_scale), as
 *     zero_step does from its fold.
 * With one micro-batch, the state this writes is bit-identical to zero_step's
 * over the same replicas when clipping is off (the norm's summation tree
 * differs, so a clipped step may differ by the last bit of the coefficient).
 * ------------------------------------------------------------------------ */

/* flags of zero_bucket_reduce */
#define ZERO_BUCKET_ACCUMULATE 1 /* add the fold to acc; otherwise store it (first micro-batch) */
#define ZERO_BUCKET_FINAL 2      /* last micro-batch of the step: also write the bucket partial */
/* flag of zero_bucket_step: the state stores of the pass stream out to memory
 * (non-temporal, system scope) instead of waiting in the caches. Results are
 * the same either way; it is faster when the step's buckets together write
 * more than the GPU's 256 MiB Infinity Cache holds, i.e. above
 * ZERO_STREAM_STORES_MIN_PARAMS parameters (12 bytes of state and 2 of bf16
 * output each), and slower below. zero_step and zero_step_accumulated make
 * this choice themselves from the size of the step. */
#define ZERO_BUCKET_STREAM_STORES 4
#define ZERO_STREAM_STORES_MIN_PARAMS ((256ll << 20) / 14)

/* One tensor shard of a gradient bucket. Host memory. */
typedef struct zero_grad_shard {
    int64_t n;                /* elements in this shard, >= 0 */
    const void* const* grads; /* HOST array of M device pointers, n bf16 each (read only) */
    float* grad_acc;          /* device, n fp32: the shard's accumulated gradient, updated */
} zero_grad_shard;

/* One bucket's share of the step's norm and flag, 32 bytes, device memory. */
typedef struct zero_bucket_partial {
    double sumsq;      /* sum over the bucket of g^2, g = acc * fl32(grad_scale) (binary64) */
    uint64_t stamp;    /* the stamp of the final zero_bucket_reduce that wrote it */
    int32_t found_inf; /* 1 when any g of the bucket is inf or NaN */
    float grad_scale;  /* fl32(grad_scale) of that call */
    int64_t reserved;  /* written 0 */
} zero_bucket_partial;

/* One tensor shard of a zero_step_accumulated list. Host memory. */
typedef struct zero_acc_tensor {
    int64_t n;              /* elements in this shard, >= 0 */
    const float* grad_acc;  /* device, n fp32: the accumulated gradient (read only) */
    float* master;          /* device, n fp32, updated in place */
    float* exp_avg;         /* device, n fp32, updated in place */
    float* exp_avg_sq;      /* device, n fp32, updated in place */
    void* param_out;        /* device, n bf16 codes, written */
} zero_acc_tensor;

/*
 * zero_bucket_reduce_workspace_bytes -- workspace size for zero_bucket_reduce
 * over this bucket (pointers inside `shards` are not read); 0 on invalid
 * arguments.
 */
size_t zero_bucket_reduce_workspace_bytes(const zero_grad_shard* shards, int32_t T, int32_t M);

/*
 * zero_bucket_reduce -- fold one micro-batch of one bucket (T tensor shards,
 * M bf16 replicas each) into the shards' fp32 accumulators, per `flags`
 * (ZERO_BUCKET_ACCUMULATE, ZERO_BUCKET_FINAL; other bits are an error).
 * With ZERO_BUCKET_FINAL, grad_scale (finite, > 0; the step's) and stamp (any
 * value that differs from the previous step's, e.g. an iteration count) go
 * into *partial_dev (device, 32 bytes); without it they are ignored and
 * partial_dev may be NULL. ws: device workspace of
 * zero_bucket_reduce_workspace_bytes(...) bytes, 256-byte aligned, one per
 * bucket (it caches the bucket's tables; calls that share one must not run
 * concurrently). A workspace that no longer holds this bucket's tables is
 * detected on the device: nothing is written but *partial_dev, whose stamp is
 * then invalid (zero_step_accumulated reports it; a later final call on a
 * valid workspace would overwrite it, so call zero_workspace_forget before
 * reusing a bucket workspace for anything else). The accumulators must not
 * overlap the replicas or each other.
 */
int zero_bucket_reduce(const zero_grad_shard* shards, int32_t T, int32_t M, int32_t flags, double grad_scale,
                       uint64_t stamp, zero_bucket_partial* partial_dev, void* ws, size_t ws_bytes,
                       hipStream_t stream);

/*
 * zero_bucket_reduce_amp -- zero_bucket_reduce under the dynamic loss scale
 * ls_dev (device): the final pass squares acc * (fl32(grad_scale) *
 * inv_scale), the binary32 product read from ls_dev on the device, and
 * stores that product in the partial's grad_scale. ls_dev is only read; it
 * must not move between a bucket's final pass and the step that consumes the
 * partials (zero_step_accumulated_amp moves it at the end of the step).
 */
int zero_bucket_reduce_amp(const zero_grad_shard* shards, int32_t T, int32_t M, int32_t flags, double grad_scale,
                           const zero_loss_scale* ls_dev, uint64_t stamp, zero_bucket_partial* partial_dev, void* ws,
                           size_t ws_bytes, hipStream_t stream);

/*
 * zero_step_accumulated_workspace_bytes -- workspace size for
 * zero_step_accumulated over this tensor list; 0 on invalid arguments.
 */
size_t zero_step_accumulated_workspace_bytes(const zero_acc_tensor* tensors, int32_t T);

/*
 * zero_step_accumulated -- the step from the accumulated shard gradients:
 * partials_dev (device, nbuckets >= 0 records, each written by the final
 * zero_bucket_reduce of one bucket with this `stamp` and hp->grad_scale) are
 * combined in index order, with external_sumsq, into res_dev (norm, clip
 * coefficient, skip, as zero_step); unless skipped, AdamW and the bf16 emit
 * are applied to every tensor from g = acc * fl32(hp->grad_scale). A partial
 * with another stamp or scale sets res_dev->status = ZERO_ERR_BUCKET_PARTIALS
 * and nothing is written. The state stores stream out above
 * ZERO_STREAM_STORES_MIN_PARAMS parameters, as in zero_step. ws: device
 * workspace of zero_step_accumulated_workspace_bytes(...) bytes, 256-byte
 * aligned, as for zero_step.
 */
int zero_step_accumulated(const zero_acc_tensor* tensors, int32_t T, const zero_adamw_hparams* hp,
                          const zero_bucket_partial* partials_dev, int32_t nbuckets, uint64_t stamp,
                          double external_sumsq, void* ws, size_t ws_bytes, zero_result* res_dev,
                          hipStream_t stream);

/*
 * zero_step_accumulated_amp -- zero_step_accumulated under the dynamic loss
 * scale ls_dev (device, with its config cfg): the multiplier is
 * fl32(hp->grad_scale) * inv_scale read on the device (the partials must
 * carry that product, as zero_bucket_reduce_amp writes it); a step with any
 * inf/NaN is always skipped (skip_on_nonfinite is ignored); after the update
 * the state moves on the step's found_inf (one more small launch). Workspace
 * as for zero_step_accumulated.
 */
int zero_step_accumulated_amp(const zero_acc_tensor* tensors, int32_t T, const zero_adamw_hparams* hp,
                              const zero_loss_scale_config* cfg, zero_loss_scale* ls_dev,
                              const zero_bucket_partial* partials_dev, int32_t nbuckets, uint64_t stamp,
                              double external_sumsq, void* ws, size_t ws_bytes, zero_result* res_dev,
                              hipStream_t stream);

/* ------------------------------------------------------------------------
 * ZeRO-2, the final micro-batch fused with the update.
 *
 * Without clipping and without skipping, no element's update waits for the
 * global norm, so the last micro-batch of a bucket can be folded and applied
 * in one pass instead of being stored to the accumulator and read back by
 * zero_step_accumulated ("CS336 Lecture 7", "ZeRO Stage 2": each bucket is
 * reduced to its owner as soon as backward has produced it; here its owner
 * also updates it then). Per element of the bucket:
 *   g   = (acc + fold(replicas)) * fl32(grad_scale)   with ZERO_BUCKET_ACCUMULATE
 *   g   = fold(replicas) * fl32(grad_scale)           without (one micro-batch)
 *   AdamW on master, m, v and the bf16 emit, exactly as zero_step; acc is read,
 *   never written. The bucket's sum of squares and non-finite flag of g go to
 *   a stamped bucket partial, as a final zero_bucket_reduce writes it.
 * The step's result record then comes from zero_step_accumulated with no
 * tensors (T = 0, ws may be NULL): it combines the bucket partials in index
 * order with external_sumsq. The state equals, bit for bit, what
 * zero_bucket_reduce (FINAL) followed by zero_step_accumulated writes.
 * Traffic per element: 2M + 26 bytes for one micro-batch (2M + 30 with the
 * accumulator), against 2M + 4 + 30 in two passes.
 * ------------------------------------------------------------------------ */

/* One tensor shard of a fused final bucket pass. Host memory. */
typedef struct zero_bucket_tensor {
    int64_t n;                /* elements in this shard, >= 0 */
    const void* const* grads; /* HOST array of M device pointers, n bf16 each (read only) */
    const float* grad_acc;    /* device, n fp32: the earlier micro-batches' sum, read with
                                 ZERO_BUCKET_ACCUMULATE (may be NULL otherwise); not written */
    float* master;            /* device, n fp32, updated in place */
    float* exp_avg;           /* device, n fp32, updated in place */
    float* exp_avg_sq;        /* device, n fp32, updated in place */
    void* param_out;          /* device, n bf16 codes, written */
} zero_bucket_tensor;

/*
 * zero_bucket_step_workspace_bytes -- workspace size for zero_bucket_step over
 * this bucket (pointers inside `tensors` are not read); 0 on invalid arguments.
 */
size_t zero_bucket_step_workspace_bytes(const zero_bucket_tensor* tensors, int32_t T, int32_t M);

/*
 * zero_bucket_step -- the final micro-batch of one bucket (T tensor shards,
 * M bf16 replicas each), folded, added to the accumulator when `flags` has
 * ZERO_BUCKET_ACCUMULATE (without it: the bucket's only micro-batch), scaled
 * and applied with AdamW and the bf16 emit in one pass, its state stores
 * streamed when `flags` has ZERO_BUCKET_STREAM_STORES (any other bit is an
 * error);
 * the bucket partial *partial_dev (device, 32 bytes) gets the bucket's sum of
 * squares and flag with `stamp` and fl32(hp->grad_scale). hp must have
 * max_grad_norm <= 0 and skip_on_nonfinite == 0 (otherwise
 * ZERO_ERR_INVALID_ARGUMENT: the update would have to wait for the norm).
 * A non-finite gradient is flagged in the partial and still applied, as
 * zero_step does without skipping. ws: device workspace of
 * zero_bucket_step_workspace_bytes(...) bytes, 256-byte aligned, one per
 * bucket (it caches the bucket's tables; calls that share one must not run
 * concurrently); a workspace that no longer holds the bucket's tables is
 * detected on the device, and then nothing is written but an invalid
 * partial. Buckets are independent: different buckets may run on different
 * streams.
 */
int zero_bucket_step(const zero_bucket_tensor* tensors, int32_t T, int32_t M, int32_t flags,
                     const zero_adamw_hparams* hp, uint64_t stamp, zero_bucket_partial* partial_dev, void* ws,
                     size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * CPU-offloaded step (ZeRO-Offload).
 *
 * "第2章 软件程序与专用硬件的结合" section 2.3.4 names ZeRO-Offload, which
 * moves the optimizer state to CPU memory; gsyq.cn/news/457874 section 4.2
 * configures it (offload_optimizer: device cpu, pin_memory true) and reports
 * its trade: less GPU memory, a slower step, CPU-GPU transfers of ~20 GB/s.
 * Here the fp32 master, m and v of the shard live in host memory. The GPU
 * folds the M replicas, unscales, flags and squares (the first pass of the
 * two-pass step, into a device fp32 gradient); the gradient goes to pinned
 * host memory in chunks; host threads apply AdamW to each chunk as it lands
 * (binary64, the same formula and rounding as the GPU kernels) and emit bf16;
 * each bf16 chunk goes back to the device shard. The result equals zero_step's
 * over the same replicas: 4 + 2 bytes per parameter cross the host link
 * instead of 12 bytes of state living in HBM.
 * ------------------------------------------------------------------------ */

/* One tensor shard of an offloaded step. Host memory. */
typedef struct zero_offload_tensor {
    int64_t n;                /* elements in this shard, >= 0 */
    const void* const* grads; /* HOST array of M device pointers, n bf16 each (read only) */
    float* master;            /* HOST memory, n fp32, updated in place */
    float* exp_avg;           /* HOST memory, n fp32, updated in place */
    float* exp_avg_sq;        /* HOST memory, n fp32, updated in place */
    void* param_out;          /* DEVICE, n bf16 codes, written by host-to-device copies */
} zero_offload_tensor;

/* Device workspace size of zero_offload_step (plan, result record, the fp32
 * gradient, one 32-byte partial per fold group); 0 on invalid arguments. */
size_t zero_offload_workspace_bytes(const zero_offload_tensor* tensors, int32_t T, int32_t M);

/* Pinned host workspace size of zero_offload_step (staging: 4 bytes of
 * gradient and 2 bytes of bf16 output per element); 0 on invalid arguments. */
size_t zero_offload_host_workspace_bytes(const zero_offload_tensor* tensors, int32_t T);

/*
 * zero_offload_step -- the step with the optimizer state in host memory.
 * hp, external_sumsq and the result as for zero_step (*res_host, HOST memory,
 * is written before the call returns). ws: device workspace of
 * zero_offload_workspace_bytes(...) bytes, 256-byte aligned (it caches the
 * call's tables, as for zero_step). host_ws: PINNED host memory
 * (hipHostMalloc) of zero_offload_host_workspace_bytes(...) bytes, 64-byte
 * aligned. threads: host threads of the update (0: the size of the process's
 * CPU affinity mask). The call waits for the GPU's fold and returns once
 * master, m and v are updated on the host (or the step is skipped); the
 * bf16 copies into param_out are then enqueued, and `stream` is made to wait
 * for them, so work later on `stream` sees the new shard. Those copies read
 * host_ws: it stays allocated and untouched until `stream` has passed them,
 * and calls that share a host workspace must be issued on one stream.
 * Argument errors are reported before anything is launched; a HIP error
 * during the transfers (ZERO_ERR_HIP) can leave the host state partly
 * updated, and the call drains its copies before returning it.
 * Without clipping, skipping or a dynamic loss scale the update needs nothing
 * global, so the fold runs in groups of tiles and the host updates each piece
 * of the gradient as it arrives; the state is the same as with one fold pass
 * (and as zero_step's), while the reported sum of squares combines the group
 * partials in group order (it may differ from zero_step's in the last bits).
 */
int zero_offload_step(const zero_offload_tensor* tensors, int32_t T, int32_t M, const zero_adamw_hparams* hp,
                      double external_sumsq, void* ws, size_t ws_bytes, void* host_ws, size_t host_ws_bytes,
                      zero_result* res_host, int32_t threads, hipStream_t stream);

/*
 * zero_offload_step_amp -- zero_offload_step under the dynamic loss scale
 * ls_dev (device, with its config cfg): the GPU's fold multiplies by
 * fl32(hp->grad_scale) * inv_scale read on the device, a step with any inf/NaN
 * is always skipped, and the fold's last workgroup moves the state, as in
 * zero_step_amp; the host update is unchanged. Workspaces as for
 * zero_offload_step.
 */
int zero_offload_step_amp(const zero_offload_tensor* tensors, int32_t T, int32_t M, const zero_adamw_hparams* hp,
                          const zero_loss_scale_config* cfg, zero_loss_scale* ls_dev, double external_sumsq, void* ws,
                          size_t ws_bytes, void* host_ws, size_t host_ws_bytes, zero_result* res_host,
                          int32_t threads, hipStream_t stream);

/*
 * zero_offload_adamw_host -- the host half alone: AdamW on host fp32
 * master/exp_avg/exp_avg_sq (n each, in place) from the host fp32 gradient g
 * (multiplied by clip_coef in binary64), bf16 output into host param_out;
 * hp as for zero_adamw_step; threads as above. For a caller that moves the
 * gradient itself. Synchronous; launches nothing on the GPU.
 */
int zero_offload_adamw_host(float* master, float* exp_avg, float* exp_avg_sq, const float* g, void* param_out,
                            int64_t n, const zero_adamw_hparams* hp, double clip_coef, int32_t threads);

/* ------------------------------------------------------------------------
 * Around a training block: 8-bit activation checkpoints and the gradients
 * taken from them.
 *
 * "CS336 Lecture 7: Parallelism 1" counts activations (34 s*b*h bytes a layer,
 * P2 section "激活内存") next to the 16 bytes per parameter that the calls above
 * manage. These calls keep the rows that a block's backward pass needs in 8
 * bits, and write the gradients of its matrices and norm vectors in the form
 * that the calls above read: one bf16 gradient replica, or a sum added to an
 * fp32 accumulator (micro-batch after micro-batch).
 *
 * A row-major operand is a zero_rows: any row stride ld >= the columns, any
 * base that is a multiple of its element size (16-byte accesses are used at
 * any alignment). Rows and columns beyond a call's sizes are neither read nor
 * written. Vectors are zero_rows with one row, whose ld is ignored.
 *
 * The 8-bit form of rows x cols values (an "act8"): every row is cut into
 * blocks of 32 columns (the last may be short); a block is stored as codes
 * and one power of two 2^k, k the smallest integer >= -117 with
 *   max |x| <= F * 2^k,   F = 448 (ZERO_ACT8_E4M3) or 127 (ZERO_ACT8_INT8),
 * and code = x * 2^-k rounded to nearest even (e4m3 with its subnormals, or an
 * integer). The scale is a power of two so that a decoded value, code * 2^k,
 * has at most 7 significant bits and is exact in bf16: products of decoded
 * values are products of what was saved. A block that holds an inf or NaN
 * decodes to NaN in every element, so that it reaches the gradients and their
 * found_inf. (A finite value that rounds up to 2^128 decodes to infinity.)
 * In memory, P = cols rounded up to 32: rows * P code bytes, row by row, the
 * columns from cols on 0, then rows * P/32 scale bytes k + 127 (255: NaN).
 * The buffer is 16-byte aligned, zero_act8_bytes(rows, cols) bytes.
 * ------------------------------------------------------------------------ */

/* Element types of a zero_rows. */
#define ZERO_BF16 1
#define ZERO_F32 2

/* 8-bit code formats. e4m3 keeps small values beside large ones (half a step
 * is 2^-4 of the value); int8 has an even step (half of it is at most 1/127 of
 * the block's largest value, and no less than 1/254). */
#define ZERO_ACT8_E4M3 1
#define ZERO_ACT8_INT8 2

/* flag of zero_act8_wgrad, zero_block_norm_grad, zero_layer_norm_grad and
 * zero_block_ffn_grad: add to the gradient buffers, which are then fp32;
 * otherwise they are overwritten */
#define ZERO_GRAD_ACCUMULATE 1

/* Largest cols of zero_block_norm and zero_layer_norm, whose rows stay in the
 * registers of one workgroup, and of zero_block_norm_grad and
 * zero_layer_norm_grad, which take wider rows than those of 6144 columns (8192
 * from act8 buffers with few gate rows), the latter than those of 8192, in
 * strips and read them twice. */
#define ZERO_BLOCK_NORM_MAX_COLS 16384

/* A row-major matrix in device memory (the struct itself is host memory). */
typedef struct zero_rows {
    void* data;       /* device; NULL: the operand is absent */
    int64_t ld;       /* elements from one row to the next, >= the columns */
    int32_t dtype;    /* ZERO_BF16 or ZERO_F32 */
    int32_t reserved; /* must be 0 */
} zero_rows;

/* zero_act8_bytes -- size of an act8 buffer; 0 on invalid sizes. */
size_t zero_act8_bytes(int64_t rows, int64_t cols);

/*
 * zero_act8_save -- x (rows x cols, bf16 or fp32) into the act8 buffer ckpt.
 * zero_act8_load -- the act8 buffer ckpt into out (rows x cols, bf16 or fp32),
 * exactly. 0 <= rows < 2^31, 0 <= cols <= 2^30, rows * P < 2^36; rows or cols 0
 * is a no-op.
 */
int zero_act8_save(const zero_rows* x, int64_t rows, int64_t cols, int32_t format, void* ckpt, hipStream_t stream);
int zero_act8_load(const void* ckpt, int64_t rows, int64_t cols, int32_t format, const zero_rows* out,
                   hipStream_t stream);

/*
 * zero_act8_wgrad_workspace_bytes -- workspace size of zero_act8_wgrad (the
 * partial sums of a product that is split over its rows; often 0); also 0 on
 * invalid sizes.
 */
size_t zero_act8_wgrad_workspace_bytes(int64_t rows, int64_t outs, int64_t cols);

/*
 * zero_act8_wgrad -- the weight gradient of a linear layer out = in * W^T from
 * the gradient dy of its output (rows x outs, bf16) and its input saved in 8
 * bits (rows x cols):
 *   dw[o][i] (+)= col_scale[i] * sum_t dy[t][o] * x[t][i]
 * summed in fp32 in an order that depends only on the sizes. col_scale (cols
 * values, bf16 or fp32; NULL: ones) is the weight of the norm before the
 * layer when the checkpoint holds that norm's rows before their weight, as
 * zero_block_norm saves them. dw (outs x cols): bf16 (a gradient replica) or
 * fp32; with ZERO_GRAD_ACCUMULATE in flags, fp32 and added to. rows == 0
 * writes zeros (nothing with ZERO_GRAD_ACCUMULATE). rows, outs < 2^31, cols <=
 * 2^30, and dw has fewer than 2^20 tiles of 128 x 128 (1.7e10 elements).
 * ws: device workspace of zero_act8_wgrad_workspace_bytes(...) bytes, 16-byte
 * aligned (NULL if that is 0), contents irrelevant on entry and not kept; two
 * calls that share one must not run concurrently. The plan that a step keeps in
 * any part of it is forgotten, as by zero_workspace_forget.
 */
int zero_act8_wgrad(const zero_rows* dy, const void* ckpt, int64_t rows, int64_t outs, int64_t cols, int32_t format,
                    const zero_rows* col_scale, const zero_rows* dw, int32_t flags, void* ws, size_t ws_bytes,
                    hipStream_t stream);

/*
 * The boundary between two blocks: the norm after a block, its gate, the
 * residual scale, the residual add, and the norm before the next block, in
 * one pass. With n(z) = z / sqrt(mean(z^2) + eps) over a row, per row t:
 *   yn    = n(y) when w_post is given, else y
 *   x_out = x + residual_scale * gate[t / gate_rows] * (w_post * yn)
 *   xn    = n(x_out)                       of x_out as stored, in its type
 *   h     = w_pre * xn
 * Absent operands (data NULL): y (then x_out is x itself and is not written),
 * w_post (no norm after the block), gate (ones), w_pre (no norm before the
 * next block). rstd_post and rstd_pre (fp32, one per row) are the reciprocal
 * roots; ckpt_post and ckpt_pre the act8 buffers of yn and xn. Two outputs at
 * one address are refused.
 *
 * Rounding. Arithmetic is fp32, the mean of squares and its root fp64 from
 * sums of squares in fp32 (at most two waves each). x_out and h are rounded to
 * their own type once, at the end; the fp32 steps before that (the row's sum,
 * the quotient, the products of residual_scale, gate and weight, the sum with
 * x) are together within 56 * 2^-24 of the sum of the terms' magnitudes. The
 * 8-bit codes are those of the quotient by the root in two fp32 parts, not of
 * its fp32 rounding: an fp32 quotient that ends in 16 zero bits, as codes and
 * the middles between them do, is moved one fp32 step towards the exact one, in
 * x_out and h as in the codes and whether or not a checkpoint is written.
 *
 * Range. Where a row's squares pass the range of fp32 (some |z| of 2^64 or
 * more) its reciprocal root is 0, and so is its n(z) (NaN where z is infinite).
 * With eps 0, a row whose squares all vanish in fp32 (every |z| below 2^-75) has
 * an infinite root, so that n(z) is infinite, or NaN where z is 0. A NaN in a
 * row makes all of its n(z) NaN.
 */
typedef struct zero_block_norm_args {
    int64_t rows;          /* 0 <= rows < 2^31 */
    int64_t cols;          /* 0 <= cols <= ZERO_BLOCK_NORM_MAX_COLS */
    int64_t gate_rows;     /* rows in a row that share one row of gate, >= 1 with a gate */
    double residual_scale; /* finite; rounded to fp32 */
    double eps;            /* finite, >= 0; rounded to fp32 */
    zero_rows x;           /* residual stream, bf16 or fp32 */
    zero_rows y;           /* block output, bf16 */
    zero_rows w_post;      /* cols, bf16 or fp32 */
    zero_rows gate;        /* ceil(rows / gate_rows) x cols, bf16 or fp32; needs y */
    zero_rows w_pre;       /* cols, bf16 or fp32 */
    zero_rows x_out;       /* residual stream, the type of x; written with y, may be x itself */
    zero_rows h;           /* bf16, written with w_pre */
    float* rstd_post;      /* rows, or NULL */
    float* rstd_pre;       /* rows, or NULL */
    void* ckpt_post;       /* act8 buffer, or NULL */
    void* ckpt_pre;        /* act8 buffer, or NULL; needs w_pre */
    int32_t format;        /* of both act8 buffers */
    int32_t reserved;      /* must be 0 */
} zero_block_norm_args;

int zero_block_norm(const zero_block_norm_args* args, hipStream_t stream);

/*
 * zero_block_norm_grad -- the gradients of zero_block_norm. yn and xn come
 * from act8 buffers, or (ckpt_* NULL) from y * rstd_post and x_out *
 * rstd_pre. With g = residual_scale * gate, per row:
 *   d    = dx_out + rstd_pre * (w_pre * dh - xn * mean(w_pre * dh * xn))
 *   dx   = d                       (the gradient of x)
 *   dy   = rstd_post * (w_post * g * d - yn * mean(w_post * g * d * yn)),
 *          or g * d without w_post
 * and, summed over rows in fp32 in an order that depends only on the sizes:
 *   dw_pre = sum dh * xn,   dw_post = sum g * d * yn,
 *   dgate[j] = sum over the rows of gate row j of residual_scale * d * w_post * yn.
 * Arithmetic is fp32, and d enters dy and the sums as it is before the rounding
 * to dx's type; each result is rounded to its own type once, at the end. Before
 * that dx is within 112 * 2^-24 of the sum of its terms' magnitudes, dy within
 * 224 * 2^-24, a sum over rows within (rows + 288) * 2^-24.
 * Absent (data NULL): dh (no norm before the next block; then dx_out is
 * given), dx_out (zeros), dy and what only it needs (no block output: dx
 * alone), and each of dw_pre, dw_post and dgate that is not wanted. dx may be
 * dx_out itself. Two outputs at one address are refused: where w_pre and w_post
 * are one vector, its two gradients still need a buffer each. rows == 0 writes
 * zeros to dw_pre and dw_post, or adds them.
 */
typedef struct zero_block_norm_grad_args {
    int64_t rows;
    int64_t cols;
    int64_t gate_rows;
    double residual_scale;
    zero_rows dh;     /* gradient of h, bf16 */
    zero_rows dx_out; /* gradient of x_out from what follows, the type of dx */
    zero_rows w_post; /* as in zero_block_norm */
    zero_rows gate;
    zero_rows w_pre;           /* with dh */
    zero_rows x_out;           /* when dh is given and ckpt_pre is NULL: the type of dx */
    zero_rows y;               /* when yn is needed and ckpt_post is NULL: bf16 */
    const void* ckpt_pre;      /* act8 buffer of xn, or NULL */
    const void* ckpt_post;     /* act8 buffer of yn, or NULL */
    const float* rstd_pre;     /* rows, with dh */
    const float* rstd_post;    /* rows, with w_post */
    zero_rows dx;              /* the gradient of x, bf16 or fp32 */
    zero_rows dy;              /* bf16 */
    zero_rows dw_pre;          /* cols, bf16 or fp32 */
    zero_rows dw_post;         /* cols, bf16 or fp32; needs w_post */
    zero_rows dgate;           /* ceil(rows / gate_rows) x cols, bf16 or fp32; needs gate */
    int32_t format;            /* of the act8 buffers */
    int32_t flags;             /* ZERO_GRAD_ACCUMULATE: dw_pre, dw_post and dgate are fp32 and added to */
} zero_block_norm_grad_args;

/* Workspace size of zero_block_norm_grad (partial column sums); gate_rows 0
 * without a gate; 0 on invalid sizes. */
size_t zero_block_norm_grad_workspace_bytes(int64_t rows, int64_t cols, int64_t gate_rows);

/* ws: device workspace of that size, 16-byte aligned (NULL if it is 0),
 * contents irrelevant on entry and not kept; two calls that share one must not
 * run concurrently. The plan that a step keeps in any part of it is forgotten,
 * as by zero_workspace_forget. */
int zero_block_norm_grad(const zero_block_norm_grad_args* args, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * zero_layer_norm -- the residual add and the layer norm before a block, in
 * one pass. Per row of cols values:
 *   x_out = x + y                       (stored in x's type)
 *   mean  = sum(x_out) / cols           of x_out as stored
 *   rstd  = 1 / sqrt(sum((x_out - mean)^2) / cols + eps)
 *   xn    = (x_out - mean) * rstd
 *   h     = w * xn + b
 * Absent operands (data NULL): y (then x_out is x itself and is not written),
 * w (ones), b (zeros). mean and rstd (fp32, one per row) are optional;
 * ckpt_xn is the act8 buffer of xn, from which zero_layer_norm_grad can take
 * it, and ckpt_h that of h before its rounding to bf16, from which
 * zero_act8_wgrad and zero_block_ffn_grad take the gradients of what h goes
 * into. x_out may be x itself; two outputs at one address are refused.
 *
 * Rounding. Arithmetic is fp32. The mean is taken in two steps, a first one and
 * the mean difference to it, and the squares about it, so that rows far from 0
 * keep their variance. With f = 1 + 22 * 2^-24 * mean(|x_out|) * rstd, xn is
 * within 100 * 2^-24 * (|xn| + f), rstd within 100 * 2^-24 * f of itself, mean
 * within 84 * 2^-24 * mean(|x_out|); each result is then rounded to its own type
 * once.
 *
 * Range. A row with an inf or NaN has NaN in its mean, rstd, xn and h, and so
 * may one whose sum passes fp32's range; one whose squares pass it may have rstd
 * 0. With eps 0 a row of equal values has a large or infinite rstd, and anything
 * in xn.
 */
typedef struct zero_layer_norm_args {
    int64_t rows;     /* 0 <= rows < 2^31 */
    int64_t cols;     /* 0 <= cols <= ZERO_BLOCK_NORM_MAX_COLS */
    double eps;       /* finite, >= 0; rounded to fp32 */
    zero_rows x;      /* residual stream, bf16 or fp32 */
    zero_rows y;      /* what is added to it, bf16 */
    zero_rows w;      /* cols, bf16 or fp32 */
    zero_rows b;      /* cols, bf16 or fp32 */
    zero_rows x_out;  /* the type of x; written with y, may be x itself */
    zero_rows h;      /* bf16 */
    float* mean;      /* rows, or NULL */
    float* rstd;      /* rows, or NULL */
    void* ckpt_xn;    /* act8 buffer, or NULL */
    void* ckpt_h;     /* act8 buffer, or NULL */
    int32_t format;   /* of both act8 buffers */
    int32_t reserved; /* must be 0 */
} zero_layer_norm_args;

int zero_layer_norm(const zero_layer_norm_args* args, hipStream_t stream);

/*
 * zero_layer_norm_grad -- the gradients of zero_layer_norm. xn comes from an
 * act8 buffer, or (ckpt_xn NULL) from x_out, mean and rstd. With v = w * dh,
 * per row:
 *   dx = dx_out + rstd * (v - mean(v) - xn * mean(v * xn))
 * which is the gradient of both x and y; dy is the same values in bf16, for a
 * block whose output y is bf16 beside an fp32 residual stream. Summed over rows
 * in fp32 in an order that depends only on the sizes:
 *   dw = sum dh * xn,   db = sum dh.
 * Absent (data NULL): dx_out (zeros), w (ones), and each of dy, dw and db that
 * is not wanted. dx may be dx_out itself. Two outputs at one address are
 * refused. rows == 0 writes zeros to dw and db, or adds them.
 */
typedef struct zero_layer_norm_grad_args {
    int64_t rows;
    int64_t cols;
    zero_rows dh;        /* gradient of h, bf16 */
    zero_rows dx_out;    /* gradient of x_out from what follows, the type of dx */
    zero_rows w;         /* as in zero_layer_norm */
    zero_rows x_out;     /* when ckpt_xn is NULL: the type of dx */
    const float* mean;   /* rows, when ckpt_xn is NULL */
    const float* rstd;   /* rows */
    const void* ckpt_xn; /* act8 buffer of xn, or NULL */
    zero_rows dx;        /* bf16 or fp32 */
    zero_rows dy;        /* bf16 */
    zero_rows dw;        /* cols, bf16 or fp32 */
    zero_rows db;        /* cols, bf16 or fp32 */
    int32_t format;      /* of the act8 buffer */
    int32_t flags;       /* ZERO_GRAD_ACCUMULATE: dw and db are fp32 and added to */
} zero_layer_norm_grad_args;

/* Workspace size of zero_layer_norm_grad (partial column sums, and for rows of
 * more than 8192 columns two values a row), the same whichever of dw and db are
 * wanted; 0 on invalid sizes. */
size_t zero_layer_norm_grad_workspace_bytes(int64_t rows, int64_t cols);

/* ws: as in zero_block_norm_grad. */
int zero_layer_norm_grad(const zero_layer_norm_grad_args* args, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * The gated feed-forward block of a layer, from its normalised input to what
 * goes into its down projection:
 *   gate = h * w_gate^T,   up = h * w_up^T,   a = act(gate) * up
 * with h rows x cols and the two weights hidden x cols, all bf16.
 */
#define ZERO_FFN_SILU 1      /* g / (1 + exp(-g)) */
#define ZERO_FFN_GELU 2      /* g * (1 + erf(g / sqrt(2))) / 2 */
#define ZERO_FFN_GELU_TANH 3 /* g * (1 + tanh(sqrt(2 / pi) * (g + 0.044715 g^3))) / 2 */

/*
 * zero_block_ffn -- both projections, the activation and the product in one
 * pass. gate and up are summed in fp32 in an order that depends only on the
 * sizes, on which operands' rows lie on 16 bytes and on whether one's lie more
 * than 2^22 elements apart, and a is made from these sums: within
 * (32 + 4 |gate|) 2^-24 |gate * up| of the formula of them. (Where act(gate) is
 * far smaller than gate that is more than bf16's half step: of ZERO_FFN_GELU from
 * gate = -5 down; at -8, where it is -5e-15, 1% of it.) For the backward pass the
 * sums can be kept as bf16 rows (gate, up) or as act8 buffers (ckpt_gate,
 * ckpt_up), or neither; each result is rounded to its own type once. cols == 0:
 * the sums are 0.
 * rows < 2^31, cols and hidden <= 2^30, rows times either (rounded up to 32)
 * < 2^36, and fewer than 2^20 tiles of 128 x 128 of rows x hidden, rows x cols
 * and hidden x cols. Two outputs at one address are refused.
 */
typedef struct zero_block_ffn_args {
    int64_t rows;
    int64_t cols;
    int64_t hidden;
    zero_rows h;      /* rows x cols, bf16 */
    zero_rows w_gate; /* hidden x cols, bf16 */
    zero_rows w_up;   /* hidden x cols, bf16 */
    zero_rows a;      /* rows x hidden, bf16 */
    zero_rows gate;   /* rows x hidden, bf16, or absent */
    zero_rows up;     /* rows x hidden, bf16, or absent */
    void* ckpt_gate;  /* act8 buffer of rows x hidden, or NULL */
    void* ckpt_up;    /* act8 buffer of rows x hidden, or NULL */
    int32_t format;   /* of both act8 buffers */
    int32_t act;      /* ZERO_FFN_* */
} zero_block_ffn_args;

/* Workspace size of zero_block_ffn: partial sums where few rows leave the
 * chip's units to the summed columns (often none), and where cols is not a
 * multiple of 8 and rows are many, aligned copies of h and the weights. 0 on
 * invalid sizes. */
size_t zero_block_ffn_workspace_bytes(int64_t rows, int64_t cols, int64_t hidden);

/* ws: as in zero_act8_wgrad. */
int zero_block_ffn(const zero_block_ffn_args* args, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * zero_block_ffn_grad -- the gradients of zero_block_ffn from da, the gradient
 * of a, and the saved gate and up: bf16 rows, or act8 buffers.
 *   dgate = da * up * act'(gate),   dup = da * act(gate)        (bf16)
 *   dh      = dgate * w_gate + dup * w_up
 *   dw_gate (+)= dgate^T * h,   dw_up (+)= dup^T * h
 * dgate and dup are the nearest bf16 values of the formulas (computed in fp32,
 * and in fp64 where that leaves the rounding open); dh and the weight gradients
 * are those of dgate and dup as stored, summed in fp32 in an order that depends
 * only on the sizes, on which of them are wanted and on how the operands lie
 * (which rows lie on 16 bytes, whether dgate and dup have one stride and w_gate
 * and w_up one, whether a stride is over 2^22 elements), each rounded to its own
 * type once.
 * The block's input comes as bf16 rows h, or as the act8 buffer ckpt_h whose
 * decoded columns are multiplied with col_scale (cols values, bf16 or fp32;
 * absent: ones), as in zero_act8_wgrad. ckpt_a, if given, is written: the act8
 * buffer of act(gate) * up, for the weight gradient of the down projection
 * without a kept from the forward pass.
 * Absent (data NULL): dh with w_gate and w_up, and each of dw_gate and dw_up
 * that is not wanted; without both, h, ckpt_h and col_scale. Two outputs at one
 * address are refused. rows == 0 writes zeros to dw_gate and dw_up, or adds
 * them; hidden == 0 writes zeros to dh. Sizes as in zero_block_ffn.
 */
typedef struct zero_block_ffn_grad_args {
    int64_t rows;
    int64_t cols;
    int64_t hidden;
    zero_rows da;          /* rows x hidden, bf16 */
    zero_rows gate;        /* rows x hidden, bf16, when ckpt_gate is NULL */
    zero_rows up;          /* rows x hidden, bf16, when ckpt_up is NULL */
    const void* ckpt_gate; /* act8 buffers, both or neither */
    const void* ckpt_up;
    zero_rows w_gate;      /* hidden x cols, bf16, with dh */
    zero_rows w_up;        /* hidden x cols, bf16, with dh */
    zero_rows h;           /* rows x cols, bf16, when a weight gradient is wanted and ckpt_h is NULL */
    const void* ckpt_h;    /* act8 buffer of rows x cols, or NULL */
    zero_rows col_scale;   /* cols, bf16 or fp32, with ckpt_h */
    zero_rows dgate;       /* rows x hidden, bf16, written */
    zero_rows dup;         /* rows x hidden, bf16, written */
    zero_rows dh;          /* rows x cols, bf16 */
    zero_rows dw_gate;     /* hidden x cols, bf16 or fp32 */
    zero_rows dw_up;       /* hidden x cols, bf16 or fp32 */
    void* ckpt_a;          /* act8 buffer of rows x hidden, written, or NULL */
    int32_t format;        /* of all act8 buffers */
    int32_t act;           /* ZERO_FFN_* */
    int32_t flags;         /* ZERO_GRAD_ACCUMULATE: dw_gate and dw_up are fp32 and added to */
    int32_t reserved;      /* must be 0 */
} zero_block_ffn_grad_args;

/* Workspace size of zero_block_ffn_grad, whichever of its gradients are wanted
 * and however h comes: partial sums, and where cols or hidden is not a multiple
 * of 8 and rows are many, aligned copies of a product's operands. 0 on invalid
 * sizes. */
size_t zero_block_ffn_grad_workspace_bytes(int64_t rows, int64_t cols, int64_t hidden);

/* ws: as in zero_act8_wgrad. */
int zero_block_ffn_grad(const zero_block_ffn_grad_args* args, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * zero_workspace_forget -- drop the host-side record that `ws` holds the
 * tensor table of an earlier zero_step, zero_step_amp, zero_bucket_reduce,
 * zero_step_accumulated or zero_offload_step call. Call it before freeing or
 * repurposing such a workspace; the next zero_step on it then rewrites the
 * table. (A workspace whose table was overwritten without this call is
 * detected on the device: zero_result.status = ZERO_ERR_STALE_WORKSPACE and
 * nothing is written.) Host only; launches nothing.
 */
int zero_workspace_forget(const void* ws);

/* Human-readable text of a status code (static storage). */
const char* zero_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_STEP_H */
