/*
 * ob_adam.h -- C ABI of the 1-bit Adam step on one AMD MI355X (gfx950).
 *
 * The library (libobadam.so) runs every step of the optimizer in hand-written HIP kernels.  All data
 * pointers are DEVICE pointers owned by the caller; every call is asynchronous on the caller's
 * `stream` and returns once its kernels are enqueued.  No torch types cross this boundary.
 *
 * Pages cited (title and section):
 *   [P1] "1bit Adam" tutorial (intelliparadigm.com article 2150495): sec. 2.1 quantization and error
 *        compensation, sec. 2.2 momentum on the compressed gradient, sec. 3.1 per-parameter state,
 *        sec. 3.2 compress routine (clip, NaN check, int8 signs), sec. 4.2 packing into one buffer.
 *   [P2] "DeepSpeed Communication Compression and Hiding": section "baseline: why Adam is hard to
 *        compress" (Adam moments), section "1-bit Adam: warmup, frozen variance, error feedback"
 *        (the two-phase step and compressed_allreduce), section "0/1 Adam" (variance refresh),
 *        section "1-bit LAMB: also protect the layer-wise trust ratio".
 *   [P3] gradient-compression survey (bmjup.com post 14450): Q&A on the memory cost of error
 *        feedback (the error term kept in a 16-bit format such as FP16).
 *
 * Definitions used by every call
 *   - Elements are a flat index 0..n-1 over one contiguous buffer per state array (the parameters
 *     packed into one block, [P1] sec. 4.2).  n may exceed 2^32.
 *   - A plan splits 0..n-1 into K chunks; every chunk has its own fp32 scale.  Chunk c spans
 *     [o_c, o_{c+1}).  Interior chunk boundaries must be multiples of 64.
 *   - sign(x) = +1 iff x >= 0.0f (so +0 and -0 give +1, NaN gives -1).
 *   - Packed signs: bit j of uint32 word w is 1 iff sign(x[32w + j]) = +1; ceil(n/32) words; bits
 *     for indices >= n are 0.  The packing ignores chunk boundaries.
 *   - scale_c = ||x_c||_2 / sqrt(n_c), with ||x_c||^2 accumulated in double and sqrt(S/n_c) taken in
 *     double, then rounded to fp32.  g_hat = +scale_c or -scale_c by the sign.
 *
 * Alignment: fp32 state and fp32 gradient pointers 16 bytes; bf16 gradient and 16-bit error buffer
 * 8 bytes; words, scales and int8 signs 4 bytes; the non-finite counter 8 bytes.  (torch allocations
 * are 256-byte aligned.)
 *
 * Errors: arguments are validated on the host before anything is enqueued, and a failed check
 * returns a status without touching the GPU: OB_ERR_ARG (null required pointer, bad size, bad chunk
 * table, W < 1, n differs from the plan), OB_ERR_ALIGN (pointer or chunk-boundary alignment),
 * OB_ERR_DTYPE (unknown dtype).  A failed launch returns OB_ERR_HIP; faults during execution surface
 * at the caller's next synchronisation.  OB_ERR_OOM: an allocation failed (a plan's device memory, or
 * host memory for its tables or for timing records).  n = 0 is a no-op.
 * No C++ exception crosses the ABI and nothing aborts.  NaN and Inf propagate per IEEE.
 *
 * Threads and streams: distinct plans are independent.  A plan holds a small workspace (one double
 * per work block), so one plan must not be used by two calls that may run concurrently on the GPU;
 * calls on one stream are ordered and therefore safe.
 */
#ifndef OB_ADAM_H
#define OB_ADAM_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    OB_OK = 0,
    OB_ERR_ARG = 1,
    OB_ERR_ALIGN = 2,
    OB_ERR_DTYPE = 3,
    OB_ERR_HIP = 4,
    OB_ERR_OOM = 5,
    OB_ERR_SIZE = 6     /* ob_adam_compress_step_noalloc: the problem needs more than its static buffer */
} ob_status;

/* Element types.  Gradients and packed inputs: OB_F32 or OB_BF16.  The error buffer of the compressed
 * step may also be OB_F16 (IEEE binary16). */
typedef enum { OB_F32 = 0, OB_BF16 = 1, OB_F16 = 2 } ob_dtype;

/* Error feedback rule: PLAIN replaces the error with x - g_hat ([P2] 1-bit Adam pseudo-code);
 * EMA keeps ef_beta*err + (1-ef_beta)*(x - g_hat) ([P1] sec. 2.1). */
typedef enum { OB_EF_PLAIN = 0, OB_EF_EMA = 1 } ob_ef_mode;

/* How a new error is stored in a 16-bit error buffer: to nearest, ties to even, or stochastically
 * (round up with probability equal to the fraction of the quantum; 16 random bits per element from
 * Philox4x32-10 at counter (i >> 2, step) with key sr_seed; see ob_adam_compress_step). */
typedef enum { OB_ROUND_NEAREST = 0, OB_ROUND_STOCHASTIC = 1 } ob_rounding;

/* Hyperparameters, fp32 as in the per-parameter state of [P1] sec. 3.1. */
typedef struct {
    float lr;
    float beta1;
    float beta2;            /* dense step only */
    float eps;
    float clip;             /* compressed step: clamp g to [-clip, clip] before adding the error
                               ([P1] sec. 3.2); <= 0 disables; NaN passes through */
    int32_t ef_mode;        /* ob_ef_mode */
    float ef_beta;          /* EMA coefficient ([P1] sec. 2.1 uses beta1 = 0.9) */
    int32_t bias_correction;/* dense step only: divide m, v by 1 - beta^step (textbook Adam);
                               the pages' step has none, so 0 is the default */
    int64_t step;           /* dense step with bias_correction: t >= 1; compressed step with
                               stochastic rounding: the random stream (use a new value every step) */
    int32_t err_rounding;   /* ob_rounding; compressed steps with a 16-bit error buffer only */
    int32_t reserved;       /* 0 */
    uint64_t sr_seed;       /* stochastic rounding: the generator's key, with step */
} ob_hparams;

typedef struct ob_plan_s* ob_plan;

/* Create a plan for n elements on the current HIP device.
 *   chunk_offsets == NULL: uniform chunks of chunk_size elements (the last one ends at n);
 *                          chunk_size > 0 and, when n > chunk_size, a multiple of 64.
 *   chunk_offsets != NULL: n_chunks + 1 host int64 offsets, 0 = o_0 < o_1 < ... < o_K = n, interior
 *                          offsets multiples of 64 (one chunk per parameter tensor).
 * The plan owns its device tables and workspace (hipMalloc here, hipFree in ob_plan_destroy);
 * *out is set to NULL on failure. */
ob_status ob_plan_create(int64_t n, int64_t chunk_size, const int64_t* chunk_offsets,
                         int64_t n_chunks, ob_plan* out);
ob_status ob_plan_destroy(ob_plan plan);
int64_t ob_plan_num_elements(ob_plan plan);   /* -1 for a NULL plan */
int64_t ob_plan_num_chunks(ob_plan plan);     /* -1 for a NULL plan */
int64_t ob_plan_num_blocks(ob_plan plan);     /* work blocks = grid size of the per-element kernels */
int64_t ob_plan_block_elems(ob_plan plan);    /* elements per work block (except chunk tails) */
/* Chunk groups of the compressed step (ob_adam_compress_step, ob_adam_worker_compress): the step runs
 * its two kernels group by group, each group being consecutive chunks whose bytes read by the first
 * kernel (g and err) stay within a budget sized to the GPU's last-level cache (320 MB; the environment
 * variable OB_GROUP_BYTES, read when the plan is created, overrides it and 0 turns grouping off), so
 * that the second kernel re-reads them from that cache.  A chunk above the budget is a group of its
 * own; plans whose chunks need a per-chunk sums launch (more than 4096 first-kernel blocks in a chunk)
 * are one group, and so is 1-bit LAMB (lamb != 0: ob_lamb_compress_step, whose first kernel also reads
 * p).  Returns the number of groups, i.e. the launches of each of the two kernels per step; -1 for a
 * NULL plan or an invalid dtype. */
int64_t ob_plan_num_groups(ob_plan plan, ob_dtype g_dtype, ob_dtype err_dtype, int32_t lamb);

/* Dense Adam step ([P2] baseline section; the step used before freeze_step in [P2] 1-bit Adam and for
 * the variance refresh of [P2] 0/1 Adam):
 *   m = beta1*m + (1-beta1)*g;  v = beta2*v + (1-beta2)*g^2;
 *   p -= lr * mh / (sqrt(vh) + eps)   with mh = m, vh = v, or m/(1-beta1^t), v/(1-beta2^t) when
 *   hp->bias_correction.  The error buffer is not touched.
 * g: n elements of `g_dtype` (read only); m, v, p: fp32[n], updated in place. */
ob_status ob_adam_warmup_step(ob_plan plan, const void* g, ob_dtype g_dtype, float* m, float* v,
                              float* p, const ob_hparams* hp, hipStream_t stream);

/* Compressed step ([P2] 1-bit Adam, compressed branch with W = 1; [P1] sec. 2.1-2.2, 3.2):
 *   g' = clip(widen(g));  x = g' + err (fp32);  words = pack(sign(x));  scales_c per chunk;
 *   g_hat = +-scale_c;  err = x - g_hat (PLAIN) or ef_beta*err + (1-ef_beta)*(x - g_hat) (EMA);
 *   m = beta1*m + (1-beta1)*g_hat;  p -= lr * m / (sqrt(v) + eps)  (v frozen, read only).
 * Runs two kernels: a per-chunk sum of squares, then one fused streaming pass, one pair of launches
 * per chunk group (ob_plan_num_groups; the results do not depend on the grouping).
 * g: n elements (read only); err: n elements of err_dtype, in place; m, p: fp32[n] in place;
 * v: fp32[n] read only; words_out: uint32[ceil(n/32)]; scales_out: fp32[K];
 * err_dtype ([P3] Q&A on error-feedback memory): OB_F32, or OB_BF16 / OB_F16 -- the stored error is
 *   widened exactly when read, and the new error, computed in fp32 as above, is rounded to the format
 *   (nearest, ties to even; beyond the largest finite value, +-Inf) when stored.  With
 *   hp->err_rounding = OB_ROUND_STOCHASTIC it is stored as lo or hi = lo + q (lo its truncation toward
 *   zero, q the format's quantum there), hi iff r*q < (|e| - lo)*65536 with r the element's 16
 *   random bits: the high half of output word i & 3 of Philox4x32-10 (Salmon et al., SC 2011) at the
 *   128-bit counter (i >> 2, hp->step) under the 64-bit key hp->sr_seed (32-bit words, low first).
 *   OB_ERR_ARG for an fp32 error buffer;
 * signs_out (optional, NULL = off): int8[n] of +1/-1 ([P1] sec. 3.2);
 * nonfinite_out (optional, NULL = off): device uint64 counter to which the number of non-finite
 * STORED new error elements is added ([P1] sec. 3.2 NaN check; the caller zeroes it), so an fp16
 * overflow is counted.
 * Outputs must not alias inputs. */
ob_status ob_adam_compress_step(ob_plan plan, const void* g, ob_dtype g_dtype, void* err, ob_dtype err_dtype,
                                float* m, const float* v, float* p, uint32_t* words_out, float* scales_out,
                                int8_t* signs_out, uint64_t* nonfinite_out, const ob_hparams* hp,
                                hipStream_t stream);

/* ---- 1-bit LAMB ([P2] section "1-bit LAMB: also protect the layer-wise trust ratio") ----
 * LAMB scales the Adam direction of each layer by the trust ratio r = ||w|| / ||u|| and updates
 * w -= lr * r * u; in 1-bit LAMB the direction is built from the reconstructed (compressed) gradient.
 * Here a layer is a chunk of the plan (create the plan with one chunk per parameter tensor):
 *   u_i = mh_i / (sqrt(vh_i) + eps)      (double, not stored; mh = m, vh = v unless bias-corrected)
 *   r_c = ||p_c|| / ||u_c||               (p before the update; sums of squares in double, rounded
 *                                         once to fp32; r_c = 1 when either norm is 0, NaN/Inf propagate)
 *   p_i -= lr * r_c * u_i                 (double, rounded once)
 * No weight decay and no clamp of r.  ratios_out: fp32[K], the ratio each layer used.
 * Each call runs 4 kernels (compressed) or 3 (dense): the passes below, one block per layer for the
 * ratios, and the update. */

/* Compressed 1-bit LAMB step: exactly ob_adam_compress_step's compensate / quantize / pack / error /
 * momentum (same arguments and outputs), then the trust ratio on the new m and the frozen v, and the
 * update of p. */
ob_status ob_lamb_compress_step(ob_plan plan, const void* g, ob_dtype g_dtype, void* err, ob_dtype err_dtype,
                                float* m, const float* v, float* p, uint32_t* words_out, float* scales_out,
                                float* ratios_out, int8_t* signs_out, uint64_t* nonfinite_out,
                                const ob_hparams* hp, hipStream_t stream);

/* Dense LAMB step (the warmup of 1-bit LAMB): m and v as in ob_adam_warmup_step (bias correction by
 * hp->bias_correction / hp->step), then the trust ratio and the update of p. */
ob_status ob_lamb_warmup_step(ob_plan plan, const void* g, ob_dtype g_dtype, float* m, float* v, float* p,
                              float* ratios_out, const ob_hparams* hp, hipStream_t stream);

/* Server half of compressed_allreduce ([P2] 1-bit Adam) on this GPU's share of n elements:
 *   avg_i = (sum_{w<W} (bit_w(i) ? s_{w,c} : -s_{w,c})) / W, summed in double in ascending w and
 *           rounded once to fp32;
 *   x = avg + server_err;  words_out = pack(sign(x));  scales_out per chunk of x;
 *   server_err = x - g_hat (plain error feedback kept by the server).
 * worker_words: W rows of ceil(n/32) uint32 (row w starts at w*ceil(n/32)); pad bits are ignored;
 * worker_scales: W rows of K fp32; server_err: fp32[n] in place; words_out: uint32[ceil(n/32)];
 * scales_out: fp32[K].  1 <= W <= 1024. */
ob_status ob_server_reduce(ob_plan plan, int32_t W, const uint32_t* worker_words,
                           const float* worker_scales, float* server_err, uint32_t* words_out,
                           float* scales_out, hipStream_t stream);

/* ---- the worker's compressed step split at the exchange (more than one worker; [P2] "1-bit Adam:
 * warmup, frozen variance, error feedback", compressed branch: the quantize line runs before
 * compressed_allreduce, the dequantize, momentum and update lines after it) ----
 * ob_adam_worker_compress: ob_adam_compress_step up to the packed signs, scales and error: the error
 *   uses the worker's own g_hat; m, v and p are not touched.  Arguments, layout and errors as there.
 * ob_adam_worker_update: g_hat_i = bit(i) ? scales[c] : -scales[c] from the exchanged words
 *   (uint32[ceil(n/32)], pad bits ignored) and scales (fp32[K]), e.g. the output of ob_server_reduce
 *   gathered back; then m = beta1*m + (1-beta1)*g_hat and p -= lr * m / (sqrt(v) + eps), m and p in
 *   place, v read only (hp: lr, beta1, eps).
 * With one worker and a zero server error the exchange returns the worker's own words and scales, and
 * the two calls give bit for bit the results of ob_adam_compress_step.
 * ob_lamb_worker_update ([P2] "1-bit LAMB"): the same g_hat and m, then the layer-wise trust ratio on
 *   the reconstructed direction and the update, as in ob_lamb_compress_step (ratios_out: fp32[K]).
 *   Its sums of p^2 and u^2 are grouped by other blocks than the fused step's, so a ratio may differ
 *   from that step's in the last bit. */
ob_status ob_adam_worker_compress(ob_plan plan, const void* g, ob_dtype g_dtype, void* err, ob_dtype err_dtype,
                                  uint32_t* words_out, float* scales_out, int8_t* signs_out,
                                  uint64_t* nonfinite_out, const ob_hparams* hp, hipStream_t stream);
ob_status ob_adam_worker_update(ob_plan plan, const uint32_t* words, const float* scales, float* m,
                                const float* v, float* p, const ob_hparams* hp, hipStream_t stream);
ob_status ob_lamb_worker_update(ob_plan plan, const uint32_t* words, const float* scales, float* m,
                                const float* v, float* p, float* ratios_out, const ob_hparams* hp,
                                hipStream_t stream);

/* Pack signs of x (OB_F32 or OB_BF16, n elements) into ceil(n/32) words ([P2] one_bit_quantize, sign part).
 * n at most (2^31 - 1) * 16384 (one block per 16384 elements); OB_ERR_ARG beyond. */
ob_status ob_pack(const void* x, ob_dtype x_dtype, int64_t n, uint32_t* words_out, hipStream_t stream);

/* Unpack + dequantize ([P2] dequantize): out_i = bit(i) ? s_c : -s_c, s_c = scales[c] for the plan's
 * chunk c of i; with scales == NULL, s = 1 and plan may be NULL.  With scales, plan is required and n
 * must equal the plan's n.  out: fp32[n].  Without a plan's tables (scales == NULL) n is at most
 * (2^31 - 1) * 16384, as for ob_pack. */
ob_status ob_unpack(ob_plan plan, const uint32_t* words, int64_t n, const float* scales, float* out,
                    hipStream_t stream);

const char* ob_status_str(ob_status s);

/* ---- the compressed step without any allocation ----
 * For callers that cannot allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  ob_adam_compress_step for uniform chunks of chunk_size elements
 * (the last chunk ends at n; chunk_size > 0 and, when n > chunk_size, a multiple of 64 -- the chunking
 * of ob_plan_create with chunk_offsets == NULL), without a plan.  Arguments, layouts, outputs and
 * errors otherwise as ob_adam_compress_step; the results are bit for bit those of
 * ob_adam_compress_step with a plan of the same n and chunk_size.
 * It calls no hipMalloc, hipFree or other allocating routine.  Its block tables and per-block sums of
 * squares live in a static device buffer of OB_NOALLOC_SCRATCH_BYTES that the library holds on every
 * GPU it runs on until the process ends; the first call on a device looks up that device's copy.
 * Each call rewrites the tables it needs (one small kernel ahead of the two passes), so consecutive
 * calls may change n and chunk_size.  The two passes run by chunk groups as in ob_adam_compress_step
 * (groups of equal numbers of chunks within the same budget, OB_GROUP_BYTES read on every call).  All calls on one GPU share its buffer: calls that may overlap on
 * one GPU (other streams, other host threads) race and must not be issued; calls on one stream are
 * ordered.  Space needed: 24 bytes per first-pass block, 16 per 4096-element block of the fused pass,
 * 16 per chunk (plus 12 per chunk for chunks of more than 4096 first-pass blocks), each region rounded
 * up to 256 bytes -- with chunks of 2^24 elements about 1.3e10 elements fit.  A larger problem returns
 * OB_ERR_SIZE before any HIP call.  No diagnostics and no timing (those belong to a plan). */
#define OB_NOALLOC_SCRATCH_BYTES (64ll << 20)
ob_status ob_adam_compress_step_noalloc(int64_t n, int64_t chunk_size, const void* g, ob_dtype g_dtype,
                                        void* err, ob_dtype err_dtype, float* m, const float* v, float* p,
                                        uint32_t* words_out, float* scales_out, int8_t* signs_out,
                                        uint64_t* nonfinite_out, const ob_hparams* hp, hipStream_t stream);

/* ---- kernel timing (measurement support) ----
 * With timing on, every call made with this plan records hipEvents around each kernel it launches, on
 * the call's stream: a pair per launch, except that the launches a compressed step makes one after the
 * other for its chunk groups share them (each starts at the event that ended the one before), one
 * event per launch.  ob_plan_read_timing waits for the recorded events and returns the summed
 * milliseconds and launch count of one kernel kind since timing was switched on.  The events are
 * created with hipEventDisableSystemFence: they measure time only and order no memory. */
typedef enum {
    OB_KERNEL_CHUNK_SUMSQ = 0,     /* compressed step (Adam or LAMB), pass 1 */
    OB_KERNEL_COMPRESS = 1,        /* compressed step (Adam or LAMB), pass 2 (fused streaming pass) */
    OB_KERNEL_DENSE = 2,           /* dense step (Adam, or the moments pass of dense LAMB) */
    OB_KERNEL_SERVER_SUMSQ = 3,    /* server reduce, pass 1 */
    OB_KERNEL_SERVER_APPLY = 4,    /* server reduce, pass 2 */
    OB_KERNEL_UNPACK = 5,
    OB_KERNEL_TRUST_RATIO = 6,     /* LAMB: per-layer ratios */
    OB_KERNEL_LAMB_APPLY = 7,      /* LAMB: parameter update */
    OB_KERNEL_DIAG = 8,            /* diagnostics: per-chunk totals */
    OB_KERNEL_SCALE = 9,           /* per-chunk sums of squares formed before pass 2 (plans with a
                                      chunk of more than 4096 pass-1 blocks) */
    OB_KERNEL_WORKER_COMPRESS = 10,/* worker compress, pass 2 (pass 1 is OB_KERNEL_CHUNK_SUMSQ) */
    OB_KERNEL_WORKER_UPDATE = 11,  /* worker update */
    OB_KERNEL_COUNT = 12
} ob_kernel;

ob_status ob_plan_set_timing(ob_plan plan, int32_t enable);
ob_status ob_plan_read_timing(ob_plan plan, int32_t kernel, double* total_ms, int64_t* launches);

/* ---- diagnostics ([P1] sec. 6.2: warn when a parameter's error-buffer L2 norm is below 1e-6;
 * [P1] sec. 8: monitor that norm and the quantization rate) ----
 * With both pointers set (device arrays of K elements, 8-byte aligned), every later compressed step
 * with this plan (ob_adam_compress_step or ob_lamb_compress_step) also writes, per chunk c:
 *   err_sumsq_out[c]  = sum of squares (double) of the error buffer as that step read it, i.e. the
 *                       error left by the previous step; sqrt gives the L2 norm;
 *   plus_count_out[c] = number of elements of the chunk whose sign bit is +1 (the bit balance).
 * The first pass accumulates the first, the fused pass the second, and a one-block-per-chunk kernel
 * writes both.  The first call that enables them allocates two workspaces for the plan.  Both NULL
 * switches them off; exactly one NULL is OB_ERR_ARG. */
ob_status ob_plan_set_diagnostics(ob_plan plan, double* err_sumsq_out, uint64_t* plus_count_out);

/* ---- steps that a norm leaves out ----
 * For gradients clipped by their norm (ob_tensor_norms, ob_clip_grads), which are NaN if it is not finite.  With norm set (one fp32 in
 * device memory, 4-byte aligned), a step that is made with this plan afterwards (ob_adam_warmup_step, ob_adam_compress_step,
 * ob_lamb_warmup_step, ob_lamb_compress_step) reads it on the GPU; if it is not finite then, the step writes nothing: no state, no
 * parameter and none of its outputs, diagnostics among them.  NULL (as after ob_plan_create): every step is made.  The worker's and
 * the server's calls, whose outputs are exchanged, do not look at it.  A captured step keeps the address, and looks at every replay. */
ob_status ob_plan_set_guard(ob_plan plan, const float* norm);

/* ---- AdamW over many tensors at once ----
 * For models whose parameters are separate tensors (or views into buckets) rather than one flat buffer:
 * the dense Adam step of ob_adam_warmup_step with decoupled weight decay, per-tensor rates, parameters
 * and gradients of mixed types, clipping by the global gradient norm, and states in fp32 or in 8 bits.
 *
 * A list (ob_tensors) describes T tensors by size and type.  Their addresses are given with every call,
 * as host arrays of T device pointers, so gradients may move from step to step.  Parameter and gradient
 * pointers need the alignment of their element type only.  g[t] == NULL: tensor t has no gradient and the
 * call leaves it and its states alone.  Tensors of 0 elements are allowed (their pointers are ignored).
 * The parameters (and 16-bit copies) of two tensors must not overlap: OB_ERR_ARG.
 *
 * States (m, v, the master copy, 8-bit codes) are flat buffers of ob_tensors_state_elems(list) elements:
 * tensor t's state starts at ob_tensors_state_offset(list, t), the sum of the sizes before it with each
 * rounded up to a multiple of OB_STATE_BLOCK.  The gaps are neither read into a result nor written.
 *
 * Threads and streams: a list is read-only after its creation and holds no workspace, so calls with one
 * list may overlap if their buffers (parameters, states, control) differ.  No call synchronises,
 * allocates device memory or records anything but kernels, so all can be captured into a HIP graph; a
 * captured call keeps its addresses, hparams and list (which must outlive the graph), while what the control
 * block holds is read on replay. */
#define OB_STATE_BLOCK 256

typedef struct ob_tensors_s* ob_tensors;

/* sizes: T >= 0 host int64, each >= 0.  g_dtypes, p_dtypes: T ob_dtype values each (OB_F32, OB_BF16 or
 * OB_F16).  lr_mults, wd_mults: T host factors of the rate and of the weight decay (parameter groups), or
 * NULL for 1; finite.  At most 2^31 - 1 work blocks of 4096 elements in all (OB_ERR_ARG beyond).  The list belongs to the
 * device that is current here; it owns its device tables (hipMalloc here, hipFree in ob_tensors_destroy). */
ob_status ob_tensors_create(int64_t n_tensors, const int64_t* sizes, const int32_t* g_dtypes, const int32_t* p_dtypes,
                            const float* lr_mults, const float* wd_mults, ob_tensors* out);
ob_status ob_tensors_destroy(ob_tensors list);
int64_t ob_tensors_count(ob_tensors list);                    /* -1 for a NULL list */
int64_t ob_tensors_num_elements(ob_tensors list);             /* sum of the sizes; -1 for a NULL list */
int64_t ob_tensors_state_elems(ob_tensors list);              /* multiple of OB_STATE_BLOCK; -1 for a NULL list */
int64_t ob_tensors_state_offset(ob_tensors list, int64_t t);  /* -1 for a NULL list or t outside 0..T-1 */

/* Parameters of the AdamW step.  beta1, beta2 in [0, 1), eps >= 0 (8-bit states: eps >= 1e-30),
 * weight_decay and lr finite; OB_ERR_ARG otherwise. */
typedef struct {
    float lr;
    float beta1;
    float beta2;
    float eps;
    float weight_decay;      /* decoupled: p -= lr * weight_decay * p */
    int32_t bias_correction; /* divide m, v by 1 - beta^t */
    int64_t step;            /* t >= 1 without a control block; ignored with one */
    int32_t rounding;        /* ob_rounding: of 8-bit states and of 16-bit parameters without a master */
    int32_t reserved;        /* 0 */
    uint64_t sr_seed;        /* OB_ROUND_STOCHASTIC: the generator's key, with t */
} ob_adamw_hparams;

/* The control block: OB_CONTROL_BYTES of device memory owned by the caller, 8-byte aligned, all zero but
 * lr_scale (1) before its first use.  The fields below are followed by the norm's partial sums. */
typedef struct {
    float norm;          /* |g_mult| times the L2 norm of all gradients */
    float grad_scale;    /* what the step multiplies every gradient with */
    int64_t step;        /* t: steps taken, the coming one included */
    int64_t skipped;     /* steps not taken because their norm was not finite */
    double bc1, bc2;     /* 1 - beta1^t, 1 - beta2^t */
    float lr_scale;      /* written by the caller: factor of the rate (schedules under a captured graph) */
    int32_t skip;        /* 1: the norm was not finite, and a step with this block changes nothing */
    float root_factor;   /* bc1 / sqrt(bc2) */
    uint32_t ticket;     /* the norm's own: 0 between calls */
    uint32_t reserved[2];
} ob_control;
#define OB_CONTROL_PARTIALS 2048
#define OB_CONTROL_BYTES (64 + 8 * OB_CONTROL_PARTIALS)

/* Global gradient norm and clipping:
 *   norm = |g_mult| * sqrt(sum over all tensors of g^2), squares and sums in double, in an order that
 *          depends on the list alone (the same bits on every call);
 *   grad_scale = g_mult * min(1, max_norm / (norm + 1e-6)) in double, rounded once; max_norm <= 0 or
 *          infinite: g_mult.  g_mult (finite, not 0) removes a loss scale.
 * hp != NULL: also the step's bookkeeping.  norm finite: step += 1, bc1 and bc2 from it, skip = 0;
 * otherwise skipped += 1, skip = 1 (grad_scale then is 0 for an infinite norm with clipping, NaN for a NaN).
 * hp == NULL: skip is set as above, step, skipped, bc1 and bc2 stay (a step that corrects the bias or rounds
 * by chance needs them: give hp). */
ob_status ob_grad_norm(ob_tensors list, const void* const* g, float g_mult, float max_norm,
                       const ob_adamw_hparams* hp, ob_control* control, hipStream_t stream);

/* AdamW step with fp32 states.  With t, bc1, bc2, s = grad_scale and r = lr_scale from `control`, as the last
 * ob_grad_norm left it (NULL: t = hp->step, s = r = 1), for tensor j: a = lr * r * lr_mults[j], d = weight_decay * wd_mults[j],
 *   g' = fl32(widen(g) * s);  m = beta1*m + (1-beta1)*g';  v = beta2*v + (1-beta2)*g'^2;
 *   p -= a * ( (m/bc1) / (sqrt(v/bc2) + eps) + d*p )     (bc1 = bc2 = 1 without hp->bias_correction)
 * each line in double, rounded once, as in ob_adam_warmup_step; with d = 0, s = 1
 * and finite p the same bits as there.
 * Outputs must not alias inputs or each other.
 * p[t]: the parameters, updated in place.  master != NULL (fp32[state_elems]): for tensors of a 16-bit
 * type the master copy is the parameter, and p[t] gets its rounding to nearest; fp32 tensors do not use
 * it.  16-bit parameters without a master are widened, updated, rounded to fp32 and then to their type:
 * to nearest, ties to even, or stochastically by the rule of ob_adam_compress_step's error buffer, with i
 * the state index and the counter (i >> 2, t + 2^63). */
ob_status ob_adamw_step(ob_tensors list, const void* const* g, void* const* p, float* master, float* m, float* v,
                        const ob_adamw_hparams* hp, const ob_control* control, hipStream_t stream);

/* The 8-bit format: blocks of OB_STATE_BLOCK consecutive state elements, one fp32 scale q per block and
 * moment, fl = rounding to fp32:
 *   m: code c in -127..127, q = fl(max|m| * fl(1/127^2)), value fl(c*|c| * q);
 *   v: code k in 0..255, q = fl(fl(sqrt(max v)) * fl(1/255^2)), root r = fl(k^2 * q), value fl(r^2).
 * (Square-law codes: the step between neighbours is 2/c of an m and 4/k of a v, finest for the largest
 * values of a block and widening to 1/127^2 and 1/255^4 of it at the smallest.)
 * Rounding to nearest in the code: |c| is the largest k with k = 0 or |m| >= fl((k-1/2)^2 * q); k the
 * largest with k = 0 or v >= fl(T^2), T = fl((k-1/2)^2 * q).  Stochastic (steps only): k the largest with
 * value(k) <= x, then up iff fl(u * fl(value(k+1) - value(k))) < fl(fl(x - value(k)) * 65536), at most the
 * largest code; u: 16 bits of output word i & 3 of Philox4x32-10 at the counter (i >> 2, t) under the key
 * sr_seed, the low half for m, the high half for v (i: state index).  A v > 0 gets at least code 1, so that
 * no denominator collapses.  A block whose largest value is below 2^-96 is held as zeros (q = 0); in a
 * block with a NaN, an infinity or a negative v, q = NaN and the codes are 0: the block reads as NaN. */

/* AdamW step with states in that format: m_codes int8[state_elems], v_codes uint8[state_elems], m_scales and
 * v_scales fp32[state_elems / 256]; all zero is the state before the first step.  Arguments as
 * ob_adamw_step; the moments of the step are
 *   m = fma(beta1, m, fl(fl(1-beta1) * g')), v = fma(beta2, v, fl(fl(1-beta2) * fl(g'^2))) in fp32,
 * and the parameters' line is evaluated in fp32 (relative error of the update below 2^-20; values of v
 * below 2^-126 count as zero in its denominator). */
ob_status ob_adamw8_step(ob_tensors list, const void* const* g, void* const* p, float* master, int8_t* m_codes,
                         float* m_scales, uint8_t* v_codes, float* v_scales, const ob_adamw_hparams* hp,
                         const ob_control* control, hipStream_t stream);

/* The status with which ob_adamw_step (ob_adamw8_step) would refuse these arguments, or OB_OK; no GPU work.  For
 * callers that count a step with ob_grad_norm, which does not see the step's own arguments: called before it, a step
 * that is refused is not counted. */
ob_status ob_adamw_check(ob_tensors list, const void* const* g, void* const* p, const float* master, const float* m,
                         const float* v, const ob_adamw_hparams* hp, const ob_control* control);
ob_status ob_adamw8_check(ob_tensors list, const void* const* g, void* const* p, const float* master,
                          const int8_t* m_codes, const float* m_scales, const uint8_t* v_codes, const float* v_scales,
                          const ob_adamw_hparams* hp, const ob_control* control);

/* n fp32 moments into the 8-bit format, to nearest (v >= 0), and back; n >= 0, the last block may be short
 * (ceil(n / 256) scales).  Either moment may be left out: all its pointers NULL.  fp32 pointers 16-byte
 * aligned, codes 4 bytes, scales 4 bytes.  Runs on the current device. */
ob_status ob_state8_encode(int64_t n, const float* m, const float* v, int8_t* m_codes, float* m_scales,
                           uint8_t* v_codes, float* v_scales, hipStream_t stream);
ob_status ob_state8_decode(int64_t n, const int8_t* m_codes, const float* m_scales, const uint8_t* v_codes,
                           const float* v_scales, float* m, float* v, hipStream_t stream);

/* ---- norms of many tensors, and clipped gradients ----
 * For gradients that more than one optimizer steps, that another type holds, or that are clipped tensor by tensor; a step over
 * one list alone takes its norm from ob_grad_norm.
 *
 * ob_tensor_norms, with T = ob_tensors_count(list), into device memory:
 *   norms[t] = |g_mult| * sqrt(sum g_t^2)   OB_NORM_2    squares and sums in double, in an order that depends on the
 *            = |g_mult| * max |g_t|         OB_NORM_MAX  list alone (the same bits on every call)
 *   norms[T] = the same over all tensors.  Rounded to fp32 once; a tensor without a gradient or elements has norm 0, a
 *   NaN in a tensor gives NaN.
 * norms: fp32[T + 1].  workspace: ob_tensor_norms_workspace(list) bytes, 8-byte aligned, of any content; calls that may
 * overlap need their own.
 *
 * ob_clip_grads: out_t = fl(widen(g_t) * f), rounded once more to out_t's type, to nearest;
 *   f = g_mult * min(1, max_norm / (norm + 1e-6)) in double, rounded once; norm = norms[T], or norms[t] with per_tensor;
 *   max_norm <= 0 or infinite: f = g_mult;  norm not finite: f = NaN, so that whatever steps over these gradients and leaves out
 *   steps whose norm is not finite leaves out this one in all its parts.
 * norms: fp32[T + 1], as ob_tensor_norms left it or joined over workers by the caller; read on the GPU.
 * out == NULL: the gradients themselves, in their types (with f = 1 nothing is written); they must not overlap each other then.
 * Otherwise out[t]: tensors of the list's parameter types, for every t that has a gradient; each may be g[t] if the types are
 * of one width, and overlaps no other gradient or output.
 * g_mult: finite, not 0 (the same in both calls); removes a loss scale. */
typedef enum { OB_NORM_2 = 0, OB_NORM_MAX = 1 } ob_norm_kind;

int64_t ob_tensor_norms_workspace(ob_tensors list);   /* bytes; -1 for a NULL list */
ob_status ob_tensor_norms(ob_tensors list, const void* const* g, float g_mult, int32_t kind, float* norms, void* workspace,
                          hipStream_t stream);
ob_status ob_clip_grads(ob_tensors list, const void* const* g, void* const* out, const float* norms, float max_norm,
                        float g_mult, int32_t per_tensor, hipStream_t stream);

/* ---- matrix products ----
 * D = alpha * A B + beta * C over a batch, 16-bit operands, sums in fp32: statistics of gradients (L = b L + a G G^T),
 * projections of gradients, and what the Muon step below is made of.
 *
 * A is m x k, B k x n, C and D m x n; element (i, j) of a matrix is at i*row + j*col (elements), and a batch's next
 * matrix at + batch.  Of A's (B's) two strides one is 1 and the other arbitrary (>= 0), so that an operand
 * may be a transposed view; C and D lie by rows, col = 1.  Stride 0 repeats an operand's row, column or matrix.
 * Every pointer needs the alignment of its element only; operands whose pointers are 16-byte aligned, whose row (or
 * column) and batch strides are multiples of 8 and whose extent along the unit stride is one are read faster.
 *   in_type   of A and B: OB_BF16 or OB_F16
 *   out_type  of C and D: OB_F32, OB_BF16 or OB_F16; every element is fma(alpha, sum, fl(beta * C)) in fp32, rounded once
 *   beta = 0  C is not read and may be NULL
 *   k = 0     the sums are 0
 *   symmetric 1: m = n, and the caller knows that A B is symmetric (B = A^T, or powers of one symmetric matrix) and
 *             C is: what is below the diagonal is computed, and written above it too.
 * D may be C itself (same pointer and strides) and overlaps nothing else (OB_ERR_ARG where it starts at A or B).  Zero extents give
 * no work.
 * Extents are at most 2^31 - 1 - 256, offsets within a matrix and a batch below 2^60 elements; OB_ERR_ARG beyond.
 * workspace: ob_matmul_workspace(product) bytes of device memory, 16-byte aligned, of any content, or NULL: with it, tiles that
 * would not fill the card are shared by several work groups, which add their parts of K; calls that may overlap need their own.
 * Sums run in an order that depends on the extents, layouts and alignment, and on whether there is a workspace, alone.  Runs on
 * the current device; allocates nothing, synchronises nothing and records kernels only. */
typedef struct {
    int64_t batch, m, n, k;
    const void* a;
    int64_t a_row, a_col, a_batch;
    const void* b;
    int64_t b_row, b_col, b_batch;
    const void* c;
    int64_t c_row, c_batch;
    void* d;
    int64_t d_row, d_batch;
    int32_t in_type, out_type;
    float alpha, beta;       /* finite */
    int32_t symmetric;       /* 0 or 1 */
    int32_t reserved;        /* 0 */
    void* workspace;         /* or NULL */
} ob_product;

/* Bytes of the workspace that this product (its workspace aside) has use for; 0: none, or ob_matmul would refuse it. */
int64_t ob_matmul_workspace(const ob_product* product);
ob_status ob_matmul(const ob_product* product, hipStream_t stream);

/* ---- Muon over lists of matrices ----
 * The step of the Muon optimizer, for the matrices of a model (AdamW steps the rest): momentum, the momentum's nearest
 * semi-orthogonal matrix by a polynomial iteration, decoupled decay and the update.  With f = grad_scale and r = lr_scale
 * of `control` (NULL: 1), for each matrix of R rows and C columns:
 *   g' = fl32(widen(g) * f);  m = fl32(mu*m + (1-mu)*g');  u = nesterov ? (1-mu)*g' + mu*m : m
 *   X = u / (|u| + eps), |u| the Frobenius norm, its sum in double
 *   `iterations` times, with X taken with its smaller side first:  A = X X^T,  X = a X + (b A + c A^2) X,
 *     a, b, c = 3.4445, -4.7750, 2.0315: singular values in (0, 1] are driven into about [0.7, 1.2]
 *   p -= l * (weight_decay * wd_mults[j] * p + s * X),  l = lr * r * lr_mults[j],
 *     s = 1 (OB_MUON_PLAIN), sqrt(max(1, R / C)) (OB_MUON_SHAPE) or 0.2 sqrt(max(R, C)) (OB_MUON_MATCH_RMS: updates of about
 *     the size of AdamW's, so that both take one rate and decay)
 * Operands of the products are fp16 times powers of two (X 2^9, A and b A + c A^2 2^10; the iteration's bounds keep them in
 * range), sums fp32: X is off by 1 to 4 parts in 1000 (2-norm, five iterations), the more the smaller its smallest singular
 * values; directions whose singular value is below 2^-12 of |u| may come out as noise of that size, grown by the iteration as they
 * would be themselves.
 * The decay and the update are one fp32 expression, fma(-l, fma(d, p, s X), p), rounded once more to a 16-bit p without
 * master.  control with skip set: nothing changes.
 *
 * The plan holds the matrices' shapes for a list: tensor t has sizes[t] = E * rows[t] * cols[t] elements, E >= 0 matrices behind
 * each other, each by rows.  rows, cols: T host int64, 1 to 2^30, and of a matrix that is not small, with its sides s <= l rounded up
 * to 8, (min(s, 64) - 1) l + 256 below 2^30 (64 rows of 17 million, 8 of 153 million: OB_ERR_ARG beyond).  It belongs to the list's
 * device, copies what it needs of the list, and owns its device tables; it must outlive a captured step.
 * m, master: flat, ob_tensors_state_elems(list) fp32 in the list's layout; g, p, master otherwise as in ob_adamw_step.
 * workspace: ob_muon_workspace(plan) bytes of device memory, 16-byte aligned, of any content (NULL where that is 0: small matrices
 * need none); calls that may overlap (other streams, captured graphs replayed at once) need their own.
 * ob_muon_check: the status with which ob_muon_step would refuse these arguments; no GPU work. */
typedef struct ob_muon_s* ob_muon;

typedef enum { OB_MUON_PLAIN = 0, OB_MUON_SHAPE = 1, OB_MUON_MATCH_RMS = 2 } ob_muon_scale;

typedef struct {
    float lr;               /* finite */
    float momentum;         /* mu in [0, 1) */
    float weight_decay;     /* finite */
    float eps;              /* > 0: at least 1e-30 */
    int32_t nesterov;       /* 0 or 1 */
    int32_t iterations;     /* 1 to 16 */
    int32_t scale;          /* ob_muon_scale */
    int32_t reserved;       /* 0 */
} ob_muon_hparams;

ob_status ob_muon_create(ob_tensors list, const int64_t* rows, const int64_t* cols, ob_muon* out);
ob_status ob_muon_destroy(ob_muon plan);
int64_t ob_muon_workspace(ob_muon plan);   /* bytes; -1 for a NULL plan */
ob_status ob_muon_step(ob_muon plan, const void* const* g, void* const* p, float* master, float* m, void* workspace,
                       const ob_muon_hparams* hp, const ob_control* control, hipStream_t stream);
ob_status ob_muon_check(ob_muon plan, const void* const* g, void* const* p, const float* master, const float* m,
                        const void* workspace, const ob_muon_hparams* hp, const ob_control* control);

#ifdef __cplusplus
}
#endif

#endif /* OB_ADAM_H */
