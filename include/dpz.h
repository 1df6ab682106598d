/*
 * dpz — the data-parallel / ZeRO-1 gradient-synchronisation and optimizer step
 * for N simulated ranks whose replicas all live in one GPU's memory.
 *
 * A "rank" is a replica slab of an arena.  The collectives of the pages become
 * in-memory kernels: a ring "send" of a chunk is a load from another slab, the
 * ring's hop order is a fixed per-element fold order, and an all-gather is N
 * coalesced stores.  Every compute call is asynchronous on the caller's CUDA
 * stream, never synchronises the host, allocates nothing, and launches only
 * this library's own kernels (dpz_device_status, a read of a device flag, is
 * the one synchronous call).
 *
 * ------------------------------------------------------------------------
 * Layout (all buffers are owned and allocated by the caller, device memory)
 *
 *   N   number of ranks, 1 <= N <= 64
 *   P   elements per replica (a flat parameter / gradient arena), P % (8N) == 0
 *   C   chunk = shard = P / N; chunk c is elements [c*C, (c+1)*C)
 *   grads    [N][P] gradient dtype: slab r = grads + r*P = rank r's gradients
 *   weights  [N][P] weight dtype:   slab r = rank r's weight replica
 *   master, m, v   [P] fp32 each: the N ranks' shards laid end to end, so rank
 *            r's shard (A4 — Multi-GPU with NCCL and ZeRO-1, Part 2:
 *            shard_offset = rank * shard_size) is elements [r*C, (r+1)*C)
 *   ws       dpz_workspace_bytes(P, N) bytes, 16-byte aligned: norm partials
 *            and the global norm, written and read only by this library
 *
 * Chunk ownership: rank c owns chunk c.  The reduce-scatter is the ring of
 * "Lab 09 — Parallelism, simulated", §1, rotated so that its last receiver of
 * chunk c is rank c; element i of chunk c is therefore summed as the left fold
 *     acc = x[(c+1)%N][i];  acc = R(acc + x[(c+j)%N][i]) for j = 2..N
 * where R rounds to the gradient dtype (identity for fp32; round to nearest
 * even for bf16, so a bf16 ring rounds once per hop: 13.5 Multi-GPU from First
 * Principles, Exercise 8).  The average is R(acc / N): sum, then divide by N
 * (Lab 09 §2; A4 Part 3, ncclAvg).  The fold order never depends on the
 * launch configuration, so results are bit-for-bit reproducible.
 *
 * Alignment: bf16 buffers 16-byte aligned, fp32 buffers (master, m, v and
 * fp32 gradients or weights) 32-byte aligned, the workspace 16-byte aligned;
 * P % (8N) == 0, so that every chunk is a whole number of 8-element groups
 * (each lane moves 8 elements with one 128- or 256-bit access).
 *
 * Status: every call returns DPZ_OK or an error code without launching
 * anything when an argument is invalid (null pointer, N out of range,
 * P <= 0, P % N != 0, bad dtype, step < 1, overlapping buffers), and
 * DPZ_ERR_ALIGN for misaligned pointers or chunks (P/N not a multiple of 8).
 * A CUDA launch failure returns DPZ_ERR_CUDA.  dpz_last_error() gives the
 * calling thread's last message.  NaN and Inf inputs are not special-cased:
 * they propagate.
 *
 * Streams: the caller orders producers of `grads` before the call with
 * events (A4 Part 3: record an event on the compute stream, make the
 * communication stream wait on it), and consumers after it.  Every kernel is
 * launched with programmatic stream serialisation: its blocks may be placed
 * while the kernel before it on the same stream still runs, and they wait
 * for that kernel to complete (its writes visible) before they touch memory.
 * So the calls keep the stream's order after a kernel, a copy or an event
 * wait alike.
 *
 * CUDA graphs: every compute call except dp_grad_global_norm_static only
 * enqueues kernels on `stream`, so it can be captured into a CUDA graph and
 * replayed.  Call each once outside capture first (its launch configuration
 * is cached per device) and keep profiling off while capturing.
 */
#ifndef DPZ_H
#define DPZ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define DPZ_API __attribute__((visibility("default")))
#else
#define DPZ_API
#endif

/* element types */
#define DPZ_F32 0
#define DPZ_BF16 1
/* Gradients only: bf16 storage whose ring accumulates in fp32 (13.5 Multi-GPU
 * from First Principles, Exercise 8, second variant: each rank's vector is
 * rounded to bf16 once and the sum is accumulated in fp32).  The fold is
 *     acc = x[(c+1)%N][i];  acc = acc + x[(c+j)%N][i]  (fp32, j = 2..N)
 * and the stored average is RNE_bf16(acc / N), one rounding in all.  The
 * arena, the stored averages and every byte moved are those of DPZ_BF16; in
 * a ring of processes the partial sums would travel as fp32 (twice the
 * reduce-scatter's bytes), here they stay in registers. */
#define DPZ_BF16_ACC32 2

/* status codes */
#define DPZ_OK 0
#define DPZ_ERR_INVALID_ARG 1
#define DPZ_ERR_ALIGN 2
#define DPZ_ERR_CUDA 3

#define DPZ_MAX_RANKS 64

/* Per-call status in the workspace.  Three kernels stage their tiles through
 * shared memory with asynchronous bulk copies and wait for them on a barrier,
 * bounded by the SM clock (about two seconds): the norm of the owner chunks
 * (dp_grad_global_norm, dp_grad_global_norm_static), the one-kernel step
 * without clip (dp_zero1_step), and the AdamW + all-gather update from stored
 * averages (dp_zero1_step with clip, dp_zero1_update, dp_zero2_update).  If a
 * wait runs out the kernel gives up on that tile instead of hanging, and says
 * so in stream order, for a consumer on the same stream to see without
 * synchronising:
 *   - the uint32 at byte DPZ_WS_STATUS_OFFSET of the call's workspace holds
 *     DPZ_STATUS_* bits.  Every norm finalisation (dp_grad_global_norm,
 *     dp_grad_norm_finalize, dp_zero1_step with clip or with norm_out) writes
 *     the whole word; the update kernels that follow it only set
 *     DPZ_STATUS_UPDATE_SKIPPED.  So after dp_zero1_step with a workspace and
 *     a clip or a norm_out, and after dp_grad_norm_finalize followed by
 *     dp_zero1_update / dp_zero2_update, the word describes that step alone;
 *   - the norm written to the workspace and to norm_out is NaN;
 *   - an update with clipping whose norm has DPZ_STATUS_NORM_SKIPPED set is not
 *     applied at all: master/m/v and the weights keep their values and
 *     DPZ_STATUS_UPDATE_SKIPPED is set.
 * dp_zero1_step without clip and without norm_out runs no finalisation and
 * has no per-call word; there, and in every case, the device-wide flag of
 * dpz_device_status is raised as well.  NaN or Inf in the data is not a
 * status: it propagates into the norm and the update as any value does. */
#define DPZ_WS_STATUS_OFFSET 20
#define DPZ_STATUS_NORM_SKIPPED 1u   /* a tile of the norm's input was not read */
#define DPZ_STATUS_UPDATE_SKIPPED 2u /* a tile of master/m/v and the weights was
                                        not updated (it keeps the old values) */

/* AdamW hyperparameters for one step (A4 Part 4: the optimizer runs on the
 * owned shard).  The update, in fp32 with every operation rounded:
 *   g  = avg * s          s = clip/norm if clip_norm > 0 and norm > clip_norm,
 *                         else 1 (norm: of the averaged gradient, before the
 *                         step)
 *   m  = beta1*m + (1-beta1)*g
 *   v  = beta2*v + (1-beta2)*(g*g)
 *   mh = m / bc1,  vh = v / bc2,  bc = 1 - beta^step (host, double -> float)
 *   theta = theta - lr * (mh / (sqrt(vh) + eps) + weight_decay * theta)
 * weights = theta cast to the weight dtype (round to nearest even for bf16). */
typedef struct dpz_adamw_cfg {
    float lr;
    float beta1;
    float beta2;
    float eps;
    float weight_decay;
    int64_t step;        /* t >= 1, passed by the caller; the library keeps no state */
    float clip_norm;     /* > 0: global-norm clip to this value; <= 0: no clip */
    int store_avg;       /* dp_zero1_step without clip: nonzero also stores the
                            averaged gradient into chunk c of slab c */
} dpz_adamw_cfg;

/* Per-kernel timing collected while profiling is on (see dpz_profile_start). */
typedef struct dpz_kernel_stat {
    char name[48];
    int64_t launches;
    double total_ms;     /* sum of per-launch CUDA-event durations */
} dpz_kernel_stat;

/* Bytes of device workspace `ws` must provide for an arena of N slabs of P
 * elements: a 256-byte header (the norm), 256 first-stage sums and one fp64
 * sum of squares per 256-element segment of every chunk (about P/32 bytes).
 * Returns 0 for invalid P or N. */
DPZ_API size_t dpz_workspace_bytes(int64_t P, int N);

/* Ring reduce-scatter + average, in place (A4 Part 3: ncclReduceScatter of
 * pointers[i] into pointers[i] + shard_offset with ncclAvg; Lab 09 §1 ring).
 * grads: [N][P] device, dtype gdtype.  On return chunk c of slab c holds the
 * average of chunk c over the N ranks; every other chunk of every slab is
 * untouched.  Reads N*P and writes P elements. */
DPZ_API int dp_reduce_scatter_avg(void* grads, int64_t P, int N, int gdtype,
                                  void* stream);

/* Ring all-reduce + average (ZeRO-0), in place (A4 Part 3, zero_stage 0:
 * ncclAllReduce with ncclAvg; Lab 09 §1: reduce-scatter then all-gather).
 * On return every slab holds the average; chunk c equals what the
 * reduce-scatter leaves in chunk c of slab c.  Reads and writes N*P. */
DPZ_API int dp_allreduce_avg(void* grads, int64_t P, int N, int gdtype,
                             void* stream);

/* Global L2 norm of the averaged gradient held in the owner chunks (chunk c of
 * slab c, as left by dp_reduce_scatter_avg): each rank's sum of squares of its
 * shard, then the sum over ranks ("Distributed training", Gates: ZeRO stages
 * differ from DDP only in the order the global norm is summed).  Squares are
 * summed in fp32 within each 256-element segment (a fixed pairwise tree); the
 * segment sums are then added in a fixed two-level order (compensated fp32
 * chains, fp64 beyond them), which depends on P and N alone, so every entry
 * point and every launch configuration gives the same bits.
 * Writes the norm into ws (for zero1_adamw_step) and, if norm_out is not
 * NULL, to *norm_out (device pointer to one float). */
DPZ_API int dp_grad_global_norm(const void* grads, int64_t P, int N, int gdtype,
                                void* ws, float* norm_out, void* stream);

/* Sharded AdamW (A4 Part 4, step 1: adamw_update on this rank's shard only).
 * For every rank c: reads the averaged chunk c of slab c, updates master/m/v
 * elements [c*C, (c+1)*C) and writes the cast weights into chunk c of slab c
 * of `weights` only (the all-gather is dp_allgather).  If cfg->clip_norm > 0
 * the clip scale uses the norm that dp_grad_global_norm left in ws (ws may be
 * NULL otherwise).  gdtype/wdtype: DPZ_F32 or DPZ_BF16. */
DPZ_API int zero1_adamw_step(const void* grads, float* master, float* m,
                             float* v, void* weights, int64_t P, int N,
                             int gdtype, int wdtype, const dpz_adamw_cfg* cfg,
                             const void* ws, void* stream);

/* All-gather (A4 Part 4, step 2: ncclAllGather of the updated shards; Lab 09
 * §1 all-gather phase): chunk c of slab c is copied into chunk c of every
 * other slab, in place.  Reads P and writes (N-1)*P elements. */
DPZ_API int dp_allgather(void* weights, int64_t P, int N, int wdtype,
                         void* stream);

/* The whole ZeRO-1 step, fused: reduce-scatter + average -> (global norm and
 * clip) -> AdamW on each rank's shard -> cast -> all-gather into all N weight
 * slabs.  Bit-identical to calling dp_reduce_scatter_avg,
 * dp_grad_global_norm (when clipping), zero1_adamw_step and dp_allgather in
 * turn.  Without clipping it is one kernel that reads each gradient byte once
 * and writes the averages only if cfg->store_avg, plus the norm's
 * finalisation when norm_out is given (for arenas of at most 32 segments of
 * 256 elements, one kernel on a thread-block cluster does both); with clipping it is three
 * (reduce + norm partials and averages store, norm finalize, AdamW + cast +
 * broadcast), because the clip scale depends on every element.  norm_out
 * (device, may be NULL) receives the global norm; ws is required when
 * clipping or when norm_out is given. */
DPZ_API int dp_zero1_step(void* grads, float* master, float* m, float* v,
                          void* weights, int64_t P, int N, int gdtype,
                          int wdtype, const dpz_adamw_cfg* cfg, void* ws,
                          float* norm_out, void* stream);

/* ---------------------------------------------------------------------
 * Buckets (overlap with the backward pass) and ZeRO-2 (sharded gradients)
 *
 * A backward pass produces the gradients layer by layer, from the last layer
 * to the first, so a bucket of the arena can be reduced while the rest is
 * still being computed ("A4 — Multi-GPU with NCCL and ZeRO-1", Part 3: each
 * layer's reduction runs on a separate stream after an event recorded on the
 * compute stream; "Lab 09 — Parallelism, simulated", §2: DDP all-reduces 25
 * MB buckets as backward produces them; "Distributed training", "Overlap and
 * graphs").  Record an event on the producing stream after each bucket is
 * written and make the stream of these calls wait on it.
 *
 * Buckets reduce element ranges [lo, lo+n) of the arena (lo and n multiples
 * of 8; any ranges, in any order, each element once per step).  With ws,
 * each range must start and end on 256-element segment boundaries of its
 * chunks ((lo mod C) and ((lo+n) mod C) multiples of 256) and its norm
 * partials are written; once every bucket is reduced, dp_grad_norm_finalize
 * gives the same norm, bit for bit, as the whole-arena calls.
 *
 * max_ctas bounds the thread blocks of the reduction kernel.  0: one pass
 * with as many blocks as the range needs, the fastest when nothing else runs.
 * > 0: at most max(max_ctas, c) blocks, where c is the number of chunks the
 * range touches, each looping over its part of the range.  A reduction that
 * runs beside compute kernels on other streams (a backward pass) should leave
 * them most of the GPU: with one block per SM it hid about 60 % of its time
 * behind a compute-bound stand-in on GB300, against about 10 % with 0, whose
 * blocks take every SM slot that the compute kernels free.  The result is the
 * same, bit for bit, for every max_ctas.  Negative: DPZ_ERR_INVALID_ARG.
 * ------------------------------------------------------------------- */

/* ZeRO-1 with buckets: reduce + average elements [lo, lo+n) of the arena in
 * place (the average of element e of chunk c goes to slab c), as
 * dp_reduce_scatter_avg does for the whole arena.  ws may be NULL (no norm
 * partials). */
DPZ_API int dp_reduce_scatter_avg_range(void* grads, int64_t P, int N, int gdtype,
                                        int64_t lo, int64_t n, void* ws, int max_ctas,
                                        void* stream);

/* ZeRO-2: gradients are sharded too ("Lab 09 — Parallelism, simulated", §4:
 * stage 2 shards the gradients, 2Ψ + 14Ψ/N bytes per rank; "Distributed
 * training": ZeroSharded[M, N, 2]).  Reduce + average a bucket of N ranks' gradients for
 * arena elements [lo, lo+n), held in a staging buffer [N][n] (rank r's
 * values at staging + r*n), into `shards` [P]: the average of element e is
 * written at shards[e], which belongs to rank e / C's shard.  The staging
 * buffer can be reused for the next bucket once this call has run, so no
 * rank keeps a full gradient replica. */
DPZ_API int dp_reduce_scatter_avg_bucket(const void* staging, int64_t lo, int64_t n,
                                         void* shards, int64_t P, int N, int gdtype,
                                         void* ws, int max_ctas, void* stream);

/* The global norm from the partials that the range or bucket calls left in
 * ws (all of [0, P) reduced, with ws); writes it into ws and, if not NULL,
 * *norm_out. */
DPZ_API int dp_grad_norm_finalize(void* ws, int64_t P, int N, float* norm_out,
                                  void* stream);

/* The second half of dp_zero1_step: AdamW on every rank's shard reading the
 * averaged chunk c of slab c, cast, and the all-gather into all N weight
 * slabs (one kernel).  Clip scale from the norm in ws when clip_norm > 0. */
DPZ_API int dp_zero1_update(const void* grads, float* master, float* m, float* v,
                            void* weights, int64_t P, int N, int gdtype, int wdtype,
                            const dpz_adamw_cfg* cfg, const void* ws, void* stream);

/* The same for ZeRO-2: the averages are read from shards [P]. */
DPZ_API int dp_zero2_update(const void* shards, float* master, float* m, float* v,
                            void* weights, int64_t P, int N, int gdtype, int wdtype,
                            const dpz_adamw_cfg* cfg, const void* ws, void* stream);

/* The global norm of dp_grad_global_norm for callers that cannot allocate
 * device memory.  The pages have no counterpart to this call.  It serves code
 * that must not call cudaMalloc or any allocator of its own: a plug-in running
 * inside a host framework whose caching allocator owns all device memory, or
 * a service that reserves its whole memory budget up front.  Such a caller
 * cannot provide the workspace of dp_grad_global_norm.  Here the partial sums
 * live in a fixed 4 MiB array of device memory that the library declares at
 * file scope, so the call allocates nothing; it needs
 * dpz_workspace_bytes(P, N) <= 4 MiB (for example the GPT-2 124M arena at
 * N = 8) and returns DPZ_ERR_INVALID_ARG with a clear message beyond that.
 * Inputs and output are as in dp_grad_global_norm; norm_out (one float of
 * device memory) is required.
 *
 * The first call on a device looks up the array's address on that device
 * (cudaGetSymbolAddress), so make that first call before any stream capture.
 * Every later call made outside a stream capture looks it up again (after a
 * device reset the array may sit elsewhere).
 * Every GPU that loads the library holds the 4 MiB array until the process
 * exits.  All calls share it: each call clears what must start at zero, but
 * calls whose kernels overlap on the GPU (unordered streams) race with each
 * other and give wrong results. */
DPZ_API int dp_grad_global_norm_static(const void* grads, int64_t P, int N,
                                       int gdtype, float* norm_out, void* stream);

/* ---------------------------------------------------------------------
 * The two ends of a language model's training step
 *
 * The arena calls above take over once every gradient slab is filled.  These
 * calls sit at the other end of a replica's forward and backward pass, where
 * it meets the vocabulary: the embedding lookup that reads a table in a
 * weight slab, the loss that reads the logits, the gradient of the logits,
 * and the table's gradient in a gradient slab.  They have no counterpart on
 * the pages (which start from filled gradients), run on one replica's
 * buffers, and keep the library's rules: asynchronous on `stream`, nothing
 * allocated, and the same bits from every run, because no sum's order depends
 * on the launch or on the order of atomics.
 *
 *   T   tokens (rows), 0 <= T < 2^31;   V  vocabulary, 1 <= V < 2^30
 *   D   width of an embedding row, 1 <= D < 2^20
 *   Matrices are row-major with a row stride in elements (ld_*, at least the
 *   row's length), so that a table inside an arena or logits with padded rows
 *   need no copy.  Any stride and any element-aligned address is accepted;
 *   the fastest accesses need the alignment each call states.  (A matrix of
 *   one row is the same matrix whatever its stride.)
 *   Ids are DPZ_I32 or DPZ_I64; an id outside [0, V) names no token.
 *   Element types are DPZ_F32 or DPZ_BF16; arithmetic is fp32, with one
 *   rounding to the output's type at the end.
 *   Kernels run on the current device, where all of a call's buffers must be.
 *   A call with T = 0 writes no row (lm_embedding_grad still writes dtable).
 *   Errors are as above: DPZ_ERR_INVALID_ARG for a NULL pointer, a size out
 *   of range, a stride below the row length, an unknown type, a scale that is
 *   not finite, a factor of the logits (scale, temperature or its inverse)
 *   outside (0, 1e30], or buffers of which one is written and that overlap,
 *   except where a call allows it (two matrices of one stride may interleave,
 *   as column ranges of a larger one do); DPZ_ERR_ALIGN for an address that is
 *   not a multiple of its element.
 * ------------------------------------------------------------------- */

/* id types */
#define DPZ_I32 16
#define DPZ_I64 17

#define DPZ_LM_MAX_TOP 32       /* most alternatives of lm_logprobs */
#define DPZ_LM_MAX_TEACHER 256  /* most teacher logits per row of lm_distill* */

/* Embedding lookup: out[t, :] = R(scale * table[ids[t], :]), a row of zeros
 * where ids[t] names no token.  table [V][D] (wdtype), out [T][D] (odtype).
 * Fastest with 32-byte aligned fp32 (16-byte bf16) rows and D % 8 == 0. */
DPZ_API int lm_embedding(const void* table, int64_t ld_table, int64_t V, int64_t D, int wdtype,
                         const void* ids, int itype, int64_t T, float scale, void* out,
                         int64_t ld_out, int odtype, void* stream);

/* Bytes of device workspace of lm_embedding_grad; 0 for invalid sizes. */
DPZ_API size_t lm_embedding_workspace_bytes(int64_t T, int64_t V, int64_t D);

/* Gradient of lm_embedding with respect to the table, added to `base`:
 *     dtable[v, :] = R(base[v, :] + scale * sum over t with ids[t] = v of dout[t, :])
 * dout [T][D] (ddtype); base and dtable [V][D] (gdtype).  base NULL: zeros,
 * so that every row of dtable is written.  base may be dtable itself (same
 * address and stride): rows whose token does not occur are then left
 * untouched, which is how a tied output layer's gradient in the slab gets the
 * lookup's part.  The tokens are sorted first and each row is summed in fp32
 * in the order of t (rows of very frequent tokens in pieces of fixed length,
 * joined in order), so the result does not depend on the launch.  Tokens
 * whose id names none contribute nothing.  ws: lm_embedding_workspace_bytes
 * bytes, 16-byte aligned. */
DPZ_API int lm_embedding_grad(const void* dout, int64_t ld_dout, int ddtype, const void* ids,
                              int itype, int64_t T, float scale, const void* base,
                              int64_t ld_base, void* dtable, int64_t ld_dtable, int gdtype,
                              int64_t V, int64_t D, void* ws, void* stream);

/* Log probabilities of given tokens.  With z = scale * logits[t, :] (scale:
 * the inverse temperature, > 0) and lse = log sum_j exp(z_j):
 *     logprob[t] = z[targets[t]] - lse          (0 where the id names no token)
 *     lse[t], and entropy[t] = lse - sum_j p_j z_j,  p = exp(z - lse)
 *     top_ids[t, k], top_logprobs[t, k]: the K largest logits in descending
 *     order, the lowest id first among equal ones (+0 equals -0, NaN counts
 *     as the largest), and their log probabilities
 * logits [T][V] (dtype); targets and top_ids of type itype; logprob, lse,
 * entropy and top_logprobs fp32; top_ids and top_logprobs [T][K], densely.
 * lse and entropy may be NULL; with K = 0 (at most DPZ_LM_MAX_TOP and V) the
 * top pointers are not used.  logprob may be NULL with targets NULL.
 * A logit of -inf is masked: p = 0.  A row of -inf alone gives lse -inf,
 * log probabilities -inf and entropy 0; a row that holds NaN or +inf gives
 * NaN for all of them. */
DPZ_API int lm_logprobs(const void* logits, int64_t ld, int64_t T, int64_t V, int dtype,
                        float scale, const void* targets, int itype, float* logprob, float* lse,
                        float* entropy, int K, void* top_ids, float* top_logprobs, void* stream);

/* Gradient of lm_logprobs with respect to the logits, from the lse and the
 * entropy that it gave and the gradients of its outputs:
 *     dlogits[t, j] = R(scale * (dlogprob[t] * (1[j = targets[t]] - p_j)
 *                                - dentropy[t] * p_j * (log p_j + entropy[t])))
 * dentropy may be NULL (zero; entropy is then not read).  Where the id names
 * no token, dlogprob counts as 0.  A row whose two gradients are 0, or whose
 * lse is -inf, is zeros (its logits are not read).  dlogits [T][V] (dtype)
 * may be logits itself (same address and stride).
 * p_j = exp(z_j - lse[t]) with lse as given, in fp32: lse's own rounding is an
 * error of p of up to 2^-24 |lse|, relative, and an lse beyond 1e6 no longer
 * holds log V.  A row wholly masked by a large finite value instead of -inf
 * wants weights of 0. */
DPZ_API int lm_logprobs_grad(const void* logits, int64_t ld, int64_t T, int64_t V, int dtype,
                             float scale, const void* targets, int itype, const float* lse,
                             const float* entropy, const float* dlogprob, const float* dentropy,
                             void* dlogits, int64_t ld_dlogits, void* stream);

/* Distillation from a teacher's top logits.  Row t has K teacher entries:
 * token teacher_ids[t, k] with logit teacher_logits[t, k] ([T][K], densely,
 * tdtype).  With tau = temperature, z = logits / tau, p = softmax(z) over the
 * vocabulary and q = softmax(teacher_logits / tau) over the row's entries:
 *     loss[t] = sum_k q_k * (log q_k - log p[teacher_ids[t, k]])
 * An entry whose id names no token, or whose logit is -inf, is absent; a row
 * without entries has loss 0.  Entries that name one token twice each count.
 * lse[t] = log sum_j exp(z_j) (may be NULL).  q_k > 0 on a token of p = 0
 * gives loss +inf; rows with NaN or +inf among the logits give NaN. */
DPZ_API int lm_distill(const void* logits, int64_t ld, int64_t T, int64_t V, int dtype,
                       const void* teacher_ids, int itype, const void* teacher_logits,
                       int tdtype, int K, float temperature, float* loss, float* lse,
                       void* stream);

/* Gradient of sum_t dloss[t] * loss[t] with respect to the logits, from lse:
 *     dlogits[t, j] = R(dloss[t] / tau * (p_j - sum over k with id j of q_k))
 * Rows with dloss 0, without entries or with lse -inf are zeros.  dlogits
 * [T][V] (dtype) may be logits itself (same address and stride).  p_j comes
 * from lse as lm_logprobs_grad's does, with the same error. */
DPZ_API int lm_distill_grad(const void* logits, int64_t ld, int64_t T, int64_t V, int dtype,
                            const void* teacher_ids, int itype, const void* teacher_logits,
                            int tdtype, int K, float temperature, const float* lse,
                            const float* dloss, void* dlogits, int64_t ld_dlogits, void* stream);

/* lm_distill and lm_distill_grad in one pass, for a training step that knows
 * its rows' weights dloss beforehand (1 / tokens, or 0 for padding): the
 * logits are read from memory once.  Here a row with dloss 0 still gets its
 * loss and lse, and p_j does not pass through lse's rounding: a value common
 * to a row's logits does not change its gradient. */
DPZ_API int lm_distill_step(const void* logits, int64_t ld, int64_t T, int64_t V, int dtype,
                            const void* teacher_ids, int itype, const void* teacher_logits,
                            int tdtype, int K, float temperature, const float* dloss, float* loss,
                            float* lse, void* dlogits, int64_t ld_dlogits, void* stream);

/* ---------------------------------------------------------------------
 * The attention block of a replica's training step
 *
 * Between the vocabulary-sized ends: the norm of each head of queries and keys
 * with the rotation by position, attention, and their gradients.  They have
 * no counterpart on the pages and keep the library's rules: asynchronous on
 * `stream`, nothing allocated, no sum's order left to atomics, so that every
 * call repeats bit for bit.
 *
 *   T, Tq, Tk  tokens, 0 .. 2^30;   Hq, Hk  heads of queries and of keys (and
 *   values), up to 65535;   D  elements of a head
 *   A tensor of heads is a dpz_heads: element [t][h][d] at
 *   p + (t * ld + h * hs + d) elements.  So the parts of a fused projection
 *   [T][(Hq + 2 Hk) * D], tokens first or heads first, need no copy.  Strides
 *   are at least D, the elements distinct, the address a multiple of the
 *   element; those of a single token or head are not looked at.
 *   Element types are DPZ_F32 or DPZ_BF16, one for all tensors of heads of a
 *   call; results are rounded to it once.
 *   Errors are as above: DPZ_ERR_INVALID_ARG for a NULL pointer (a tensor
 *   without elements may be NULL), a size or stride out of range, an unknown type,
 *   or buffers of which one is written and that overlap, except where a call
 *   allows it (tensors of heads may interleave, as column ranges of a larger
 *   one do); DPZ_ERR_ALIGN for an address that is not a multiple of its element.
 * ------------------------------------------------------------------- */

typedef struct dpz_heads {
    void* p;
    int64_t ld; /* elements between tokens */
    int64_t hs; /* elements between heads */
} dpz_heads;

/* Norm of every head of q [T][Hq][D] and k [T][Hk][D] and rotation by position,
 * D <= 256:
 *     y = w * x * (mean_d x^2 + eps)^(-1/2),   rounded once after the rotation of
 *     its first R elements (R even, <= D): pair i (elements i and i + R/2, or
 *     2 i and 2 i + 1 with `interleaved`) turns by positions[t] * inv_freq[i],
 *     (a, b) -> (a cos - b sin, b cos + a sin)
 * wq and wk [D] (wdtype) or NULL for ones; positions [T] (itype, any value),
 * inv_freq [R/2] fp32 (radians per position, finite); R = 0: no rotation, neither is
 * read.  The angle is taken modulo a turn exactly for |inv_freq| < 2^40, so
 * far positions lose nothing.  q_out may be q and k_out k (same address and
 * strides).  Fastest where addresses and strides are multiples of 16 bytes and R / 2 of 8
 * elements (4 in fp32). */
DPZ_API int attn_qk_norm_rope(const dpz_heads* q, const dpz_heads* k, int64_t T, int64_t Hq,
                              int64_t Hk, int64_t D, int dtype, const void* wq, const void* wk,
                              int wdtype, float eps, const void* positions, int itype,
                              const float* inv_freq, int64_t R, int interleaved,
                              const dpz_heads* q_out, const dpz_heads* k_out, void* stream);

/* Bytes of device workspace of attn_qk_norm_rope_grad; 0 for invalid sizes. */
DPZ_API size_t attn_qk_norm_rope_workspace_bytes(int64_t T, int64_t Hq, int64_t Hk, int64_t D);

/* Gradient of attn_qk_norm_rope: from its inputs q and k (not its outputs) and the
 * gradients dq_out and dk_out of its outputs, dq and dk (which may be dq_out
 * and dk_out) and, where not NULL, dwq and dwk [D] (wdtype), summed over all
 * tokens and heads in fp32 and joined in fp64, in an order that the sizes and the
 * alignment fix.  ws: attn_qk_norm_rope_workspace_bytes bytes, 16-byte aligned;
 * not used without dwq and dwk. */
DPZ_API int attn_qk_norm_rope_grad(const dpz_heads* q, const dpz_heads* k, const dpz_heads* dq_out,
                                   const dpz_heads* dk_out, int64_t T, int64_t Hq, int64_t Hk,
                                   int64_t D, int dtype, const void* wq, const void* wk, int wdtype,
                                   float eps, const void* positions, int itype,
                                   const float* inv_freq, int64_t R, int interleaved,
                                   const dpz_heads* dq, const dpz_heads* dk, void* dwq, void* dwk,
                                   void* ws, void* stream);

/* Attention over B sequences packed one after another: q and out [Tq][Hq][D],
 * k and v [Tk][Hk][D], D <= 128, Hq a multiple of Hk (query head h reads key
 * head h / (Hq / Hk)).  Sequence b has queries [cu_q[b], cu_q[b+1]) and keys
 * [cu_k[b], cu_k[b+1]): offsets [B + 1] of type itype in device memory,
 * ascending, within [0, Tq] and [0, Tk] (values outside are taken as the
 * nearest bound; sequences that overlap give undefined results within the outputs).
 * cu_q and cu_k NULL: B sequences of Tq / B and Tk / B rows.
 *     s_ij = scale * q_i . k_j,   p = softmax_j(s),   out_i = sum_j p_ij v_j,
 *     lse[h][i] = log sum_j exp(s_ij)        (natural; fp32 [Hq][Tq] or NULL)
 * causal: of nq queries and nk keys, query i sees keys j <= i + nk - nq (the
 * last query sees all).  A query that sees no key has out 0 and lse -inf.
 * Rows outside every sequence are neither read nor written.  scale in (0, 1e30].
 * Scores, softmax and sums are fp32; for bf16 tensors the probabilities are
 * rounded to bf16 before their product with v, as operands of the tensor
 * cores.  A score of NaN or +inf makes its row NaN.  A value row that holds NaN or an
 * infinity may make NaN of any query of its sequence, also of one that the
 * causal mask keeps from seeing it (0 times infinity); keys and values behind a
 * sequence's end never do.
 * bf16 with addresses and strides that are multiples of 16 bytes runs on the
 * tensor cores. */
DPZ_API int attn_forward(const dpz_heads* q, const dpz_heads* k, const dpz_heads* v, int64_t Tq,
                         int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int dtype, int64_t B,
                         const void* cu_q, const void* cu_k, int itype, int causal, float scale,
                         const dpz_heads* out, float* lse, void* stream);

/* Bytes of device workspace of attn_grad; 0 for invalid sizes. */
DPZ_API size_t attn_grad_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hk,
                                         int64_t D);

/* Gradient of attn_forward's out: from its inputs, its out and lse, and dout
 * [Tq][Hq][D], the gradients dq, dk and dv.  The probabilities are computed again,
 * p_ij = exp(s_ij - lse_i):
 *     delta_i = dout_i . out_i,   ds_ij = p_ij (dout_i . v_j - delta_i)
 *     dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i,
 *     dv_j = sum_i p_ij dout_i
 * dk and dv are summed over the query heads that share a key head.  A query
 * that sees no key, or whose lse is -inf, has dq 0 and adds nothing.  For bf16
 * tensors p and ds are rounded to bf16 as operands of the tensor cores.  lse's own
 * rounding is an error of p of up to 2^-24 |lse|, relative.  ws:
 * attn_grad_workspace_bytes bytes, 16-byte aligned. */
DPZ_API int attn_grad(const dpz_heads* q, const dpz_heads* k, const dpz_heads* v,
                      const dpz_heads* out, const float* lse, const dpz_heads* dout, int64_t Tq,
                      int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int dtype, int64_t B,
                      const void* cu_q, const void* cu_k, int itype, int causal, float scale,
                      const dpz_heads* dq, const dpz_heads* dk, const dpz_heads* dv, void* ws,
                      void* stream);

/* ---------------------------------------------------------------------
 * The global norm and clip of a list of tensors
 *
 * dp_grad_global_norm and the step's clip work on an arena.  These calls do
 * the same for gradients that a program holds as separate tensors, of any
 * sizes and both types, and can write the clipped values into the arena's
 * slab on the way.
 * ------------------------------------------------------------------- */

#define DPZ_MAX_TENSORS 8192

/* A dense tensor of n elements in device memory (n = 0: p is not looked at).
 * The list itself is host memory, read during the call. */
typedef struct dpz_tensor {
    void* p;
    int64_t n;
    int64_t dtype; /* DPZ_F32 or DPZ_BF16 */
} dpz_tensor;

/* Bytes of device workspace of tensors_norm; 0 for an invalid list. */
DPZ_API size_t tensors_workspace_bytes(const dpz_tensor* tensors, int n);

/* *norm_out = sqrt(sum of the squares of all elements of n <= DPZ_MAX_TENSORS
 * tensors), fp32 in device memory.  Squares are taken and summed in fp32 within
 * 64 KB of a tensor by each thread, and in fp64 beyond, in an order that depends on the
 * list alone.  So an element beyond 1.8e19 gives +inf and one below 1e-23
 * nothing, as in dp_grad_global_norm; NaN gives NaN.  ws:
 * tensors_workspace_bytes bytes, 16-byte aligned. */
DPZ_API int tensors_norm(const dpz_tensor* tensors, int n, float* norm_out, void* ws,
                            void* stream);

/* out[i] = R(tensors[i] * s), s = clip_norm / *norm if *norm > clip_norm, else 1
 * (as in the AdamW step's clip; a NaN norm clips nothing).  out[i] has the
 * elements of tensors[i], of either type, and may be tensors[i] itself (same
 * address and type), which is then not written where s = 1.  Other overlaps of an output
 * are refused.  clip_norm > 0 and finite. */
DPZ_API int tensors_clip(const dpz_tensor* tensors, const dpz_tensor* out, int n,
                            const float* norm, float clip_norm, void* stream);

/* The calling thread's last error message ("" if none). */
DPZ_API const char* dpz_last_error(void);

/* Library version string. */
DPZ_API const char* dpz_version(void);

/* Device-side error flag of the current device, read and cleared: 1 if any
 * bulk-copy staged kernel (see DPZ_WS_STATUS_OFFSET) gave up on a tile, or any
 * attention kernel on a wait of its own (its rows of out or of the gradients are
 * then not written, and lse is NaN there), since the last call, else 0.  Synchronous: call it after the work in question has
 * finished (for example after cudaStreamSynchronize), not inside a stream
 * capture.  Returns DPZ_ERR_INVALID_ARG for a NULL flag_out, DPZ_ERR_CUDA if
 * the read fails. */
DPZ_API int dpz_device_status(int* flag_out);

/* Self-test of the timeout path (no counterpart on the pages).  Launches, on
 * `stream`, one of the staged kernels on a one-tile arena (N = 1, P = 8) laid
 * out in `buf`, DPZ_SELFTEST_BUF_BYTES bytes of caller device memory, 256-byte
 * aligned:
 *   +0     the arena's workspace (DPZ_WS_STATUS_OFFSET is relative to it)
 *   +2560  norm_out, one float
 *   +2816  gradients (bf16, 8 elements); +2848, +2880, +2912 master, m, v
 *          (fp32, 8 each); +2944 weights (bf16, 8)
 * The kernel's barrier expects 16 bytes more than its bulk loads deliver and
 * its wait is bounded by about 10^8 SM cycles (some 0.05 to 0.1 s) instead of
 * the usual two seconds.  Every copy it issues completes, so the wait runs out
 * and nothing is in flight when the kernel gives up.  kernel:
 *   DPZ_SELFTEST_UPDATE  the AdamW + all-gather update (without clip): sets
 *                        DPZ_STATUS_UPDATE_SKIPPED in the workspace's status
 *                        word and NaN in norm_out;
 *   DPZ_SELFTEST_NORM    the norm of the owner chunks, then the finalisation:
 *                        status DPZ_STATUS_NORM_SKIPPED, norm_out NaN;
 *   DPZ_SELFTEST_STEP    the step without clip with norm partials, then the
 *                        finalisation: status NORM_SKIPPED | UPDATE_SKIPPED,
 *                        norm_out NaN.
 * No kernel writes the arena's gradients, master/m/v or weights, and each
 * raises the device flag of dpz_device_status; the context stays usable.
 * Returns DPZ_ERR_INVALID_ARG for a NULL buf or an unknown kernel,
 * DPZ_ERR_ALIGN for a buf not 256-byte aligned, DPZ_ERR_CUDA if a launch
 * fails. */
#define DPZ_SELFTEST_BUF_BYTES 4096
#define DPZ_SELFTEST_UPDATE 0
#define DPZ_SELFTEST_NORM 1
#define DPZ_SELFTEST_STEP 2
DPZ_API int dpz_selftest_staged_timeout(int kernel, void* buf, void* stream);

/* Self-test of the division inside the average (no counterpart on the pages,
 * which fix only that the reduced sum is divided by N).  For N not a power of
 * two the library divides with Markstein's correction of a reciprocal
 * product instead of an IEEE division; this call checks that the two agree
 * for every float.  It sets, on `stream`, the 8-byte device counter
 * `mismatches` (caller memory, 16-byte aligned) to the number of (pattern,
 * path) cases, over all 2^32 float bit patterns a, where the library's
 * quotient a/N differs bit for bit from the IEEE round-to-nearest quotient
 * (two NaNs count as equal).  Each pattern is checked twice: in a group of
 * 8 consecutive patterns, as the streaming kernels divide them, and in a
 * group of 8 copies of itself.  0 means the average is correctly rounded for
 * this N.  It takes a few milliseconds.  Returns DPZ_ERR_INVALID_ARG for
 * N outside [1, DPZ_MAX_RANKS] or a NULL pointer, DPZ_ERR_ALIGN for one not 16-byte aligned,
 * DPZ_ERR_CUDA if the launch fails. */
DPZ_API int dpz_selftest_average_division(int N, unsigned long long* mismatches,
                                          void* stream);

/* Number of kernels this library has launched since it was loaded. */
DPZ_API int64_t dpz_launch_count(void);

/* Profiling: while on, every kernel launch is bracketed by a pair of CUDA
 * events recorded on the launch's own stream (capacity: max_launches
 * launches; later launches are not timed).  dpz_profile_stop synchronises
 * those events, fills up to max_stats per-kernel totals, sets *n_stats and
 * turns profiling off. */
DPZ_API int dpz_profile_start(int max_launches);
DPZ_API int dpz_profile_stop(dpz_kernel_stat* stats, int max_stats, int* n_stats);

#ifdef __cplusplus
}
#endif

#endif /* DPZ_H */
