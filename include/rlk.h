/*
 * rlk.h -- C ABI of the deterministic, batch-invariant selected-token
 * log-probability operator `linear_logp` for NVIDIA GB300 (sm_103a).
 *
 * Operation ("Announcing RL-Kernel for vime", section "Key Capabilities", first
 * bullet, and the operator boundary "hidden + lm_head_weight + target_ids ->
 * selected logprob" in section "Why the Fused Path Wins"):
 *
 *   z[t][v]  = h[t] . W[v]                        (bf16 inputs, fp32 accumulation)
 *   lse[t]   = log sum_{v < V_true} exp(z[t][v])   (columns >= V_true are masked:
 *              "true vocabulary range", table "Boundary Fixes in the RL-Kernel
 *              Strict Path", row "Linear logprob", of "vLLM RL-Kernel v0.1.0:
 *              Bitwise Train-Rollout Consistency on ROCm")
 *   logp[t]  = z[t][y[t]] - lse[t]
 *
 * computed without materialising the [T, V] logits (the fused kernel keeps
 * running max / sum-exp / target-logit statistics while it walks vocab tiles,
 * second reason in "Why the Fused Path Wins"). The backward returns dH and dW of
 * L = sum_t g[t] * logp[t] ("Full-gradient support" bullet), recomputing the
 * logits tile by tile and forming dz = g * (onehot - softmax).
 *
 * Numerical contract (the six observables of "The Numerical Execution
 * Contract" in the ROCm consistency article, fixed here once for every shape):
 *  1. Input dependency: logp[t], lse[t] and dH[t] depend only on h[t], y[t], W,
 *     V_true (and g[t], lse[t] for dH[t]); never on T, on other rows, on the
 *     stream, on the launch shape or on the GPU's SM count.
 *  2. Partitioning: the hidden dimension is reduced in steps of 64 (one K=16
 *     tensor-core instruction at a time, ascending). The vocabulary is cut into
 *     leaves of RLK_LEAF_WIDTH = 1024 global columns, each walked in 256-column
 *     tiles in ascending order. No split-K, no atomics on data (one atomic
 *     counter per launch only hands out work items; which CTA pair computes an
 *     output tile never changes how it is computed).
 *  3. Merge order: leaves are merged by a balanced pairwise tree defined on
 *     global leaf indices: nLeaves = ceil(V_true / 1024) leaves are grouped into
 *     RLK_MAX_SHARDS = 8 super-shards of L = ceil(nLeaves / 8) leaves; inside a
 *     super-shard the leaves sit in P = next_pow2(L) slots (missing leaves are
 *     the identity) and are merged pairwise; the 8 super-shard results are then
 *     merged pairwise (8 -> 4 -> 2 -> 1). Because the tree depends only on V_true,
 *     a vocab-sharded run (S in {1, 2, 4, 8} contiguous shards, each a
 *     power-of-two-aligned run of super-shards) followed by rlk_lse_merge gives
 *     bit-identical logp and lse to the unsharded run.
 *  4. Precision: bf16 inputs; fp32 accumulation, statistics, logp and lse; dz
 *     is rounded once to bf16 (it is an operand of the dH/dW products); dH is
 *     rounded once to bf16 from its fp32 accumulator; dW is fp32.
 *  5. Rounding: every floating-point step is an explicitly rounded operation
 *     (round-to-nearest fmul / fadd / fma); nothing is left to compiler contraction.
 *  6. Primitives: e(x) = ex2.approx.ftz(fma(x, log2 e, -rn(b * log2 e))) for
 *     exp(x - b) everywhere; log is logf (fp32, CUDA math library).
 *
 * Conventions for every entry point:
 *  - The caller owns every buffer. The library allocates and frees nothing and
 *    keeps no state between calls (apart from per-device kernel attributes),
 *    so calls are re-entrant.
 *  - All work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) with no host synchronisation. Device pointers must be valid in the
 *    current CUDA context.
 *  - Argument errors are returned before anything is launched; T == 0 returns
 *    RLK_OK and launches nothing (per-token pointers may then be NULL). A
 *    launch failure returns RLK_ERR_CUDA.
 *  - Row-major, contiguous tensors. h, W and dz-style bf16 rows need a 16-byte
 *    aligned base and H % 8 == 0 (tensor-memory-access strides).
 *  - Targets outside [0, V_true) cannot be checked on the host without a sync:
 *    their logp is NaN, their gradient row is zero, and RLK_FLAG_BAD_TARGET is
 *    ORed into *err_flag when err_flag is not NULL.
 *  - Every internal wait of a kernel is bounded; on expiry the kernel stops,
 *    ORs RLK_FLAG_TIMEOUT into *err_flag (if given) and the outputs are invalid.
 */
#ifndef RLK_H_
#define RLK_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define RLK_API __attribute__((visibility("default")))
#else
#define RLK_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  RLK_OK = 0,
  RLK_ERR_INVALID_ARG = 1, /* null pointer, negative size, misaligned pointer, H % 8 != 0 */
  RLK_ERR_UNSUPPORTED = 2, /* a shard split the fixed merge tree cannot express; sizes beyond limits */
  RLK_ERR_WORKSPACE = 3,   /* workspace missing or smaller than the query returns */
  RLK_ERR_CUDA = 4         /* a CUDA runtime/driver call failed (launch, tensor-map encode) */
} rlk_status;

/* bits ORed into *err_flag by the kernels */
#define RLK_FLAG_BAD_TARGET 1
#define RLK_FLAG_TIMEOUT 2
#define RLK_FLAG_NONFINITE 4 /* rlk_quantize_rows_e4m3: a row held a NaN or an infinity; operators over
                                logits: a row held a NaN or +inf */
#define RLK_FLAG_BOUNDS 8    /* debug-checks builds only: an index or tensor-copy coordinate
                                check failed; the access was skipped (see rlk_debug_checks) */

/* tiling constants that are part of the numerical contract */
#define RLK_LEAF_WIDTH 1024
#define RLK_MAX_SHARDS 8

/* size limits (RLK_ERR_UNSUPPORTED beyond them) */
#define RLK_MAX_VOCAB (1 << 24)
#define RLK_MAX_HIDDEN (1 << 16)

/*
 * Per-token statistics of one vocab shard, natural-log units: m is the largest
 * logit of the shard's valid columns, s = sum exp(z - m) over them, zt the
 * target logit if the shard owns y[t], else -inf (NaN for an invalid target).
 * The identity (empty shard) is {-inf, 0, -inf}. Layout: 12 bytes, no padding.
 * ("Why the Fused Path Wins", third reason: only statistics cross shards.)
 */
typedef struct {
  float m;
  float s;
  float zt;
} rlk_lse_partial;

/* Bytes of device workspace rlk_linear_logp_fwd needs (256-byte aligned base): the
 * per-(token, leaf) statistics, then 256 bytes of work-item counters that the call
 * zeroes on its stream before its kernels use them. */
RLK_API size_t rlk_linear_logp_fwd_workspace(int64_t T, int64_t H, int64_t V_local);

/*
 * Forward. The shard holds W rows for global vocab columns
 * [vocab_start, vocab_start + V_local); the unsharded call is vocab_start = 0,
 * V_local = V >= V_true.
 *
 *   h        device bf16 [T][H]
 *   W        device bf16 [V_local][H] (this shard's rows)
 *   y        device int64 [T], global vocab ids
 *   V_true   global true-vocab bound; columns >= V_true are masked
 *   logp,lse device fp32 [T] each, or NULL; used when partial == NULL, which
 *            requires the shard to cover [0, V_true)
 *   partial  device rlk_lse_partial [T] or NULL: when given, the call writes
 *            this shard's triple per token instead of logp / lse; combine the
 *            shards with rlk_lse_merge
 *   err_flag device int32 or NULL (RLK_FLAG_* bits are ORed in, never cleared)
 *   workspace, workspace_bytes: device scratch of at least
 *            rlk_linear_logp_fwd_workspace(T, H, V_local) bytes, 256-byte aligned
 *
 * A shard must start at a multiple of the super-shard width
 * L * RLK_LEAF_WIDTH (L = ceil(ceil(V_true / 1024) / 8)), cover n = ceil(V_local /
 * (L * 1024)) super-shards with n a power of two and vocab_start / (L * 1024) a
 * multiple of n, and contain every column of those super-shards below V_true;
 * otherwise RLK_ERR_UNSUPPORTED.
 */
RLK_API rlk_status rlk_linear_logp_fwd(const void* h, const void* W, const int64_t* y, int64_t T,
                               int64_t H, int64_t V_local, int64_t vocab_start, int64_t V_true,
                               float* logp, float* lse, rlk_lse_partial* partial,
                               int32_t* err_flag, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * Merge S per-shard triples per token (partials laid out [S][T], shards in
 * ascending vocab order) by the top levels of the fixed tree, then
 * lse = m + log(s), logp = zt - lse. S must be 1, 2, 4 or 8. logp, lse: device
 * fp32 [T]. ("vLLM RL-Kernel v0.1.0 ... on ROCm", "Boundary Fixes" table,
 * "Linear logprob" row: cross-rank LSE merge; fixed merge order, item 3 of
 * "The Numerical Execution Contract".)
 */
RLK_API rlk_status rlk_lse_merge(const rlk_lse_partial* partials, int32_t S, int64_t T, float* logp,
                         float* lse, void* stream);

/* Bytes of device workspace rlk_linear_logp_bwd needs: the bf16 dz tile store
 * [T][round_up(V_local, 256)] (the "controlled workspace" of the fourth reason
 * in "Why the Fused Path Wins"), plus, when V_local > 65536, an fp32 [T][H]
 * running sum for dH's chunked accumulation, plus 256 bytes of work-item counters
 * (zeroed by the call on its stream). */
RLK_API size_t rlk_linear_logp_bwd_workspace(int64_t T, int64_t H, int64_t V_local);

/*
 * Backward of L = sum_t g[t] logp[t] for one shard (or the whole vocabulary).
 *
 *   h, W, y, T, H, V_local, vocab_start, V_true: as in the forward
 *   lse      device fp32 [T], the GLOBAL log-sum-exp from the forward / merge
 *   g        device fp32 [T], upstream gradient
 *   dH       device [T][H] or NULL: bf16 when dH_fp32_partial == 0, else fp32
 *            (a shard's partial; sum the shards with rlk_shard_sum_bf16)
 *   dW       device fp32 [V_local][H] or NULL; rows at or above V_true get 0
 *   err_flag, workspace, workspace_bytes, stream: as in the forward
 *
 * dz[t][v] = g[t] (1[v == y[t]] - exp(z[t][v] - lse[t])) is recomputed from a
 * fresh z tile with the forward's exact tensor-core sequence, rounded once to
 * bf16; dH = dz W sums the vocabulary in ascending 64-column steps, dW = dz^T h
 * sums the tokens in ascending 64-row steps, each output tile by one CTA pair.
 * Both reductions run in fixed chunks of 65536 (tensor-core fp32 accumulation
 * within a chunk, then round-to-nearest fp32 adds of the chunk results in
 * ascending order), which keeps the accumulation bias of very long reductions
 * bounded; the chunking depends on neither T's batch composition nor the launch.
 */
RLK_API rlk_status rlk_linear_logp_bwd(const void* h, const void* W, const int64_t* y, const float* lse,
                               const float* g, int64_t T, int64_t H, int64_t V_local,
                               int64_t vocab_start, int64_t V_true, void* dH,
                               int32_t dH_fp32_partial, float* dW, int32_t* err_flag,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same backward, launched in separate stages. The backward's three products
 * meet in its workspace ("tiled logits / dlogits and linear-gradient work ... with
 * a controlled workspace", "Announcing RL-Kernel for vime", section "Why the Fused
 * Path Wins", fourth reason): the dz tiles are written there once and read by both
 * gradient products. `stages` is a nonzero OR of
 *   RLK_BWD_DZ  recompute the logits and write dz into the workspace
 *   RLK_BWD_DH  dH = dz W from the dz the workspace holds (dH must not be NULL)
 *   RLK_BWD_DW  dW = dz^T h from the dz the workspace holds (dW must not be NULL)
 * and every other argument is as in rlk_linear_logp_bwd. A stage launches the kernel
 * that rlk_linear_logp_bwd launches for it, on the same operands in the same work order
 * (only how it follows the launch before it differs), so stages run one call at a time
 * in the order DZ, DH, DW with one workspace give the bits of a single
 * rlk_linear_logp_bwd call. The workspace must stay untouched
 * from the DZ call until the last call that reads its dz. Each stage has its own
 * work-item counter in the workspace and only RLK_BWD_DH uses its fp32 running sum,
 * so once the DZ stage has completed, the DH and DW stages may run on two streams
 * at the same time. Uses: pipeline schedules that need the input gradient dH at once
 * and defer the weight gradient dW; timing each stage on its own.
 */
#define RLK_BWD_DZ 1
#define RLK_BWD_DH 2
#define RLK_BWD_DW 4

RLK_API rlk_status rlk_linear_logp_bwd_stages(const void* h, const void* W, const int64_t* y,
                                              const float* lse, const float* g, int64_t T,
                                              int64_t H, int64_t V_local, int64_t vocab_start,
                                              int64_t V_true, void* dH, int32_t dH_fp32_partial,
                                              float* dW, int32_t stages, int32_t* err_flag,
                                              void* workspace, size_t workspace_bytes,
                                              void* stream);

/*
 * Saved-logits variant of the pair above: the forward also stores the fp32
 * logits it computed and the backward forms dz from them instead of recomputing
 * the logits GEMM (the "save-logits fused-tile full-gradient path" named in
 * "Announcing RL-Kernel for vime", section "Validation and Benchmarks"). The
 * saved logits are the accumulator values bit for bit and dz uses the same
 * arithmetic, so logp, lse, dH and dW are bit-identical to the recompute path;
 * the price is rlk_saved_logits_bytes of device memory between the two calls.
 *
 *   z_saved  device fp32 [T][round_up(V_local, 256)], 16-byte aligned, caller-owned;
 *            written by rlk_linear_logp_fwd_save for the shard's columns below
 *            V_true, read by rlk_linear_logp_bwd_saved; z_saved_bytes must be at
 *            least rlk_saved_logits_bytes(T, V_local) (else RLK_ERR_INVALID_ARG)
 * Every other argument is as in rlk_linear_logp_fwd / rlk_linear_logp_bwd.
 */
RLK_API size_t rlk_saved_logits_bytes(int64_t T, int64_t V_local);

RLK_API rlk_status rlk_linear_logp_fwd_save(const void* h, const void* W, const int64_t* y,
                                            int64_t T, int64_t H, int64_t V_local,
                                            int64_t vocab_start, int64_t V_true, float* logp,
                                            float* lse, rlk_lse_partial* partial, float* z_saved,
                                            size_t z_saved_bytes, int32_t* err_flag,
                                            void* workspace, size_t workspace_bytes, void* stream);

RLK_API rlk_status rlk_linear_logp_bwd_saved(const void* h, const void* W, const int64_t* y,
                                             const float* lse, const float* g,
                                             const float* z_saved, size_t z_saved_bytes, int64_t T,
                                             int64_t H, int64_t V_local, int64_t vocab_start,
                                             int64_t V_true, void* dH, int32_t dH_fp32_partial,
                                             float* dW, int32_t* err_flag, void* workspace,
                                             size_t workspace_bytes, void* stream);

/*
 * Saved-probabilities variant (the bf16 "save probs" option of the pages'
 * linear_logp settings, "Announcing RL-Kernel for vime", section "Quick Start"):
 * the forward stores, for every logit, e(z - m) rounded to bf16 together with the
 * row's fp32 running max m after each 64-column chunk, and the backward forms
 * p = e(z - m) * e(m - lse) from them. Half the memory of the saved logits; dz
 * carries an extra relative error of at most 2^-9 (bf16) per element, so dH / dW
 * are NOT bit-identical to the recompute path (logp and lse are).
 *
 *   p_saved  device buffer of rlk_saved_probs_bytes(T, V_local) bytes, 256-byte
 *            aligned, caller-owned: bf16 [T][round_up(V_local, 256)], then fp32
 *            [T][round_up(V_local, 256) / 64] at a 256-byte aligned offset
 * Every other argument is as in rlk_linear_logp_fwd / rlk_linear_logp_bwd.
 */
RLK_API size_t rlk_saved_probs_bytes(int64_t T, int64_t V_local);

RLK_API rlk_status rlk_linear_logp_fwd_save_probs(const void* h, const void* W, const int64_t* y,
                                                  int64_t T, int64_t H, int64_t V_local,
                                                  int64_t vocab_start, int64_t V_true,
                                                  float* logp, float* lse,
                                                  rlk_lse_partial* partial, void* p_saved,
                                                  size_t p_saved_bytes, int32_t* err_flag,
                                                  void* workspace, size_t workspace_bytes,
                                                  void* stream);

RLK_API rlk_status rlk_linear_logp_bwd_saved_probs(const void* h, const void* W, const int64_t* y,
                                                   const float* lse, const float* g,
                                                   const void* p_saved, size_t p_saved_bytes,
                                                   int64_t T, int64_t H, int64_t V_local,
                                                   int64_t vocab_start, int64_t V_true, void* dH,
                                                   int32_t dH_fp32_partial, float* dW,
                                                   int32_t* err_flag, void* workspace,
                                                   size_t workspace_bytes, void* stream);

/*
 * out[i] = bf16(((p[0][i] + p[1][i]) + p[2][i]) + ...), the fixed ascending-order
 * sum of S fp32 partials laid out [S][n], rounded once to bf16 (RNE). Used to
 * combine per-shard dH partials. partials, out: device, 16-byte aligned.
 */
RLK_API rlk_status rlk_shard_sum_bf16(const float* partials, int32_t S, int64_t n, void* out,
                              void* stream);

/*
 * FP8 LM head. An RL trainer whose rollouts run an FP8 output layer reproduces it
 * in the training forward: the weights are quantized to FP8 again at every
 * forward, both sides use one quantization rounding rule and one batch-invariant
 * GEMM for every batch size, and the backward takes gradients for the bf16 master
 * weights with the quantization treated as the identity (straight-through
 * estimator) (AREX feed article on vLLM's bitwise-consistent RL training, sections
 * "训练前向直接调用推理内核" and "对齐的代价：逐算子拆解"). The pages fix neither the
 * FP8 format nor the scale granularity; this library uses OCP E4M3 (no infinities,
 * largest magnitude 448) with one power-of-two scale per row, so a token's codes
 * never depend on the rest of the batch and quantization is exactly reproducible.
 *
 * rlk_quantize_rows_e4m3: for each row r of x (bf16 [rows][cols], device, 16-byte
 * aligned, cols % 8 == 0):
 *   e       = the smallest integer with max_k |x[r][k]| <= 448 * 2^e (0 if the row is all zero)
 *   scale[r] = 2^e                                   (fp32 [rows], device)
 *   q[r][k]  = E4M3 code nearest to x[r][k] / 2^e, ties to even (uint8 [rows][cols], device,
 *             16-byte aligned)
 * A row holding a NaN or an infinity gets scale NaN and zero codes, and
 * RLK_FLAG_NONFINITE is ORed into *err_flag (device int32, or NULL). rows == 0 or
 * cols == 0 launches nothing. Asynchronous on `stream`; argument errors are returned
 * before any launch.
 */
RLK_API rlk_status rlk_quantize_rows_e4m3(const void* x, int64_t rows, int64_t cols, void* q,
                                          float* scale, int32_t* err_flag, void* stream);

/*
 * FP8 forward: the forward of rlk_linear_logp_fwd on E4M3 operands,
 *   z[t][v] = (sum_k hq[t][k] * Wq[v][k]) * h_scale[t] * W_scale[v]
 * (products exact, fp32 tensor-core accumulation over K in ascending 128-element
 * steps, then the two power-of-two scales), with the same fixed merge tree, shard
 * statistics, masking, outputs and errors.
 *   hq       E4M3 codes [T][H] (device, 16-byte aligned), h_scale fp32 [T]
 *   Wq       E4M3 codes [V_local][H] (device, 16-byte aligned), W_scale fp32 [V_local]
 *            (device, 16-byte aligned)
 * as produced by rlk_quantize_rows_e4m3; H % 16 == 0. Workspace: as
 * rlk_linear_logp_fwd_workspace(T, H, V_local).
 */
RLK_API rlk_status rlk_linear_logp_fwd_fp8(const void* hq, const float* h_scale, const void* Wq,
                                           const float* W_scale, const int64_t* y, int64_t T,
                                           int64_t H, int64_t V_local, int64_t vocab_start,
                                           int64_t V_true, float* logp, float* lse,
                                           rlk_lse_partial* partial, int32_t* err_flag,
                                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * Straight-through FP8 backward: dz[t][v] = g[t] (1[v = y[t]] - e(z[t][v] - lse[t]))
 * with z the E4M3 logits of rlk_linear_logp_fwd_fp8 (recomputed tile by tile, the
 * same bits as that forward's), then dH = dz W and dW = dz^T h with the bf16
 * operands h, W exactly as in rlk_linear_logp_bwd (outputs, shard partials, workspace
 * rlk_linear_logp_bwd_workspace(T, H, V_local), errors). hq, h_scale, Wq, W_scale as
 * in rlk_linear_logp_fwd_fp8; lse is the FP8 forward's.
 */
RLK_API rlk_status rlk_linear_logp_bwd_fp8(const void* h, const void* W, const void* hq,
                                           const float* h_scale, const void* Wq,
                                           const float* W_scale, const int64_t* y,
                                           const float* lse, const float* g, int64_t T, int64_t H,
                                           int64_t V_local, int64_t vocab_start, int64_t V_true,
                                           void* dH, int32_t dH_fp32_partial, float* dW,
                                           int32_t* err_flag, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * Operators over logits that already exist, next to the fused head: a serving engine has
 * them after sampling, rlk_linear_logp_fwd_save leaves them as saved logits. All of them
 * take the rows' scaled logits x = s z, s = 1 / temperature (rounded once to fp32), over the
 * columns below V_true; what the columns at and beyond V_true hold is never read. Common
 * arguments:
 *   logits   device [T][ld] of type dtype (RLK_DTYPE_*), rows `ld` elements apart, aligned to
 *            its element size only (rows of an odd length may start anywhere)
 *   ld       row distance in elements, at least V_true
 *   V_true   1 .. RLK_MAX_LOGITS_VOCAB
 *   temperature  RLK_MIN_TEMPERATURE .. RLK_MAX_TEMPERATURE
 *   err_flag device int32 or NULL, as everywhere
 * Numerical contract: fp32 statistics in one fixed order over column indices (leaves of 1024
 * columns about their own maximum, then all leaves about the row's), so every output of a row
 * depends on that row's inputs alone: not on T, on the other rows, on alignment or strides, on
 * the launch shape or on the GPU's SM count. e^x = ex2.approx.ftz(x log2 e), log is logf.
 * Log probabilities (logp, top_logp and those in the distillation loss) are formed as
 * s (z - M) - log S about the row's maximum M, S = sum e^{s (z - M)}, and are as good for logits far
 * from zero -- an offset, a low temperature, a row masked wholly by a finite value -- as for others; they
 * are never above 0; entropy is never below 0. lse = s M + log S is one fp32: it loses 2^-24 |lse|, and where s M is beyond
 * fp32's range (bf16 or fp32 logits of the type's lowest value at a temperature below 1, say) it is
 * +inf or, below, fp32's lowest value: -inf marks an empty row alone.
 * The gradients take log p = s z - lse from the caller's lse while what it has lost is small against
 * what p has lost anyway: up to |lse| = 4096 for a gradient in bf16, 512 in f16, 256 in fp32. Rows beyond
 * that are read once more for M and log S, several times slower (8192 rows of 151936 in bf16, all of
 * them so: 4.0 ms instead of 0.71); rlk_distill_topk_fwd_bwd has both at hand where it runs in one launch.
 * Nothing needs a workspace. T == 0 returns RLK_OK and launches nothing.
 *
 * Special rows. -inf logits are masked columns: probability 0. A row of nothing but -inf has
 * lse -inf, logp -inf, entropy 0, no alternatives, and a zero gradient. A row with a NaN or
 * +inf below V_true has NaN in lse, logp, entropy and loss, rank 0, no alternatives (id -1, log
 * probability NaN), a zero gradient, and RLK_FLAG_NONFINITE is ORed into *err_flag. A target
 * outside [0, V_true) has logp NaN, rank 0 and a zero gradient row, and RLK_FLAG_BAD_TARGET is
 * ORed in.
 */
typedef enum { RLK_DTYPE_BF16 = 0, RLK_DTYPE_F16 = 1, RLK_DTYPE_F32 = 2 } rlk_dtype;

#define RLK_MAX_TOP_K 128
#define RLK_MAX_LOGITS_VOCAB (1 << 20)
#define RLK_MAX_LOGITS_ROWS (1 << 28)
#define RLK_MIN_TEMPERATURE 1e-6
#define RLK_MAX_TEMPERATURE 1e6

/*
 * Log probabilities of given tokens, with entropy and top alternatives. Per row t:
 *   lse      = log sum_v e^{x_v}
 *   logp     = x_y - lse
 *   rank     = 1 + #{v : z_v > z_y, or z_v = z_y and v < y}     (1: the most likely token)
 *   entropy  = -sum_v p_v log p_v,  p_v = e^{x_v - lse}
 *   top_ids, top_logp: the top_k best columns in the order of rank and their x_v - lse
 *            (so a token of rank r <= top_k stands in place r - 1); places beyond the columns
 *            that are not -inf hold id -1 and -inf
 *   y        device int64 [T], or NULL (then logp and rank must be NULL)
 *   logp, lse, entropy  device fp32 [T], rank device int32 [T], each may be NULL
 *   top_k    0 .. RLK_MAX_TOP_K; top_ids device int64 [T][top_k] and top_logp device fp32
 *            [T][top_k], both given when top_k > 0
 */
RLK_API rlk_status rlk_token_logprobs(const void* logits, int32_t dtype, int64_t T, int64_t ld,
                                      int64_t V_true, double temperature, const int64_t* y,
                                      int32_t top_k, float* logp, int32_t* rank, float* lse,
                                      float* entropy, int64_t* top_ids, float* top_logp,
                                      int32_t* err_flag, void* stream);

/*
 * Gradient of sum_t (g_logp[t] logp[t] + g_entropy[t] entropy[t]) with respect to the logits:
 *   dlogits[t][v] = s (g_logp (1[v = y] - p_v) - g_entropy p_v (log p_v + entropy))
 * in fp32 and rounded once to out_dtype; columns V_true .. V - 1 get 0. A row whose two
 * gradients are 0 gets zeros whatever its logits hold (padding tokens).
 *   lse, entropy  device fp32 [T], as rlk_token_logprobs gave them (entropy may be NULL when
 *            g_entropy is); g_logp device fp32 [T]; g_entropy device fp32 [T] or NULL
 *   dlogits  device [T][out_ld] of type out_dtype, out_ld >= V >= V_true: the logits' type, or
 *            RLK_DTYPE_BF16 for fp32 logits. The first round_up(V_local, 256) * T elements of
 *            rlk_linear_logp_bwd's workspace are such an array (bf16, V = out_ld =
 *            round_up(V_local, 256)): with dlogits there, RLK_BWD_DH and RLK_BWD_DW of
 *            rlk_linear_logp_bwd_stages give this loss's dH and dW. dlogits may be the logits
 *            themselves (same type, base and row distance). Else no row of one may meet a
 *            row of the other: the arrays' address ranges are apart, or the rows are the same
 *            number of bytes apart and lie side by side (column slices of one wider buffer).
 */
RLK_API rlk_status rlk_token_logprobs_bwd(const void* logits, int32_t dtype, int64_t T, int64_t ld,
                                          int64_t V_true, double temperature, const int64_t* y,
                                          const float* lse, const float* entropy,
                                          const float* g_logp, const float* g_entropy,
                                          void* dlogits, int32_t out_dtype, int64_t V,
                                          int64_t out_ld, int32_t* err_flag, void* stream);

/*
 * Distillation from a teacher's top logits. q = softmax(s t_k) over the row's entries, and
 *   loss[t] = sum_k q_k (log q_k - (x_{id_k} - lse))       (the KL divergence from q to p)
 *   dlogits[t][v] = s g[t] (p_v - sum_{k : id_k = v} q_k)  of sum_t g[t] loss[t]
 * (no factor temperature^2: a caller who wants gradients of one size at every temperature has it in g).
 * (teacher log probabilities serve as well as logits: q does not change under a shift).
 *   ids      device int64 [T][K], K in 1 .. RLK_MAX_TOP_K; id -1: no entry (as rlk_token_logprobs
 *            marks missing alternatives); an id may come twice, then both count
 *   teacher  device fp32 [T][K]; -inf: probability 0
 *   g        device fp32 [T]
 *   loss, lse  device fp32 [T]; lse (of the student's logits) feeds the backward; in
 *            rlk_distill_topk_fwd it may be NULL
 * A row without entries (or with all teacher values -inf) has loss 0 and a zero gradient. A row
 * with an id outside [-1, V_true) (RLK_FLAG_BAD_TARGET) or a teacher value of NaN or +inf
 * (RLK_FLAG_NONFINITE) has loss NaN and a zero gradient. Where the student's logit of an entry
 * with q > 0 is -inf the loss is +inf. dlogits, out_dtype, V, out_ld as in
 * rlk_token_logprobs_bwd, with rows of g = 0 zero.
 *
 * rlk_distill_topk_fwd_bwd gives both at once, for weights g that are known before the loss (a
 * token mask over a count): the same bits as the two calls. The logits are read once for rows of up to
 * 53248 columns in 16-bit types and 13312 in fp32, and for longer ones where they are few: up to
 * 608 rows of 106496 (53248 in fp32), 304 of 212992 (106496). Else they are read twice, which is faster there.
 */
RLK_API rlk_status rlk_distill_topk_fwd(const void* logits, int32_t dtype, int64_t T, int64_t ld,
                                        int64_t V_true, double temperature, const int64_t* ids,
                                        const float* teacher, int32_t K, float* loss, float* lse,
                                        int32_t* err_flag, void* stream);

RLK_API rlk_status rlk_distill_topk_bwd(const void* logits, int32_t dtype, int64_t T, int64_t ld,
                                        int64_t V_true, double temperature, const int64_t* ids,
                                        const float* teacher, int32_t K, const float* lse,
                                        const float* g, void* dlogits, int32_t out_dtype, int64_t V,
                                        int64_t out_ld, int32_t* err_flag, void* stream);

RLK_API rlk_status rlk_distill_topk_fwd_bwd(const void* logits, int32_t dtype, int64_t T, int64_t ld,
                                            int64_t V_true, double temperature, const int64_t* ids,
                                            const float* teacher, int32_t K, const float* g,
                                            float* loss, float* lse, void* dlogits,
                                            int32_t out_dtype, int64_t V, int64_t out_ld,
                                            int32_t* err_flag, void* stream);

/*
 * Operators around the head in a training step: what turns tokens into the first hidden values and the
 * last ones into h, each with its gradient, and the norm of all gradients. The table of an embedding is a
 * [V][H] array like W; a tied model has one for both, and its dW is the head's with the embedding's added.
 * Common arguments:
 *   dtype    RLK_DTYPE_* of the rows; results have the same type, or RLK_DTYPE_BF16 for fp32 rows
 *   H        1 .. RLK_MAX_HIDDEN; rows `ld` elements apart (at least H), aligned to their element size only.
 *            Rows that all start on 16-byte boundaries (fp32 ones, weight, bias and dW on 32-byte ones), with
 *            H % 8 == 0, are the fast case
 *   T        0 .. RLK_MAX_TOKENS
 *   err_flag device int32 or NULL, as everywhere
 *   workspace, workspace_bytes: device scratch of the size that the query returns, 256-byte aligned; what it
 *            holds before a call does not matter
 * A result may not meet an input, but for the cases that an entry point names: the arrays are apart, or
 * their rows are the same number of bytes apart and lie side by side (column slices of one wider buffer).
 * Numerical contract: fp32 sums in fixed orders that follow from columns, and for sums over tokens from the
 * order of the tokens, so that a result never depends on alignment, strides, the launch shape or the GPU's SM count;
 * a row of a lookup, of a norm or of dx depends on that row's inputs alone, and a row of an embedding's dW on that
 * token's rows alone.
 */
#define RLK_MAX_TOKENS (1 << 24)

/*
 * out[t] = scale * table[ids[t] - vocab_start], the product in fp32 (scale as well), then rounded to out_dtype: the rows of a
 * table, or of a shard of one that holds the tokens [vocab_start, vocab_start + V_local).
 *   table    device [V_local][ld];  ids: device int64 [T];  out: device [T][out_ld]
 *   V_true   tokens are 0 .. V_true - 1
 * The row of a token that is not in the shard is zero, and so is that of id -1 (padding); any other id outside
 * [0, V_true) gets a row of NaN, and RLK_FLAG_BAD_TARGET is ORed into *err_flag.
 */
RLK_API rlk_status rlk_embedding_fwd(const void* table, int32_t dtype, int64_t V_local, int64_t H, int64_t ld,
                                     int64_t vocab_start, int64_t V_true, const int64_t* ids, int64_t T, double scale,
                                     void* out, int32_t out_dtype, int64_t out_ld, int32_t* err_flag, void* stream);

/* Bytes of device workspace rlk_embedding_bwd needs; 0 (and workspace may be NULL) for up to 256 tokens. Beyond, with n = T / 16 + 1 and
 * H rounded up to 8: the sorted tokens and their runs (32 T + 16 bytes), the sums of tokens that come more than 16 times (8 n H) and
 * counters of those sums (12 n for every 256 columns begun, beyond 2048 columns for every 2048 begun 8 times that), each of the five arrays
 * rounded up to 256 bytes. */
RLK_API size_t rlk_embedding_bwd_workspace(int64_t T, int64_t H);

/*
 * The table's gradient: dW[v - vocab_start] = scale * sum of dout[t] over the t with ids[t] = v.
 *   dout     device [T][ld] of type dtype;  ids: device int64 [T]
 *   dW       device fp32 [V_local][H], as rlk_linear_logp_bwd writes it (any 4-byte alignment)
 *   accumulate  0: dW is written, with zeros in the rows of tokens that do not come; 1: the gradient is added to what dW
 *            holds (a tied model's head has been there), one rounding an element, and other rows are not touched
 * Ids of -1 and of other shards add nothing; any other id outside [0, V_true) adds nothing and ORs RLK_FLAG_BAD_TARGET
 * in. A token's rows are added in the order of t, in runs of 16, the runs' sums in groups of 8, and the groups' sums:
 * the order does not depend on the other tokens or on the shard. T == 0 with accumulate == 0 writes zeros.
 */
RLK_API rlk_status rlk_embedding_bwd(const void* dout, int32_t dtype, int64_t T, int64_t H, int64_t ld,
                                     const int64_t* ids, int64_t V_local, int64_t vocab_start, int64_t V_true,
                                     double scale, float* dW, int32_t accumulate, int32_t* err_flag, void* workspace,
                                     size_t workspace_bytes, void* stream);

/*
 * Layer norm of each row:
 *   y_c = (x_c - mean) rstd weight_c + bias_c,   rstd = (mean_c (x_c - mean)^2 + eps)^(-1/2)
 * or, with centered == 0, the same with mean = 0 (the root-mean-square norm).
 *   x        device [T][ld] of type dtype;  y: device [T][out_ld] of type out_dtype, which may be x itself
 *   weight, bias  device [H] of type weight_dtype (the rows' type or RLK_DTYPE_F32), either may be NULL
 *   eps      RLK_MIN_NORM_EPS .. 1
 *   mean, rstd  device fp32 [T], for the backward; either may be NULL
 * The variance is summed about the mean, which is corrected by what its own rounding lost; rows whose sums are beyond
 * fp32 are summed once more at a smaller scale. A row that holds a NaN or an infinity is NaN throughout, and
 * RLK_FLAG_NONFINITE is ORed into *err_flag.
 */
#define RLK_MIN_NORM_EPS 1e-18

RLK_API rlk_status rlk_layer_norm_fwd(const void* x, int32_t dtype, int64_t T, int64_t H, int64_t ld,
                                      const void* weight, const void* bias, int32_t weight_dtype, int32_t centered,
                                      double eps, void* y, int32_t out_dtype, int64_t out_ld, float* mean, float* rstd,
                                      int32_t* err_flag, void* stream);

/* Bytes of device workspace rlk_layer_norm_bwd needs: 8 T bytes, and the parts of dw and db of every strip of rows (below). */
RLK_API size_t rlk_layer_norm_bwd_workspace(int64_t T, int64_t H);

/*
 * Gradients of the layer norm, with h = (x - mean) rstd and g = dy weight:
 *   dx_c = rstd (g_c - mean_c g - h_c mean_c(g h)),   dw_c = sum_t dy h,   db_c = sum_t dy
 * (without the term mean_c g when the norm is not centered).
 *   dy       device [T][dy_ld] of type dy_dtype (the forward's out_dtype)
 *   x, dtype, ld, T, H, weight, weight_dtype: as in the forward
 *   mean, rstd  device fp32 [T] from the forward; mean NULL: not centered
 *   dx       device [T][dx_ld] of type dtype, or NULL; it may be dy or x itself (same type and row distance)
 *   dw, db   device fp32 [H], each may be NULL; at least one of dx, dw and db is wanted. T == 0 writes zeros to them
 * Rows are dealt to S strips, row t to strip t mod S, with S = T, or 304, 608, 1216 and 2432 for H above 2048, 1024, 512 and
 * otherwise where T is larger; a strip adds its rows in ascending order. Of the strips' sums, those of strips i, i + 32, ... are
 * added in ascending order, and the 32 results as a balanced tree. Finite rows of any size have the h of their statistics: a row that
 * differs from its mean by more than fp32 holds is halved first. The mean is the forward's, rounded to fp32: h carries half a step of
 * mean rstd. Sums of dy weight, and of their products with h, are to stay inside fp32. A row whose x, dy or statistics hold a NaN
 * makes that row of dx and all or those columns of dw and db NaN, whatever its dy: rows of padding are to hold finite values in both.
 */
RLK_API rlk_status rlk_layer_norm_bwd(const void* dy, int32_t dy_dtype, int64_t dy_ld, const void* x, int32_t dtype,
                                      int64_t ld, int64_t T, int64_t H, const void* weight, int32_t weight_dtype,
                                      const float* mean, const float* rstd, void* dx, int64_t dx_ld, float* dw,
                                      float* db, int32_t* err_flag, void* workspace, size_t workspace_bytes,
                                      void* stream);

/*
 * The 2-norm over all elements of n tensors, and gradients scaled so that it is at most max_norm:
 *   norm = sqrt(sum g^2),   out = g if norm <= max_norm, else g (max_norm / norm)
 *   grads, sizes, dtypes  host arrays of n: device pointers (aligned to their element size only), element counts
 *            (0 .. RLK_MAX_TENSOR_ELEMENTS), RLK_DTYPE_*; read before the call returns
 *   n        0 .. RLK_MAX_TENSORS
 *   outs, out_dtypes  host arrays of n: where the results go (same count; same type, or RLK_DTYPE_BF16 for fp32), a
 *            gradient itself among them. Results meet neither one another nor any other gradient
 *   max_norm above 0 (infinity: never scaled)
 *   norm     device fp32 [1]: the norm before scaling; with outs, it meets no gradient and no result
 * Squares that would overflow or vanish in fp32 are summed at another scale. A norm that is not finite (a NaN or an
 * infinity among the gradients, or a norm beyond fp32) leaves the gradients unscaled, and RLK_FLAG_NONFINITE is ORed
 * into *err_flag: a trainer skips that step. It is NaN where there is a NaN, and infinite otherwise. Sums are taken in an order that
 * follows from sizes and types.
 */
#define RLK_MAX_TENSORS (1 << 14)
#define RLK_MAX_TENSOR_ELEMENTS ((int64_t)1 << 40)

RLK_API size_t rlk_grad_norm_workspace(int32_t n);

RLK_API rlk_status rlk_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                                 float* norm, int32_t* err_flag, void* workspace, size_t workspace_bytes, void* stream);

RLK_API rlk_status rlk_clip_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                                      double max_norm, void* const* outs, const int32_t* out_dtypes, float* norm,
                                      int32_t* err_flag, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Forward without a workspace argument, for callers that cannot allocate device
 * memory: runtimes whose device memory is fully reserved up front by another
 * allocator (a serving engine that pre-plans every buffer), or latency-critical
 * loops where cudaMalloc / cudaFree would synchronise the device and stall the
 * other streams. The pages have no counterpart to this entry point.
 *
 * Same arguments, results and errors as rlk_linear_logp_fwd, minus workspace and
 * workspace_bytes. The scratch it needs instead is one static device array of
 * RLK_FWD_NOALLOC_SCRATCH_BYTES (16 MiB), held by every GPU that loads the library
 * until the process exits; the call itself allocates nothing. A shape whose
 * rlk_linear_logp_fwd_workspace(T, H, V_local) exceeds that size is rejected with
 * RLK_ERR_WORKSPACE before anything runs (e.g. at most 9383 tokens for a 151936-row
 * W). The first call on a device looks up the array's device address (with that
 * device current) and keeps it for the life of the process; make that first call
 * before any stream capture. Calling it after cudaDeviceReset on that device is not
 * supported (the array may then live at another address). All calls on a
 * device share the array: calls that can overlap on the GPU (different streams with
 * no ordering between them) race and give wrong results.
 */
#define RLK_FWD_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

RLK_API rlk_status rlk_linear_logp_fwd_noalloc(const void* h, const void* W, const int64_t* y,
                                               int64_t T, int64_t H, int64_t V_local,
                                               int64_t vocab_start, int64_t V_true, float* logp,
                                               float* lse, rlk_lse_partial* partial,
                                               int32_t* err_flag, void* stream);

/*
 * Self-test of the kernels' bounded waits. Runs the unsharded forward (arguments
 * as rlk_linear_logp_fwd with vocab_start = 0) with the first shared-memory stage
 * of one CTA deliberately left unfilled, so the pipeline's first wait can never
 * complete. After the wait limit (2 s) the kernel gives up: it raises its abort
 * flag in both CTAs of the pair, drains the copies and tensor-core work already in
 * flight, frees its tensor memory, ORs RLK_FLAG_TIMEOUT into *err_flag (required)
 * and returns; the kernel takes about 4 s and logp / lse are undefined. No fault,
 * trap or hang is involved, and the CUDA context stays usable afterwards.
 */
RLK_API rlk_status rlk_selftest_wait_timeout(const void* h, const void* W, const int64_t* y,
                                             int64_t T, int64_t H, int64_t V, int64_t V_true,
                                             float* logp, float* lse, int32_t* err_flag,
                                             void* workspace, size_t workspace_bytes,
                                             void* stream);

/*
 * Debug-checks builds. The library can also be compiled with device-side checks
 * (RLK_DEBUG_CHECKS=1; `python -m deterministic_token_logprob_gb300.build --debug-checks`
 * writes _build_debug/librlk.so): before every global-memory access whose address the
 * kernels compute from an index (statistics, saved maxima, running sums, plain output
 * stores, the dz passes, the leaf-tree reads) they check the index against the extent of
 * the buffer, and before every tensor copy they check the rules of its coordinates (the
 * innermost one a multiple of 16 bytes, a store's never negative). A failed check ORs
 * RLK_FLAG_BOUNDS into *err_flag instead of trapping and skips the access (a load's
 * misaligned coordinate is rounded down instead, so the pipeline's byte counts still
 * complete), so the context stays usable. Results of a build with checks are bit-identical
 * to the plain build's.
 *
 * rlk_debug_checks: 1 for a library built with the checks, else 0.
 * rlk_selftest_bounds_check: the unsharded forward (arguments as rlk_linear_logp_fwd) told
 * that its statistics workspace is one (token, leaf) entry shorter than it is, so the last
 * entry's store and read fail their checks: afterwards *err_flag (required) holds
 * RLK_FLAG_BOUNDS, and every access stayed inside the real buffers. logp / lse are
 * undefined. Without the checks it returns RLK_ERR_UNSUPPORTED and launches nothing.
 */
RLK_API int32_t rlk_debug_checks(void);

RLK_API rlk_status rlk_selftest_bounds_check(const void* h, const void* W, const int64_t* y,
                                             int64_t T, int64_t H, int64_t V, int64_t V_true,
                                             float* logp, float* lse, int32_t* err_flag,
                                             void* workspace, size_t workspace_bytes,
                                             void* stream);

/* Static description of a status code. */
RLK_API const char* rlk_status_string(rlk_status s);

/* Library version string, e.g. "rlk 0.1.0 sm_103a". */
RLK_API const char* rlk_version(void);

#ifdef __cplusplus
}
#endif

#endif /* RLK_H_ */
