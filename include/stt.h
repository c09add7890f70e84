/*
 * stt.h -- C ABI of the EAGLE-3 training-time-test (TTT) draft-step core on
 * NVIDIA GB300 (sm_103a).
 *
 * Two operations, as defined by the xllm-io review of "SpecForge: A Flexible
 * and Efficient Open-Source Training Framework for Speculative Decoding"
 * (cited as "SpecForge review"):
 *
 *  1. Sparse-tree TTT attention (SpecForge review, §三 "稀疏树注意力" and §四
 *     "BlockMask 构造").  At TTT step k the queries q attend to the
 *     concatenation of k+1 KV blocks (each Q_LEN rows) under the mask
 *         M = (q >= kv AND kv < T) OR
 *             (kv >= Q_LEN AND kv mod Q_LEN < T AND (kv - q) mod Q_LEN == 0)
 *     i.e. block 0 is causal with the padded columns kv >= T cut, and a query
 *     q < T additionally sees exactly key q of every later block j = 1..k.
 *     Queries q >= T ("padded rows") see the T keys kv < T and nothing else.
 *
 *  2. Masked soft-target softmax cross-entropy with the gradient written in
 *     place over the logits (SpecForge review, §三 "内存高效梯度计算", §四
 *     "掩码 Softmax 损失" / "原地反向传播"):
 *         pi = softmax(z_r), l_r = -sum_v p_rv log pi_rv,
 *         s_r = sum_v p_rv g_r,  z_rv <- -(p_rv g_r - pi_rv s_r),
 *         L = sum_r g_r l_r.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All tensor arguments are DEVICE pointers into memory the caller owns
 *    (cudaMalloc'd, or a framework's allocator); arrays of pointers and T are
 *    HOST arrays.  The library allocates no device memory, never synchronises
 *    the device, and enqueues all work on `stream` (a cudaStream_t passed as
 *    void*; NULL means the legacy default stream).
 *  - Argument errors are detected on the host before any launch and returned
 *    as a negative stt_status; nothing is enqueued in that case.  A CUDA
 *    launch error is returned as STT_ERR_CUDA.  No C++ exception crosses the
 *    ABI.  Functions are thread-safe; calls that share output buffers must be
 *    ordered by the caller.
 *  - Asynchronous device-side failures (a bounded wait that ran out inside a
 *    kernel) are recorded in a library-wide error word that
 *    stt_device_error() reads and clears.
 *  - Layouts are dense row-major (C order), innermost dimension last.
 */
#ifndef STT_H_
#define STT_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define STT_API __attribute__((visibility("default")))
#else
#define STT_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  STT_OK = 0,
  STT_ERR_INVALID_ARG = -1, /* null pointer, bad size, bad T, H % H_kv != 0 ... */
  STT_ERR_UNSUPPORTED = -2, /* valid but not implemented (e.g. D not 64/128)  */
  STT_ERR_MISALIGNED = -3,  /* a pointer is not 16-byte aligned               */
  STT_ERR_CUDA = -4,        /* a CUDA call failed (launch or driver)          */
  STT_ERR_TIMEOUT = -5,     /* a kernel's bounded wait ran out (device word)  */
  STT_ERR_WORKSPACE = -6    /* workspace missing or smaller than required     */
} stt_status;

/* Limits of this build. */
#define STT_MAX_BATCH 1024   /* B: T[] travels in the kernel parameters */
#define STT_MAX_STEP 31      /* k: at most 32 KV blocks                 */

/* Static, NUL-terminated description of a status code.  Thread-safe. */
STT_API const char* stt_status_string(int status);

/* Library version as 10000*major + 100*minor + patch. */
STT_API int stt_version(void);

/*
 * The cudaError_t code of the last CUDA failure (a status of STT_ERR_CUDA or
 * STT_ERR_UNSUPPORTED from a CUDA call) of a library call made by the calling
 * thread, 0 if none since the last read; reading clears it.  If `name` is not
 * NULL it receives the code's static name (cudaGetErrorName).  Every
 * launching entry point first clears an error that an earlier runtime call of
 * the same thread left pending, so a failure reported by the library is its
 * own.
 */
STT_API int stt_last_cuda_error(const char** name);

/*
 * Reads and clears the device-side error word (bitwise OR of the STT_DEVERR_*
 * sites whose bounded wait ran out since the last call).  Synchronises
 * `stream` first, then stores the word in *word and returns STT_ERR_TIMEOUT
 * if any STT_DEVERR_*_WAIT bit is set, STT_OK otherwise (the word is stored
 * in both cases), or STT_ERR_CUDA if the synchronisation or a read failed.
 */
STT_API int stt_device_error(void* stream, uint32_t* word);

/*
 * Failure-detection test hooks (no counterpart on the pages).  Every wait of
 * the kernels on an mbarrier is bounded by a wall-clock budget (2 s by
 * default); when it runs out, the waiting thread records its site in the
 * device error word and gives up, the other roles of the CTA give up in turn,
 * and the kernel returns (its outputs are then undefined).
 *
 * stt_debug_set_wait_budget(ns) sets that budget, in nanoseconds, on the
 * current device for every kernel of the library launched afterwards; 0
 * restores the default.  Returns STT_OK or STT_ERR_CUDA.
 *
 * stt_debug_inject(what) makes every later launch of the named kernels skip
 * one step on purpose, so that a bounded wait runs out without any fault:
 *   STT_INJECT_FWD_WITHHOLD_Q  the attention forward's producer never loads
 *                              the query tile, so the wait for it runs out;
 *                              every copy already issued is waited for before
 *                              the CTA exits, and no tensor-core product is
 *                              issued.
 *   STT_INJECT_LOGITS_WITHHOLD_PAIRS  the first CTA of a row that several share
 *                              does not send the others its maximum and sum.
 *   STT_INJECT_PAGED_WITHHOLD_Q  the paged attention's producer never loads
 *                              queries, as the attention forward's.
 *   STT_INJECT_CE_TOPK_WITHHOLD_PARTS  the first CTA of a row that several share
 *                              does not send the others its part of the soft-CE against
 *                              top logits.
 *   STT_INJECT_SLICE_WITHHOLD_COPIES  the first CTA of a row does not fetch its logits, in the
 *                              soft-CE against top logits and in sampling.
 * 0 switches injection off.  Unknown bits return STT_ERR_INVALID_ARG.  The
 * setting is process-wide; it is meant for tests, never for production runs.
 */
STT_API int stt_debug_set_wait_budget(uint64_t ns);
STT_API int stt_debug_inject(uint32_t what);
#define STT_INJECT_FWD_WITHHOLD_Q 0x1u
#define STT_INJECT_LOGITS_WITHHOLD_PAIRS 0x2u
#define STT_INJECT_PAGED_WITHHOLD_Q 0x4u
#define STT_INJECT_CE_TOPK_WITHHOLD_PARTS 0x8u
#define STT_INJECT_SLICE_WITHHOLD_COPIES 0x10u

/* --------------------------------------------------------------------------
 * Sparse-tree attention, forward.
 *
 *  q        bf16 [B, H, Q_LEN, D], the step-k queries.
 *  k_blocks host array of k+1 device pointers; k_blocks[j] is bf16
 *           [B, H_kv, Q_LEN, D], the keys of TTT block j (block 0 = causal).
 *  v_blocks host array of k+1 device pointers, same shape as k_blocks[j].
 *  T_host   host int32 [B], valid length of each sequence, 0 <= T[b] <= Q_LEN.
 *  B        1 <= B <= STT_MAX_BATCH.
 *  H, H_kv  query / KV heads; H % H_kv == 0; query head h reads KV head
 *           h / (H / H_kv).
 *  D        head dimension, 64 or 128.
 *  Q_LEN    block length, >= 1.
 *  k        TTT step, 0 <= k <= STT_MAX_STEP.
 *  scale    softmax scale applied to q.K (1/sqrt(D) in the usual case); finite
 *           and > 0 (STT_ERR_INVALID_ARG otherwise).
 *  out      bf16 [B, H, Q_LEN, D]: O = softmax(scale q Kc^T + mask) Vc,
 *           rounded to nearest even.  A row with no visible key (T[b] = 0)
 *           is written as zeros.
 *  lse      fp32 [B, H, Q_LEN]: natural-log logsumexp of the visible scaled
 *           scores (-inf for a row with no visible key).
 *  All device pointers must be 16-byte aligned (TMA requirement).
 * ------------------------------------------------------------------------ */
STT_API int stt_attn_fwd(const void* q, const void* const* k_blocks, const void* const* v_blocks,
                 const int32_t* T_host, int B, int H, int H_kv, int D, int Q_LEN, int k,
                 float scale, void* out, float* lse, void* stream);

/* Bytes of device workspace stt_attn_bwd needs for these sizes (>= 16). */
STT_API size_t stt_attn_bwd_workspace_size(int B, int H, int H_kv, int D, int Q_LEN, int k);

/* --------------------------------------------------------------------------
 * Sparse-tree attention, backward: the gradient of sum(O * dout) with respect
 * to q and every K/V block (the page trains through this attention; the
 * backward is the derivative of the definition, recomputing P from lse).
 *
 *  q, k_blocks, v_blocks, T_host, B, H, H_kv, D, Q_LEN, k, scale: as forward.
 *  out      bf16 [B, H, Q_LEN, D], the forward output.
 *  dout     bf16 [B, H, Q_LEN, D], upstream gradient of out.
 *  lse      fp32 [B, H, Q_LEN], the forward logsumexp.
 *  dq       fp32 [B, H, Q_LEN, D], OVERWRITTEN with dL/dq.
 *  dk_blocks host array of k+1 device pointers, fp32 [B, H_kv, Q_LEN, D],
 *           each OVERWRITTEN with dL/dK_j (summed over the query heads of the
 *           group; zero for rows no query sees).
 *  dv_blocks same for dL/dV_j.
 *  workspace device scratch of at least stt_attn_bwd_workspace_size() bytes,
 *           256-byte aligned; contents on entry are ignored.
 * ------------------------------------------------------------------------ */
STT_API int stt_attn_bwd(const void* q, const void* const* k_blocks, const void* const* v_blocks,
                 const int32_t* T_host, int B, int H, int H_kv, int D, int Q_LEN, int k,
                 float scale, const void* out, const void* dout, const float* lse, float* dq,
                 float* const* dk_blocks, float* const* dv_blocks, void* workspace,
                 size_t workspace_bytes, void* stream);

/* --------------------------------------------------------------------------
 * Sparse-tree attention, backward with options.  Same operation and
 * arguments as stt_attn_bwd, plus `flags`:
 *
 *  STT_BWD_ACCUMULATE_KV  dL/dK_j and dL/dV_j are ADDED to what dk_blocks[j]
 *           and dv_blocks[j] hold instead of overwriting them (dq is still
 *           overwritten).  This is the training use of the TTT step loop
 *           (SpecForge review, §三 "稀疏树注意力", TTT length 7, and §六
 *           "训练时测试（TTT）长度的影响"): block j is read by every step k >= j,
 *           so its gradient is the sum over those steps; each step's call adds
 *           its part in place, with no separate pass over the block gradients.
 *           Rows that no query of the step sees are left unchanged.
 *  STT_BWD_BF16_GRADS  dq, dk_blocks[j] and dv_blocks[j] are bf16 (round to
 *           nearest even) instead of fp32.  Sums across key tiles and heads
 *           are taken in fp32 in the workspace and rounded once at the end;
 *           with STT_BWD_ACCUMULATE_KV the existing bf16 value is added in fp32
 *           and the sum rounded once per call.
 *
 *  dq, dk_blocks, dv_blocks  device pointers of the element type the flags
 *           select, layouts as in stt_attn_bwd.
 *  workspace at least stt_attn_bwd_ex_workspace_size(..., flags) bytes,
 *           256-byte aligned (STT_ERR_MISALIGNED otherwise); contents on entry
 *           are ignored.
 * Unknown flag bits return STT_ERR_INVALID_ARG.  stt_attn_bwd is this call
 * with flags = 0.
 * ------------------------------------------------------------------------ */
#define STT_BWD_ACCUMULATE_KV 0x1u
#define STT_BWD_BF16_GRADS 0x2u
STT_API size_t stt_attn_bwd_ex_workspace_size(int B, int H, int H_kv, int D, int Q_LEN, int k,
                                              uint32_t flags);
STT_API int stt_attn_bwd_ex(const void* q, const void* const* k_blocks,
                            const void* const* v_blocks, const int32_t* T_host, int B, int H,
                            int H_kv, int D, int Q_LEN, int k, float scale, const void* out,
                            const void* dout, const float* lse, void* dq, void* const* dk_blocks,
                            void* const* dv_blocks, uint32_t flags, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Bytes of device workspace soft_ce_fwd_bwd_inplace needs (>= 16). */
STT_API size_t soft_ce_workspace_size(int64_t N, int64_t V);

/* --------------------------------------------------------------------------
 * Masked soft-target cross-entropy, loss and in-place gradient, one pass.
 *
 *  z        fp32 [N, V] logits; OVERWRITTEN with dL/dz = pi*s - p*g.
 *  p        fp32 [N, V] target distribution (rows need not sum to 1).
 *  g        fp32 [N] per-row upstream gradient / loss weight (mask / N).
 *  N        rows, >= 0.   V  vocabulary, >= 1.
 *  row_loss fp32 [N] or NULL: l_r = -sum_v p log softmax(z_r) for rows with
 *           g_r != 0, and 0 for rows with g_r == 0 (masked rows are not read).
 *  loss     fp32 scalar (device): L = sum_r g_r l_r, summed in a fixed order
 *           (deterministic).  0 when N == 0.
 *  workspace device scratch of at least soft_ce_workspace_size(N, V) bytes.
 *  Rows with g_r == 0 get an exact-zero gradient.  z and p should be 16-byte
 *  aligned with V % 4 == 0 for the bulk-copy path; other layouts take a
 *  slower element-wise path with identical results.
 * ------------------------------------------------------------------------ */
STT_API int soft_ce_fwd_bwd_inplace(float* z, const float* p, const float* g, int64_t N, int64_t V,
                            float* row_loss, float* loss, void* workspace,
                            size_t workspace_bytes, void* stream);

/* --------------------------------------------------------------------------
 * Soft-CE variants the formula admits (SpecForge review, §三 "内存高效梯度计算":
 * s = sum(p * g), z <- -(p * g - pi * s)).  `flags`:
 *
 *  STT_CE_BF16           z and p are bf16 [N, V]; every sum is taken in fp32
 *                        and the gradient is written over z rounded to bf16
 *                        (nearest even).
 *  STT_CE_G_PER_ELEMENT  g is fp32 [N, V], one upstream gradient per logit:
 *                            s_r = sum_v p_rv g_rv,  z_rv <- pi_rv s_r - p_rv g_rv,
 *                            row_loss_r = -sum_v g_rv p_rv log pi_rv,
 *                            L = sum_r row_loss_r
 *                        (row_loss is then already weighted, and every row is
 *                        read).
 * flags = 0 is soft_ce_fwd_bwd_inplace (fp32 z and p, per-row g).  Other
 * arguments, the workspace and the status codes as there; V may be at most
 * 16 slices of the shared memory a CTA can hold (above ~270000 for fp32 with
 * a per-element g) and STT_ERR_UNSUPPORTED is returned beyond that.  Unknown
 * flag bits return STT_ERR_INVALID_ARG.  Rows whose addresses are 16-byte
 * aligned with V % 8 == 0 take bulk copies; others an element-wise path with
 * identical results.
 * ------------------------------------------------------------------------ */
#define STT_CE_BF16 0x1u
#define STT_CE_G_PER_ELEMENT 0x2u
STT_API int soft_ce_fwd_bwd_inplace_ex(void* z, const void* p, const float* g, int64_t N,
                                       int64_t V, uint32_t flags, float* row_loss, float* loss,
                                       void* workspace, size_t workspace_bytes, void* stream);

/* --------------------------------------------------------------------------
 * Allocation-free soft-CE (the paper has no counterpart; this is a library
 * convenience).  Identical results to soft_ce_fwd_bwd_inplace, but it takes no
 * workspace: its per-row scratch is a fixed 256 KB array inside the library
 * (allocated when the library is loaded, held on every GPU that loads it until
 * the process exits).  It is for callers that cannot call cudaMalloc: for
 * example an operator plugged into a host framework that hands it only its
 * input and output buffers and owns all device memory itself, or code in a
 * phase where device allocation is not permitted.  The call itself allocates
 * nothing and calls no allocating routine.
 *
 *  z, p, g, N, V, row_loss, loss: as soft_ce_fwd_bwd_inplace.
 *  N must be <= 65536 rows (the scratch size); larger N returns
 *  STT_ERR_WORKSPACE without launching anything.
 *  Every call looks up the scratch array's device address on the current
 *  device (cudaGetSymbolAddress), so the address stays right after a
 *  cudaDeviceReset or a new primary context; the first call on a device also
 *  loads the library's kernels there, so make that first call before any
 *  stream capture.  All calls share the one array, so calls whose kernels
 *  overlap on the GPU (different streams, or threads without ordering) race
 *  on it and must be serialised by the caller.  Every scratch entry a call
 *  reads is written earlier in the same call, so the previous call's
 *  leftovers never affect the result.  Status codes are those of
 *  soft_ce_fwd_bwd_inplace (a CUDA failure the device does not support is
 *  STT_ERR_UNSUPPORTED, any other STT_ERR_CUDA).
 * ------------------------------------------------------------------------ */
STT_API int soft_ce_fwd_bwd_inplace_noalloc(float* z, const float* p, const float* g, int64_t N,
                                            int64_t V, float* row_loss, float* loss,
                                            void* stream);

/* --------------------------------------------------------------------------
 * The draft's LM head fused with the soft-CE, chunked over the vocabulary
 * (SpecForge review, §三 "内存高效梯度计算": the logits are the activation the
 * in-place gradient saves memory on; §四 "原地反向传播").  With hidden states
 * h, head weights W, targets p and per-row upstream gradients g:
 *     z = h W^T,  L = sum_r g_r l_r (l_r and dL/dz as soft_ce_fwd_bwd_inplace),
 *     dh = (dL/dz) W,  dW = (dL/dz)^T h.
 * The logits are never stored: a tensor-core pass computes per-row softmax
 * statistics from z tile by tile, and a second pass recomputes z one
 * vocabulary chunk at a time and turns it into dL/dz (bf16, in the
 * workspace), which feeds dh and dW at once.
 *
 *  h        bf16 [N, Hd] row-major.      W  bf16 [V, Hd] row-major.
 *  p        fp32 [N, V].                 g  fp32 [N].
 *  N >= 0; Hd and V multiples of 8 (STT_ERR_UNSUPPORTED otherwise), >= 8.
 *  dh       fp32 [N, Hd], OVERWRITTEN with dL/dh.
 *  dW       fp32 [V, Hd], OVERWRITTEN with dL/dW.
 *  row_loss fp32 [N] or NULL: l_r (0 for rows with g_r = 0).
 *  loss     fp32 scalar (device): L, summed in a fixed order.
 *  workspace at least stt_lm_head_ce_workspace_size(N, Hd, V) bytes,
 *           256-byte aligned; h, W, p, dh, dW 16-byte aligned.
 * dL/dz enters the two gradient products rounded to bf16 (as the operands of
 * any bf16 training step); sums are fp32.
 * ------------------------------------------------------------------------ */
STT_API size_t stt_lm_head_ce_workspace_size(int64_t N, int64_t Hd, int64_t V);
STT_API int stt_lm_head_ce(const void* h, const void* W, const float* p, const float* g,
                           int64_t N, int64_t Hd, int64_t V, float* dh, float* dW,
                           float* row_loss, float* loss, void* workspace,
                           size_t workspace_bytes, void* stream);

/* --------------------------------------------------------------------------
 * Speculative-decoding verification by rejection sampling (the "FlashSpec"
 * practice page, §3.4 "验证器的具体实现").  For each sequence b the draft's
 * tokens x_0..x_{gamma-1} are tested in order: x_i is accepted with
 * probability min(1, p_t[x_i] / p_d[x_i]), evaluated as
 * u_accept[b, i] * p_d < p_t in fp64 (a token with p_d = 0 is accepted iff
 * p_t > 0; a token outside [0, V) never).  At the first rejection one token
 * is drawn from norm(max(0, p_t - p_d)) at that position -- the smallest y
 * whose running residual sum (fp64) exceeds u_sample[b] times the total, or
 * from p_t itself if the residual is all zero -- and the sequence stops.
 * Nothing is drawn when every token is accepted.
 *
 *  p_target   fp32 [B, gamma, V]: the target model's distribution at each
 *             draft position.
 *  p_draft    fp32 [B, gamma, V]: the draft's distribution there.
 *  draft_tokens int32 [B, gamma].
 *  u_accept   fp32 [B, gamma], uniform in [0, 1): the acceptance draws.
 *  u_sample   fp32 [B], uniform in [0, 1): the resampling draw.
 *  B >= 0 (0 does nothing), 1 <= gamma <= STT_VERIFY_MAX_GAMMA, V >= 1.
 *  n_accepted int32 [B]: accepted draft tokens per sequence.
 *  out_tokens int32 [B, gamma]: the accepted tokens, then the drawn token if
 *             n_accepted < gamma, then -1.
 * All pointers device, 4-byte aligned (rows that are 16-byte aligned with
 * V % 4 == 0 are read with 16-byte loads).  V above 16 x 51200 returns
 * STT_ERR_UNSUPPORTED (a rejected row is split over at most 16 CTAs, each
 * holding its slice in shared memory).  The random numbers are inputs, so a
 * call is deterministic.
 * ------------------------------------------------------------------------ */
#define STT_VERIFY_MAX_GAMMA 32
STT_API int stt_verify(const float* p_target, const float* p_draft, const int32_t* draft_tokens,
                       const float* u_accept, const float* u_sample, int B, int gamma, int64_t V,
                       int32_t* n_accepted, int32_t* out_tokens, void* stream);

/* --------------------------------------------------------------------------
 * Query/key norm and position rotation.  The fused QKV projection gives each
 * token one row of H query heads, H_kv key heads and H_kv value heads of D
 * elements each.  For every query and key head x of a token at position t:
 *     x^  = x * (mean(x^2) + eps)^(-1/2),   n = x^ * w     (n = x if w is NULL)
 *     y_a = amplitude * (n_a cos(t f_i) - n_b sin(t f_i)),
 *     y_b = amplitude * (n_b cos(t f_i) + n_a sin(t f_i))
 * for the pairs i = 0..R/2-1 of the head's first R elements: (a, b) =
 * (i, i + R/2), or (2i, 2i + 1) with STT_ROPE_INTERLEAVED; elements R..D-1 are
 * y = n.  Values pass through.  Sums are fp32, y is rounded once.
 *
 * The frequencies are the caller's, so any scaling for long contexts is a
 * matter of the array.  Angles are exact for far positions: t f_i is reduced
 * modulo a full turn in 64-bit fixed point before its sine is taken.
 *
 *  freq     fp64 [R/2] (device): radians per position, finite; NULL iff R = 0.
 *  R        rotated elements of a head: a multiple of 16, 0 <= R <= D
 *           (0: norms only; STT_ERR_UNSUPPORTED for other values).
 *  flags    STT_ROPE_INTERLEAVED or 0.
 *  amplitude  finite; multiplies the rotated elements (1 in the usual case).
 *  w_q, w_k bf16 [D] (device) or NULL, each 16-byte aligned.
 *  eps      finite and > 0 where a weight is given.
 * ------------------------------------------------------------------------ */
#define STT_ROPE_INTERLEAVED 0x1u
typedef struct {
  const double* freq;
  const void* w_q;
  const void* w_k;
  int R;
  uint32_t flags;
  float amplitude;
  float eps;
} stt_rope;

/* --------------------------------------------------------------------------
 * Training form: projection rows to the attention's layout.
 *
 *  qkv      bf16, row b S + s at qkv + (b S + s) ld: heads in the order q, k, v.
 *  ld       elements between rows, >= (H + 2 H_kv) D, a multiple of 8.
 *  positions int32 [B, S] (device), any values, or NULL for 0..S-1.
 *  B, S >= 0; H, H_kv >= 1 (H need not be a multiple of H_kv here); D 64 or 128.
 *  q        bf16 [B, H, S, D];  k, v  bf16 [B, H_kv, S, D].
 * Device pointers 16-byte aligned (positions 4, freq 8).
 * ------------------------------------------------------------------------ */
STT_API int stt_qkv_rope_fwd(const void* qkv, int64_t ld, const int32_t* positions, int B, int S,
                             int H, int H_kv, int D, const stt_rope* rope, void* q, void* k,
                             void* v, void* stream);

/* Bytes of device workspace stt_qkv_rope_bwd needs (>= 16). */
STT_API size_t stt_qkv_rope_bwd_workspace_size(int D);

/* --------------------------------------------------------------------------
 * Its gradient.  With u the transposed rotation of dL/dy:
 *     dL/dw = sum over tokens and heads of u x^,
 *     dL/dx = r (u w - x^ mean(u w x^)),  r = (mean(x^2) + eps)^(-1/2)
 * (dL/dx = u without a weight).
 *
 *  dq, dk, dv  gradients of q, k, v in their layout, fp32 as stt_attn_bwd writes
 *           them, or bf16 with STT_ROPE_BF16_GRADS.
 *  qkv, ld  as forward; qkv may be NULL when neither weight is given.
 *  dqkv     bf16, rows ld_d elements apart (as ld), OVERWRITTEN: the operand
 *           of the projection's own gradient products, rounded once.
 *  dw_q, dw_k  fp32 [D], OVERWRITTEN; NULL exactly where the weight is NULL.
 *           Summed in an order fixed by the sizes and the device.
 *  workspace at least stt_qkv_rope_bwd_workspace_size(D) bytes, 16-byte aligned
 *           (NULL allowed when neither weight is given); contents on entry are
 *           ignored, calls that may overlap need one each.
 * ------------------------------------------------------------------------ */
#define STT_ROPE_BF16_GRADS 0x2u
STT_API int stt_qkv_rope_bwd(const void* dq, const void* dk, const void* dv, const void* qkv,
                             int64_t ld, const int32_t* positions, int B, int S, int H, int H_kv,
                             int D, const stt_rope* rope, uint32_t flags, void* dqkv, int64_t ld_d,
                             float* dw_q, float* dw_k, void* workspace, size_t workspace_bytes,
                             void* stream);

/* --------------------------------------------------------------------------
 * A paged KV cache and a ragged batch of new tokens on it, shared by
 * stt_kv_append and stt_paged_attn.  Everything but the sizes is read on the
 * device, so a captured call follows the batch as it changes.
 *
 *  k, v     bf16 caches: key x of page p, head h is the D elements at
 *           p stride_page + h stride_head + x stride_tok (elements; both caches
 *           alike).  16-byte aligned, strides multiples of 8.  Any order of the
 *           page's heads and tokens, and a k/v pair in one allocation, are a
 *           matter of the strides.
 *  table    int32 [B, max_pages]: page of keys x page_size.. of each sequence.
 *           Entries past a sequence's last page are not read.
 *  cu_q     int32 [B + 1], cu_q[0] = 0, nondecreasing: sequence b's new tokens
 *           are rows cu_q[b]..cu_q[b+1]-1 of the call's N rows.  A sequence may
 *           have none.  Rows from cu_q[B] on are left as they are.
 *  seq_lens int32 [B]: keys of each sequence, its new tokens among them; new
 *           token i of n is key seq_len - n + i.
 *  B        0 <= B <= STT_MAX_BATCH.   H_kv >= 1.   D 64 or 128.
 *  page_size a power of two, 8..1024 (STT_ERR_UNSUPPORTED otherwise).
 *  num_pages >= 1, max_pages >= 1; max_pages * page_size <= 2^30.
 *
 * A page outside [0, num_pages), or a key at or past max_pages * page_size, is
 * never read or written: it is skipped and reported as STT_DEVERR_PAGE in the
 * device error word, and the attention of that sequence is undefined.  A key
 * before 0 (a sequence with more new tokens than keys): stt_kv_append skips and
 * reports it too; stt_paged_attn reports nothing, there is no such key to see, and
 * a row whose own key lies there sees none (zeros, -inf) unless a tree's bit shows
 * it a later one.
 * ------------------------------------------------------------------------ */
typedef struct {
  void* k;
  void* v;
  const int32_t* table;
  const int32_t* cu_q;
  const int32_t* seq_lens;
  int64_t stride_page, stride_head, stride_tok;
  int B, H_kv, D, page_size, num_pages, max_pages;
} stt_pages;

/* --------------------------------------------------------------------------
 * Serving form of the norm and rotation: new tokens into the cache.
 *
 *  qkv      bf16 [N, .], rows ld elements apart, as stt_qkv_rope_fwd.
 *  positions int32 [N] or NULL: the rotation's position of each row where it is
 *           not its key index (the depth of a token in a draft tree).
 *  N        rows, >= 0.
 *  q        bf16 [N, H, D]: the normed and rotated queries.
 * Two rows of one call may not have the same key slot.
 * ------------------------------------------------------------------------ */
STT_API int stt_kv_append(const void* qkv, int64_t ld, const int32_t* positions, int64_t N, int H,
                          const stt_pages* pages, const stt_rope* rope, void* q, void* stream);

/* Bytes of device workspace stt_paged_attn needs (>= 16). */
STT_API size_t stt_paged_attn_workspace_size(int64_t N, int B, int H, int H_kv, int D);

/* --------------------------------------------------------------------------
 * Attention of the new tokens over their sequences' pages, whose new keys are
 * already there (stt_kv_append).  New token i of a sequence with n new tokens
 * and L keys sees keys 0..L-n+i, or, with `tree`, keys 0..L-n-1 and those of the
 * n new ones whose bit is set in its row.
 *
 *  q        bf16, row r at q + r ld_q: H heads of D; ld_q >= H D, a multiple
 *           of 8.  Query head h reads KV head h / (H / H_kv); H % H_kv == 0,
 *           H / H_kv <= 16.
 *  N        rows, >= 0, N H < 2^31.
 *  scale    finite and > 0.
 *  tree     uint32 [N, tree_words] or NULL: bit j % 32 of word j / 32 of a row
 *           is set iff it sees new token j of its sequence (itself only if its
 *           own bit is set).  New tokens from 32 tree_words on are not seen.
 *  out      bf16 [N, H, D], rounded to nearest even; zeros for a row that sees
 *           nothing.  May not overlap q.
 * Slots behind a sequence's last key may hold anything.  The values of its own keys
 * must be finite even where a row does not see them (they meet a zero probability);
 * keys that a row does not see may hold anything.
 *  lse      fp32 [N, H] or NULL: natural logarithm of the sum of exponentials
 *           of the visible scaled scores, -inf for a row that sees nothing.
 *  workspace at least stt_paged_attn_workspace_size() bytes, 256-byte aligned;
 *           contents on entry are ignored.  Calls that may overlap (two
 *           streams, two graphs) need one each.
 * ------------------------------------------------------------------------ */
STT_API int stt_paged_attn(const void* q, int64_t ld_q, int64_t N, int H, const stt_pages* pages,
                           float scale, const uint32_t* tree, int tree_words, void* out,
                           float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* --------------------------------------------------------------------------
 * Logits to the distributions stt_verify tests against.  Rows come `rows` to a
 * sequence: row r is position i = r % rows of sequence b = r / rows.  With c the
 * number of times token v occurs in the sequence's output so far:
 *     z <- z > 0 ? z / repetition : z * repetition   if v occurs in its history
 *     z <- z - frequency * c - presence * [c > 0]
 *     z <- z + bias,   z <- -inf where the mask forbids v
 *     out = softmax(z / temperature)
 * The history of row (b, i) is tokens[cu_tokens[b]..cu_tokens[b+1]), the first
 * n_prompt[b] of them the prompt and the rest output, and then the draft's
 * tokens 0..i-1, output too.  Tokens outside [0, V) count for nothing.  (The draft
 * is a chain, as in stt_verify; each path of a tree goes as a sequence of its own.)
 *
 *  z        fp32 [N, V], or bf16 with STT_LOGITS_BF16.  A forbidden element may
 *           hold anything; NaN or +inf elsewhere makes its row's probabilities
 *           NaN (greedy: NaN is passed over).
 *  N        rows, >= 0, a multiple of `rows` >= 1.   V  >= 1.
 *  temperature, repetition, frequency, presence  fp32 [N / rows] or NULL (1, 1,
 *           0, 0).  temperature = 0 is greedy: the distribution is 1 at the
 *           largest z (the lowest such v) and 0 elsewhere.  That all are finite,
 *           temperature >= 0 and repetition > 0 is the caller's to see to.
 *  tokens, cu_tokens, n_prompt  int32; all NULL without a history (n_prompt
 *           NULL alone: no prompt).  n_tokens: length of tokens, past which
 *           nothing is read.
 *  draft    int32 [N / rows, draft_ld] or NULL; draft_ld >= rows - 1.
 *  bias     fp32 [bias_rows, V]; bias_rows 0 (none), 1, or N / rows.
 *  mask     uint32 [N, ceil(V / 32)] or NULL: bit v % 32 of word v / 32 set iff
 *           row r allows v.
 *  out      fp32 [N, V]; may be z itself when that is fp32.  With
 *           STT_LOGITS_RAW it receives z / temperature instead (z itself where
 *           temperature is 0).  A row with nothing allowed gets zeros (-inf raw).
 * V above 16 x 24576 returns STT_ERR_UNSUPPORTED.
 * ------------------------------------------------------------------------ */
#define STT_LOGITS_BF16 0x1u
#define STT_LOGITS_RAW 0x2u
typedef struct {
  const float* temperature;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* tokens;
  const int32_t* cu_tokens;
  const int32_t* n_prompt;
  const int32_t* draft;
  const float* bias;
  const uint32_t* mask;
  int n_tokens;
  int draft_ld;
  int bias_rows;
} stt_logits;
STT_API int stt_logits_process(const void* z, int64_t N, int64_t V, int rows,
                               const stt_logits* params, uint32_t flags, float* out,
                               void* stream);

/* --------------------------------------------------------------------------
 * The K largest logits of every row, the largest first and the lower index first
 * among equals, with the row's log-sum-exp: a teacher's targets as they are stored
 * for training (soft_ce_topk_fwd_bwd reads them), or the candidates that a draft
 * tree grows by (values[k] / temperature - lse is a candidate's log-probability).
 *
 *  z        fp32 [N, V], or bf16 with STT_LOGITS_BF16; rows ld_z elements apart,
 *           any alignment of the element.  -inf is never taken (a forbidden
 *           token); NaN counts as the largest, and makes the row's lse NaN, as
 *           +inf does.
 *  N        rows, >= 0.   V  1..STT_ROW_MAX_V.   K  1..min(V, STT_TOP_MAX_K)
 *           (K > V is STT_ERR_INVALID_ARG).
 *  temperature  finite and at least 2^-126; of lse alone.
 *  values   fp32 [N, K]: logits as they are, -inf past the row's last.
 *  indices  int32 [N, K], -1 past the row's last.
 *  lse      fp32 [N] or NULL: log sum_v exp(z_v / temperature); -inf for a row
 *           without logits.
 * ------------------------------------------------------------------------ */
#define STT_ROW_MAX_V (16 * 45056)
#define STT_TOP_MAX_K 1024
STT_API int stt_top_logits(const void* z, int64_t ld_z, int64_t N, int64_t V, int K,
                           float temperature, uint32_t flags, float* values, int32_t* indices,
                           float* lse, void* stream);

/* --------------------------------------------------------------------------
 * Soft-CE against a teacher's top logits, loss and gradient: the target
 * distribution is K logits a row (SpecForge review, §三 "内存高效梯度计算", with the
 * targets kept as their top entries in place of [N, V]).  With tau = temperature:
 *     p_k = exp(t_values[k] / tau - L),  s = sum_k p_k,  pi = softmax(z / tau)
 *     l_r = s log sum_v exp(z_v / tau) - sum_k p_k z[t_indices[k]] / tau
 *     L = sum_r g_r l_r,   dz_v = g_r / tau (s pi_v - sum_{k: t_indices[k] = v} p_k)
 *
 *  z        fp32 [N, V], or bf16 with STT_CE_BF16; rows ld_z elements apart.
 *  t_values fp32 [N, K];  t_indices int32 [N, K].  An entry whose index lies
 *           outside [0, V) is none (so is one of -inf); entries of one token add up.
 *  t_lse    fp32 [N]: the teacher's log sum_v exp(t_v / tau) over its whole row, as
 *           stt_top_logits gives it: p are then the teacher's probabilities and s
 *           their sum (0 under an lse of +inf).  NULL: over the row's entries alone,
 *           s = 1.
 *  g        fp32 [N], as soft_ce_fwd_bwd_inplace: rows with g_r = 0 are not read,
 *           their gradient and row_loss are 0.
 *  N        rows, >= 0.   V  1..STT_ROW_MAX_V.   K  1..STT_TOP_MAX_K.
 *  temperature  finite and at least 2^-126; that g_r / temperature is finite is the
 *           caller's to see to.
 *  dz       the gradient, of z's type, rows ld_dz apart, OVERWRITTEN, rounded once.
 *           It may be z (with ld_dz = ld_z); otherwise it may not overlap z.
 *  row_loss fp32 [N] or NULL;  loss  fp32 scalar (device), summed in a fixed order.
 *  workspace at least soft_ce_workspace_size(N, V) bytes, as soft_ce_fwd_bwd_inplace.
 * A logit of -inf has probability 0; its loss is +inf where the teacher's is not 0.
 * A row of -inf alone is left out (gradient and row_loss 0); NaN or +inf in a row
 * makes its gradient and loss NaN.
 * ------------------------------------------------------------------------ */
STT_API int soft_ce_topk_fwd_bwd(const void* z, int64_t ld_z, const float* t_values,
                                 const int32_t* t_indices, const float* t_lse, const float* g,
                                 int64_t N, int64_t V, int K, float temperature, uint32_t flags,
                                 void* dz, int64_t ld_dz, float* row_loss, float* loss,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* --------------------------------------------------------------------------
 * Logits to the distribution that temperature, top-k, top-p and min-p leave, and a
 * token drawn from it with a given random number: the draft's tokens with the
 * p_draft that stt_verify tests them against, the target's p_target (stt_logits_process
 * with STT_LOGITS_RAW before it where there are penalties, and no temperature here),
 * or plain decoding.  Rows come `rows` to a sequence, as there.
 *
 * The order of a row's tokens is by logit, the largest first, the lower index first
 * among equals.  Kept are, of that order, the first top_k; of those the shortest
 * beginning that holds top_p of their probability, at least one token; of those the
 * ones at least min_p times as probable as the first.
 *     probs_v = e^(z_v / temperature) / (its sum over the kept),  0 for the others
 *     token   = the smallest v with probs_0 + .. + probs_v > u
 * A token less than 2^-63 times as probable as the first may count as 0.
 *
 *  z        fp32 [N, V], or bf16 with STT_LOGITS_BF16; rows ld_z elements apart.
 *           -inf is a forbidden token.
 *  N        rows, >= 0, a multiple of `rows` >= 1.   V  1..STT_ROW_MAX_V.
 *  temperature, top_p, min_p  fp32 [N / rows], top_k  int32 [N / rows]; each may be
 *           NULL (1, 1, 0, off).  temperature = 0, like top_k = 1, keeps the first
 *           token alone; top_k <= 0 or >= V, top_p >= 1 and min_p <= 0 cut nothing,
 *           top_p <= 0 leaves one token, and min_p > 1 counts as 1.
 *           That none is NaN and temperature >= 0 is the caller's to see to.
 *  u        fp32 [N] in [0, 1), or NULL: nothing is drawn (tokens and logprobs NULL).
 *           Weights have 31 bits; their running sums, and u times the whole, are exact.
 *  tokens   int32 [N].   logprobs  fp32 [N] or NULL: log probs[token].
 *  probs    fp32, rows ld_probs elements apart, or NULL (with u); may be z where that
 *           is fp32 (with ld_probs = ld_z), otherwise it may not overlap z.
 * A row with nothing allowed gives token -1, logprob -inf and probabilities 0; one with
 * NaN or +inf gives -1, NaN and NaN.
 * ------------------------------------------------------------------------ */
STT_API int stt_sample(const void* z, int64_t ld_z, int64_t N, int64_t V, int rows,
                       const float* temperature, const int32_t* top_k, const float* top_p,
                       const float* min_p, const float* u, uint32_t flags, int32_t* tokens,
                       float* logprobs, float* probs, int64_t ld_probs, void* stream);

/* --------------------------------------------------------------------------
 * Per-launch timing (measurement support; no counterpart on the pages).
 * stt_profile_start(capacity) makes every subsequent kernel launch of the
 * library (from any thread) record a CUDA event pair around itself on its
 * launch stream, for up to `capacity` launches.  stt_profile_stop() waits for
 * the recorded events, writes up to `capacity` (kernel id, milliseconds)
 * pairs into the caller's host arrays (either may be NULL), stores the count
 * in *n and disables recording.  Events are host-side objects: no device
 * memory is allocated.  Returns STT_ERR_INVALID_ARG when not in the right
 * state, STT_ERR_CUDA if an event call failed.
 * ------------------------------------------------------------------------ */
STT_API int stt_profile_start(int capacity);
STT_API int stt_profile_stop(int* n, int* kernel_ids, float* ms, int capacity);
/* Static name of a kernel id ("attn_fwd", ...). */
STT_API const char* stt_kernel_name(int kernel_id);

#define STT_KERNEL_SOFT_CE 1
/* The soft-CE row kernel and its loss sum are recorded together as
 * STT_KERNEL_SOFT_CE; STT_KERNEL_SOFT_CE_LOSS_SUM only names the second. */
#define STT_KERNEL_SOFT_CE_LOSS_SUM 2
#define STT_KERNEL_ATTN_FWD 3
#define STT_KERNEL_ATTN_BWD_PREP 4
#define STT_KERNEL_ATTN_BWD_CAUSAL 5
#define STT_KERNEL_ATTN_BWD_CAST 6
#define STT_KERNEL_SOFT_CE_VARIANT 7
#define STT_KERNEL_VERIFY 8
#define STT_KERNEL_LM_HEAD_CE 9
#define STT_KERNEL_QKV_ROPE 10
#define STT_KERNEL_QKV_ROPE_BWD 11
#define STT_KERNEL_KV_APPEND 12
#define STT_KERNEL_PAGED_ATTN 13
#define STT_KERNEL_LOGITS 14
#define STT_KERNEL_TOP_LOGITS 15
#define STT_KERNEL_SOFT_CE_TOPK 16 /* with its loss sum, as STT_KERNEL_SOFT_CE */
#define STT_KERNEL_SAMPLE 17

/* Device error-word bits: sites of bounded waits that gave up, and blocks
 * whose dynamic shared memory did not have the 1024-byte alignment the
 * swizzled tiles need (such a block skips its work). */
#define STT_DEVERR_FWD_WAIT 0x1u
#define STT_DEVERR_BWD_WAIT 0x2u
#define STT_DEVERR_CE_WAIT 0x4u
#define STT_DEVERR_SMEM_ALIGN 0x8u
#define STT_DEVERR_LM_WAIT 0x10u
#define STT_DEVERR_PAGE 0x20u /* a page or key slot out of range, skipped */
#define STT_DEVERR_PAGED_WAIT 0x40u
#define STT_DEVERR_LOGITS_WAIT 0x80u
#define STT_DEVERR_SAMPLE_WAIT 0x100u
#define STT_DEVERR_WAIT_MASK                                                           \
  (STT_DEVERR_FWD_WAIT | STT_DEVERR_BWD_WAIT | STT_DEVERR_CE_WAIT | STT_DEVERR_LM_WAIT | \
   STT_DEVERR_PAGED_WAIT | STT_DEVERR_LOGITS_WAIT | STT_DEVERR_SAMPLE_WAIT)

#ifdef __cplusplus
}
#endif

#endif /* STT_H_ */
