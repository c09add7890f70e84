// internal.h -- declarations shared by the host-side ABI (stt_api.cu) and the
// kernel translation units.  Not part of the public interface.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace stt {

// ------------------------------------------------------------- soft-CE ----
struct CePlan {
  bool bulk;     // bulk-copy (TMA) path: 16-byte aligned rows
  int C;         // CTAs per row (thread-block cluster size)
  int slice;     // elements of a row per CTA
  int smem;      // dynamic shared memory bytes per CTA
  bool persistent;  // persistent clusters walking the rows, nb row buffers per CTA
  bool split;       // persistent with z and p in separate buffers (large slices)
  int nb;
};
CePlan soft_ce_plan(const float* z, const float* p, int64_t N, int64_t V);
constexpr int64_t kCeMaxV = 409600;  // 16 CTAs x 25600 elements
cudaError_t soft_ce_launch(const CePlan& plan, float* z, const float* p, const float* g, int64_t N,
                           int64_t V, float* row_loss, float* loss, float* wl, cudaStream_t s);

// Fixed-order sum of the per-row weighted losses wl[0..N) into *loss, launched
// as a programmatic dependent of the kernel before it on the stream.
cudaError_t soft_ce_loss_sum_launch(const float* wl, int64_t N, float* loss, cudaStream_t s);

// Variants (the STT_CE_* bits of the public header).
constexpr uint32_t kCeBf16 = 0x1u;         // z and p are bf16
constexpr uint32_t kCeGPerElement = 0x2u;  // g is fp32 [N, V]
struct CeVariantPlan {
  bool ok;     // the slice fits in shared memory
  bool bulk;   // 16-byte aligned rows (bulk copies)
  int C;       // CTAs per row (cluster size)
  int slice;   // elements per CTA
  int chunk;   // elements per bulk-copy chunk
  int smem;    // dynamic shared bytes per CTA
};
CeVariantPlan soft_ce_variant_plan(const void* z, const void* p, const float* g, int64_t V,
                                   uint32_t flags);
cudaError_t soft_ce_variant_launch(const CeVariantPlan& plan, uint32_t flags, void* z,
                                   const void* p, const float* g, int64_t N, int64_t V,
                                   float* row_loss, float* loss, float* wl, cudaStream_t s);
// The variants on the persistent cluster kernel (rows 16-byte aligned, V a
// multiple of 8, slices within its registers' reach); cudaErrorNotSupported
// when a call does not fit it, before anything is launched.
cudaError_t soft_ce_variant_persistent_launch(uint32_t flags, void* z, const void* p,
                                              const float* g, int64_t N, int64_t V,
                                              float* row_loss, float* loss, float* wl,
                                              cudaStream_t s);

// ------------------------------------------------------- LM head + soft-CE --
size_t lm_head_ce_workspace(int64_t N, int64_t V);
cudaError_t lm_head_ce_launch(const void* h, const void* W, const float* p, const float* g,
                              int64_t N, int64_t Hd, int64_t V, float* dh, float* dW,
                              float* row_loss, float* loss, void* workspace, cudaStream_t s);
cudaError_t lm_head_error_word(uint32_t* w);
cudaError_t lm_head_set_wait_budget(uint64_t ns);

// ---------------------------------------------------------- verification --
cudaError_t verify_launch(const float* p_t, const float* p_d, const int32_t* tokens,
                          const float* u_accept, const float* u_sample, int B, int gamma,
                          int64_t V, int32_t* n_acc, int32_t* out, cudaStream_t s);

// ----------------------------------------------------------- attention ----
constexpr int kMaxBatch = 1024;
constexpr int kMaxBlocks = 32;

struct AttnArgs {
  const void* q;
  const void* k_blocks[kMaxBlocks];
  const void* v_blocks[kMaxBlocks];
  int B, H, H_kv, D, Q_LEN, k;
  float scale;
  int T[kMaxBatch];
};

cudaError_t attn_fwd_launch(const AttnArgs& a, void* out, float* lse, cudaStream_t s);

// Flags of the backward (the STT_BWD_* bits of the public header).
constexpr uint32_t kBwdAccumulate = 0x1u;  // add into dK_j / dV_j instead of overwriting
constexpr uint32_t kBwdBf16 = 0x2u;        // dq, dK_j, dV_j are bf16

struct AttnBwdArgs {
  const void* out;
  const void* dout;
  const float* lse;
  void* dq;                     // fp32, or bf16 with kBwdBf16
  void* dk_blocks[kMaxBlocks];  // same element type as dq
  void* dv_blocks[kMaxBlocks];
  uint32_t flags;
  void* workspace;  // attn_bwd_workspace(...) bytes, 256-byte aligned
};
// Workspace: Delta [B, H, Q_LEN] fp32; with kBwdBf16 also fp32 accumulators
// for dq [B, H, Q_LEN, D] and dK_0, dV_0 [B, H_kv, Q_LEN, D].
size_t attn_bwd_workspace(int B, int H, int H_kv, int D, int Q_LEN, uint32_t flags);
cudaError_t attn_bwd_launch(const AttnArgs& a, const AttnBwdArgs& g, cudaStream_t s);

// ------------------------------------------- rotation, paged cache, logits --
struct RopeArgs {
  const double* freq;
  const __nv_bfloat16* w_q;
  const __nv_bfloat16* w_k;
  int R;
  bool inter;
  float amplitude, eps;
};
struct PagesArgs {
  void* k;
  void* v;
  const int32_t* table;
  const int32_t* cu_q;
  const int32_t* seq_lens;
  int64_t stride_page, stride_head, stride_tok;
  int B, H_kv, D, page_shift, num_pages, max_pages;
};
constexpr int kRopeBwdMaxGrid = 1024;  // blocks of the rotation's gradient
cudaError_t qkv_rope_launch(const RopeArgs& r, const void* qkv, int64_t ld,
                            const int32_t* positions, int B, int S, int H, int H_kv, int D, void* q,
                            void* k, void* v, cudaStream_t s);
size_t qkv_rope_bwd_workspace(int D);
cudaError_t qkv_rope_bwd_launch(const RopeArgs& r, const void* dq, const void* dk, const void* dv,
                                const void* qkv, int64_t ld, const int32_t* positions, int B,
                                int S, int H, int H_kv, int D, bool bf16, void* dqkv, int64_t ld_d,
                                float* dw_q, float* dw_k, void* workspace, cudaStream_t s);
cudaError_t kv_append_launch(const RopeArgs& r, const PagesArgs& pg, const void* qkv, int64_t ld,
                             const int32_t* positions, int64_t N, int H, void* q, cudaStream_t s);

struct PagedAttnArgs {
  const void* q;
  int64_t ld_q;
  int N, H;
  float scale;
  const uint32_t* tree;
  int tree_words;
  void* out;
  float* lse;
  void* workspace;
};
size_t paged_attn_workspace(int64_t N, int B, int H, int H_kv, int D);
cudaError_t paged_attn_launch(const PagesArgs& pg, const PagedAttnArgs& a, cudaStream_t s);

struct LogitsArgs {
  const void* z;
  int N, rows;
  int V;
  bool bf16, raw;
  const float *temperature, *repetition, *frequency, *presence;
  const int32_t *tokens, *cu_tokens, *n_prompt, *draft;
  const float* bias;
  const uint32_t* mask;
  int draft_ld, bias_rows, n_tokens;
  float* out;
};
constexpr int64_t kLogitsMaxV = 16 * 24576;
cudaError_t logits_launch(const LogitsArgs& a, cudaStream_t s);

// --------------------------- top logits, soft-CE against them, sampling --
constexpr int kRowMaxCtas = 16;                     // CTAs of a cluster that share a row
constexpr int64_t kRowMaxV = kRowMaxCtas * 45056;  // 16 slices that fit into shared memory
constexpr int kTopMaxK = 1024;
struct TopLogitsArgs {
  const void* z;
  int64_t ld_z, N;
  int V, K;
  bool bf16;
  float temperature;
  float* values;
  int32_t* indices;
  float* lse;
};
cudaError_t top_logits_launch(const TopLogitsArgs& a, cudaStream_t s);

constexpr int kSoftCeTopkMaxK = 1024;
struct SoftCeTopkArgs {
  const void* z;
  int64_t ld_z;
  void* dz;
  int64_t ld_dz, N;
  int V, K;
  bool bf16;
  float temperature;
  const float* values;
  const int32_t* indices;
  const float* lse;
  const float* g;
  float *row_loss, *loss, *wl;
};
cudaError_t soft_ce_topk_launch(const SoftCeTopkArgs& a, cudaStream_t s);

struct SampleArgs {
  const void* z;
  int64_t ld_z, N;
  int V, rows;
  bool bf16;
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p, *u;
  int32_t* tokens;
  float* logprobs;
  float* probs;
  int64_t ld_p;
};
cudaError_t sample_launch(const SampleArgs& a, cudaStream_t s);

// Per-file device error words (read and cleared).
cudaError_t qkv_rope_error_word(uint32_t* w);
cudaError_t paged_attn_error_word(uint32_t* w);
cudaError_t logits_error_word(uint32_t* w);
cudaError_t soft_ce_topk_error_word(uint32_t* w);
cudaError_t sample_error_word(uint32_t* w);
cudaError_t soft_ce_error_word(uint32_t* w);
cudaError_t attn_fwd_error_word(uint32_t* w);
cudaError_t attn_bwd_error_word(uint32_t* w);
// Per-file bounded-wait budgets (nanoseconds; 0 restores the default).
cudaError_t soft_ce_set_wait_budget(uint64_t ns);
cudaError_t attn_fwd_set_wait_budget(uint64_t ns);
cudaError_t attn_bwd_set_wait_budget(uint64_t ns);
cudaError_t paged_attn_set_wait_budget(uint64_t ns);
cudaError_t logits_set_wait_budget(uint64_t ns);
cudaError_t soft_ce_topk_set_wait_budget(uint64_t ns);
cudaError_t sample_set_wait_budget(uint64_t ns);

// Streaming multiprocessors of the current device (cached per device; 1 if
// the query fails, which only shrinks persistent grids).
int sm_count();

// Test hooks set by stt_debug_inject (STT_INJECT_* bits), read at launch.
uint32_t debug_inject();

// Status code of a CUDA error: cudaErrorNotSupported (an unsupported device
// or driver feature) is STT_ERR_UNSUPPORTED (-2), every other failure
// STT_ERR_CUDA (-4).
inline int status_from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return 0;
  if (e == cudaErrorNotSupported) return -2;
  return -4;
}

// Per-launch timing hooks (profile.cu); no-ops unless stt_profile_start ran.
void prof_before(cudaStream_t s, int kernel_id);
void prof_after(cudaStream_t s);

// Resolves cuTensorMapEncodeTiled through the runtime (no link against libcuda).
void* tensor_map_encoder();

// Makes the current device's primary context current on the calling thread.
// The tensor-map encoder is a driver call: on a thread that has not yet made
// a runtime call that binds the context (a fresh thread, e.g. the autograd
// engine's), it fails.  Called before any encoding.
cudaError_t bind_device_context();

}  // namespace stt
