// stt_api.cu -- the C ABI declared in include/stt.h: argument validation,
// status codes, and dispatch to the kernel launchers.  No entry point
// allocates device memory or synchronises (except stt_device_error, which is
// documented to synchronise its stream).
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "../../include/stt.h"
#include "internal.h"

namespace stt {

void* tensor_map_encoder() {
  static void* fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = f;
  });
  return fn;
}

cudaError_t bind_device_context() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return cudaSetDevice(dev);
}

namespace {
std::atomic<uint32_t> g_inject{0};
constexpr int kMaxDevices = 64;
std::atomic<int> g_sm_count[kMaxDevices];
}  // namespace

int sm_count() {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 1;
  if (dev < kMaxDevices) {
    const int c = g_sm_count[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
    return 1;
  if (dev < kMaxDevices) g_sm_count[dev].store(v, std::memory_order_relaxed);
  return v;
}

uint32_t debug_inject() { return g_inject.load(std::memory_order_relaxed); }

}  // namespace stt

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The CUDA error the last failing call of this thread returned (read and
// cleared by stt_last_cuda_error).
thread_local int t_last_cuda_error = 0;

int from_cuda(cudaError_t e) {
  if (e != cudaSuccess) t_last_cuda_error = (int)e;
  return stt::status_from_cuda(e);
}

// Every launching entry point starts here: an error that an earlier runtime
// call of this thread left behind (someone else's) is cleared, so that the
// check after our own launches reports only them.  A sticky error (a faulted
// context) cannot be cleared and still fails the launches.
inline void begin_call() { (void)cudaGetLastError(); }

static_assert(STT_ERR_UNSUPPORTED == -2 && STT_ERR_CUDA == -4, "status_from_cuda codes");
static_assert(STT_CE_BF16 == stt::kCeBf16 && STT_CE_G_PER_ELEMENT == stt::kCeGPerElement,
              "soft-CE flags");
static_assert(STT_BWD_ACCUMULATE_KV == stt::kBwdAccumulate && STT_BWD_BF16_GRADS == stt::kBwdBf16,
              "backward flags");

// Shared validation of the attention arguments; fills `a` on success.
int check_attn(const void* q, const void* const* k_blocks, const void* const* v_blocks,
               const int32_t* T_host, int B, int H, int H_kv, int D, int Q_LEN, int k, float scale,
               stt::AttnArgs* a) {
  if (!q || !k_blocks || !v_blocks || !T_host) return STT_ERR_INVALID_ARG;
  if (B < 1 || B > STT_MAX_BATCH || H < 1 || H_kv < 1 || Q_LEN < 1) return STT_ERR_INVALID_ARG;
  if (H % H_kv != 0) return STT_ERR_INVALID_ARG;
  if (k < 0 || k > STT_MAX_STEP) return STT_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return STT_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return STT_ERR_UNSUPPORTED;
  if (H / H_kv > 8) return STT_ERR_UNSUPPORTED;
  if ((long long)B * H * Q_LEN > (1ll << 31) - 1) return STT_ERR_UNSUPPORTED;
  if (!aligned16(q)) return STT_ERR_MISALIGNED;
  for (int j = 0; j <= k; ++j) {
    if (!k_blocks[j] || !v_blocks[j]) return STT_ERR_INVALID_ARG;
    if (!aligned16(k_blocks[j]) || !aligned16(v_blocks[j])) return STT_ERR_MISALIGNED;
  }
  for (int b = 0; b < B; ++b)
    if (T_host[b] < 0 || T_host[b] > Q_LEN) return STT_ERR_INVALID_ARG;
  std::memset(a, 0, sizeof(*a));
  a->q = q;
  for (int j = 0; j <= k; ++j) {
    a->k_blocks[j] = k_blocks[j];
    a->v_blocks[j] = v_blocks[j];
  }
  a->B = B;
  a->H = H;
  a->H_kv = H_kv;
  a->D = D;
  a->Q_LEN = Q_LEN;
  a->k = k;
  a->scale = scale;
  for (int b = 0; b < B; ++b) a->T[b] = T_host[b];
  return STT_OK;
}

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Validation of the rotation's arguments; fills `r` on success.
int check_rope(const stt_rope* rope, int D, stt::RopeArgs* r) {
  if (!rope) return STT_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return STT_ERR_UNSUPPORTED;
  if (rope->R < 0 || rope->R > D) return STT_ERR_INVALID_ARG;
  if (rope->R % 16 != 0) return STT_ERR_UNSUPPORTED;
  if ((rope->R > 0) != (rope->freq != nullptr)) return STT_ERR_INVALID_ARG;
  if (rope->flags & ~(uint32_t)STT_ROPE_INTERLEAVED) return STT_ERR_INVALID_ARG;
  if (!std::isfinite(rope->amplitude)) return STT_ERR_INVALID_ARG;
  if ((rope->w_q || rope->w_k) && (!std::isfinite(rope->eps) || !(rope->eps > 0.f)))
    return STT_ERR_INVALID_ARG;
  if (!aligned(rope->freq, 8) || !aligned16(rope->w_q) || !aligned16(rope->w_k))
    return STT_ERR_MISALIGNED;
  r->freq = rope->freq;
  r->w_q = static_cast<const __nv_bfloat16*>(rope->w_q);
  r->w_k = static_cast<const __nv_bfloat16*>(rope->w_k);
  r->R = rope->R;
  r->inter = (rope->flags & STT_ROPE_INTERLEAVED) != 0;
  r->amplitude = rope->amplitude;
  r->eps = rope->eps;
  return STT_OK;
}

// Rows of the projection: N of them, ld elements apart.
int check_rows(const void* rows, int64_t ld, int64_t heads, int D) {
  if (!rows) return STT_ERR_INVALID_ARG;
  if (ld < heads * D) return STT_ERR_INVALID_ARG;
  if (ld % 8 != 0 || !aligned16(rows)) return STT_ERR_MISALIGNED;
  return STT_OK;
}

int check_pages(const stt_pages* p, int64_t N, stt::PagesArgs* g) {
  if (!p) return STT_ERR_INVALID_ARG;
  if (p->B < 0 || p->B > STT_MAX_BATCH || p->H_kv < 1 || N < 0) return STT_ERR_INVALID_ARG;
  if (p->D != 64 && p->D != 128) return STT_ERR_UNSUPPORTED;
  if (p->page_size < 1 || p->num_pages < 1 || p->max_pages < 1) return STT_ERR_INVALID_ARG;
  int shift = 3;
  while (shift < 10 && (1 << shift) != p->page_size) ++shift;
  if ((1 << shift) != p->page_size) return STT_ERR_UNSUPPORTED;
  if ((int64_t)p->max_pages * p->page_size > (1ll << 30)) return STT_ERR_UNSUPPORTED;
  if (p->B > 0 && N > 0) {
    if (!p->k || !p->v || !p->table || !p->cu_q || !p->seq_lens) return STT_ERR_INVALID_ARG;
    if (!aligned16(p->k) || !aligned16(p->v) || !aligned(p->table, 4) || !aligned(p->cu_q, 4) ||
        !aligned(p->seq_lens, 4))
      return STT_ERR_MISALIGNED;
    // Every key of a cache at its own place, in any order of page, head and key.
    if (p->stride_page < 1 || p->stride_head < 1 || p->stride_tok < p->D)
      return STT_ERR_INVALID_ARG;
    if (p->stride_page % 8 || p->stride_head % 8 || p->stride_tok % 8) return STT_ERR_MISALIGNED;
    if (p->stride_page > (1ll << 38) || p->stride_head > (1ll << 38) ||
        p->stride_tok > (1ll << 38))
      return STT_ERR_UNSUPPORTED;  // a tensor map's strides are 40-bit byte counts
  }
  g->k = p->k;
  g->v = p->v;
  g->table = p->table;
  g->cu_q = p->cu_q;
  g->seq_lens = p->seq_lens;
  g->stride_page = p->stride_page;
  g->stride_head = p->stride_head;
  g->stride_tok = p->stride_tok;
  g->B = p->B;
  g->H_kv = p->H_kv;
  g->D = p->D;
  g->page_shift = shift;
  g->num_pages = p->num_pages;
  g->max_pages = p->max_pages;
  return STT_OK;
}

static_assert(STT_ROPE_INTERLEAVED == 1u && STT_ROPE_BF16_GRADS == 2u, "rotation flags");

}  // namespace

extern "C" {

const char* stt_status_string(int status) {
  switch (status) {
    case STT_OK: return "ok";
    case STT_ERR_INVALID_ARG: return "invalid argument";
    case STT_ERR_UNSUPPORTED: return "unsupported configuration";
    case STT_ERR_MISALIGNED: return "pointer not 16-byte aligned";
    case STT_ERR_CUDA: return "CUDA error";
    case STT_ERR_TIMEOUT: return "device-side bounded wait ran out";
    case STT_ERR_WORKSPACE: return "workspace missing or too small";
    default: return "unknown status";
  }
}

int stt_version(void) { return 100; }

int stt_device_error(void* stream, uint32_t* word) {
  if (!word) return STT_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return STT_ERR_CUDA;
  uint32_t w = 0, part = 0;
  if (stt::soft_ce_error_word(&part) != cudaSuccess) return STT_ERR_CUDA;
  w |= part;
  if (stt::attn_fwd_error_word(&part) != cudaSuccess) return STT_ERR_CUDA;
  w |= part;
  if (stt::attn_bwd_error_word(&part) != cudaSuccess) return STT_ERR_CUDA;
  w |= part;
  if (stt::lm_head_error_word(&part) != cudaSuccess) return STT_ERR_CUDA;
  w |= part;
  if (stt::qkv_rope_error_word(&part) != cudaSuccess) return STT_ERR_CUDA;
  w |= part;
  if (stt::paged_attn_error_word(&part) != cudaSuccess) return STT_ERR_CUDA;
  w |= part;
  if (stt::logits_error_word(&part) != cudaSuccess) return STT_ERR_CUDA;
  w |= part;
  *word = w;
  return (w & STT_DEVERR_WAIT_MASK) ? STT_ERR_TIMEOUT : STT_OK;
}

int stt_last_cuda_error(const char** name) {
  const int e = t_last_cuda_error;
  t_last_cuda_error = 0;
  if (name) *name = cudaGetErrorName(static_cast<cudaError_t>(e));
  return e;
}

int stt_debug_set_wait_budget(uint64_t ns) {
  cudaError_t e = stt::soft_ce_set_wait_budget(ns);
  if (e == cudaSuccess) e = stt::attn_fwd_set_wait_budget(ns);
  if (e == cudaSuccess) e = stt::attn_bwd_set_wait_budget(ns);
  if (e == cudaSuccess) e = stt::lm_head_set_wait_budget(ns);
  if (e == cudaSuccess) e = stt::paged_attn_set_wait_budget(ns);
  if (e == cudaSuccess) e = stt::logits_set_wait_budget(ns);
  return from_cuda(e);
}

int stt_debug_inject(uint32_t what) {
  if (what & ~(uint32_t)(STT_INJECT_FWD_WITHHOLD_Q | STT_INJECT_LOGITS_WITHHOLD_PAIRS |
                         STT_INJECT_PAGED_WITHHOLD_Q))
    return STT_ERR_INVALID_ARG;
  stt::g_inject.store(what, std::memory_order_relaxed);
  return STT_OK;
}

int stt_attn_fwd(const void* q, const void* const* k_blocks, const void* const* v_blocks,
                 const int32_t* T_host, int B, int H, int H_kv, int D, int Q_LEN, int k,
                 float scale, void* out, float* lse, void* stream) {
  try {
    begin_call();
    static thread_local stt::AttnArgs a;
    int st = check_attn(q, k_blocks, v_blocks, T_host, B, H, H_kv, D, Q_LEN, k, scale, &a);
    if (st != STT_OK) return st;
    if (!out || !lse) return STT_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(lse)) return STT_ERR_MISALIGNED;
    return from_cuda(stt::attn_fwd_launch(a, out, lse, static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return STT_ERR_CUDA;
  }
}

size_t stt_attn_bwd_workspace_size(int B, int H, int H_kv, int D, int Q_LEN, int k) {
  return stt_attn_bwd_ex_workspace_size(B, H, H_kv, D, Q_LEN, k, 0u);
}

size_t stt_attn_bwd_ex_workspace_size(int B, int H, int H_kv, int D, int Q_LEN, int k,
                                      uint32_t flags) {
  (void)k;
  if (B < 1 || H < 1 || H_kv < 1 || Q_LEN < 1 || D < 1) return 16;
  return stt::attn_bwd_workspace(B, H, H_kv, D, Q_LEN, flags);
}

int stt_attn_bwd_ex(const void* q, const void* const* k_blocks, const void* const* v_blocks,
                    const int32_t* T_host, int B, int H, int H_kv, int D, int Q_LEN, int k,
                    float scale, const void* out, const void* dout, const float* lse, void* dq,
                    void* const* dk_blocks, void* const* dv_blocks, uint32_t flags,
                    void* workspace, size_t workspace_bytes, void* stream) {
  try {
    begin_call();
    static thread_local stt::AttnArgs a;
    int st = check_attn(q, k_blocks, v_blocks, T_host, B, H, H_kv, D, Q_LEN, k, scale, &a);
    if (st != STT_OK) return st;
    if (flags & ~(uint32_t)(STT_BWD_ACCUMULATE_KV | STT_BWD_BF16_GRADS)) return STT_ERR_INVALID_ARG;
    if (!out || !dout || !lse || !dq || !dk_blocks || !dv_blocks) return STT_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(dout) || !aligned16(lse) || !aligned16(dq))
      return STT_ERR_MISALIGNED;
    stt::AttnBwdArgs g;
    std::memset(&g, 0, sizeof(g));
    for (int j = 0; j <= k; ++j) {
      if (!dk_blocks[j] || !dv_blocks[j]) return STT_ERR_INVALID_ARG;
      if (!aligned16(dk_blocks[j]) || !aligned16(dv_blocks[j])) return STT_ERR_MISALIGNED;
      g.dk_blocks[j] = dk_blocks[j];
      g.dv_blocks[j] = dv_blocks[j];
    }
    const size_t need = stt::attn_bwd_workspace(B, H, H_kv, D, Q_LEN, flags);
    if (!workspace || workspace_bytes < need) return STT_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return STT_ERR_MISALIGNED;
    g.out = out;
    g.dout = dout;
    g.lse = lse;
    g.dq = dq;
    g.flags = flags;
    g.workspace = workspace;
    return from_cuda(stt::attn_bwd_launch(a, g, static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return STT_ERR_CUDA;
  }
}

int stt_attn_bwd(const void* q, const void* const* k_blocks, const void* const* v_blocks,
                 const int32_t* T_host, int B, int H, int H_kv, int D, int Q_LEN, int k,
                 float scale, const void* out, const void* dout, const float* lse, float* dq,
                 float* const* dk_blocks, float* const* dv_blocks, void* workspace,
                 size_t workspace_bytes, void* stream) {
  return stt_attn_bwd_ex(q, k_blocks, v_blocks, T_host, B, H, H_kv, D, Q_LEN, k, scale, out, dout,
                         lse, dq, reinterpret_cast<void* const*>(dk_blocks),
                         reinterpret_cast<void* const*>(dv_blocks), 0u, workspace,
                         workspace_bytes, stream);
}

size_t soft_ce_workspace_size(int64_t N, int64_t V) {
  (void)V;
  if (N < 0) return 16;
  size_t b = (size_t)N * sizeof(float);
  b = (b + 15) / 16 * 16;
  return b < 16 ? 16 : b;
}

int soft_ce_fwd_bwd_inplace(float* z, const float* p, const float* g, int64_t N, int64_t V,
                            float* row_loss, float* loss, void* workspace,
                            size_t workspace_bytes, void* stream) {
  try {
    begin_call();
    if (N < 0 || V < 1 || !loss) return STT_ERR_INVALID_ARG;
    if (N > 0 && (!z || !p || !g)) return STT_ERR_INVALID_ARG;
    if (N > 0 && V > INT64_MAX / N) return STT_ERR_INVALID_ARG;
    if (V > stt::kCeMaxV) return STT_ERR_UNSUPPORTED;
    if (N * (V > 16 ? 16 : V) > 0x7fffffffLL) return STT_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < soft_ce_workspace_size(N, V)) return STT_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 3u) != 0) return STT_ERR_MISALIGNED;
    const stt::CePlan plan = stt::soft_ce_plan(z, p, N, V);
    if (N * (int64_t)plan.C > 0x7fffffffLL) return STT_ERR_UNSUPPORTED;
    return from_cuda(stt::soft_ce_launch(plan, z, p, g, N, V, row_loss, loss,
                                         static_cast<float*>(workspace),
                                         static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return STT_ERR_CUDA;
  }
}

int soft_ce_fwd_bwd_inplace_ex(void* z, const void* p, const float* g, int64_t N, int64_t V,
                               uint32_t flags, float* row_loss, float* loss, void* workspace,
                               size_t workspace_bytes, void* stream) {
  try {
    begin_call();
    if (flags & ~(uint32_t)(STT_CE_BF16 | STT_CE_G_PER_ELEMENT)) return STT_ERR_INVALID_ARG;
    if (flags == 0)
      return soft_ce_fwd_bwd_inplace(static_cast<float*>(z), static_cast<const float*>(p), g, N,
                                     V, row_loss, loss, workspace, workspace_bytes, stream);
    if (N < 0 || V < 1 || !loss) return STT_ERR_INVALID_ARG;
    if (N > 0 && (!z || !p || !g)) return STT_ERR_INVALID_ARG;
    if (N > 0 && V > INT64_MAX / N) return STT_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < soft_ce_workspace_size(N, V)) return STT_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 3u) != 0) return STT_ERR_MISALIGNED;
    const stt::CeVariantPlan plan = stt::soft_ce_variant_plan(z, p, g, V, flags);
    if (!plan.ok) return STT_ERR_UNSUPPORTED;
    if (N * (int64_t)plan.C > 0x7fffffffLL) return STT_ERR_UNSUPPORTED;
    return from_cuda(stt::soft_ce_variant_launch(plan, flags, z, p, g, N, V, row_loss, loss,
                                                 static_cast<float*>(workspace),
                                                 static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return STT_ERR_CUDA;
  }
}

size_t stt_lm_head_ce_workspace_size(int64_t N, int64_t Hd, int64_t V) {
  (void)Hd;
  if (N < 0 || V < 1) return 16;
  return stt::lm_head_ce_workspace(N, V);
}

int stt_lm_head_ce(const void* h, const void* W, const float* p, const float* g, int64_t N,
                   int64_t Hd, int64_t V, float* dh, float* dW, float* row_loss, float* loss,
                   void* workspace, size_t workspace_bytes, void* stream) {
  try {
    begin_call();
    if (N < 0 || Hd < 8 || V < 8 || !loss) return STT_ERR_INVALID_ARG;
    if (Hd % 8 != 0 || V % 8 != 0) return STT_ERR_UNSUPPORTED;
    if (N > 0x7fffffffLL || Hd > 0x7fffffffLL || V > 0x7fffffffLL) return STT_ERR_UNSUPPORTED;
    if (N > 0 && (!h || !W || !p || !g || !dh || !dW)) return STT_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < stt::lm_head_ce_workspace(N, V)) return STT_ERR_WORKSPACE;
    const uintptr_t a = reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(W) |
                        reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(dh) |
                        reinterpret_cast<uintptr_t>(dW);
    if ((a & 15u) != 0 || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
      return STT_ERR_MISALIGNED;
    return from_cuda(stt::lm_head_ce_launch(h, W, p, g, N, Hd, V, dh, dW, row_loss, loss,
                                            workspace, static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return STT_ERR_CUDA;
  }
}

int stt_verify(const float* p_target, const float* p_draft, const int32_t* draft_tokens,
               const float* u_accept, const float* u_sample, int B, int gamma, int64_t V,
               int32_t* n_accepted, int32_t* out_tokens, void* stream) {
  try {
    begin_call();
    if (B < 0 || gamma < 1 || gamma > STT_VERIFY_MAX_GAMMA || V < 1) return STT_ERR_INVALID_ARG;
    if (B == 0) return STT_OK;
    if (!p_target || !p_draft || !draft_tokens || !u_accept || !u_sample || !n_accepted ||
        !out_tokens)
      return STT_ERR_INVALID_ARG;
    if ((long long)B * gamma > INT64_MAX / V) return STT_ERR_INVALID_ARG;
    if (V > 0x7fffffffLL) return STT_ERR_UNSUPPORTED;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p_target) |
                        reinterpret_cast<uintptr_t>(p_draft) |
                        reinterpret_cast<uintptr_t>(draft_tokens) |
                        reinterpret_cast<uintptr_t>(u_accept) |
                        reinterpret_cast<uintptr_t>(u_sample) |
                        reinterpret_cast<uintptr_t>(n_accepted) |
                        reinterpret_cast<uintptr_t>(out_tokens);
    if (a & 3u) return STT_ERR_MISALIGNED;
    return from_cuda(stt::verify_launch(p_target, p_draft, draft_tokens, u_accept, u_sample, B,
                                        gamma, V, n_accepted, out_tokens,
                                        static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return STT_ERR_CUDA;
  }
}

int stt_qkv_rope_fwd(const void* qkv, int64_t ld, const int32_t* positions, int B, int S, int H,
                     int H_kv, int D, const stt_rope* rope, void* q, void* k, void* v,
                     void* stream) {
  try {
    begin_call();
    stt::RopeArgs r{};
    if (B < 0 || S < 0 || H < 1 || H_kv < 1) return STT_ERR_INVALID_ARG;
    int st = check_rope(rope, D, &r);
    if (st != STT_OK) return st;
    if ((int64_t)B * S == 0) return STT_OK;
    if ((int64_t)B * S > 0x7fffffffll || (int64_t)H + 2ll * H_kv > (1 << 20))
      return STT_ERR_UNSUPPORTED;
    st = check_rows(qkv, ld, (int64_t)H + 2ll * H_kv, D);
    if (st != STT_OK) return st;
    if (!q || !k || !v) return STT_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned(positions, 4))
      return STT_ERR_MISALIGNED;
    return from_cuda(stt::qkv_rope_launch(r, qkv, ld, positions, B, S, H, H_kv, D, q, k, v,
                                          static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return STT_ERR_CUDA;
  }
}

size_t stt_qkv_rope_bwd_workspace_size(int D) {
  return D > 0 && D <= 128 ? stt::qkv_rope_bwd_workspace(D) : 16;
}

int stt_qkv_rope_bwd(const void* dq, const void* dk, const void* dv, const void* qkv, int64_t ld,
                     const int32_t* positions, int B, int S, int H, int H_kv, int D,
                     const stt_rope* rope, uint32_t flags, void* dqkv, int64_t ld_d, float* dw_q,
                     float* dw_k, void* workspace, size_t workspace_bytes, void* stream) {
  try {
    begin_call();
    stt::RopeArgs r{};
    if (B < 0 || S < 0 || H < 1 || H_kv < 1) return STT_ERR_INVALID_ARG;
    if (flags & ~(uint32_t)STT_ROPE_BF16_GRADS) return STT_ERR_INVALID_ARG;
    int st = check_rope(rope, D, &r);
    if (st != STT_OK) return st;
    const bool norm = r.w_q || r.w_k;
    if ((r.w_q != nullptr) != (dw_q != nullptr) || (r.w_k != nullptr) != (dw_k != nullptr))
      return STT_ERR_INVALID_ARG;
    if (!aligned(dw_q, 4) || !aligned(dw_k, 4)) return STT_ERR_MISALIGNED;
    if (norm) {
      if (!workspace || workspace_bytes < stt::qkv_rope_bwd_workspace(D))
        return STT_ERR_WORKSPACE;
      if (!aligned16(workspace)) return STT_ERR_MISALIGNED;
    }
    if ((int64_t)B * S > 0x7fffffffll || (int64_t)H + 2ll * H_kv > (1 << 20))
      return STT_ERR_UNSUPPORTED;
    if ((int64_t)B * S > 0) {
      st = check_rows(dqkv, ld_d, (int64_t)H + 2ll * H_kv, D);
      if (st == STT_OK && norm) st = check_rows(qkv, ld, (int64_t)H + 2ll * H_kv, D);
      if (st != STT_OK) return st;
      if (!dq || !dk || !dv) return STT_ERR_INVALID_ARG;
      if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned(positions, 4))
        return STT_ERR_MISALIGNED;
    } else if (!norm) {
      return STT_OK;
    }
    return from_cuda(stt::qkv_rope_bwd_launch(
        r, dq, dk, dv, qkv, ld, positions, B, S, H, H_kv, D, (flags & STT_ROPE_BF16_GRADS) != 0,
        dqkv, ld_d, dw_q, dw_k, workspace, static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return STT_ERR_CUDA;
  }
}

int stt_kv_append(const void* qkv, int64_t ld, const int32_t* positions, int64_t N, int H,
                  const stt_pages* pages, const stt_rope* rope, void* q, void* stream) {
  try {
    begin_call();
    stt::RopeArgs r{};
    stt::PagesArgs g{};
    if (H < 1) return STT_ERR_INVALID_ARG;
    int st = check_pages(pages, N, &g);
    if (st != STT_OK) return st;
    st = check_rope(rope, g.D, &r);
    if (st != STT_OK) return st;
    if (N == 0 || g.B == 0) return STT_OK;
    if (N > 0x7fffffffll || (int64_t)H + 2ll * g.H_kv > (1 << 20)) return STT_ERR_UNSUPPORTED;
    st = check_rows(qkv, ld, (int64_t)H + 2ll * g.H_kv, g.D);
    if (st != STT_OK) return st;
    if (!q) return STT_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned(positions, 4)) return STT_ERR_MISALIGNED;
    return from_cuda(stt::kv_append_launch(r, g, qkv, ld, positions, N, H, q,
                                           static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return STT_ERR_CUDA;
  }
}

size_t stt_paged_attn_workspace_size(int64_t N, int B, int H, int H_kv, int D) {
  if (N < 1 || B < 1 || H < 1 || H_kv < 1 || D < 1 || H % H_kv != 0) return 16;
  return stt::paged_attn_workspace(N, B, H, H_kv, D);
}

int stt_paged_attn(const void* q, int64_t ld_q, int64_t N, int H, const stt_pages* pages,
                   float scale, const uint32_t* tree, int tree_words, void* out, float* lse,
                   void* workspace, size_t workspace_bytes, void* stream) {
  try {
    begin_call();
    stt::PagesArgs g{};
    int st = check_pages(pages, N, &g);
    if (st != STT_OK) return st;
    if (H < 1 || H % g.H_kv != 0) return STT_ERR_INVALID_ARG;
    if (H / g.H_kv > 16) return STT_ERR_UNSUPPORTED;
    if (!std::isfinite(scale) || !(scale > 0.f)) return STT_ERR_INVALID_ARG;
    if (tree && (tree_words < 1 || tree_words > (1 << 20))) return STT_ERR_INVALID_ARG;
    if (N == 0 || g.B == 0) return STT_OK;
    if (N > 0x7fffffffll || N * H > 0x7fffffffll) return STT_ERR_UNSUPPORTED;
    st = check_rows(q, ld_q, H, g.D);
    if (st != STT_OK) return st;
    if (ld_q > (1ll << 38)) return STT_ERR_UNSUPPORTED;
    if (!out) return STT_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned(lse, 4) || !aligned(tree, 4)) return STT_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < stt::paged_attn_workspace(N, g.B, H, g.H_kv, g.D))
      return STT_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return STT_ERR_MISALIGNED;
    stt::PagedAttnArgs a{};
    a.q = q;
    a.ld_q = ld_q;
    a.N = (int)N;
    a.H = H;
    a.scale = scale;
    a.tree = tree;
    a.tree_words = tree_words;
    a.out = out;
    a.lse = lse;
    a.workspace = workspace;
    return from_cuda(stt::paged_attn_launch(g, a, static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return STT_ERR_CUDA;
  }
}

int stt_logits_process(const void* z, int64_t N, int64_t V, int rows, const stt_logits* params,
                       uint32_t flags, float* out, void* stream) {
  try {
    begin_call();
    if (!params || N < 0 || V < 1 || rows < 1) return STT_ERR_INVALID_ARG;
    if (flags & ~(uint32_t)(STT_LOGITS_BF16 | STT_LOGITS_RAW)) return STT_ERR_INVALID_ARG;
    if (N % rows != 0) return STT_ERR_INVALID_ARG;
    if (V > stt::kLogitsMaxV || N > 0x7fffffffll / 16) return STT_ERR_UNSUPPORTED;
    const stt_logits& p = *params;
    if (!p.tokens != !p.cu_tokens || (p.n_prompt && !p.tokens)) return STT_ERR_INVALID_ARG;
    if (p.n_tokens < 0) return STT_ERR_INVALID_ARG;
    if (p.draft && p.draft_ld < rows - 1) return STT_ERR_INVALID_ARG;
    if (p.bias_rows < 0 || (p.bias_rows > 0) != (p.bias != nullptr)) return STT_ERR_INVALID_ARG;
    if (p.bias_rows > 1 && p.bias_rows != N / rows) return STT_ERR_INVALID_ARG;
    if (N == 0) return STT_OK;
    if (!z || !out) return STT_ERR_INVALID_ARG;
    const bool bf16 = (flags & STT_LOGITS_BF16) != 0;
    if (bf16 && z == out) return STT_ERR_INVALID_ARG;
    const uintptr_t all =
        reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(p.temperature) |
        reinterpret_cast<uintptr_t>(p.repetition) | reinterpret_cast<uintptr_t>(p.frequency) |
        reinterpret_cast<uintptr_t>(p.presence) | reinterpret_cast<uintptr_t>(p.tokens) |
        reinterpret_cast<uintptr_t>(p.cu_tokens) | reinterpret_cast<uintptr_t>(p.n_prompt) |
        reinterpret_cast<uintptr_t>(p.draft) | reinterpret_cast<uintptr_t>(p.bias) |
        reinterpret_cast<uintptr_t>(p.mask);
    if ((all & 3u) || !aligned(z, bf16 ? 2 : 4)) return STT_ERR_MISALIGNED;
    stt::LogitsArgs a{};
    a.z = z;
    a.N = (int)N;
    a.rows = rows;
    a.V = (int)V;
    a.bf16 = bf16;
    a.raw = (flags & STT_LOGITS_RAW) != 0;
    a.temperature = p.temperature;
    a.repetition = p.repetition;
    a.frequency = p.frequency;
    a.presence = p.presence;
    a.tokens = p.tokens;
    a.cu_tokens = p.cu_tokens;
    a.n_prompt = p.n_prompt;
    a.draft = p.draft;
    a.bias = p.bias;
    a.mask = p.mask;
    a.draft_ld = p.draft_ld;
    a.bias_rows = p.bias_rows;
    a.n_tokens = p.n_tokens;
    a.out = out;
    return from_cuda(stt::logits_launch(a, static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return STT_ERR_CUDA;
  }
}

}  // extern "C"
