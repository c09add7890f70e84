// paged_attn.cu -- attention of each sequence's new tokens over its pages.
//
// One warp per (row, query head): its lanes split D, keys come one after
// another, with a running maximum and sum (the softmax's result does not depend
// on the order).
#include <algorithm>

#include "../../include/stt.h"
#include "attn_common.cuh"

namespace stt {
namespace {

constexpr int kThreads = 128;

struct Params {
  PagesArgs g;
  PagedAttnArgs a;
};

template <int D>
__global__ void __launch_bounds__(kThreads) paged_attn_simple(const __grid_constant__ Params P) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = w / P.a.H;
  const int h = (int)(w - row * P.a.H);
  if (row >= P.a.N) return;
  const PagesArgs& G = P.g;
  int b = 0;
  for (int j = 0; j < G.B; j += 32) {
    const bool ends = j + lane < G.B && __ldg(G.cu_q + 1 + j + lane) <= (int)row;
    b += __popc(__ballot_sync(0xffffffffu, ends));
  }
  if (b >= G.B) return;
  const int first = __ldg(G.cu_q + b), n = __ldg(G.cu_q + b + 1) - first;
  const int len = __ldg(G.seq_lens + b), ctx = len - n, i = (int)row - first;
  const int kvh = h / (P.a.H / G.H_kv);

  float q[E], o[E];
  const __nv_bfloat16* qr =
      static_cast<const __nv_bfloat16*>(P.a.q) + row * P.a.ld_q + (int64_t)h * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(qr[e]) * P.a.scale;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int end = P.a.tree ? len : ctx + i + 1;
  bool bad = false;
  for (int key = 0; key < end; ++key) {
    if (P.a.tree && key >= ctx) {
      const int j = key - ctx;
      if (j >= 32 * P.a.tree_words) break;
      if (!((__ldg(P.a.tree + row * P.a.tree_words + (j >> 5)) >> (j & 31)) & 1u)) continue;
    }
    const int slot = key >> G.page_shift;
    if (slot >= G.max_pages) {
      bad = true;
      break;
    }
    const int page = __ldg(G.table + (int64_t)b * G.max_pages + slot);
    if (page < 0 || page >= G.num_pages) {
      bad = true;
      continue;
    }
    const int64_t at = (int64_t)page * G.stride_page + (int64_t)kvh * G.stride_head +
                       (int64_t)(key & ((1 << G.page_shift) - 1)) * G.stride_tok + lane * E;
    const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(G.k) + at;
    const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(G.v) + at;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], __bfloat162float(kr[e]), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s);
    const float alpha = expf(m - mn), p = expf(s - mn);
    l = l * alpha + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(p, __bfloat162float(vr[e]), o[e] * alpha);
    m = mn;
  }
  if (bad && lane == 0) record_error(STT_DEVERR_PAGE);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(P.a.out) + (row * P.a.H + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = __float2bfloat16_rn(o[e] * inv);
  if (P.a.lse && lane == 0) P.a.lse[row * P.a.H + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t paged_attn_workspace(int64_t, int, int, int, int) { return 16; }

cudaError_t paged_attn_launch(const PagesArgs& pg, const PagedAttnArgs& a, cudaStream_t s) {
  Params P{pg, a};
  const int64_t warps = (int64_t)a.N * a.H;
  const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
  prof_before(s, STT_KERNEL_PAGED_ATTN);
  if (pg.D == 128) paged_attn_simple<128><<<grid, kThreads, 0, s>>>(P);
  else paged_attn_simple<64><<<grid, kThreads, 0, s>>>(P);
  prof_after(s);
  return cudaGetLastError();
}

STT_DEFINE_ERROR_ACCESSOR(paged_attn_error_word)
STT_DEFINE_BUDGET_SETTER(paged_attn_set_wait_budget)

}  // namespace stt
