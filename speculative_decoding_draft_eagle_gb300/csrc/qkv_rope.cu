// qkv_rope.cu -- per-head norm and position rotation of queries and keys: from
// the fused QKV projection's rows to the attention's layout (training), to the
// queries and a paged KV cache (serving), and the training form's gradient.
//
// All three are one pass over memory: a warp takes a token (or a part of its
// heads, where there are too few tokens to fill the GPU), makes the token's
// tables of cosines, sines and weights once (rope.cuh), and streams the token's
// heads through them, 32 / (D / 8) heads a step, 16-byte loads and stores, a few
// steps' loads in flight at a time.
#include <algorithm>

#include "rope.cuh"

namespace stt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 4;
constexpr int kUnroll = 4;  // steps whose loads are in flight together

struct FwdP {
  RopeArgs r;
  PagesArgs pg;  // append only
  const __nv_bfloat16* qkv;
  int64_t ld;
  const int32_t* positions;
  __nv_bfloat16 *q, *k, *v;
  uint32_t N, items, parts, steps_per_part;
  int S, H, H_kv;
};

// Where one token's heads go.
struct Dest {
  __nv_bfloat16 *q, *k, *v;
  int64_t q_head, kv_head;
  bool kv;  // the key and value rows are written
  int pos;
};

__device__ __forceinline__ Dest train_dest(const FwdP& P, uint32_t t, int D) {
  Dest d;
  const uint32_t b = t / (uint32_t)P.S, s = t - b * (uint32_t)P.S;
  d.q_head = d.kv_head = (int64_t)P.S * D;
  d.q = P.q + ((int64_t)b * P.H * P.S + s) * D;
  d.k = P.k + ((int64_t)b * P.H_kv * P.S + s) * D;
  d.v = P.v + ((int64_t)b * P.H_kv * P.S + s) * D;
  d.kv = true;
  d.pos = P.positions ? __ldg(P.positions + t) : (int)s;
  return d;
}

// False for a row behind the last sequence.
__device__ __forceinline__ bool append_dest(const FwdP& P, uint32_t t, int D, Dest& d) {
  const PagesArgs& G = P.pg;
  const int lane = threadIdx.x & 31;
  // The row's sequence: how many sequences end at or before it (warp-wide count).
  int b = 0;
  for (int j = 0; j < G.B; j += 32) {
    const bool ends = j + lane < G.B && __ldg(G.cu_q + 1 + j + lane) <= (int)t;
    b += __popc(__ballot_sync(0xffffffffu, ends));
  }
  if (b >= G.B) return false;
  const int key = __ldg(G.seq_lens + b) - __ldg(G.cu_q + b + 1) + (int)t;
  d.q = P.q + (int64_t)t * P.H * D;
  d.q_head = D;
  d.kv_head = G.stride_head;
  d.pos = P.positions ? __ldg(P.positions + t) : key;
  d.kv = false;
  const int slot = key >> G.page_shift;
  if (key >= 0 && slot < G.max_pages) {
    const int page = __ldg(G.table + (int64_t)b * G.max_pages + slot);
    if (page >= 0 && page < G.num_pages) {
      d.kv = true;
      const int64_t at = (int64_t)page * G.stride_page +
                         (int64_t)(key & ((1 << G.page_shift) - 1)) * G.stride_tok;
      d.k = static_cast<__nv_bfloat16*>(G.k) + at;
      d.v = static_cast<__nv_bfloat16*>(G.v) + at;
    }
  }
  if (!d.kv && lane == 0) record_error(STT_DEVERR_PAGE);
  return true;
}

template <int D, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kThreads)
    qkv_rope_kernel(const __grid_constant__ FwdP P) {
  using L = RopeLane<D, INTER>;
  L L_;
  L_.init(P.r.freq, P.r.R);
  const int nq = (P.H + L::kHeads - 1) / L::kHeads, nk = (P.H_kv + L::kHeads - 1) / L::kHeads;
  const uint32_t warp = blockIdx.x * kWarps + (threadIdx.x >> 5), warps = gridDim.x * kWarps;

  for (uint32_t item = warp; item < P.items; item += warps) {
    const uint32_t t = item / P.parts, part = item - t * P.parts;
    Dest d;
    if constexpr (APPEND) {
      if (!append_dest(P, t, D, d)) continue;
    } else {
      d = train_dest(P, t, D);
    }
    const __nv_bfloat16* row = P.qkv + (int64_t)t * P.ld;
    const int lo = (int)(part * P.steps_per_part), hi = lo + (int)P.steps_per_part;
    float c[8], s[8];
    L_.angles(d.pos, P.r.amplitude, c, s);

    // Steps [lo, hi) of one kind of head: `first` its first step, `n` its heads.
    auto run = [&](int first, int steps, int n, int head0, const __nv_bfloat16* w, bool rotate,
                   __nv_bfloat16* dst, int64_t dst_head) {
      const int from = max(lo, first) - first, to = min(hi, first + steps) - first;
      if (from >= to) return;
      float a[8], b[8];
      if (rotate) L_.tables(w, c, s, a, b);
      for (int u0 = from; u0 < to; u0 += kUnroll) {
        uint4 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int h = (u0 + u) * L::kHeads + L_.sub;
          x[u] = make_uint4(0, 0, 0, 0);
          if (u0 + u < to && h < n)
            x[u] = __ldg(reinterpret_cast<const uint4*>(row + (int64_t)(head0 + h) * D) + L_.chunk);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (u0 + u >= to) break;
          const int h = (u0 + u) * L::kHeads + L_.sub;
          const uint4 y = rotate ? L_.apply(x[u], w != nullptr, P.r.eps, a, b) : x[u];
          if (h < n) reinterpret_cast<uint4*>(dst + (int64_t)h * dst_head)[L_.chunk] = y;
        }
      }
    };
    run(0, nq, P.H, 0, P.r.w_q, true, d.q, d.q_head);
    if (d.kv) {
      run(nq, nk, P.H_kv, P.H, P.r.w_k, true, d.k, d.kv_head);
      run(nq + nk, nk, P.H_kv, P.H + P.H_kv, nullptr, false, d.v, d.kv_head);
    }
  }
}

// Splits each token's steps over enough warps to fill the GPU, down to kUnroll
// steps a warp.
void split_items(int64_t N, int steps, int64_t warps_wanted, uint32_t* parts, uint32_t* per) {
  int64_t p = std::max<int64_t>(1, warps_wanted / std::max<int64_t>(N, 1));
  p = std::min<int64_t>(p, (steps + kUnroll - 1) / kUnroll);
  *per = (uint32_t)((steps + p - 1) / p);
  *parts = (uint32_t)((steps + *per - 1) / *per);
}

template <bool APPEND>
cudaError_t launch_fwd(FwdP& P, int D, cudaStream_t s) {
  if (P.N == 0) return cudaSuccess;
  const int heads = 32 / (D / 8);
  const int steps = (P.H + heads - 1) / heads + 2 * ((P.H_kv + heads - 1) / heads);
  const int64_t blocks_max = (int64_t)sm_count() * kBlocksPerSm;
  split_items(P.N, steps, blocks_max * kWarps, &P.parts, &P.steps_per_part);
  const int64_t items = (int64_t)P.N * P.parts;
  if (items > 0x7fffffffll) return cudaErrorNotSupported;
  P.items = (uint32_t)items;
  const unsigned grid = (unsigned)std::min<int64_t>((items + kWarps - 1) / kWarps, blocks_max);
  const bool inter = P.r.inter;
  prof_before(s, APPEND ? STT_KERNEL_KV_APPEND : STT_KERNEL_QKV_ROPE);
  if (D == 128) {
    if (inter) qkv_rope_kernel<128, true, APPEND><<<grid, kThreads, 0, s>>>(P);
    else qkv_rope_kernel<128, false, APPEND><<<grid, kThreads, 0, s>>>(P);
  } else {
    if (inter) qkv_rope_kernel<64, true, APPEND><<<grid, kThreads, 0, s>>>(P);
    else qkv_rope_kernel<64, false, APPEND><<<grid, kThreads, 0, s>>>(P);
  }
  prof_after(s);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- gradient --
struct BwdP {
  RopeArgs r;
  const void *dq, *dk, *dv;  // T
  const __nv_bfloat16* qkv;
  int64_t ld, ld_d;
  const int32_t* positions;
  __nv_bfloat16* dqkv;
  float* partial;  // [grid][2][D], with a weight
  uint32_t items, parts, steps_per_part;
  int S, H, H_kv;
};

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  unpack8(__ldg(reinterpret_cast<const uint4*>(p)), x);
}

constexpr int kBwdUnroll = 2;

template <int D, bool INTER, class T>
__global__ void __launch_bounds__(kThreads) qkv_rope_bwd_kernel(const __grid_constant__ BwdP P) {
  using L = RopeLane<D, INTER>;
  __shared__ float s_dw[kWarps][2][D];
  L L_;
  L_.init(P.r.freq, P.r.R);
  const int nq = (P.H + L::kHeads - 1) / L::kHeads, nk = (P.H_kv + L::kHeads - 1) / L::kHeads;
  const int wib = threadIdx.x >> 5;
  const uint32_t warp = blockIdx.x * kWarps + wib, warps = gridDim.x * kWarps;
  float dwq[8], dwk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;

  for (uint32_t item = warp; item < P.items; item += warps) {
    const uint32_t t = item / P.parts, part = item - t * P.parts;
    const uint32_t bi = t / (uint32_t)P.S, si = t - bi * (uint32_t)P.S;
    const int pos = P.positions ? __ldg(P.positions + t) : (int)si;
    const int lo = (int)(part * P.steps_per_part), hi = lo + (int)P.steps_per_part;
    float c[8], s[8];
    L_.angles(pos, P.r.amplitude, c, s);
    __nv_bfloat16* drow = P.dqkv + (int64_t)t * P.ld_d;
    const __nv_bfloat16* xrow = P.qkv + (int64_t)t * P.ld;

    auto run = [&](int first, int steps, int n, int head0, const void* dsrc,
                   const __nv_bfloat16* w, bool rotate, float (&dw)[8]) {
      const int from = max(lo, first) - first, to = min(hi, first + steps) - first;
      if (from >= to) return;
      const T* dy0 = static_cast<const T*>(dsrc) + ((int64_t)bi * n * P.S + si) * D + L_.chunk * 8;
      float wv[8];
      if (w) L_.weight(w, wv);
      for (int u0 = from; u0 < to; u0 += kBwdUnroll) {
        float dy[kBwdUnroll][8];
        uint4 xr[kBwdUnroll];
#pragma unroll
        for (int u = 0; u < kBwdUnroll; ++u) {
          const int h = (u0 + u) * L::kHeads + L_.sub;
          const bool live = u0 + u < to && h < n;
          xr[u] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 8; ++e) dy[u][e] = 0.f;
          if (live) {
            load8(dy0 + (int64_t)h * P.S * D, dy[u]);
            if (w)
              xr[u] = __ldg(reinterpret_cast<const uint4*>(xrow + (int64_t)(head0 + h) * D) +
                            L_.chunk);
          }
        }
#pragma unroll
        for (int u = 0; u < kBwdUnroll; ++u) {
          if (u0 + u >= to) break;
          const int h = (u0 + u) * L::kHeads + L_.sub;
          float g[8];
          if (rotate) {
            float o[8];
            L_.other(dy[u], o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              g[e] = L_.rot ? fmaf(dy[u][e], c[e], -(o[e] * s[e])) : dy[u][e];
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = dy[u][e];
          }
          if (w) {
            float x[8], ss = 0.f, sd = 0.f;
            unpack8(xr[u], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
            const float r = rsqrtf(L::head_sum(ss) * (1.f / D) + P.r.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x[e] *= r;
              dw[e] = fmaf(g[e], x[e], dw[e]);
              g[e] *= wv[e];
              sd = fmaf(g[e], x[e], sd);
            }
            sd = L::head_sum(sd) * (1.f / D);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = r * fmaf(-x[e], sd, g[e]);
          }
          if (h < n) reinterpret_cast<uint4*>(drow + (int64_t)(head0 + h) * D)[L_.chunk] = pack8(g);
        }
      }
    };
    float none[8];
    run(0, nq, P.H, 0, P.dq, P.r.w_q, true, dwq);
    run(nq, nk, P.H_kv, P.H, P.dk, P.r.w_k, true, dwk);
    run(nq + nk, nk, P.H_kv, P.H + P.H_kv, P.dv, nullptr, false, none);
  }

  if (P.r.w_q || P.r.w_k) {
    // Heads of one warp step, then the block's warps, in fixed order.
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = L::kLanes; o < 32; o <<= 1) {
        dwq[e] += __shfl_xor_sync(0xffffffffu, dwq[e], o);
        dwk[e] += __shfl_xor_sync(0xffffffffu, dwk[e], o);
      }
    }
    if (L_.sub == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s_dw[wib][0][L_.chunk * 8 + e] = dwq[e];
        s_dw[wib][1][L_.chunk * 8 + e] = dwk[e];
      }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += (&s_dw[w][0][0])[x];
      P.partial[(int64_t)blockIdx.x * 2 * D + x] = v;
    }
  }
}

// dw = sum of the blocks' partials, in a fixed order: thread (y, x) adds rows y,
// y + 8, ..., then the eight of an element are added.
__global__ void __launch_bounds__(1024) qkv_rope_dw_kernel(const float* partial, int rows, int D,
                                                           float* dw_q, float* dw_k) {
  __shared__ float sm[8][128];
  const int x = threadIdx.x & 127, y = threadIdx.x >> 7;
  float* const dst = blockIdx.x ? dw_k : dw_q;
  if (!dst) return;
  float v = 0.f;
  if (x < D)
    for (int r = y; r < rows; r += 8) v += partial[((int64_t)r * 2 + blockIdx.x) * D + x];
  sm[y][x] = v;
  __syncthreads();
  if (y == 0 && x < D) {
#pragma unroll
    for (int j = 1; j < 8; ++j) v += sm[j][x];
    dst[x] = v;
  }
}

template <int D, class T>
void launch_bwd(const BwdP& P, unsigned grid, cudaStream_t s) {
  if (P.r.inter) qkv_rope_bwd_kernel<D, true, T><<<grid, kThreads, 0, s>>>(P);
  else qkv_rope_bwd_kernel<D, false, T><<<grid, kThreads, 0, s>>>(P);
}

}  // namespace

cudaError_t qkv_rope_launch(const RopeArgs& r, const void* qkv, int64_t ld,
                            const int32_t* positions, int B, int S, int H, int H_kv, int D, void* q,
                            void* k, void* v, cudaStream_t s) {
  FwdP P{};
  P.r = r;
  P.qkv = static_cast<const __nv_bfloat16*>(qkv);
  P.ld = ld;
  P.positions = positions;
  P.q = static_cast<__nv_bfloat16*>(q);
  P.k = static_cast<__nv_bfloat16*>(k);
  P.v = static_cast<__nv_bfloat16*>(v);
  P.N = (uint32_t)((int64_t)B * S);
  P.S = S;
  P.H = H;
  P.H_kv = H_kv;
  return launch_fwd<false>(P, D, s);
}

cudaError_t kv_append_launch(const RopeArgs& r, const PagesArgs& pg, const void* qkv, int64_t ld,
                             const int32_t* positions, int64_t N, int H, void* q, cudaStream_t s) {
  FwdP P{};
  P.r = r;
  P.pg = pg;
  P.qkv = static_cast<const __nv_bfloat16*>(qkv);
  P.ld = ld;
  P.positions = positions;
  P.q = static_cast<__nv_bfloat16*>(q);
  P.N = (uint32_t)N;
  P.S = 1;
  P.H = H;
  P.H_kv = pg.H_kv;
  return launch_fwd<true>(P, pg.D, s);
}

size_t qkv_rope_bwd_workspace(int D) { return (size_t)kRopeBwdMaxGrid * 2 * D * sizeof(float); }

cudaError_t qkv_rope_bwd_launch(const RopeArgs& r, const void* dq, const void* dk, const void* dv,
                                const void* qkv, int64_t ld, const int32_t* positions, int B,
                                int S, int H, int H_kv, int D, bool bf16, void* dqkv, int64_t ld_d,
                                float* dw_q, float* dw_k, void* workspace, cudaStream_t s) {
  BwdP P{};
  P.r = r;
  P.dq = dq;
  P.dk = dk;
  P.dv = dv;
  P.qkv = static_cast<const __nv_bfloat16*>(qkv);
  P.ld = ld;
  P.ld_d = ld_d;
  P.positions = positions;
  P.dqkv = static_cast<__nv_bfloat16*>(dqkv);
  P.partial = static_cast<float*>(workspace);
  P.S = S > 0 ? S : 1;
  P.H = H;
  P.H_kv = H_kv;
  const int64_t N = (int64_t)B * S;
  const int heads = 32 / (D / 8);
  const int steps = (H + heads - 1) / heads + 2 * ((H_kv + heads - 1) / heads);
  const int64_t blocks_max = std::min<int64_t>((int64_t)sm_count() * 3, kRopeBwdMaxGrid);
  split_items(N, steps, blocks_max * kWarps, &P.parts, &P.steps_per_part);
  const int64_t items = N * P.parts;
  if (items > 0x7fffffffll) return cudaErrorNotSupported;
  P.items = (uint32_t)items;
  const unsigned grid = (unsigned)std::min<int64_t>((items + kWarps - 1) / kWarps, blocks_max);
  prof_before(s, STT_KERNEL_QKV_ROPE_BWD);
  if (grid > 0) {
    if (D == 128) {
      if (bf16) launch_bwd<128, __nv_bfloat16>(P, grid, s);
      else launch_bwd<128, float>(P, grid, s);
    } else {
      if (bf16) launch_bwd<64, __nv_bfloat16>(P, grid, s);
      else launch_bwd<64, float>(P, grid, s);
    }
  }
  // No tokens: the weights' gradients are zero.
  if (dw_q || dw_k) qkv_rope_dw_kernel<<<2, 1024, 0, s>>>(P.partial, (int)grid, D, dw_q, dw_k);
  prof_after(s);
  return cudaGetLastError();
}

STT_DEFINE_ERROR_ACCESSOR(qkv_rope_error_word)

}  // namespace stt
