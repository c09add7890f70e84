// soft_ce_topk.cu -- cross-entropy of a row's softmax against a teacher's top
// logits, with its gradient: the soft-CE for targets that are stored as K logits a
// token and not as a whole row.
//
//   p_k = exp(t_k / tau - L),  L = lse, or the logarithm of their sum of exponentials
//   s = sum_k p_k,  pi = softmax(z / tau)
//   l = s log sum_v exp(z_v / tau) - sum_k p_k z_{i_k} / tau
//   dz_v = g / tau (s pi_v - sum over k with i_k = v of p_k)
//
// Bound by HBM: a logit is read once and its gradient written once.  A cluster of C
// CTAs takes a row, each its slice in shared memory (bulk copies); the maximum and sum
// of every slice, and its part of sum p z, are exchanged through distributed shared
// memory, and the gradient is written out of shared memory.  The teacher's entries are
// held by the threads: an entry's CTA writes its element again after the dense pass.
// Entries of the same token are found with a bit map over the slice; only then are
// they added up, in their order.
#include <algorithm>
#include <cmath>

#include "../../include/stt.h"
#include "row_slice.cuh"

namespace stt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunks = 8;
constexpr int kEntries = kSoftCeTopkMaxK / kThreads;  // of the teacher's, to a thread
constexpr int kSliceBytes = 40 * 1024;  // preferred bytes of a slice
constexpr float kLog2E = 1.4426950408889634f;

struct Params {
  SoftCeTopkArgs a;
  float inv_tau, c;   // 1 / tau, log2(e) / tau
  int C, per, chunk;  // CTAs of a row, pieces of a CTA, pieces of a copy
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The block's sum, in a fixed order; ends with a __syncthreads().
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float all = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) all += s[w];
  __syncthreads();
  return all;
}
__device__ __forceinline__ float block_max(float v, float* s) {
  v = warp_max(v);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float all = s[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) all = fmaxf(all, s[w]);
  __syncthreads();
  return all;
}

template <class T>
__device__ __forceinline__ void store_piece(T* dst, const float (&y)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    st_global_cs_f4(reinterpret_cast<float*>(dst), make_float4(y[0], y[1], y[2], y[3]));
  } else {
    st_global_cs_f4(reinterpret_cast<float*>(dst),
                    make_float4(__uint_as_float(pack_bf16(y[0], y[1])),
                                __uint_as_float(pack_bf16(y[2], y[3])),
                                __uint_as_float(pack_bf16(y[4], y[5])),
                                __uint_as_float(pack_bf16(y[6], y[7]))));
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads) soft_ce_topk_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(128) unsigned char smem[];  // the slice, its bit map, the entries
  __shared__ uint64_t bars[kMaxChunks];
  __shared__ float red[2 * kWarps];
  __shared__ __align__(16) float4 s_part;
  __shared__ int s_twice;
  constexpr int G = RowSlice<T>::G;
  const SoftCeTopkArgs& A = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)P.C);
  const int64_t row = blockIdx.x / (unsigned)P.C;
  const float g = A.g[row];
  const RowSlice<T> S(static_cast<const T*>(A.z) + row * A.ld_z, A.V, rank, P.per);
  T* const out = static_cast<T*>(A.dz) + row * A.ld_dz;
  // The gradient's pieces lie as the logits' do, or it goes element by element.
  const bool vec = ((reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(S.row)) & 15u) == 0;

  // Writes piece p of the gradient.
  auto put = [&](int p, const float (&y)[G]) {
    const int v = S.index(p);
    if (vec && S.whole(p)) {
      store_piece<T>(out + v, y);
    } else {
#pragma unroll
      for (int e = 0; e < G; ++e)
        if (v + e >= 0 && v + e < A.V) out[v + e] = (T)y[e];
    }
  };
  auto masked = [&] {
    const float zero[G] = {};
    for (int p = tid; p < S.pieces; p += kThreads) put(p, zero);
    if (rank == 0 && tid == 0) {
      if (A.row_loss) A.row_loss[row] = 0.f;
      A.wl[row] = 0.f;
    }
  };
  if (g == 0.f) {  // the same in every CTA of the row
    masked();
    return;
  }
  T* const zs = reinterpret_cast<T*>(smem);
  const int words = (P.per * G + 31) / 32;
  uint32_t* const bits = reinterpret_cast<uint32_t*>(smem + (size_t)P.per * 16);
  int* const ent_v = reinterpret_cast<int*>(bits + words);
  float* const ent_p = reinterpret_cast<float*>(ent_v + A.K);
  for (int w = tid; w < words; w += kThreads) bits[w] = 0;
  if (tid == 0) s_twice = 0;
  fetch_slice(S, zs, bars, P.chunk);

  // ---- the teacher's entries, k = tid, tid + kThreads, ..
  float p[kEntries];
  int at[kEntries];  // place in the slice, -1: not here
  float s = 0.f;
  {
    float L;
    int v[kEntries];
#pragma unroll
    for (int j = 0; j < kEntries; ++j) {
      const int k = tid + j * kThreads;
      v[j] = -1;
      p[j] = -INFINITY;
      if (k < A.K) {
        v[j] = __ldg(A.indices + row * A.K + k);
        if (v[j] >= 0 && v[j] < A.V) p[j] = __ldg(A.values + row * A.K + k) * P.inv_tau;
        else v[j] = -1;
      }
    }
    if (A.lse) {
      L = __ldg(A.lse + row);
    } else {
      float m = p[0], e = 0.f;
#pragma unroll
      for (int j = 1; j < kEntries; ++j) m = fmaxf(m, p[j]);
      m = block_max(m, red);
      if (m == -INFINITY) m = 0.f;
#pragma unroll
      for (int j = 0; j < kEntries; ++j) e += ex2((p[j] - m) * kLog2E);
      e = block_sum(e, red);
      L = e == 0.f ? 0.f : m + logf(e);
    }
#pragma unroll
    for (int j = 0; j < kEntries; ++j) {
      p[j] = v[j] < 0 ? 0.f : ex2((p[j] - L) * kLog2E);
      s += p[j];
      const int x = v[j] - S.first;
      at[j] = v[j] >= 0 && x >= 0 && x < S.pieces * G ? x : -1;
      if (at[j] >= 0 && atomicOr(&bits[at[j] >> 5], 1u << (at[j] & 31)) >> (at[j] & 31) & 1u)
        s_twice = 1;
    }
    s = block_sum(s, red);
  }

  // ---- the slice's maximum and sum of exponentials, as it arrives
  constexpr int U = 16 / G;  // pieces taken together
  float m = -INFINITY, l = 0.f;
  const int n_chunks = (S.pieces + P.chunk - 1) / P.chunk;
  for (int c = 0; c < n_chunks; ++c) {
    mbar_wait(&bars[c], 0, STT_DEVERR_CE_WAIT);
    const int end = min(S.pieces, (c + 1) * P.chunk);
    for (int q = c * P.chunk + tid; q < end; q += U * kThreads) {
      float x[U][G];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (q + u * kThreads < end) {
          unpack_piece(*reinterpret_cast<const uint4*>(zs + (q + u * kThreads) * G), x[u]);
        } else {
#pragma unroll
          for (int e = 0; e < G; ++e) x[u][e] = -INFINITY;
        }
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < G; ++e) top = fmaxf(top, x[u][e]);
      const float base = top == -INFINITY ? 0.f : top;
      l *= ex2((m - base) * P.c);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < G; ++e) l += ex2((x[u][e] - base) * P.c);
      m = top;
    }
  }
  // What the entries here contribute to sum p z; p = 0 counts for nothing whatever z is.
  float d = 0.f;
#pragma unroll
  for (int j = 0; j < kEntries; ++j)
    if (at[j] >= 0 && p[j] != 0.f) d = fmaf(p[j], (float)zs[at[j]] * P.inv_tau, d);

  // ---- the row's, through distributed shared memory
  {
    const float top = warp_max(m), base = top == -INFINITY ? 0.f : top;
    l = warp_sum(l == 0.f ? 0.f : l * ex2((m - base) * P.c));
    if (lane == 0) {
      red[warp] = top;
      red[kWarps + warp] = l;
    }
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = fmaxf(m, red[w]);
    l = 0.f;
    const float b = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) l += red[kWarps + w] == 0.f ? 0.f : red[kWarps + w] * ex2((red[w] - b) * P.c);
    __syncthreads();
    d = block_sum(d, red);
  }
  if (P.C > 1) {
    if (tid == 0) s_part = make_float4(m, l, d, 0.f);
    cluster_sync();
    float4 o = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    if (lane < P.C) o = ld_shared_cluster_f4(mapa_shared(smem_u32(&s_part), (uint32_t)lane));
    cluster_arrive_release();  // done with the neighbours' shared memory; waited for at the end
    m = warp_max(o.x);
    const float b = m == -INFINITY ? 0.f : m;
    l = warp_sum(o.y == 0.f ? 0.f : o.y * ex2((o.x - b) * P.c));
    d = warp_sum(o.z);
  }

  if (m == -INFINITY && l == 0.f) {
    masked();  // no logit at all: nothing to learn
  } else {
    const float scale = g * P.inv_tau, a = scale * s / l;
    for (int q = tid; q < S.pieces; q += kThreads) {
      float x[G];
      unpack_piece(*reinterpret_cast<const uint4*>(zs + q * G), x);
#pragma unroll
      for (int e = 0; e < G; ++e) x[e] = ex2((x[e] - m) * P.c) * a;
      put(q, x);
    }
    const bool twice = s_twice != 0;  // set before the last barriers
    if (twice) {
#pragma unroll
      for (int j = 0; j < kEntries; ++j) {
        const int k = tid + j * kThreads;
        if (k < A.K) {
          ent_v[k] = at[j];
          ent_p[k] = p[j];
        }
      }
    }
    __syncthreads();  // the dense gradient is written
#pragma unroll
    for (int j = 0; j < kEntries; ++j) {
      if (at[j] < 0) continue;
      float t = p[j];
      bool mine = true;
      if (twice) {
        t = 0.f;
        for (int k = 0; k < A.K; ++k) {
          if (ent_v[k] != at[j]) continue;
          if (k < tid + j * kThreads) mine = false;  // the first of a token's entries writes
          t += ent_p[k];
        }
      }
      if (mine)
        out[S.first + at[j]] = (T)fmaf(ex2(((float)zs[at[j]] - m) * P.c), a, -t * scale);
    }
    if (rank == 0 && tid == 0) {
      const float loss = fmaf(s, m * P.inv_tau + logf(l), -d);
      if (A.row_loss) A.row_loss[row] = loss;
      A.wl[row] = g * loss;
    }
  }
  __syncwarp();
  if (P.C > 1) cluster_wait_acquire();
}

}  // namespace

cudaError_t soft_ce_topk_launch(const SoftCeTopkArgs& a, cudaStream_t s) {
  const int size = a.bf16 ? 2 : 4;
  Params P{};
  P.a = a;
  P.inv_tau = 1.f / a.temperature;
  P.c = (float)(1.4426950408889634 / (double)a.temperature);
  int C = (int)((a.V * (int64_t)size + kSliceBytes - 1) / kSliceBytes);
  C = std::max(1, std::min(C, kRowMaxCtas));
  while (C < kRowMaxCtas && a.N * 2 * C <= sm_count() && slice_pieces(a.V, size, C) >= 2 * kThreads) C *= 2;
  C = std::min(C, kRowMaxCtas);
  P.C = C;
  P.per = (int)slice_pieces(a.V, size, C);
  const int round = 512;
  P.chunk = ((P.per + kMaxChunks - 1) / kMaxChunks + round - 1) / round * round;
  const int smem = P.per * 16 + (P.per * (16 / size) + 31) / 32 * 4 + a.K * 8;
  prof_before(s, STT_KERNEL_SOFT_CE_TOPK);
  cudaError_t e = a.N == 0 ? cudaSuccess
                  : a.bf16 ? launch_rows(soft_ce_topk_kernel<__nv_bfloat16>, P, a.N, C, kThreads, smem, s)
                           : launch_rows(soft_ce_topk_kernel<float>, P, a.N, C, kThreads, smem, s);
  if (e == cudaSuccess) e = soft_ce_loss_sum_launch(a.wl, a.N, a.loss, s);
  prof_after(s);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

STT_DEFINE_ERROR_ACCESSOR(soft_ce_topk_error_word)
STT_DEFINE_BUDGET_SETTER(soft_ce_topk_set_wait_budget)

}  // namespace stt
