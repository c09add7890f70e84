// logits.cu -- the target's logits to the distributions that verification tests
// against: penalties for repeated tokens, bias, grammar mask, temperature,
// softmax.
//
// A cluster of C CTAs takes a row, each a slice of the vocabulary, and reads it
// once: the slice stays in registers from the load to the store.  While the loads
// are under way the CTA counts the row's history over its slice in shared memory
// (whole numbers, so the order of the atomics does not matter; every CTA scans the
// whole history, which is short against the row).  Each thread then applies
// penalties, bias and mask to its elements, the CTA takes its maximum m and its
// sum l of e^(y - m), the C pairs are exchanged through distributed shared memory
// (one cluster barrier), and the exponentials leave scaled by e^(m - M) / L.  A
// greedy row exchanges the largest value and then the lowest index that has it.
// Bounded by HBM: 2 or 4 bytes read and 4 written per logit.
#include <algorithm>

#include "../../include/stt.h"
#include "internal.h"
#include "ptx.cuh"

namespace stt {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxCluster = 16;
constexpr int kMaxNv = 6;                  // 8-element chunks a thread holds at most
constexpr uint32_t kPrompt = 0x80000000u;  // the token is in the prompt
constexpr float kLog2E = 1.4426950408889634f;

struct Params {
  LogitsArgs a;
  int C, slice;  // CTAs per row, elements per CTA (a multiple of 8)
};

// A logit after the penalties, each step rounded as written.
struct Penalty {
  float rep, freq, pres;
  __device__ __forceinline__ float operator()(float z, uint32_t seen) const {
    if (seen) {
      z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
      const uint32_t c = seen & ~kPrompt;
      if (c) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)c)), pres);
    }
    return z;
  }
};

__device__ __forceinline__ void st_cluster_f2(uint32_t addr, float a, float b) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

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

// VEC: rows 16-byte aligned, a thread's chunk is 8 consecutive elements (vector
// loads and stores); else its elements are a block apart (any alignment).
template <class T, bool VEC, int NV>
__global__ void __launch_bounds__(kMaxThreads, NV <= 5 ? 2 : 1)
    logits_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(16) uint32_t count[];
  __shared__ float s_red[kMaxThreads / 32];
  __shared__ int s_idx[kMaxThreads / 32];
  __shared__ __align__(16) float2 s_pair[kMaxCluster];
  const LogitsArgs& A = P.a;
  const int tid = threadIdx.x, nt = blockDim.x, warps = nt >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)P.C), r = (int)(blockIdx.x / (unsigned)P.C);
  if (P.C > 1) cluster_arrive_release();  // everyone runs before anyone writes to a neighbour
  const int b = r / A.rows, i = r - b * A.rows;
  const int begin = rank * P.slice, len = min(P.slice, A.V - begin);
  const T* z = static_cast<const T*>(A.z) + (int64_t)r * A.V + begin;

  // Element e of chunk k, relative to the slice.
  auto at = [&](int k, int e) { return VEC ? (k * nt + tid) * 8 + e : (k * 8 + e) * nt + tid; };

  float x[NV][8];
  uint4 raw[NV];  // bf16 chunks as loaded
  if constexpr (VEC) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (at(k, 0) < len) {
        if constexpr (sizeof(T) == 2) {
          raw[k] = *reinterpret_cast<const uint4*>(z + at(k, 0));
        } else {
          const float4 p = *reinterpret_cast<const float4*>(z + at(k, 0));
          const float4 q = *reinterpret_cast<const float4*>(z + at(k, 4));
          x[k][0] = p.x; x[k][1] = p.y; x[k][2] = p.z; x[k][3] = p.w;
          x[k][4] = q.x; x[k][5] = q.y; x[k][6] = q.z; x[k][7] = q.w;
        }
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] = at(k, e) < len ? (float)z[at(k, e)] : 0.f;
  }

  const bool hist = A.tokens != nullptr || (A.draft != nullptr && i > 0);
  if (hist) {
    for (int v = tid * 4; v < P.slice; v += nt * 4)
      *reinterpret_cast<uint4*>(count + v) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (A.tokens) {
      const int t0 = A.cu_tokens[b], n = A.cu_tokens[b + 1] - t0;
      const int np = A.n_prompt ? A.n_prompt[b] : 0;
      const int32_t* tok = A.tokens + t0;
#pragma unroll 4
      for (int j = tid; j < n; j += nt) {
        const int v = __ldg(tok + j) - begin;
        if (v >= 0 && v < len) {
          if (j < np) atomicOr(&count[v], kPrompt);
          else atomicAdd(&count[v], 1u);
        }
      }
    }
    if (A.draft) {
      for (int j = tid; j < i; j += nt) {
        const int v = A.draft[(int64_t)b * A.draft_ld + j] - begin;
        if (v >= 0 && v < len) atomicAdd(&count[v], 1u);
      }
    }
    __syncthreads();
  }

  const float temp = A.temperature ? A.temperature[b] : 1.f;
  const Penalty pen{A.repetition ? A.repetition[b] : 1.f, A.frequency ? A.frequency[b] : 0.f,
                    A.presence ? A.presence[b] : 0.f};
  const float* bias =
      A.bias_rows ? A.bias + (A.bias_rows > 1 ? (int64_t)b * A.V : 0) + begin : nullptr;
  const uint32_t* mask = A.mask ? A.mask + (int64_t)r * ((A.V + 31) / 32) : nullptr;
  const bool bias_vec = VEC && (reinterpret_cast<uintptr_t>(bias) & 15u) == 0;

  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const bool live = at(k, 0) < len;
    if (VEC && !live) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] = -INFINITY;
      continue;
    }
    if constexpr (VEC && sizeof(T) == 2) {
      const uint32_t u[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[k][2 * e] = __uint_as_float(u[e] << 16);
        x[k][2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
      }
    }
    if (hist) {
      uint32_t c[8];
      if constexpr (VEC) {
        const uint4 p = *reinterpret_cast<const uint4*>(count + at(k, 0));
        const uint4 q = *reinterpret_cast<const uint4*>(count + at(k, 4));
        c[0] = p.x; c[1] = p.y; c[2] = p.z; c[3] = p.w;
        c[4] = q.x; c[5] = q.y; c[6] = q.z; c[7] = q.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = at(k, e) < len ? count[at(k, e)] : 0u;
      }
      if ((c[0] | c[1] | c[2] | c[3]) | (c[4] | c[5] | c[6] | c[7])) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] = pen(x[k][e], c[e]);
      }
    }
    if (bias) {
      if (bias_vec) {
        const float4 p = __ldg(reinterpret_cast<const float4*>(bias + at(k, 0)));
        const float4 q = __ldg(reinterpret_cast<const float4*>(bias + at(k, 4)));
        x[k][0] += p.x; x[k][1] += p.y; x[k][2] += p.z; x[k][3] += p.w;
        x[k][4] += q.x; x[k][5] += q.y; x[k][6] += q.z; x[k][7] += q.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at(k, e) < len) x[k][e] += __ldg(bias + at(k, e));
      }
    }
    if (mask) {
      if constexpr (VEC) {
        const int v = begin + at(k, 0);
        const uint32_t bits = __ldg(mask + (v >> 5)) >> (v & 31);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!((bits >> e) & 1u)) x[k][e] = -INFINITY;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int v = begin + at(k, e);
          if (at(k, e) < len && !((__ldg(mask + (v >> 5)) >> (v & 31)) & 1u)) x[k][e] = -INFINITY;
        }
      }
    }
    if constexpr (!VEC) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at(k, e) >= len) x[k][e] = -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, x[k][e]);
  }

  float* out = A.out + (int64_t)r * A.V + begin;
  auto store = [&](int k, const float (&y)[8]) {
    if constexpr (VEC) {
      if (at(k, 0) < len) {
        st_global_cs_f4(out + at(k, 0), make_float4(y[0], y[1], y[2], y[3]));
        st_global_cs_f4(out + at(k, 4), make_float4(y[4], y[5], y[6], y[7]));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at(k, e) < len) out[at(k, e)] = y[e];
    }
  };

  if (A.raw) {
    if (P.C > 1) cluster_wait_acquire();
    const float t = temp > 0.f ? temp : 1.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] = __fdiv_rn(x[k][e], t);
      store(k, x[k]);
    }
    return;
  }

  // The CTA's maximum.
  m = warp_max(m);
  if ((tid & 31) == 0) s_red[tid >> 5] = m;
  __syncthreads();
  m = s_red[0];
  for (int w = 1; w < warps; ++w) m = fmaxf(m, s_red[w]);
  const bool greedy = temp == 0.f;
  float l = 0.f;
  if (!greedy) {
    // y - m as (x - m) / temperature: exact zeros at the maximum, whatever its size.
    const float c = __fdiv_rn(kLog2E, temp), base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[k][e] = ex2((x[k][e] - base) * c);
        l += x[k][e];
      }
    l = warp_sum(l);
    __syncthreads();
    if ((tid & 31) == 0) s_red[tid >> 5] = l;
    __syncthreads();
    l = s_red[0];
    for (int w = 1; w < warps; ++w) l += s_red[w];
  }
  if (P.C > 1) {
    cluster_wait_acquire();
    if (tid < P.C) st_cluster_f2(mapa_shared(smem_u32(&s_pair[rank]), (uint32_t)tid), m, l);
    cluster_arrive_release();
    cluster_wait_acquire();
  } else {
    if (tid == 0) s_pair[0] = make_float2(m, l);
    __syncthreads();
  }
  float M = -INFINITY;
  for (int c = 0; c < P.C; ++c) M = fmaxf(M, s_pair[c].x);

  if (!greedy) {
    const float c = __fdiv_rn(kLog2E, temp), base = M == -INFINITY ? 0.f : M;
    float total = 0.f;
    for (int q = 0; q < P.C; ++q) {
      const float2 p = s_pair[q];
      total += p.y == 0.f ? 0.f : p.y * ex2((p.x - base) * c);
    }
    const float f = total == 0.f ? 0.f : ex2(((m == -INFINITY ? base : m) - base) * c) / total;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] *= f;
      store(k, x[k]);
    }
    return;
  }

  // The lowest index of the row's largest value.
  int best = 0x7fffffff;
#pragma unroll
  for (int k = NV - 1; k >= 0; --k)
#pragma unroll
    for (int e = 7; e >= 0; --e)
      if (x[k][e] == M && at(k, e) < len) best = begin + at(k, e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
  if ((tid & 31) == 0) s_idx[tid >> 5] = best;
  __syncthreads();
  for (int w = 0; w < warps; ++w) best = min(best, s_idx[w]);
  if (P.C > 1) {
    // s_pair has been read by every CTA before anyone writes it again.
    cluster_arrive_release();
    cluster_wait_acquire();
    if (tid < P.C)
      st_cluster_f2(mapa_shared(smem_u32(&s_pair[rank]), (uint32_t)tid), __int_as_float(best), 0.f);
    cluster_arrive_release();
    cluster_wait_acquire();
    for (int q = 0; q < P.C; ++q) best = min(best, __float_as_int(s_pair[q].x));
  }
  if (M == -INFINITY) best = -1;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[k][e] = begin + at(k, e) == best ? 1.f : 0.f;
    store(k, x[k]);
  }
}

using Kernel = void (*)(const Params);

template <class T, bool VEC>
Kernel pick(int nv) {
  switch (nv) {
    case 1: return logits_kernel<T, VEC, 1>;
    case 2: return logits_kernel<T, VEC, 2>;
    case 3: return logits_kernel<T, VEC, 3>;
    case 4: return logits_kernel<T, VEC, 4>;
    case 5: return logits_kernel<T, VEC, 5>;
    default: return logits_kernel<T, VEC, 6>;
  }
}

}  // namespace

cudaError_t logits_launch(const LogitsArgs& a, cudaStream_t s) {
  // CTAs per row: the fewest whose slice a CTA's registers hold at two CTAs an SM;
  // more while the rows alone leave SMs idle and a slice is worth splitting.
  int C = 1;
  auto slice_of = [&](int c) { return ((a.V + c - 1) / c + 7) / 8 * 8; };
  while (C < kMaxCluster && slice_of(C) > 5 * 8 * kMaxThreads) C *= 2;
  while (C < kMaxCluster && (int64_t)a.N * C * 2 <= sm_count() && slice_of(C) >= 4096) C *= 2;
  const int slice = slice_of(C);
  int threads = kMaxThreads;
  while (threads > 128 && slice <= 8 * (threads / 2)) threads /= 2;
  const int nv = (slice + 8 * threads - 1) / (8 * threads);
  if (nv > kMaxNv) return cudaErrorNotSupported;
  const uintptr_t zo = reinterpret_cast<uintptr_t>(a.z) | reinterpret_cast<uintptr_t>(a.out);
  const bool vec = a.V % 8 == 0 && (zo & 15u) == 0;
  const Kernel kern = a.bf16 ? (vec ? pick<__nv_bfloat16, true>(nv) : pick<__nv_bfloat16, false>(nv))
                             : (vec ? pick<float, true>(nv) : pick<float, false>(nv));
  const int smem = (a.tokens || a.draft) ? slice * 4 : 0;
  cudaError_t e;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  if (C > 8) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  Params P{a, C, slice};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.N * C), 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  prof_before(s, STT_KERNEL_LOGITS);
  e = cudaLaunchKernelEx(&cfg, kern, P);
  prof_after(s);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace stt
