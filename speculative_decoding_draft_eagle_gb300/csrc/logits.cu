// logits.cu -- the target's logits to the distributions that verification tests
// against: penalties for repeated tokens, bias, grammar mask, temperature,
// softmax.
//
// One block per row.  The vocabulary is taken in slices whose token counts fit
// in shared memory: the block counts the row's history over the slice, applies
// the penalties, bias and mask, writes the result and keeps a running maximum,
// sum and argmax; a second pass turns the row into probabilities.
#include <algorithm>

#include "../../include/stt.h"
#include "internal.h"
#include "ptx.cuh"

namespace stt {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSlice = 8192;
constexpr uint32_t kPrompt = 0x80000000u;  // the token is in the prompt

// The row's logit after penalties, bias and mask, each step rounded as written.
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

// Argmax order: larger first, then the lower index.
__device__ __forceinline__ bool better(float a, int ia, float b, int ib) {
  return a > b || (a == b && ia < ib);
}

template <class T>
__global__ void __launch_bounds__(kThreads) logits_simple(const __grid_constant__ LogitsArgs P) {
  __shared__ uint32_t count[kSlice];
  __shared__ float s_m[kWarps], s_l[kWarps];
  __shared__ int s_i[kWarps];
  const int tid = threadIdx.x, r = blockIdx.x, b = r / P.rows, i = r - b * P.rows;
  const float T_ = P.temperature ? P.temperature[b] : 1.f;
  const float t = T_ > 0.f ? T_ : 1.f;
  const Penalty pen{P.repetition ? P.repetition[b] : 1.f, P.frequency ? P.frequency[b] : 0.f,
                    P.presence ? P.presence[b] : 0.f};
  const int t0 = P.tokens ? P.cu_tokens[b] : 0, t1 = P.tokens ? P.cu_tokens[b + 1] : 0;
  const int np = P.n_prompt ? P.n_prompt[b] : 0;
  const T* z = static_cast<const T*>(P.z) + (int64_t)r * P.V;
  float* out = P.out + (int64_t)r * P.V;
  const float* bias =
      P.bias_rows ? P.bias + (P.bias_rows > 1 ? (int64_t)b * P.V : 0) : nullptr;
  const uint32_t* mask = P.mask ? P.mask + (int64_t)r * ((P.V + 31) / 32) : nullptr;

  float m = -INFINITY, l = 0.f;
  int best = P.V;
  for (int v0 = 0; v0 < P.V; v0 += kSlice) {
    const int v1 = min(P.V, v0 + kSlice);
    for (int v = tid; v < kSlice; v += kThreads) count[v] = 0;
    __syncthreads();
    for (int x = t0 + tid; x < t1; x += kThreads) {
      const int v = P.tokens[x];
      if (v >= v0 && v < v1) {
        if (x - t0 < np) atomicOr(&count[v - v0], kPrompt);
        else atomicAdd(&count[v - v0], 1u);
      }
    }
    for (int x = tid; P.draft && x < i; x += kThreads) {
      const int v = P.draft[(int64_t)b * P.draft_ld + x];
      if (v >= v0 && v < v1) atomicAdd(&count[v - v0], 1u);
    }
    __syncthreads();
    for (int v = v0 + tid; v < v1; v += kThreads) {
      float x = pen((float)z[v], count[v - v0]);
      if (bias) x = __fadd_rn(x, bias[v]);
      if (mask && !((mask[v >> 5] >> (v & 31)) & 1u)) x = -INFINITY;
      const float y = __fdiv_rn(x, t);
      out[v] = y;
      if (T_ == 0.f) {
        if (better(x, v, m, best)) {
          m = x;
          best = v;
        }
      } else {
        if (y > m || isnan(y)) {
          l = l * expf(m - y);
          m = y;
        }
        if (y > -INFINITY || isnan(y)) l += expf(y - m);
      }
    }
    __syncthreads();
  }
  if (P.raw) return;
  // Block-wide maximum and sum, or argmax.
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
    const int i2 = __shfl_xor_sync(0xffffffffu, best, o);
    if (T_ == 0.f) {
      if (better(m2, i2, m, best)) { m = m2; best = i2; }
    } else {
      const float mn = fmaxf(m, m2);
      l = (mn == -INFINITY) ? l + l2 : l * expf(m - mn) + l2 * expf(m2 - mn);
      m = mn;
    }
  }
  if ((tid & 31) == 0) { s_m[tid >> 5] = m; s_l[tid >> 5] = l; s_i[tid >> 5] = best; }
  __syncthreads();
  m = s_m[0]; l = s_l[0]; best = s_i[0];
  for (int w = 1; w < kWarps; ++w) {
    if (T_ == 0.f) {
      if (better(s_m[w], s_i[w], m, best)) { m = s_m[w]; best = s_i[w]; }
    } else {
      const float mn = fmaxf(m, s_m[w]);
      l = (mn == -INFINITY) ? l + s_l[w] : l * expf(m - mn) + s_l[w] * expf(s_m[w] - mn);
      m = mn;
    }
  }
  for (int v = tid; v < P.V; v += kThreads) {
    if (T_ == 0.f) out[v] = (v == best && m > -INFINITY) ? 1.f : 0.f;
    else out[v] = (m == -INFINITY && l == 0.f) ? 0.f : expf(out[v] - m) / l;
  }
}

}  // namespace

cudaError_t logits_launch(const LogitsArgs& a, cudaStream_t s) {
  prof_before(s, STT_KERNEL_LOGITS);
  if (a.bf16) logits_simple<__nv_bfloat16><<<a.N, kThreads, 0, s>>>(a);
  else logits_simple<float><<<a.N, kThreads, 0, s>>>(a);
  prof_after(s);
  return cudaGetLastError();
}

}  // namespace stt
