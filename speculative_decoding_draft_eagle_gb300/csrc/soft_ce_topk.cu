// soft_ce_topk.cu -- cross-entropy of a row's softmax against a teacher's top
// logits, with its gradient: the soft-CE for targets that are stored as K logits a
// token and not as a whole row.
//
//   p_k = exp(t_k / tau - L),  L = lse, or the logarithm of their sum of exponentials
//   s = sum_k p_k,  pi = softmax(z / tau)
//   l = s log sum_v exp(z_v / tau) - sum_k p_k z_{i_k} / tau
//   dz_v = g / tau (s pi_v - sum over k with i_k = v of p_k)
//
// The loss is taken as s log sum_v exp((z_v - m) / tau) + sum_k p_k (m - z_{i_k}) / tau, m = max z:
// two sums without a minus, the same for logits that are all larger by a constant.
//
// Bound by HBM: a logit is read once and its gradient written once.  A cluster of C
// CTAs takes a row, each its slice in shared memory (bulk copies); the maximum and sum
// of every slice, and its parts of sum p z and sum p, go to the others by st.async, which signals
// an mbarrier there (a cluster barrier would wait for stores to drain), and the gradient is
// written out of shared memory.  One warp looks through the teacher's entries meanwhile
// and lists the slice's own; their elements are written again after the dense pass.
// Entries of the same token are found by comparison, or among more than 32 with a bit map
// over the slice; only then are they added up, in their order.
//
// 8192 fp32 rows of 151936, a fifth masked, K 128: 1387 us, 6.5 TB/s (0.97); 4096 bf16 rows of
// 128256, K 64: 376 us, 5.6 TB/s (0.84); 999 fp32 rows of 50257: 66 us (0.80); 64 bf16 rows of
// 32000, K 8, with the loss's sum: 11 us.  On the way: cluster barriers that order memory, which
// wait for stores on their way, and entries found by atomics 2220 us for the first, without them
// 1446; slices of three CTAs on an SM 1374; the loss from differences and waits that give up once
// 1387.  A persistent form took 2778 and was left out.
#include <algorithm>
#include <cmath>

#include "../../include/stt.h"
#include "attn_common.cuh"
#include "row_slice.cuh"

namespace stt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunks = 8;
// Preferred bytes of a slice: three CTAs on an SM.  (8192 fp32 rows of 151936 / 4096 bf16 rows of
// 128256: 24 KB 1470 / 463 us, 40 KB 1447 / 397, 56 KB 1507 / 372, 62 KB 1383 / 373, 72 KB
// 1376 / 396, 76 KB, which is two on an SM, 1582 / 396.)
constexpr int kSliceBytes = 62 * 1024;

struct Params {
  SoftCeTopkArgs a;
  float inv_tau, inv_lo, c;  // 1 / tau, what its rounding left, log2(e) / tau
  int C, per, chunk;         // CTAs of a row, pieces of a CTA, pieces of a copy
  bool withhold, no_copies;  // test hooks: the first CTA of a row sends no part, fetches nothing
};

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
  extern __shared__ __align__(128) unsigned char smem[];  // the slice, its bit map, its entries
  __shared__ uint64_t bars[kMaxChunks], bar_part;
  __shared__ __align__(16) float red[4][kWarps];
  __shared__ __align__(16) float4 s_part[kRowMaxCtas];
  __shared__ int s_entries, s_twice;
  __shared__ float s_sum;
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
  int* const ent_v = reinterpret_cast<int*>(bits + words);  // place in the slice
  float* const ent_p = reinterpret_cast<float*>(ent_v + A.K);
  if (tid == 0) {
    mbar_init(&bar_part, 1);
    fence_mbar_init();
    if (P.C > 1) mbar_arrive_expect_tx(&bar_part, (uint32_t)P.C * 16u);
  }
  fetch_slice(S, zs, bars, P.chunk, P.no_copies && rank == 0);
  if (P.C > 1) cluster_arrive_relaxed();  // everyone runs before anyone writes to a neighbour

  // ---- the teacher's entries, by the last warp: p of all, and the list of the slice's own in
  // their order
  if (warp == kWarps - 1) {
    constexpr int kAhead = 4;  // groups of 32 entries whose loads are in flight
    const int32_t* const idx = A.indices + row * A.K;
    const float* const val = A.values + row * A.K;
    // f(group's tokens or -1, their t or -inf), kAhead groups at a time
    auto each = [&](auto&& f) {
      for (int k0 = 0; k0 < A.K; k0 += 32 * kAhead) {
        int v[kAhead];
        float t[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int k = k0 + u * 32 + lane;
          v[u] = k < A.K ? __ldg(idx + k) : -1;
          t[u] = k < A.K ? __ldg(val + k) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          // (A logit of -inf is no entry, whatever L is: with an L of -inf, a teacher row without
          // any, its exponent would be -inf + inf.)
          const bool there = v[u] >= 0 && v[u] < A.V && t[u] != -INFINITY;
          v[u] = there ? v[u] : -1;
          t[u] = there ? t[u] : -INFINITY;
        }
        f(v, t);
      }
    };
    float s = 0.f;
    int n = 0;
    auto list = [&](auto&& share) {
      each([&](const int (&v)[kAhead], const float (&t)[kAhead]) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const float p = v[u] < 0 ? 0.f : share(t[u]);
          s += p;
          const int at = v[u] - S.first;
          const bool here = v[u] >= 0 && at >= 0 && at < S.pieces * G;
          const uint32_t mask = __ballot_sync(0xffffffffu, here);
          if (here) {
            const int i = n + __popc(mask & ((1u << lane) - 1u));
            ent_v[i] = at;
            ent_p[i] = p;
          }
          n += __popc(mask);
        }
      });
    };
    // p = e^(t / tau - L) in one rounding at the difference's size, or e^((t - max t) / tau) over
    // their sum: t / tau by itself would cost its own size's bits, and may not be finite.
    if (A.lse) {
      const float L = __ldg(A.lse + row);
      list([&](float t) { return ex2(fmaf(t, P.inv_lo, fmaf(t, P.inv_tau, -L)) * kLog2e); });
    } else {
      float top = -INFINITY, e = 0.f;
      each([&](const int (&)[kAhead], const float (&t)[kAhead]) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) top = fmaxf(top, t[u]);
      });
      top = warp_max(top);
      const float first = top == -INFINITY ? 0.f : top;
      each([&](const int (&)[kAhead], const float (&t)[kAhead]) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) e += ex2((t[u] - first) * P.c);
      });
      e = warp_sum(e);
      const float inv_sum = e == 0.f ? 0.f : 1.f / e;
      list([&](float t) { return ex2((t - first) * P.c) * inv_sum; });
    }
    s = warp_sum(s);
    __syncwarp();
    // A token twice: up to 32 entries by comparison, more with the bit map.
    bool twice = false;
    if (n <= 32) {
      const int at = lane < n ? ent_v[lane] : -1 - lane;
      twice = __popc(__match_any_sync(0xffffffffu, at)) > 1;
    } else {
      for (int w = lane; w < words; w += 32) bits[w] = 0;
      __syncwarp();
      for (int i = lane; i < n; i += 32) {
        const int at = ent_v[i];
        twice |= atomicOr(&bits[at >> 5], 1u << (at & 31)) >> (at & 31) & 1u;
      }
    }
    twice = __any_sync(0xffffffffu, twice);
    if (lane == 0) {
      s_sum = s;
      s_entries = n;
      s_twice = twice;
    }
  }

  // ---- the slice's maximum and sum of exponentials, as it arrives
  constexpr int U = 16 / G;  // pieces taken together
  const uint64_t cc = f32x2(P.c, P.c);
  float m = -INFINITY, l = 0.f;
  const int n_chunks = (S.pieces + P.chunk - 1) / P.chunk;
  for (int c = 0; c < n_chunks; ++c) {
    if (!wait_slice(bars, c, n_chunks, STT_DEVERR_CE_WAIT)) break;
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
        for (int e = 0; e < G; e += 2) top = fmax3(top, x[u][e], x[u][e + 1]);
      const float base = top == -INFINITY ? 0.f : top;
      const uint64_t low = f32x2(-base, -base);
      uint64_t sum = f32x2(l * ex2((m - base) * P.c), 0.f);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < G; e += 2) {
          float y0, y1;
          unpack_f32x2(mul_f32x2(add_f32x2(f32x2(x[u][e], x[u][e + 1]), low), cc), y0, y1);
          sum = add_f32x2(sum, f32x2(ex2(y0), ex2(y1)));
        }
      float y0, y1;
      unpack_f32x2(sum, y0, y1);
      l = y0 + y1;
      m = top;
    }
  }

  // ---- the slice's, then the row's: a warp's lanes send the slice's part to the neighbours
  {
    const float top = warp_max(m), base = top == -INFINITY ? 0.f : top;
    l = warp_sum(l == 0.f ? 0.f : l * ex2((m - base) * P.c));
    if (lane == 0) {
      red[0][warp] = top;
      red[1][warp] = l;
    }
    __syncthreads();  // and the entries are listed
    // What the entries here contribute to sum p (z - max z) / tau, with the slice's maximum for the
    // row's: differences, so that an offset of all logits costs the loss no bits.  p = 0 counts for
    // nothing whatever z is.
    float d = 0.f, ps = 0.f;
    const int n = s_entries;
    if (warp * 32 < n) {
      static_assert(kWarps == 8, "two loads");
      const float4 a = *reinterpret_cast<const float4*>(&red[0][0]), b = *reinterpret_cast<const float4*>(&red[0][4]);
      float at = fmaxf(fmax3(fmax3(a.x, a.y, a.z), a.w, b.x), fmax3(b.y, b.z, b.w));
      at = at == -INFINITY ? 0.f : at;
      for (int i = tid; i < n; i += kThreads) {
        const float p = ent_p[i];
        if (p != 0.f) {
          d = fmaf(p, ((float)zs[ent_v[i]] - at) * P.inv_tau, d);
          ps += p;
        }
      }
      d = warp_sum(d);
      ps = warp_sum(ps);
    }
    if (lane == 0) {
      red[2][warp] = d;
      red[3][warp] = ps;
    }
    __syncthreads();
  }
  float d, ps;
  {
    // The slice's, from its warps'.
    auto slice = [&] {
      const bool has = lane < kWarps;
      const float a = has ? red[0][lane] : -INFINITY, b = has ? red[1][lane] : 0.f;
      m = warp_max(a);
      const float base = m == -INFINITY ? 0.f : m;
      l = warp_sum(b == 0.f ? 0.f : b * ex2((a - base) * P.c));
      d = warp_sum(has ? red[2][lane] : 0.f);
      ps = warp_sum(has ? red[3][lane] : 0.f);
    };
    if (P.C == 1) {
      slice();
    } else {
      cluster_wait_acquire();
      if (warp == 0) {
        slice();
        if (lane < P.C && !(P.withhold && rank == 0))
          st_async_f4(mapa_shared(smem_u32(&s_part[rank]), (uint32_t)lane), make_float4(m, l, d, ps),
                      mapa_shared(smem_u32(&bar_part), (uint32_t)lane));
        __syncwarp();
      }
      cluster_arrive_relaxed();  // this CTA has sent its part; waited for at the end
      mbar_wait_cluster(&bar_part, 0, STT_DEVERR_CE_WAIT);
      const float4 o = lane < P.C ? s_part[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      m = warp_max(o.x);
      const float base = m == -INFINITY ? 0.f : m;
      l = warp_sum(o.y == 0.f ? 0.f : o.y * ex2((o.x - base) * P.c));
      if (rank == 0 && warp == 0) {  // (A slice of -inf alone took its differences to 0.)
        const float shift = ((o.x == -INFINITY ? 0.f : o.x) - base) * P.inv_tau;
        d = warp_sum(o.w == 0.f ? o.z : fmaf(o.w, shift, o.z));
      }
    }
  }

  if (m == -INFINITY && l == 0.f) {
    masked();  // no logit at all: nothing to learn
  } else {
    const float scale = g * P.inv_tau, s = s_sum, a = scale * s / l;
    const uint64_t low = f32x2(-m, -m), aa = f32x2(a, a);
    auto gradient = [&](int q, float (&x)[G]) {
      unpack_piece(*reinterpret_cast<const uint4*>(zs + q * G), x);
#pragma unroll
      for (int e = 0; e < G; e += 2) {
        float y0, y1;
        unpack_f32x2(mul_f32x2(add_f32x2(f32x2(x[e], x[e + 1]), low), cc), y0, y1);
        unpack_f32x2(mul_f32x2(f32x2(ex2(y0), ex2(y1)), aa), x[e], x[e + 1]);
      }
    };
    if (vec) {
      // Whole pieces; the one or two others apart.
      const int lo = S.pieces > 0 && !S.whole(0) ? 1 : 0;
      const int hi = S.pieces > 0 && !S.whole(S.pieces - 1) ? S.pieces - 1 : S.pieces;
      T* const at = out + S.index(0);
#pragma unroll 4
      for (int q = lo + tid; q < hi; q += kThreads) {
        float x[G];
        gradient(q, x);
        store_piece<T>(at + q * G, x);
      }
      if (tid < 2 && S.pieces > 0) {
        const int q = tid == 0 ? 0 : S.pieces - 1;
        if (!S.whole(q) && (tid == 0 || S.pieces > 1)) {
          float x[G];
          gradient(q, x);
          put(q, x);
        }
      }
    } else {
      for (int q = tid; q < S.pieces; q += kThreads) {
        float x[G];
        gradient(q, x);
        put(q, x);
      }
    }
    __syncthreads();  // the dense gradient is written
    const int n = s_entries;
    const bool twice = s_twice != 0;
    for (int i = tid; i < n; i += kThreads) {
      const int at = ent_v[i];
      float t = ent_p[i];
      bool mine = true;
      if (twice) {
        t = 0.f;
        for (int k = 0; k < n; ++k) {
          if (ent_v[k] != at) continue;
          if (k < i) mine = false;  // the first of a token's entries writes
          t += ent_p[k];
        }
      }
      if (mine) out[S.first + at] = (T)fmaf(ex2(((float)zs[at] - m) * P.c), a, -t * scale);
    }
    if (rank == 0 && tid == 0) {
      const float loss = fmaf(s, logf(l), -d);  // both at least 0
      if (A.row_loss) A.row_loss[row] = loss;
      A.wl[row] = g * loss;
    }
  }
  // A CTA whose wait gave up may not leave while parts are on their way to it: everyone has
  // sent theirs, and they have landed.
  __syncwarp();
  if (P.C > 1) {
    cluster_wait_acquire();
    if (tid == 0) mbar_wait_cluster(&bar_part, 0, STT_DEVERR_CE_WAIT);
  }
}

}  // namespace

cudaError_t soft_ce_topk_launch(const SoftCeTopkArgs& a, cudaStream_t s) {
  const int size = a.bf16 ? 2 : 4;
  Params P{};
  P.a = a;
  P.inv_tau = 1.f / a.temperature;
  P.inv_lo = (float)(1.0 / (double)a.temperature - (double)P.inv_tau);
  P.c = (float)(1.4426950408889634 / (double)a.temperature);
  int C = (int)((a.V * (int64_t)size + kSliceBytes - 1) / kSliceBytes);
  C = std::max(1, std::min(C, kRowMaxCtas));
  while (C < kRowMaxCtas && a.N * 2 * C <= sm_count() && slice_pieces(a.V, size, C) >= 2 * kThreads) C *= 2;
  C = std::min(C, kRowMaxCtas);
  P.C = C;
  P.per = (int)slice_pieces(a.V, size, C);
  const int round = 1024;  // four pieces of fp32 to a thread, or eight of bf16
  P.chunk = ((P.per + kMaxChunks - 1) / kMaxChunks + round - 1) / round * round;
  const int smem = P.per * 16 + (P.per * (16 / size) + 31) / 32 * 4 + a.K * 8;
  P.no_copies = (debug_inject() & STT_INJECT_SLICE_WITHHOLD_COPIES) != 0;
  P.withhold = (debug_inject() & STT_INJECT_CE_TOPK_WITHHOLD_PARTS) != 0;
  prof_before(s, STT_KERNEL_SOFT_CE_TOPK);
  static Raised raised[2];
  cudaError_t e = a.N == 0 ? cudaSuccess
                  : a.bf16 ? launch_rows(soft_ce_topk_kernel<__nv_bfloat16>, P, a.N, C, kThreads, smem, raised[1], s)
                           : launch_rows(soft_ce_topk_kernel<float>, P, a.N, C, kThreads, smem, raised[0], s);
  if (e == cudaSuccess) e = soft_ce_loss_sum_launch(a.wl, a.N, a.loss, s);
  prof_after(s);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

STT_DEFINE_ERROR_ACCESSOR(soft_ce_topk_error_word)
STT_DEFINE_BUDGET_SETTER(soft_ce_topk_set_wait_budget)

}  // namespace stt
