// row_slice.cuh -- a row of logits cut into whole 16-byte pieces of memory, and
// the order of its elements: shared by the kernels that take, learn from and draw
// from the top of a distribution.
//
// A row of V elements starts anywhere (odd vocabularies, rows of a wider buffer).
// It is taken in the 16-byte pieces of memory that it touches; of the first and the
// last piece some elements may lie outside the row, and those are never read: such a
// piece goes element by element, with -inf for what is not the row's.
#pragma once

#include <atomic>
#include <climits>
#include <cstdint>
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace stt {

// Pieces of 16 bytes of the longest of C slices of V elements of `size` bytes, wherever
// the row starts.
inline int64_t slice_pieces(int64_t V, int size, int C) {
  const int64_t G = 16 / size;
  return ((V + 2 * G - 2) / G + C - 1) / C;
}

__device__ __forceinline__ void unpack_piece(const uint4& r, float (&x)[4]) {
  x[0] = __uint_as_float(r.x);
  x[1] = __uint_as_float(r.y);
  x[2] = __uint_as_float(r.z);
  x[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack_piece(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// The part of a row that CTA `rank` takes, `per` pieces to a CTA.
template <class T>
struct RowSlice {
  static constexpr int G = 16 / (int)sizeof(T);  // elements of a piece
  const T* row;
  int V;
  int first;   // index in the row of the slice's first element; negative before the row
  int pieces;

  __device__ __forceinline__ RowSlice(const T* row_, int V_, int rank, int per) : row(row_), V(V_) {
    const int shift = (int)((reinterpret_cast<uintptr_t>(row_) / sizeof(T)) % G);
    const int all = (V_ + shift + G - 1) / G;
    const int p0 = min(rank * per, all);
    pieces = min(per, all - p0);
    first = p0 * G - shift;
  }
  __device__ __forceinline__ int index(int piece) const { return first + piece * G; }
  __device__ __forceinline__ bool whole(int piece) const {
    const int v = index(piece);
    return v >= 0 && v + G <= V;
  }
  // A piece's elements, -inf outside the row.
  __device__ __forceinline__ void edge(int piece, float (&x)[G]) const {
#pragma unroll
    for (int e = 0; e < G; ++e) {
      const int v = index(piece) + e;
      x[e] = v >= 0 && v < V ? (float)row[v] : -INFINITY;
    }
  }
  __device__ __forceinline__ uint4 load(int piece) const {
    return *reinterpret_cast<const uint4*>(row + index(piece));
  }
};

// Brings a slice into shared memory at `dst`: whole pieces by bulk copies, `chunk`
// pieces on each of `bars` (initialised here), the others by the threads, before the
// __syncthreads() in here.  Called by all threads, at least 64 of them.  `withhold`, a test hook:
// no copy is issued, and no wait for one can end.
template <class T>
__device__ __forceinline__ void fetch_slice(const RowSlice<T>& s, T* dst, uint64_t* bars, int chunk,
                                            bool withhold) {
  constexpr int G = RowSlice<T>::G;
  const int tid = threadIdx.x;
  const int n_chunks = (s.pieces + chunk - 1) / chunk;
  if (tid == 0) {
    for (int c = 0; c < n_chunks; ++c) mbar_init(&bars[c], 1);
    fence_mbar_init();
    const int a = s.pieces > 0 && !s.whole(0) ? 1 : 0;
    const int b = s.pieces > 0 && !s.whole(s.pieces - 1) ? s.pieces - 1 : s.pieces;
    for (int c = 0; c < n_chunks && !withhold; ++c) {
      const int lo = max(a, c * chunk), hi = min(b, (c + 1) * chunk);
      const uint32_t bytes = hi > lo ? (uint32_t)(hi - lo) * 16u : 0u;
      mbar_arrive_expect_tx(&bars[c], bytes);
      if (bytes) bulk_load(dst + lo * G, s.row + s.index(lo), bytes, &bars[c]);
    }
  }
  if (tid >= 32 && tid < 32 + 2 * G) {
    const int e = (tid - 32) % G, piece = tid - 32 < G ? 0 : s.pieces - 1;
    if (piece < s.pieces && piece >= 0 && !s.whole(piece)) {
      const int v = s.index(piece) + e;
      dst[piece * G + e] = v >= 0 && v < s.V ? s.row[v] : (T)(-INFINITY);
    }
  }
  __syncthreads();
}
// Waits for a slice's c-th copies.  False: that gave up, and the caller waits for no more of them;
// they have been waited for once more, within one budget for all together, so that a CTA does not
// leave while they are on their way.  (Here and not at its end, where it took 2 % of a gradient's
// time.)
__device__ __forceinline__ bool wait_slice(uint64_t* bars, int c, int n_chunks, uint32_t site) {
  if (mbar_wait(&bars[c], 0, site)) return true;
  const uint64_t t0 = globaltimer_ns(), budget = *(volatile uint64_t*)&g_wait_budget_ns;
  for (int i = 0; i < n_chunks; ++i)
    while (!mbar_try_wait_suspend(&bars[i], 0, 20000u))
      if (globaltimer_ns() - t0 > budget) return false;
  return false;
}

// ------------------------------------------------------------------ order --
// Larger logits first, the lower index first among equals: one whole number for a
// logit and its index, larger for what comes earlier.  -0 counts as 0; NaN comes
// before everything.
__device__ __forceinline__ uint32_t order_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  if (z != z) return 0xffffffffu;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t place_key(float z, int v) {
  return (uint64_t)order_of(z) << 32 | (0xffffffffu - (uint32_t)v);
}
__device__ __forceinline__ int key_index(uint64_t key) {
  return (int)(0xffffffffu - (uint32_t)key);
}

// Sorts n keys (a power of two) in shared memory, the largest first: a bitonic network.
// Ends with a __syncthreads().
template <int kThreads>
__device__ __forceinline__ void sort_keys(uint64_t* a, int n) {
  for (int size = 2; size <= n; size *= 2) {
    for (int step = size / 2; step > 0; step /= 2) {
      for (int t = threadIdx.x; t < n / 2; t += kThreads) {
        const int i = 2 * t - (t & (step - 1)), j = i + step;
        const uint64_t x = a[i], y = a[j];
        const bool down = (i & size) == 0;
        if ((x < y) == down) {
          a[i] = y;
          a[j] = x;
        }
      }
      __syncthreads();
    }
  }
}
// How many of a descending run's n keys are above `key`; n is below 2^steps.
template <int steps>
__device__ __forceinline__ int above(const uint64_t* run, int n, uint64_t key) {
  int at = 0;
#pragma unroll
  for (int s = 1 << (steps - 1); s > 0; s /= 2)
    if (at + s <= n && run[at + s - 1] > key) at += s;
  return at;
}

// Sorts n <= E kThreads different keys in shared memory, the largest first, as far as the
// first K: each warp sorts 32 E by shuffles alone, and a key's place is the sum of its
// places among the warps' runs.  Ends with a __syncthreads().
template <int kThreads, int E>
__device__ __forceinline__ void sort_runs(uint64_t* a, int n, int K) {
  constexpr int kRun = 32 * E;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = warp * kRun;
  uint64_t key[E];
#pragma unroll
  for (int e = 0; e < E; ++e) key[e] = first + e * 32 + lane < n ? a[first + e * 32 + lane] : 0;
  if (first < n) {
    // Key e of a lane is number lane + 32 e of the run.
#pragma unroll
    for (int size = 2; size <= kRun; size *= 2) {
#pragma unroll
      for (int step = size / 2; step > 0; step /= 2) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const bool down = ((lane + 32 * e) & size) == 0;
          if (step >= 32) {
            const int f = e | (step / 32);
            if (f != e && (key[e] < key[f]) == down) {
              const uint64_t x = key[e];
              key[e] = key[f];
              key[f] = x;
            }
          } else {
            const uint64_t other = __shfl_xor_sync(0xffffffffu, key[e], step);
            const bool larger = ((lane & step) == 0) == down;
            key[e] = (key[e] < other) == larger ? other : key[e];
          }
        }
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (first + e * 32 + lane < n) a[first + e * 32 + lane] = key[e];
  }
  __syncthreads();
  int place[E];
#pragma unroll
  for (int e = 0; e < E; ++e) place[e] = lane + 32 * e;
  for (int r = 0; r * kRun < n && first < n; ++r) {
    if (r == warp) continue;
#pragma unroll
    for (int e = 0; e < E; ++e)
      place[e] += above<E == 2 ? 7 : 8>(a + r * kRun, min(kRun, n - r * kRun), key[e]);
  }
  static_assert(E == 2 || E == 4, "runs of 64 or 128");
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (first + e * 32 + lane < n && place[e] < K) a[place[e]] = key[e];
  __syncthreads();
}
__device__ __forceinline__ int next_power(int n) { return n <= 1 ? 1 : 1 << (32 - __clz(n - 1)); }
// Sorts n <= kMost different keys as far as the first K; where kMost is above 4 kThreads there
// is room for the next power of two.
template <int kThreads, int kMost>
__device__ __forceinline__ void sort_top(uint64_t* a, int n, int K) {
  if (n <= 2 * kThreads) return sort_runs<kThreads, 2>(a, n, K);
  if (kMost <= 4 * kThreads || n <= 4 * kThreads) return sort_runs<kThreads, 4>(a, n, K);
  if constexpr (kMost > 4 * kThreads) {
    const int size = next_power(n);
    for (int i = n + (int)threadIdx.x; i < size; i += kThreads) a[i] = 0;
    __syncthreads();
    sort_keys<kThreads>(a, size);
  }
}

// ------------------------------------------------- neighbours in a cluster --
// Arrives without ordering any memory access: it does not wait for stores on their way.
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  cluster_arrive_release();
  cluster_wait_acquire();
}
template <class U>
__device__ __forceinline__ U ld_cluster(const U* p, int rank) {
  const uint32_t a = mapa_shared(smem_u32(p), (uint32_t)rank);
  U v;
  if constexpr (sizeof(U) == 8) {
    uint64_t w;
    asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(w) : "r"(a) : "memory");
    v = *reinterpret_cast<U*>(&w);
  } else {
    static_assert(sizeof(U) == 4, "words of 4 or 8 bytes");
    uint32_t w;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(w) : "r"(a) : "memory");
    v = *reinterpret_cast<U*>(&w);
  }
  return v;
}
__device__ __forceinline__ void st_cluster(const uint64_t* p, int rank, uint64_t v) {
  const uint32_t a = mapa_shared(smem_u32(p), (uint32_t)rank);
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
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
// max(a, b, c) that passes NaN on.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Devices (the first 64) on which a kernel's limits have been raised, one for each kernel.
using Raised = std::atomic<uint64_t>;

// Launches `kern` with C CTAs of a row to a cluster; raises its limits first, to all that a
// device has, once on each.
template <class P>
inline cudaError_t launch_rows(void (*kern)(const P), const P& p, int64_t rows, int C, int threads,
                               int smem, Raised& raised, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (!(raised.load(std::memory_order_relaxed) & bit)) {
    cudaFuncAttributes fa;
    int most = 0;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               most - (int)fa.sharedSizeBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    raised.fetch_or(bit, std::memory_order_relaxed);
  }
  if (rows * C > 0x7fffffffll) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C), 1, 1);
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
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace stt
