// sample.cu -- logits to the distribution that temperature, top-k, top-p and min-p leave,
// and a token drawn from it with a given random number.
//
// The order of a row's tokens is: larger logits first, the lower index first among
// equals.  What is kept is a beginning of that order:
//   top-k  the first k;
//   top-p  of those, the shortest beginning whose weight is at least p times theirs,
//          one token at least;
//   min-p  of those, the tokens of at least min_p times the largest weight,
// with weights w = e^((z - max z) / T).  The result is w / (sum of the kept), and the
// token is the smallest index at which the running sum of the kept exceeds u times their
// sum.
//
// A cluster of C CTAs takes a row, each its slice in shared memory: HBM sees one read of
// the logits and one write of the probabilities.  The cut is found in two steps.  A
// histogram of the slice over 2048 bins of 1/32 octave of weight gives, summed over the
// cluster, the bin where the cut lies; the bin's tokens, a few hundred in practice, are
// then gathered in the row's first CTA and sorted there.  (A bin that holds more, as
// equal logits make it, is halved by key and counted over the slices instead.)
//
// Neighbours at the border of the kept weight differ by little, and so do a draw's, so
// sums are exact and weights are good to about 2^-31: a weight is 2^(-bin / 32) (1 + E),
// z log2(e) / T being a product of two floats in full; E, below 2^-6, comes from a
// polynomial of degree 4 and is summed as a whole number of 2^-32.  A histogram's bin
// holds the count and the sum of E in 64 bits, split over two words of shared memory; its
// weight is a whole number of 2^-42 of the first token's.  A draw's sums take 128 bits, in
// which the least weight keeps its 31.  A weight more than 2048 bins, about 2^-64, below the
// largest is taken as 0.
//
// 320 fp32 rows of 151936 by top-p, with probabilities: 291 us, against 58 at HBM's rate; 64
// bf16 rows of 128256 with all cuts, tokens alone: 41 (2.5); 99 bf16 rows of 50257: 40 (4.5);
// one fp32 row of 32000: 16 by top-p, 8.4 with nothing cut (19 of a call through the binding).
// HBM is at 11 % of its rate: bound by instructions (113 of a warp for 32 logits, half of the
// issue slots) and by the row's CTAs waiting at barriers (a quarter of the stalls); few rows by
// the chain of a row's steps.  Off the usual path: 64 bf16 rows of 128256 at T = 30 by top-p,
// whose cut is found by halving, 612; of equal logits 744; 320 fp32 rows of 151936 at T = 30 3890.
// Left out after measuring: a row to one CTA that reads its logits again from L2 (266 to 290 us
// for the first, but 50, 60 and 23 on the others); threads' own lists of the kept (295).
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "../../include/stt.h"
#include "row_slice.cuh"

namespace stt {
namespace {

constexpr int kThreads = 512;  // (320 rows of 151936: 256 threads 335 us, 384 301, 512 294, 640 301)
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunks = 8;
constexpr int kOctaves = 64;
constexpr uint32_t kBins = 32 * kOctaves;
constexpr int kList = 2048;                // tokens of a bin that are sorted
// Preferred bytes of a slice: with the bins, the list, the groups' sums, 4 KB of static and reserved
// shared memory, and a piece more where the row starts off a piece, two CTAs fit on an SM's 228 KB.
// (Of 80 KB, where one fits: 320 fp32 rows of 100000 by top-p 307 us, of 77 KB 220; 320 bf16 rows of
// 40960 106 and 88.)
constexpr int kSliceBytes = 77 * 1024;
constexpr int kSegment = 8 * (int)kBins / 2 / kWarps;  // kept tokens that a warp lists, in the bins' memory
constexpr int64_t kBias = 1ll << 26;       // keeps 2^32 E positive
constexpr int kGroup = 4;                  // runs of 32 pieces whose kept weight a warp notes as one
constexpr float kMagic = 393216.f;         // 1.5 2^18: floats there are 1/32 apart

struct Params {
  SampleArgs a;
  int C, per, chunk;
  bool no_copies;      // test hook: the first CTA of a row fetches nothing
  int runs, groups;    // runs of 32 pieces that a warp takes, and groups of those
  uint64_t table[32];  // 2^(63 - j / 32)
};

// A row's grid: bins and weights of its logits.
struct Grid {
  float m0, c, c_lo;  // subtracted first; log2(e) / T in two parts
  int top;            // bits of the maximum's place on the grid
  // z's product with c, its place on the grid, and its bin.
  struct At {
    float zz, p, ks;
    uint32_t bin;
  };
  __device__ __forceinline__ At at(float z) const {
    At a;
    // (Each rounded by itself, never as one product-and-sum: all uses of a logit, and `top`,
    // have to put it at the same place.)
    a.zz = __fsub_rn(z, m0);
    a.p = __fmul_rn(a.zz, c);
    a.ks = __fadd_rn(a.p, kMagic);
    // (Products too far below for the grid, down to -inf, give smaller floats, or ones with a
    // sign: both are far from `top` as whole numbers, too.)
    a.bin = (uint32_t)(top - __float_as_int(a.ks));
    return a;
  }
  // 2^32 E of an element whose bin is below kBins.
  __device__ __forceinline__ int e32(const At& a) const {
    const float r = __fsub_rn(a.p, __fsub_rn(a.ks, kMagic)) + fmaf(a.zz, c_lo, fmaf(a.zz, c, -a.p));
    // 2^r - 1, times 2^32: (r ln 2)^n / n!, |r| <= 2^-6 and the product's low part.
    constexpr double s = 4294967296.0, l = 0.693147180559945309;
    constexpr float a1 = (float)(s * l), a2 = (float)(s * l * l / 2), a3 = (float)(s * l * l * l / 6),
                    a4 = (float)(s * l * l * l * l / 24);
    return __float2int_rn(r * fmaf(r, fmaf(r, fmaf(r, a4, a3), a2), a1));
  }
};

// A cut of the order: kept are logits above z, and at z the indices up to v.
struct Cut {
  float z;
  int v;
  __device__ __forceinline__ bool keeps(float x, int i) const { return x > z || (x == z && i <= v); }
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan64(uint64_t v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}
// A draw's weights are whole numbers of 2^-94 (of a token at its place on the grid that is as
// probable as the first): all of a weight's 31 bits down to the last octave, and room for the
// sum of 2^20.
using Whole = unsigned __int128;
__device__ __forceinline__ Whole warp_sum(Whole v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v += (Whole)__shfl_xor_sync(0xffffffffu, (uint64_t)(v >> 64), o) << 64 |
         __shfl_xor_sync(0xffffffffu, (uint64_t)v, o);
  return v;
}
template <int n = 32>
__device__ __forceinline__ Whole warp_scan(Whole v) {  // inclusive, of the first n lanes
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < n; o <<= 1) {
    const Whole t = (Whole)__shfl_up_sync(0xffffffffu, (uint64_t)(v >> 64), o) << 64 |
                    __shfl_up_sync(0xffffffffu, (uint64_t)v, o);
    if (lane >= o) v += t;
  }
  return v;
}
__device__ __forceinline__ Whole from_lane(Whole v, int lane) {
  return (Whole)__shfl_sync(0xffffffffu, (uint64_t)(v >> 64), lane) << 64 |
         __shfl_sync(0xffffffffu, (uint64_t)v, lane);
}
struct Weight {
  uint32_t w;  // in 2^-31 of the octave
  uint32_t o;  // below 64
  __device__ __forceinline__ Whole whole() const {
    return (Whole)((uint64_t)(w >> 1) >> o) << 64 | (uint64_t)w << (63 - o);
  }
};
// floor(u total) for 0 <= u < 1 and a total below 2^115: exceeded where u total is.
__device__ __forceinline__ Whole share_of(Whole total, float u) {
  const uint32_t bits = __float_as_uint(u), e = max(bits >> 23, 1u);
  const uint32_t mant = (bits & 0x7fffffu) | (bits >> 23 ? 0x800000u : 0u);  // u = mant 2^(e - 150)
  const Whole t = (total >> 24) * mant + ((uint64_t)((uint32_t)total & 0xffffffu) * mant >> 24);
  return t >> (126 - e);
}
// Ends with a __syncthreads().
__device__ __forceinline__ uint64_t block_sum64(uint64_t v, uint64_t* s) {
  v = warp_sum64(v);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  uint64_t all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) all += s[w];
  __syncthreads();
  return all;
}

// The weight of `count` tokens of a bin, `sum` being that of their 2^32 E + 2^26, in units
// of 2^-42; `table` is that of 2^(63 - j / 32).  (Rounded once for a bin of a slice, so that the
// scans over the bins stay in 64 bits: half a unit each, of either sign.  A sum of fp64 weights,
// one token after another, rounds 2^-53 a token, which over a row of 2^17 is no less.)
__device__ __forceinline__ uint64_t weight_of(uint32_t bin, int64_t count, int64_t sum,
                                              const uint64_t* table) {
  const uint64_t n = (uint64_t)((count << 32) + (sum - count * kBias));  // below 2^53
  const uint64_t w = __umul64hi(n << 11, table[bin & 31]);               // in 2^-42 of the octave
  const uint32_t o = bin >> 5;
  return o == 0 ? w : ((w >> (o - 1)) + 1) >> 1;
}

static_assert(2 * (kSliceBytes + 16 + 8 * (int)kBins + 8 * kList +
                   kWarps * (kSliceBytes / 16 / 32 / kWarps / kGroup + 1) * (int)sizeof(Whole) + 4096) <= 228 * 1024,
              "two CTAs on an SM");

template <class T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t bars[kMaxChunks];
  __shared__ uint64_t s_red[kWarps];
  __shared__ float s_max[kWarps];
  __shared__ float s_top;
  __shared__ int s_index;
  __shared__ uint64_t s_mass[kOctaves];  // the slice's, read by the cluster
  __shared__ int s_count[kOctaves];
  __shared__ uint64_t s_run[kOctaves];   // the row's, with all octaves before
  __shared__ int s_run_n[kOctaves];
  __shared__ uint64_t s_tab[32];
  __shared__ float s_c[2];
  __shared__ double s_log;               // T log(min_p)
  __shared__ uint64_t s_target;
  __shared__ int s_n;
  __shared__ __align__(16) uint64_t s_total[2];
  __shared__ Whole s_part[kWarps];
  __shared__ uint64_t s_sum[2][2];  // of the halving steps: counts and sums, in turn
  struct Found {
    uint32_t bin;
    int before, in_bin, offset;  // tokens before it, in it, and of those in slices before
    uint64_t mass;               // weight before it
  };
  __shared__ Found s_found;
  struct Chosen {
    uint64_t key, count, sum;
  };
  __shared__ Chosen s_cut;
  constexpr int G = RowSlice<T>::G;
  const SampleArgs& A = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = P.C;
  const int rank = (int)(blockIdx.x % (unsigned)C);
  const int64_t row = blockIdx.x / (unsigned)C;
  const int64_t b = row / A.rows;
  const RowSlice<T> S(static_cast<const T*>(A.z) + row * A.ld_z, A.V, rank, P.per);
  T* const zs = reinterpret_cast<T*>(smem);
  uint32_t* const bin_lo = reinterpret_cast<uint32_t*>(smem + (size_t)P.per * 16);  // sums of 2^32 E
  uint32_t* const bin_n = bin_lo + kBins;  // counts, and in the upper half the sums' carries
  uint64_t* const list = reinterpret_cast<uint64_t*>(bin_n + kBins);
  Whole* const group_sum = reinterpret_cast<Whole*>(list + kList) + warp * P.groups;  // this warp's
  uint16_t* const kept = reinterpret_cast<uint16_t*>(bin_lo) + warp * kSegment;  // this warp's, places in the slice

  const float temp = A.temperature ? A.temperature[b] : 1.f;
  const int top_k = A.top_k ? A.top_k[b] : 0;
  const float top_p = A.top_p ? A.top_p[b] : 1.f;
  const float min_p = A.min_p ? A.min_p[b] : 0.f;
  const bool greedy = temp == 0.f || top_k == 1;
  const bool want_k = !greedy && top_k > 0 && top_k < A.V;
  const bool want_p = !greedy && top_p < 1.f;
  // (In 64-bit floats, of which an SM does two at a time, by one thread.)
  if (tid == 64) {
    const double c = 1.4426950408889634074 / (double)(greedy ? 1.f : temp);
    const float hi = (float)fmin(c, (double)FLT_MAX);
    s_c[0] = hi;
    s_c[1] = c < (double)FLT_MAX ? (float)(c - (double)hi) : 0.f;
    if (min_p > 0.f) s_log = (double)temp * log((double)fminf(min_p, 1.f));
  }
  if (tid < 32) s_tab[tid] = P.table[tid];
  if (want_k || want_p)
    for (int i = tid; i < 2 * (int)kBins; i += kThreads) bin_lo[i] = 0;
  if (tid == 0) s_index = INT_MAX;
  fetch_slice(S, zs, bars, P.chunk, P.no_copies && rank == 0);

  auto each_piece = [&](auto&& f) {
    for (int q = tid; q < S.pieces; q += kThreads) {
      float x[G];
      unpack_piece(*reinterpret_cast<const uint4*>(zs + q * G), x);
      f(x, S.index(q));
    }
  };

  // ---- the row's largest logit
  float m = -INFINITY;
  const int n_chunks = (S.pieces + P.chunk - 1) / P.chunk;
  {
    for (int c = 0; c < n_chunks; ++c) {
      if (!wait_slice(bars, c, n_chunks, STT_DEVERR_SAMPLE_WAIT)) break;
      const int end = min(S.pieces, (c + 1) * P.chunk);
      for (int q = c * P.chunk + tid; q < end; q += kThreads) {
        float x[G];
        unpack_piece(*reinterpret_cast<const uint4*>(zs + q * G), x);
#pragma unroll
        for (int e = 0; e < G; e += 2) m = max3_nan(m, x[e], x[e + 1]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    m = s_max[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = max_nan(m, s_max[w]);
    if (tid == 0) s_top = m;
    cluster_sync();
    m = lane < C ? ld_cluster(&s_top, lane) : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  float* const probs = A.probs ? A.probs + row * A.ld_p : nullptr;
  const bool vec = ((reinterpret_cast<uintptr_t>(probs) + 4 * (intptr_t)S.first) & 15) == 0;
  // Writes a piece's probabilities.
  auto put = [&](int v, const float (&y)[G]) {
    if (vec && v >= 0 && v + G <= A.V) {
#pragma unroll
      for (int e = 0; e < G; e += 4)
        st_global_cs_f4(probs + v + e, make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]));
    } else {
#pragma unroll
      for (int e = 0; e < G; ++e)
        if (v + e >= 0 && v + e < A.V) probs[v + e] = y[e];
    }
  };
  if (!(fabsf(m) < INFINITY)) {
    // Nothing allowed: no token, no probability.  NaN or +inf: no distribution.
    const float none = m == -INFINITY ? 0.f : NAN;
    if (probs) {
      float y[G];
#pragma unroll
      for (int e = 0; e < G; ++e) y[e] = none;
      for (int q = tid; q < S.pieces; q += kThreads) put(S.index(q), y);
    }
    if (rank == 0 && tid == 0) {
      if (A.tokens) A.tokens[row] = -1;
      if (A.logprobs) A.logprobs[row] = m == -INFINITY ? -INFINITY : NAN;
    }
    cluster_sync();  // nobody leaves while its maximum is read
    return;
  }

  const bool truncated = greedy || want_k || want_p || min_p > 0.f;

  // ---- the grid
  Grid grid;
  {
    grid.top = 0;
    grid.c = s_c[0];
    grid.c_lo = s_c[1];
    // Where the products would leave the grid's range the maximum is taken off first: the
    // logits that matter are then within a 2^10th of it and the difference is exact.
    grid.m0 = fabsf(m) * grid.c < 65536.f ? 0.f : m;
    grid.top = __float_as_int(grid.at(m).ks);
  }

  Cut cut{-INFINITY, INT_MAX};  // (the weight of -inf is 0)
  auto cut_at = [&](float z, int v) {  // the stricter of the two
    if (z > cut.z || (z == cut.z && v < cut.v)) cut = Cut{z, v};
  };
  if (greedy) {
    int first = INT_MAX;
    each_piece([&](const float (&x)[G], int v) {
#pragma unroll
      for (int e = G - 1; e >= 0; --e)
        if (x[e] == m) first = min(first, v + e);
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) atomicMin(&s_index, first);
    cluster_sync();
    first = lane < C ? ld_cluster(&s_index, lane) : INT_MAX;
    cut = Cut{m, __reduce_min_sync(0xffffffffu, first)};
  } else if (want_k || want_p) {
    // ---- the histogram of the slice
    each_piece([&](const float (&x)[G], int) {
#pragma unroll
      for (int e = 0; e < G; ++e) {
        const auto a = grid.at(x[e]);
        const uint32_t v = (uint32_t)(grid.e32(a) + (int)kBias);
        if (a.bin < kBins) {
          const uint32_t old = atomicAdd(&bin_lo[a.bin], v);
          atomicAdd(&bin_n[a.bin], 1u + (old + v < old ? 1u << 16 : 0u));
        }
      }
    });
    __syncthreads();
    auto bin_count = [&](uint32_t n) { return (int)(n & 0xffffu); };
    auto bin_sum = [&](uint32_t lo, uint32_t n) { return (int64_t)((uint64_t)(n >> 16) << 32 | lo); };
    // Octaves: a warp's lanes take an octave's bins.
    for (int o = warp; o < kOctaves; o += kWarps) {
      const uint32_t lo = bin_lo[o * 32 + lane], n = bin_n[o * 32 + lane];
      const uint64_t w = warp_sum64(weight_of(o * 32 + lane, bin_count(n), bin_sum(lo, n), s_tab));
      const int k = __reduce_add_sync(0xffffffffu, bin_count(n));
      if (lane == 0) {
        s_mass[o] = w;
        s_count[o] = k;
      }
    }
    cluster_sync();
    if (tid < kOctaves) {
      uint64_t w = 0;
      int k = 0;
      for (int r = 0; r < C; ++r) {
        w += ld_cluster(&s_mass[tid], r);
        k += ld_cluster(&s_count[tid], r);
      }
      s_run[tid] = w;
      s_run_n[tid] = k;
    }
    __syncthreads();
    if (warp == 0) {
      uint64_t w[2] = {s_run[2 * lane], s_run[2 * lane + 1]};
      uint32_t n[2] = {(uint32_t)s_run_n[2 * lane], (uint32_t)s_run_n[2 * lane + 1]};
      const uint64_t run = warp_scan64(w[0] + w[1]), run_n = warp_scan64((uint64_t)(n[0] + n[1]));
      s_run[2 * lane] = run - w[1];
      s_run[2 * lane + 1] = run;
      s_run_n[2 * lane] = (int)run_n - (int)n[1];
      s_run_n[2 * lane + 1] = (int)run_n;
    }
    __syncthreads();
    uint64_t whole = s_run[kOctaves - 1];  // the row's weight
    const int many = s_run_n[kOctaves - 1];

    // Finds the bin where the running count reaches `k`, or (k < 0) the running weight
    // reaches `target`: into s_found, by warp 0.  One does.
    auto find_bin = [&](int k, uint64_t target) {
      if (warp == 0) {
        int o = 0;
        for (int half = 0; half < 2; ++half) {
          const int i = half * 32 + lane;
          const bool reached = k >= 0 ? s_run_n[i] >= k : s_run[i] >= target;
          o += __popc(~__ballot_sync(0xffffffffu, reached));
        }
        o = min(o, kOctaves - 1);
        const uint64_t before = o ? s_run[o - 1] : 0;
        const int before_n = o ? s_run_n[o - 1] : 0;
        // The octave's bins over the cluster, a lane to each.
        int n = 0, offset = 0;
        int64_t sum = 0;
        for (int r = 0; r < C; ++r) {
          const uint32_t lo = ld_cluster(&bin_lo[o * 32 + lane], r), c = ld_cluster(&bin_n[o * 32 + lane], r);
          if (r < rank) offset += bin_count(c);
          n += bin_count(c);
          sum += bin_sum(lo, c);
        }
        const uint64_t w = weight_of(o * 32 + lane, n, sum, s_tab);
        const uint64_t run = before + warp_scan64(w);
        const int run_n = before_n + (int)warp_scan64((uint64_t)n);
        const uint32_t reached =
            __ballot_sync(0xffffffffu, n > 0 && (k >= 0 ? run_n >= k : run >= target));
        const uint32_t any = __ballot_sync(0xffffffffu, n > 0);
        // (The octave's own weight is a sum of rounded ones: its last bin with tokens.)
        const int hit = reached ? __ffs((int)reached) - 1 : any ? 31 - __clz((int)any) : 0;
        if (lane == hit) s_found = Found{(uint32_t)(o * 32 + lane), run_n - n, n, offset, run - w};
      }
      __syncthreads();
    };
    // Halves the found bin by key: kept are the tokens down to the one at which the
    // running count in the bin reaches `need`, or (need < 0) the row's weight `target`.
    // Returns their count and sum of 2^32 E + 2^26, and cuts there.
    int turn = 0;
    auto halve = [&](const Found& f, int need, uint64_t target, int64_t& count, int64_t& sum) {
      auto reaches = [&](uint64_t key, int64_t& n, int64_t& s) {
        uint64_t my_n = 0, my_s = 0;
        each_piece([&](const float (&x)[G], int v) {
#pragma unroll
          for (int e = 0; e < G; ++e) {
            const auto a = grid.at(x[e]);
            if (a.bin == f.bin && place_key(x[e], v + e) >= key) {
              ++my_n;
              my_s += (uint64_t)(grid.e32(a) + (int)kBias);
            }
          }
        });
        my_n = block_sum64(my_n, s_red);
        my_s = block_sum64(my_s, s_red);
        if (tid == 0) {
          s_sum[turn][0] = my_n;
          s_sum[turn][1] = my_s;
        }
        cluster_sync();
        // (Read by all before the next step but one writes them again.)
        uint64_t on = lane < C ? ld_cluster(&s_sum[turn][0], lane) : 0;
        uint64_t os = lane < C ? ld_cluster(&s_sum[turn][1], lane) : 0;
        turn ^= 1;
        n = (int64_t)warp_sum64(on);
        s = (int64_t)warp_sum64(os);
        // (The whole bin always does: see the rounding in find_bin.)
        return need >= 0 ? n >= need
                         : n == f.in_bin || (n > 0 && f.mass + weight_of(f.bin, n, s, s_tab) >= target);
      };
      // The logit first, then the index.
      uint64_t lo = 0, hi = (uint64_t)order_of(m) + 1;  // `lo` reaches, `hi` does not
      int64_t n, s;
      while (hi - lo > 1) {
        const uint64_t mid = lo + (hi - lo) / 2;
        if (reaches(mid << 32, n, s)) lo = mid;
        else hi = mid;
      }
      const uint64_t z = lo << 32;
      lo = 0xffffffffu - (uint32_t)(A.V - 1);  // the last index's
      hi = 0x100000000ull;
      while (hi - lo > 1) {
        const uint64_t mid = lo + (hi - lo) / 2;
        if (reaches(z | mid, n, s)) lo = mid;
        else hi = mid;
      }
      reaches(z | lo, count, sum);
      cut_at(logit_of((uint32_t)(z >> 32)), key_index(z | lo));
    };
    // Gathers the found bin's tokens in the row's first CTA, which sorts them and cuts as
    // halve() does.
    auto select = [&](const Found& f, int need, uint64_t target, int64_t& count, int64_t& sum) {
      const int n = f.in_bin;
      if (tid == 0) s_n = 0;
      cluster_sync();  // and the first CTA is done with its list
      each_piece([&](const float (&x)[G], int v) {
#pragma unroll
        for (int e = 0; e < G; ++e) {
          if (grid.at(x[e]).bin == f.bin) {
            const int at = f.offset + atomicAdd(&s_n, 1);
            if (at < kList) st_cluster(&list[at], 0, place_key(x[e], v + e));
          }
        }
      });
      cluster_sync();
      if (rank == 0) {
        sort_top<kThreads, kList>(list, n, n);
        // Running sums over the sorted tokens, a run of them to a thread.
        const int each = (n + kThreads - 1) / kThreads, i0 = min(n, tid * each), i1 = min(n, i0 + each);
        uint64_t mine = 0;
        auto e_of = [&](uint64_t key) {
          return (uint64_t)(grid.e32(grid.at(logit_of((uint32_t)(key >> 32)))) + (int)kBias);
        };
        for (int i = i0; i < i1; ++i) mine += e_of(list[i]);
        const uint64_t incl = warp_scan64(mine);
        if (lane == 31) s_red[warp] = incl;
        if (tid == 0) s_cut = Chosen{};
        __syncthreads();
        uint64_t run = incl - mine;
        for (int w = 0; w < warp; ++w) run += s_red[w];
        // The last token that is kept, whose next one is not.
        for (int i = i0; i < i1; ++i) {
          const uint64_t next = run + e_of(list[i]);
          const bool keep = need >= 0 ? i < need
                                      : i == 0 || f.mass + weight_of(f.bin, i, (int64_t)run, s_tab) < target;
          const bool more = need >= 0 ? i + 1 < need
                                      : f.mass + weight_of(f.bin, i + 1, (int64_t)next, s_tab) < target;
          if (keep && (i + 1 == n || !more)) s_cut = Chosen{list[i], (uint64_t)(i + 1), next};
          run = next;
        }
      }
      cluster_sync();
      const uint64_t last = ld_cluster(&s_cut.key, 0);
      count = (int64_t)ld_cluster(&s_cut.count, 0);
      sum = (int64_t)ld_cluster(&s_cut.sum, 0);
      cut_at(logit_of((uint32_t)(last >> 32)), key_index(last));
    };
    auto cut_bin = [&](int need, uint64_t target) {
      const Found f = s_found;
      int64_t count, sum;
      if (f.in_bin <= kList) select(f, need < 0 ? -1 : need - f.before, target, count, sum);
      else halve(f, need < 0 ? -1 : need - f.before, target, count, sum);
      return f.mass + weight_of(f.bin, count, sum, s_tab);
    };
    if (want_k && many > top_k) {
      find_bin(top_k, 0);
      whole = cut_bin(top_k, 0);
    }
    if (want_p) {
      // A beginning is short of p times the whole if, as a whole number, it is below this.
      if (tid == 0) s_target = (uint64_t)ceil(fmax(0.0, (double)top_p) * (double)whole);
      __syncthreads();
      const uint64_t target = s_target;
      find_bin(-1, target);
      cut_bin(-1, target);
    }
  }
  if (!greedy && min_p > 0.f) {
    // w >= min_p: z >= max + T log(min_p), as the smallest float that satisfies it.
    cut_at(__double2float_ru((double)m + s_log), INT_MAX);
  }

  // ---- the kept weights in whole numbers
  auto weight = [&](float x) -> Weight {
    const auto a = grid.at(x);
    const uint32_t t = (uint32_t)(s_tab[a.bin & 31] >> 32);
    const uint32_t w = t + (uint32_t)((int64_t)((uint64_t)t) * grid.e32(a) >> 32);
    return a.bin < kBins ? Weight{w, a.bin >> 5} : Weight{0, 0};
  };
  // A warp takes its slice's pieces in order, as runs of 32, and lists what is kept of
  // them; where that is too much for its list, `dense`, it adds up run by run.
  const int q_begin = min(S.pieces, warp * P.runs * 32), q_end = min(S.pieces, q_begin + P.runs * 32);
  int n_kept = 0;
  bool dense = !truncated;
  // (The bins' memory: no neighbour reads bins after the barriers of the cut.)
  for (int q0 = q_begin; q0 < q_end && !dense; q0 += 32) {
    const int q = q0 + lane, v = S.index(q);
    float x[G];
    uint32_t keep = 0;
    if (q < q_end) {
      unpack_piece(*reinterpret_cast<const uint4*>(zs + q * G), x);
#pragma unroll
      for (int e = 0; e < G; ++e) keep |= x[e] >= cut.z ? 1u << e : 0u;
      if (keep) {
#pragma unroll
        for (int e = 0; e < G; ++e)
          if (x[e] == -INFINITY || !cut.keeps(x[e], v + e)) keep &= ~(1u << e);
      }
    }
    if (__any_sync(0xffffffffu, keep != 0)) {
      const int n = __popc(keep);
      int at = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += t;
      }
      const int all = __shfl_sync(0xffffffffu, at, 31);
      if (n_kept + all > kSegment) {
        dense = true;
      } else {
        at += n_kept - n;
        for (uint32_t k = keep; k; k &= k - 1) kept[at++] = (uint16_t)(q * G + __ffs((int)k) - 1);
        n_kept += all;
      }
    }
  }
  __syncwarp();
  // What is kept of the piece that this lane has of a run.
  auto kept_of = [&](int q) -> Whole {
    Whole w = 0;
    if (q < q_end) {
      float x[G];
      unpack_piece(*reinterpret_cast<const uint4*>(zs + q * G), x);
#pragma unroll
      for (int e = 0; e < G; ++e) {
        const Whole t = weight(x[e]).whole();  // (0 for -inf)
        if (cut.keeps(x[e], S.index(q) + e)) w += t;
      }
    }
    return w;
  };
  Whole mine = 0;
  if (!dense) {
    for (int i = lane; i < n_kept; i += 32) mine += weight((float)zs[kept[i]]).whole();
    mine = warp_sum(mine);
  } else {
    for (int g = 0; g < P.groups; ++g) {
      Whole w = 0;
      const int q0 = q_begin + g * kGroup * 32;
      for (int q = q0; q < min(q0 + kGroup * 32, q_end); q += 32) w += kept_of(q + lane);
      w = warp_sum(w);
      if (lane == 0) group_sum[g] = w;
      mine += w;
    }
  }
  if (lane == 0) s_part[warp] = mine;
  __syncthreads();
  Whole slice_before;  // what the slice's warps before this one have
  {
    const Whole part = lane < kWarps ? s_part[lane] : 0, run = warp_scan<kWarps>(part);
    slice_before = from_lane(run - part, warp);
    if (tid == kWarps - 1) {
      s_total[0] = (uint64_t)run;
      s_total[1] = (uint64_t)(run >> 64);
    }
  }
  cluster_sync();
  Whole total, before;
  {
    Whole o = 0;
    if (lane < C) o = (Whole)ld_cluster(&s_total[1], lane) << 64 | ld_cluster(&s_total[0], lane);
    const Whole run = warp_scan<kRowMaxCtas>(o);
    total = from_lane(run, kRowMaxCtas - 1);
    before = from_lane(run - o, rank) + slice_before;
  }
  __syncwarp();
  cluster_arrive_release();  // done with the neighbours' shared memory; waited for at the end
  const float total_f = (float)(uint64_t)(total >> 50);  // in 2^-44

  // ---- the token: its warp finds it
  if (A.u && before < total) {
    const float u = A.u[row];
    Whole at = u >= 1.f ? total - 1 : u > 0.f ? share_of(total, u) : 0;
    // (The logarithm of the weight's own bits, over the total's.)
    auto drawn = [&](int v, const Weight& w) {
      if (A.tokens) A.tokens[row] = v;
      if (A.logprobs) A.logprobs[row] = logf((float)w.w * __uint_as_float((127 + 13 - w.o) << 23) / total_f);
    };
    if (before <= at && at < before + mine) {
      at -= before;
      if (!dense) {
        for (int i0 = 0; i0 < n_kept; i0 += 32) {
          const int place = i0 + lane < n_kept ? kept[i0 + lane] : 0;
          const Weight of = i0 + lane < n_kept ? weight((float)zs[place]) : Weight{0, 0};
          const Whole w = of.whole(), run = warp_scan(w);
          if (run > at && run - w <= at) drawn(S.first + place, of);
          const Whole all = from_lane(run, 31);
          if (all > at) break;
          at -= all;
        }
      } else {
        // The group of runs, then the run, the lane's piece, and the element.
        int g = 0;
        while (g + 1 < P.groups && group_sum[g] <= at) at -= group_sum[g++];
        for (int q0 = q_begin + g * kGroup * 32; q0 < q_end; q0 += 32) {
          const Whole w = kept_of(q0 + lane), run = warp_scan(w), all = from_lane(run, 31);
          if (all <= at) {
            at -= all;
            continue;
          }
          if (run > at && run - w <= at) {
            float x[G];
            unpack_piece(*reinterpret_cast<const uint4*>(zs + (q0 + lane) * G), x);
            const int v = S.index(q0 + lane);
            Whole acc = run - w;
            bool done = false;
#pragma unroll
            for (int e = 0; e < G; ++e) {
              const Weight of = weight(x[e]);
              if (cut.keeps(x[e], v + e)) acc += of.whole();
              if (!done && acc > at) {
                done = true;
                drawn(v + e, of);
              }
            }
          }
          break;
        }
      }
    }
  }

  // ---- the probabilities
  if (probs) {
    // 1 / total, for weights in units of the maximum's bin.
    const float inv = 1.f / (total_f * 0x1p-44f);
    auto probability = [&](float x) {
      const auto a = grid.at(x);
      const float p = ex2((float)a.bin * (-1.f / 32.f)) * fmaf((float)grid.e32(a), 0x1p-32f, 1.f) * inv;
      return a.bin < kBins ? p : 0.f;
    };
    if (truncated) {  // most of the row; what is kept is written over it
      const float zero[G] = {};
      for (int q = tid; q < S.pieces; q += kThreads) put(S.index(q), zero);
      __syncthreads();
    }
    if (!dense) {
      for (int i = lane; i < n_kept; i += 32) {
        const int place = kept[i];
        probs[S.first + place] = probability((float)zs[place]);
      }
    } else {
      for (int q = q_begin + lane; q < q_end; q += 32) {
        const int v = S.index(q);
        float x[G], y[G];
        unpack_piece(*reinterpret_cast<const uint4*>(zs + q * G), x);
#pragma unroll
        for (int e = 0; e < G; ++e) {
          const float p = probability(x[e]);
          y[e] = cut.keeps(x[e], v + e) ? p : 0.f;
        }
        put(v, y);
      }
    }
  }
  __syncwarp();
  cluster_wait_acquire();
}

}  // namespace

cudaError_t sample_launch(const SampleArgs& a, cudaStream_t s) {
  const int size = a.bf16 ? 2 : 4;
  Params P{};
  P.a = a;
  for (int j = 0; j < 32; ++j)  // (exact in a double, but for its last bits)
    P.table[j] = j == 0 ? 1ull << 63 : (uint64_t)std::ldexp(std::exp2(-j / 32.0), 63);
  // CTAs of a row: as few as leave room for two on an SM; more while all rows run at once,
  // but none below 16 KB (99 bf16 rows of 50257 in two CTAs 42.9 us, in three 41.5; one row of
  // 32000 in 15 CTAs 23.0, in seven 18.6, all at the time).
  int C = (int)((a.V * (int64_t)size + kSliceBytes - 1) / kSliceBytes);
  C = std::max(1, std::min(C, kRowMaxCtas));
  while (C < kRowMaxCtas && a.N * (C + 1) <= 2 * sm_count() && slice_pieces(a.V, size, C + 1) >= 2 * kThreads) ++C;
  P.C = C;
  P.per = (int)slice_pieces(a.V, size, C);
  const int round = 512;
  P.chunk = ((P.per + kMaxChunks - 1) / kMaxChunks + round - 1) / round * round;
  P.runs = ((P.per + 31) / 32 + kWarps - 1) / kWarps;
  P.groups = (P.runs + kGroup - 1) / kGroup;
  const int smem = P.per * 16 + kBins * 8 + kList * 8 + kWarps * P.groups * (int)sizeof(Whole);
  P.no_copies = (debug_inject() & STT_INJECT_SLICE_WITHHOLD_COPIES) != 0;
  prof_before(s, STT_KERNEL_SAMPLE);
  static Raised raised[2];
  const cudaError_t e =
      a.bf16 ? launch_rows(sample_kernel<__nv_bfloat16>, P, a.N, C, kThreads, smem, raised[1], s)
             : launch_rows(sample_kernel<float>, P, a.N, C, kThreads, smem, raised[0], s);
  prof_after(s);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

STT_DEFINE_ERROR_ACCESSOR(sample_error_word)
STT_DEFINE_BUDGET_SETTER(sample_set_wait_budget)

}  // namespace stt
