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
// then gathered from the cluster and sorted by every CTA.  (A bin that holds more, as
// equal logits make it, is halved by key and counted over the slices instead.)
//
// Neighbours at the border of the kept weight differ by little, and so do a draw's, so
// sums are exact and weights are good to about 2^-31: a weight is 2^(-bin / 32) (1 + E),
// z log2(e) / T being a product of two floats in full; E, below 2^-6, comes from a
// polynomial of degree 4 and is summed as a whole number of 2^-32.  A histogram's bin
// holds the count and the sum of E in 64 bits, split over two words of shared memory.
// A weight more than 2048 bins, about 2^-64, below the largest is taken as 0.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "../../include/stt.h"
#include "row_slice.cuh"

namespace stt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunks = 8;
constexpr int kOctaves = 64;
constexpr uint32_t kBins = 32 * kOctaves;
constexpr int kList = 2048;                // tokens of a bin that are sorted
constexpr int kSliceBytes = 40 * 1024;     // preferred bytes of a slice
constexpr int64_t kBias = 1ll << 26;       // keeps 2^32 E positive
constexpr int kUnitShift = 42;             // a weight of 1 in whole numbers is 2^42
constexpr float kMagic = 393216.f;         // 1.5 2^18: floats there are 1/32 apart

struct Params {
  SampleArgs a;
  int C, per, chunk;
  int units;         // runs of 32 pieces in a slice, at most
  double octave[32]; // 2^(-j / 32)
};

// A row's grid: bins and weights of its logits.
struct Grid {
  float m0, c, c_lo, low;  // subtracted first; log2(e) / T in two parts; smallest product kept
  int top;                 // bits of the maximum's place on the grid
  // z's product with c, its place on the grid, and its bin.
  struct At {
    float zz, p, ks;
    uint32_t bin;
  };
  __device__ __forceinline__ At at(float z) const {
    At a;
    a.zz = z - m0;
    a.p = a.zz * c;
    a.ks = fmaxf(a.p, low) + kMagic;
    a.bin = (uint32_t)(top - __float_as_int(a.ks));
    return a;
  }
  // 2^32 E of an element whose bin is below kBins.
  __device__ __forceinline__ int e32(const At& a) const {
    const float r = (a.p - (a.ks - kMagic)) + fmaf(a.zz, c_lo, fmaf(a.zz, c, -a.p));
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

// The weight of `count` tokens of a bin with the sum of their 2^32 E + 2^26, in units of
// the bin's own weight.
__device__ __forceinline__ double weight_of(int64_t count, int64_t sum) {
  return (double)count + (double)(sum - count * kBias) * (1.0 / 4294967296.0);
}
__device__ __forceinline__ double octave_scale(int o) {  // 2^-o
  return __longlong_as_double((long long)(1023 - o) << 52);
}

template <class T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t bars[kMaxChunks];
  __shared__ uint64_t s_red[kWarps];
  __shared__ float s_max[kWarps];
  __shared__ float s_top;
  __shared__ int s_index;
  __shared__ double s_mass[kOctaves];    // the slice's, then read by the cluster
  __shared__ int s_count[kOctaves];
  __shared__ double s_all_mass[kOctaves];
  __shared__ int s_all_count[kOctaves];
  __shared__ double s_tab[32];
  __shared__ uint32_t s_tab32[32];
  __shared__ int s_n;
  __shared__ uint64_t s_total;
  __shared__ uint64_t s_sum[2][2];  // of the halving steps: counts and sums, in turn
  struct Found {
    uint32_t bin;
    int before, in_bin, offset;  // tokens before it, in it, and of those in slices before
    double mass;                 // weight before it
  };
  __shared__ Found s_found;
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
  uint64_t* const unit = list + kList;

  const float temp = A.temperature ? A.temperature[b] : 1.f;
  const int top_k = A.top_k ? A.top_k[b] : 0;
  const float top_p = A.top_p ? A.top_p[b] : 1.f;
  const float min_p = A.min_p ? A.min_p[b] : 0.f;
  const bool greedy = temp == 0.f || top_k == 1;
  const bool want_k = !greedy && top_k > 0 && top_k < A.V;
  const bool want_p = !greedy && top_p < 1.f;
  if (tid < 32) {
    s_tab[tid] = P.octave[tid];
    s_tab32[tid] = (uint32_t)(P.octave[tid] * 2147483648.0 + 0.5);
  }
  if (want_k || want_p)
    for (int i = tid; i < 2 * (int)kBins; i += kThreads) bin_lo[i] = 0;
  if (tid == 0) s_index = INT_MAX;
  fetch_slice(S, zs, bars, P.chunk);

  auto each_piece = [&](auto&& f) {
    for (int q = tid; q < S.pieces; q += kThreads) {
      float x[G];
      unpack_piece(*reinterpret_cast<const uint4*>(zs + q * G), x);
      f(x, S.index(q));
    }
  };

  // ---- the row's largest logit
  float m = -INFINITY;
  {
    const int n_chunks = (S.pieces + P.chunk - 1) / P.chunk;
    for (int c = 0; c < n_chunks; ++c) {
      mbar_wait(&bars[c], 0, STT_DEVERR_SAMPLE_WAIT);
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

  // ---- the grid
  Grid grid;
  {
    const double c = 1.4426950408889634074 / (double)(greedy ? 1.f : temp);
    grid.c = (float)fmin(c, (double)FLT_MAX);
    grid.c_lo = c < (double)FLT_MAX ? (float)(c - (double)grid.c) : 0.f;
    // Where the products would leave the grid's range the maximum is taken off first: the
    // logits that matter are then within a 2^10th of it and the difference is exact.
    grid.m0 = fabsf(m) * grid.c < 65536.f ? 0.f : m;
    grid.low = -FLT_MAX;
    const float p = (m - grid.m0) * grid.c;
    grid.top = __float_as_int(p + kMagic);
    grid.low = p - (kOctaves + 1.f);
  }

  Cut cut{-INFINITY, -1};
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
        if (a.bin < kBins) {
          const uint32_t v = (uint32_t)(grid.e32(a) + (int)kBias);
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
      double w = weight_of(bin_count(n), bin_sum(lo, n)) * s_tab[lane];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
      const int k = __reduce_add_sync(0xffffffffu, bin_count(n));
      if (lane == 0) {
        s_mass[o] = w * octave_scale(o);
        s_count[o] = k;
      }
    }
    cluster_sync();
    if (tid < kOctaves) {
      double w = 0.0;
      int k = 0;
      for (int r = 0; r < C; ++r) {
        w += ld_cluster(&s_mass[tid], r);
        k += ld_cluster(&s_count[tid], r);
      }
      s_all_mass[tid] = w;
      s_all_count[tid] = k;
    }
    __syncthreads();
    double whole = 0.0;  // the row's weight, every thread's in the same order
    int many = 0;
    for (int o = 0; o < kOctaves; ++o) {
      whole += s_all_mass[o];
      many += s_all_count[o];
    }

    // Finds the bin where the running count reaches `k`, or (k < 0) the running weight
    // reaches `target`: into s_found, by warp 0.  False: no bin does.
    auto find_bin = [&](int k, double target) {
      double before = 0.0;
      int count = 0, o = 0;
      for (; o < kOctaves; ++o) {
        const double w = before + s_all_mass[o];
        const int n = count + s_all_count[o];
        if (k >= 0 ? n >= k : w >= target) break;
        before = w;
        count = n;
      }
      if (o == kOctaves) return false;
      if (warp == 0) {
        // The octave's bins over the cluster, a lane to each.
        int n = 0, offset = 0;
        int64_t sum = 0;
        for (int r = 0; r < C; ++r) {
          const uint32_t lo = ld_cluster(&bin_lo[o * 32 + lane], r), c = ld_cluster(&bin_n[o * 32 + lane], r);
          if (r < rank) offset += bin_count(c);
          n += bin_count(c);
          sum += bin_sum(lo, c);
        }
        const double w = weight_of(n, sum) * s_tab[lane] * octave_scale(o);
        // (One after another, as the octaves: what a bin holds before it is the same sum
        // for everyone.)
        double run = before, mine = before;
        int at = count, mine_n = count, hit = 32;
        int last = -1;
        for (int j = 0; j < 32; ++j) {
          const double wj = __shfl_sync(0xffffffffu, w, j);
          const int nj = __shfl_sync(0xffffffffu, n, j);
          if (lane == j) {
            mine = run;
            mine_n = at;
          }
          run += wj;
          at += nj;
          if (nj > 0) last = j;
          if (hit == 32 && nj > 0 && (k >= 0 ? at >= k : run >= target)) hit = j;
        }
        // (The octave's weight was summed in another order: its last bin with tokens.)
        if (hit == 32) hit = last < 0 ? 0 : last;
        if (lane == hit) s_found = Found{(uint32_t)(o * 32 + lane), mine_n, n, offset, mine};
      }
      __syncthreads();
      return true;
    };
    // Halves the found bin by key: kept are the tokens down to the one at which the
    // running count in the bin reaches `need`, or (need < 0) the row's weight `target`.
    // Returns their count and sum of 2^32 E + 2^26, and cuts there.
    int turn = 0;
    auto halve = [&](const Found& f, int need, double target, int64_t& count, int64_t& sum) {
      const double scale = s_tab[f.bin & 31] * octave_scale((int)(f.bin >> 5));
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
        return need >= 0 ? n >= need : n > 0 && f.mass + scale * weight_of(n, s) >= target;
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
    // Gathers the found bin's tokens, sorts them and cuts as halve() does.
    auto select = [&](const Found& f, int need, double target, int64_t& count, int64_t& sum) {
      const double scale = s_tab[f.bin & 31] * octave_scale((int)(f.bin >> 5));
      const int n = f.in_bin;
      if (tid == 0) s_n = 0;
      cluster_sync();  // and everyone is done with its list
      each_piece([&](const float (&x)[G], int v) {
#pragma unroll
        for (int e = 0; e < G; ++e) {
          if (grid.at(x[e]).bin == f.bin) {
            const int at = f.offset + atomicAdd(&s_n, 1);
            const uint64_t key = place_key(x[e], v + e);
            if (at < kList)
              for (int r = 0; r < C; ++r) st_cluster(&list[at], r, key);
          }
        }
      });
      const int size = next_power(n);
      for (int i = n + tid; i < size; i += kThreads) list[i] = 0;
      cluster_sync();
      sort_keys<kThreads>(list, size);
      // Running sums over the sorted tokens, a run of them to a thread.
      const int each = (size + kThreads - 1) / kThreads, i0 = min(n, tid * each), i1 = min(n, i0 + each);
      uint64_t mine = 0;
      auto e_of = [&](uint64_t key) {
        return (uint64_t)(grid.e32(grid.at(logit_of((uint32_t)(key >> 32)))) + (int)kBias);
      };
      for (int i = i0; i < i1; ++i) mine += e_of(list[i]);
      const uint64_t incl = warp_scan64(mine);
      if (lane == 31) s_red[warp] = incl;
      __syncthreads();
      uint64_t run = incl - mine;
      for (int w = 0; w < warp; ++w) run += s_red[w];
      __syncthreads();
      int kept = 0;
      uint64_t kept_sum = 0;
      for (int i = i0; i < i1; ++i) {
        const bool keep = need >= 0 ? i < need
                                    : i == 0 || f.mass + scale * weight_of(i, (int64_t)run) < target;
        if (!keep) break;
        const uint64_t v = e_of(list[i]);
        run += v;
        ++kept;
        kept_sum += v;
      }
      count = (int64_t)block_sum64((uint64_t)kept, s_red);
      sum = (int64_t)block_sum64(kept_sum, s_red);
      const uint64_t last = list[count - 1];
      cut_at(logit_of((uint32_t)(last >> 32)), key_index(last));
    };
    auto cut_bin = [&](int need, double target, int64_t& count, int64_t& sum) {
      const Found f = s_found;
      if (f.in_bin <= kList) select(f, need < 0 ? -1 : need - f.before, target, count, sum);
      else halve(f, need < 0 ? -1 : need - f.before, target, count, sum);
      return f.mass + s_tab[f.bin & 31] * octave_scale((int)(f.bin >> 5)) * weight_of(count, sum);
    };
    int64_t count, sum;
    if (want_k && many > top_k && find_bin(top_k, 0.0)) whole = cut_bin(top_k, 0.0, count, sum);
    __syncthreads();
    if (want_p && find_bin(-1, fmin((double)top_p, 1.0) * whole))
      cut_bin(-1, fmin((double)top_p, 1.0) * whole, count, sum);
  }
  if (!greedy && min_p > 0.f) {
    // w >= min_p: z >= max + T log(min_p), as the smallest float that satisfies it.
    const double z = (double)m + (double)temp * log((double)fminf(min_p, 1.f));
    cut_at(__double2float_ru(z), INT_MAX);
  }

  // ---- the kept weights in whole numbers, by runs of 32 pieces in the order of indices
  auto weight = [&](float x) -> uint64_t {
    const auto a = grid.at(x);
    if (a.bin >= kBins) return 0;
    const uint32_t t = s_tab32[a.bin & 31];
    const uint32_t w = t + (uint32_t)((int64_t)((uint64_t)t) * grid.e32(a) >> 32);
    // w / 2^31 2^-octave, in units of 2^-42, rounded.
    const uint64_t u = (uint64_t)w << (kUnitShift - 31 + 1) >> (a.bin >> 5);
    return (u + 1) >> 1;
  };
  uint64_t mine = 0;
  for (int q0 = warp * 32; q0 < S.pieces; q0 += kThreads) {
    const int q = q0 + lane;
    float x[G];
    bool any = false;
    const int v = S.index(q);
    if (q < S.pieces) {
      unpack_piece(*reinterpret_cast<const uint4*>(zs + q * G), x);
#pragma unroll
      for (int e = 0; e < G; ++e) any |= x[e] >= cut.z && x[e] > -INFINITY;
    }
    uint64_t w = 0;
    if (__any_sync(0xffffffffu, any)) {
      if (any) {
#pragma unroll
        for (int e = 0; e < G; ++e)
          if (cut.keeps(x[e], v + e)) w += weight(x[e]);
      }
      w = warp_sum64(w);
    }
    if (lane == 0) unit[q0 / 32] = w;
    mine += w;  // the same in every lane
  }
  if (lane == 0) s_red[warp] = mine;
  __syncthreads();
  mine = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mine += s_red[w];
  if (tid == 0) s_total = mine;
  cluster_sync();
  uint64_t total, before;
  {
    const uint64_t o = lane < C ? ld_cluster(&s_total, lane) : 0;
    const uint64_t run = warp_scan64(o);
    total = __shfl_sync(0xffffffffu, run, 31);
    before = __shfl_sync(0xffffffffu, run - o, rank);
  }
  cluster_arrive_release();  // done with the neighbours' shared memory; waited for at the end

  // ---- the token
  if (A.u && warp == 0) {
    uint64_t at = (uint64_t)fmax(0.0, (double)A.u[row] * (double)total);
    at = min(at, total - 1);
    if (before <= at && at < before + mine) {
      at -= before;
      // The run of pieces, then the lane's piece, then the element.
      const int n = (S.pieces + 31) / 32;
      int q0 = 0;
      for (int u0 = 0; u0 < n; u0 += 32) {
        const uint64_t w = u0 + lane < n ? unit[u0 + lane] : 0;
        const uint64_t run = warp_scan64(w);
        const uint32_t over = __ballot_sync(0xffffffffu, run > at);
        if (over) {
          const int j = __ffs((int)over) - 1;
          at -= __shfl_sync(0xffffffffu, run - w, j);
          q0 = (u0 + j) * 32;
          break;
        }
        at -= __shfl_sync(0xffffffffu, run, 31);
      }
      const int q = q0 + lane, v = S.index(q);
      float x[G];
      uint64_t w[G], sum = 0;
#pragma unroll
      for (int e = 0; e < G; ++e) w[e] = 0;
      if (q < S.pieces) {
        unpack_piece(*reinterpret_cast<const uint4*>(zs + q * G), x);
#pragma unroll
        for (int e = 0; e < G; ++e) {
          if (x[e] > -INFINITY && cut.keeps(x[e], v + e)) w[e] = weight(x[e]);
          sum += w[e];
        }
      }
      const uint64_t run = warp_scan64(sum);
      if (run - sum <= at && at < run) {
        uint64_t acc = run - sum;
        bool done = false;
#pragma unroll
        for (int e = 0; e < G; ++e) {
          acc += w[e];
          if (!done && acc > at) {
            done = true;
            if (A.tokens) A.tokens[row] = v + e;
            if (A.logprobs) A.logprobs[row] = logf((float)w[e] / (float)total);
          }
        }
      }
    }
  }

  // ---- the probabilities
  if (probs) {
    // 1 / total, for weights in units of the maximum's bin.
    const float inv = (float)((double)(1ull << kUnitShift) / (double)total);
    each_piece([&](const float (&x)[G], int v) {
      float y[G];
#pragma unroll
      for (int e = 0; e < G; ++e) {
        y[e] = 0.f;
        if (x[e] >= cut.z && x[e] > -INFINITY && cut.keeps(x[e], v + e)) {
          const auto a = grid.at(x[e]);
          if (a.bin < kBins)
            y[e] = ex2((float)a.bin * (-1.f / 32.f)) * fmaf((float)grid.e32(a), 0x1p-32f, 1.f) * inv;
        }
      }
      put(v, y);
    });
  }
  __syncwarp();
  cluster_wait_acquire();
}

}  // namespace

cudaError_t sample_launch(const SampleArgs& a, cudaStream_t s) {
  const int size = a.bf16 ? 2 : 4;
  Params P{};
  P.a = a;
  for (int j = 0; j < 32; ++j) P.octave[j] = std::exp2(-j / 32.0);
  int C = (int)((a.V * (int64_t)size + kSliceBytes - 1) / kSliceBytes);
  C = std::max(1, std::min(C, kRowMaxCtas));
  while (C < kRowMaxCtas && a.N * 2 * C <= sm_count() && slice_pieces(a.V, size, C) >= 2 * kThreads) C *= 2;
  C = std::min(C, kRowMaxCtas);
  P.C = C;
  P.per = (int)slice_pieces(a.V, size, C);
  const int round = 512;
  P.chunk = ((P.per + kMaxChunks - 1) / kMaxChunks + round - 1) / round * round;
  P.units = (P.per + 31) / 32;
  const int smem = P.per * 16 + kBins * 8 + kList * 8 + P.units * 8;
  prof_before(s, STT_KERNEL_SAMPLE);
  const cudaError_t e = a.bf16 ? launch_rows(sample_kernel<__nv_bfloat16>, P, a.N, C, kThreads, smem, s)
                               : launch_rows(sample_kernel<float>, P, a.N, C, kThreads, smem, s);
  prof_after(s);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

STT_DEFINE_ERROR_ACCESSOR(sample_error_word)
STT_DEFINE_BUDGET_SETTER(sample_set_wait_budget)

}  // namespace stt
