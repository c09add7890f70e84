// top_logits.cu -- the K largest logits of every row, in order, with their indices and
// the logarithm of the row's sum of exponentials.
//
// Bound by HBM: a row is read once.  A CTA (or, with few rows, each CTA of a cluster on
// its slice) looks at a sample of 4096 elements spread over its slice and takes a lower
// bound of the K-th largest from it: a sample's r-th largest, with r so far above the
// K / n share that fewer than K elements of the slice reach it about once in a
// million rows of independent logits.  Then it reads the slice, sums the exponentials
// and keeps what reaches the bound, a few times K elements, as 64-bit keys of logit and
// index, narrows those where they are many, sorts them and has the first K.  Where the
// bound was too high, or too many reach it (equal logits, orders that the sample does not
// show), the K-th largest key is found digit by digit over the slice instead, whatever it
// holds.  The K largest of each slice go to the row's first CTA, which merges them.
//
// 4096 bf16 rows of 151936, K 128: 238 us, 5.2 TB/s (0.78); 777 fp32 rows of 50257, K 64: 46
// us against 23 (1.3 waves of CTAs, and what a row takes apart from its logits).  Bound by
// instructions beside HBM: 10 of a warp for 32 logits, 65 % of the issue slots.  On the way:
// elements kept in the loop 489 us, pieces listed and looked at afterwards 336, listed with
// their bits, narrowed and sorted in the warps' runs 260, exponentials from one product and
// sum 238.  Logits that crowd by index make the runs of 32 pieces a poor sample, and the digits
// cost up to nine more passes: the first case with -a log(index + 100) added takes 232 us for a =
// 0.5, 395 for 0.75, 970 for 1, 5240 for 1.5; with equal logits 8240.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "../../include/stt.h"
#include "attn_common.cuh"
#include "row_slice.cuh"

namespace stt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSample = 16 * kThreads;  // elements looked at first
constexpr int kHeld = 1024;             // listed pieces that are kept with their places
constexpr int kCap = 4096;              // keys that are kept for the sort, at most
constexpr int kMerge = 2048;            // keys that the first CTA of a row sorts, at most

struct Params {
  TopLogitsArgs a;
  float c;            // log2(e) / tau
  float far;          // the difference of logits whose ratio is 2^64
  int C, per;         // CTAs of a row, pieces of a CTA
  int cap;            // keys kept, and pieces listed
};

__device__ __forceinline__ float warp_min(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fminf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <class T>
__global__ void __launch_bounds__(kThreads, 4) top_logits_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(16) uint64_t keys[];  // [cap], [C K] of the row's slices, kHeld pieces, the places of [cap]
  __shared__ int s_n, s_pieces, s_count[3];
  __shared__ float red[2 * kWarps];
  __shared__ uint32_t hist[256];
  __shared__ uint64_t s_cut;
  __shared__ int s_digit, s_need, s_done;
  __shared__ float s_m, s_l;
  constexpr int G = RowSlice<T>::G;
  constexpr int PS = kSample / kThreads / G;  // pieces of the sample, to a thread
  const TopLogitsArgs& A = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)P.C);
  const int64_t row = blockIdx.x / (unsigned)P.C;
  const RowSlice<T> S(static_cast<const T*>(A.z) + row * A.ld_z, A.V, rank, P.per);
  const int K = A.K, cap = P.cap;
  if (tid == 0) s_n = s_pieces = 0;
  __syncwarp();
  if (P.C > 1) cluster_arrive_relaxed();  // everyone runs before anyone writes to the first CTA

  // ---- a bound from the sample; -inf where the slice is kept whole
  float bound = -INFINITY, start = -INFINITY;  // `start`: a first maximum for the sums
  if (S.pieces * G > cap) {
    float x[PS * G];
    // The sample's place whose logit is the bound.
    const float q = (float)K * ((float)kSample / (float)(S.pieces * G));
    const int want = (int)ceilf(q + 4.5f * sqrtf(q) + 4.f);
    // Each warp takes PS runs of 32 pieces, spread evenly over the slice (there are
    // more than 32, and in short slices the runs overlap).
#pragma unroll
    for (int j = 0; j < PS; ++j) {
      const int run = warp * PS + j;
      const int q = (int)((int64_t)(S.pieces - 32) * run / (kWarps * PS - 1)) + lane;
      float y[G];
      if (S.whole(q)) unpack_piece(S.load(q), y);
      else S.edge(q, y);
#pragma unroll
      for (int e = 0; e < G; ++e) x[j * G + e] = y[e];
    }
    float hi = -INFINITY, lo = INFINITY;
#pragma unroll
    for (int i = 0; i < PS * G; ++i) {
      hi = fmaxf(hi, x[i]);
      if (x[i] > -INFINITY) lo = fminf(lo, x[i]);
    }
    const float mine = hi;
    hi = warp_max(hi);
    lo = warp_min(lo);
    if (lane == 0) {
      red[warp] = hi;
      red[kWarps + warp] = lo;
    }
    if (tid < 3) s_count[tid] = 0;
    __syncthreads();
    hi = red[0];
    lo = red[kWarps];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      hi = fmaxf(hi, red[w]);
      lo = fminf(lo, red[kWarps + w]);
    }
    start = hi;
    // Halving until a third more than wanted reach it at most.  `lo` is reached by enough, or
    // is the smallest of all.  (Few wanted ones are hardly ever in one thread's 16: then its
    // largest stands for them, and a step is a barrier that counts.)
    const bool few = want <= kThreads / 4;
    if (hi > lo) {
      for (int it = 0; it < 18; ++it) {
        // Halfway between them, or between their places among the floats where they are
        // far apart (a mask of the type's lowest value).
        const uint32_t below = order_of(lo);
        const float mid = hi - lo < 1024.f ? lo + 0.5f * (hi - lo)
                                           : logit_of(below + (order_of(hi) - below) / 2);
        int n = 0;
        if (few) {
          n = __syncthreads_count(mine >= mid);
        } else {
#pragma unroll
          for (int i = 0; i < PS * G; ++i) n += x[i] >= mid ? 1 : 0;
          n = __reduce_add_sync(0xffffffffu, n);
          if (lane == 0) atomicAdd(&s_count[it % 3], n);
          __syncthreads();
          n = s_count[it % 3];
          if (tid == 0) s_count[(it + 2) % 3] = 0;  // read before this barrier, used after the next
        }
        if (n >= want) lo = mid;
        else hi = mid;
        if (n >= want && n <= want + want / 3) break;
      }
    }
    bound = lo;
    if (!(bound < INFINITY)) bound = -INFINITY;  // nothing in the sample
  }
  __syncthreads();

  // ---- the slice, once: its sum of exponentials, and the pieces in which something
  // reaches the bound.  (Few do, and the elements of those are looked at afterwards: the
  // loop is a subtraction, a product, an exponential and a sum to an element, and half a
  // maximum.)
  uint4* const listed = reinterpret_cast<uint4*>(keys + cap + (P.C > 1 ? kMerge : 0));
  uint32_t* const listed_at = reinterpret_cast<uint32_t*>(listed + kHeld);
  // The reference of the sums, as an exponent of 2: 2^(z c - m) takes one product-and-sum.
  // (Within a range that leaves room to the float's; see the end for logits beyond.)
  auto exponent = [&](float z) { return fminf(fmaxf(z * P.c, -1e38f), 1e38f); };
  float m = -INFINITY, limit = -INFINITY, l = 0.f;  // none yet
  if (fabsf(start) < INFINITY) {
    m = exponent(start);
    limit = start + P.far;
  }
  uint64_t low = f32x2(m == -INFINITY ? 0.f : -m, m == -INFINITY ? 0.f : -m);
  uint64_t sum = 0;  // two sums side by side
  const uint64_t cc = f32x2(P.c, P.c);
  const bool all = bound == -INFINITY;
  const float least = all ? -FLT_MAX : bound;  // (-inf is never taken)
  auto take = [&](int q, const float (&x)[G], const uint4& raw) {
    float top = max3_nan(x[0], x[1], x[2]);
#pragma unroll
    for (int e = 3; e < G; e += 2) top = e + 1 < G ? max3_nan(top, x[e], x[e + 1]) : max_nan(top, x[e]);
    // (NaN, too, is not below the bound.)
    if (!(top < least)) {
      const int at = atomicAdd(&s_pieces, 1);
      if (at < cap) listed_at[at] = (uint32_t)q;
      if (at < kHeld) listed[at] = raw;
      if (top > limit) {  // the reference is too low, or there is none yet
        const float to = exponent(top);
        float s0, s1;
        unpack_f32x2(sum, s0, s1);
        const float f = m == -INFINITY ? 0.f : ex2(m - to);
        sum = f32x2(s0 == 0.f ? 0.f : s0 * f, s1 == 0.f ? 0.f : s1 * f);
        m = to;
        low = f32x2(-m, -m);
        limit = top + P.far;
      }
    }
#pragma unroll
    for (int e = 0; e < G; e += 2) {
      float y0, y1;
      unpack_f32x2(fma_f32x2(f32x2(x[e], x[e + 1]), cc, low), y0, y1);
      sum = add_f32x2(sum, f32x2(ex2(y0), ex2(y1)));
    }
  };
  {
    constexpr int U = 4;
    // Whole pieces, and the one or two others.
    const int first = S.pieces > 0 && !S.whole(0) ? 1 : 0;
    const int last = S.pieces > 0 && !S.whole(S.pieces - 1) ? S.pieces - 1 : S.pieces;
    const uint4* const src = reinterpret_cast<const uint4*>(S.row + S.index(0));
    int q = first + tid;
    if (q + (U - 1) * kThreads < last) {
      uint4 raw[U], then[U];  // the next pieces are on their way
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = __ldg(src + q + u * kThreads);
      auto use = [&](const uint4 (&r)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float x[G];
          unpack_piece(r[u], x);
          take(q + u * kThreads, x, r[u]);
        }
        q += U * kThreads;
      };
      // True if there was another group, which is then in r once its loads are done.
      auto fetch = [&](uint4 (&r)[U]) {
        if (q + (2 * U - 1) * kThreads >= last) return false;
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = __ldg(src + q + (U + u) * kThreads);
        return true;
      };
      while (true) {
        bool more = fetch(then);
        use(raw);
        if (!more) break;
        more = fetch(raw);
        use(then);
        if (!more) break;
      }
    }
    for (; q < last; q += kThreads) {
      float x[G];
      const uint4 raw = __ldg(src + q);
      unpack_piece(raw, x);
      take(q, x, raw);
    }
    if (tid < 2 && S.pieces > 0) {
      const int edge = tid == 0 ? 0 : S.pieces - 1;
      if (!S.whole(edge) && (tid == 0 || S.pieces > 1)) {
        // (As the type's own bits again, which -inf outside the row has too.)
        float x[G];
        S.edge(edge, x);
        uint4 raw;
        if constexpr (G == 4)
          raw = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                           __float_as_uint(x[3]));
        else
          raw = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                           pack_bf16(x[6], x[7]));
        take(edge, x, raw);
      }
    }
    float s0, s1;
    unpack_f32x2(sum, s0, s1);
    l = s0 + s1;
  }
  {
    const float top = warp_max(m);
    l = warp_sum(l == 0.f ? 0.f : l * (m == top ? 1.f : ex2(m - top)));
    if (lane == 0) {
      red[warp] = top;
      red[kWarps + warp] = l;
    }
  }
  __syncthreads();
  // ---- the elements of the listed pieces
  const int n_pieces = s_pieces;
  if (n_pieces <= cap) {
    for (int i0 = warp * 32; i0 < n_pieces; i0 += kThreads) {
      const int i = i0 + lane;
      float x[G];
      int q = 0;
      uint32_t in = 0;
      if (i < n_pieces) {
        q = (int)listed_at[i];
        if (i < kHeld) unpack_piece(listed[i], x);
        else if (S.whole(q)) unpack_piece(S.load(q), x);
        else S.edge(q, x);
#pragma unroll
        for (int e = 0; e < G; ++e) in |= x[e] < least ? 0u : 1u << e;
      }
      // A warp's keys side by side.
      int at = __popc(in);
      const int mine = at;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += t;
      }
      int base = 0;
      if (lane == 31) base = atomicAdd(&s_n, at);
      at += __shfl_sync(0xffffffffu, base, 31) - mine;
      while (in) {
        const int e = __ffs((int)in) - 1;
        in &= in - 1;
        float y = x[0];
#pragma unroll
        for (int i = 1; i < G; ++i) y = e == i ? x[i] : y;
        if (at < cap) keys[at] = place_key(y, S.index(q) + e);
        ++at;
      }
    }
  }
  __syncthreads();
  int n = n_pieces > cap ? cap + 1 : s_n;

  // ---- the K-th largest key digit by digit, where the bound did not do
  if (n > cap || (!all && n < K)) {
    auto each = [&](auto&& f) {
      for (int q = tid; q < (S.pieces + 31) / 32 * 32; q += kThreads) {
        float x[G];
        const bool in = q < S.pieces;
        if (in && S.whole(q)) unpack_piece(S.load(q), x);
        else if (in) S.edge(q, x);
#pragma unroll
        for (int e = 0; e < G; ++e) {
          const bool take = in && !(x[e] == -INFINITY);
          f(take, take ? place_key(x[e], S.index(q) + e) : 0ull);
        }
      }
    };
    uint64_t prefix = 0;
    int need = K;
    for (int shift = 56; shift >= 0; shift -= 8) {
      hist[tid] = 0;
      static_assert(kThreads == 256, "a thread for each digit");
      __syncthreads();
      each([&](bool take, uint64_t key) {
        const bool in = take && (shift == 56 || key >> ((shift + 8) & 63) == prefix);
        const uint32_t d = (uint32_t)(key >> shift) & 255u;
        // A warp of equal digits, as equal logits give, counts at once.
        int same;
        __match_all_sync(0xffffffffu, in ? d : 256u, &same);
        if (same) {
          if (lane == 0 && in) atomicAdd(&hist[d], 32u);
        } else if (in) {
          atomicAdd(&hist[d], 1u);
        }
      });
      __syncthreads();
      if (tid == 0) {
        int above = 0, total = 0, digit = 255;
        if (shift == 56) {
          for (int d = 0; d < 256; ++d) total += (int)hist[d];
          need = min(need, total);
        }
        s_done = need == 0;
        if (need > 0) {
          while (digit > 0 && above + (int)hist[digit] < need) above += (int)hist[digit--];
          need -= above;
          s_done = need == (int)hist[digit];
        }
        s_digit = digit;
        s_need = need;
      }
      __syncthreads();
      need = s_need;
      prefix = prefix << 8 | (uint64_t)s_digit;
      if (s_done || shift == 0) {
        if (tid == 0) {
          s_cut = need == 0 ? ~0ull : prefix << shift;
          s_n = 0;
        }
        break;
      }
    }
    __syncthreads();
    const uint64_t cut = s_cut;
    each([&](bool take, uint64_t key) {
      if (take && key >= cut) {
        const int at = atomicAdd(&s_n, 1);
        if (at < cap) keys[at] = key;
      }
    });
    __syncthreads();
    n = min(s_n, cap);
  }

  // ---- fewer of them, by halving their range of logits: a quarter more than K are enough
  constexpr int kEach = 8;
  if (n > 128 && n > K + K / 2 && n <= kEach * kThreads) {
    uint64_t key[kEach];
    uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      key[j] = tid + j * kThreads < n ? keys[tid + j * kThreads] : 0;
      if (key[j]) lo = min(lo, (uint32_t)(key[j] >> 32));
      hi = max(hi, (uint32_t)(key[j] >> 32));
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      hist[warp] = lo;
      hist[kWarps + warp] = hi;
    }
    if (tid < 3) s_count[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      lo = min(lo, hist[w]);
      hi = max(hi, hist[kWarps + w]);
    }
    for (int it = 0; it < 12 && hi - lo > 1; ++it) {
      const uint32_t mid = lo + (hi - lo) / 2;
      int above_mid = 0;
#pragma unroll
      for (int j = 0; j < kEach; ++j) above_mid += (uint32_t)(key[j] >> 32) >= mid ? 1 : 0;
      above_mid = __reduce_add_sync(0xffffffffu, above_mid);
      if (lane == 0) atomicAdd(&s_count[it % 3], above_mid);
      __syncthreads();
      above_mid = s_count[it % 3];
      if (tid == 0) s_count[(it + 2) % 3] = 0;
      if (above_mid >= K) lo = mid;
      else hi = mid;
      if (above_mid >= K && above_mid <= K + K / 4) break;
    }
    __syncthreads();
    if (tid == 0) s_n = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if ((uint32_t)(key[j] >> 32) >= lo && key[j]) keys[atomicAdd(&s_n, 1)] = key[j];
    __syncthreads();
    n = s_n;
  }

  // ---- in order
  sort_top<kThreads, kCap>(keys, n, K);
  n = min(n, K);

  m = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) m = fmaxf(m, red[w]);
  l = 0.f;
  {
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      l += red[kWarps + w] == 0.f ? 0.f : red[kWarps + w] * (red[w] == m ? 1.f : ex2(red[w] - m));
  }
  auto give = [&](int place, uint64_t key) {
    float z = key ? logit_of((uint32_t)(key >> 32)) : -INFINITY;
    if (z == 0.f) z = (float)S.row[key_index(key)];  // the order knows no sign of it
    A.values[row * K + place] = z;
    A.indices[row * K + place] = key ? key_index(key) : -1;
  };
  if (P.C == 1) {
    for (int i = tid; i < K; i += kThreads) give(i, i < n ? keys[i] : 0ull);
  } else {
    // Every slice's first K to the row's first CTA, where a key's place is the sum of its
    // places among the slices.
    uint64_t* const all_keys = keys + cap;
    if (tid == 0) {
      s_m = m;
      s_l = l;
    }
    __syncwarp();
    cluster_wait_acquire();
    for (int i = tid; i < K; i += kThreads) st_cluster(all_keys + rank * K + i, 0, i < n ? keys[i] : 0ull);
    if (rank == 0)
      for (int i = tid; i < K; i += kThreads) give(i, 0ull);  // where the row has fewer
    cluster_sync();
    if (rank == 0) {
      float om = -INFINITY, ol = 0.f;
      if (lane < P.C) {
        om = ld_cluster(&s_m, lane);
        ol = ld_cluster(&s_l, lane);
      }
      m = warp_max(om);
      l = warp_sum(ol == 0.f ? 0.f : ol * (om == m ? 1.f : ex2(om - m)));
    }
    __syncwarp();
    cluster_arrive_release();  // the sums have been read
    if (rank == 0) {
      // Of every slice's first K / C the last, the least of which has K keys at or above it:
      // what is below is not among the row's (8 bf16 rows of 151936, K 128, 16 CTAs: 61 us
      // without this).
      const int share = (K + P.C - 1) / P.C;
      uint64_t floor_key = ~0ull;
      for (int c = 0; c < P.C; ++c) floor_key = min(floor_key, all_keys[c * K + share - 1]);
      for (int i = tid; i < P.C * K; i += kThreads) {
        const uint64_t key = all_keys[i];
        if (!key || key < floor_key) continue;
        const int own = i / K;
        int place = i - own * K;
        for (int c = 0; c < P.C && place < K; ++c)
          if (c != own) place += above<11>(all_keys + c * K, K, key);
        if (place < K) give(place, key);
      }
    }
    __syncwarp();
    cluster_wait_acquire();  // nobody leaves while its sum is read
    if (rank != 0) return;
  }
  if (A.lse && tid == 0) {
    float lse = fmaf(m, kLn2, logf(l));
    if (l == 0.f || l == INFINITY) {
      // No logit; or the largest is so far from 0 that it alone is left after rounding.
      uint64_t key = P.C == 1 ? (n > 0 ? keys[0] : 0) : 0;
      for (int c = 0; c < P.C && P.C > 1; ++c) key = max(key, keys[cap + c * K]);
      const float z = logit_of((uint32_t)(key >> 32));
      lse = !key ? -INFINITY : z < INFINITY ? __fdiv_rn(z, A.temperature) : NAN;
    }
    A.lse[row] = lse;
  }
}

}  // namespace

cudaError_t top_logits_launch(const TopLogitsArgs& a, cudaStream_t s) {
  const int size = a.bf16 ? 2 : 4;
  Params P{};
  P.a = a;
  P.c = (float)(1.4426950408889634 / (double)a.temperature);
  P.far = 64.f / P.c;
  // CTAs of a row: one while the rows fill the GPU; more for few rows of more than 128 KB,
  // or for rows so long that the sample says little; as many as the first one can merge.
  // (Splitting from 16 KB on: 64 fp32 rows of 32000, K 8: 10.3 us, unsplit 10.1; one bf16 row
  // of 151936: 13.1, unsplit 14.6, from 128 KB on 11.1; 8 of them, K 128: from 128 KB on
  // 14.7, unsplit 19.8; 40 fp32 rows of 151936: 18.2, unsplit 27.2.)
  const int most = std::max(1, std::min(kRowMaxCtas, kMerge / a.K));
  int C = 1;
  while (2 * C <= most && slice_pieces(a.V, 1, C) * 16 > 262144) C *= 2;
  while (2 * C <= most && a.N * 2 * C <= 2 * sm_count() && slice_pieces(a.V, size, C) >= 32 * kThreads) C *= 2;
  P.C = C;
  P.per = (int)slice_pieces(a.V, size, C);
  P.cap = a.K <= 512 ? kCap / 2 : kCap;
  const int smem = P.cap * 12 + kHeld * 16 + (C > 1 ? kMerge * 8 : 0);
  prof_before(s, STT_KERNEL_TOP_LOGITS);
  static Raised raised[2];
  const cudaError_t e =
      a.bf16 ? launch_rows(top_logits_kernel<__nv_bfloat16>, P, a.N, C, kThreads, smem, raised[1], s)
             : launch_rows(top_logits_kernel<float>, P, a.N, C, kThreads, smem, raised[0], s);
  prof_after(s);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace stt
