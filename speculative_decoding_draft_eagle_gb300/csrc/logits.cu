// logits.cu -- the target's logits to the distributions that verification tests
// against: penalties for repeated tokens, bias, grammar mask, temperature,
// softmax.
//
// A cluster of C CTAs takes up to eight consecutive rows of a sequence, each CTA
// every C-th block of 2048 logits (tokens crowd at the low end of a vocabulary, and
// contiguous slices would leave most of the history to one CTA).  It counts the
// sequence's history over its blocks in shared memory (whole numbers: the atomics'
// order does not matter).  A first pass over a row applies everything, writes the
// processed logits to the output and takes their maximum m and the sum l of
// e^(y - m); the pairs of all rows are exchanged with the other CTAs at once; and a
// second pass turns the output into e^(y - M) / L in place, out of L2, which a CTA's
// rows do not leave in between: HBM sees 2 or 4 bytes read and 4 written per logit.
// 320 bf16 rows of 151936 with histories, bias and mask take 129 us against 44 at HBM's
// rate.  Without any of them they take 66, with the bias 85, the mask 87, the history 109
// alone: each CTA of each row (group) scans its sequence's history twice and ranks its
// bit map, the filter costs instructions and a second write of the output, and between
// the passes a row's CTAs wait for one another, with 32 warps an SM to cover it (the same
// with twice the loads in flight; five rows together 137; C half as large, 145).  Keeping
// a row in registers between the passes left fewer warps, 136 to 205 us.  Histories of
// 20000 tokens: 341 us.  Rows that are not aligned to four elements go one element at a
// time: 320 bf16 rows of 50257 take 162 us, of 50256 62.
//
// The tokens that occur in the history are few against the vocabulary.  A bit map
// holds the ones seen; a seen token's rank in it, from the running sum of its words'
// bit counts, is the place of its count, so the counts take 8 KB and not 4 bytes a
// logit, which would keep CTAs off the SM.  The first pass takes seen and forbidden
// elements out with one bit each, and the seen ones are done apart, with their
// penalties, a window of 2048 ranks at a time, and written over what it left.
//
// The pairs go to the other CTAs by st.async, which signals an mbarrier there.  A
// greedy row's pair is its largest value and the lowest index that has it.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <type_traits>

#include "../../include/stt.h"
#include "attn_common.cuh"

namespace stt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxRows = 8;             // rows a cluster takes together
constexpr int kBlock = 8 * kThreads;    // consecutive logits of a CTA
constexpr int kBlocksMax = 10;          // blocks of a CTA at most, where C allows (*)
constexpr int kCtasPerSm = 4;           // by registers
constexpr int kFill = 16;               // CTAs an SM before rows are taken together (*)
// (*) Chosen on 64 x 5 rows of 151936; other values were not tried on other vocabularies.
constexpr int kWindow = 2048;           // seen tokens counted at a time
constexpr uint32_t kPrompt = 0x80000000u;  // the token is in the prompt
constexpr float kLog2E = 1.4426950408889634f;

struct Params {
  LogitsArgs a;
  int C, log_c;            // CTAs per row (a power of two)
  int groups, group_rows;  // row groups of a sequence, rows of a group
  int words;               // of the bit map
  bool withhold;           // test hook: the first CTA of a row sends no pairs
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

// Four elements as loaded.  Four, because a warp then stores whole lines: with eight
// to a thread its 16-byte stores cover half of every sector they touch.  A thread
// takes two such chunks, kApart elements apart, at a time.
constexpr int kChunk = 4;
constexpr int kApart = kThreads * kChunk;
constexpr uint32_t kNibble = (1u << kChunk) - 1u;
template <int bytes> struct RawChunk { using type = uint4; };
template <> struct RawChunk<2> { using type = uint2; };
__device__ __forceinline__ void unpack(const uint4& r, float* x) {
  x[0] = __uint_as_float(r.x);
  x[1] = __uint_as_float(r.y);
  x[2] = __uint_as_float(r.z);
  x[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(const uint2& r, float* x) {
  x[0] = __uint_as_float(r.x << 16);
  x[1] = __uint_as_float(r.x & 0xffff0000u);
  x[2] = __uint_as_float(r.y << 16);
  x[3] = __uint_as_float(r.y & 0xffff0000u);
}
// 2^((x - base) c) of n values.
template <int n>
__device__ __forceinline__ void exponentials(const float (&x)[n], float base, float c,
                                             float (&y)[n]) {
#pragma unroll
  for (int e = 0; e < n; ++e) y[e] = ex2((x[e] - base) * c);
}

// A row's running maximum and sum, or (greedy) maximum and its lowest index.
struct Stat {
  float m, l;
};

// Adds n values to a row's statistics; at(e) is the index of value e.
template <bool GREEDY, int n, class At>
__device__ __forceinline__ void add_values(Stat& s, const float (&x)[n], float c, At&& at) {
  float top = x[0];
#pragma unroll
  for (int e = 1; e < n; ++e) top = fmaxf(top, x[e]);
  if constexpr (GREEDY) {
    if (top > s.m) s.l = __int_as_float(0x7fffffff);
    s.m = fmaxf(s.m, top);
    int best = __float_as_int(s.l);
#pragma unroll
    for (int e = 0; e < n; ++e)
      if (x[e] == s.m) best = min(best, at(e));
    s.l = __int_as_float(best);
  } else {
    // y - m as (x - m) / temperature: exact zeros at the maximum, whatever its size.
    const float m = fmaxf(s.m, top), base = m == -INFINITY ? 0.f : m;
    float l = s.l == 0.f ? 0.f : s.l * ex2((s.m - base) * c), y[n];
    exponentials(x, base, c, y);
#pragma unroll
    for (int e = 0; e < n; ++e) l += y[e];
    s.m = m;
    s.l = l;
  }
}

// Combines the lanes' statistics; every lane gets the result.
__device__ __forceinline__ Stat warp_stat(Stat s, bool greedy, float c) {
  const float M = warp_max(s.m);
  if (greedy) {
    int best = s.m == M ? __float_as_int(s.l) : 0x7fffffff;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
    return Stat{M, __int_as_float(best)};
  }
  const float base = M == -INFINITY ? 0.f : M;
  return Stat{M, warp_sum(s.l == 0.f ? 0.f : s.l * ex2((s.m - base) * c))};
}

// VEC: rows aligned to whole chunks, which a thread takes; else its elements are a
// block apart.  FILTER: there is a mask or a history.
template <class T, bool VEC, bool FILTER>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) logits_kernel(const __grid_constant__ Params P) {
  extern __shared__ uint32_t seen_bits[];  // [words], then [words] ranks before each
  __shared__ Stat s_warp[kMaxRows][kWarps];
  __shared__ __align__(16) float4 s_pair[kMaxRows][kMaxCluster];
  __shared__ uint64_t bar_pair;
  __shared__ uint32_t count[kWindow];
  __shared__ uint16_t list[kWindow];
  __shared__ float s_y[kWindow];  // the listed elements' results, each thread's own
  __shared__ uint32_t s_scan[kWarps];
  const LogitsArgs& A = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)P.C), item = (int)(blockIdx.x / (unsigned)P.C);
  const int b = item / P.groups, i0 = (item - b * P.groups) * P.group_rows;
  const int n_rows = min(P.group_rows, A.rows - i0);
  const int64_t r0 = (int64_t)b * A.rows + i0;
  uint32_t* const rank0 = seen_bits + P.words;
  const bool hist = A.tokens != nullptr || A.draft != nullptr;
  const uint32_t V = (uint32_t)A.V, words = (V + 31) / 32;
  // This CTA's blocks, and the logit where its k-th begins.
  const int n_blocks = ((A.V + kBlock - 1) / kBlock - rank + P.C - 1) >> P.log_c;
  auto block_at = [&](int k) { return ((k << P.log_c) + rank) * kBlock; };

  const float temp = A.temperature ? A.temperature[b] : 1.f;
  const Penalty pen{A.repetition ? A.repetition[b] : 1.f, A.frequency ? A.frequency[b] : 0.f,
                    A.presence ? A.presence[b] : 0.f};
  if (tid == 0) {
    mbar_init(&bar_pair, 1);
    fence_mbar_init();
    if (P.C > 1) mbar_arrive_expect_tx(&bar_pair, (uint32_t)(P.C * n_rows * 16));
  }
  // The first row's logits into L2 while the history is counted (129 -> 124 us).
  if (FILTER && VEC && tid < n_blocks) {
    const int first = block_at(tid), n = min(kBlock, A.V - first) * (int)sizeof(T) & ~15;
    const T* const at = static_cast<const T*>(A.z) + r0 * A.V + first;
    if (n > 0 && (reinterpret_cast<uintptr_t>(at) & 15u) == 0)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(n) : "memory");
  }
  const int32_t* const draft = A.draft ? A.draft + (int64_t)b * A.draft_ld : nullptr;
  if (hist)
    for (int w = tid; w < P.words; w += kThreads) seen_bits[w] = 0;
  __syncthreads();
  if (P.C > 1) cluster_arrive_release();  // everyone runs before anyone writes to a neighbour

  // A token's place among this CTA's logits, or -1.
  auto mine = [&](int token) {
    const uint32_t t = (uint32_t)token, block = t / kBlock;
    return t < V && (block & (uint32_t)(P.C - 1)) == (uint32_t)rank
               ? (int)((block >> P.log_c) * kBlock + t % kBlock)
               : -1;
  };
  // Hands f(place, what) every token of the slice in the history: `what` is kPrompt, 1
  // for one of the output (draft tokens before this group among it), or 0 for a draft
  // token of the group, which its later rows count themselves.
  auto scan_history = [&](auto&& f) {
    if (A.tokens) {
      const int t0 = max(0, min(A.cu_tokens[b], A.n_tokens));
      const int n = min(A.cu_tokens[b + 1], A.n_tokens) - t0;
      const int np = A.n_prompt ? A.n_prompt[b] : 0;
      const int32_t* tok = A.tokens + t0;
#pragma unroll 4
      for (int j = tid; j < n; j += kThreads) {
        const int v = mine(__ldg(tok + j));
        if (v >= 0) f(v, j < np ? kPrompt : 1u);
      }
    }
    if (draft) {
      for (int j = tid; j < i0 + n_rows - 1; j += kThreads) {
        const int v = mine(__ldg(draft + j));
        if (v >= 0) f(v, j < i0 ? 1u : 0u);
      }
    }
  };
  int n_seen = 0;
  if (hist) {
    scan_history([&](int v, uint32_t) { atomicOr(&seen_bits[v >> 5], 1u << (v & 31)); });
    __syncthreads();
    // Ranks: bits before each word.
    const int per = (P.words + kThreads - 1) / kThreads, w0 = min(tid * per, P.words);
    const int w1 = min(w0 + per, P.words);
    uint32_t mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(seen_bits[w]);
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    uint32_t before = incl - mine;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_scan[w];
      n_seen += (int)s_scan[w];
    }
    for (int w = w0; w < w1; ++w) {
      rank0[w] = before;
      before += __popc(seen_bits[w]);
    }
  }
  // Lists and counts the seen tokens of ranks [from, from + kWindow).
  auto window = [&](int from) {
    for (int j = tid; j < kWindow; j += kThreads) count[j] = 0;
    __syncthreads();  // and the ranks, the first time
    scan_history([&](int v, uint32_t what) {
      const int at = (int)(rank0[v >> 5] + __popc(seen_bits[v >> 5] & ((1u << (v & 31)) - 1u))) - from;
      if (at >= 0 && at < kWindow) {
        list[at] = (uint16_t)v;  // every occurrence writes the same
        if (what == kPrompt) atomicOr(&count[at], kPrompt);
        else if (what) atomicAdd(&count[at], 1u);
      }
    });
    __syncthreads();
  };

  const float* const bias =
      A.bias_rows ? A.bias + (A.bias_rows > 1 ? (int64_t)b * A.V : 0) : nullptr;
  const uint32_t* const mask = A.mask ? A.mask + r0 * words : nullptr;
  const bool bias_vec = VEC && (reinterpret_cast<uintptr_t>(bias) & 15u) == 0;
  const T* const z0 = static_cast<const T*>(A.z) + r0 * A.V;
  float* const out0 = A.out + r0 * A.V;

  // The logit of a place.
  auto logit_of = [&](int at) { return block_at(at / kBlock) + at % kBlock; };
  // Element j of the window in row q, with everything applied.
  auto listed = [&](int j, int q) {
    const int v = logit_of(list[j]);
    uint32_t c = count[j];
    if (draft)
      for (int d = i0; d < i0 + q; ++d) c += __ldg(draft + d) == v ? 1u : 0u;
    float x = (float)z0[(uint32_t)q * V + v];
    const float add = bias ? __ldg(bias + v) : 0.f;
    const uint32_t ok =
        mask ? __ldg(mask + (uint32_t)q * words + (v >> 5)) >> (v & 31) : 1u;
    x = pen(x, c) + add;
    return ok & 1u ? x : -INFINITY;
  };
  // f(j, v, q) for every seen element and row.
  int counted = -1;
  auto each_listed = [&](auto&& f) {
    for (int from = 0; from < n_seen; from += kWindow) {
      if (counted != from) {
        if (counted >= 0) __syncthreads();  // the last window is done with
        window(from);
        counted = from;
      }
      const int n = min(kWindow, n_seen - from);
      for (int j = tid; j < n; j += kThreads) f(j, logit_of(list[j]));
    }
  };

  // Hands the elements of row q to f(values, seen bits, first): seen elements (those
  // are the list's) and forbidden ones come as -inf.  A value's index is index(first, e).
  auto sweep = [&](int q, auto&& f) {
    const T* const z = z0 + (uint32_t)q * V;
    const uint32_t* const allowed = mask ? mask + (uint32_t)q * words : nullptr;
    if constexpr (VEC) {
      using Raw = typename RawChunk<sizeof(T)>::type;
      struct Pair {
        Raw raw[2];
        uint32_t allow[2];
      };
      // A pair of chunks; `tail`: the slice may end in it.
      auto load = [&](Pair& p, int k, auto tail) {
        const int v = block_at(k) + tid * kChunk;
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const int at = v + d * kApart;
          if (!decltype(tail)::value || at < A.V) {
            p.raw[d] = *reinterpret_cast<const Raw*>(z + at);
            if (FILTER && allowed) p.allow[d] = __ldg(allowed + ((uint32_t)at >> 5));
          }
        }
      };
      auto work = [&](const Pair& p, int k, auto tail) {
        const int v = block_at(k) + tid * kChunk;
        [[maybe_unused]] const int at = k * kBlock + tid * kChunk;  // its place
        if (decltype(tail)::value && v >= A.V) return;
        const bool second = !decltype(tail)::value || v + kApart < A.V;
        float x[2 * kChunk];
        unpack(p.raw[0], x);
        unpack(p.raw[1], x + kChunk);
        if (bias) {
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            if (d == 0 || second) {
              const float* bb = bias + v + d * kApart;
              if (bias_vec) {
                const float4 t = __ldg(reinterpret_cast<const float4*>(bb));
                x[4 * d] += t.x; x[4 * d + 1] += t.y; x[4 * d + 2] += t.z; x[4 * d + 3] += t.w;
              } else {
#pragma unroll
                for (int e = 0; e < kChunk; ++e) x[4 * d + e] += __ldg(bb + e);
              }
            }
          }
        }
        uint32_t seen = 0;
        if constexpr (FILTER) {
          const int sh = v & 31;
          uint32_t keep = 0xffu;
          if (allowed) keep = (p.allow[0] >> sh & kNibble) | (p.allow[1] >> sh & kNibble) << kChunk;
          if (hist) {
            seen = seen_bits[at >> 5] >> sh & kNibble;
            if (second) seen |= (seen_bits[(at + kApart) >> 5] >> sh & kNibble) << kChunk;
          }
          keep &= ~seen;
#pragma unroll
          for (int e = 0; e < 2 * kChunk; ++e) x[e] = keep & (1u << e) ? x[e] : -INFINITY;
        }
        if (!second) {
#pragma unroll
          for (int e = kChunk; e < 2 * kChunk; ++e) x[e] = -INFINITY;
        }
        f(x, seen, v, second);
      };
      constexpr int U = sizeof(T) == 2 ? 3 : 2;  // blocks whose loads are in flight
      int k = 0;
      Pair p[U];
      for (; k + U <= n_blocks && block_at(k + U - 1) + kBlock <= A.V; k += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) load(p[u], k + u, std::false_type{});
#pragma unroll
        for (int u = 0; u < U; ++u) work(p[u], k + u, std::false_type{});
      }
      for (; k < n_blocks; ++k) {
        load(p[0], k, std::true_type{});
        work(p[0], k, std::true_type{});
      }
    } else {
      for (int at = tid; at < n_blocks * kBlock; at += kThreads) {
        const int v = logit_of(at);
        if (v >= A.V) break;
        const uint32_t seen = hist ? (seen_bits[at >> 5] >> (at & 31)) & 1u : 0u;
        float x[1] = {(float)z[v]};
        if (bias) x[0] += __ldg(bias + v);
        if (seen || (FILTER && allowed && !((__ldg(allowed + (v >> 5)) >> (v & 31)) & 1u)))
          x[0] = -INFINITY;
        f(x, seen, v, false);
      }
    }
  };
  // Seen elements of one window are written over what the first pass stores, after
  // it; of more, the first pass leaves them out.
  const bool over = n_seen <= kWindow;
  const bool in_place = A.z == static_cast<const void*>(A.out);
  auto store = [&](float* dst, const auto& y, uint32_t seen, bool second) {
    if constexpr (VEC) {
      if (!FILTER || over || seen == 0) {
        *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[2], y[3]);
        if (second) *reinterpret_cast<float4*>(dst + kApart) = make_float4(y[4], y[5], y[6], y[7]);
      } else {
#pragma unroll
        for (int e = 0; e < 2 * kChunk; ++e)
          if (!((seen >> e) & 1u) && (e < kChunk || second))
            dst[(e / kChunk) * kApart + e % kChunk] = y[e];
      }
    } else {
      if (over || !seen) dst[0] = y[0];
    }
  };
  // Index of the sweep's value e.
  auto index = [&](int v, int e) {
    return v + (VEC ? (e / kChunk) * kApart + e % kChunk : 0);
  };

  // ------------------------------------------ first pass: processed logits --
  const bool greedy = temp == 0.f && !A.raw;
  // (Below about 2^-127 the quotient is infinite: the largest number instead, by which
  // any difference of logits gives a probability of 0 and none stays 0, not NaN.)
  const float c = temp > 0.f ? fminf(__fdiv_rn(kLog2E, temp), FLT_MAX) : 1.f;
  const float t_raw = temp > 0.f ? temp : 1.f;
  const Stat none = {-INFINITY, greedy ? __int_as_float(0x7fffffff) : 0.f};
  // Without mask and history the second pass takes the logits again, which are in L2 as
  // well: nothing is written twice (320 bf16 rows of 151936: 80 -> 66 us, with a bias 91 ->
  // 83, fp32 97 -> 80).  With them, applying them twice costs more than the writes (130 ->
  // 149 us).
  constexpr bool again = !FILTER;
  auto first_pass = [&](auto mode) {
    constexpr int M = decltype(mode)::value;  // 0: softmax, 1: greedy, 2: raw
    for (int q = 0; q < n_rows; ++q) {
      float* const out = out0 + (uint32_t)q * V;
      Stat st = none;
      // A listed element's value.
      auto single = [&](int j, int v) {
        const float x[1] = {listed(j, q)};
        if constexpr (M == 2) return __fdiv_rn(x[0], t_raw);
        if constexpr (M < 2) add_values<M == 1>(st, x, c, [&](int) { return v; });
        return x[0];
      };
      if (over && n_seen > 0) {
        each_listed([&](int j, int v) { s_y[j] = single(j, v); });
        if (in_place) __syncthreads();  // the sweep below writes over those logits
      }
      sweep(q, [&](auto& x, uint32_t seen, int v, bool second) {
        if constexpr (M == 2) {
#pragma unroll
          for (auto& y : x) y = __fdiv_rn(y, t_raw);
        } else {
          add_values<M == 1>(st, x, c, [&](int e) { return index(v, e); });
        }
        if constexpr (M == 2 || !again) store(out + v, x, seen, second);
      });
      if (over && n_seen > 0) {
        __syncthreads();
        each_listed([&](int j, int v) { out[v] = s_y[j]; });
      }
      if (!over) each_listed([&](int j, int v) { out[v] = single(j, v); });
      if constexpr (M < 2) {
        st = warp_stat(st, M == 1, c);
        if (lane == 0) s_warp[q][warp] = st;
      }
    }
  };
  if (A.raw) {
    if (P.C > 1) cluster_wait_acquire();
    first_pass(std::integral_constant<int, 2>{});
    return;
  }
  if (greedy) first_pass(std::integral_constant<int, 1>{});
  else first_pass(std::integral_constant<int, 0>{});
  __syncthreads();
  if (P.C > 1) cluster_wait_acquire();
  if (warp < n_rows) {  // warp q: row q
    const Stat s = warp_stat(lane < kWarps ? s_warp[warp][lane] : none, greedy, c);
    const float4 p = make_float4(s.m, s.l, 0.f, 0.f);
    if (P.C == 1) {
      if (lane == 0) s_pair[warp][0] = p;
    } else if (lane < P.C && !(P.withhold && rank == 0)) {
      st_async_f4(mapa_shared(smem_u32(&s_pair[warp][rank]), (uint32_t)lane), p,
                  mapa_shared(smem_u32(&bar_pair), (uint32_t)lane));
    }
  }
  if (P.C > 1) {
    cluster_arrive_release();  // this CTA has sent its pairs
    mbar_wait_cluster(&bar_pair, 0, STT_DEVERR_LOGITS_WAIT);
  } else {
    __syncthreads();
  }

  // ----------------------------------------------- second pass: the results --
  for (int q = 0; q < n_rows; ++q) {
    const float4 p = s_pair[q][lane < P.C ? lane : 0];
    const Stat s = warp_stat(lane < P.C ? Stat{p.x, p.y} : none, greedy, c);
    const int best = s.m == -INFINITY ? -1 : __float_as_int(s.l);
    const float top = s.m == -INFINITY ? 0.f : s.m, inv = s.l == 0.f ? 0.f : 1.f / s.l;
    float* const out = out0 + (uint32_t)q * V;
    if constexpr (again) {
      sweep(q, [&](auto& x, uint32_t seen, int v, bool second) {
#pragma unroll
        for (int e = 0; e < (int)(sizeof(x) / sizeof(float)); ++e)
          x[e] = greedy ? (index(v, e) == best ? 1.f : 0.f) : ex2((x[e] - top) * c) * inv;
        store(out + v, x, seen, second);
      });
    } else if constexpr (VEC) {
      auto result = [&](float4 y, int v) {
        if (greedy)
          return make_float4(v == best ? 1.f : 0.f, v + 1 == best ? 1.f : 0.f,
                             v + 2 == best ? 1.f : 0.f, v + 3 == best ? 1.f : 0.f);
        return make_float4(ex2((y.x - top) * c) * inv, ex2((y.y - top) * c) * inv,
                           ex2((y.z - top) * c) * inv, ex2((y.w - top) * c) * inv);
      };
      constexpr int U = 4;  // chunks in flight
      int k = 0;
      for (; k + U / 2 <= n_blocks && block_at(k + U / 2 - 1) + kBlock <= A.V; k += U / 2) {
        float4 y[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          y[u] = *reinterpret_cast<const float4*>(out + block_at(k + u / 2) + (u % 2) * kApart + tid * kChunk);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int v = block_at(k + u / 2) + (u % 2) * kApart + tid * kChunk;
          const float4 r = result(y[u], v);
          st_global_cs_f4(out + v, r);
        }
      }
      for (; k < n_blocks; ++k)
        for (int v = block_at(k) + tid * kChunk; v < min(block_at(k) + kBlock, A.V); v += kApart)
          st_global_cs_f4(out + v, result(*reinterpret_cast<const float4*>(out + v), v));
    } else {
      for (int at = tid; at < n_blocks * kBlock; at += kThreads) {
        const int v = logit_of(at);
        if (v >= A.V) break;
        out[v] = greedy ? (v == best ? 1.f : 0.f) : ex2((out[v] - top) * c) * inv;
      }
    }
  }
  // A CTA whose wait gave up may not leave while pairs are on their way to it: everyone
  // has sent theirs, and they have landed.
  if (P.C > 1) {
    cluster_wait_acquire();
    if (tid == 0) mbar_wait_cluster(&bar_pair, 0, STT_DEVERR_LOGITS_WAIT);
  }
}

using Kernel = void (*)(const Params);

// Raises a kernel's cluster limit, once per device (the first 64).
cudaError_t allow(Kernel kern, int which, int dev) {
  static std::atomic<uint64_t> done[8];
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done[which].load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done[which].fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace

cudaError_t logits_launch(const LogitsArgs& a, cudaStream_t s) {
  // CTAs per row: as few as leave a CTA ten blocks or less; more while the
  // rows alone leave SMs idle.
  const int blocks = (a.V + kBlock - 1) / kBlock;
  auto blocks_of = [&](int c) { return (blocks + c - 1) / c; };
  int C = 1;
  while (C < kMaxCluster && blocks_of(C) > kBlocksMax) C *= 2;
  while (C < kMaxCluster && (int64_t)a.N * C * 2 <= sm_count() && blocks_of(C) >= 2) C *= 2;
  Params P{};
  P.a = a;
  P.C = C;
  while ((1 << P.log_c) < C) ++P.log_c;
  // Rows of a sequence that share its counts: up to eight, fewer while that makes less
  // than kFill CTAs an SM (64 sequences of five rows: one at a time or two together 129 us,
  // three 137).
  const int64_t B = a.N / a.rows;
  int most = std::min(kMaxRows, a.rows);
  while (most > 1 && B * ((a.rows + most - 1) / most) * C < kFill * sm_count()) --most;
  P.groups = (a.rows + most - 1) / most;
  P.group_rows = (a.rows + P.groups - 1) / P.groups;
  P.groups = (a.rows + P.group_rows - 1) / P.group_rows;
  const uintptr_t zo = reinterpret_cast<uintptr_t>(a.z) | reinterpret_cast<uintptr_t>(a.out);
  const bool vec = a.V % kChunk == 0 && (zo & 15u) == 0;
  const bool filter = a.mask || a.tokens || a.draft;
  const int which = (a.bf16 ? 4 : 0) + (vec ? 2 : 0) + (filter ? 1 : 0);
  static const Kernel kernels[8] = {
      logits_kernel<float, false, false>, logits_kernel<float, false, true>,
      logits_kernel<float, true, false>, logits_kernel<float, true, true>,
      logits_kernel<__nv_bfloat16, false, false>, logits_kernel<__nv_bfloat16, false, true>,
      logits_kernel<__nv_bfloat16, true, false>, logits_kernel<__nv_bfloat16, true, true>};
  const Kernel kern = kernels[which];
  P.words = blocks_of(C) * (kBlock / 32);
  P.withhold = (debug_inject() & STT_INJECT_LOGITS_WITHHOLD_PAIRS) != 0;
  const int smem = (a.tokens || a.draft) ? P.words * 8 : 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = allow(kern, which, dev);
  if (e != cudaSuccess) return e;
  const int64_t ctas = B * P.groups * C;
  if (ctas > 0x7fffffffll) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
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

STT_DEFINE_ERROR_ACCESSOR(logits_error_word)
STT_DEFINE_BUDGET_SETTER(logits_set_wait_budget)

}  // namespace stt
