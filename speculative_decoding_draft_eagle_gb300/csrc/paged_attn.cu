// paged_attn.cu -- attention of each sequence's new tokens over its pages.
//
// A unit of work is a query tile of one KV head: up to 128 rows, row t G + g
// being head g of the group of G query heads at new token t of the tile, so that
// every key a CTA loads serves the whole group and, when there are few new
// tokens, all of them.  A unit runs over the 128-key tiles that its last token
// sees, flash-style: S = Q K^T and O += P V on the tensor cores (tcgen05, S and O
// in tensor memory), keys and values brought page by page by TMA into swizzled
// shared memory, softmax with a running maximum and sum in between.
//
// Persistent, one CTA per SM.  Every key tile of every unit counts one, and a share
// is a run of tiles in the order (sequence, KV head, query tile, key tile), cut where
// it comes: CTA c takes the tiles [c W / G, (c + 1) W / G) of all W, so that whatever
// the lengths, the shares differ by one tile at most.  Where there are two units or
// more to a CTA, whole ones are dealt first, a round of G neighbours at a time: they
// are query tiles of a few heads, which go through the same keys side by side, out of
// L2 (dealt in runs alone, chunks on 170 MB of keys read 1.9 GB from HBM, 0.18 this
// way).  The units left, between one and two to a CTA, go in runs that make the CTAs'
// totals even.  With 0.8 to 2 units to a CTA one round is dealt if the keys that several
// query tiles read are more than L2 keeps and the units are about as long as one
// another (500 tokens on 120 thousand keys: 888 TFLOP/s in runs, 1232 dealt).  A unit
// cut by a share's border leaves partial results
// (normalised rows and their logarithms of the sum) in the workspace, at most two
// per CTA, and a second small kernel, launched as a programmatic dependent, joins
// them in a fixed order.  The lengths are read on the device: nothing here depends
// on what the host knows of the batch.
//
// What bounds it: HBM for few new tokens (six tokens on each of four contexts of 90 to
// 131 thousand keys, 32 query and 8 KV heads of 128: 255 us, 6.79 TB/s, all of the copy
// rate), the tensor cores with the softmax between them for chunks (500 to 2048 tokens
// on 4 to 16 thousand keys: 561 us, 1284 TFLOP/s, 0.67 of cuBLAS's burst; 520 repeated
// on one state.  A row's two warps taking whole tiles in turn, not halves, made that 510,
// and units of few tiles 5 to 20 % longer).  With units of a few tiles the fixed parts
// show (4 us until the batch is laid out, 3 to the first scores, 5 for the join; a unit's
// end of 2 us passes while the next tiles load): trees of 16 tokens on 32 sequences of 500
// to 4000 keys take 63 us, 0.67 of the copy rate, although the tiles themselves pass at
// all of it; 64 prompts of 128 tokens, units of one tile, 72 us.  One token on 777 keys
// takes 13 us (14.5 launched behind what came before, not beside its end): this kernel's
// chain for a single tile, and 4 the join's.  With one warp per row and head, and no
// tensor cores, these took 130, 154, 6.7 and 0.4 ms.
//
// Warp roles (384 threads), as in the training forward (attn_fwd.cu):
//   warps 0-7  softmax: warps w and w + 4 own the 32 rows of TMEM lane quarter
//              w % 4 and half of the 128 keys each; a quarter without live rows
//              only keeps the barriers going.
//   warp 8     queries and key pages (TMA); lanes look the pages up, a tile ahead.
//   warp 9     issues S(g) into TMEM buffer g % 3.
//   warp 10    issues O += P(g) V(g), P read from TMEM.
//   warp 11    value pages (TMA).
// Barrier phases count S products, stage uses and units over the CTA's whole share.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../../include/stt.h"
#include "attn_common.cuh"

namespace stt {
namespace {

constexpr int kStages = 2;
constexpr int kSoftmaxWarps = 8;
constexpr int kWarpK = 8, kWarpMma = 9, kWarpPv = 10, kWarpV = 11;
constexpr int kThreads = 384;
constexpr int kMaxCtas = 160;  // CTAs the workspace has room for
constexpr unsigned long long kL2Keeps = 64ull << 20;  // bytes of keys and values, about
constexpr int kJoinThreads = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P <= 2^8 between rescales
constexpr uint32_t kTmemCols = 512;
constexpr int kSBufs = 3;
constexpr uint32_t kColO = kSBufs * kTile;

// 4-D tiled load global -> shared, completion counted on `bar` in bytes.
__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, uint64_t* bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// A unit cut by share borders, as seen from the CTA whose share begins inside it.
struct JoinDesc {
  int c0, c1;  // first and last CTA with a part; c0 < 0: none
  int tok0, ntok, kvh, pad[3];
};

struct Params {
  PagesArgs g;
  const uint32_t* tree;
  __nv_bfloat16* out;
  float* lse;
  JoinDesc* join;
  float* part;       // [2 ctas][slot]: O [slot_rows][D], then lse [slot_rows]
  int tree_words, N, H, G, TT, slot_rows;
  int64_t slot;      // floats from slot to slot
  int key_cap;       // max_pages * page_size
  int d_tok, d_head, d_page;  // place of each among the cache map's outer dimensions
  float scale_log2;
  uint32_t inject;  // STT_INJECT_* test hooks (0 in normal use)
};

template <int D>
struct Smem {
  static constexpr int kQ = kTile * D * 2;
  static constexpr int kKV = kTile * D * 2;
  static constexpr int q = 0;  // two Q buffers (unit parity)
  static constexpr int k0 = 2 * kQ;
  static constexpr int v0 = 2 * kQ + kStages * kKV;
  static constexpr int total = 2 * kQ + 2 * kStages * kKV;
  static constexpr int alloc = total + 1024;
};

// The batch in shared memory.
struct Batch {
  long long pref[kMaxBatch + 1];  // tiles before each sequence
  int qt[kMaxBatch + 1];          // query tiles before each sequence (a unit: one per KV head)
  int first[kMaxBatch], n[kMaxBatch], len[kMaxBatch];
  long long start[kMaxCtas + 1];  // the CTAs' runs of tiles
  long long dealt[2][kMaxCtas];   // tiles of the whole units dealt to each CTA, in halves
  unsigned long long shared;      // keys that several query tiles read
  int most;                       // tiles of the longest unit dealt (one round)
  int rounds;                     // rounds of whole units
  int at_b, at_h, at_j, at_off;   // where this CTA's run begins
};

// The last sequence whose entry of a running sum is not above x.
template <class T>
__device__ __forceinline__ int seq_of(const T* sums, int B, T x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Keys the query tile j of a sequence needs.
__device__ __forceinline__ int unit_keys(const Params& P, int n, int len, int j) {
  const int cap = min(len, P.key_cap);
  if (P.tree) return max(cap, 0);
  const int last = min((j + 1) * P.TT, n);  // tokens up to the tile's end
  return max(min(len - n + last, cap), 0);
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }

// a / b; in 32 bits where both fit, which is a fraction of the instructions.
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// Part of one unit in a CTA's share: key tiles [t0, t1) of `tiles`.
struct Seg {
  int b, h, j, t0, t1, tiles, keys;
  int have;  // keys of the sequence; `keys` are those that the unit sees
  int tok0, ntok, ctx;
};

__device__ __forceinline__ int unit_cost(const Params& P, const Batch& S, int b, int j) {
  return max(tiles_of(unit_keys(P, S.n[b], S.len[b], j)), 1);
}
// Unit u in the order of all: its sequence, head and query tile.
__device__ __forceinline__ void unit_at(const Params& P, const Batch& S, int u, int& b, int& h,
                                        int& j) {
  b = 0;
  for (int step = kMaxBatch / 2; step > 0; step >>= 1)
    if (b + step < P.g.B && (long long)S.qt[b + step] * P.g.H_kv <= u) b += step;
  const int tiles = S.qt[b + 1] - S.qt[b], r = u - S.qt[b] * P.g.H_kv;
  // r / tiles is a head: few enough for a quotient of floats to be off by one at most.
  h = (int)__fdividef((float)r, (float)tiles);
  j = r - h * tiles;
  if (j < 0) {
    --h;
    j += tiles;
  } else if (j >= tiles) {
    ++h;
    j -= tiles;
  }
}
// Unit that CTA c of n takes in a round (snake order).
__device__ __forceinline__ int dealt_unit(int round, int c, int n) {
  return round * n + ((round & 1) ? n - 1 - c : c);
}

// A CTA's segments: the whole units dealt to it, then its run of tiles.
struct Walk {
  long long left;  // tiles of the run to come
  int b, h, j, off, round;

  __device__ __forceinline__ void init(const Batch& S) {
    round = 0;
    left = S.start[blockIdx.x + 1] - S.start[blockIdx.x];
    b = S.at_b;
    h = S.at_h;
    j = S.at_j;
    off = S.at_off;
  }

  __device__ __forceinline__ bool next(const Params& P, const Batch& S, int ctas, Seg& s) {
    const bool whole = round < S.rounds;
    if (whole) {
      unit_at(P, S, dealt_unit(round, blockIdx.x, ctas), s.b, s.h, s.j);
      ++round;
    } else {
      if (left <= 0) return false;
      s.b = b;
      s.h = h;
      s.j = j;
    }
    const int n = S.n[s.b], len = S.len[s.b];
    s.ctx = len - n;
    s.keys = unit_keys(P, n, len, s.j);
    s.have = max(min(len, P.key_cap), 0);
    s.tiles = tiles_of(s.keys);
    s.tok0 = S.first[s.b] + s.j * P.TT;
    s.ntok = min(P.TT, n - s.j * P.TT);
    const int cost = max(s.tiles, 1);
    s.t0 = 0;
    s.t1 = cost;
    if (!whole) {
      s.t0 = off;
      if (cost - off > left) s.t1 = off + (int)left;
      left -= s.t1 - s.t0;
      off = 0;
      if (++j * P.TT >= n) {
        j = 0;
        if (++h == P.g.H_kv) {
          h = 0;
          do ++b; while (b < P.g.B && S.n[b] <= 0);
        }
      }
    }
    if (s.tiles == 0) s.t0 = s.t1 = 0;  // its place in the order is not a tile
    return true;
  }
};

// The 32 bits of a row's tree mask over keys whose first is `o` after the context:
// ones before the context's end.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t* row, int words, int o) {
  const int w = o >> 5;
  const uint32_t lo = w < 0 ? 0xffffffffu : (w < words ? row[w] : 0u);
  const uint32_t hi = w + 1 < 0 ? 0xffffffffu : (w + 1 < words ? row[w + 1] : 0u);
  return __funnelshift_r(lo, hi, o & 31);
}

// Tiles of the query tiles before the first `count` of a sequence, for one KV head (the
// whole warp calls this).
__device__ __forceinline__ long long tiles_before(const Params& P, const Batch& S, int b,
                                                  int count) {
  long long t = 0;
  for (int x = threadIdx.x & 31; x < count; x += 32) t += unit_cost(P, S, b, x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// Where the run that begins at tile `pos` does (one warp).
__device__ __forceinline__ void locate(const Params& P, Batch& S, long long pos) {
  const int lane = threadIdx.x & 31;
  const int b = seq_of(S.pref, P.g.B, pos);
  long long rem = pos - S.pref[b];
  const int tiles = S.qt[b + 1] - S.qt[b];
  const bool one = tiles == 1;  // as for single tokens: half of the time
  const long long per_head = one ? (long long)unit_cost(P, S, b, 0)
                                 : div_ll(S.pref[b + 1] - S.pref[b], P.g.H_kv);
  const int h = (int)div_ll(rem, per_head);
  rem -= h * per_head;
  if (one) {
    if (lane == 0) {
      S.at_b = b;
      S.at_h = h;
      S.at_j = 0;
      S.at_off = (int)rem;
    }
    return;
  }
  for (int j0 = 0; j0 < tiles; j0 += 32) {
    const int cost = j0 + lane < tiles ? unit_cost(P, S, b, j0 + lane) : 0;
    int incl = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, rem < incl);
    if (past) {
      if (lane == __ffs(past) - 1) {
        S.at_b = b;
        S.at_h = h;
        S.at_j = j0 + lane;
        S.at_off = (int)rem - (incl - cost);
      }
      return;
    }
    rem -= __shfl_sync(0xffffffffu, incl, 31);
  }
}

// Deals `rounds` rounds of whole units to n CTAs, and gives the units left to their runs:
// each gets what its dealt units leave of an even total (one tile at least).  False if
// the dealt units are too uneven for that (one round only).  Every CTA works the same
// plan out; the whole block calls this.  A CTA's rounds are summed by two threads (sums
// in shared memory by 64-bit atomics, and runs in doubles, took 10 us of 64 x 128 tokens).
__device__ __noinline__ bool plan_rounds(const Params& P, Batch& S, int n, int rounds) {
  static_assert(kThreads >= 2 * kMaxCtas, "two threads to a CTA");
  const int tid = threadIdx.x;
  const long long W = S.pref[P.g.B], units = (long long)S.qt[P.g.B] * P.g.H_kv;
  if (tid < 2 * n) {
    const int part = tid >= n, c = tid - part * n;
    long long sum = 0;
#pragma unroll 1
    for (int r = part; r < rounds; r += 2) {
      int b, h, j;
      unit_at(P, S, dealt_unit(r, c, n), b, h, j);
      const int cost = unit_cost(P, S, b, j);
      if (rounds == 1) atomicMax(&S.most, cost);
      sum += cost;
    }
    S.dealt[part][c] = sum;
  }
  __syncthreads();
  const long long even = div_ll(W, n);
  const bool none_left = units == (long long)rounds * n;
  long long first = W;  // tiles before the units left
  if (!none_left) {
    int b, h, j;
    unit_at(P, S, rounds * n, b, h, j);
    first = S.pref[b] + div_ll(S.pref[b + 1] - S.pref[b], P.g.H_kv) * h +
            tiles_before(P, S, b, j);
  }
  const long long left = W - first;
  if (rounds == 1) {
    // One unit each: no longer than a quarter over an even share of all SMs.  A unit each
    // and a run: within a tenth of an even total.
    if (none_left ? (long long)S.most * gridDim.x * 4 > W * 5
                  : left < n || (long long)S.most * 10 > even * 11)
      return false;
  }
  if (none_left) {
    if (tid < 32)  // the warp that reads a border before the next barrier
      for (int c = tid; c <= n; c += 32) S.start[c] = W;
    return true;
  }
  if (tid < 32) {
    constexpr int kPer = (kMaxCtas + 31) / 32;
    const int shift = max(0, 34 - __clzll(W));  // sums below 2^30
    int need[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = tid * kPer + i;
      // (One over the quotient, less the one that every run has: where the quotient has
      // lost a fraction, all of them stay in proportion.)
      need[i] =
          c < n ? (int)(max(even - (S.dealt[0][c] + S.dealt[1][c]), 0ll) >> shift) : 0;
      sum += need[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (tid >= o) incl += v;
    }
    const int all = __shfl_sync(0xffffffffu, incl, 31);
    int before = incl - sum;
    // In floats: the shares need not be exact, only in order (and each step here keeps it).
    const float spare = (float)(left - n), scale = all > 0 ? __fdividef(1.f, (float)all) : 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = tid * kPer + i;
      if (c < n)
        S.start[c] = first + c + min((long long)((float)before * scale * spare), left - n);
      before += need[i];
    }
    if (tid == 0) S.start[n] = W;
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ Params P, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV) {
  using L = Smem<D>;
  constexpr uint32_t kSite = STT_DEVERR_PAGED_WAIT;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // Phases as in the training forward: see there why p_full and s_free are per S
  // buffer and o_done alternates.
  __shared__ uint64_t bar_q_full[2], bar_q_empty[2], bar_k_full[kStages], bar_v_full[kStages],
      bar_k_empty[kStages], bar_v_empty[kStages], bar_s_full[kSBufs], bar_s_free[kSBufs],
      bar_p_full[kSBufs], bar_o_done[2], bar_o_final, bar_drain, bar_quad[4];
  __shared__ uint32_t tmem_base;
  __shared__ float s_max[2][2][kTile], s_sum[2][2][kTile];
  __shared__ Batch S;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = P.g.B;
  // The join's blocks may take their places as CTAs leave; they wait for the rest.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (lane == 0 && (warp == kWarpK || warp == kWarpV)) {
    tma_prefetch_desc(warp == kWarpK ? &tmK : &tmV);
    if (warp == kWarpK) tma_prefetch_desc(&tmQ);
  }
  if (tid == 0) {
    S.most = 0;
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bar_q_full[x], 1);
      mbar_init(&bar_q_empty[x], 1 + kSoftmaxWarps);
      mbar_init(&bar_o_done[x], 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar_k_full[s], 1);
      mbar_init(&bar_v_full[s], 1);
      mbar_init(&bar_k_empty[s], 1);
      mbar_init(&bar_v_empty[s], 1);
    }
    for (int s = 0; s < kSBufs; ++s) {
      mbar_init(&bar_s_full[s], 1);
      mbar_init(&bar_s_free[s], 1);
      mbar_init(&bar_p_full[s], kSoftmaxWarps);
    }
    mbar_init(&bar_o_final, 1);
    mbar_init(&bar_drain, 2);
    for (int q = 0; q < 4; ++q) mbar_init(&bar_quad[q], 2);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_base, kTmemCols);
    tmem_relinquish();
  }
  // What was launched before is complete from here on; all above ran beside its end.  (It
  // may have written the lists while this kernel ran: they are read by ordinary loads, not
  // as constant data.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // The batch: rows and lengths, each sequence's tiles (by a warp where it has more than a
  // few query tiles), their sums.
  int many = 0;
  for (int b = tid; b < B; b += kThreads) {
    const int lo = max(0, min(P.g.cu_q[b], P.N));
    const int hi = max(lo, min(P.g.cu_q[b + 1], P.N));
    const int n = hi - lo, len = P.g.seq_lens[b], tiles = (n + P.TT - 1) / P.TT;
    S.first[b] = lo;
    S.n[b] = n;
    S.len[b] = len;
    if (n > 0 && len > P.key_cap) record_error(STT_DEVERR_PAGE);
    long long t = -1;
    if (tiles <= 4) {
      t = 0;
      for (int j = 0; j < tiles; ++j) t += max(tiles_of(unit_keys(P, n, len, j)), 1);
    } else {
      many = 1;
    }
    S.qt[b + 1] = tiles;
    S.pref[b + 1] = t * P.g.H_kv;
  }
  many = __syncthreads_or(many);
  if (many) {
    for (int b = warp; b < B; b += kThreads / 32)
      if (S.pref[b + 1] < 0) {
        const long long t = tiles_before(P, S, b, S.qt[b + 1]);
        __syncwarp();
        if (lane == 0) S.pref[b + 1] = t * P.g.H_kv;
      }
    __syncthreads();
  }
  if (warp == 1) {
    long long carry = 0;
    unsigned long long shared = 0;
    int carry_u = 0;
    if (lane == 0) {
      S.pref[0] = 0;
      S.qt[0] = 0;
    }
    for (int b0 = 0; b0 < B; b0 += 32) {
      long long v = b0 + lane < B ? S.pref[b0 + lane + 1] : 0;
      int u = b0 + lane < B ? S.qt[b0 + lane + 1] : 0;
      if (many && b0 + lane < B && S.n[b0 + lane] > 4 * P.TT) shared += max(S.len[b0 + lane], 0);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v1 = __shfl_up_sync(0xffffffffu, v, o);
        const int u1 = __shfl_up_sync(0xffffffffu, u, o);
        if (lane >= o) {
          v += v1;
          u += u1;
        }
      }
      v += carry;
      u += carry_u;
      if (b0 + lane < B) {
        S.pref[b0 + lane + 1] = v;
        S.qt[b0 + lane + 1] = u;
      }
      carry = __shfl_sync(0xffffffffu, v, 31);
      carry_u = __shfl_sync(0xffffffffu, u, 31);
    }
    for (int o = many ? 16 : 0; o > 0; o >>= 1) shared += __shfl_xor_sync(0xffffffffu, shared, o);
    if (lane == 0) S.shared = shared;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const long long W = S.pref[B];
  const int grid = (int)gridDim.x, units = S.qt[B] * P.g.H_kv;
  int ctas = (int)(W < (long long)grid ? W : (long long)grid), rounds = 0;
  if (units >= 2 * grid) {
    rounds = units / grid - 1;
  } else if ((long long)units * 5 >= (long long)grid * 4 &&
             S.shared * (unsigned long long)(P.g.H_kv * D * 4) > kL2Keeps) {
    rounds = 1;
  }
  if (rounds > 0) {
    const int n = min(units, grid);
    if (plan_rounds(P, S, n, rounds)) ctas = n;
    else rounds = 0;
  }
  const auto border = [&](int c) { return div_ll(W * c, max(ctas, 1)); };
  if (rounds == 0 && warp > 0)
    for (int c = tid - 32; c <= ctas; c += kThreads - 32) S.start[c] = border(c);
  if (warp == 0) {  // (the borders were written by this warp if there are rounds)
    __syncwarp();
    if (lane == 0) S.rounds = rounds;
    const long long pos =
        (int)blockIdx.x >= ctas ? W : (rounds == 0 ? border(blockIdx.x) : S.start[blockIdx.x]);
    if (pos < W) locate(P, S, pos);
  }
  __syncthreads();
  Walk walk;
  walk.left = 0;
  walk.round = rounds;
  if ((int)blockIdx.x < ctas) walk.init(S);
  Seg s, nx;

  if (warp == kWarpK || warp == kWarpV) {
    // --------------------------------------------------- page producers ----
    const bool is_k = warp == kWarpK;
    const CUtensorMap* const tm = is_k ? &tmK : &tmV;
    unsigned char* const base = smem + (is_k ? L::k0 : L::v0);
    uint64_t* const full = is_k ? bar_k_full : bar_v_full;
    uint64_t* const empty = is_k ? bar_k_empty : bar_v_empty;
    const int page = 1 << P.g.page_shift;
    const int box = min(page, kTile);      // keys a copy brings
    const int copies = kTile / box;        // copies a tile takes, one lane each
    uint32_t g = 0, i = 0, q_issued = 0;
    bool ok = true;
    while (ok && walk.next(P, S, ctas, s)) {
      if (s.tiles == 0) continue;
      if (is_k) {
        const int qs = i & 1;
        if (i >= 2) ok = warp_wait(&bar_q_empty[qs], ((i >> 1) - 1u) & 1u, kSite);
        if (!ok) break;
        // Test hook: queries are never loaded, the S issuer's wait for them runs out, and
        // every role gives up in turn.
        const bool withhold = (P.inject & STT_INJECT_PAGED_WITHHOLD_Q) != 0;
        if (lane == 0 && !withhold) {
          mbar_arrive_expect_tx(&bar_q_full[qs], (uint32_t)(P.G * P.TT * D * 2));
          for (int cb = 0; cb < D / kColBlock; ++cb)
            tma_load_3d(smem + L::q + qs * L::kQ + cb * kTile * 128, &tmQ, &bar_q_full[qs],
                        cb * kColBlock, s.h * P.G, s.tok0);
        }
        if (!withhold) q_issued = i + 1;
      }
      const int32_t* table = P.g.table + (int64_t)s.b * P.g.max_pages;
      // This lane's page of a tile (-1: past the sequence's keys).
      auto look = [&](int t) {
        const int key = t * kTile + lane * box;
        return lane < copies && t < s.t1 && key < s.have ? table[key >> P.g.page_shift]
                                                          : -1;
      };
      int pg = look(s.t0);
      for (int t = s.t0; t < s.t1; ++t, ++g) {
        const int st = g & 1;
        const int key = t * kTile + lane * box;
        const bool mine = lane < copies && key < s.have;
        int p = pg;
        pg = look(t + 1);
        if (mine && (p < 0 || p >= P.g.num_pages)) {
          record_error(STT_DEVERR_PAGE);
          p = 0;
        }
        if (g >= (uint32_t)kStages) ok = warp_wait(&empty[st], ((g >> 1) - 1u) & 1u, kSite);
        if (!ok) break;
        const int n_copies = __popc(__ballot_sync(0xffffffffu, mine));
        if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(n_copies * box * D * 2));
        __syncwarp();
        if (mine) {
          const int in_page = key & (page - 1);
          const int c1 = P.d_tok == 1 ? in_page : (P.d_head == 1 ? s.h : p);
          const int c2 = P.d_tok == 2 ? in_page : (P.d_head == 2 ? s.h : p);
          const int c3 = P.d_tok == 3 ? in_page : (P.d_head == 3 ? s.h : p);
          for (int cb = 0; cb < D / kColBlock; ++cb)
            tma_load_4d(base + st * L::kKV + cb * kTile * 128 + lane * box * 128, tm, &full[st],
                        cb * kColBlock, c1, c2, c3);
        }
      }
      ++i;
    }
    // Every copy issued lands before the CTA exits (on the way out after a wait that
    // gave up, too).
    for (uint32_t x = g > (uint32_t)kStages ? g - kStages : 0; x < g; ++x)
      mbar_wait(&full[x & 1], (x >> 1) & 1u, kSite);
    for (uint32_t x = q_issued > 2 ? q_issued - 2 : 0; x < q_issued; ++x)
      mbar_wait(&bar_q_full[x & 1], (x >> 1) & 1u, kSite);
  } else if (warp == kWarpMma || warp == kWarpPv) {
    // ------------------------------------------------------- MMA issuers --
    if (lane == 0) {
      const uint32_t idS = idesc_bf16(128, kTile, false, false);
      const uint32_t idO = idesc_bf16(128, D, false, true);
      const uint64_t dK0 = sdesc_sw128(smem_u32(smem + L::k0), 16, 1024);
      const uint64_t dV0 = sdesc_sw128(smem_u32(smem + L::v0), kTile * 128, 1024);
      uint32_t g = 0, i = 0;
      bool ok = true;
      while (ok && walk.next(P, S, ctas, s)) {
        if (s.tiles == 0) continue;
        if (warp == kWarpMma) {
          ok = mbar_wait(&bar_q_full[i & 1], (i >> 1) & 1u, kSite);
          const uint64_t dQ = sdesc_sw128(smem_u32(smem + L::q + (i & 1) * L::kQ), 16, 1024);
          for (int t = s.t0; ok && t < s.t1; ++t, ++g) {
            const int st = g & 1, sb = (int)(g % kSBufs);
            ok = mbar_wait(&bar_k_full[st], (g >> 1) & 1u, kSite);
            if (ok && g >= (uint32_t)kSBufs)
              ok = mbar_wait(&bar_s_free[sb], (g / kSBufs - 1u) & 1u, kSite);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dK = sdesc_add(dK0, st * L::kKV);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * kTile * 128 + (kk & 3) * 32;
              umma_bf16_ss(tmem + sb * kTile, sdesc_add(dQ, off), sdesc_add(dK, off), idS,
                           kk > 0 ? 1u : 0u);
            }
            umma_commit(&bar_s_full[sb]);
            umma_commit(&bar_k_empty[st]);
          }
          if (ok) umma_commit(&bar_q_empty[i & 1]);
        } else {
          for (int t = s.t0; ok && t < s.t1; ++t, ++g) {
            const int st = g & 1, sb = (int)(g % kSBufs);
            ok = mbar_wait(&bar_p_full[sb], (g / kSBufs) & 1u, kSite) &&
                 mbar_wait(&bar_v_full[st], (g >> 1) & 1u, kSite);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dV = sdesc_add(dV0, st * L::kKV);
            const uint32_t aP = tmem + sb * kTile;
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              umma_bf16_ts(tmem + kColO, aP + (kk >> 2) * 64 + (kk & 3) * 8,
                           sdesc_add(dV, kk * 2048), idO, (t > s.t0 || kk > 0) ? 1u : 0u);
            umma_commit(&bar_o_done[g & 1]);
            umma_commit(&bar_s_free[sb]);
            umma_commit(&bar_v_empty[st]);
          }
          if (ok) umma_commit(&bar_o_final);
        }
        ++i;
      }
      umma_commit(&bar_drain);
      mbar_wait(&bar_drain, 0, kSite);
    }
  } else {
    // ------------------------------------------------------------ softmax --
    constexpr int DH = D / 2;  // O columns per thread
    const int quarter = warp & 3, part = warp >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const float sl2 = P.scale_log2;
    const int t_row = r / P.G, g_row = r - t_row * P.G;
    uint32_t quad_uses = 0, g = 0, n_final = 0;
    const int row_off = t_row * P.H + g_row;  // in rows of `out`
    // Where this warp turns rows held by lanes into rows held by chunks: its eighth of
    // the unit's query buffer, which its last S has read.
    constexpr int kChunks = DH / 8, kRowsAt = 32 / kChunks;  // 16-byte chunks, rows a pass
    const int put_x = D == 128 ? lane & 7 : (lane >> 1) & 3;
    const int get_r = lane / kChunks, get_c = lane % kChunks;
    bool ok = true, joined = false;
    s = Seg{};
    s.b = -1;  // none yet
    for (uint32_t i = 0;;) {
      const bool whole = s.t0 == 0 && s.t1 == s.tiles;
      // A share's first segment that begins inside its unit leaves what the join
      // needs to know.
      if (!whole && s.t0 > 0 && tid == 0) {
        joined = true;
        const long long first = S.start[blockIdx.x] - s.t0, last = first + s.tiles - 1;
        JoinDesc d;
        d.c0 = seq_of(S.start, ctas, first);
        d.c1 = seq_of(S.start, ctas, last);
        d.tok0 = s.tok0;
        d.ntok = s.ntok;
        d.kvh = s.h;
        P.join[blockIdx.x] = d;
      }
      const int live = s.ntok * P.G;             // live rows of the tile
      const bool dead = quarter * 32 >= live;    // none in this quarter
      const bool row_live = r < live;
      // Rows behind the live ones go with the last of them, so that a warp that has both
      // stays on one path (masked on their own they cost every tile a second one, half
      // as long again); nothing of them is written.
      const int t_seen = min(t_row, s.ntok - 1);
      const int q_tok = s.j * P.TT + t_seen;     // new token of this row
      const int lim = P.tree ? s.keys - 1 : min(s.ctx + q_tok, s.keys - 1);
      const uint32_t* tree_row =
          P.tree ? P.tree + (int64_t)(s.tok0 + t_seen) * P.tree_words : nullptr;

      float m_run = -INFINITY, l_run = 0.f;
      for (int t = s.t0; ok && t < s.t1; ++t, ++g) {
        const int sb = (int)(g % kSBufs);
        ok = warp_wait(&bar_s_full[sb], (g / kSBufs) & 1u, kSite);
        if (!ok) break;
        // Values behind the sequence's last key may be anything: zeros, so that the
        // products with their zero probabilities vanish.  These warps do not follow
        // v_full's phases in turn, so they make sure first that the phase before
        // V(g)'s is over: O += P(g-2) V, which consumed that stage's last values.
        // (S(g) is there, so O += P(g-3) V and all before it are complete, and the
        // phase of o_done waited for is its barrier's current or latest one.)
        const int behind = s.have - t * kTile;
        if (behind < kTile) {
          const int st = g & 1;
          if (g >= (uint32_t)kStages) ok = warp_wait(&bar_o_done[g & 1], ((g >> 1) - 1u) & 1u, kSite);
          ok = ok && warp_wait(&bar_v_full[st], (g >> 1) & 1u, kSite);
          if (!ok) break;
          unsigned char* const v = smem + L::v0 + st * L::kKV;
          for (int x = behind * (D / 8) + tid; x < kTile * (D / 8); x += kSoftmaxWarps * 32)
            *reinterpret_cast<uint4*>(v + swz_chunk_offset(x / (D / 8), x % (D / 8), kTile)) =
                make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        if (dead) {
          warp_arrive(&bar_p_full[sb]);
          continue;
        }
        tc_fence_after();
        const uint32_t scol = tmem + lane_off + sb * kTile + part * 64;
        uint32_t sc[2][32];
        tmem_ld32x2(scol, scol + 32, sc[0], sc[1]);

        const int cbase = t * kTile + part * 64;
        float mp[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mp[k] = -INFINITY;
        if (cbase + 63 <= (P.tree ? min(lim, s.ctx - 1) : lim)) {
#pragma unroll
          for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
            for (int x = 0; x < 32; x += 2)
              mp[(x >> 1) & 7] = fmax3(mp[(x >> 1) & 7], __uint_as_float(sc[c2][x]),
                                       __uint_as_float(sc[c2][x + 1]));
        } else {
#pragma unroll
          for (int c2 = 0; c2 < 2; ++c2) {
            // Bit x: key cbase + 32 c2 + x is visible.
            const int k0 = cbase + c2 * 32, left = lim + 1 - k0;
            uint32_t bits = left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1u);
            if (tree_row) bits &= tree_bits(tree_row, P.tree_words, k0 - s.ctx);
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const float v = (bits >> x) & 1u ? __uint_as_float(sc[c2][x]) : -INFINITY;
              sc[c2][x] = __float_as_uint(v);
              mp[x & 7] = fmaxf(mp[x & 7], v);
            }
          }
        }
        float mt = fmaxf(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])),
                         fmaxf(fmaxf(mp[4], mp[5]), fmaxf(mp[6], mp[7]))) * sl2;
        s_max[g & 1][part][r] = mt;
        ok = group_sync(&bar_quad[quarter], quad_uses, kSite);
        if (!ok) break;
        mt = fmaxf(mt, s_max[g & 1][part ^ 1][r]);

        float alpha = 1.f;
        bool rescale_o = false;
        const float m_new = fmaxf(m_run, mt);
        if (m_new > m_run + kRescaleThreshold) {
          alpha = ex2(m_run - m_new);
          l_run *= alpha;
          m_run = m_new;
          rescale_o = t > s.t0;
        }
        const float m_use = (m_run == -INFINITY) ? 0.f : m_run;
        uint32_t pk[32];
        const uint64_t sl2x2 = f32x2(sl2, sl2), negm2 = f32x2(-m_use, -m_use);
        uint64_t rp[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) rp[k] = f32x2(0.f, 0.f);
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            float x0, x1;
            unpack_f32x2(fma_f32x2(f32x2(__uint_as_float(sc[c2][x]), __uint_as_float(sc[c2][x + 1])),
                                   sl2x2, negm2),
                         x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            // The sum takes P in fp32, the product with V in bf16, as in the training forward
            // (the tensor cores have tf32 at half the rate, and fp32 not at all): an output's
            // error of 2.3e-3, relative and in norm, against 1.7e-3 by its own rounding alone.
            rp[(x >> 1) & 3] = add_f32x2(rp[(x >> 1) & 3], f32x2(p0, p1));
            pk[(c2 * 32 + x) >> 1] = pack_bf16(p0, p1);
          }
        float ra, rb;
        unpack_f32x2(add_f32x2(add_f32x2(rp[0], rp[1]), add_f32x2(rp[2], rp[3])), ra, rb);
        l_run += ra + rb;

        if (__any_sync(0xffffffffu, rescale_o)) {
          ok = warp_wait(&bar_o_done[(g - 1u) & 1u], ((g - 1u) >> 1) & 1u, kSite);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ocol = tmem + lane_off + kColO + part * DH;
#pragma unroll
          for (int c2 = 0; c2 < DH / 32; ++c2) {
            uint32_t o[32];
            tmem_ld32(ocol + c2 * 32, o);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
            tmem_st32(ocol + c2 * 32, o);
          }
          tmem_st_wait();
        }
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
          uint32_t pp[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) pp[c] = pk[c2 * 16 + c];
          tmem_st16(scol + c2 * 16, pp);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&bar_p_full[sb]);
      }
      if (!ok) break;
      const bool more = walk.next(P, S, ctas, nx);  // while the last product runs
      if (s.b < 0) {
        if (!more) break;
        s = nx;
        continue;
      }

      // ------------------------------------------------------- results ----
      // In a unit without keys there is no query buffer, nor a part to leave.
      float o[DH];
      unsigned char* const turn = smem + L::q + (int)(i & 1) * L::kQ + warp * (L::kQ / kSoftmaxWarps);
      uint64_t* const q_empty = &bar_q_empty[i & 1];
      if (s.tiles == 0) {
#pragma unroll
        for (int x = 0; x < DH; ++x) o[x] = 0.f;
      } else {
        ok = warp_wait(&bar_o_final, n_final & 1u, kSite);
        ++n_final;
        ++i;
        if (!ok) break;
        if (dead) {
          warp_arrive(q_empty);
          if (!more) break;
          s = nx;
          continue;
        }
        tc_fence_after();
        const uint32_t ocol = tmem + lane_off + kColO + part * DH;
#pragma unroll
        for (int c2 = 0; c2 < DH / 32; ++c2) {
          uint32_t u[32];
          tmem_ld32(ocol + c2 * 32, u);
#pragma unroll
          for (int x = 0; x < 32; ++x) o[c2 * 32 + x] = __uint_as_float(u[x]);
        }
        tc_fence_before();
        s_sum[i & 1][part][r] = l_run;
        ok = group_sync(&bar_quad[quarter], quad_uses, kSite);
        if (!ok) break;
        l_run += s_sum[i & 1][part ^ 1][r];
      }
      // A row that saw nothing has l = 0 and O = 0.
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      const float lse2 = l_run == 0.f ? -INFINITY : m_run + log2f(l_run);
      // Rows go out through shared memory: stored by the lanes that hold them, each
      // store would touch 32 rows, and the eight warps' took 2.9 thousand cycles a unit,
      // 1.9 now.  Chunks are placed by an exclusive or, so that neither side meets a bank
      // twice.
      auto put = [&](int c, const uint4& v) {
        *reinterpret_cast<uint4*>(turn + (lane * kChunks + (c ^ put_x)) * 16) = v;
      };
      auto get = [&](int row) {
        const int x = D == 128 ? row & 7 : (row >> 1) & 3;
        return *reinterpret_cast<const uint4*>(turn + (row * kChunks + (get_c ^ x)) * 16);
      };
      const int64_t first = (int64_t)s.tok0 * P.H + s.h * P.G;
      if (s.tiles == 0) {
        if (row_live) {
          uint4* dst = reinterpret_cast<uint4*>(P.out + (first + row_off) * D + part * DH);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) dst[c] = make_uint4(0, 0, 0, 0);
        }
      } else if (whole) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          put(c, make_uint4(pack_bf16(o[c * 8 + 0] * inv, o[c * 8 + 1] * inv),
                            pack_bf16(o[c * 8 + 2] * inv, o[c * 8 + 3] * inv),
                            pack_bf16(o[c * 8 + 4] * inv, o[c * 8 + 5] * inv),
                            pack_bf16(o[c * 8 + 6] * inv, o[c * 8 + 7] * inv)));
        __syncwarp();
        uint4 v[kChunks];
#pragma unroll
        for (int k = 0; k < kChunks; ++k) v[k] = get(k * kRowsAt + get_r);
        fence_proxy_async_smem();  // the next queries come here by TMA
        warp_arrive(q_empty);
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          const int row = k * kRowsAt + get_r;
          const int off = __shfl_sync(0xffffffffu, row_off, row);
          if (quarter * 32 + row < live)
            *reinterpret_cast<uint4*>(P.out + (first + off) * D + part * DH + get_c * 8) = v[k];
        }
      } else {
        float* slot = P.part + (int64_t)(2 * blockIdx.x + (s.t0 > 0 ? 0 : 1)) * P.slot;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          constexpr int kHalf = DH / 2;
          __syncwarp();
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const float* v = o + half * kHalf + c * 4;
            put(c, make_uint4(__float_as_uint(v[0] * inv), __float_as_uint(v[1] * inv),
                              __float_as_uint(v[2] * inv), __float_as_uint(v[3] * inv)));
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            const int row = k * kRowsAt + get_r;
            if (quarter * 32 + row < live)
              *reinterpret_cast<uint4*>(slot + (int64_t)(quarter * 32 + row) * D + part * DH +
                                        half * kHalf + get_c * 4) = get(row);
          }
        }
        fence_proxy_async_smem();
        warp_arrive(q_empty);
        if (row_live && part == 0) slot[(int64_t)P.slot_rows * D + r] = lse2;
      }
      if ((whole || s.tiles == 0) && row_live && part == 0 && P.lse)
        P.lse[first + row_off] = lse2 * kLn2;
      if (!more) break;
      s = nx;
    }
    if (tid == 0 && !joined) P.join[blockIdx.x].c0 = -1;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the units cut by share borders.  The CTAs c0 + 1 .. c1 whose
// shares begin inside a unit divide its rows among their blocks.  A warp takes four rows
// at a time, so that their loads are in flight together; with few rows, several warps
// share a row's parts.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_attn_join(const __grid_constant__ Params P) {
  constexpr int E = D / 32, kW = kJoinThreads / 32, R = 4;
  __shared__ __align__(16) float s_o[kW][D];
  __shared__ float s_l[kW];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinDesc d = P.join[blockIdx.x];
  if (d.c0 < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = d.c1 - d.c0 + 1, rows = d.ntok * P.G;
  const int share = parts - 1, first = (int)blockIdx.x - d.c0 - 1;
  const int mine = first < rows ? (rows - first + share - 1) / share : 0;
  if (mine == 0) return;

  // Part p's slot.
  auto slot = [&](int p) { return P.part + (int64_t)(2 * (d.c0 + p) + (p == 0 ? 1 : 0)) * P.slot; };
  using V = typename std::conditional<E == 4, float4, float2>::type;
  struct Sum {
    float acc[E], l, m;
  };
  auto add = [&](Sum& s, float lse, const V& v) {
    if (lse != -INFINITY) {
      const float mn = fmaxf(s.m, lse), a = ex2(s.m - mn), w = ex2(lse - mn);
      s.l = s.l * a + w;
      const float* x = reinterpret_cast<const float*>(&v);
#pragma unroll
      for (int e = 0; e < E; ++e) s.acc[e] = fmaf(w, x[e], s.acc[e] * a);
      s.m = mn;
    }
  };
  auto write = [&](const Sum& s, int r) {
    const int t = r / P.G, g = r - t * P.G;
    const int64_t at = (int64_t)(d.tok0 + t) * P.H + d.kvh * P.G + g;
    const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
    uint32_t* dst = reinterpret_cast<uint32_t*>(P.out + at * D) + lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16(s.acc[e] * inv, s.acc[e + 1] * inv);
    if (P.lse && lane == 0) P.lse[at] = s.l == 0.f ? -INFINITY : (s.m + log2f(s.l)) * kLn2;
  };

  int wpr = 1;  // warps per row
  while (wpr * 2 * mine <= kW && wpr * 2 <= parts) wpr *= 2;
  if (wpr == 1) {
    for (int x0 = warp * R; x0 < mine; x0 += kW * R) {
      Sum s[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int e = 0; e < E; ++e) s[i].acc[e] = 0.f;
        s[i].l = 0.f;
        s[i].m = -INFINITY;
      }
      for (int p = 0; p < parts; ++p) {
        const float* src = slot(p);
        float lse[R];
        V v[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int r = first + min(x0 + i, mine - 1) * share;
          lse[i] = src[(int64_t)P.slot_rows * D + r];
          v[i] = reinterpret_cast<const V*>(src + (int64_t)r * D)[lane];
        }
#pragma unroll
        for (int i = 0; i < R; ++i) add(s[i], lse[i], v[i]);
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (x0 + i < mine) write(s[i], first + (x0 + i) * share);
    }
    return;
  }
  // One row to each wpr warps.
  const int sub = warp % wpr, x = warp / wpr, r = first + x * share;
  Sum s;
#pragma unroll
  for (int e = 0; e < E; ++e) s.acc[e] = 0.f;
  s.l = 0.f;
  s.m = -INFINITY;
  if (x < mine) {
#pragma unroll 4
    for (int p = sub; p < parts; p += wpr) {
      const float* src = slot(p);
      add(s, src[(int64_t)P.slot_rows * D + r], reinterpret_cast<const V*>(src + (int64_t)r * D)[lane]);
    }
  }
  const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = s.acc[e] * inv;
  if (lane == 0) s_l[warp] = s.l == 0.f ? -INFINITY : s.m + log2f(s.l);
  __syncthreads();
  if (sub == 0 && x < mine) {  // the row's warps, in order
#pragma unroll
    for (int e = 0; e < E; ++e) s.acc[e] = 0.f;
    s.l = 0.f;
    s.m = -INFINITY;
    for (int y = 0; y < wpr; ++y)
      add(s, s_l[warp + y], reinterpret_cast<const V*>(s_o[warp + y])[lane]);
    write(s, r);
  }
}

int slot_rows(int64_t N, int G) { return (int)std::min<int64_t>(N * G, kTile); }

// Floats of a partial result, each starting on a 128-byte line.
int64_t slot_floats(int rows, int D) { return ((int64_t)rows * (D + 1) + 31) / 32 * 32; }

constexpr size_t kJoinBytes = (kMaxCtas * sizeof(JoinDesc) + 255) / 256 * 256;

// A cache as a tensor map: elements, then keys, heads and pages by increasing
// stride; a box is `box` keys of one head.
cudaError_t encode_cache(CUtensorMap* map, const void* base, const PagesArgs& g, int box, int* place) {
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return cudaErrorNotSupported;
  struct Dim { int64_t stride; cuuint64_t size; int what; } d[3] = {
      {g.stride_tok, (cuuint64_t)1 << g.page_shift, 0},
      {g.stride_head, (cuuint64_t)g.H_kv, 1},
      {g.stride_page, (cuuint64_t)g.num_pages, 2}};
  std::stable_sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  cuuint64_t dims[4] = {(cuuint64_t)g.D, d[0].size, d[1].size, d[2].size};
  cuuint64_t strides[3];
  cuuint32_t boxes[4] = {(cuuint32_t)kColBlock, 1, 1, 1}, es[4] = {1, 1, 1, 1};
  for (int x = 0; x < 3; ++x) {
    strides[x] = (cuuint64_t)d[x].stride * 2;
    place[d[x].what] = x + 1;
    if (d[x].what == 0) boxes[x + 1] = (cuuint32_t)box;
  }
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                   boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The queries: elements, heads, rows; a box is a group's heads at TT rows.
cudaError_t encode_q(CUtensorMap* map, const PagedAttnArgs& a, int D, int G, int TT) {
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.H, (cuuint64_t)a.N};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.ld_q * 2};
  cuuint32_t box[3] = {(cuuint32_t)kColBlock, (cuuint32_t)G, (cuuint32_t)TT}, es[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch(const PagesArgs& pg, const PagedAttnArgs& a, cudaStream_t s) {
  Params P{};
  P.g = pg;
  P.tree = a.tree;
  P.tree_words = a.tree_words;
  P.out = static_cast<__nv_bfloat16*>(a.out);
  P.lse = a.lse;
  P.N = a.N;
  P.H = a.H;
  P.G = a.H / pg.H_kv;
  P.TT = std::min(kTile / P.G, a.N);
  P.slot_rows = slot_rows(a.N, P.G);
  P.slot = slot_floats(P.slot_rows, D);
  P.key_cap = pg.max_pages << pg.page_shift;
  P.scale_log2 = a.scale * kLog2e;
  P.inject = debug_inject();
  P.join = static_cast<JoinDesc*>(a.workspace);
  P.part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.workspace) + kJoinBytes);
  CUtensorMap tmQ, tmK, tmV;
  cudaError_t e;
  const int box = std::min(1 << pg.page_shift, kTile);
  int place[3];
  if ((e = bind_device_context()) != cudaSuccess) return e;
  if ((e = encode_q(&tmQ, a, D, P.G, P.TT)) != cudaSuccess) return e;
  if ((e = encode_cache(&tmK, pg.k, pg, box, place)) != cudaSuccess) return e;
  if ((e = encode_cache(&tmV, pg.v, pg, box, place)) != cudaSuccess) return e;
  P.d_tok = place[0];
  P.d_head = place[1];
  P.d_page = place[2];
  static std::atomic<uint64_t> raised{0};  // devices whose limit is raised, the first 64
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(raised.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(paged_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Smem<D>::alloc);
    if (e != cudaSuccess) return e;
    raised.fetch_or(bit, std::memory_order_relaxed);
  }
  const unsigned grid = (unsigned)std::min(sm_count(), kMaxCtas);
  prof_before(s, STT_KERNEL_PAGED_ATTN);
  // Both as programmatic dependents: this kernel's set-up overlaps the end of what came
  // before, the join's launch this kernel.
  cudaLaunchAttribute la[1];
  la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  la[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<D>::alloc;
  cfg.stream = s;
  cfg.attrs = la;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_attn_kernel<D>, P, tmQ, tmK, tmV);
  if (e == cudaSuccess) {
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, paged_attn_join<D>, P);
  }
  prof_after(s);
  return e;
}

}  // namespace

size_t paged_attn_workspace(int64_t N, int B, int H, int H_kv, int D) {
  (void)B;
  return kJoinBytes +
         (size_t)(2 * kMaxCtas * slot_floats(slot_rows(N, H / H_kv), D)) * sizeof(float);
}

cudaError_t paged_attn_launch(const PagesArgs& pg, const PagedAttnArgs& a, cudaStream_t s) {
  if (pg.D == 128) return launch<128>(pg, a, s);
  return launch<64>(pg, a, s);
}

STT_DEFINE_ERROR_ACCESSOR(paged_attn_error_word)
STT_DEFINE_BUDGET_SETTER(paged_attn_set_wait_budget)

}  // namespace stt
