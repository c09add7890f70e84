// qkv_rope.cu -- per-head norm and position rotation of queries and keys: from
// the fused QKV projection's rows to the attention's layout (training), to the
// queries and a paged KV cache (serving), and the training form's gradient.
//
// All three are one pass over memory: a warp takes a token (or a part of its
// heads), fills its table of cosines and sines, and streams the token's heads, 32 / (D
// / 8) of them a step, four steps' loads in flight.  HBM bounds them where there are
// many tokens: 8192 tokens of 32 + 16 heads of 128 take 37 us forward (5.5 TB/s, 0.81 of
// the copy rate; 38.5 with norms), 2 x 4096 tokens of 64 + 16 heads 110 us backward with
// norms and fp32 gradients (5.95 TB/s, 0.88), 93 with bf16 gradients (5.2 TB/s, 0.77).
// What moved them there was fewer instructions, not more bytes in flight: 185 a step
// became about 80 when both elements of a pair came to one lane and arithmetic went in
// pairs of floats (166 to 113 us backward), while a ring of bulk copies ahead of the
// warps took 166 to 276 us, and tiles of eight tokens with the warps dividing the heads
// 147.  Few tokens are bound by the launch and a chain of dependent loads (8 us for 64
// sequences of 8 tokens).
#include <algorithm>
#include <type_traits>

#include "rope.cuh"

namespace stt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 3;     // forward; by registers
constexpr int kBwdBlocksPerSm = 2;  // gradient
constexpr int kUnroll = 4;  // steps whose loads are in flight together

struct FwdP {
  RopeArgs r;
  PagesArgs pg;  // append only
  const __nv_bfloat16* qkv;
  int64_t ld;
  const int32_t* positions;
  __nv_bfloat16 *q, *k, *v;
  uint32_t N, items, parts, steps_per_part;
  int S, H, H_kv;
};

// Where one token's heads go.
struct Dest {
  __nv_bfloat16 *q, *k, *v;
  int64_t q_head, kv_head;
  bool kv;  // the key and value rows are written
  int pos;
};

__device__ __forceinline__ Dest train_dest(const FwdP& P, uint32_t t, int D) {
  Dest d;
  const uint32_t b = t / (uint32_t)P.S, s = t - b * (uint32_t)P.S;
  d.q_head = d.kv_head = (int64_t)P.S * D;
  d.q = P.q + ((int64_t)b * P.H * P.S + s) * D;
  d.k = P.k + ((int64_t)b * P.H_kv * P.S + s) * D;
  d.v = P.v + ((int64_t)b * P.H_kv * P.S + s) * D;
  d.kv = true;
  d.pos = P.positions ? __ldg(P.positions + t) : (int)s;
  return d;
}

// False for a row behind the last sequence.
__device__ __forceinline__ bool append_dest(const FwdP& P, uint32_t t, int D, Dest& d) {
  const PagesArgs& G = P.pg;
  const int lane = threadIdx.x & 31;
  // The row's sequence: how many sequences end at or before it (warp-wide count).
  int b = 0;
  for (int j = 0; j < G.B; j += 32) {
    const bool ends = j + lane < G.B && __ldg(G.cu_q + 1 + j + lane) <= (int)t;
    b += __popc(__ballot_sync(0xffffffffu, ends));
  }
  if (b >= G.B) return false;
  const int key = __ldg(G.seq_lens + b) - __ldg(G.cu_q + b + 1) + (int)t;
  d.q = P.q + (int64_t)t * P.H * D;
  d.q_head = D;
  d.kv_head = G.stride_head;
  d.pos = P.positions ? __ldg(P.positions + t) : key;
  d.kv = false;
  const int slot = key >> G.page_shift;
  if (key >= 0 && slot < G.max_pages) {
    const int page = __ldg(G.table + (int64_t)b * G.max_pages + slot);
    if (page >= 0 && page < G.num_pages) {
      d.kv = true;
      const int64_t at = (int64_t)page * G.stride_page +
                         (int64_t)(key & ((1 << G.page_shift) - 1)) * G.stride_tok;
      d.k = static_cast<__nv_bfloat16*>(G.k) + at;
      d.v = static_cast<__nv_bfloat16*>(G.v) + at;
    }
  }
  if (!d.kv && lane == 0) record_error(STT_DEVERR_PAGE);
  return true;
}

template <int D, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    qkv_rope_kernel(const __grid_constant__ FwdP P) {
  using L = RopeLane<D, INTER>;
  __shared__ __align__(16) RopeTable<D> s_table[kWarps];
  RopeTable<D>& table = s_table[threadIdx.x >> 5];
  L L_;
  L_.init(P.r.freq, P.r.R);
  const int nq = (P.H + L::kHeads - 1) / L::kHeads, nk = (P.H_kv + L::kHeads - 1) / L::kHeads;
  const uint32_t warp = blockIdx.x * kWarps + (threadIdx.x >> 5), warps = gridDim.x * kWarps;
  const int lane = threadIdx.x & 31;

  for (uint32_t item = warp; item < P.items; item += warps) {
    const uint32_t t = item / P.parts, part = item - t * P.parts;
    // Where the row goes takes a few dependent loads; the row is fetched meanwhile.
    for (int line = lane; line < (int)P.steps_per_part * 4; line += 32) {
      const int64_t at = ((int64_t)part * P.steps_per_part * 4 + line) * 64;
      if (at < (int64_t)(P.H + 2 * P.H_kv) * D)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(P.qkv + (int64_t)t * P.ld + at));
    }
    Dest d;
    if constexpr (APPEND) {
      if (!append_dest(P, t, D, d)) continue;
    } else {
      d = train_dest(P, t, D);
    }
    const __nv_bfloat16* row = P.qkv + (int64_t)t * P.ld;
    const int lo = (int)(part * P.steps_per_part), hi = lo + (int)P.steps_per_part;
    if (P.r.R > 0) L_.fill(table, d.pos, P.r.amplitude);

    // Steps [lo, hi) of one kind of head: `first` its first step, `n` its heads.
    auto run = [&](int first, int steps, int n, int head0, const __nv_bfloat16* w, auto rotate,
                   __nv_bfloat16* dst, int64_t dst_head) {
      constexpr bool kRotate = decltype(rotate)::value;
      const int from = max(lo, first) - first, to = min(hi, first + steps) - first;
      if (from >= to) return;
      Eight a, b;
      if constexpr (kRotate) {
        L_.factors(table, a, b);
        if (w) {
          const Eight own = L_.weight(w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a.p[i] = mul_f32x2(a.p[i], own.p[i]);
            b.p[i] = mul_f32x2(b.p[i], L::other(own, i));
          }
        }
      }
      const __nv_bfloat16* src = row + (head0 + from * L::kHeads + L_.sub) * D;
      dst += (int64_t)(from * L::kHeads + L_.sub) * dst_head;
      const int64_t dst_step = dst_head * L::kHeads;
      // kUnroll steps from u0; `check`: there may be fewer, or fewer heads.
      auto group = [&](int u0, auto check) {
        constexpr bool kCheck = decltype(check)::value;
        auto live = [&](int u) {
          return !kCheck || (u0 + u < to && (u0 + u) * L::kHeads + L_.sub < n);
        };
        uint4 raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          raw[u] = make_uint4(0, 0, 0, 0);
          if (live(u)) {
            const __nv_bfloat16* p = src + u * L::kHeads * D;
            raw[u] = kRotate ? L_.load(p) : __ldg(reinterpret_cast<const uint4*>(p) + L_.chunk);
          }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (kCheck && u0 + u >= to) break;
          if constexpr (kRotate) {
            const Eight x = L::get(raw[u]);
            Eight y = L_.turn(x, a, b);
            if (w) {
              uint64_t ss = mul_f32x2(x.p[0], x.p[0]);
#pragma unroll
              for (int i = 1; i < 4; ++i) ss = fma_f32x2(x.p[i], x.p[i], ss);
              const float r = rsqrtf(L::head_sum(sum_pair(ss)) * (1.f / D) + P.r.eps);
#pragma unroll
              for (int i = 0; i < 4; ++i) y.p[i] = mul_f32x2(y.p[i], f32x2(r, r));
            }
            if (live(u)) L_.store(dst, y);
          } else {
            if (live(u)) reinterpret_cast<uint4*>(dst)[L_.chunk] = raw[u];
          }
          dst += dst_step;
        }
        src += kUnroll * L::kHeads * D;
      };
      int u0 = from;
      for (; u0 + kUnroll <= to && (u0 + kUnroll) * L::kHeads <= n; u0 += kUnroll)
        group(u0, std::false_type{});
      for (; u0 < to; u0 += kUnroll) group(u0, std::true_type{});
    };
    run(0, nq, P.H, 0, P.r.w_q, std::true_type{}, d.q, d.q_head);
    if (d.kv) {
      run(nq, nk, P.H_kv, P.H, P.r.w_k, std::true_type{}, d.k, d.kv_head);
      run(nq + nk, nk, P.H_kv, P.H + P.H_kv, nullptr, std::false_type{}, d.v, d.kv_head);
    }
  }
}

// Splits each token's steps into the fewest parts that give the resident warps even
// shares (within 7 %; 8192 tokens on 3648 warps would leave a quarter of them idle in
// the last round), down to `least` steps a part; the evenest split where none does.
void split_items(int64_t N, int steps, int64_t warps, int least, uint32_t* parts, uint32_t* per) {
  double best = 0;
  for (int p = 1; p <= (steps + least - 1) / least; ++p) {
    const int64_t each = (steps + p - 1) / p, n = (steps + each - 1) / each;
    const int64_t rounds = (N * n + warps - 1) / warps;
    // Steps there are over steps the slowest warp's rounds have room for.
    const double even = (double)(N * steps) / (double)(rounds * warps * each);
    if (even > best) {
      best = even;
      *per = (uint32_t)each;
      *parts = (uint32_t)n;
      if (even > 0.93) break;
    }
  }
}

template <bool APPEND>
cudaError_t launch_fwd(FwdP& P, int D, cudaStream_t s) {
  if (P.N == 0) return cudaSuccess;
  const int heads = 32 / (D / 8);
  const int steps = (P.H + heads - 1) / heads + 2 * ((P.H_kv + heads - 1) / heads);
  const int64_t blocks_max = (int64_t)sm_count() * kBlocksPerSm;
  split_items(P.N, steps, blocks_max * kWarps, kUnroll, &P.parts, &P.steps_per_part);
  const int64_t items = (int64_t)P.N * P.parts;
  if (items > 0x7fffffffll) return cudaErrorNotSupported;
  P.items = (uint32_t)items;
  const unsigned grid = (unsigned)std::min<int64_t>((items + kWarps - 1) / kWarps, blocks_max);
  const bool inter = P.r.inter;
  prof_before(s, APPEND ? STT_KERNEL_KV_APPEND : STT_KERNEL_QKV_ROPE);
  if (D == 128) {
    if (inter) qkv_rope_kernel<128, true, APPEND><<<grid, kThreads, 0, s>>>(P);
    else qkv_rope_kernel<128, false, APPEND><<<grid, kThreads, 0, s>>>(P);
  } else {
    if (inter) qkv_rope_kernel<64, true, APPEND><<<grid, kThreads, 0, s>>>(P);
    else qkv_rope_kernel<64, false, APPEND><<<grid, kThreads, 0, s>>>(P);
  }
  prof_after(s);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- gradient --
struct BwdP {
  RopeArgs r;
  const void *dq, *dk, *dv;  // T
  const __nv_bfloat16* qkv;
  int64_t ld, ld_d;
  const int32_t* positions;
  __nv_bfloat16* dqkv;
  float* partial;  // [grid][2][D], with a weight
  uint32_t items, parts, steps_per_part;
  int S, H, H_kv;
};

// A lane's elements of a gradient head as loaded.
template <class T>
struct RawGrad {
  uint4 v[sizeof(T) / 2];
  template <class L>
  __device__ __forceinline__ void load(const L& l, const float* p) {
    v[0] = __ldg(reinterpret_cast<const uint4*>(p + l.off0));
    v[1] = __ldg(reinterpret_cast<const uint4*>(p + l.off1));
  }
  template <class L>
  __device__ __forceinline__ void load(const L& l, const __nv_bfloat16* p) {
    v[0] = l.load(p);
  }
  __device__ __forceinline__ Eight get() const {
    if constexpr (sizeof(T) == 2)
      return Eight{{pair_of(v[0].x), pair_of(v[0].y), pair_of(v[0].z), pair_of(v[0].w)}};
    else
      return Eight{{f32x2(__uint_as_float(v[0].x), __uint_as_float(v[0].y)),
                    f32x2(__uint_as_float(v[0].z), __uint_as_float(v[0].w)),
                    f32x2(__uint_as_float(v[1].x), __uint_as_float(v[1].y)),
                    f32x2(__uint_as_float(v[1].z), __uint_as_float(v[1].w))}};
  }
};

constexpr int kBwdUnroll = 4;

template <int D, bool INTER, class T>
__global__ void __launch_bounds__(kThreads, kBwdBlocksPerSm)
    qkv_rope_bwd_kernel(const __grid_constant__ BwdP P) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  using L = RopeLane<D, INTER>;
  __shared__ __align__(16) float s_dw[kWarps][2][32][8];  // each lane's own, by kind
  __shared__ __align__(16) RopeTable<D> s_table[kWarps];
  L L_;
  L_.init(P.r.freq, P.r.R);
  const int nq = (P.H + L::kHeads - 1) / L::kHeads, nk = (P.H_kv + L::kHeads - 1) / L::kHeads;
  const int wib = threadIdx.x >> 5, lane = threadIdx.x & 31;
  RopeTable<D>& table = s_table[wib];
  const uint32_t warp = blockIdx.x * kWarps + wib, warps = gridDim.x * kWarps;
#pragma unroll
  for (int e = 0; e < 8; ++e) s_dw[wib][0][lane][e] = s_dw[wib][1][lane][e] = 0.f;

  for (uint32_t item = warp; item < P.items; item += warps) {
    const uint32_t t = item / P.parts, part = item - t * P.parts;
    const uint32_t bi = t / (uint32_t)P.S, si = t - bi * (uint32_t)P.S;
    const int pos = P.positions ? __ldg(P.positions + t) : (int)si;
    const int lo = (int)(part * P.steps_per_part), hi = lo + (int)P.steps_per_part;
    if (P.r.R > 0) L_.fill(table, pos, P.r.amplitude);
    __nv_bfloat16* drow = P.dqkv + (int64_t)t * P.ld_d;
    const __nv_bfloat16* xrow = P.qkv + (int64_t)t * P.ld;

    auto run = [&](int first, int steps, int n, int head0, const void* dsrc,
                   const __nv_bfloat16* w, auto rotate, int kind) {
      constexpr bool kRotate = decltype(rotate)::value;
      const int from = max(lo, first) - first, to = min(hi, first + steps) - first;
      if (from >= to) return;
      const int64_t step = (int64_t)L::kHeads * P.S * D;
      const T* dy = static_cast<const T*>(dsrc) +
                    (((int64_t)bi * n + from * L::kHeads + L_.sub) * P.S + si) * D;
      const int col = (head0 + from * L::kHeads + L_.sub) * D;
      const __nv_bfloat16* xp = xrow + col;
      __nv_bfloat16* dst = drow + col;
      Eight a, b, wv, dw;
      if constexpr (kRotate) {
        L_.factors(table, a, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) b.p[i] ^= 0x8000000080000000ull;  // the transpose
        if (w) wv = L_.weight(w);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) dw.p[i] = 0;
      auto group = [&](int u0, auto check) {
        constexpr bool kCheck = decltype(check)::value;
        auto live = [&](int u) {
          return !kCheck || (u0 + u < to && (u0 + u) * L::kHeads + L_.sub < n);
        };
        RawGrad<T> raw[kBwdUnroll];
        uint4 xr[kBwdUnroll];
#pragma unroll
        for (int u = 0; u < kBwdUnroll; ++u) {
          raw[u] = RawGrad<T>{};
          xr[u] = make_uint4(0, 0, 0, 0);
          if (live(u)) {
            raw[u].load(L_, dy);
            if (kRotate && w) xr[u] = L_.load(xp + u * L::kHeads * D);
          }
          dy += step;
        }
#pragma unroll
        for (int u = 0; u < kBwdUnroll; ++u) {
          if (kCheck && u0 + u >= to) break;
          Eight g = raw[u].get();
          if constexpr (kRotate) {
            g = L_.turn(g, a, b);
            if (w) {
              // dx = r u w - x r^2 (r sum(u w x) / D): both sums go over the lanes together.
              const Eight x = L::get(xr[u]);
              Eight gw;
              uint64_t s2 = 0, d2 = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                gw.p[i] = mul_f32x2(g.p[i], wv.p[i]);
                s2 = fma_f32x2(x.p[i], x.p[i], s2);
                d2 = fma_f32x2(gw.p[i], x.p[i], d2);
              }
              float ss = sum_pair(s2), sd = sum_pair(d2);
#pragma unroll
              for (int m = L::kLanes / 2; m > 0; m >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, m);
                sd += __shfl_xor_sync(0xffffffffu, sd, m);
              }
              const float r = rsqrtf(ss * (1.f / D) + P.r.eps), k = -(r * r * (r * sd) * (1.f / D));
              const uint64_t r2 = f32x2(r, r), k2 = f32x2(k, k);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                dw.p[i] = fma_f32x2(mul_f32x2(g.p[i], r2), x.p[i], dw.p[i]);
                g.p[i] = fma_f32x2(x.p[i], k2, mul_f32x2(gw.p[i], r2));
              }
            }
          }
          if (live(u)) L_.store(dst + u * L::kHeads * D, g);
        }
        xp += kBwdUnroll * L::kHeads * D;
        dst += kBwdUnroll * L::kHeads * D;
      };
      int u0 = from;
      for (; u0 + kBwdUnroll <= to && (u0 + kBwdUnroll) * L::kHeads <= n; u0 += kBwdUnroll)
        group(u0, std::false_type{});
      for (; u0 < to; u0 += kBwdUnroll) group(u0, std::true_type{});
      if (kRotate && w) {
        uint64_t* acc = reinterpret_cast<uint64_t*>(s_dw[wib][kind][lane]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = add_f32x2(acc[i], dw.p[i]);
      }
    };
    run(0, nq, P.H, 0, P.dq, P.r.w_q, std::true_type{}, 0);
    run(nq, nk, P.H_kv, P.H, P.dk, P.r.w_k, std::true_type{}, 1);
    run(nq + nk, nk, P.H_kv, P.H + P.H_kv, P.dv, nullptr, std::false_type{}, 0);
  }

  if (P.r.w_q || P.r.w_k) {
    // The block's warps and the heads of one warp step, in fixed order.
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
      const int kind = x / D, e = x % D, half = P.r.R / 2;
      int c = e / 8, slot = e % 8;  // the lane of the head that holds element e, and where
      if (!INTER && e < P.r.R) {
        c = (e < half ? e : e - half) / 4;
        slot = e % 4 + (e < half ? 0 : 4);
      }
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int h = 0; h < L::kHeads; ++h) v += s_dw[w][kind][h * L::kLanes + c][slot];
      P.partial[(int64_t)blockIdx.x * 2 * D + x] = v;
    }
  }
}

// dw = sum of the blocks' partials, in a fixed order: block (kind, 32 elements); warp w
// adds rows w, w + 32, ..., then the 32 sums of an element are added.
__global__ void __launch_bounds__(1024) qkv_rope_dw_kernel(const float* partial, int rows, int D,
                                                           float* dw_q, float* dw_k) {
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, x = blockIdx.y * 32 + lane;
  float* const dst = blockIdx.x ? dw_k : dw_q;
  if (!dst) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float v = 0.f;
#pragma unroll 8
  for (int r = warp; r < rows; r += 32) v += partial[((int64_t)r * 2 + blockIdx.x) * D + x];
  sm[warp][lane] = v;
  __syncthreads();
  v = sm[lane][warp];  // warp w: element w's sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) dst[blockIdx.y * 32 + warp] = v;
}

template <int D, class T>
void launch_bwd(const BwdP& P, unsigned grid, cudaStream_t s) {
  if (P.r.inter) qkv_rope_bwd_kernel<D, true, T><<<grid, kThreads, 0, s>>>(P);
  else qkv_rope_bwd_kernel<D, false, T><<<grid, kThreads, 0, s>>>(P);
}

}  // namespace

cudaError_t qkv_rope_launch(const RopeArgs& r, const void* qkv, int64_t ld,
                            const int32_t* positions, int B, int S, int H, int H_kv, int D, void* q,
                            void* k, void* v, cudaStream_t s) {
  FwdP P{};
  P.r = r;
  P.qkv = static_cast<const __nv_bfloat16*>(qkv);
  P.ld = ld;
  P.positions = positions;
  P.q = static_cast<__nv_bfloat16*>(q);
  P.k = static_cast<__nv_bfloat16*>(k);
  P.v = static_cast<__nv_bfloat16*>(v);
  P.N = (uint32_t)((int64_t)B * S);
  P.S = S;
  P.H = H;
  P.H_kv = H_kv;
  return launch_fwd<false>(P, D, s);
}

cudaError_t kv_append_launch(const RopeArgs& r, const PagesArgs& pg, const void* qkv, int64_t ld,
                             const int32_t* positions, int64_t N, int H, void* q, cudaStream_t s) {
  FwdP P{};
  P.r = r;
  P.pg = pg;
  P.qkv = static_cast<const __nv_bfloat16*>(qkv);
  P.ld = ld;
  P.positions = positions;
  P.q = static_cast<__nv_bfloat16*>(q);
  P.N = (uint32_t)N;
  P.S = 1;
  P.H = H;
  P.H_kv = pg.H_kv;
  return launch_fwd<true>(P, pg.D, s);
}

size_t qkv_rope_bwd_workspace(int D) { return (size_t)kRopeBwdMaxGrid * 2 * D * sizeof(float); }

cudaError_t qkv_rope_bwd_launch(const RopeArgs& r, const void* dq, const void* dk, const void* dv,
                                const void* qkv, int64_t ld, const int32_t* positions, int B,
                                int S, int H, int H_kv, int D, bool bf16, void* dqkv, int64_t ld_d,
                                float* dw_q, float* dw_k, void* workspace, cudaStream_t s) {
  BwdP P{};
  P.r = r;
  P.dq = dq;
  P.dk = dk;
  P.dv = dv;
  P.qkv = static_cast<const __nv_bfloat16*>(qkv);
  P.ld = ld;
  P.ld_d = ld_d;
  P.positions = positions;
  P.dqkv = static_cast<__nv_bfloat16*>(dqkv);
  P.partial = static_cast<float*>(workspace);
  P.S = S > 0 ? S : 1;
  P.H = H;
  P.H_kv = H_kv;
  const int64_t N = (int64_t)B * S;
  const int heads = 32 / (D / 8);
  const int steps = (H + heads - 1) / heads + 2 * ((H_kv + heads - 1) / heads);
  const int64_t blocks_max = std::min<int64_t>((int64_t)sm_count() * kBwdBlocksPerSm, kRopeBwdMaxGrid);
  split_items(N, steps, blocks_max * kWarps, kBwdUnroll, &P.parts, &P.steps_per_part);
  if (N == 0) P.parts = P.steps_per_part = 1;
  const int64_t items = N * P.parts;
  if (items > 0x7fffffffll) return cudaErrorNotSupported;
  P.items = (uint32_t)items;
  const unsigned grid = (unsigned)std::min<int64_t>((items + kWarps - 1) / kWarps, blocks_max);
  prof_before(s, STT_KERNEL_QKV_ROPE_BWD);
  if (grid > 0) {
    if (D == 128) {
      if (bf16) launch_bwd<128, __nv_bfloat16>(P, grid, s);
      else launch_bwd<128, float>(P, grid, s);
    } else {
      if (bf16) launch_bwd<64, __nv_bfloat16>(P, grid, s);
      else launch_bwd<64, float>(P, grid, s);
    }
  }
  // No tokens: the weights' gradients are zero.
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && (dw_q || dw_k)) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, (unsigned)(D / 32), 1);
    cfg.blockDim = dim3(1024, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute la[1];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = la;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, qkv_rope_dw_kernel, (const float*)P.partial, (int)grid, D, dw_q, dw_k);
  }
  prof_after(s);
  return e;
}

STT_DEFINE_ERROR_ACCESSOR(qkv_rope_error_word)

}  // namespace stt
