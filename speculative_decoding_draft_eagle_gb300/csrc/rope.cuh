// rope.cuh -- pieces shared by the rotation kernels (qkv_rope.cu): angles, and what a
// lane holds of a head.
//
// A head takes D / 8 lanes, a lane 8 of its elements, and both elements of each of
// its pairs: lane c has elements 8 c .. 8 c + 7 for interleaved pairs and for elements
// that are not rotated, and 4 c .. 4 c + 3 with R / 2 + 4 c .. for halves.  A lane has
// four pairs either way, whose cosines and sines it reads from its warp's table, and
// nothing of the rotation crosses lanes.  Elements are kept as four pairs of floats
// (the instructions that take two at a time halve what the kernels issue, which bound
// them before).
#pragma once

#include "../../include/stt.h"
#include "attn_common.cuh"

namespace stt {

// Radians per position as turns per position, modulo one turn, in 64-bit fixed
// point.  The mantissa times 2/pi (0.A2F9836E4E44152A in hexadecimal, scaled by
// 2^64) is a 117-bit product; in integers, because fp64 arithmetic is slow here.
// A position times this wraps modulo a turn by itself, and is off by at most
// |position| 2^-64 turns besides the fp64 frequency's own rounding.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int ex = (int)((bits >> 52) & 0x7ffu);
  const uint64_t m = (bits & 0xfffffffffffffull) | (ex ? 1ull << 52 : 0ull);
  const uint64_t c = 0xA2F9836E4E44152Aull;
  const uint64_t lo = m * c, hi = __umul64hi(m, c);
  // f = m 2^(ex - 1075) radians; over 2 pi = times c 2^-66; in units of 2^-64.
  const int s = (ex ? ex : 1) - 1075 - 2;
  uint64_t t;
  if (s >= 0)
    t = s < 64 ? lo << s : 0;
  else if (s > -64)
    t = (hi << (64 + s)) | (lo >> -s);
  else
    t = s > -128 ? hi >> (-s - 64) : 0;
  return (bits >> 63) ? 0 - t : t;
}

// cos and sin of `pos` times the frequency: the top 32 bits of the turn
// fraction as a signed number of half turns in [-1, 1).
__device__ __forceinline__ void turn_sincos(uint64_t frac, int pos, float& c, float& s) {
  const uint64_t t = frac * (uint64_t)(int64_t)pos;
  sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f, &s, &c);
}

// Eight elements as four pairs.
struct Eight {
  uint64_t p[4];
};
__device__ __forceinline__ uint64_t pair_of(uint32_t v) { return f32x2(bf16lo(v), bf16hi(v)); }
__device__ __forceinline__ uint64_t swapped(uint64_t v) {
  float a, b;
  unpack_f32x2(v, a, b);
  return f32x2(b, a);
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
  float a, b;
  unpack_f32x2(v, a, b);
  return pack_bf16(a, b);
}
__device__ __forceinline__ float sum_pair(uint64_t v) {
  float a, b;
  unpack_f32x2(v, a, b);
  return a + b;
}

// A warp's table of its token's cosines and sines (amplitude applied), in shared
// memory: each pair's angle is taken once.
template <int D>
struct RopeTable {
  float cos[D / 2], sin[D / 2];
};

// What one lane knows of its elements for the whole kernel.
template <int D, bool INTER>
struct RopeLane {
  static constexpr int kLanes = D / 8;         // lanes per head
  static constexpr int kHeads = 32 / kLanes;   // heads per warp step
  static constexpr int kAngles = D / 64;       // pairs whose angles a lane takes
  int chunk, sub;   // lane of the head, head of the warp step
  int off0, off1;   // first of its two runs of four elements
  bool rot;         // rotated
  uint64_t frac[kAngles];

  __device__ __forceinline__ void init(const double* freq, int R) {
    const int lane = threadIdx.x & 31;
    chunk = lane % kLanes;
    sub = lane / kLanes;
    rot = chunk * 8 < R;
    off0 = !INTER && rot ? chunk * 4 : chunk * 8;
    off1 = !INTER && rot ? R / 2 + chunk * 4 : chunk * 8 + 4;
#pragma unroll
    for (int i = 0; i < kAngles; ++i)
      frac[i] = lane + 32 * i < R / 2 ? turn_fraction(__ldg(freq + lane + 32 * i)) : 0;
  }

  // Fills the warp's table for a position.
  __device__ __forceinline__ void fill(RopeTable<D>& t, int pos, float amplitude) const {
    const int lane = threadIdx.x & 31;
    __syncwarp();  // the last token's readers
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
      float c, s;
      turn_sincos(frac[i], pos, c, s);
      t.cos[lane + 32 * i] = c * amplitude;
      t.sin[lane + 32 * i] = s * amplitude;
    }
    __syncwarp();
  }

  // Factors of a rotation: y = x a + x' b, x' the other element of each one's pair.
  // Elements that are not rotated: a = 1, and no x'.
  __device__ __forceinline__ void factors(const RopeTable<D>& t, Eight& a, Eight& b) const {
    if (!rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a.p[i] = f32x2(1.f, 1.f);
        b.p[i] = 0;
      }
      return;
    }
    const float4 c = *reinterpret_cast<const float4*>(t.cos + chunk * 4);
    const float4 s = *reinterpret_cast<const float4*>(t.sin + chunk * 4);
    if (INTER) {
      a.p[0] = f32x2(c.x, c.x); a.p[1] = f32x2(c.y, c.y);
      a.p[2] = f32x2(c.z, c.z); a.p[3] = f32x2(c.w, c.w);
      b.p[0] = f32x2(-s.x, s.x); b.p[1] = f32x2(-s.y, s.y);
      b.p[2] = f32x2(-s.z, s.z); b.p[3] = f32x2(-s.w, s.w);
    } else {
      a.p[0] = a.p[2] = f32x2(c.x, c.y);
      a.p[1] = a.p[3] = f32x2(c.z, c.w);
      b.p[0] = f32x2(-s.x, -s.y); b.p[1] = f32x2(-s.z, -s.w);
      b.p[2] = f32x2(s.x, s.y); b.p[3] = f32x2(s.z, s.w);
    }
  }
  // The other element of each pair.
  __device__ __forceinline__ static uint64_t other(const Eight& x, int i) {
    return INTER ? swapped(x.p[i]) : x.p[i ^ 2];
  }
  // x a + x' b (unrotated: x a; not 0 times an infinity).
  __device__ __forceinline__ Eight turn(const Eight& x, const Eight& a, const Eight& b) const {
    Eight y;
    if (rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y.p[i] = fma_f32x2(x.p[i], a.p[i], mul_f32x2(other(x, i), b.p[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) y.p[i] = mul_f32x2(x.p[i], a.p[i]);
    }
    return y;
  }

  // This lane's elements of a bf16 head at p, as loaded; and its elements.
  __device__ __forceinline__ uint4 load(const __nv_bfloat16* p) const {
    if (INTER) return __ldg(reinterpret_cast<const uint4*>(p + off0));
    const uint2 lo = __ldg(reinterpret_cast<const uint2*>(p + off0));
    const uint2 hi = __ldg(reinterpret_cast<const uint2*>(p + off1));
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  __device__ __forceinline__ static Eight get(const uint4& v) {
    return Eight{{pair_of(v.x), pair_of(v.y), pair_of(v.z), pair_of(v.w)}};
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, const Eight& y) const {
    const uint4 v = make_uint4(pack_pair(y.p[0]), pack_pair(y.p[1]), pack_pair(y.p[2]),
                               pack_pair(y.p[3]));
    if (INTER) {
      *reinterpret_cast<uint4*>(p + off0) = v;
    } else {
      *reinterpret_cast<uint2*>(p + off0) = make_uint2(v.x, v.y);
      *reinterpret_cast<uint2*>(p + off1) = make_uint2(v.z, v.w);
    }
  }
  // A weight's elements (ones without a weight).
  __device__ __forceinline__ Eight weight(const __nv_bfloat16* w) const {
    if (w) return get(load(w));
    return Eight{{f32x2(1.f, 1.f), f32x2(1.f, 1.f), f32x2(1.f, 1.f), f32x2(1.f, 1.f)}};
  }

  // Sum over the lanes of a head.
  __device__ __forceinline__ static float head_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
};

}  // namespace stt
