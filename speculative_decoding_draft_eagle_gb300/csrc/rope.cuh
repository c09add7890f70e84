// rope.cuh -- pieces shared by the rotation kernels (qkv_rope.cu):
// angles, and the per-lane tables of the fused norm + rotation.
//
// A lane holds 8 consecutive elements of a head (one 16-byte load), so a head
// takes D / 8 lanes.  With x the raw elements, r = (mean x^2 + eps)^(-1/2) (1
// without a weight), and x' the other element of each one's pair,
//     y[e] = r (x[e] a[e] + x'[e] b[e]),
// a = amplitude w cos, b = -+ amplitude w' sin for rotated elements, a = w,
// b = 0 for the rest: two multiply-adds an element once the token's tables are
// made, and the tables serve every head of the token.  x' is in the lane itself
// for interleaved pairs, and in the lane R / 16 further (or back) for halves.
#pragma once

#include "../../include/stt.h"
#include "internal.h"
#include "ptx.cuh"

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

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ uint4 shfl4(const uint4& v, int src) {
  return make_uint4(__shfl_sync(0xffffffffu, v.x, src), __shfl_sync(0xffffffffu, v.y, src),
                    __shfl_sync(0xffffffffu, v.z, src), __shfl_sync(0xffffffffu, v.w, src));
}

// What one lane knows of its chunk for the whole kernel.
template <int D, bool INTER>
struct RopeLane {
  static constexpr int kLanes = D / 8;         // lanes per head
  static constexpr int kHeads = 32 / kLanes;   // heads per warp step
  static constexpr int kAngles = INTER ? 4 : 8;
  int chunk, sub, partner;  // chunk of the head, head of the warp step, lane of x'
  bool rot, first;          // rotated; first half (of halves)
  uint64_t frac[kAngles];

  __device__ __forceinline__ void init(const double* freq, int R) {
    const int lane = threadIdx.x & 31;
    chunk = lane % kLanes;
    sub = lane / kLanes;
    rot = chunk * 8 < R;
    const int half = R / 16;
    first = INTER || chunk < half;
    partner = lane;
    if (!INTER && rot) partner = first ? lane + half : lane - half;
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
      const int pair = INTER ? chunk * 4 + i : (first ? chunk : chunk - half) * 8 + i;
      frac[i] = rot ? turn_fraction(__ldg(freq + pair)) : 0;
    }
  }

  // cos and +-sin of this lane's elements at a position (amplitude applied); the
  // sign is that of x' in y.  Unrotated elements: 1 and 0.
  __device__ __forceinline__ void angles(int pos, float amplitude, float (&c)[8],
                                         float (&s)[8]) const {
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
      float ci = 1.f, si = 0.f;
      if (rot) {
        turn_sincos(frac[i], pos, ci, si);
        ci *= amplitude;
        si *= amplitude;
      }
      if (INTER) {
        c[2 * i] = c[2 * i + 1] = ci;
        s[2 * i] = -si;
        s[2 * i + 1] = si;
      } else {
        c[i] = ci;
        s[i] = first ? -si : si;
      }
    }
  }

  // This chunk of a weight (ones without one), and of its pair elements.
  __device__ __forceinline__ void weight(const __nv_bfloat16* w, float (&own)[8]) const {
    if (w) {
      unpack8(__ldg(reinterpret_cast<const uint4*>(w) + chunk), own);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) own[e] = 1.f;
    }
  }
  __device__ __forceinline__ void other(const float (&x)[8], float (&o)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = INTER ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], partner);
  }

  // a = w cos, b = w' sin.
  __device__ __forceinline__ void tables(const __nv_bfloat16* w, const float (&c)[8],
                                         const float (&s)[8], float (&a)[8], float (&b)[8]) const {
    float own[8], oth[8];
    weight(w, own);
    other(own, oth);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] = own[e] * c[e];
      b[e] = oth[e] * s[e];
    }
  }

  // Sum over the lanes of a head.
  __device__ __forceinline__ static float head_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }

  // y of one 16-byte chunk x; every lane of the warp calls it.
  __device__ __forceinline__ uint4 apply(const uint4& raw, bool norm, float eps,
                                         const float (&a)[8], const float (&b)[8]) const {
    float x[8], o[8], y[8];
    unpack8(raw, x);
    if constexpr (INTER) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = x[e ^ 1];
    } else {
      unpack8(shfl4(raw, partner), o);
    }
    if (!rot) {  // b is 0 there, but 0 times an infinity is not
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = 0.f;
    }
    float r = 1.f;
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      r = rsqrtf(head_sum(ss) * (1.f / D) + eps);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = r * fmaf(x[e], a[e], o[e] * b[e]);
    return pack8(y);
  }
};

}  // namespace stt
