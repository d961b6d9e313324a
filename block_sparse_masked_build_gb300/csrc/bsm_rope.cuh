// Cosines and sines of a row's position angles, shared by the kernels that
// rotate rows (bsm_rope.cu, the cache's append).
#pragma once

#include <cstdint>

#include "bsm_internal.h"

namespace bsm {

// cos and sin of position * step turns.  The product modulo 2^64 drops whole
// turns exactly; its upper half, to the nearest quarter turn, leaves an angle in
// [-pi/4, pi/4), a + low with 2 pi / 2^32 as a sum of two f32, so that what it
// is off by is the integer's rounding, 2^-24 of at most pi / 4.  The Taylor series
// are summed to a^9 and a^8 (they leave out at most (pi/4)^11 / 11! < 2^-29 and
// (pi/4)^10 / 10! < 2^-25) and moved by low.  With the sums' own roundings that
// is less than 2^-23.  (__sincosf, within 2^-20, moved enough keys to the
// neighbouring e4m3 value to be seen in a cache's error.)
__device__ __forceinline__ void turn_of(uint64_t step, int32_t position,
                                        float* c, float* s) {
  const uint64_t turns =
      static_cast<uint64_t>(static_cast<int64_t>(position)) * step;
  const uint32_t t = static_cast<uint32_t>(turns >> 32);
  const uint32_t q = t + 0x20000000u;  // the nearest quarter in its two top bits
  const float r = static_cast<float>(static_cast<int32_t>(t - (q & 0xc0000000u)));
  constexpr float kTurn = 1.462918119976564e-09f, kTurnLow = -4.070940267922164e-17f;
  const float a = r * kTurn;
  const float low = fmaf(r, kTurnLow, fmaf(r, kTurn, -a));
  const float z = a * a;
  float sn = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  sn = fmaf(sn, z, 1.f / 120.f);
  sn = fmaf(sn, z, -1.f / 6.f);
  float cs = fmaf(z, 1.f / 40320.f, -1.f / 720.f);
  cs = fmaf(cs, z, 1.f / 24.f);
  cs = fmaf(cs, z, -0.5f);
  // + low cos a and - low sin a, to the terms that count; the small parts first
  sn = a + fmaf(sn * z, a, fmaf(-0.5f * z, low, low));
  cs = 1.f + fmaf(cs, z, -low * a);
  const bool odd = q & 0x40000000u;  // a quarter turn exchanges them
  const float x = odd ? sn : cs, y = odd ? cs : sn;
  *c = __uint_as_float(__float_as_uint(x) ^
                       ((q + 0x40000000u) & 0x80000000u));
  *s = __uint_as_float(__float_as_uint(y) ^ (q & 0x80000000u));
}

// Where a lane's 16 elements of a row lie, and which frequencies turn them: the
// two elements of a pair lie in one lane.
struct LanePart {
  int at0, at1;  // its first eight elements, and the other eight
  int freq;      // frequencies freq .. freq + 7; -1: not turned
};

// Halves: lane l of dim / 16 holds elements 8 l .. and dim / 2 + 8 l ..;
// neighbouring pairs, and what is not turned: 16 elements in a row.
__device__ __forceinline__ LanePart lane_part(int l, int dim, bool halves) {
  LanePart p;
  const bool turned = l < dim / 16;
  p.freq = turned ? 8 * l : -1;
  p.at0 = halves && turned ? 8 * l : 16 * l;
  p.at1 = halves && turned ? dim / 2 + 8 * l : 16 * l + 8;
  return p;
}

// Of N frequencies from f on, whose steps the caller holds; pos: the token's
// first axis.
template <int N>
__device__ __forceinline__ void turns_of(const bsm_rope& rope,
                                         const uint64_t* steps, int f,
                                         const int32_t* pos, int64_t axis_stride,
                                         int32_t index, float* c, float* s) {
  if (pos == nullptr || rope.axes == 1) {
    const int32_t at = pos == nullptr ? index : *pos;
#pragma unroll
    for (int i = 0; i < N; ++i) turn_of(steps[i], at, &c[i], &s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      turn_of(steps[i], pos[rope.axis[f + i] * axis_stride], &c[i], &s[i]);
  }
}

// Eight elements of a norm's weight from `at` on; ones where there is none.
__device__ __forceinline__ void weights_of(const void* w, int bf16, int at,
                                           float* out) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = 1.f;
  } else if (bf16) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      out[i] = __uint_as_float(
          static_cast<uint32_t>(static_cast<const uint16_t*>(w)[at + i]) << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = static_cast<const float*>(w)[at + i];
  }
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

}  // namespace bsm
