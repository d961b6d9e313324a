// Cosines and sines of a row's position angles, shared by the kernels that
// rotate rows (bsm_rope.cu, the cache's append).
#pragma once

#include <cstdint>

#include "bsm_internal.h"

namespace bsm {

// cos and sin of position * step turns.  The product modulo 2^64 drops whole
// turns exactly; its upper half is a signed fraction of a turn in [-1/2, 1/2),
// whose angle __sincosf takes within its bound for [-pi, pi] (2^-21.2
// absolute); with the roundings of the angle itself (3 of 2^-25 of at most pi)
// that is less than 2^-20, eleven bits below bf16's half step of a result of
// size 1.
__device__ __forceinline__ void turn_of(uint64_t step, int32_t position,
                                        float* c, float* s) {
  // (the product's upper half in 32 bits: a negative position is 2^32 less
  // than its bits)
  const uint32_t p = static_cast<uint32_t>(position);
  const uint32_t lo = static_cast<uint32_t>(step);
  const uint32_t turns = __umulhi(p, lo) + p * static_cast<uint32_t>(step >> 32) -
                         (position < 0 ? lo : 0u);
  const float a = static_cast<float>(static_cast<int32_t>(turns)) *
                  1.4629180792671596e-9f;  // 2 pi / 2^32
  __sincosf(a, s, c);
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
