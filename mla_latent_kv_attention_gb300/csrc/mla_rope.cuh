// mla_rope.cuh -- the rotation of RoPE pairs, shared by the query rotation and the cache write.
#pragma once

#include <math.h>
#include <stdint.h>

#include "../../include/mla.h"

namespace mla {

// amplitude * (cos, sin) of a pair's angle at a position. The phase is position * turns modulo
// 2^64 in units of 2^-64 turns. The product is exact, so the phase is off by the position times
// what `turns` is off by (2^-65 turns, and float64's 2^-50 of the frequency: 1.4e-10 turns at
// position 10^6 for the fastest pair), where a float32 angle keeps only 24 bits of a number of
// radians that grows with the position. The top 32 bits, as a signed number of half turns in
// [-1, 1), go through one rounding to float32 (at most 2^-25 half turns, 9e-8 rad) into sincospif.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t turns, int64_t position, float amplitude) {
  const int32_t half_turns = (int32_t)(uint32_t)((turns * (uint64_t)position) >> 32);
  float s, c;
  sincospif((float)half_turns * 0x1p-31f, &s, &c);
  return make_float2(amplitude * c, amplitude * s);
}

// (a, b) turned by (cos, sin).
__device__ __forceinline__ float2 rope_turn(float a, float b, float2 cs) {
  return make_float2(fmaf(a, cs.x, -b * cs.y), fmaf(a, cs.y, b * cs.x));
}

}  // namespace mla
