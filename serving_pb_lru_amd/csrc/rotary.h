// Rotary positions: the sines of a pair's angle and the turn, shared by the row
// writer, the turn and the norms of queries and keys.
#pragma once

#include "row_format.h"

namespace ula {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__bf16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }

// cos and sin of 2 pi x turns.
__device__ __forceinline__ float2 cos_sin_turns(double turns) {
  turns -= rint(turns);                        // [-1/2, 1/2]
  const double q = rint(4.0 * turns);          // quarter turns
  const float x = (float)(__builtin_fma(q, -0.25, turns) * 6.283185307179586476925);   // [-pi/4, pi/4]
  const float y = x * x;
  // every fused step spelled out, so that all kernels get the same bits
  auto f = [](float a, float b, float c) { return __builtin_fmaf(a, b, c); };
  const float s = f(x * y, f(y, f(y, f(y, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
  const float c = f(y, f(y, f(y, f(y, f(y, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  switch ((int)q & 3) {
    case 0: return make_float2(c, s);
    case 1: return make_float2(-s, c);
    case 2: return make_float2(-c, -s);
    default: return make_float2(s, -c);
  }
}

// The pair (p, q) turned by (cos, sin), with the rounding steps spelled out: the
// compiler's own fusing differs from kernel to kernel, and strides must not change
// bits. (The empty assembly keeps a following conversion to fp16 out of the fma:
// the fused form rounds once, the others twice, which differs in one of 10^5.)
__device__ __forceinline__ float2 turned(float p, float q, float2 cs) {
  float a = __builtin_fmaf(p, cs.x, -(q * cs.y)), b = __builtin_fmaf(p, cs.y, q * cs.x);
  asm("" : "+v"(a), "+v"(b));
  return make_float2(a, b);
}

// Turn of pair i at a token whose positions start at pos.
__device__ __forceinline__ float2 rotary_of(const RotaryDev& r, const int32_t* __restrict__ pos, int i) {
  const int axis = i < r.end0 ? 0 : (i < r.end1 ? 1 : 2);
  return cos_sin_turns((double)pos[axis] * r.turns[i]);
}

}  // namespace ula
