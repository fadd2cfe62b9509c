// The writer of rows in the two formats, and rotary positions.
//
// UlaCache summary (paper-daily.com), section 4: the KV cache is held in FP8.
//
// Quantisation, per scale block (128 latent channels, or one head's keys or
// values in a block of tokens): scale = max(amax / 448, 2^-126), code =
// e4m3(x / scale), both divisions correctly rounded in 32 bits and the code
// rounded to nearest even. An infinity takes the largest code and a NaN the NaN
// code; neither enters amax.
//
// Rotary positions: pair i of R / 2 turns by the angle pos[axis(i)] x
// theta^(-2i / R). The angle is taken in turns in 64 bits (a far position times
// a rounded frequency would lose the angle in 32), reduced to an eighth of a
// turn either way, and its sine and cosine come from their series in 32 bits
// (truncation below 2^-27 there).
//
// All three kernels read and write every byte once and are bound by HBM, or for
// a decode step's few rows by the launch.
#include <algorithm>

#include "row_format.h"

namespace ula {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__bf16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }

// N consecutive elements from p as fp32, as one vector where p allows it.
template <typename T, int N, bool ALIGNED>
__device__ __forceinline__ void load_f32(const T* p, float* x) {
  typedef T vec __attribute__((ext_vector_type(N)));
  if constexpr (ALIGNED) {
    const vec v = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(p[i]);
  }
}

__device__ __forceinline__ float scale_of(float amax) { return fmaxf(amax / kE4m3Max, 0x1p-126f); }

// x / scale clamped to e4m3's range; a NaN stays one.
__device__ __forceinline__ float to_e4m3_range(float x, float scale) {
  const float y = x / scale;
  return y != y ? y : fminf(fmaxf(y, -kE4m3Max), kE4m3Max);
}

// cos and sin of 2 pi x turns.
__device__ __forceinline__ float2 cos_sin_turns(double turns) {
  turns -= rint(turns);                        // [-1/2, 1/2]
  const double q = rint(4.0 * turns);          // quarter turns
  const float x = (float)((turns - 0.25 * q) * 6.283185307179586476925);   // [-pi/4, pi/4]
  const float y = x * x;
  const float s = x + x * y * (-1.0f / 6 + y * (1.0f / 120 + y * (-1.0f / 5040 + y * (1.0f / 362880))));
  const float c = 1.0f + y * (-0.5f + y * (1.0f / 24 + y * (-1.0f / 720 + y * (1.0f / 40320 + y * (-1.0f / 3628800)))));
  switch ((int)q & 3) {
    case 0: return make_float2(c, s);
    case 1: return make_float2(-s, c);
    case 2: return make_float2(-c, -s);
    default: return make_float2(s, -c);
  }
}

// Turn of pair i at a token whose positions start at pos.
__device__ __forceinline__ float2 rotary_of(const RotaryDev& r, const int32_t* __restrict__ pos, int i) {
  const int axis = i < r.end0 ? 0 : (i < r.end1 ? 1 : 2);
  return cos_sin_turns((double)pos[axis] * r.turns[i]);
}

// Latent rows: one wave per row, lane i channels 8 i .. 8 i + 7 (16 lanes share
// a scale), then lane i < 32 rotary pair i.
template <typename T, bool ALIGNED>
__global__ __launch_bounds__(256) void k_pack_latent(PackDev a, RotaryDev rot) {
  const int lane = lane_id();
  const int row = blockIdx.x * 4 + threadIdx.x / kWave;
  if (row >= a.n * a.layers) return;
  const int entry = row / a.layers, layer = row % a.layers;
  const T* latent = static_cast<const T*>(a.a) + entry * a.a_stride[0] + layer * a.a_stride[1];
  const T* rope = static_cast<const T*>(a.b) + entry * a.b_stride[0] + layer * a.b_stride[1];
  uint8_t* out = a.rows + (size_t)row * kLatentRow;
  float x[8];
  load_f32<T, 8, ALIGNED>(latent + 8 * lane, x);
  const int pair = lane % 32;
  const int at0 = rot.interleaved ? 2 * pair : pair, at1 = rot.interleaved ? 2 * pair + 1 : pair + kRope / 2;
  const float r0 = to_f32(rope[at0]), r1 = to_f32(rope[at1]);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, finite_abs(x[i]));
#pragma unroll
  for (int d = 1; d < 16; d *= 2) amax = fmaxf(amax, __shfl_xor(amax, d, kWave));
  const float scale = scale_of(amax);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_e4m3_range(x[i], scale);
  reinterpret_cast<uint2*>(out)[lane] = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
  if (lane % 16 == 0) *reinterpret_cast<float*>(out + kLatentScaleAt + lane / 16 * 4) = scale;
  if (lane < 32) {
    float y0 = r0, y1 = r1;
    if (a.positions) {
      const float2 cs = rotary_of(rot, a.positions + (size_t)entry * rot.axes, pair);
      y0 = r0 * cs.x - r1 * cs.y;
      y1 = r0 * cs.y + r1 * cs.x;
    }
    __bf16* ro = reinterpret_cast<__bf16*>(out + kRopeAt);
    ro[at0] = (__bf16)y0;
    ro[at1] = (__bf16)y1;
  }
}

// Heads rows: one wave per (row, KV head, keys or values): the block's values,
// keys turned, go to LDS in 32 bits while amax is taken, then to codes.
constexpr int kBlockMost = 2048;   // block_tokens x head_dim of a row of at most 4096 bytes

template <typename T>
__global__ __launch_bounds__(kWave) void k_pack_heads(PackDev a, RotaryDev rot) {
  __shared__ float s[kBlockMost];
  const int lane = lane_id();
  const int per_row = 2 * a.kv_heads;
  const int row = blockIdx.x / per_row;
  const int h = blockIdx.x % per_row % a.kv_heads;
  const bool value = blockIdx.x % per_row >= a.kv_heads;
  const int entry = row / a.layers, layer = row % a.layers;
  const int block = a.block_tokens, dim = a.head_dim, half = dim / 2;
  const long long* st = value ? a.b_stride : a.a_stride;
  const T* src = static_cast<const T*>(value ? a.b : a.a) + entry * st[0] + layer * st[1] + h * st[3];
  const int count = a.count ? min(max(a.count[entry], 0), block) : block;
  float amax = 0.0f;
  for (int e = lane; e < block * half; e += kWave) {
    const int tok = e / half, i = e % half;
    const int at0 = rot.interleaved ? 2 * i : i, at1 = rot.interleaved ? 2 * i + 1 : i + half;
    float y0 = 0.0f, y1 = 0.0f;
    if (tok < count) {
      const float x0 = to_f32(src[tok * st[2] + at0]), x1 = to_f32(src[tok * st[2] + at1]);
      y0 = x0;
      y1 = x1;
      if (!value && a.positions) {
        const float2 cs = rotary_of(rot, a.positions + ((size_t)entry * block + tok) * rot.axes, i);
        y0 = x0 * cs.x - x1 * cs.y;
        y1 = x0 * cs.y + x1 * cs.x;
      }
    }
    s[tok * dim + at0] = y0;
    s[tok * dim + at1] = y1;
    amax = fmaxf(amax, fmaxf(finite_abs(y0), finite_abs(y1)));
  }
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) amax = fmaxf(amax, __shfl_xor(amax, d, kWave));
  __syncthreads();
  const float scale = scale_of(amax);
  uint8_t* out = a.rows + (size_t)row * a.row_bytes;
  const int part = block * dim;
  uint32_t* codes = reinterpret_cast<uint32_t*>(out + (value ? a.kv_heads * part : 0) + h * part);
  for (int e = lane; e < part / 4; e += kWave) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(&s[4 * e]);
    codes[e] = e4m3x4(to_e4m3_range(x[0], scale), to_e4m3_range(x[1], scale), to_e4m3_range(x[2], scale),
                      to_e4m3_range(x[3], scale));
  }
  uint8_t* tail = out + 2 * a.kv_heads * part;
  if (lane == 0) reinterpret_cast<float*>(tail)[(value ? a.kv_heads : 0) + h] = scale;
  if (h == 0 && !value) {   // the token count and the zeros behind it
    int32_t* words = reinterpret_cast<int32_t*>(tail + 8 * a.kv_heads);
    const int n = (int)(out + a.row_bytes - reinterpret_cast<uint8_t*>(words)) / 4;
    if (lane < n) words[lane] = lane == 0 ? count : 0;
  }
}

// Rotary positions of [n][heads][dim] tensors. A workgroup takes `tokens` tokens
// and a range of heads: the tokens' sines and cosines once into LDS, then V
// pairs per lane. In place is fine: a lane reads its pairs before it writes them.
template <typename T, int V>
__global__ __launch_bounds__(256) void k_rotate(RotateDev a, RotaryDev rot) {
  extern __shared__ float2 s_cs[];   // [tokens][pairs]
  const int pairs = a.dim / 2;
  const int head_parts = (a.heads + a.heads_per_block - 1) / a.heads_per_block;
  const int tok0 = blockIdx.x / head_parts * a.tokens_per_block;
  const int head0 = blockIdx.x % head_parts * a.heads_per_block;
  const int tokens = min(a.tokens_per_block, a.n - tok0);
  const int heads = min(a.heads_per_block, a.heads - head0);
  for (int e = threadIdx.x; e < tokens * pairs; e += 256) {
    const int t = e / pairs;
    float2 cs = rotary_of(rot, a.positions + (size_t)(tok0 + t) * rot.axes, e % pairs);
    if (a.inverse) cs.y = -cs.y;
    s_cs[e] = cs;
  }
  __syncthreads();
  const int units = pairs / V;
  typedef T vec __attribute__((ext_vector_type(V)));
  typedef T vec2 __attribute__((ext_vector_type(2 * V)));
  for (int e = threadIdx.x; e < tokens * heads * units; e += 256) {
    const int i = e % units * V;
    const int h = e / units % heads, t = e / units / heads;
    const T* x = static_cast<const T*>(a.x) + (tok0 + t) * a.x_stride[0] + (head0 + h) * a.x_stride[1];
    T* y = static_cast<T*>(a.out) + (tok0 + t) * a.out_stride[0] + (head0 + h) * a.out_stride[1];
    const float2* cs = s_cs + t * pairs + i;
    if (rot.interleaved) {
      vec2 v;
      if constexpr (V > 1) v = *reinterpret_cast<const vec2*>(x + 2 * i);
      else v = vec2{x[2 * i], x[2 * i + 1]};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float p = to_f32(v[2 * j]), q = to_f32(v[2 * j + 1]);
        v[2 * j] = (T)(p * cs[j].x - q * cs[j].y);
        v[2 * j + 1] = (T)(p * cs[j].y + q * cs[j].x);
      }
      if constexpr (V > 1) {
        *reinterpret_cast<vec2*>(y + 2 * i) = v;
      } else {
        y[2 * i] = v[0];
        y[2 * i + 1] = v[1];
      }
    } else {
      vec v, w;
      if constexpr (V > 1) {
        v = *reinterpret_cast<const vec*>(x + i);
        w = *reinterpret_cast<const vec*>(x + i + pairs);
      } else {
        v = vec{x[i]};
        w = vec{x[i + pairs]};
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float p = to_f32(v[j]), q = to_f32(w[j]);
        v[j] = (T)(p * cs[j].x - q * cs[j].y);
        w[j] = (T)(p * cs[j].y + q * cs[j].x);
      }
      if constexpr (V > 1) {
        *reinterpret_cast<vec*>(y + i) = v;
        *reinterpret_cast<vec*>(y + i + pairs) = w;
      } else {
        y[i] = v[0];
        y[i + pairs] = w[0];
      }
    }
  }
}

template <typename T>
static hipError_t pack_of(const PackDev& a, const RotaryDev& rot, hipStream_t s) {
  const int rows = a.n * a.layers;
  if (a.latent) {
    const int blocks = (rows + 3) / 4;
    if (a.aligned) k_pack_latent<T, true><<<blocks, 256, 0, s>>>(a, rot);
    else k_pack_latent<T, false><<<blocks, 256, 0, s>>>(a, rot);
  } else {
    k_pack_heads<T><<<rows * 2 * a.kv_heads, kWave, 0, s>>>(a, rot);
  }
  return hipGetLastError();
}

hipError_t launch_pack(const PackDev& a, const RotaryDev& rot, int type, hipStream_t s) {
  if (type == ULA_BF16) return pack_of<__bf16>(a, rot, s);
  if (type == ULA_FP16) return pack_of<_Float16>(a, rot, s);
  return pack_of<float>(a, rot, s);
}

template <typename T>
static hipError_t rotate_of(RotateDev a, const RotaryDev& rot, hipStream_t s) {
  constexpr int V = 4;
  const int pairs = a.dim / 2;
  const int units = a.aligned ? pairs / V : pairs;
  // about 512 units per workgroup: two per lane, enough workgroups for a decode step
  constexpr int kUnits = 512;
  a.heads_per_block = std::max(1, std::min(a.heads, kUnits / units));
  a.tokens_per_block = std::max(1, std::min(a.n, std::min(kUnits / (units * a.heads_per_block), 4096 / pairs)));
  const long long blocks = (long long)((a.n + a.tokens_per_block - 1) / a.tokens_per_block) *
                           ((a.heads + a.heads_per_block - 1) / a.heads_per_block);
  const size_t lds = (size_t)a.tokens_per_block * pairs * sizeof(float2);
  if (a.aligned) k_rotate<T, V><<<(unsigned)blocks, 256, lds, s>>>(a, rot);
  else k_rotate<T, 1><<<(unsigned)blocks, 256, lds, s>>>(a, rot);
  return hipGetLastError();
}

hipError_t launch_rotate(const RotateDev& a, const RotaryDev& rot, int type, hipStream_t s) {
  if (type == ULA_BF16) return rotate_of<__bf16>(a, rot, s);
  if (type == ULA_FP16) return rotate_of<_Float16>(a, rot, s);
  return rotate_of<float>(a, rot, s);
}

}  // namespace ula
