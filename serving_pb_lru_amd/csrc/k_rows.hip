// The writer of rows in the two formats, and rotary positions.
//
// UlaCache summary (paper-daily.com), section 4: the KV cache is held in FP8.
//
// Quantisation, per scale block (128 latent channels, or one head's keys or
// values in a block of tokens): scale = max(amax / 448, 2^-126), code =
// e4m3(x / scale), both quotients in 32 bits and the code rounded to nearest
// even. An infinity takes the largest code and a NaN the NaN
// code; neither enters amax.
//
// Rotary positions: pair i of R / 2 turns by the angle pos[axis(i)] x
// theta^(-2i / R). The angle is taken in turns in 64 bits (a far position times
// a rounded frequency would lose the angle in 32), reduced to an eighth of a
// turn either way, and its sine and cosine come from their series in 32 bits
// (truncation below 2^-27 there).
//
// All three kernels read and write every byte once. The writer of latent rows and
// the turn are bound by HBM, the writer of heads rows by its vector instructions,
// and all by the launch for a decode step's few rows.
#include <algorithm>
#include <type_traits>

#include "rotary.h"
#include "row_format.h"

namespace ula {

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

// x / b by b's correctly rounded reciprocal and one correction: off by less than
// 2^-46 of the quotient before its own rounding, given that neither the product
// nor the remainder leaves the normal range.
__device__ __forceinline__ float divide_by(float x, float b, float inv_b) {
  const float q = x * inv_b;
  return __builtin_fmaf(__builtin_fmaf(-q, b, x), inv_b, q);
}

// The largest of 16 lanes' values, in all of them.
__device__ __forceinline__ float max_of_16(float x) {
  auto rotated = [](float v, auto n) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x120 + n.value, 0xF, 0xF, true));
  };
  x = fmaxf(x, rotated(x, std::integral_constant<int, 8>{}));
  x = fmaxf(x, rotated(x, std::integral_constant<int, 4>{}));
  x = fmaxf(x, rotated(x, std::integral_constant<int, 2>{}));
  return fmaxf(x, rotated(x, std::integral_constant<int, 1>{}));
}

// Latent rows: a wave takes two rows, lane i channels 8 i .. 8 i + 7 of either (16
// lanes share a scale) and rotary pair i % 32 of row i / 32. Instructions, not
// bytes, would bound it with a division per channel: hence one reciprocal per
// scale where every value is finite and far enough from the least ones (65536 rows, 118 MB read and
// written: 36 us with a row a wave and IEEE divisions, 22 us so).
constexpr int kPackRows = 2;

template <typename T, bool ALIGNED>
__global__ __launch_bounds__(256) void k_pack_latent(PackDev a, RotaryDev rot, FastDiv by_layers) {
  const int lane = lane_id();
  const uint32_t row0 = (blockIdx.x * 4 + threadIdx.x / kWave) * kPackRows;
  const uint32_t rows = (uint32_t)a.n * (uint32_t)a.layers;
  if (row0 >= rows) return;
  float x[kPackRows][8];
#pragma unroll
  for (int r = 0; r < kPackRows; ++r) {
    const uint32_t row = min(row0 + r, rows - 1), entry = by_layers.div(row), layer = row - entry * a.layers;
    load_f32<T, 8, ALIGNED>(static_cast<const T*>(a.a) + entry * a.a_stride[0] + layer * a.a_stride[1] + 8 * lane, x[r]);
  }
  {
    const uint32_t row = row0 + lane / 32;
    static_assert(kPackRows == 2, "a row's rotary pairs for either half of the wave");
    if (row < rows) {
      const uint32_t entry = by_layers.div(row), layer = row - entry * a.layers;
      const T* rope = static_cast<const T*>(a.b) + entry * a.b_stride[0] + layer * a.b_stride[1];
      const int pair = lane % 32;
      const int at0 = rot.interleaved ? 2 * pair : pair, at1 = rot.interleaved ? 2 * pair + 1 : pair + kRope / 2;
      const float r0 = to_f32(rope[at0]), r1 = to_f32(rope[at1]);
      float y0 = r0, y1 = r1;
      if (a.positions) {
        const float2 cs = rotary_of(rot, a.positions + (size_t)entry * rot.axes, pair);
        const float2 y = turned(r0, r1, cs);
        y0 = y.x;
        y1 = y.y;
      }
      __bf16* ro = reinterpret_cast<__bf16*>(a.rows + (size_t)row * kLatentRow + kRopeAt);
      ro[at0] = (__bf16)y0;
      ro[at1] = (__bf16)y1;
    }
  }
#pragma unroll
  for (int r = 0; r < kPackRows; ++r) {
    if (row0 + r >= rows) break;
    float amax = 0.0f, odd = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      amax = fmaxf(amax, fabsf(x[r][i]));
      odd = __builtin_fmaf(x[r][i], 0.0f, odd);   // NaN after an infinity or a NaN
    }
    amax = max_of_16(amax);
    float scale = divide_by(amax, kE4m3Max, 1.0f / kE4m3Max);
    if (__any(odd != 0.0f || !(scale >= 0x1p-60f))) {
      amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, finite_abs(x[r][i]));
      scale = scale_of(max_of_16(amax));
#pragma unroll
      for (int i = 0; i < 8; ++i) x[r][i] = to_e4m3_range(x[r][i], scale);
    } else {
      const float inv = 1.0f / scale;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[r][i] = divide_by(x[r][i], scale, inv);
    }
    uint8_t* out = a.rows + (size_t)(row0 + r) * kLatentRow;
    reinterpret_cast<uint2*>(out)[lane] =
        make_uint2(e4m3x4(x[r][0], x[r][1], x[r][2], x[r][3]), e4m3x4(x[r][4], x[r][5], x[r][6], x[r][7]));
    if (lane % 16 == 0) *reinterpret_cast<float*>(out + kLatentScaleAt + lane / 16 * 4) = scale;
  }
}

// V pairs of a row as they are in memory, first .. first + V - 1 of `pairs`.
template <typename T, int V>
struct Pairs {
  typedef T vec __attribute__((ext_vector_type(V)));
  typedef T vec2 __attribute__((ext_vector_type(2 * V)));
  T a[V], b[V];
  __device__ __forceinline__ void load(const T* x, int first, int pairs, bool interleaved) {
    if (interleaved) {
      vec2 v;
      if constexpr (V > 1) v = *reinterpret_cast<const vec2*>(x + 2 * first);
      else v = vec2{x[2 * first], x[2 * first + 1]};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        a[j] = v[2 * j];
        b[j] = v[2 * j + 1];
      }
    } else if constexpr (V > 1) {
      const vec v = *reinterpret_cast<const vec*>(x + first), w = *reinterpret_cast<const vec*>(x + first + pairs);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        a[j] = v[j];
        b[j] = w[j];
      }
    } else {
      a[0] = x[first];
      b[0] = x[first + pairs];
    }
  }
  __device__ __forceinline__ void turn(const float2* cs) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float2 y = turned(to_f32(a[j]), to_f32(b[j]), cs[j]);
      a[j] = (T)y.x;
      b[j] = (T)y.y;
    }
  }
  __device__ __forceinline__ void store(T* y, int first, int pairs, bool interleaved) const {
    if (interleaved) {
      if constexpr (V > 1) {
        vec2 v;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[2 * j] = a[j];
          v[2 * j + 1] = b[j];
        }
        *reinterpret_cast<vec2*>(y + 2 * first) = v;
      } else {
        y[2 * first] = a[0];
        y[2 * first + 1] = b[0];
      }
    } else if constexpr (V > 1) {
      vec v, w;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[j] = a[j];
        w[j] = b[j];
      }
      *reinterpret_cast<vec*>(y + first) = v;
      *reinterpret_cast<vec*>(y + first + pairs) = w;
    } else {
      y[first] = a[0];
      y[first + pairs] = b[0];
    }
  }
};

// Heads rows. A workgroup takes 256 units of four pairs of one side (keys in the
// first half of the grid, values in the second): whole scale blocks (a row, a KV
// head), of `units` lanes each (a power of two, 8 to 128), whose largest value is
// found by shuffles, and through LDS where a block is more than a wave. The sines
// of the workgroup's tokens are computed once for all their heads, into LDS, while
// the values are on their way. (65536 rows of 8 KV heads of 128, turned, 403 MB
// read and written: 683 us with a wave per scale block and single elements,
// 114 us so. 71 thousand vector instructions a SIMD bound it.)
constexpr int kPackThreads = 256;

template <typename T, bool ALIGNED>
__global__ __launch_bounds__(kPackThreads) void k_pack_heads(PackDev a, RotaryDev rot, int units, uint32_t side_blocks,
                                                            FastDiv by_heads, FastDiv by_layers) {
  extern __shared__ float2 s_cs[];   // [entry][token][pair] from the workgroup's first entry on
  __shared__ float s_max[kPackThreads / kWave];
  const bool value = blockIdx.x >= side_blocks;
  const int dim = a.head_dim, half = dim / 2, block = a.block_tokens, per_token = dim / 8;
  const uint32_t per = kPackThreads / units;                      // scale blocks here
  const uint32_t all = (uint32_t)a.n * (uint32_t)a.layers * (uint32_t)a.kv_heads;
  const uint32_t first = (blockIdx.x - (value ? side_blocks : 0u)) * per;
  const uint32_t mine = first + threadIdx.x / units;
  const bool there = mine < all;
  const uint32_t at = min(mine, all - 1);
  const uint32_t row = by_heads.div(at), h = at - row * a.kv_heads;
  const uint32_t entry = by_layers.div(row), layer = row - entry * a.layers;
  const int unit = (int)threadIdx.x % units, tok = unit / per_token, pair = unit % per_token * 4;
  const int count = a.count ? min(max(a.count[entry], 0), block) : block;
  const bool live = tok < count;

  Pairs<T, 4> x;
  if (live) {
    const long long* st = value ? a.b_stride : a.a_stride;
    const T* src = static_cast<const T*>(value ? a.b : a.a) + entry * st[0] + layer * st[1] + tok * st[2] + h * st[3];
    if constexpr (ALIGNED) {
      x.load(src, pair, half, rot.interleaved);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x.a[j] = src[rot.interleaved ? 2 * (pair + j) : pair + j];
        x.b[j] = src[rot.interleaved ? 2 * (pair + j) + 1 : pair + j + half];
      }
    }
  }
  const uint32_t entry0 = by_layers.div(by_heads.div(first));
  if (!value && a.positions) {
    const uint32_t last = by_layers.div(by_heads.div(min(first + per, all) - 1));
    const int tokens = (int)(last - entry0 + 1) * block;
    for (int e = threadIdx.x; e < tokens * half; e += kPackThreads)
      s_cs[e] = rotary_of(rot, a.positions + ((size_t)entry0 * block + e / half) * rot.axes, e % half);
    __syncthreads();
  }
  float y[2][4];                                                  // first and second of each pair
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[0][j] = live ? to_f32(x.a[j]) : 0.0f;
    y[1][j] = live ? to_f32(x.b[j]) : 0.0f;
  }
  if (!value && a.positions) {
    const float2* cs = s_cs + ((size_t)(entry - entry0) * block + tok) * half + pair;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 t = turned(y[0][j], y[1][j], cs[j]);
      y[0][j] = t.x;
      y[1][j] = t.y;
    }
  }
  auto largest = [&](float v) {                                   // of the scale block; every lane calls it
    for (int d = 1; d < min(units, kWave); d *= 2) v = fmaxf(v, __shfl_xor(v, d, kWave));
    if (units > kWave) {
      __syncthreads();
      if (lane_id() == 0) s_max[threadIdx.x / kWave] = v;
      __syncthreads();
      const int w0 = (int)threadIdx.x / units * (units / kWave);
      for (int w = 0; w < units / kWave; ++w) v = fmaxf(v, s_max[w0 + w]);
    }
    return v;
  };
  float amax = 0.0f, odd = 0.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      amax = fmaxf(amax, fabsf(y[i][j]));
      odd = __builtin_fmaf(y[i][j], 0.0f, odd);                   // NaN after an infinity or a NaN
    }
  amax = largest(odd == 0.0f ? amax : __builtin_inff());
  float scale = divide_by(amax, kE4m3Max, 1.0f / kE4m3Max);
  const bool far = !(scale >= 0x1p-60f && scale < __builtin_inff());
  // one answer for the whole workgroup where a scale block is more than a wave: largest() has barriers then
  if (units > kWave ? __syncthreads_or(far) : __any(far)) {
    float finite = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) finite = fmaxf(finite, finite_abs(y[i][j]));
    scale = scale_of(largest(finite));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) y[i][j] = to_e4m3_range(y[i][j], scale);
  } else {
    const float inv = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) y[i][j] = divide_by(y[i][j], scale, inv);
  }
  if (!there) return;
  uint8_t* out = a.rows + (size_t)row * a.row_bytes;
  const int part = block * dim;
  uint8_t* codes = out + (value ? a.kv_heads * part : 0) + h * part + tok * dim;
  if (rot.interleaved) {
    *reinterpret_cast<uint2*>(codes + 2 * pair) = make_uint2(e4m3x4(y[0][0], y[1][0], y[0][1], y[1][1]),
                                                            e4m3x4(y[0][2], y[1][2], y[0][3], y[1][3]));
  } else {
    *reinterpret_cast<uint32_t*>(codes + pair) = e4m3x4(y[0][0], y[0][1], y[0][2], y[0][3]);
    *reinterpret_cast<uint32_t*>(codes + half + pair) = e4m3x4(y[1][0], y[1][1], y[1][2], y[1][3]);
  }
  uint8_t* tail = out + 2 * a.kv_heads * part;
  if (unit == 0) reinterpret_cast<float*>(tail)[(value ? a.kv_heads : 0) + h] = scale;
  if (h == 0 && !value) {   // the token count and the zeros behind it, fewer words than a block has lanes
    int32_t* words = reinterpret_cast<int32_t*>(tail + 8 * a.kv_heads);
    const int n = (int)(out + a.row_bytes - reinterpret_cast<uint8_t*>(words)) / 4;
    if (unit < n) words[unit] = unit == 0 ? count : 0;
  }
}

// Units of a scale block, and workgroups of either side.
static int pack_units(const PackDev& a) { return a.block_tokens * a.head_dim / 8; }
long long pack_heads_blocks(const PackDev& a) {
  const long long per = kPackThreads / pack_units(a);
  return ((long long)a.n * a.layers * a.kv_heads + per - 1) / per;
}

// Rotary positions of [n][heads][dim] tensors. A workgroup takes `tokens` tokens
// and a range of heads, V pairs of a row a unit, U units a lane: their loads are
// on their way while the tokens' sines and cosines are computed, once each, into
// LDS. In place is fine: a lane reads its pairs before it writes them. (8191 x 32
// heads x 128 fp32, 268 MB read and written: 42 us.)
template <typename T, int V, int U>
__global__ __launch_bounds__(256) void k_rotate(RotateDev a, RotaryDev rot, FastDiv by_units, FastDiv by_heads) {
  extern __shared__ float2 s_cs[];   // [tokens][pairs]
  const int pairs = a.dim / 2, units = pairs / V;
  const int head_parts = 1 + (a.heads - 1) / a.heads_per_block;   // heads may be near 2^31
  const int tok0 = blockIdx.x / head_parts * a.tokens_per_block;
  const int head0 = blockIdx.x % head_parts * a.heads_per_block;
  const int tokens = min(a.tokens_per_block, a.n - tok0);
  const int heads = min(a.heads_per_block, a.heads - head0);
  Pairs<T, V> x[U];
  int first[U], head[U], tok[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // the whole range's division, whatever part of it this workgroup has: heads beyond it do nothing
    const uint32_t e = threadIdx.x + u * 256, row = by_units.div(e);
    tok[u] = (int)by_heads.div(row);
    first[u] = (int)(e - row * units) * V;
    head[u] = (int)row - tok[u] * a.heads_per_block;
    if (head[u] >= heads) tok[u] = tokens;
    if (tok[u] < tokens)
      x[u].load(static_cast<const T*>(a.x) + (tok0 + tok[u]) * a.x_stride[0] + (head0 + head[u]) * a.x_stride[1],
                first[u], pairs, rot.interleaved);
  }
  for (int e = threadIdx.x; e < tokens * pairs; e += 256) {
    const int t = e / pairs;
    float2 cs = rotary_of(rot, a.positions + (size_t)(tok0 + t) * rot.axes, e % pairs);
    if (a.inverse) cs.y = -cs.y;
    s_cs[e] = cs;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (tok[u] >= tokens) continue;
    x[u].turn(s_cs + tok[u] * pairs + first[u]);
    x[u].store(static_cast<T*>(a.out) + (tok0 + tok[u]) * a.out_stride[0] + (head0 + head[u]) * a.out_stride[1],
               first[u], pairs, rot.interleaved);
  }
}

template <typename T>
static hipError_t pack_of(const PackDev& a, const RotaryDev& rot, hipStream_t s) {
  const int rows = a.n * a.layers;
  if (a.latent) {
    const int blocks = (rows + 4 * kPackRows - 1) / (4 * kPackRows);
    const FastDiv by_layers(a.layers);
    if (a.aligned) k_pack_latent<T, true><<<blocks, 256, 0, s>>>(a, rot, by_layers);
    else k_pack_latent<T, false><<<blocks, 256, 0, s>>>(a, rot, by_layers);
  } else {
    const int units = pack_units(a), per = kPackThreads / units;
    const uint32_t blocks = (uint32_t)pack_heads_blocks(a);
    // entries that `per` scale blocks touch, which need not begin with a row's first
    const size_t entries = (per + a.kv_heads - 1) / a.kv_heads + 1;
    const size_t lds = a.positions ? entries * a.block_tokens * (a.head_dim / 2) * sizeof(float2) : 0;
    const FastDiv by_heads(a.kv_heads), by_layers(a.layers);
    if (a.aligned) k_pack_heads<T, true><<<2 * blocks, kPackThreads, lds, s>>>(a, rot, units, blocks, by_heads, by_layers);
    else k_pack_heads<T, false><<<2 * blocks, kPackThreads, lds, s>>>(a, rot, units, blocks, by_heads, by_layers);
  }
  return hipGetLastError();
}

hipError_t launch_pack(const PackDev& a, const RotaryDev& rot, int type, hipStream_t s) {
  if (type == ULA_BF16) return pack_of<__bf16>(a, rot, s);
  if (type == ULA_FP16) return pack_of<_Float16>(a, rot, s);
  return pack_of<float>(a, rot, s);
}

// Workgroups of a turn: two units a lane, which is enough of them for a decode step
// and holds a head's units (at most 128).
constexpr int kRotateUnits = 2, kRotateVector = 4;
long long plan_rotate(RotateDev* a) {
  constexpr int kUnits = 256 * kRotateUnits;
  const int pairs = a->dim / 2, units = a->aligned ? pairs / kRotateVector : pairs;
  a->heads_per_block = std::max(1, std::min(a->heads, kUnits / units));
  a->tokens_per_block = std::max(1, std::min(a->n, std::min(kUnits / (units * a->heads_per_block), 4096 / pairs)));
  return (long long)((a->n + (long long)a->tokens_per_block - 1) / a->tokens_per_block) *
         (1 + (a->heads - 1) / a->heads_per_block);
}

template <typename T, int V>
static void rotate_units(RotateDev a, const RotaryDev& rot, hipStream_t s) {
  const long long blocks = plan_rotate(&a);
  const int pairs = a.dim / 2;
  const size_t lds = (size_t)a.tokens_per_block * pairs * sizeof(float2);
  k_rotate<T, V, kRotateUnits><<<(unsigned)blocks, 256, lds, s>>>(a, rot, FastDiv(pairs / V), FastDiv(a.heads_per_block));
}

template <typename T>
static hipError_t rotate_of(const RotateDev& a, const RotaryDev& rot, hipStream_t s) {
  if (a.aligned) rotate_units<T, kRotateVector>(a, rot, s);
  else rotate_units<T, 1>(a, rot, s);
  return hipGetLastError();
}

hipError_t launch_rotate(const RotateDev& a, const RotaryDev& rot, int type, hipStream_t s) {
  if (type == ULA_BF16) return rotate_of<__bf16>(a, rot, s);
  if (type == ULA_FP16) return rotate_of<_Float16>(a, rot, s);
  return rotate_of<float>(a, rot, s);
}

}  // namespace ula
