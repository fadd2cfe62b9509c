// Norms of queries and keys for each head, with rotary positions in the same pass.
//
// For a row x of `dim` channels, weights w (or 1):
//   y_i = w_i x_i / sqrt(sum_j x_j^2 / dim + eps)
// and then the first R channels' pairs turn by the angles of their token's
// positions (rotary.h); channels from R on stay as y. Sums, products and the turn
// are in 32 bits, the result is rounded to its type once. Squares that overflow are
// summed again scaled by 2^-100, so finite rows of any size have finite norms.
//
// Bound by HBM for a prompt and by the launch for a decode step. Queries and keys
// go in one launch: a token's rows are its query heads and then its key heads.
// L lanes share a row, 8 channels (a unit) each, 16 bytes at a time for 16-bit
// types; a lane's unit is the same in every row it takes, so its weights stay in
// registers. A workgroup takes whole tokens (or, where those are too few to fill the
// card, a part of one token's heads), whose sines it computes once into LDS while
// the first rows are on their way.
#include <algorithm>

#include "rotary.h"
#include "row_format.h"

namespace ula {

constexpr int kNormThreads = 256;
constexpr int kNormAhead = 4;          // rows a lane has on their way

// The sum over the L lanes of a row, in all of them, in one order whatever the lane.
template <int L>
__device__ __forceinline__ float sum_of_lanes(float x) {
#define ULA_DPP(v, ctrl) __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), ctrl, 0xF, 0xF, true))
  x += ULA_DPP(x, 0xB1);                              // the lane 1 away
  x += ULA_DPP(x, 0x4E);                              // 2 away
  x += ULA_DPP(x, 0x141);                             // the other four of eight
  if constexpr (L > 8) x += ULA_DPP(x, 0x140);        // the other eight of 16
#undef ULA_DPP
  if constexpr (L > 16) {
    const float2 v = swap_quads(x);
    x = v.x + v.y;
  }
  return x;
}

// 1 / sqrt(mean square + eps) of a row whose lane sums of squares `sum` adds up;
// again(factor) is the same sum of the values times factor.
template <typename F>
__device__ __forceinline__ float inverse_rms(float sum, float inv_dim, float eps, F again) {
  float inv = 1.0f / sqrtf(__builtin_fmaf(sum, inv_dim, eps));
  if (__any(!(sum < __builtin_inff()))) {
    const float far = 0x1p-100f / sqrtf(again(0x1p-100f) * inv_dim);
    if (!(sum < __builtin_inff())) inv = far;
  }
  return inv;
}

// The row of a token's head (queries', then keys').
template <typename T>
__device__ __forceinline__ const T* norm_source(const NormDev& a, int token, int head) {
  const bool key = head >= a.q_heads;
  const long long* st = key ? a.k_stride : a.q_stride;
  return static_cast<const T*>(key ? a.k : a.q) + token * st[0] + (key ? head - a.q_heads : head) * st[1];
}
template <typename T>
__device__ __forceinline__ T* norm_target(const NormDev& a, int token, int head) {
  const bool key = head >= a.q_heads;
  const long long* st = key ? a.k_out_stride : a.q_out_stride;
  return static_cast<T*>(key ? a.k_out : a.q_out) + token * st[0] + (key ? head - a.q_heads : head) * st[1];
}

// Weight of a channel of queries or keys.
template <typename T>
__device__ __forceinline__ float norm_weight(const NormDev& a, bool key, int channel) {
  const void* w = key ? a.k_weight : a.q_weight;
  if (!w) return 1.0f;
  return a.wide_weights ? static_cast<const float*>(w)[channel] : to_f32(static_cast<const T*>(w)[channel]);
}

// The sines of the workgroup's tokens into LDS, [token][pair].
__device__ __forceinline__ void norm_sines(const NormDev& a, const RotaryDev& rot, float2* cs, int tok0, int tokens) {
  const int pairs = a.rotary / 2;
  for (int e = threadIdx.x; e < tokens * pairs; e += kNormThreads) {
    const int t = e / pairs;
    cs[e] = rotary_of(rot, a.positions + (size_t)(tok0 + t) * rot.axes, e - t * pairs);
  }
}

// dim and R multiples of 8. L >= dim / 8.
template <typename T, int L, bool ALIGNED>
__global__ __launch_bounds__(kNormThreads) void k_norm(NormDev a, RotaryDev rot, FastDiv by_heads) {
  extern __shared__ float2 s_cs[];
  typedef T vec4 __attribute__((ext_vector_type(4)));
  typedef T vec8 __attribute__((ext_vector_type(8)));
  constexpr int kAtOnce = kNormThreads / L;            // rows
  const int all_heads = a.q_heads + a.k_heads;
  const int head_parts = (all_heads + a.heads_per_block - 1) / a.heads_per_block;
  const int tok0 = blockIdx.x / head_parts * a.tokens_per_block;
  const int head0 = blockIdx.x % head_parts * a.heads_per_block;
  const int tokens = min(a.tokens_per_block, a.n - tok0);
  const int heads = min(a.heads_per_block, all_heads - head0);
  const int unit = threadIdx.x % L;
  const bool mine = unit < a.dim / 8;
  const bool turns = unit < a.rotary / 8;
  const bool halves = turns && !rot.interleaved;       // pairs (i, i + R / 2): four channels from either half
  const int at0 = halves ? 4 * unit : 8 * unit;
  const int at1 = halves ? a.rotary / 2 + 4 * unit : 8 * unit + 4;

  struct Unit {
    vec4 lo, hi;
    bool there;
    int token, head;
  };
  auto load = [&](Unit& u, int row) {
    u.token = (int)by_heads.div(row);
    u.head = row - u.token * a.heads_per_block;
    u.there = u.token < tokens && u.head < heads;
    u.lo = u.hi = vec4{};
    if (!u.there || !mine) return;
    const T* p = norm_source<T>(a, tok0 + u.token, head0 + u.head);
    if constexpr (ALIGNED) {
      if (rot.interleaved) {                           // uniform
        const vec8 v = *reinterpret_cast<const vec8*>(p + at0);
        u.lo = v.lo;
        u.hi = v.hi;
      } else {
        u.lo = *reinterpret_cast<const vec4*>(p + at0);
        u.hi = *reinterpret_cast<const vec4*>(p + at1);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u.lo[j] = p[at0 + j];
        u.hi[j] = p[at1 + j];
      }
    }
  };
  const int rows = tokens * a.heads_per_block;         // with a last part's missing heads
  Unit u[kNormAhead];
  const int row0 = threadIdx.x / L;
#pragma unroll
  for (int i = 0; i < kNormAhead; ++i) load(u[i], row0 + i * kAtOnce);
  float w[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) w[k][j] = mine ? norm_weight<T>(a, k, j < 4 ? at0 + j : at1 + j - 4) : 0.0f;
  if (a.rotary) {
    norm_sines(a, rot, s_cs, tok0, tokens);
    __syncthreads();
  }
  const float inv_dim = 1.0f / a.dim;
  for (int base = 0; base < rows; base += kNormAhead * kAtOnce) {
#pragma unroll
    for (int i = 0; i < kNormAhead; ++i) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = to_f32(u[i].lo[j]);
        x[4 + j] = to_f32(u[i].hi[j]);
      }
      const bool there = u[i].there && mine;
      const int token = u[i].token, head = head0 + u[i].head;
      if (base + kNormAhead * kAtOnce < rows) load(u[i], base + kNormAhead * kAtOnce + row0 + i * kAtOnce);
      auto squares = [&](float factor) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = x[j] * factor;
          s = __builtin_fmaf(y, y, s);
        }
        return sum_of_lanes<L>(s);
      };
      const float inv = inverse_rms(squares(1.0f), inv_dim, a.eps, squares);
      if (!there) continue;
      const bool key = head >= a.q_heads;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * (key ? w[1][j] : w[0][j]);
      if (turns) {
        const float2* cs = s_cs + token * (a.rotary / 2) + 4 * unit;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int p = halves ? j : 2 * j, q = halves ? 4 + j : 2 * j + 1;
          const float2 y = turned(x[p], x[q], cs[j]);
          x[p] = y.x;
          x[q] = y.y;
        }
      }
      // (the empty assembly keeps the conversion to fp16 apart: fused with the product it rounds
      // once instead of twice, and strides must not change bits)
      vec4 lo, hi;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        asm("" : "+v"(x[j]), "+v"(x[4 + j]));
        lo[j] = (T)x[j];
        hi[j] = (T)x[4 + j];
      }
      T* out = norm_target<T>(a, tok0 + token, head);
      if constexpr (ALIGNED) {
        if (rot.interleaved) {
          vec8 v;
          v.lo = lo;
          v.hi = hi;
          *reinterpret_cast<vec8*>(out + at0) = v;
        } else {
          *reinterpret_cast<vec4*>(out + at0) = lo;
          *reinterpret_cast<vec4*>(out + at1) = hi;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          out[at0 + j] = lo[j];
          out[at1 + j] = hi[j];
        }
      }
    }
  }
}

// Any even dim and R: a wave a row, lane i pairs i and i + 64; pairs from R / 2 on are
// the channels that do not turn.
template <typename T>
__global__ __launch_bounds__(kNormThreads) void k_norm_any(NormDev a, RotaryDev rot) {
  extern __shared__ float2 s_cs[];
  const int all_heads = a.q_heads + a.k_heads;
  const int head_parts = (all_heads + a.heads_per_block - 1) / a.heads_per_block;
  const int tok0 = blockIdx.x / head_parts * a.tokens_per_block;
  const int head0 = blockIdx.x % head_parts * a.heads_per_block;
  const int tokens = min(a.tokens_per_block, a.n - tok0);
  const int heads = min(a.heads_per_block, all_heads - head0);
  if (a.rotary) {
    norm_sines(a, rot, s_cs, tok0, tokens);
    __syncthreads();
  }
  const int half = a.rotary / 2;
  for (int row = threadIdx.x / kWave; row < tokens * heads; row += kNormThreads / kWave) {
    const int token = row / heads, head = head0 + row % heads;
    const T* p = norm_source<T>(a, tok0 + token, head);
    float x[2][2];
    int at[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int pair = lane_id() + kWave * i;
      const bool split = pair < half && !rot.interleaved;
      at[i][0] = split ? pair : 2 * pair;
      at[i][1] = split ? pair + half : 2 * pair + 1;
#pragma unroll
      for (int j = 0; j < 2; ++j) x[i][j] = 2 * pair < a.dim ? to_f32(p[at[i][j]]) : 0.0f;
    }
    auto squares = [&](float factor) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) s = __builtin_fmaf(x[i][j] * factor, x[i][j] * factor, s);
      return sum_halves(sum_of_lanes<32>(s));
    };
    const float inv = inverse_rms(squares(1.0f), 1.0f / a.dim, a.eps, squares);
    T* out = norm_target<T>(a, tok0 + token, head);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int pair = lane_id() + kWave * i;
      if (2 * pair >= a.dim) continue;
      const bool key = head >= a.q_heads;
#pragma unroll
      for (int j = 0; j < 2; ++j) x[i][j] = x[i][j] * inv * norm_weight<T>(a, key, at[i][j]);
      if (pair < half) {
        const float2 y = turned(x[i][0], x[i][1], s_cs[token * half + pair]);
        x[i][0] = y.x;
        x[i][1] = y.y;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) out[at[i][j]] = (T)x[i][j];
    }
  }
}

// Lanes of a row; 0: the form for any sizes.
static int norm_lanes(const NormDev& a) {
  if (a.dim % 8 || a.rotary % 8) return 0;
  return a.dim <= 64 ? 8 : (a.dim <= 128 ? 16 : 32);
}

// Tokens and heads of a workgroup. A step of it takes `step` rows (those its lanes have
// on their way); whole tokens, up to 16, that fill their steps best, if 1024 workgroups
// (four a compute unit) have them, else one token and as few heads as a quarter of a
// step. (8191 tokens x 36 heads of 128: 45 us with two tokens in two steps, 38 us so; the
// bytes take 28 us at the rate of a copy.)
long long plan_norm(NormDev* a) {
  const int lanes = norm_lanes(*a);
  const int at_once = lanes ? kNormThreads / lanes : kNormThreads / kWave;
  const int heads = a->q_heads + a->k_heads, step = kNormAhead * at_once;
  a->heads_per_block = heads;
  a->tokens_per_block = 0;
  double best = -1;                                    // a single token always has a plan
  for (int tokens = 1; tokens <= 16 && (tokens == 1 || a->n / tokens >= 1024); ++tokens) {
    const long long rows = (long long)tokens * heads;
    const double full = (double)rows / ((rows + step - 1) / step * step);
    if (full > best + 0.02) {
      best = full;
      a->tokens_per_block = tokens;
    }
  }
  if (a->n < 1024) {
    a->tokens_per_block = std::max(1, std::min(a->n, at_once / heads));
    a->heads_per_block = std::min(heads, at_once);
  }
  if (a->rotary) a->tokens_per_block = std::max(1, std::min(a->tokens_per_block, 4096 / (a->rotary / 2)));
  return ((a->n + (long long)a->tokens_per_block - 1) / a->tokens_per_block) *
         ((heads + a->heads_per_block - 1) / a->heads_per_block);
}

template <typename T, bool ALIGNED>
static void norm_lanes_of(const NormDev& a, const RotaryDev& rot, int lanes, unsigned blocks, size_t lds, hipStream_t s) {
  const FastDiv by_heads(a.heads_per_block);
  if (lanes == 8) k_norm<T, 8, ALIGNED><<<blocks, kNormThreads, lds, s>>>(a, rot, by_heads);
  else if (lanes == 16) k_norm<T, 16, ALIGNED><<<blocks, kNormThreads, lds, s>>>(a, rot, by_heads);
  else k_norm<T, 32, ALIGNED><<<blocks, kNormThreads, lds, s>>>(a, rot, by_heads);
}

template <typename T>
static hipError_t norm_of(NormDev a, const RotaryDev& rot, hipStream_t s) {
  const unsigned blocks = (unsigned)plan_norm(&a);
  const int lanes = norm_lanes(a);
  const size_t lds = (size_t)a.tokens_per_block * (a.rotary / 2) * sizeof(float2);
  if (!lanes) k_norm_any<T><<<blocks, kNormThreads, lds, s>>>(a, rot);
  else if (a.aligned) norm_lanes_of<T, true>(a, rot, lanes, blocks, lds, s);
  else norm_lanes_of<T, false>(a, rot, lanes, blocks, lds, s);
  return hipGetLastError();
}

hipError_t launch_norm(const NormDev& a, const RotaryDev& rot, int type, hipStream_t s) {
  if (type == ULA_BF16) return norm_of<__bf16>(a, rot, s);
  if (type == ULA_FP16) return norm_of<_Float16>(a, rot, s);
  return norm_of<float>(a, rot, s);
}

}  // namespace ula
