// Attention of each selection set over its selected rows in the heads format:
// keys and values of every KV head in e4m3 with a scale for each block of tokens
// and head, read from the GPU pool where they lie.
//
// With k8, v8 a token's codes and ks, vs the scales of its block for this KV
// head, c = scale log2(e):
//   S_j = c ks_j (q . k8_j),  p_j = 2^(S_j - m),  o = sum_j p_j vs_j v8_j / l
// e4m3 values are exact in bf16 and fp16, so both products run on 16-bit matrix
// instructions and the scales are applied in 32 bits, to S and to p. p vs is then
// rounded to fp16 (at most 2^-11 of its value). m follows the largest p vs, not
// the largest p, so that fp16's range serves scales from 2^-60 to 2^80 (p itself
// stays in the range of 32 bits): the largest p vs lies between 2^7 and 2^15, and
// one below fp16's least value (its rounding: 2^-25) is off by less than 2^-32 of
// it. For fp16 results, which show that rounding (their own is as large), what it
// leaves goes through a second product: off by 2.1e-4 of their size instead of
// 3.4e-4, 21 -> 22 us for 64 sets x 500 blocks of 8 tokens x 2 KV heads of 64.
//
// Only 2 x heads / kv_heads operations per byte, so loads in flight count most (two
// waves a SIMD still wait half of their time, and 2.2 TB/s come from HBM). A wave
// works by itself, on one KV head's up to 16 query heads and one range of tokens,
// with no barrier, and many waves per compute unit keep loads in flight; waves of
// one workgroup take neighbouring KV heads of the same tokens, whose parts of a
// row share cache lines. 32 tokens at a time: keys go from memory to registers
// as the operand of S^T = K Q^T (heads in the lanes' columns), values through a
// few KB of LDS, from which a transposing read makes the operand of
// O^T = V^T P^T; p stays in the lane that computed it. The loads of tile i + 1
// and the slots of tile i + 2 are in flight while tile i is computed.
#include <algorithm>

#include "row_format.h"

namespace ula {

constexpr int kTok = 32;             // tokens per tile
constexpr int kHeadWaves = 4;
constexpr int kHeadsPerWave = 16;

template <typename Q8, int D>
__global__ __launch_bounds__(kHeadWaves * kWave) void k_attend_heads(GroupDev g, AttendDev a, int n_items) {
  constexpr bool kRest = !__is_same(Q8, bf16x8);   // see above: p vs in two parts
  constexpr int kPieces = D / 16;              // 16-byte pieces of a token's key or value
  constexpr int kKeyLoads = D / 64;            // pieces of its key a lane holds (a quarter)
  constexpr int kValLoads = kTok * kPieces / kWave;
  struct WaveLds {
    alignas(1024) uint8_t v[kTok * D];
    alignas(16) float ks[kTok], vs[kTok];
  };
  __shared__ WaveLds s_all[kHeadWaves];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int quad = lane / 16, col = lane % 16;
  const int item = blockIdx.x * kHeadWaves + wave;
  if (item >= n_items) return;                 // waves are independent: no barrier below
  const ReaderState state = reader_state(g);
  WaveLds& s = s_all[wave];

  const int unit = item % a.head_blocks;
  const int split = item / a.head_blocks % a.splits;
  const int set = item / a.head_blocks / a.splits;
  const int shared = a.heads / a.kv_heads;     // query heads per KV head
  const int blocks = (shared + kHeadsPerWave - 1) / kHeadsPerWave;
  const int kvh = unit / blocks;
  const int hi = unit % blocks * kHeadsPerWave + col;
  const bool has_head = hi < shared;
  const int head = kvh * shared + hi;
  const int block = 1 << a.block_shift;
  const int tok0 = split * a.split_keys;
  const int ntok = max(0, min(a.split_keys, (a.k << a.block_shift) - tok0));
  const int tiles = (ntok + kTok - 1) / kTok;

  Q8 q[D / 32];
  if (has_head) {
    const uint16_t* p = static_cast<const uint16_t*>(a.q) + set * a.q_set_stride + head * a.q_head_stride + quad * (D / 4);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) q[j] = a.q_aligned ? load8<Q8, true>(p + 8 * j) : load8<Q8, false>(p + 8 * j);
  } else {
#pragma unroll
    for (int j = 0; j < D / 32; ++j) q[j] = Q8{};
  }

  const uint8_t* pool = g.pool + (size_t)a.layer * g.row_bytes;
  const int head_at = kvh * block * D;                         // this head's keys inside a row
  const int val_at = a.kv_heads * block * D;                   // from keys to values
  const int scale_at = 2 * val_at + 4 * kvh;
  int err = 0;

  // the selection entry of this lane's token (lane % 32) of a tile
  auto look = [&](int tile) -> Lookup {
    const int t = tile * kTok + lane % kTok;
    if (t >= ntok) return {make_uint2(kAbsent, kAbsent), -1};
    return look_up(g, a.sel, set * a.k + ((tok0 + t) >> a.block_shift), a.n_res);
  };
  vec4u kreg[2][kKeyLoads], vreg[kValLoads];
  float ks = 0.0f, vs = 0.0f;
  uint32_t live = 0;                                           // bit per token
  // loads of a tile whose slots are known
  auto load = [&](int tile, uint32_t slot) {
    const int t0 = tok0 + tile * kTok;
    int count = 0;
    ks = vs = 0.0f;
    if (slot != kAbsent) {
      const uint8_t* row = pool + (size_t)slot * g.slot_bytes + scale_at;
      ks = *reinterpret_cast<const float*>(row);
      vs = *reinterpret_cast<const float*>(row + 4 * a.kv_heads);
      count = *reinterpret_cast<const int32_t*>(row - 4 * kvh + 8 * a.kv_heads);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = 8 * (col / 4) + 4 * u + col % 4;
      const uint32_t sl = (uint32_t)__shfl((int)slot, t, kWave);
      const uint8_t* p = pool + (size_t)sl * g.slot_bytes + head_at + ((t0 + t) & (block - 1)) * D + quad * (D / 4);
#pragma unroll
      for (int j = 0; j < kKeyLoads; ++j)
        kreg[u][j] = sl != kAbsent ? *reinterpret_cast<const vec4u*>(p + 16 * j) : vec4u{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) {
      const int t = (i * kWave + lane) / kPieces, c = lane % kPieces;
      const uint32_t sl = (uint32_t)__shfl((int)slot, t, kWave);
      const uint8_t* p = pool + (size_t)sl * g.slot_bytes + head_at + val_at + ((t0 + t) & (block - 1)) * D + 16 * c;
      vreg[i] = sl != kAbsent ? *reinterpret_cast<const vec4u*>(p) : vec4u{0u, 0u, 0u, 0u};
    }
    const bool mine = slot != kAbsent && ((t0 + lane % kTok) & (block - 1)) < count;
    if (!mine) ks = vs = 0.0f;
    live = (uint32_t)__ballot(mine);
  };

  f32x4 o[D / 16];
#pragma unroll
  for (int t = 0; t < D / 16; ++t) o[t] = f32x4{};
  float m = -__builtin_inff(), l = 0.0f;
  // transposed reads: this lane names token 8 quad + col / 2, piece 0; piece x is ^ (x << 4)
  const int vtok = 8 * quad + col / 2;
  auto swizzle = [](int tok) { return D == 128 ? (tok >> 1) & 7 : (tok >> 2) & 1; };
  const uint32_t vrow = lds_address(s.v) + vtok * D + (swizzle(vtok) << 4) + (col & 1) * 8;

  const Lookup first = look(0);
  Lookup next = look(1);
  int ok = 0;
  if (lane == 0) ok = reader_ready(g, state, a.want_flag);
  if (!__builtin_amdgcn_readfirstlane(ok)) return;
  if (tiles > 0) load(0, slot_of(g, first, a.n_res, err));
#pragma unroll 1
  for (int tile = 0; tile < tiles; ++tile) {
    // this tile out of the staging registers
    vec4u k8[2][kKeyLoads];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < kKeyLoads; ++j) k8[u][j] = kreg[u][j];
    const uint32_t now = live;
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) {
      const int t = (i * kWave + lane) / kPieces, c = lane % kPieces;
      // a token out of use must not reach the product: 0 x NaN
      const vec4u v = (now >> t & 1u) ? vreg[i] : vec4u{0u, 0u, 0u, 0u};
      *reinterpret_cast<vec4u*>(&s.v[t * D + ((c ^ swizzle(t)) << 4)]) = v;
    }
    if (lane < kTok) {
      s.ks[lane] = ks;
      s.vs[lane] = vs;
    }
    // the next tile's loads, and the slots of the one after it
    if (tile + 1 < tiles) {
      const uint32_t cur = slot_of(g, next, a.n_res, err);
      next = look(tile + 2);
      load(tile + 1, cur);
    }
    if (now == 0) continue;
    f32x4 S[2] = {}, sv[2];
    float top = -__builtin_inff();               // of log2(p vs), to 1 upwards; vs below 2^-60 counts as that
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int j = 0; j < kKeyLoads; ++j) {
        S[u] = mfma16(widen8<Q8>(k8[u][j].x, k8[u][j].y), q[2 * j], S[u]);
        S[u] = mfma16(widen8<Q8>(k8[u][j].z, k8[u][j].w), q[2 * j + 1], S[u]);
      }
      const f32x4 sc = lds_get<f32x4>(lds_address(s.ks) + (8 * quad + 4 * u) * 4);
      sv[u] = lds_get<f32x4>(lds_address(s.vs) + (8 * quad + 4 * u) * 4);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        S[u][r] *= sc[r] * a.scale_log2;
        if (!(now >> (8 * quad + 4 * u + r) & 1u)) S[u][r] = -__builtin_inff();
        top = fmaxf(top, S[u][r] + (float)__builtin_amdgcn_frexp_expf(fmaxf(fabsf(sv[u][r]), 0x1p-60f)));
      }
    }
    // p vs in fp16: the reference m moves when p vs could pass 2^15, and then so that
    // the largest is between 2^7 and 2^8
    top = max_quads(top);
    if (__any(top > m + 15.0f)) {
      const bool move = top > m + 15.0f;
      const float nm = move ? top - 8.0f : m;
      const float al = move ? __builtin_amdgcn_exp2f(m - nm) : 1.0f;
      m = nm;
      l *= al;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) o[t] *= al;
    }
    const float base = m == -__builtin_inff() ? 0.0f : m;
    f16x8 p, rest;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float w = __builtin_amdgcn_exp2f(S[u][r] - base);
        l += w;
        const float x = w * sv[u][r];
        p[4 * u + r] = (_Float16)x;
        if constexpr (kRest) rest[4 * u + r] = (_Float16)(x - (float)p[4 * u + r]);
      }
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      const i32x2 v8 = lds_read_transposed(vrow ^ (t << 4));
      const f16x8 v = widen8<f16x8>((uint32_t)v8.x, (uint32_t)v8.y);
      o[t] = mfma16(v, p, o[t]);
      if constexpr (kRest) o[t] = mfma16(v, rest, o[t]);
    }
  }
  if (err) latch_gather(g.ctr, err);
  l = sum_quads(l);
  if (!has_head) return;
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  const float lse2 = l != 0.0f ? m + log2f(l) : -__builtin_inff();
  if (a.splits > 1) {
    const size_t row = ((size_t)set * a.heads + head) * a.splits + split;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) *reinterpret_cast<f32x4*>(a.part_o + row * D + 16 * t + 4 * quad) = o[t] * inv;
    if (quad == 0) a.part_lse[row] = lse2;
    return;
  }
  uint16_t* out = static_cast<uint16_t*>(a.out) + set * a.out_set_stride + head * a.out_head_stride + 4 * quad;
#pragma unroll
  for (int t = 0; t < D / 16; ++t) {
    const float v[4] = {o[t][0] * inv, o[t][1] * inv, o[t][2] * inv, o[t][3] * inv};
    store4<Q8>(out + 16 * t, v, a.out_aligned);
  }
  if (quad == 0 && a.lse) a.lse[(size_t)set * a.heads + head] = lse2 * kLn2;
}

// Splits so that about kWaveTarget waves run (8 per compute unit), each with at
// least kLeastTiles tiles: a split costs its start and the join's traffic.
// Measured, kernel + join, us, for 16 sets x 2048 tokens x 8 KV heads of 128 (70 MB)
// and 64 sets x 500 blocks of 8 tokens x 2 KV heads of 64 (65 MB):
//   1024 waves 24 + 4 and 28 + 4;  2048 waves 21 + 4 and 21 + 5;  4096 the same;
//   2048 waves of at least 8 tiles 25 + 4 and 22 + 5, of at least 2 as of 4.
// The rows alone take 15 us and 14 us at the rate of a copy of their size.
AttendPlan plan_attend_heads(int n_sets, int tokens, int heads, int kv_heads) {
  constexpr int kWaveTarget = 256 * 8, kLeastTiles = 4;
  AttendPlan p{};
  const int shared = heads / kv_heads;
  p.head_blocks = kv_heads * ((shared + kHeadsPerWave - 1) / kHeadsPerWave);
  const long long base = std::max<long long>(1, (long long)n_sets * p.head_blocks);
  const int tiles = std::max(1, (tokens + kTok - 1) / kTok);
  const int want = (int)std::min<long long>(std::min<long long>((kWaveTarget + base - 1) / base, kAttendMaxSplits), std::max(1, tiles / kLeastTiles));
  const int per = (tiles + want - 1) / want;
  p.splits = (tiles + per - 1) / per;
  p.split_keys = per * kTok;
  return p;
}

template <typename Q8>
static hipError_t launch_heads_of(const GroupDev& g, const AttendDev& a, int n_sets, int head_dim, hipStream_t s) {
  const int items = n_sets * a.head_blocks * a.splits;
  const int blocks = (items + kHeadWaves - 1) / kHeadWaves;
  if (head_dim == 64) k_attend_heads<Q8, 64><<<blocks, kHeadWaves * kWave, 0, s>>>(g, a, items);
  else k_attend_heads<Q8, 128><<<blocks, kHeadWaves * kWave, 0, s>>>(g, a, items);
  return hipGetLastError();
}

hipError_t launch_attend_heads(const GroupDev& g, const AttendDev& a, int type, int n_sets, int head_dim,
                               hipStream_t s) {
  return type == ULA_BF16 ? launch_heads_of<bf16x8>(g, a, n_sets, head_dim, s)
                          : launch_heads_of<f16x8>(g, a, n_sets, head_dim, s);
}

}  // namespace ula
