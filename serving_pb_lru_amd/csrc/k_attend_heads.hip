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

constexpr int kTok = kTileTokens;    // tokens per tile
constexpr int kHeadWaves = 4;
constexpr int kHeadsPerWave = 16;

// RT: groups of 16 query heads (a tree: of nodes and heads) that share a wave's keys and values.
template <typename Q8, int D, int RT, bool TREE>
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
  const int shared = a.heads / a.kv_heads;     // query heads (a tree: of all its nodes) per KV head
  constexpr int kRows = kHeadsPerWave * RT;
  const int blocks = (shared + kRows - 1) / kRows;
  const int kvh = unit / blocks;
  const int block = 1 << a.block_shift;
  const int tok0 = split * a.split_keys;
  // a tree's keys: the selected entries' tokens, padding up to history_tiles, then the drafted tokens
  const int all = TREE ? a.history_tiles * kTok + a.nodes : a.k << a.block_shift;
  const int ntok = max(0, min(a.split_keys, all - tok0));
  const int tiles = (ntok + kTok - 1) / kTok;
  const int draft0 = a.history_tiles - tok0 / kTok;            // the first tile of drafted tokens (a tree)

  // this lane's query rows: their heads, and for a tree their nodes
  bool has_head[RT];
  int head[RT], node[RT];
  unsigned long long sees[RT];                 // a tree: the drafted tokens that the node sees
  Q8 q[RT][D / 32];
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const int hi = unit % blocks * kRows + 16 * x + col;
    has_head[x] = hi < shared;
    node[x] = 0;
    sees[x] = 0;
    head[x] = kvh * shared + hi;
    if constexpr (TREE) {
      const int per = (int)a.by_heads.d;       // query heads of a node per KV head
      node[x] = (int)a.by_heads.div(hi);
      head[x] = kvh * per + hi - node[x] * per;
    }
    if (has_head[x]) {
      const uint16_t* p = static_cast<const uint16_t*>(a.q) + set * a.q_set_stride + head[x] * a.q_head_stride + quad * (D / 4);
      if constexpr (TREE) {
        p += node[x] * a.q_node_stride;
        sees[x] = a.visible[(size_t)set * a.nodes + node[x]];
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j) q[x][j] = a.q_aligned ? load8<Q8, true>(p + 8 * j) : load8<Q8, false>(p + 8 * j);
    } else {
#pragma unroll
      for (int j = 0; j < D / 32; ++j) q[x][j] = Q8{};
    }
  }

  const uint8_t* pool = g.pool + (size_t)a.layer * g.row_bytes;
  const int head_at = kvh * block * D;                         // this head's keys inside a row
  const int val_at = a.kv_heads * block * D;                   // from keys to values
  const int scale_at = 2 * val_at + 4 * kvh;
  int err = 0;

  // the selection entry of this lane's token (lane % 32) of a tile
  auto look = [&](int tile) -> Lookup {
    const int t = tile * kTok + lane % kTok;
    if constexpr (TREE) {
      if (t >= ntok || tok0 + t >= a.sel_k << a.block_shift) return {make_uint2(kAbsent, kAbsent), -1};
      return look_up(g, a.sel, set * a.sel_k + ((tok0 + t) >> a.block_shift), a.n_res);
    } else {
      if (t >= ntok) return {make_uint2(kAbsent, kAbsent), -1};
      return look_up(g, a.sel, set * a.k + ((tok0 + t) >> a.block_shift), a.n_res);
    }
  };
  vec4u kreg[2][kKeyLoads], vreg[kValLoads];
  float ks = 0.0f, vs = 0.0f;
  uint32_t live = 0;                                           // bit per token
  // loads of a tile whose slots are known
  auto load = [&](int tile, uint32_t slot) {
    const int t0 = tok0 + tile * kTok;
    int count = 0;
    ks = vs = 0.0f;
    const uint8_t* from = pool;
    size_t stride = g.slot_bytes;
    if constexpr (TREE) {
      if (tile >= draft0) {                                    // the drafted tokens' blocks in the place of slots
        const int d = (tile - draft0) * kTok + lane % kTok;
        const int per_set = (a.nodes + block - 1) >> a.block_shift;
        slot = d < a.nodes ? (uint32_t)(set * per_set + (d >> a.block_shift)) : kAbsent;
        from = a.drafts;
        stride = (size_t)a.draft_stride;
      }
    }
    if (slot != kAbsent) {
      const uint8_t* row = from + (size_t)slot * stride + scale_at;
      ks = *reinterpret_cast<const float*>(row);
      vs = *reinterpret_cast<const float*>(row + 4 * a.kv_heads);
      count = *reinterpret_cast<const int32_t*>(row - 4 * kvh + 8 * a.kv_heads);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = 8 * (col / 4) + 4 * u + col % 4;
      const uint32_t sl = (uint32_t)__shfl((int)slot, t, kWave);
      const uint8_t* p = from + (size_t)sl * stride + head_at + ((t0 + t) & (block - 1)) * D + quad * (D / 4);
#pragma unroll
      for (int j = 0; j < kKeyLoads; ++j)
        kreg[u][j] = sl != kAbsent ? *reinterpret_cast<const vec4u*>(p + 16 * j) : vec4u{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) {
      const int t = (i * kWave + lane) / kPieces, c = lane % kPieces;
      const uint32_t sl = (uint32_t)__shfl((int)slot, t, kWave);
      const uint8_t* p = from + (size_t)sl * stride + head_at + val_at + ((t0 + t) & (block - 1)) * D + 16 * c;
      vreg[i] = sl != kAbsent ? *reinterpret_cast<const vec4u*>(p) : vec4u{0u, 0u, 0u, 0u};
    }
    const bool mine = slot != kAbsent && ((t0 + lane % kTok) & (block - 1)) < count;
    if (!mine) ks = vs = 0.0f;
    live = (uint32_t)__ballot(mine);
  };

  f32x4 o[RT][D / 16];
  float m[RT], l[RT];
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    m[x] = -__builtin_inff();
    l[x] = 0.0f;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) o[x][t] = f32x4{};
  }
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
    uint32_t bad = 0;                          // a tree: drafted tokens whose values hold a NaN
    const bool drafted = TREE && tile >= draft0;
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) {
      const int t = (i * kWave + lane) / kPieces, c = lane % kPieces;
      // a token out of use must not reach the product: 0 x NaN
      vec4u v = (now >> t & 1u) ? vreg[i] : vec4u{0u, 0u, 0u, 0u};
      if constexpr (TREE) {
        // nor may a drafted token reach the nodes that do not see it: its NaN codes become 0, and the
        // logits of those that see it NaN
        if (drafted) {
          bool any = false;
          v = without_nan_codes(v, any);
          unsigned long long lanes = __ballot(any);
          while (lanes) {
            const int first = __builtin_ctzll(lanes) / kPieces;
            bad |= 1u << ((i * kWave) / kPieces + first);
            lanes &= ~(((1ull << kPieces) - 1) << (first * kPieces));
          }
        }
      }
      *reinterpret_cast<vec4u*>(&s.v[t * D + ((c ^ swizzle(t)) << 4)]) = v;
    }
    if constexpr (TREE) {
      if (drafted) {
        const bool odd = !(fabsf(vs) < __builtin_inff());
        bad |= (uint32_t)__ballot(odd);
        if (odd) vs = 0.0f;
      }
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
    f32x4 S[RT][2], sv[2];
    float top[RT];                               // of log2(p vs), to 1 upwards; vs below 2^-60 counts as that
#pragma unroll
    for (int x = 0; x < RT; ++x) top[x] = -__builtin_inff();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int x = 0; x < RT; ++x) S[x][u] = f32x4{};
#pragma unroll
      for (int j = 0; j < kKeyLoads; ++j) {
        const Q8 k0 = widen8<Q8>(k8[u][j].x, k8[u][j].y), k1 = widen8<Q8>(k8[u][j].z, k8[u][j].w);
#pragma unroll
        for (int x = 0; x < RT; ++x) {
          S[x][u] = mfma16(k0, q[x][2 * j], S[x][u]);
          S[x][u] = mfma16(k1, q[x][2 * j + 1], S[x][u]);
        }
      }
      const f32x4 sc = lds_get<f32x4>(lds_address(s.ks) + (8 * quad + 4 * u) * 4);
      sv[u] = lds_get<f32x4>(lds_address(s.vs) + (8 * quad + 4 * u) * 4);
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        uint32_t mine = now;
        if constexpr (TREE) {
          if (drafted) mine &= (uint32_t)(sees[x] >> (32 * ((tile - draft0) & 1)));
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          S[x][u][r] *= sc[r] * a.scale_log2;
          if constexpr (TREE) {
            if (bad >> (8 * quad + 4 * u + r) & 1u) S[x][u][r] = __builtin_nanf("");
          }
          if (!(mine >> (8 * quad + 4 * u + r) & 1u)) S[x][u][r] = -__builtin_inff();
          top[x] = fmaxf(top[x], S[x][u][r] + (float)__builtin_amdgcn_frexp_expf(fmaxf(fabsf(sv[u][r]), 0x1p-60f)));
        }
      }
    }
    f16x8 p[RT], rest[RT];
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      // p vs in fp16: the reference m moves when p vs could pass 2^15, and then so that
      // the largest is between 2^7 and 2^8
      top[x] = max_quads(top[x]);
      if (__any(top[x] > m[x] + 15.0f)) {
        const bool move = top[x] > m[x] + 15.0f;
        const float nm = move ? top[x] - 8.0f : m[x];
        const float al = move ? __builtin_amdgcn_exp2f(m[x] - nm) : 1.0f;
        m[x] = nm;
        l[x] *= al;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) o[x][t] *= al;
      }
      const float base = m[x] == -__builtin_inff() ? 0.0f : m[x];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float w = __builtin_amdgcn_exp2f(S[x][u][r] - base);
          l[x] += w;
          const float v = w * sv[u][r];
          p[x][4 * u + r] = (_Float16)v;
          if constexpr (kRest) rest[x][4 * u + r] = (_Float16)(v - (float)p[x][4 * u + r]);
        }
    }
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      const i32x2 v8 = lds_read_transposed(vrow ^ (t << 4));
      const f16x8 v = widen8<f16x8>((uint32_t)v8.x, (uint32_t)v8.y);
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        o[x][t] = mfma16(v, p[x], o[x][t]);
        if constexpr (kRest) o[x][t] = mfma16(v, rest[x], o[x][t]);
      }
    }
  }
  if (err) latch_gather(g.ctr, err);
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    l[x] = sum_quads(l[x]);
    if (!has_head[x]) continue;
    const float inv = l[x] != 0.0f ? 1.0f / l[x] : 0.0f;
    const float lse2 = l[x] != 0.0f ? m[x] + log2f(l[x]) : -__builtin_inff();
    const int nth = TREE ? node[x] * (a.heads / a.nodes) + head[x] : head[x];
    const size_t row = (size_t)set * a.heads + nth;
    if (a.splits > 1) {
      const size_t part = row * a.splits + split;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) *reinterpret_cast<f32x4*>(a.part_o + part * D + 16 * t + 4 * quad) = o[x][t] * inv;
      if (quad == 0) a.part_lse[part] = lse2;
      continue;
    }
    uint16_t* out = static_cast<uint16_t*>(a.out) + set * a.out_set_stride + head[x] * a.out_head_stride + 4 * quad;
    if constexpr (TREE) out += node[x] * a.out_node_stride;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      const float v[4] = {o[x][t][0] * inv, o[x][t][1] * inv, o[x][t][2] * inv, o[x][t][3] * inv};
      store4<Q8>(out + 16 * t, v, a.out_aligned);
    }
    if (quad == 0 && a.lse) a.lse[row] = lse2 * kLn2;
  }
}

// Splits so that about kWaveTarget waves run (8 per compute unit), each with at
// least kLeastTiles tiles: a split costs its start and the join's traffic.
// Measured, kernel + join, us, for 16 sets x 2048 tokens x 8 KV heads of 128 (70 MB)
// and 64 sets x 500 blocks of 8 tokens x 2 KV heads of 64 (65 MB):
//   1024 waves 24 + 4 and 28 + 4;  2048 waves 21 + 4 and 21 + 5;  4096 the same;
//   2048 waves of at least 8 tiles 25 + 4 and 22 + 5, of at least 2 as of 4.
// The rows alone take 15 us and 14 us at the rate of a copy of their size.
static AttendPlan plan_heads(int n_sets, int tiles, int head_blocks) {
  constexpr int kWaveTarget = 256 * 8, kLeastTiles = 4;
  AttendPlan p{};
  p.head_blocks = head_blocks;
  const long long base = std::max<long long>(1, (long long)n_sets * p.head_blocks);
  const int want = (int)std::min<long long>(std::min<long long>((kWaveTarget + base - 1) / base, kAttendMaxSplits), std::max(1, tiles / kLeastTiles));
  const int per = (tiles + want - 1) / want;
  p.splits = (tiles + per - 1) / per;
  p.split_keys = per * kTok;
  return p;
}

AttendPlan plan_attend_heads(int n_sets, int tokens, int heads, int kv_heads) {
  const int shared = heads / kv_heads;
  return plan_heads(n_sets, std::max(1, (tokens + kTok - 1) / kTok),
                    kv_heads * ((shared + kHeadsPerWave - 1) / kHeadsPerWave));
}

// Groups of 16 rows that a wave of a tree takes.
static int tree_groups(int shared) { return shared > 32 ? 4 : (shared > 16 ? 2 : 1); }

AttendPlan plan_tree_heads(int n_sets, int tiles, int rows, int kv_heads) {
  const int shared = rows / kv_heads, per = kHeadsPerWave * tree_groups(shared);
  return plan_heads(n_sets, tiles, kv_heads * ((shared + per - 1) / per));
}

template <typename Q8, int D, int RT, bool TREE>
static hipError_t launch_heads(const GroupDev& g, const AttendDev& a, int n_sets, hipStream_t s) {
  const int items = n_sets * a.head_blocks * a.splits;
  const int blocks = (items + kHeadWaves - 1) / kHeadWaves;
  k_attend_heads<Q8, D, RT, TREE><<<blocks, kHeadWaves * kWave, 0, s>>>(g, a, items);
  return hipGetLastError();
}

template <typename Q8>
static hipError_t launch_heads_of(const GroupDev& g, const AttendDev& a, int n_sets, int head_dim, hipStream_t s) {
  return head_dim == 64 ? launch_heads<Q8, 64, 1, false>(g, a, n_sets, s) : launch_heads<Q8, 128, 1, false>(g, a, n_sets, s);
}

hipError_t launch_attend_heads(const GroupDev& g, const AttendDev& a, int type, int n_sets, int head_dim,
                               hipStream_t s) {
  return type == ULA_BF16 ? launch_heads_of<bf16x8>(g, a, n_sets, head_dim, s)
                          : launch_heads_of<f16x8>(g, a, n_sets, head_dim, s);
}

template <typename Q8, int D>
static hipError_t launch_tree_of(const GroupDev& g, const AttendDev& a, int n_sets, hipStream_t s) {
  switch (tree_groups(a.heads / a.kv_heads)) {
    case 1: return launch_heads<Q8, D, 1, true>(g, a, n_sets, s);
    case 2: return launch_heads<Q8, D, 2, true>(g, a, n_sets, s);
    default: return launch_heads<Q8, D, 4, true>(g, a, n_sets, s);
  }
}

hipError_t launch_tree_heads(const GroupDev& g, const AttendDev& a, int type, int n_sets, int head_dim, hipStream_t s) {
  if (type == ULA_BF16) return head_dim == 64 ? launch_tree_of<bf16x8, 64>(g, a, n_sets, s) : launch_tree_of<bf16x8, 128>(g, a, n_sets, s);
  return head_dim == 64 ? launch_tree_of<f16x8, 64>(g, a, n_sets, s) : launch_tree_of<f16x8, 128>(g, a, n_sets, s);
}

}  // namespace ula
