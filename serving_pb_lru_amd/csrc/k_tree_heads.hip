// Attention of trees of drafted tokens over rows in the heads format: every node of
// a set's tree attends to the set's selected tokens and to the drafted tokens that
// its mask has.
//
// As in k_attend_heads.hip, with k8, v8 a token's codes, ks, vs its scales and
// c = scale log2(e), but the value scale goes into the exponent:
//   T_j = c ks_j (q . k8_j) + log2 |vs_j|,  w_j = 2^(T_j - m),
//   o = sum_j w_j (+-v8_j) / l,  l = sum_j w_j / |vs_j|,  lse = (m + log2 l) ln 2
// so that w_j is what the second product takes, in two fp16 parts whatever the type of the
// results (bf16 ones of one part were 2.9e-4 of their size from those of weights in 32
// bits, 6e-5 so; 16 sets x 16 nodes x 2048 tokens x 32 heads of 128 34.7 -> 35.3 us a call):
// a scaled sum, a maximum, a difference, an exponential, a fused add and the roundings
// for each logit. (With 64 query rows to a key, vector
// instructions on logits bound this, not bytes; masks, a product with vs and an
// exponent of it for each logit, in four waves that each had their own rows' tokens, took
// 410 us a call where this takes 130 us for 32 sets x 61 nodes x 500 blocks of 8 tokens x
// 24 heads of 64, fp16, and 80 us where this takes 35 us, 30 of them the kernel's, for 16
// sets x 16 nodes x 2048 tokens x 32 heads of 128 over 8, bf16. In the first of the two vector
// instructions fill 57% of a SIMD's cycles and matrix instructions 22%; its form, 64 rows of 64
// channels, spills 17 registers, most of them where drafted tiles branch; 48 rows spill none
// and take 134 us.) m follows the largest w as
// there: it moves, to leave the largest at 2^8, when one could pass 2^15, which each lane
// tells from its own tokens. A negative vs turns the signs of its codes; one below 2^-80
// makes them 0 (so l, which adds up to 2^95 for a token then, stays finite); from the first
// beyond 2^40 either way on, l adds up powers of its own (w / |vs| would vanish beside a
// token of large scale); one that is not finite, or a NaN code in a drafted token's values,
// makes T NaN, which a node that does not see the token replaces with its mask.
//
// A workgroup is one KV head's RT x 16 query rows (of nodes and heads) and one range of
// tokens; its four or eight waves take every fourth or eighth tile of 32 tokens, each by
// itself as there, and join their results in LDS. So a set's tokens are split over fewer
// workgroups, whose parts go through memory, than over waves. With up to 32 rows q is in
// LDS, and a tile's products with all of them come first, a half of the keys at a time:
// so two waves of 32 rows and heads of 128 fit a SIMD (the second of the two above: 32 us a
// call, weights in one part, 36 us with one wave and q in registers). With more rows q stays
// in registers, which leaves fewer accumulators waiting (the first of the two: 130 us so,
// 132 us with q in LDS).
#include <algorithm>
#include <cmath>

#include "row_format.h"

namespace ula {

constexpr int kTok = kTileTokens;
constexpr float kLeastScale = 0x1p-80f;        // of a value; what is below it counts as 0

// Waves on a SIMD, by registers, and waves of a workgroup.
constexpr int tree_waves(int dim, int groups) { return dim == 64 ? (groups == 1 ? 3 : 2) : (groups <= 2 ? 2 : 1); }
constexpr int tree_group(int dim, int groups) { return dim == 128 && groups == 2 ? 8 : 4; }

template <typename Q8, int D, int RT>
__global__ __launch_bounds__(tree_group(D, RT) * kWave, tree_waves(D, RT)) void k_tree_heads(GroupDev g, AttendDev a) {
  constexpr int kTreeWaves = tree_group(D, RT);
  constexpr int kPieces = D / 16;              // 16-byte pieces of a token's key or value
  constexpr int kKeyLoads = D / 64;            // pieces of its key a lane holds (a quarter)
  constexpr int kValLoads = kTok * kPieces / kWave;
  constexpr int kRows = 16 * RT;
  constexpr bool kKeepValues = D == 64;        // of a tile, widened, or else the weights of all rows: the fewer registers
  constexpr int kRow = D + 4;                  // floats of a row in the join
  constexpr bool kAhead = RT <= 2;             // q in LDS, the first products of all rows at once
  struct WaveLds {
    alignas(1024) uint8_t v[kTok * D];
    alignas(16) float scale[kTok], shift[kTok], inverse[kTok];   // c ks, log2 |vs|, 1 / |vs|
  };
  union Lds {
    WaveLds wave[kTreeWaves];
    float o[kTreeWaves][16][kRow];
  };
  __shared__ Lds s;
  __shared__ float s_lse[kTreeWaves][kRows];
  __shared__ bool s_ok[kTreeWaves];
  __shared__ Q8 s_q[kAhead ? RT * D / 32 : 1][kWave];   // q in operand order, the same for all waves
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int quad = lane / 16, col = lane % 16;
  WaveLds& mine_lds = s.wave[wave];

  // consecutive items (which share rows) on one XCD at about the same time
  int item = blockIdx.x;
  {
    const int per = gridDim.x / 8, rest = gridDim.x % 8, x = item % 8;
    item = x * per + min(x, rest) + item / 8;
  }
  const int unit = item % a.head_blocks;
  const int split = item / a.head_blocks % a.splits;
  const int set = item / a.head_blocks / a.splits;
  const int rows = a.heads / a.kv_heads;       // of one KV head: nodes x query heads
  const int per = (int)a.by_heads.d;           // query heads of a node per KV head
  const int blocks = (rows + kRows - 1) / kRows;
  const int kvh = unit / blocks, row0 = unit % blocks * kRows;
  const int block = 1 << a.block_shift;
  const int draft_blocks = (a.nodes + block - 1) >> a.block_shift;
  const int all_tiles = a.history_tiles + (a.nodes + kTok - 1) / kTok;
  const int tile0 = split * (a.split_keys / kTok) + wave;
  const int tile1 = min(all_tiles, (split + 1) * (a.split_keys / kTok));
  const ReaderState state = reader_state(g);

  const uint8_t* pool = g.pool + (size_t)a.layer * g.row_bytes;
  const int head_at = kvh * block * D;                         // this head's keys inside a row
  const int val_at = a.kv_heads * block * D;                   // from keys to values
  const int scale_at = 2 * val_at + 4 * kvh;
  int err = 0;

  // Lookups and loads have no branches, so that the compiler knows how many are in flight behind the ones it
  // waits for: what is not there, or is of a tile behind the last, reads something else that is.
  const int32_t* sel = a.sel_k ? a.sel : reinterpret_cast<const int32_t*>(g.ctr);
  // the selection entry of this lane's token (lane % 32) of a tile, 0 in the place of one that is not there
  auto entry_of = [&](int tile, bool& there) {
    const int t = tile * kTok + lane % kTok;
    there = tile < min(tile1, a.history_tiles) && t < a.sel_k << a.block_shift;
    return there ? set * a.sel_k + (t >> a.block_shift) : 0;
  };
  auto look = [&](int tile) -> Lookup {
    bool there;
    const int r = entry_of(tile, there);
    return {g.res[r], sel[r]};                                 // res has room for every selection of the engine
  };
  auto slot_at = [&](int tile, Lookup at) {
    bool there;
    const int r = entry_of(tile, there);
    if (!there) at.la = -1;
    if (r >= a.n_res) at.res = make_uint2(kAbsent, kAbsent);
    return slot_of(g, at, a.n_res, err);
  };
  struct Loads {
    vec4u k[2][kKeyLoads], v[kValLoads];
    float ks, vs;
    int used;                                                  // tokens in use of this lane's token's block
  };
  Loads in;                                                    // of the next tile
  // loads of a tile whose slots are known; tokens that are not there read slot 0 or the last drafted token,
  // which `used` leaves out
  auto load = [&](int tile, uint32_t slot) {
    const uint8_t* from = pool;
    uint32_t stride = (uint32_t)g.slot_bytes;
    bool there = slot != kAbsent;
    if (!there) slot = 0;
    if (tile >= a.history_tiles) {                             // blocks of drafted tokens in the place of slots
      const int d = (tile - a.history_tiles) * kTok + lane % kTok;
      there = d < a.nodes && tile < tile1;
      slot = (uint32_t)(set * draft_blocks + (min(d, a.nodes - 1) >> a.block_shift));
      from = a.drafts;
      stride = (uint32_t)a.draft_stride;
    }
    const uint8_t* row = from + (uint64_t)slot * stride + scale_at;
    in.ks = *reinterpret_cast<const float*>(row);
    in.vs = *reinterpret_cast<const float*>(row + 4 * a.kv_heads);
    const int count = *reinterpret_cast<const int32_t*>(row - 4 * kvh + 8 * a.kv_heads);
    uint32_t ksl[2], vsl[kValLoads];                           // all exchanges in flight together
#pragma unroll
    for (int u = 0; u < 2; ++u) ksl[u] = (uint32_t)__shfl((int)slot, 8 * (col / 4) + 4 * u + col % 4, kWave);
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) vsl[i] = (uint32_t)__shfl((int)slot, (i * kWave + lane) / kPieces, kWave);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = 8 * (col / 4) + 4 * u + col % 4;
      const uint8_t* p = from + (uint64_t)ksl[u] * stride + (head_at + (t & (block - 1)) * D + quad * 16);
#pragma unroll
      for (int j = 0; j < kKeyLoads; ++j) in.k[u][j] = *reinterpret_cast<const vec4u*>(p + 64 * j);
    }
#pragma unroll
    for (int i = 0; i < kValLoads; ++i) {
      const int t = (i * kWave + lane) / kPieces, c = lane % kPieces;
      const uint8_t* p = from + (uint64_t)vsl[i] * stride + (head_at + val_at + (t & (block - 1)) * D + 16 * c);
      in.v[i] = *reinterpret_cast<const vec4u*>(p);
    }
    in.used = there ? count : 0;
  };

  const Lookup first = look(tile0);
  Lookup next = look(tile0 + kTreeWaves);
  // this lane's query rows and what their nodes see of the drafted tokens
  unsigned long long sees[RT];
  constexpr int kQ = D / 32;                   // operands of a row group
  Q8 q[kAhead ? 1 : RT][kQ];
  // row hi of q from this lane's first channel on; operand j is 64 (j / 2) + 8 (j % 2) further
  auto query = [&](int hi) {
    const int node = (int)a.by_heads.div(hi), head = kvh * per + hi - node * per;
    return static_cast<const uint16_t*>(a.q) + set * a.q_set_stride + node * a.q_node_stride + head * a.q_head_stride +
           16 * quad;
  };
  auto operand = [&](const uint16_t* p) { return a.q_aligned ? load8<Q8, true>(p) : load8<Q8, false>(p); };
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const int hi = row0 + 16 * x + col;
    sees[x] = 0;
    if constexpr (!kAhead) {
#pragma unroll
      for (int j = 0; j < kQ; ++j) q[x][j] = Q8{};
    }
    if (hi < rows) {
      sees[x] = a.visible[(size_t)set * a.nodes + (int)a.by_heads.div(hi)];
      if constexpr (!kAhead) {
        const uint16_t* p = query(hi);
#pragma unroll
        for (int j = 0; j < kQ; ++j) q[x][j] = operand(p + 64 * (j / 2) + 8 * (j % 2));
      }
    }
  }
  if constexpr (kAhead) {
    for (int e = wave; e < RT * kQ; e += kTreeWaves) {
      const int hi = row0 + 16 * (e / kQ) + col, j = e % kQ;
      s_q[e][lane] = hi < rows ? operand(query(hi) + 64 * (j / 2) + 8 * (j % 2)) : Q8{};
    }
    __syncthreads();
  }
  f32x4 o[RT][D / 16];
  // bit x: value scales beyond 2^40 either way have come to the lane's row x, so that w / |vs| may vanish
  uint32_t wide = 0;
  float m[RT], base[RT], l[RT];                // base: m, or 0 as long as there is none
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    m[x] = -__builtin_inff();
    base[x] = l[x] = 0.0f;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) o[x][t] = f32x4{};
  }
  // transposed reads: this lane names token 8 quad + col / 2, piece 0; piece x is ^ (x << 4)
  const int vtok = 8 * quad + col / 2;
  auto swizzle = [](int tok) { return D == 128 ? (tok >> 1) & 7 : (tok >> 2) & 1; };
  const uint32_t vrow = lds_address(mine_lds.v) + vtok * D + (swizzle(vtok) << 4) + (col & 1) * 8;

  float minus = -1.0f;                         // one the compiler does not know: a fused step takes it, a difference two
  asm volatile("" : "+s"(minus));
  int ok = 0;
  if (lane == 0) ok = reader_ready(g, state, a.want_flag);
  ok = __builtin_amdgcn_readfirstlane(ok);     // the same in every wave but for a race with an error: see the join
  // q is there before the tiles' loads start: a wait for it in the loop would be one for them too
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    asm volatile("" : "+v"(sees[x]));
    if constexpr (!kAhead) {
#pragma unroll
      for (int j = 0; j < kQ; ++j) asm volatile("" : "+v"(q[x][j]));
    }
  }
  if (ok) load(tile0, slot_at(tile0, first));
#pragma unroll 1
  for (int tile = tile0; ok && tile < tile1; tile += kTreeWaves) {
    const bool drafted = tile >= a.history_tiles;
    const uint32_t now = (uint32_t)__ballot((lane % kTok & (block - 1)) < in.used);   // bit per token
    {
      const bool use = now >> (lane % kTok) & 1u;
      const float vs = in.vs, big = fmaxf(fabsf(vs), kLeastScale);   // NaN: that, and the shift says so
      float shift = __builtin_amdgcn_logf(big);
      if (!(fabsf(vs) < __builtin_inff())) shift = __builtin_nanf("");
      // Most tiles go to LDS as they are. Else: a token out of use must not reach the products (0 x NaN); codes of
      // negative scales change sign, those of vanishing ones are 0; NaN codes of drafted tokens are 0 as well.
      if (drafted || __any(!use || !(vs >= 0x1p-40f && vs <= 0x1p40f))) {
        const uint32_t flips = (uint32_t)__ballot(vs < 0.0f), keep = now & (uint32_t)__ballot(fabsf(vs) >= kLeastScale);
        uint32_t nan = 0;                                      // drafted tokens with NaN codes
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < kKeyLoads; ++j)
            if (!(now >> (8 * (col / 4) + 4 * u + col % 4) & 1u)) in.k[u][j] = vec4u{0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < kValLoads; ++i) {
          const int t = (i * kWave + lane) / kPieces;
          if (!(keep >> t & 1u)) in.v[i] = vec4u{0u, 0u, 0u, 0u};
          const uint32_t sign = (flips >> t & 1u) * 0x80808080u;
#pragma unroll
          for (int w = 0; w < 4; ++w) in.v[i][w] ^= sign;
          if (drafted) {
            bool any = false;
            in.v[i] = without_nan_codes(in.v[i], any);
            unsigned long long lanes = __ballot(any);
            while (lanes) {
              const int at = __builtin_ctzll(lanes) / kPieces;
              nan |= 1u << (i * kWave / kPieces + at);
              lanes &= ~(((1ull << kPieces) - 1) << (at * kPieces));
            }
          }
        }
        const uint32_t far = (uint32_t)__ballot(use && fabsf(shift) > 40.0f);
        if (far) {
#pragma unroll
          for (int x = 0; x < RT; ++x)
            if (far & (drafted ? (uint32_t)(sees[x] >> (32 * ((tile - a.history_tiles) & 1))) : ~0u)) wide |= 1u << x;
        }
        if (nan >> (lane % kTok) & 1u) shift = __builtin_nanf("");
      }
#pragma unroll
      for (int i = 0; i < kValLoads; ++i) {
        const int t = (i * kWave + lane) / kPieces, c = lane % kPieces;
        *reinterpret_cast<vec4u*>(&mine_lds.v[t * D + ((c ^ swizzle(t)) << 4)]) = in.v[i];
      }
      if (lane < kTok) {
        mine_lds.scale[lane] = use ? in.ks * a.scale_log2 : 0.0f;
        mine_lds.shift[lane] = use ? shift : -__builtin_inff();
        mine_lds.inverse[lane] = use ? __builtin_amdgcn_rcpf(big) : 0.0f;
      }
    }
    Q8 kw[kAhead ? 1 : 2][2 * kKeyLoads];
    f32x4 products[kAhead ? RT : 1][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Q8(&k)[2 * kKeyLoads] = kw[kAhead ? 0 : u];
#pragma unroll
      for (int j = 0; j < kKeyLoads; ++j) {
        k[2 * j] = widen8<Q8>(in.k[u][j].x, in.k[u][j].y);
        k[2 * j + 1] = widen8<Q8>(in.k[u][j].z, in.k[u][j].w);
      }
      if constexpr (kAhead) {
#pragma unroll
        for (int x = 0; x < RT; ++x) products[x][u] = f32x4{};
#pragma unroll
        for (int j = 0; j < 2 * kKeyLoads; ++j)
#pragma unroll
          for (int x = 0; x < RT; ++x) products[x][u] = mfma16(k[j], s_q[x * kQ + j][lane], products[x][u]);
        __builtin_amdgcn_sched_barrier(0);         // the widened keys' registers are free from here
      }
    }
    // loads into the registers that are free now, and the slots of the tile after that
    {
      const uint32_t slot = slot_at(tile + kTreeWaves, next);
      next = look(tile + 2 * kTreeWaves);
      load(tile + kTreeWaves, slot);
    }
    if (now == 0) continue;
    f32x4 scale[2], shift[2], inverse[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      scale[u] = lds_get<f32x4>(lds_address(mine_lds.scale) + (8 * quad + 4 * u) * 4);
      shift[u] = lds_get<f32x4>(lds_address(mine_lds.shift) + (8 * quad + 4 * u) * 4);
      if constexpr (!kAhead) inverse[u] = lds_get<f32x4>(lds_address(mine_lds.inverse) + (8 * quad + 4 * u) * 4);
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int x = 0; x < RT; ++x)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) products[x][u][r] = __builtin_fmaf(products[x][u][r], scale[u][r], shift[u][r]);
      __builtin_amdgcn_sched_barrier(0);           // and the factors'
#pragma unroll
      for (int u = 0; u < 2; ++u) inverse[u] = lds_get<f32x4>(lds_address(mine_lds.inverse) + (8 * quad + 4 * u) * 4);
    }
    i32x2 v8[D / 16];                            // on their way during the first product
#pragma unroll
    for (int t = 0; t < D / 16; ++t) v8[t] = lds_read_transposed(vrow ^ (t << 4));
    auto values = [&](int at) { return widen8<f16x8>((uint32_t)v8[at].x, (uint32_t)v8[at].y); };
    auto add = [&](int x, int at, const f16x8& v, const f16x8& p, const f16x8& rest) {
      o[x][at] = mfma16(v, p, o[x][at]);
      o[x][at] = mfma16(v, rest, o[x][at]);
    };
    const bool any_wide = __any(wide);
    f16x8 v[kKeepValues ? D / 16 : 1], p[kKeepValues ? 1 : RT], rest[kKeepValues ? 1 : RT];
    if constexpr (kKeepValues) {
#pragma unroll
      for (int t = 0; t < D / 16; ++t) v[t] = values(t);
    }
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      constexpr auto at = [](int i) { return kKeepValues ? 0 : i; };
      f32x4 T[2] = {};
      float top = -__builtin_inff();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if constexpr (kAhead) {
          T[u] = products[x][u];
        } else {
#pragma unroll
          for (int j = 0; j < 2 * kKeyLoads; ++j) T[u] = mfma16(kw[u][j], q[x][j], T[u]);
#pragma unroll
          for (int r = 0; r < 4; ++r) T[u][r] = __builtin_fmaf(T[u][r], scale[u][r], shift[u][r]);
        }
      }
      if (drafted) {
        const uint32_t mine = (uint32_t)(sees[x] >> (32 * ((tile - a.history_tiles) & 1))) >> (8 * quad);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!(mine >> e & 1u)) T[e / 4][e % 4] = -__builtin_inff();
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, T[e / 4][e % 4]);
      if (__any(top > m[x] + 15.0f)) {
        top = max_quads(top);
        const bool move = top > m[x] + 15.0f;
        const float nm = move ? top - 8.0f : m[x];
        const float fall = move ? m[x] - nm : 0.0f, al = near_power(fall);
        m[x] = nm;
        base[x] = nm == -__builtin_inff() ? 0.0f : nm;
        l[x] = l[x] * far_power(fall) * al;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) o[x][t] *= al;
      }
      float plus = 0.0f;                         // what l gains
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        f32x2 w = {__builtin_amdgcn_exp2f(T[e / 4][e % 4] - base[x]), __builtin_amdgcn_exp2f(T[e / 4][e % 4 + 1] - base[x])};
        plus = __builtin_fmaf(w.x, inverse[e / 4][e % 4], plus);
        plus = __builtin_fmaf(w.y, inverse[e / 4][e % 4 + 1], plus);
        f16x2 hi = __builtin_convertvector(w, f16x2);
        asm("" : "+v"(hi));                      // one rounding for both uses
        rest[at(x)][e] = (_Float16)__builtin_fmaf((float)hi.x, minus, w.x);
        rest[at(x)][e + 1] = (_Float16)__builtin_fmaf((float)hi.y, minus, w.y);
        p[at(x)][e] = hi.x;
        p[at(x)][e + 1] = hi.y;
      }
      if (any_wide) {                            // w / |vs| may vanish
        float more = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f32x4 of_scale = kAhead ? lds_get<f32x4>(lds_address(mine_lds.shift) + (8 * quad + 4 * u) * 4) : shift[u];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (T[u][r] != -__builtin_inff()) more += __builtin_amdgcn_exp2f(T[u][r] - of_scale[r] - base[x]);
        }
        plus = wide >> x & 1u ? more : plus;
        asm volatile("" : "+v"(plus));           // a branch, not a selection
      }
      l[x] += plus;
      if constexpr (kKeepValues) {
#pragma unroll
        for (int t = 0; t < D / 16; ++t) add(x, t, v[t], p[0], rest[0]);
      }
    }
    if constexpr (!kKeepValues) {
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        const f16x8 vt = values(t);
#pragma unroll
        for (int x = 0; x < RT; ++x) add(x, t, vt, p[x], rest[x]);
      }
    }
  }
  if (err) latch_gather(g.ctr, err);

  // The waves' results as one, in units of the largest log-sum: m, which follows the largest product with a
  // value scale, may differ by more than what 32 bits hold.
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    l[x] = sum_quads(l[x]);
    if (quad == 0) s_lse[wave][16 * x + col] = l[x] != 0.0f ? m[x] + __builtin_amdgcn_logf(l[x]) : -__builtin_inff();
  }
  if (lane == 0) s_ok[wave] = ok;
  __syncthreads();
  for (int w = 0; w < kTreeWaves; ++w)
    if (!s_ok[w]) return;                                      // some wave found an error: every thread sees that
  constexpr int kLanes = kTreeWaves * kWave / 16, kPer = D / kLanes;   // threads of a row in the stores, channels of each
  const int orow = threadIdx.x / kLanes, ch = threadIdx.x % kLanes * kPer;
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    float most = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < kTreeWaves; ++w) most = fmaxf(most, s_lse[w][16 * x + col]);
    const float mine = __builtin_amdgcn_exp2f(m[x] - (most == -__builtin_inff() ? 0.0f : most));
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
      *reinterpret_cast<f32x4*>(&s.o[wave][col][16 * t + 4 * quad]) = o[x][t] * mine;
    __syncthreads();
    float sum = 0.0f, peak = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < kTreeWaves; ++w) peak = fmaxf(peak, s_lse[w][16 * x + orow]);
    const float from = peak == -__builtin_inff() ? 0.0f : peak;
#pragma unroll
    for (int w = 0; w < kTreeWaves; ++w) sum += __builtin_amdgcn_exp2f(s_lse[w][16 * x + orow] - from);
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    const float lse2 = sum != 0.0f ? from + log2f(sum) : -__builtin_inff();
    const int hi = row0 + 16 * x + orow;
    if (hi < rows) {
      float out[kPer];
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        out[c] = s.o[0][orow][ch + c];
#pragma unroll
        for (int w = 1; w < kTreeWaves; ++w) out[c] += s.o[w][orow][ch + c];
        out[c] *= inv;
      }
      const int node = (int)a.by_heads.div(hi), head = kvh * per + hi - node * per;
      const size_t row = (size_t)set * a.heads + node * (a.heads / a.nodes) + head;
      if (a.splits > 1) {
        const size_t part = row * a.splits + split;
#pragma unroll
        for (int c = 0; c < kPer; c += 4)
          *reinterpret_cast<f32x4*>(a.part_o + part * D + ch + c) = f32x4{out[c], out[c + 1], out[c + 2], out[c + 3]};
        if (ch == 0) a.part_lse[part] = lse2;
      } else {
        uint16_t* to = static_cast<uint16_t*>(a.out) + set * a.out_set_stride + node * a.out_node_stride + head * a.out_head_stride + ch;
#pragma unroll
        for (int c = 0; c < kPer; c += 4) store4<Q8>(to + c, out + c, a.out_aligned);
        if (ch == 0 && a.lse) a.lse[row] = lse2 * kLn2;
      }
    }
    __syncthreads();
  }
}

// How a call's rows and tokens are split over workgroups: 16 to 64 rows each and the
// number of splits, with the least estimated time in us. A workgroup takes 10 for its
// start and end, and for each of a wave's tiles the time in the table, that of a compute
// unit full of them; the join takes 7 and its traffic.
// Measured, us a call, rows of a workgroup 16, 32, 48, 64 (sets x rows of a KV head):
//   32 sets x 732 rows x 2 KV heads of 64, 4061 tokens, fp16, one split: 182 163 134 132; two: 185 179 150 139
//   16 sets x 64 rows x 8 KV heads of 128, 2064 tokens, bf16, one split: 43 33 47 60; two: 52 45 57 44
//   32 sets x 128 rows x 8 KV heads of 128, 1056 tokens, bf16, one split: 84 71 84 73; two: 104 104 109 97
//   1 set x 32 rows x 8 KV heads of 128, 4104 tokens, bf16, 1, 2, 4 splits of 32 rows: 45 32 25
//   1 set x 512 rows x 1 KV head of 128, 2064 tokens, fp16, one split: 30 29 46 58; four: 26 24 26 30
AttendPlan plan_tree_heads(int n_sets, int tiles, int rows, int kv_heads, int head_dim) {
  static constexpr double kTileUs[2][4] = {{1.1, 1.25, 1.75, 2.3}, {1.6, 2.1, 1.9, 2.7}};   // heads of 64, of 128
  constexpr double kStartUs = 10.0;
  AttendPlan best{};
  const int of_head = rows / kv_heads;
  double best_cost = 0;
  for (int groups = 1; groups <= 4; ++groups) {
    if (groups > 1 && of_head <= 16 * (groups - 1)) break;         // a group without rows
    const int head_blocks = kv_heads * ((of_head + 16 * groups - 1) / (16 * groups));
    const int waves = tree_waves(head_dim, groups), group = tree_group(head_dim, groups);
    for (int want = 1; want <= std::max(1, std::min(tiles / group, 64)); ++want) {
      const int per = (tiles + want - 1) / want, splits = (tiles + per - 1) / per;
      if (splits != want) continue;                                // the same split as a smaller one
      const double rounds = std::max(1.0, (double)n_sets * head_blocks * splits / (256.0 * waves * 4 / group));   // of full units
      double cost = rounds * (kStartUs + std::ceil((double)per / group) * kTileUs[head_dim / 128][groups - 1]);
      if (splits > 1) cost += 7 + (double)n_sets * rows * splits * head_dim * 2e-6;
      if (best.splits == 0 || cost < best_cost) {
        best_cost = cost;
        best = {splits, per * kTok, head_blocks, groups};
      }
    }
  }
  return best;
}

template <typename Q8, int D, int RT>
static hipError_t launch_groups(const GroupDev& g, const AttendDev& a, int n_sets, hipStream_t s) {
  k_tree_heads<Q8, D, RT><<<n_sets * a.head_blocks * a.splits, tree_group(D, RT) * kWave, 0, s>>>(g, a);
  return hipGetLastError();
}

template <typename Q8, int D>
static hipError_t launch_dim(const GroupDev& g, const AttendDev& a, int n_sets, hipStream_t s) {
  switch (a.groups) {
    case 1: return launch_groups<Q8, D, 1>(g, a, n_sets, s);
    case 2: return launch_groups<Q8, D, 2>(g, a, n_sets, s);
    case 3: return launch_groups<Q8, D, 3>(g, a, n_sets, s);
    default: return launch_groups<Q8, D, 4>(g, a, n_sets, s);
  }
}

hipError_t launch_tree_heads(const GroupDev& g, const AttendDev& a, int type, int n_sets, int head_dim, hipStream_t s) {
  if (type == ULA_BF16) return head_dim == 64 ? launch_dim<bf16x8, 64>(g, a, n_sets, s) : launch_dim<bf16x8, 128>(g, a, n_sets, s);
  return head_dim == 64 ? launch_dim<f16x8, 64>(g, a, n_sets, s) : launch_dim<f16x8, 128>(g, a, n_sets, s);
}

}  // namespace ula
