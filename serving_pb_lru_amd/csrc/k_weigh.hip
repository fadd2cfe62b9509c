// The softmax weight that each selected entry got, summed over a set's query rows,
// read from the GPU pool where the keys lie, and added to a score for each address.
//
// With S_rj the logit of row r and key j (k_attend.hip), in powers of two, and lse_r
// the row's log-sum from the attention that has run:
//   share_j = sum_r 2^(S_rj - lse_r log2(e)),   score[address of j] += round(2^32 share_j)
// The keys are read again: their weights need the whole row's log-sum, which an
// attention split over workgroups has only once it is joined. Scores are whole
// numbers in units of 2^-32 because adds of those commute: an address that several
// sets list gets the same score whatever the order. Negative scores are added to like
// others: to leave them alone, their signs read with the keys, took 9% more (256 sets
// x 2048 keys x 64 heads 102 -> 112 us a call: one more line for each key).
//
// Products are taken as Q K^T, so that a lane's column is one key: its scales are
// the lane's own, the sum over rows stays in the lane, and only its parts in the
// other half (quads) of the wave are added at the end. Accumulators, logits, and
// sums are in 32 bits; e4m3 codes are exact in bf16 and fp16.
#include <algorithm>
#include <type_traits>

#include "row_format.h"

namespace ula {

// A share is at most its rows, nodes x heads <= 2^16 for each token, with those rows' own log-sums; with
// others it may be anything, and 2^22 is the most that one entry of a selection adds. A NaN adds 0.
__device__ __forceinline__ unsigned long long score_units(float share) {
  const float x = fminf(fmaxf(share, 0.0f), 0x1p22f);   // NaN: 0
  return (unsigned long long)(long long)rint((double)x * 0x1p32);
}

// The value again, as one the compiler cannot trace back: sums of it and a constant
// become instruction offsets, not registers kept across the loop.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Whether a row of this log-sum counts.
__device__ __forceinline__ bool counts(float lse) { return fabsf(lse) < __builtin_inff(); }

// ---- latent rows ---------------------------------------------------------------
// A wave takes 32 keys, a workgroup 8 x 32 at a time and up to 64 rows, whose q is in
// LDS ([row][576], rows padded by 16 bytes for the banks), all of them for every
// key group; more rows go chunk by chunk over the same keys. A key's codes stay in
// registers as they are until a block of 128 channels is widened for both 32-row
// products; a block's registers then take the next key group's.
// Bound by the lines that a compute unit can have outstanding: 256 sets x 2048 keys x 64
// heads take 90 us, in which the units ask for 530 MB (344 MB of rows, whose ends share
// lines) and wait about 860 cycles for each line. (240 us a call with branches around the loads, whose
// waits were for all of them, where this takes 104 us a call; 125 us with 16 x 16 products, 64 bytes
// of a row at a time, and spilled registers; 109 us with rows of q asked for once their log-sum was
// known; 108 us with tiles of whole rows in LDS, five of them on their way, that all waves share.
// Of 1024 query rows: 16 sets x 2048 keys 99 us a call, 127 us with a pause in the keys' loads
// between chunks of rows, 144 us with tiles in LDS.)
constexpr int kWeighWaves = 8;
constexpr int kWeighKeys = 32;                       // of a wave
constexpr int kWeighGroup = kWeighWaves * kWeighKeys;
constexpr int kWeighRows = 64;                       // most at a time
constexpr int kWeighMaxGroups = 8;                   // key groups of a workgroup

__device__ __align__(16) uint8_t g_no_row[kLatentRow];   // zeros

template <typename Q8>
struct WeighLds {
  // fp16: rotary channels as the sum of two bf16 values, since the keys' are bf16
  static constexpr int kRopeParts = std::is_same_v<Q8, bf16x8> ? 1 : 2;
  static constexpr int kRowBytes = 2 * (kLatent + kRope * kRopeParts) + 16;
  alignas(16) uint8_t q[kWeighRows * kRowBytes];
  alignas(16) float minus[kWeighRows];               // -lse log2(e); -inf for rows that do not count
  float share[kWeighWaves][kWeighMaxGroups][kWeighKeys];
  int ok;
};

// HT: rows at a time, in 32s.
template <typename Q8, int HT>
__global__ __launch_bounds__(kWeighWaves * kWave, 2) void k_weigh_latent(GroupDev g, WeighDev a) {
  using Lds = WeighLds<Q8>;
  constexpr int kRows = 32 * HT;
  __shared__ Lds s;
  const int lane = lane_id(), half = lane / 32, col = lane % 32;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int set = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const int group0 = split * a.groups;                // of 256 keys
  const int groups = min(a.groups, (a.k + kWeighGroup - 1) / kWeighGroup - group0);
  const ReaderState state = reader_state(g);
  if (threadIdx.x == 0) s.ok = reader_ready(g, state, a.want_flag);

  const uint8_t* pool = g.pool + (size_t)a.layer * g.row_bytes;
  int err = 0;
  // This lane's key (both halves the same one) of a group. Lookups and loads have no branches, so that the
  // compiler knows how many are in flight behind the ones it waits for: a key that is not there looks entry 0 up
  // and reads zeros.
  auto key_of = [&](int group) { return (group0 + group) * kWeighGroup + wave * kWeighKeys + col; };
  // step: a chunk of rows' key group; chunks follow each other without a pause
  const int steps = (a.rows + kRows - 1) / kRows * groups;
  auto entry_of = [&](int step) {
    const int key = key_of(step % groups);
    return step < steps && key < a.k ? set * a.k + key : -1;
  };
  auto look = [&](int step) -> Lookup {
    const int r = max(entry_of(step), 0);
    return {g.res[r], a.sel[r]};                      // res has room for every selection of the engine
  };
  auto row_at = [&](int step, Lookup at) -> const uint8_t* {
    const int r = entry_of(step);
    if (r < 0) at.la = -1;
    if (r >= a.n_res) at.res = make_uint2(kAbsent, kAbsent);
    const uint32_t slot = slot_of(g, at, a.n_res, err);
    return slot != kAbsent ? pool + (size_t)slot * g.slot_bytes : g_no_row;
  };
  // 16-byte pieces of the lane's half: pieces 2 j + half of each block, and of the rotary channels
  vec4u code[kLatentGroups][4], rope[4];
  f32x4 scale;
  auto load_block = [&](const uint8_t* row, int b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) code[b][j] = *reinterpret_cast<const vec4u*>(row + b * kScaleGroup + (2 * j + half) * 16);
  };
  auto load_rest = [&](const uint8_t* row) {
#pragma unroll
    for (int j = 0; j < 4; ++j) rope[j] = *reinterpret_cast<const vec4u*>(row + kRopeAt + (2 * j + half) * 16);
    scale = *reinterpret_cast<const f32x4*>(row + kLatentScaleAt);
  };

  const Lookup first = look(0);
  Lookup ahead = look(1);
  const uint8_t* row = row_at(0, first);
  int32_t address = first.la;                          // of the row, where there is one
#pragma unroll
  for (int b = 0; b < kLatentGroups; ++b) load_block(row, b);
  load_rest(row);
  int step = 0;
  for (int row0 = 0; row0 < a.rows; row0 += kRows) {
    if (row0) __syncthreads();                         // the chunk before it is done with
    // q of this chunk into LDS, eight channels a thread at a time, all of them and the rows' log-sums on their way
    // together: a row that is not there stands for the set's first
    constexpr int kPieces = (kLatent + kRope) / 8, kEach = (kRows * kPieces + kWeighWaves * kWave - 1) / (kWeighWaves * kWave);
    Q8 v[kEach];
    float of_row[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = i * kWeighWaves * kWave + threadIdx.x, r = e / kPieces, c = e % kPieces;
      const int row = row0 + r < a.rows ? row0 + r : 0;
      const int node = (int)a.by_heads.div(row), head = row - node * (int)a.by_heads.d;
      const uint16_t* p = static_cast<const uint16_t*>(a.q) + set * a.q_set_stride + node * a.q_node_stride +
                          head * a.q_head_stride + 8 * c;
      of_row[i] = a.lse[(size_t)set * a.rows + row];
      v[i] = a.q_aligned ? load8<Q8, true>(p) : load8<Q8, false>(p);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = i * kWeighWaves * kWave + threadIdx.x, r = e / kPieces, c = e % kPieces;
      if (r >= kRows) break;
      // a row that counts for nothing may hold anything
      if (row0 + r >= a.rows || !counts(of_row[i])) v[i] = Q8{};
      uint8_t* at = s.q + r * Lds::kRowBytes + 16 * c;
      if (Lds::kRopeParts == 1 || c < kLatent / 8) {
        *reinterpret_cast<Q8*>(at) = v[i];
      } else {
        bf16x8 hi, lo;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          __bf16 top, rest;
          two_parts((_Float16)(float)v[i][x], top, rest);
          hi[x] = top;
          lo[x] = rest;
        }
        *reinterpret_cast<bf16x8*>(at) = hi;
        *reinterpret_cast<bf16x8*>(at + 2 * kRope) = lo;
      }
    }
    if (threadIdx.x < kRows) {
      const int r = row0 + threadIdx.x;
      const float lse = r < a.rows ? a.lse[(size_t)set * a.rows + r] : -__builtin_inff();
      s.minus[threadIdx.x] = counts(lse) ? lse * -kLog2e : -__builtin_inff();
    }
    __syncthreads();
    if (!s.ok) return;

    for (int group = 0; group < groups; ++group, ++step) {
      const bool live = row != g_no_row;
      const uint8_t* next = row_at(step + 1, ahead);
      const int32_t next_address = ahead.la;
      ahead = look(step + 2);
      // this lane's row of q: pieces of 16 channels, and of 8 rotary ones; the rest are instruction offsets
      const uint32_t qx = opaque(lds_address(s.q) + col * Lds::kRowBytes + half * 32);
      const uint32_t qr = opaque(lds_address(s.q) + col * Lds::kRowBytes + half * 16);
      f32x4 sc = scale;
#pragma unroll
      for (int b = 0; b < kLatentGroups; ++b) sc[b] *= a.scale_log2;
      f32x16 t[HT];
      {   // the rotary channels, and the rows' log-sums
        f32x16 part[HT];
#pragma unroll
        for (int h = 0; h < HT; ++h) part[h] = f32x16{};
#pragma unroll
        for (int i = Lds::kRopeParts - 1; i >= 0; --i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < HT; ++h) {
              const uint32_t at = 32 * h * Lds::kRowBytes + 2 * kLatent + 2 * kRope * i + 2 * j * 16;
              part[h] = mfma32(lds_get<bf16x8>(qr + at), __builtin_bit_cast(bf16x8, rope[j]), part[h]);
            }
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 m = lds_get<f32x4>(lds_address(s.minus) + (32 * h + 8 * i + 4 * half) * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) t[h][4 * i + r] = __builtin_fmaf(part[h][4 * i + r], a.scale_log2, m[r]);
          }
      }
      load_rest(next);
#pragma unroll
      for (int b = 0; b < kLatentGroups; ++b) {
        __builtin_amdgcn_sched_barrier(0);            // reads of q ahead of a block's products would spill
        Q8 k[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          k[2 * j] = widen8<Q8>(code[b][j].x, code[b][j].y);
          k[2 * j + 1] = widen8<Q8>(code[b][j].z, code[b][j].w);
        }
        load_block(next, b);
        f32x16 part[HT];
#pragma unroll
        for (int h = 0; h < HT; ++h) part[h] = f32x16{};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < HT; ++h) {
              const uint32_t at = 32 * h * Lds::kRowBytes + 2 * (b * kScaleGroup + 2 * j * 16 + 8 * i);
              part[h] = mfma32(lds_get<Q8>(qx + at), k[2 * j + i], part[h]);
            }
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
          for (int r = 0; r < 16; ++r) t[h][r] = __builtin_fmaf(part[h][r], sc[b], t[h][r]);
      }
      float share = 0.0f;
#pragma unroll
      for (int h = 0; h < HT; ++h)
#pragma unroll
        for (int r = 0; r < 16; ++r) share += __builtin_amdgcn_exp2f(t[h][r]);
      if (__any(share != share)) {                    // 0 x infinity in rows that count for nothing, it may be
        share = 0.0f;
#pragma unroll
        for (int h = 0; h < HT; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 m = lds_get<f32x4>(lds_address(s.minus) + (32 * h + 8 * i + 4 * half) * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (m[r] != -__builtin_inff()) share += __builtin_amdgcn_exp2f(t[h][4 * i + r]);
          }
      }
      share = sum_halves(share);
      if (half == 0) {
        float& sum = s.share[wave][group][col];
        if (row0) share += sum;
        if (row0 + kRows < a.rows) {
          sum = share;
        } else if (key_of(group) < a.k) {
          if (!live) share = 0.0f;
          if (a.shares) a.shares[set * a.k + key_of(group)] = share;
          if (a.scores && live) atomicAdd(a.scores + address, score_units(share));
        }
      }
      row = next;
      address = next_address;
    }
  }
  if (err) latch_gather(g.ctr, err);
}

// ---- heads rows ----------------------------------------------------------------
// Bound by the latency of reading the keys: a wave takes TT x 16 tokens by itself and
// goes through the KV heads, a head's keys being contiguous, its 16 query rows (of
// nodes and heads) at a time as the other operand; the next head's keys and the next
// step's query rows are on their way. A token's share stays in the lane's column.
// 16 sets x 2048 tokens x 32 heads of 128 over 8: 13.9 us, 36 MB (15.8 us with rows of q
// asked for when they were needed, and branches around the keys' loads).
__device__ __align__(16) uint8_t g_no_block[4096];     // zeros: a row is at most that long

constexpr int kWeighTokens = 16;
constexpr int kWeighHeadWaves = 4;

template <typename Q8, int D, int TT>
__global__ __launch_bounds__(kWeighHeadWaves * kWave) void k_weigh_heads(GroupDev g, WeighDev a, int n_items) {
  constexpr int kLoads = D / 64;                       // 16-byte pieces of a lane's quarter of a key
  const int lane = lane_id(), quad = lane / 16, col = lane % 16;
  const int item = blockIdx.x * kWeighHeadWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (item >= n_items) return;                         // waves are independent: no barrier below
  const int set = item / a.splits, tile = item % a.splits;
  const int block = 1 << a.block_shift;
  const int shared = a.rows / a.kv_heads;              // query rows per KV head
  const int per = (int)a.by_heads.d;                   // of one node
  const ReaderState state = reader_state(g);

  // Lookups and loads have no branches, so that the compiler knows how many are in flight behind the ones it
  // waits for: a token that is not there looks entry 0 up and reads zeros.
  const uint8_t* pool = g.pool + (size_t)a.layer * g.row_bytes;
  int err = 0;
  const uint8_t* row[TT];
  int tok[TT], count[TT];
  Lookup found[TT];
  auto entry_of = [&](int x) { return tok[x] < a.k << a.block_shift ? set * a.k + (tok[x] >> a.block_shift) : -1; };
#pragma unroll
  for (int x = 0; x < TT; ++x) {
    tok[x] = (tile * TT + x) * kWeighTokens + col;
    const int r = max(entry_of(x), 0);
    found[x] = {g.res[r], a.sel[r]};                   // res has room for every selection of the engine
  }
#pragma unroll
  for (int x = 0; x < TT; ++x) {
    const int r = entry_of(x);
    if (r < 0) found[x].la = -1;
    if (r >= a.n_res) found[x].res = make_uint2(kAbsent, kAbsent);
    const uint32_t slot = slot_of(g, found[x], a.n_res, err);
    row[x] = slot != kAbsent ? pool + (size_t)slot * g.slot_bytes : g_no_block;
  }
  int ok = 0;
  if (lane == 0) ok = reader_ready(g, state, a.want_flag);
  if (!__builtin_amdgcn_readfirstlane(ok)) return;
  if (err) latch_gather(g.ctr, err);

  const int scale_at = 2 * a.kv_heads * block * D;
  vec4u code[TT][kLoads];
  float ks[TT];
  auto load = [&](int kvh) {
#pragma unroll
    for (int x = 0; x < TT; ++x) {
      const uint8_t* p = row[x] + (kvh * block + (tok[x] & (block - 1))) * D + quad * 16;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) code[x][j] = *reinterpret_cast<const vec4u*>(p + 64 * j);
      ks[x] = *reinterpret_cast<const float*>(row[x] + scale_at + 4 * kvh);
    }
  };
  // Sixteen query rows of a KV head: this lane's operand of Q K^T, and the log-sum of its row.
  struct Rows {
    Q8 q[2 * kLoads];
    float lse;
  };
  auto load_rows = [&](int kvh, int r0, Rows& to) {
    const bool there = r0 + col < shared && kvh < a.kv_heads;
    const int hi = there ? r0 + col : 0;               // of those there are, the first stands in for the others
    const int node = (int)a.by_heads.div(hi), head = (there ? kvh * per : 0) + hi - node * per;
    const float lse = a.lse[(size_t)set * a.rows + node * (a.rows / a.nodes) + head];
    const uint16_t* p = static_cast<const uint16_t*>(a.q) + set * a.q_set_stride + node * a.q_node_stride +
                        head * a.q_head_stride + quad * 16;
#pragma unroll
    for (int j = 0; j < 2 * kLoads; ++j) {
      const uint16_t* at = p + 64 * (j / 2) + 8 * (j % 2);
      to.q[j] = a.q_aligned ? load8<Q8, true>(at) : load8<Q8, false>(at);
    }
    to.lse = there ? lse : __builtin_inff();
  };
  load(0);
  float share[TT];
#pragma unroll
  for (int x = 0; x < TT; ++x) {
    share[x] = 0.0f;
    count[x] = *reinterpret_cast<const int32_t*>(row[x] + scale_at + 8 * a.kv_heads);
  }
  Q8 k[TT][2 * kLoads];
  float sc[TT];
  int kvh = 0, r0 = 0;                                 // of the step at hand
  // One step: rows r0 .. of KV head kvh, which are in `now`; the next step's are on their way to `then`.
  auto step = [&](Rows& now, Rows& then) {
    if (r0 == 0) {
#pragma unroll
      for (int x = 0; x < TT; ++x) {
        sc[x] = ks[x] * a.scale_log2;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          k[x][2 * j] = widen8<Q8>(code[x][j].x, code[x][j].y);
          k[x][2 * j + 1] = widen8<Q8>(code[x][j].z, code[x][j].w);
        }
      }
      load(min(kvh + 1, a.kv_heads - 1));
    }
    r0 += 16;
    if (r0 >= shared) {
      r0 = 0;
      ++kvh;
    }
    load_rows(kvh, r0, then);
    // a row that counts for nothing may hold anything
    const bool any = counts(now.lse);
    const float minus = any ? now.lse * -kLog2e : -__builtin_inff();
    Q8 q[2 * kLoads];
#pragma unroll
    for (int j = 0; j < 2 * kLoads; ++j) q[j] = any ? now.q[j] : Q8{};
    float m[4];                                        // of the rows in this lane's registers, 4 quad + r
#pragma unroll
    for (int r = 0; r < 4; ++r) m[r] = __shfl(minus, 4 * quad + r, kWave);
#pragma unroll
    for (int x = 0; x < TT; ++x) {
      f32x4 S{};
#pragma unroll
      for (int j = 0; j < 2 * kLoads; ++j) S = mfma16(q[j], k[x][j], S);
      float part = 0.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) part += __builtin_amdgcn_exp2f(__builtin_fmaf(S[r], sc[x], m[r]));
      if (__any(part != part)) {                       // 0 x infinity in rows that count for nothing, it may be
        part = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (m[r] != -__builtin_inff()) part += __builtin_amdgcn_exp2f(__builtin_fmaf(S[r], sc[x], m[r]));
      }
      share[x] += part;
    }
  };
  Rows rows_a, rows_b;
  load_rows(0, 0, rows_a);
  while (true) {
    step(rows_a, rows_b);
    if (kvh == a.kv_heads) break;
    step(rows_b, rows_a);
    if (kvh == a.kv_heads) break;
  }
#pragma unroll
  for (int x = 0; x < TT; ++x) {
    float sum = (tok[x] & (block - 1)) < count[x] ? sum_quads(share[x]) : 0.0f;
    for (int d = 1; d < block; d *= 2) sum += __shfl_xor(sum, d, kWave);   // the tokens of an entry
    const int entry = tok[x] >> a.block_shift;
    if (quad == 0 && (col & (block - 1)) == 0 && entry < a.k) {
      const int at = set * a.k + entry;
      if (a.shares) a.shares[at] = sum;
      if (a.scores && row[x] != g_no_block) atomicAdd(a.scores + a.sel[at], score_units(sum));
    }
  }
}

// ---- launches ------------------------------------------------------------------
// Latent rows: one workgroup a compute unit (its registers), each with as many key
// groups as that leaves it.
WeighPlan plan_weigh_latent(int n_sets, int k) {
  WeighPlan p{};
  const int groups = (k + kWeighGroup - 1) / kWeighGroup;
  const int want = std::max(1, std::min(groups, (256 + n_sets - 1) / std::max(1, n_sets)));
  p.groups = std::min(kWeighMaxGroups, (groups + want - 1) / want);
  p.splits = std::max(1, (groups + p.groups - 1) / std::max(1, p.groups));
  return p;
}

// Heads rows: 16 tokens a wave, or 64 where many query rows share them.
static int weigh_tiles(int shared) { return shared > 16 ? 4 : 1; }
WeighPlan plan_weigh_heads(long long tokens, int shared) {
  WeighPlan p{};
  const int per = kWeighTokens * weigh_tiles(shared);
  p.splits = (int)((tokens + per - 1) / per);
  return p;
}

template <typename Q8>
static hipError_t weigh_latent_of(const GroupDev& g, const WeighDev& a, int n_sets, hipStream_t s) {
  if (a.rows <= 32) k_weigh_latent<Q8, 1><<<n_sets * a.splits, kWeighWaves * kWave, 0, s>>>(g, a);
  else k_weigh_latent<Q8, 2><<<n_sets * a.splits, kWeighWaves * kWave, 0, s>>>(g, a);
  return hipGetLastError();
}

hipError_t launch_weigh_latent(const GroupDev& g, const WeighDev& a, int type, int n_sets, hipStream_t s) {
  return type == ULA_BF16 ? weigh_latent_of<bf16x8>(g, a, n_sets, s) : weigh_latent_of<f16x8>(g, a, n_sets, s);
}

template <typename Q8, int D>
static hipError_t weigh_heads_of(const GroupDev& g, const WeighDev& a, int n_sets, hipStream_t s) {
  const int items = n_sets * a.splits, blocks = (items + kWeighHeadWaves - 1) / kWeighHeadWaves;
  if (weigh_tiles(a.rows / a.kv_heads) == 1) k_weigh_heads<Q8, D, 1><<<blocks, kWeighHeadWaves * kWave, 0, s>>>(g, a, items);
  else k_weigh_heads<Q8, D, 4><<<blocks, kWeighHeadWaves * kWave, 0, s>>>(g, a, items);
  return hipGetLastError();
}

hipError_t launch_weigh_heads(const GroupDev& g, const WeighDev& a, int type, int n_sets, int head_dim, hipStream_t s) {
  if (type == ULA_BF16)
    return head_dim == 64 ? weigh_heads_of<bf16x8, 64>(g, a, n_sets, s) : weigh_heads_of<bf16x8, 128>(g, a, n_sets, s);
  return head_dim == 64 ? weigh_heads_of<f16x8, 64>(g, a, n_sets, s) : weigh_heads_of<f16x8, 128>(g, a, n_sets, s);
}

}  // namespace ula
