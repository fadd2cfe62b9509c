// Attention of each selection set over its selected latent rows, read from the
// GPU pool where they lie (no gathered copy).
//
// UlaCache summary (paper-daily.com): attention reads only the KV rows at the
// selected positions (introduction), one latent representation serves every
// head (section 1), the cache is in FP8 (section 4), and readers wait for the
// completion signal (section 3).
//
// With k8 a row's e4m3 channels, s_b the scale of channel block b (128
// channels), r its rotary channels and c = scale log2(e), for head h:
//   S_j  = c (sum_b s_bj (q_b . k8_bj) + q_r . r_j)
//   p_j  = 2^(S_j - m)          m the running maximum, l = sum_j p_j
//   o_d  = sum_j p_j s_b(d)j k8_dj / l,   lse = (m + log2 l) ln 2
// e4m3 values are exact in bf16 and fp16, so both products run on 16-bit matrix
// instructions with the block scales applied in 32 bits: to the four partial
// products of S, and to p (rounded to bf16 once per block, at most 2^-8 of its value)
// before the second product.
//
// Layout. Both products are taken transposed: S^T = K Q^T puts heads in the
// lanes' columns and keys in registers, which is the operand layout that
// O^T = V^T P^T wants once V's keys are named in the same order, so p never
// crosses lanes. A wave holds 32 heads: Q in 144 registers, O (512 channels) in
// 256 accumulators, one wave per SIMD; with 16 heads per wave and two waves per
// SIMD every key would be read from LDS and widened twice as often. Of a
// workgroup's 4 waves, NHG take different heads, NKG different keys, and NCG
// different channels of O.
// Keys come in tiles of 32 rows: the first 640 bytes of each row as 16-byte
// pieces straight into LDS (no registers), the scales transposed to [block][key].
// Piece c of key j lies at c ^ ((j >> 1) & 7): without that the 640-byte row
// stride maps every other key to the same banks.
#include <algorithm>
#include <type_traits>

#include "row_format.h"

namespace ula {

constexpr int kTileKeys = 32;
constexpr int kTilePieces = kLatentScaleAt / 16;                 // 40 pieces of a row go to LDS
constexpr int kTileBytes = kTileKeys * kLatentScaleAt;           // 20 KB
constexpr int kTiles = 6;                                        // ring of tiles
constexpr int kComputeUnits = 256;
constexpr double kStartTiles = 6, kJoinTiles = 8, kJoinTilesPerRow = 2.0e-4;   // see plan_attend_latent
constexpr int kWaves = 4;
constexpr int kTileLoads = kTileBytes / 1024;                    // wave-wide 16-byte loads of a tile: 20
constexpr int kLoadsPerWave = 6;                                 // vector loads each wave issues per tile
static_assert(kTileLoads + kLatentGroups == kWaves * kLoadsPerWave, "pieces and scales fill the waves' loads");

// rows that stand in for padding: zeros, so that a masked key adds 0 x 0
__device__ __align__(16) uint8_t g_zero_row[kLatentRow];

// 16 (4) bytes per lane from `src` to LDS at address dst (uniform) + 16 (4) x
// lane. Asynchronous: counted by vmcnt, waited for with wait_loads. In assembly,
// without a data register, because the compiler waits for all such loads it
// knows of before every transposed LDS read. (m0 is never allocated; the kernel
// has nothing else that uses it.)
__device__ __forceinline__ void lds_load16(const uint8_t* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(dst), "v"(src) : "memory");
}
__device__ __forceinline__ void lds_load4(const uint8_t* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(dst), "v"(src) : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A workgroup barrier that leaves vector loads in flight (__syncthreads waits
// for them): this wave's LDS accesses are done, loads into LDS are waited for by
// wait_loads.
__device__ __forceinline__ void barrier_keep_loads() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The value again, as one the compiler cannot trace back: what is computed from
// it inside a loop is not kept in registers across the loop.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

struct LatentLds {
  alignas(1024) uint8_t ring[kTiles][kTileBytes];
  alignas(16) float scale[kTiles][kLatentGroups][kTileKeys];
  uint32_t slot[kAttendKeys];
  uint32_t live[kAttendKeys / kTileKeys];   // bit per key: not padding
  int ok;
};
static_assert(sizeof(LatentLds) <= 160 * 1024, "LDS of a compute unit");

template <typename Q8, int NHG, int NKG>
__global__ __launch_bounds__(kWaves * kWave, 1) void k_attend_latent(GroupDev g, AttendDev a) {
  constexpr int NCG = kWaves / (NHG * NKG);  // waves that share heads and keys, each with its channels of O
  constexpr int kRounds = kTiles / NKG;      // rounds of NKG tiles the ring holds
  constexpr int kOut = kLatent / 32 / NCG;   // 32-channel tiles of O per wave
  constexpr int kOutBlocks = kLatentGroups / NCG;   // scale blocks of those channels
  static_assert(kLatentGroups % NCG == 0, "a wave's channels are whole scale blocks");
  __shared__ LatentLds s;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);   // uniform: its branches are scalar
  const int hg = wave % NHG, cg = (wave / NHG) % NCG, kg = wave / (NHG * NCG);
  const int half = lane / 32;                // which 8 of an operand's 16 k
  const int col = lane % 32;

  // work item: consecutive sets (which share rows under speculative selection)
  // run on one XCD at about the same time
  int item = blockIdx.x;
  {
    const int per = gridDim.x / 8, rest = gridDim.x % 8;
    const int x = item % 8;
    item = x * per + min(x, rest) + item / 8;
  }
  const int split = item % a.splits;
  const int hb = (item / a.splits) % a.head_blocks;
  const int set = item / (a.splits * a.head_blocks);
  const int key0 = split * a.split_keys;
  const int nkeys = max(0, min(a.split_keys, a.k - key0));
  const int ntiles = (nkeys + kTileKeys - 1) / kTileKeys;
  const int rounds = (ntiles + NKG - 1) / NKG;
  const int total = rounds * NKG;

  // resolve the keys' slots once (whole waves take part: the ballot below)
  int err = 0;
  if (threadIdx.x == 0) s.ok = reader_ready(g, a.want_flag);
  for (int i0 = wave * kWave; i0 < total * kTileKeys; i0 += kWaves * kWave) {
    const int i = i0 + lane;
    const uint32_t slot = i < nkeys ? resolve_slot(g, a.sel, set * a.k + key0 + i, a.n_res, err) : kAbsent;
    s.slot[i] = slot;
    const unsigned long long live = __ballot(slot != kAbsent);
    if (lane < 2) s.live[i0 / 32 + lane] = (uint32_t)(live >> (32 * lane));
  }
  if (err) latch_gather(g.ctr, err);

  // this wave's 32 heads of q. A 32-channel piece t gives two operands: lane half
  // x holds channels 32 t + 16 x + 8 j + i, as the 16-byte key reads do.
  const int head = (hb * NHG + hg) * 32 + col;
  Q8 ql[kLatent / 16];
  Q8 qr[kRope / 16];
  if (head < a.heads) {
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + set * a.q_set_stride + head * a.q_head_stride;
    auto load_q = [&](auto aligned) {
#pragma unroll
      for (int t = 0; t < kLatent / 32; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) ql[2 * t + j] = load8<Q8, aligned>(q + 32 * t + 16 * half + 8 * j);
#pragma unroll
      for (int j = 0; j < kRope / 16; ++j) qr[j] = load8<Q8, aligned>(q + kLatent + 16 * j + 8 * half);
    };
    if (a.q_aligned) load_q(std::true_type{});
    else load_q(std::false_type{});
  } else {
#pragma unroll
    for (int t = 0; t < kLatent / 16; ++t) ql[t] = Q8{};
#pragma unroll
    for (int j = 0; j < kRope / 16; ++j) qr[j] = Q8{};
  }
  // q has arrived before any asynchronous load is issued: a wait for it inside the
  // main loop would wait for those too
#pragma unroll
  for (int t = 0; t < kLatent / 16; ++t) asm volatile("" : "+v"(ql[t]));
#pragma unroll
  for (int j = 0; j < kRope / 16; ++j) asm volatile("" : "+v"(qr[j]));
  __syncthreads();
  if (!s.ok) return;

  const uint8_t* pool = g.pool + (size_t)a.layer * g.row_bytes;
  auto row_of = [&](uint32_t slot) -> const uint8_t* {
    return slot == kAbsent ? g_zero_row : pool + (size_t)slot * g.slot_bytes;
  };
  // a tile's loads: 5 wave-wide ones for pieces and one for a scale block, per wave
  auto issue = [&](int tile) {
    const int at = tile % kTiles;
    const uint32_t slots = lds_address(s.slot) + tile * kTileKeys * 4;
    const int lane = opaque(lane_id());   // registers are scarce in the main loop
#pragma unroll
    for (int i = 0; i < kTileLoads / kWaves; ++i) {
      const int n = i * kWaves + wave;
      const int p = n * kWave + lane;
      const int key = p / kTilePieces, c = p % kTilePieces;
      lds_load16(row_of(lds_get<uint32_t>(slots + key * 4)) + (c ^ ((key >> 1) & 7)) * 16,
                 lds_address(s.ring) + at * kTileBytes + n * kWave * 16);
    }
    if (lane < kTileKeys)
      lds_load4(row_of(lds_get<uint32_t>(slots + lane * 4)) + kLatentScaleAt + 4 * wave,
                lds_address(s.scale) + (at * kLatentGroups + wave) * kTileKeys * 4);
  };

  // Keys of a tile: register r in lane half x is key 8 (r / 4) + 4 x + r % 4.
  // koff: this lane's key (col), piece `half` of a scale block; piece 2 t + half is
  // ^ (t << 5). voff: the row this lane names in a transposed read of keys 0..15
  // and the channels of its 16 lanes; 32-channel tile t is ^ (t << 5).
  int koff, voff;
  {
    koff = col * kLatentScaleAt + ((half ^ ((col >> 1) & 7)) << 4);
    const int r = lane % 16 / 2;
    const int key = 8 * (r / 4) + 4 * half + r % 4;
    voff = key * kLatentScaleAt + (((lane / 16 % 2) ^ ((key >> 1) & 7)) << 4) + (lane & 1) * 8;
  }
  static_assert(kLatentScaleAt % 128 == 0 && kTileBytes % 128 == 0, "the swizzle's bits are free in every row address");

  f32x16 o[kOut];
#pragma unroll
  for (int t = 0; t < kOut; ++t) o[t] = f32x16{};
  float m = -__builtin_inff(), l = 0.0f;

#pragma unroll 1
  for (int t = 0; t < kRounds * NKG && t < total; ++t) issue(t);
#pragma unroll 1
  for (int round = 0; round < rounds; ++round) {
    // this round's tiles are in LDS once every wave's loads for them are
    if (round + kRounds <= rounds) wait_loads<(kRounds - 1) * NKG * kLoadsPerWave>();
    else wait_loads<0>();
    barrier_keep_loads();
    const int tile = round * NKG + kg;
    const int at = tile % kTiles;
    // LDS addresses: everything below is one of these plus a constant
    const uint32_t ring = lds_address(s.ring) + at * kTileBytes;
    const uint32_t krow = ring + koff, vrow = ring + voff;
    const uint32_t scale = lds_address(s.scale) + (at * kLatentGroups * kTileKeys + 4 * half) * 4;
    const uint32_t live = __builtin_amdgcn_readfirstlane(s.live[tile]);
    if (live) {
      f32x16 S{};
#pragma unroll
      for (int j = 0; j < kRope / 16; ++j) {   // rotary part: bf16 in the row
        const bf16x8 kr = lds_get<bf16x8>((krow ^ (j << 5)) + kRopeAt);
        if constexpr (__is_same(Q8, bf16x8)) {
          S = mfma32(kr, qr[j], S);
        } else {
          // an fp16 q as the sum of two bf16 values (8 + 8 bits hold its 11)
          bf16x8 hi, lo;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            hi[e] = (__bf16)(float)qr[j][e];
            lo[e] = (__bf16)((float)qr[j][e] - (float)hi[e]);
          }
          S = mfma32(kr, hi, S);
          S = mfma32(kr, lo, S);
        }
      }
#pragma unroll
      for (int b = 0; b < kLatentGroups; ++b) {
        f32x16 part{};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const vec4u k8 = lds_get<vec4u>((krow ^ (t << 5)) + b * kScaleGroup);
          part = mfma32(widen8<Q8>(k8.x, k8.y), ql[8 * b + 2 * t], part);
          part = mfma32(widen8<Q8>(k8.z, k8.w), ql[8 * b + 2 * t + 1], part);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 sc = lds_get<f32x4>(scale + (kTileKeys * b + 8 * i) * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) S[4 * i + e] += sc[e] * part[4 * i + e];
        }
      }
      float top = -__builtin_inff();
      const uint32_t mine = live >> (4 * half);
#pragma unroll
      for (int r = 0; r < 16; ++r) S[r] *= a.scale_log2;
      if (live != 0xFFFFFFFFu) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (!(mine & (1u << (8 * (r / 4) + r % 4)))) S[r] = -__builtin_inff();
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, S[r]);
      top = max_halves(top);
      // The maximum moves only when it rises by more than 2^8: p then stays below
      // 2^8, exact in its exponent, and most tiles leave O as it is.
      if (__any(top > m + 8.0f)) {
        const float nm = fmaxf(m, top);
        const float al = nm == -__builtin_inff() ? 1.0f : exp2f(m - nm);
        m = nm;
        l *= al;
#pragma unroll
        for (int t = 0; t < kOut; ++t) o[t] *= al;
      }
      const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        S[r] = __builtin_amdgcn_exp2f(S[r] - base);
        l += S[r];
      }
#pragma unroll
      for (int bi = 0; bi < kOutBlocks; ++bi) {
        const int b = cg * kOutBlocks + bi;
        bf16x8 p[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 sc = lds_get<f32x4>(scale + (kTileKeys * b + 8 * i) * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) p[i / 2][4 * (i % 2) + e] = (__bf16)(S[4 * i + e] * sc[e]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const i32x2 v8 = lds_read_transposed((vrow ^ (t << 5)) + b * kScaleGroup + x * 16 * kLatentScaleAt);
            o[4 * bi + t] = mfma32(widen8<bf16x8>((uint32_t)v8.x, (uint32_t)v8.y), p[x], o[4 * bi + t]);
          }
      }
    }
    barrier_keep_loads();   // every wave is done with this round's tiles
#pragma unroll
    for (int x = 0; x < NKG; ++x) {
      const int next = (round + kRounds) * NKG + x;
      if (next < total) issue(next);
    }
  }
  l = sum_halves(l);

  // join the two key groups: the second hands (m, l, O) over in quarters of O
  if constexpr (NKG == 2) {
    constexpr int kPart = kOut / 4;
    float* box = reinterpret_cast<float*>(s.ring) + (wave % (NHG * NCG)) * (kPart * 16 + 2) * kWave + lane;
    static_assert((kWaves / 2) * (kPart * 16 + 2) * kWave * 4 <= kTiles * kTileBytes, "the ring holds a quarter of O");
    float w1 = 1.0f, w2 = 0.0f;
#pragma unroll
    for (int part = 0; part < 4; ++part) {
      if (kg == 1) {
#pragma unroll
        for (int t = 0; t < kPart; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r) box[(16 * t + r) * kWave] = o[part * kPart + t][r];
        box[kPart * 16 * kWave] = m;
        box[(kPart * 16 + 1) * kWave] = l;
      }
      __syncthreads();
      if (kg == 0) {
        if (part == 0) {
          const float m2 = box[kPart * 16 * kWave], l2 = box[(kPart * 16 + 1) * kWave];
          const float nm = fmaxf(m, m2);
          w1 = nm == -__builtin_inff() ? 0.0f : exp2f(m - nm);
          w2 = nm == -__builtin_inff() ? 0.0f : exp2f(m2 - nm);
          m = nm;
          l = l * w1 + l2 * w2;
        }
#pragma unroll
        for (int t = 0; t < kPart; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            o[part * kPart + t][r] = o[part * kPart + t][r] * w1 + box[(16 * t + r) * kWave] * w2;
      }
      __syncthreads();
    }
    if (kg) return;
  }

  if (head >= a.heads) return;
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  const float lse2 = l != 0.0f ? m + log2f(l) : -__builtin_inff();
  const int c0 = cg * (kLatent / NCG) + 4 * half;
  if (a.splits > 1) {   // this split's own result, joined by k_attend_join
    const size_t row = ((size_t)set * a.heads + head) * a.splits + split;
    float* po = a.part_o + row * kLatent + c0;
#pragma unroll
    for (int t = 0; t < kOut; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = o[t][4 * i + e] * inv;
        *reinterpret_cast<f32x4*>(po + 32 * t + 8 * i) = v;
      }
    if (half == 0 && cg == 0) a.part_lse[row] = lse2;
    return;
  }
  uint16_t* out = static_cast<uint16_t*>(a.out) + set * a.out_set_stride + head * a.out_head_stride + c0;
#pragma unroll
  for (int t = 0; t < kOut; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = o[t][4 * i + e] * inv;
      store4<Q8>(out + 32 * t + 8 * i, v, a.out_aligned);
    }
  if (half == 0 && cg == 0 && a.lse) a.lse[(size_t)set * a.heads + head] = lse2 * kLn2;
}

// Joins the splits of one (set, head): o = sum_s w_s o_s / sum_s w_s with
// w_s = 2^(lse_s - max lse). One wave per `kWave * 4` channels or fewer.
template <typename Q8>
__global__ __launch_bounds__(128) void k_attend_join(GroupDev g, AttendDev a, int width) {
  __shared__ int ok;
  if (threadIdx.x == 0) ok = reader_ready(g, a.want_flag);
  __syncthreads();
  if (!ok) return;
  const size_t row = blockIdx.x;
  const float* lse = a.part_lse + row * a.splits;
  float top = -__builtin_inff();
  for (int i = 0; i < a.splits; ++i) top = fmaxf(top, lse[i]);
  const float base = top == -__builtin_inff() ? 0.0f : top;
  const int c = 4 * threadIdx.x;
  f32x4 acc{};
  float sum = 0.0f;
  for (int i = 0; i < a.splits; ++i) {
    const float w = exp2f(lse[i] - base);
    sum += w;
    if (c < width) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(a.part_o + (row * a.splits + i) * width + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] += w * v[e];
    }
  }
  const int set = (int)(row / a.heads), head = (int)(row % a.heads);
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  if (c < width) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = acc[e] * inv;
    store4<Q8>(static_cast<uint16_t*>(a.out) + set * a.out_set_stride + head * a.out_head_stride + c, v, a.out_aligned);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[row] = sum != 0.0f ? (top + log2f(sum)) * kLn2 : -__builtin_inff();
}

constexpr int latent_wg_heads(int heads) { return heads <= 32 ? 32 : 64; }

// How a call's keys are split over workgroups (one per compute unit at a time):
// the number of splits with the least estimated time, in units of one tile's
// time on one compute unit. A workgroup costs its tiles plus a fixed start
// (resolving slots, loading q); with more than one split each also writes, and
// the join reads, its 32-bit results.
AttendPlan plan_attend_latent(int n_sets, int k, int heads) {
  AttendPlan best{};
  const int wg_heads = latent_wg_heads(heads);
  best.head_blocks = (heads + wg_heads - 1) / wg_heads;
  const long long base = (long long)n_sets * best.head_blocks;
  const int tiles = (k + kTileKeys - 1) / kTileKeys;
  double best_cost = 0;
  const int least = std::max(1, (k + kAttendKeys - 1) / kAttendKeys);
  for (int want = least; want <= std::max(least, std::min(tiles, 256)); ++want) {
    const int per = (tiles + want - 1) / want;            // tiles per split
    const int splits = std::max(1, (tiles + per - 1) / per);
    if (splits != want && want != least) continue;        // the same split as a smaller one
    const double waves = (double)((base * splits + kComputeUnits - 1) / kComputeUnits);
    double cost = waves * (per + kStartTiles);
    if (splits > 1) cost += kJoinTiles + (double)base * splits * std::min(heads, wg_heads) * kJoinTilesPerRow;
    if (best.splits == 0 || cost < best_cost) {
      best_cost = cost;
      best.splits = splits;
      best.split_keys = std::max(1, per) * kTileKeys;
    }
  }
  return best;
}

template <typename Q8, int NHG, int NKG>
static void launch_latent(const GroupDev& g, const AttendDev& a, int n_sets, hipStream_t s) {
  k_attend_latent<Q8, NHG, NKG><<<n_sets * a.head_blocks * a.splits, kWaves * kWave, 0, s>>>(g, a);
}

template <typename Q8>
static hipError_t launch_latent_of(const GroupDev& g, const AttendDev& a, int n_sets, hipStream_t s) {
  if (a.heads <= 32) launch_latent<Q8, 1, 2>(g, a, n_sets, s);
  else launch_latent<Q8, 2, 1>(g, a, n_sets, s);
  return hipGetLastError();
}

hipError_t launch_attend_latent(const GroupDev& g, const AttendDev& a, int type, int n_sets, hipStream_t s) {
  return type == ULA_BF16 ? launch_latent_of<bf16x8>(g, a, n_sets, s) : launch_latent_of<f16x8>(g, a, n_sets, s);
}

hipError_t launch_attend_join(const GroupDev& g, const AttendDev& a, int type, int n_sets, int width, hipStream_t s) {
  const int blocks = n_sets * a.heads;
  if (type == ULA_BF16) k_attend_join<bf16x8><<<blocks, 128, 0, s>>>(g, a, width);
  else k_attend_join<f16x8><<<blocks, 128, 0, s>>>(g, a, width);
  return hipGetLastError();
}

}  // namespace ula
