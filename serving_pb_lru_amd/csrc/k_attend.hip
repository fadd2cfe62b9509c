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
//   p_j  = 2^(S_j - m)          m a running reference, l = sum_j p_j
//   o_d  = sum_j p_j s_b(d)j k8_dj / l,   lse = (m + log2 l) ln 2
// The block scales are applied in 32 bits, to the four partial products of S and
// to p, so e4m3 codes enter the matrix instructions as they are:
//   - first product: codes widened to q's type, which holds them exactly. (The
//     8-bit matrix instruction with q as a sum of e4m3 values widens nothing, and
//     took 111 us where this takes 113 us for 256 sets of 2048 keys and 64 heads.
//     But it cuts the products of 16 channels off at 2^-13 of the largest of
//     them before it adds them up: log-sums were off by up to 5e-4, this way by
//     4e-6.)
//   - second product: codes widened to fp16, and p s_b rounded to fp16. m follows
//     the largest p_j max_b s_bj of any key, which stays within 2^7..2^15 (a scale
//     below 2^-60 counts as that), so the rounding is at most 2^-11 of the value, or
//     2^-25 (2^-32 of the largest) for small ones. bf16 results hardly show it
//     (1.68e-3 of their size off, 1.66e-3 without). fp16 results would: for them
//     what it leaves goes through a second product with the same values (2.07e-4
//     off, as a result of 64 bits rounded once, 2.9e-4 without; 384 sets of 2047 keys
//     and 128 heads 368 us, 300 us without). A tree's results of either type go that
//     way: bf16 ones of one part were 1e-3 of their size from those of weights in 32 bits, 6e-5 so
//     (16 sets x 8 nodes x 2048 keys x 128 heads 125 us, 101 us without).
// Both products have 32-bit accumulators.
//
// Layout. Both products are taken transposed: S^T = K Q^T puts heads in the
// lanes' columns and keys in registers, O^T = V^T P^T the same way. A workgroup
// has four waves for the first product and the softmax, half of its heads (16 or
// 32) and half of a tile's 32 keys each, and four for the second product, 128
// channels of O (one scale block) with all heads each: so no wave holds another's
// Q, a key is widened for all of a wave's heads at once and every value once. In
// between p goes through LDS in the operand order of the second product, scaled for
// each block (fp16 queries and trees: in 32 bits, scaled, and split, by the second waves).
// The two waves of a head tell each other their largest logits through LDS as well, a
// barrier ahead of the softmax, and so come to the same m. Each SIMD has a wave of either kind. One barrier per tile.
// Measured, 256 sets of 2048 keys and 64 heads: 206 us with a wave that kept 32
// heads to itself for both products, reading and widening every key and value
// four times; 128 us with eight equal waves that went through first product,
// softmax and second product in turn, which left the younger wave of a SIMD
// waiting; 132 us with 16 heads and a whole tile's keys per first wave; 113 us so
// (116 since the sum of the weights takes two factors; a call 121).
// Of that 18 us are start and end, and the 344 MB of rows alone take 58 us at the
// rate of a large copy. In the loop the first waves' chain of products, maximum,
// exponentials and p takes about 2500 cycles a tile; vector instructions fill 56% of
// a SIMD's cycles and matrix instructions 32%, and the two hardly overlap. Issuing
// a tile's products ahead of the softmax before it does not shorten it (116 us), nor
// does p in 32 bits scaled by the second waves, with a sixth tile in the LDS that
// frees (117 us).
// Sixteen waves of 16 heads or 64 channels read keys and p from LDS twice as often
// and widen keys twice as often: 159 us.
// A tree of drafted tokens (TREE) has nodes x heads rows where the heads are, and two
// tiles of keys at most behind the selected ones, whose rows come from the caller and
// which a row sees by its node's mask. 64 sets x 1024 rows x 2048 keys, bf16: 474 us a call, of which each
// of four rounds of workgroups spends 15 us on its start (5 us for 19 MB of q), the filling
// of the pipeline and its end.
// Tiles: the first 640 bytes of each row as 16-byte pieces straight into LDS (no
// registers), the scales transposed to [block][key]. Piece c of key j lies at
// c ^ swizzle(j), which keeps the 16 lanes that a 16-byte read serves at once
// (0-3, 12-15, 20-27 and the other such sets) and the 32 of a transposed read on
// different banks; (j >> 1) & 7 in its place took 8.3 cycles per read, this 4.6.
#include <algorithm>
#include <type_traits>

#include "row_format.h"

namespace ula {

constexpr int kTileKeys = 32;
constexpr int kTilePieces = kLatentScaleAt / 16;                 // 40 pieces of a row go to LDS
constexpr int kTileBytes = kTileKeys * kLatentScaleAt;           // 20 KB
constexpr int kComputeUnits = 256;
constexpr int kTileLoads = kTileBytes / 1024;                    // wave-wide 16-byte loads of a tile: 20

// rows that stand in for padding: zeros, so that a masked key adds 0 x 0
__device__ __align__(16) uint8_t g_zero_row[kLatentRow];

// 16 (4) bytes per lane from `src` to LDS at address dst (uniform) + 16 (4) x
// lane. Asynchronous: counted by vmcnt, waited for with wait_loads. In assembly,
// without a data register, because the compiler waits for all such loads it
// knows of before every transposed LDS read. (m0 is never allocated; the kernel
// has nothing else that uses it.)
__device__ __forceinline__ void lds_load16(const uint8_t* src, uint32_t dst) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(dst);   // a scalar register, whatever the compiler knows
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(src) : "memory");
}
__device__ __forceinline__ void lds_load4(const uint8_t* src, uint32_t dst) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(dst);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(at), "v"(src) : "memory");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The piece bits of key j in a tile that are exchanged (see above): bit 1 from the
// key's bit 1, bit 2 from bits 2 and 3.
__device__ __forceinline__ int swizzle(int key) { return (key & 2) | ((key >> 2 ^ key >> 3) & 1) << 2; }

// A workgroup barrier that leaves vector loads in flight (__syncthreads waits
// for them): this wave's LDS accesses are done, loads into LDS are waited for by
// wait_loads.
__device__ __forceinline__ void barrier_keep_loads() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The value again, as one the compiler cannot trace back: sums of it and a
// constant become instruction offsets, where it would otherwise keep the sums of
// its parts and each constant in registers across the loop.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// x *= f element by element in x's own registers. Without the empty assembly the
// compiler gathers the products into new registers, and a branch around them
// then costs a copy of the accumulators where it is not taken.
__device__ __forceinline__ void scale_in_place(f32x16& x, float f) {
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    x[r] *= f;
    asm volatile("" : "+v"(x));
  }
}

constexpr int kFewSplits = 8;                     // of a tree's rows: joined by k_tree_join
constexpr int kWaves = 8;
constexpr int kFirstWaves = 4;                    // waves 0..3: first product and softmax
constexpr int kSecondWaves = kWaves - kFirstWaves;
constexpr int kLoadsPerWave = (kTileLoads + kLatentGroups) / kSecondWaves;   // a second wave's vector loads per tile
static_assert(kSecondWaves == kLatentGroups, "one scale block per second wave");

// fp16 results, and a tree's: p x scale in two parts, which the second waves make of p in 32 bits. (Else the first waves
// make it: 256 sets x 64 heads x 2048 keys 121 us so, 125 when the second waves do it.)
template <typename Q8, bool TREE>
constexpr bool kTwoParts = TREE || !std::is_same_v<Q8, bf16x8>;

// Keys that a work item takes: a tree's drafted tokens come on top of a whole selection.
template <bool TREE>
constexpr int kItemKeys = kAttendKeys + (TREE ? kTreeNodes : 0);

template <typename Q8, int HT, int TILES, bool TREE>
struct LatentLds {
  static constexpr int HEADS = 32 * HT;
  alignas(1024) uint8_t ring[TILES][kTileBytes];
  // bytes of a key's p: one in 32 bits, or one for each block in 16
  static constexpr int kKeyBytes = kTwoParts<Q8, TREE> ? 4 : 2 * kLatentGroups;
  // p of two tiles. In 16 bits: p x scale, [block][head][key], key chunk c (8 keys) of head h at
  // c ^ ((h >> 2) & 3). In 32: p, [head][key], key chunk c (4 keys) of head h at c ^ ((h >> 1) & 7).
  alignas(1024) uint8_t p[2][HEADS * kTileKeys * kKeyBytes];
  alignas(16) float scale[TILES][kLatentGroups][kTileKeys];
  float alpha[2][HEADS];                    // factor of O before the tile's second product
  alignas(16) uint32_t moved[2][4];         // whether any head of a first wave has a factor other than 1
  alignas(8) float top[2][HEADS][2];        // of two tiles: the largest logarithm of p x scale, of either half of the keys
  const uint8_t* row[kItemKeys<TREE>];      // each key's row in this layer; zeros for padding
  uint32_t live[kItemKeys<TREE> / kTileKeys + 2];   // bit per key: not padding; none behind the last tile
  uint32_t sees[2][TREE ? HEADS : 1];       // what a row sees of the drafted tokens' two tiles
  uint32_t bad[TREE ? kItemKeys<TREE> / kTileKeys + 2 : 1];   // bit per drafted token: its row holds a NaN
  int ok;
};

// One wave's 16 heads of q as they are in memory. Lane quad x holds channels 64 t
// + 16 x + (0..15) of each 64-channel piece t, as the 16-byte key reads do.
template <typename Q8>
struct QueryRaw {
  Q8 x[kLatent / 32];
  Q8 rope[kRope / 32];
  template <bool ALIGNED>
  __device__ __forceinline__ void load(const uint16_t* q, bool any, int quad) {
#pragma unroll
    for (int t = 0; t < kLatent / 32; ++t)
      x[t] = any ? load8<Q8, ALIGNED>(q + 64 * (t / 2) + 16 * quad + 8 * (t % 2)) : Q8{};
#pragma unroll
    for (int j = 0; j < kRope / 32; ++j)
      rope[j] = any ? load8<Q8, ALIGNED>(q + kLatent + 32 * j + 8 * quad) : Q8{};
  }
};

// The same as the operands of the first product. The keys' rotary channels are
// bf16, so fp16 ones become the sum of two bf16 values (8 + 8 bits hold their 11).
template <typename Q8>
struct QueryOperand {
  static constexpr int kRopeParts = std::is_same_v<Q8, bf16x8> ? 1 : 2;
  Q8 x[kLatent / 32];
  bf16x8 rope[kRopeParts][kRope / 32];
  __device__ __forceinline__ void take(const QueryRaw<Q8>& raw) {
#pragma unroll
    for (int t = 0; t < kLatent / 32; ++t) x[t] = raw.x[t];
#pragma unroll
    for (int j = 0; j < kRope / 32; ++j) {
      if constexpr (kRopeParts == 1) {
        rope[0][j] = raw.rope[j];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          __bf16 hi, lo;
          two_parts(raw.rope[j][e], hi, lo);
          rope[0][j][e] = hi;
          rope[1][j][e] = lo;
        }
      }
    }
  }
  __device__ __forceinline__ f32x4 rope_product(const bf16x8* kr) const {
    f32x4 s{};
#pragma unroll
    for (int j = 0; j < kRope / 32; ++j)
#pragma unroll
      for (int i = kRopeParts - 1; i >= 0; --i) s = mfma16(kr[j], rope[i][j], s);
    return s;
  }
  // product of a block's keys, widened, 32 channels at a time
  __device__ __forceinline__ f32x4 block_product(int b, const Q8* k) const {
    f32x4 s{};
#pragma unroll
    for (int j = 0; j < kScaleGroup / 32; ++j) s = mfma16(k[j], x[4 * b + j], s);
    return s;
  }
};

// The second waves' O (o[t][h] of wave w: channels 128 w + 32 t .., heads 32 h ..)
// as type T, times inv, through the LDS at `box`; put(head, channel, 16 bytes) for
// heads first + 0.. below `heads`. 32 channels of every wave at a time, so that
// memory is written in whole segments (8 bytes per lane from the registers' order
// took 18 us of a 256-set call), and the stores of one step are on their way
// during the next. Rows are padded by 16 bytes for the banks.
template <typename T, int CT, int HT, typename F>
__device__ __forceinline__ void store_heads(uint8_t* box, const f32x16 (&o)[CT][HT], const float (&inv)[HT], int first,
                                            int heads, F put) {
  constexpr int kSpan = 32 * kSecondWaves;        // channels at a time
  constexpr int kRow = kSpan * sizeof(T) + 16;
  constexpr int kPer = 16 / sizeof(T);            // channels per 16 bytes
  constexpr int kLanes = kSpan / kPer;            // lanes per head
  const int lane = lane_id(), half = lane / 32, col32 = lane % 32;
  const int wave = (int)(threadIdx.x / kWave) - kFirstWaves;
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    barrier_keep_loads();
    if (wave >= 0) {
#pragma unroll
      for (int h = 0; h < HT; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          typedef T vec __attribute__((ext_vector_type(4)));
          vec v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (T)(o[t][h][4 * i + e] * inv[h]);
          *reinterpret_cast<vec*>(box + (32 * h + col32) * kRow + (32 * wave + 8 * i + 4 * half) * sizeof(T)) = v;
        }
    }
    barrier_keep_loads();
    for (int e = threadIdx.x; e < 32 * HT * kLanes; e += kWaves * kWave) {
      const int h = e / kLanes, c = e % kLanes * kPer;
      if (first + h < heads)
        put(first + h, c / 32 * (kLatent / kSecondWaves) + 32 * t + c % 32,
            *reinterpret_cast<const vec4u*>(box + h * kRow + c * sizeof(T)));
    }
  }
}

// HT tiles of 32 heads; TILES tiles in the ring.
template <typename Q8, int HT, int TILES, bool TREE>
__global__ __launch_bounds__(kWaves * kWave, 2) void k_attend_latent(GroupDev g, AttendDev a) {
  constexpr int kHeads = 32 * HT;                 // heads of a workgroup
  constexpr bool kTwo = kTwoParts<Q8, TREE>;
  constexpr int CT = kScaleGroup / 32;            // 32-channel tiles of a second wave's O
  static_assert(2 * kHeads == 16 * HT * kFirstWaves, "every head has two waves in the first product");
  static_assert(TILES >= 4, "a tile on its way beside the three in use");
  __shared__ LatentLds<Q8, HT, TILES, TREE> s;
  static_assert(sizeof(s) <= 160 * 1024, "LDS of a compute unit");
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);   // uniform: its branches are scalar
  const bool second = wave >= kFirstWaves;
  const int quad = lane / 16, col = lane % 16;    // first product: 16 heads, quads of keys
  const int half = lane / 32, col32 = lane % 32;  // second product: 32 heads

  // work item: consecutive sets (which share rows under speculative selection)
  // run on one XCD at about the same time
  int item = blockIdx.x;
  const int lead = TREE ? a.whole * a.head_blocks : 0;   // workgroups that have all of a set's keys
  const bool whole = TREE && item < lead;
  {
    const int n = whole ? lead : gridDim.x - lead, i = whole ? item : item - lead;
    const int per = n / 8, rest = n % 8;
    const int x = i % 8;
    item = x * per + min(x, rest) + i / 8;
  }
  const int splits = whole ? 1 : a.splits;
  const int hb = item % a.head_blocks;
  const int split = item / a.head_blocks % splits;
  const int set = item / (splits * a.head_blocks) + (TREE && !whole ? a.whole : 0);
  const int key0 = split * a.split_keys;
  const int nkeys = whole ? a.k : max(0, min(a.split_keys, a.k - key0));
  const int tiles = (nkeys + kTileKeys - 1) / kTileKeys;

  const int head0 = wave / 2 * 16 * HT;           // the first of a first wave's HT x 16 heads, and its half of the keys
  const int key_half = wave % 2;
  f32x16 o[CT][HT];                               // a second wave's alone: unset in the others, whose registers it would fill
  float m[HT], l[HT];                             // of a first wave's heads; l of the lane's keys alone

  // Barriers: one when the rows are known, one when tile 0 is in LDS, then one per tile i = -1, 0, ..: tile
  // i + 2 is in LDS, p of tile i is there, and nobody reads tile i - 1 any more.
  if (second) {
    // The second waves look the keys' rows up and start their loads; the first waves'
    // q, which takes longer to arrive, is on its way meanwhile.
    int err = 0;
    const uint8_t* pool = g.pool + (size_t)a.layer * g.row_bytes;
    constexpr int kAtOnce = 4;                    // lookups in flight per lane
    const int n = tiles * kTileKeys;
    for (int i0 = (wave - kFirstWaves) * kWave; i0 < n; i0 += kAtOnce * kSecondWaves * kWave) {
      Lookup at[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = i0 + j * kSecondWaves * kWave + lane;
        at[j].la = -1;
        if constexpr (TREE) {
          if (i < nkeys && key0 + i < a.sel_k) at[j] = look_up(g, a.sel, set * a.sel_k + key0 + i, a.n_res);
        } else {
          if (i < nkeys) at[j] = look_up(g, a.sel, set * a.k + key0 + i, a.n_res);
        }
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int first = i0 + j * kSecondWaves * kWave;   // uniform: whole waves take part in the ballot
        if (first >= n) break;
        const uint32_t slot = slot_of(g, at[j], a.n_res, err);
        const uint8_t* row = slot != kAbsent ? pool + (size_t)slot * g.slot_bytes : g_zero_row;
        if constexpr (TREE) {
          const int draft = key0 + first + lane - a.history_tiles * kTileKeys;
          if (draft >= 0 && draft < a.nodes) row = a.drafts + ((long long)set * a.nodes + draft) * a.draft_stride;
        }
        s.row[first + lane] = row;
        const unsigned long long live = __ballot(row != g_zero_row);
        if (lane < 2) s.live[first / 32 + lane] = (uint32_t)(live >> (32 * lane));
      }
    }
    if (err) latch_gather(g.ctr, err);
    barrier_keep_loads();
    if (!s.ok) return;
    // This wave's six loads of a tile: five of pieces, one of a scale block. The
    // rows' addresses are read from LDS one tile earlier.
    const int sw = wave - kFirstWaves;
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int h = 0; h < HT; ++h) o[t][h] = f32x16{};
    constexpr int kPieceLoads = kLoadsPerWave - 1;
    static_assert(kPieceLoads * kSecondWaves == kTileLoads, "pieces fill the waves' loads");
    int row_at[kLoadsPerWave], source[kLoadsPerWave];   // LDS offset of the row's address, offset in the row
#pragma unroll
    for (int i = 0; i < kPieceLoads; ++i) {
      const int p = (i * kSecondWaves + sw) * kWave + lane, key = p / kTilePieces;
      row_at[i] = 8 * key;
      source[i] = (p % kTilePieces ^ swizzle(key)) * 16;
    }
    row_at[kPieceLoads] = 8 * (lane % kTileKeys);
    source[kPieceLoads] = kLatentScaleAt + 4 * sw;
    const uint8_t* row[kLoadsPerWave];
    auto read_rows = [&](int tile) {
      const uint32_t rows = lds_address(s.row) + min(tile, max(tiles - 1, 0)) * kTileKeys * 8;
#pragma unroll
      for (int i = 0; i < kLoadsPerWave; ++i) row[i] = lds_get<const uint8_t*>(rows + row_at[i]);
    };
    auto issue = [&](int tile) {
      const int at = tile % TILES;
      const uint32_t ring = lds_address(s.ring) + at * kTileBytes;
#pragma unroll
      for (int i = 0; i < kPieceLoads; ++i) lds_load16(row[i] + source[i], ring + (i * kSecondWaves + sw) * kWave * 16);
      if (lane < kTileKeys)
        lds_load4(row[kPieceLoads] + source[kPieceLoads], lds_address(s.scale) + (at * kLatentGroups + sw) * kTileKeys * 4);
    };
    // A drafted token is seen by some nodes only, and 0 x NaN in the second product would reach the others: NaN
    // codes and scales that are not finite become 0, and `bad` tells the softmax of the nodes that see them. Each
    // wave looks at what it has loaded, when that has arrived and before the others are told.
    auto clean = [&](int tile) {
      if (tile >= tiles || key0 / kTileKeys + tile < a.history_tiles) return;
      const uint32_t ring = lds_address(s.ring) + tile % TILES * kTileBytes;
#pragma unroll 1
      for (int i = 0; i < kPieceLoads; ++i) {
        const int p = (i * kSecondWaves + sw) * kWave + lane, key = p / kTilePieces;
        if ((p % kTilePieces ^ swizzle(key)) >= kRopeAt / 16) continue;   // rotary channels
        bool any = false;
        const vec4u v = without_nan_codes(lds_get<vec4u>(ring + p * 16), any);
        if (any) {
          lds_put(ring + p * 16, v);
          atomicOr(&s.bad[tile], 1u << key);
        }
      }
      if (lane < kTileKeys && !(fabsf(s.scale[tile % TILES][sw][lane]) < __builtin_inff())) {
        s.scale[tile % TILES][sw][lane] = 0.0f;
        atomicOr(&s.bad[tile], 1u << lane);
      }
    };
#pragma unroll 1
    for (int t = 0; t < TILES - 1 && t < tiles; ++t) {
      read_rows(t);
      issue(t);
    }
    // voff: the row (key) this lane names in a transposed read of keys 0..15, and the
    // channels of its 16 lanes; 32-channel tile t is ^ (t << 5).
    const int vkey = 8 * half + col / 2;
    const int voff = vkey * kLatentScaleAt + (((quad % 2) ^ swizzle(vkey)) << 4) + (col & 1) * 8 + sw * kScaleGroup;
    static_assert(kLatentScaleAt % 128 == 0 && kTileBytes % 128 == 0, "the swizzle's bits are free in every row address");
    // this lane's chunk of head col32: keys 8 half .. of a tile's first 16
    const uint32_t pread = lds_address(s.p) +
                           (kTwo ? col32 * kTileKeys * 4 + ((2 * half ^ ((col32 >> 1) & 7)) << 4)
                                   : (sw * kHeads + col32) * kTileKeys * 2 + ((half ^ ((col32 >> 2) & 3)) << 4));
    float minus = -1.0f;                          // one the compiler does not know: a fused step takes it, a difference two
    asm volatile("" : "+s"(minus));
    if (tiles >= TILES - 1) wait_loads<(TILES - 2) * kLoadsPerWave>();
    else wait_loads<0>();
    if constexpr (TREE) clean(0);
    barrier_keep_loads();
    read_rows(TILES - 1);
#pragma unroll 1
    for (int tile = -1; tile < tiles; ++tile) {
      // tiles up to tile + TILES - 2 (at least TILES - 2) were issued; tile + 2 must have arrived
      if (tile < 0 ? tiles >= TILES - 1 : tile + TILES - 1 <= tiles)
        wait_loads<(TILES - 4) * kLoadsPerWave>();
      else
        wait_loads<0>();
      if constexpr (TREE) clean(tile + 2);
      barrier_keep_loads();
      if (tile < 0) continue;
      const int buf = tile & 1;
      const uint32_t vrow = opaque(lds_address(s.ring) + tile % TILES * kTileBytes + voff);
      // the second 16 keys: ^ 32, or ^ 64 in 32 bits
      const uint32_t prow = opaque(pread + buf * (uint32_t)sizeof(s.p[0]));
      const vec4u mv = lds_get<vec4u>(lds_address(s.moved) + buf * 16);
      i32x2 v8[CT][2];
      f16x8 p[HT][2], rest[HT][2];
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) v8[t][x] = lds_read_transposed((vrow ^ (t << 5)) + x * 16 * kLatentScaleAt);
#pragma unroll
      for (int h = 0; h < HT; ++h)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if constexpr (kTwo) {
            const uint32_t scale = lds_address(s.scale) + ((tile % TILES * kLatentGroups + sw) * kTileKeys + 16 * x + 8 * half) * 4;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const f32x4 w = lds_get<f32x4>((prow ^ (64 * x + 16 * y)) + 32 * h * kTileKeys * 4);
              const f32x4 sc = lds_get<f32x4>(scale + 16 * y);
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                // (the empty assembly keeps the product and its rounding one step each for both uses)
                f32x2 v = {w[e] * sc[e], w[e + 1] * sc[e + 1]};
                asm("" : "+v"(v));
                f16x2 hi = __builtin_convertvector(v, f16x2);
                asm("" : "+v"(hi));
                rest[h][x][4 * y + e] = (_Float16)__builtin_fmaf((float)hi.x, minus, v.x);
                rest[h][x][4 * y + e + 1] = (_Float16)__builtin_fmaf((float)hi.y, minus, v.y);
                p[h][x][4 * y + e] = hi.x;
                p[h][x][4 * y + e + 1] = hi.y;
              }
            }
          } else {
            p[h][x] = lds_get<f16x8>((prow ^ (32 * x)) + 32 * h * kTileKeys * 2);
          }
        }
      if (tile + TILES - 1 < tiles) issue(tile + TILES - 1);
      if (__builtin_amdgcn_readfirstlane(mv.x | mv.y | mv.z | mv.w)) {   // a reference moved: O's factors
#pragma unroll
        for (int h = 0; h < HT; ++h) {
          const float al = lds_get<float>(lds_address(s.alpha) + (buf * kHeads + 32 * h + col32) * 4);
#pragma unroll
          for (int t = 0; t < CT; ++t) scale_in_place(o[t][h], al);
        }
      }
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const f16x8 v = widen8<f16x8>((uint32_t)v8[t][x].x, (uint32_t)v8[t][x].y);
#pragma unroll
          for (int h = 0; h < HT; ++h) {
            o[t][h] = mfma32(v, p[h][x], o[t][h]);
            if constexpr (kTwo) o[t][h] = mfma32(v, rest[h][x], o[t][h]);
          }
        }
      read_rows(tile + TILES);
    }
  } else {
    QueryRaw<Q8> raw[HT];
    const ReaderState state = reader_state(g);
    if constexpr (TREE) {
      for (int i = threadIdx.x; i < kItemKeys<TREE> / kTileKeys + 2; i += kFirstWaves * kWave) s.bad[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < HT; ++i) {
      const int head = hb * kHeads + head0 + 16 * i + col;
      const bool any = head < a.heads;
      const uint16_t* p = static_cast<const uint16_t*>(a.q) + set * a.q_set_stride;
      if constexpr (TREE) {
        const int node = (int)a.by_heads.div(head);
        p += node * a.q_node_stride + (head - node * (int)a.by_heads.d) * a.q_head_stride;
        if (quad == 0 && key_half == 0) {
          const unsigned long long sees = any ? a.visible[(size_t)set * a.nodes + node] : 0;
          s.sees[0][head0 + 16 * i + col] = (uint32_t)sees;
          s.sees[1][head0 + 16 * i + col] = (uint32_t)(sees >> 32);
        }
      } else {
        p += head * a.q_head_stride;
      }
      if (a.q_aligned) raw[i].template load<true>(p, any, quad);
      else raw[i].template load<false>(p, any, quad);
    }
    if (threadIdx.x == 0) s.ok = reader_ready(g, state, a.want_flag);
    barrier_keep_loads();
    if (!s.ok) return;
    // Tiles behind the last one are computed on whatever lies in their place and
    // masked, so that the main loop has no branches. (Read a barrier later or more.)
    if (threadIdx.x < 2) s.live[tiles + threadIdx.x] = 0;
    if (threadIdx.x < 8) s.moved[threadIdx.x / 4][threadIdx.x % 4] = 0;   // one wave of two writes its heads'
    QueryOperand<Q8> q[HT];
#pragma unroll
    for (int i = 0; i < HT; ++i) {
      q[i].take(raw[i]);
      m[i] = -__builtin_inff();
      l[i] = 0.0f;
    }
    const float c_log2 = a.scale_log2;
    // Register r in quad x is key 8 x + 4 key_half + r. koff: this lane's key as an
    // operand, piece quad of a scale block; piece 4 + quad is ^ 64.
    const int key = 8 * (col / 4) + 4 * key_half + col % 4;
    const int koff = key * kLatentScaleAt + ((quad ^ swizzle(key)) << 4);
    const int head = head0 + col;
    const uint32_t pwrite = lds_address(s.p) +
                            (kTwo ? head * kTileKeys * 4 + (((2 * quad + key_half) ^ ((head >> 1) & 7)) << 4)
                                    : head * kTileKeys * 2 + ((quad ^ ((head >> 2) & 3)) << 4) + 8 * key_half);
    const uint32_t at_top = lds_address(s.top) + head * 8;
    f32x4 sc[kLatentGroups], S[HT];                // of the next tile for the softmax: scales, logits in powers of two
    // First product of a tile in LDS; the largest logarithm of p x scale of each
    // head, over this half of the keys, goes to the wave with the other half.
    vec4u ahead[2];                                // a tree: the first block's keys of the next tile
    auto first_keys = [&](int tile) {
      const uint32_t krow = lds_address(s.ring) + tile % TILES * kTileBytes + koff;
      ahead[0] = lds_get<vec4u>(krow);
      ahead[1] = lds_get<vec4u>(krow ^ 64);
    };
    auto logits = [&](int tile) {
      const uint32_t krow = opaque(lds_address(s.ring) + tile % TILES * kTileBytes + koff);
      const uint32_t krow64 = opaque(krow ^ 64);
      const uint32_t scale = opaque(lds_address(s.scale) + (tile % TILES * kLatentGroups * kTileKeys + 8 * quad + 4 * key_half) * 4);
      bf16x8 kr[2] = {lds_get<bf16x8>(krow + kRopeAt), lds_get<bf16x8>(krow64 + kRopeAt)};
      const uint32_t live = __builtin_amdgcn_readfirstlane(s.live[tile]);
      const int draft = TREE ? key0 / kTileKeys + tile - a.history_tiles : -1;   // a tile of drafted tokens, or < 0
      const bool masked = !TREE || live != ~0u || draft >= 0;   // without a tree the keys take longer than masks
      f32x4 part[HT][kLatentGroups], rope[HT];
#pragma unroll
      for (int b = 0; b < kLatentGroups; ++b) {
        sc[b] = lds_get<f32x4>(scale + kTileKeys * b * 4);
        const vec4u k0 = TREE && b == 0 ? ahead[0] : lds_get<vec4u>(krow + b * kScaleGroup);
        const vec4u k1 = TREE && b == 0 ? ahead[1] : lds_get<vec4u>(krow64 + b * kScaleGroup);
        const Q8 k[4] = {widen8<Q8>(k0.x, k0.y), widen8<Q8>(k0.z, k0.w), widen8<Q8>(k1.x, k1.y), widen8<Q8>(k1.z, k1.w)};
#pragma unroll
        for (int i = 0; i < HT; ++i) part[i][b] = q[i].block_product(b, k);
      }
#pragma unroll
      for (int i = 0; i < HT; ++i) rope[i] = q[i].rope_product(kr);
#pragma unroll
      for (int i = 0; i < HT; ++i) {
        S[i] = rope[i];
#pragma unroll
        for (int b = 0; b < kLatentGroups; ++b) S[i] += sc[b] * part[i][b];
      }
      __builtin_amdgcn_sched_barrier(0);          // the partial products' registers are free from here
      if constexpr (TREE) {
        const uint32_t spoilt = draft >= 0 ? __builtin_amdgcn_readfirstlane(s.bad[tile]) : 0;
        if (spoilt) {                               // drafted tokens that make those who see them NaN
#pragma unroll
          for (int i = 0; i < HT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (spoilt >> (8 * quad + 4 * key_half + r) & 1u) S[i][r] = __builtin_nanf("");
        }
      }
      // each key's largest scale as a power of two, from above: a key of large weight must not take a
      // neighbour's (p x scale would then vanish in fp16); scales below 2^-60 count as that
      float power[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float big = 0x1p-60f;
#pragma unroll
        for (int b = 0; b < kLatentGroups; ++b) big = fmaxf(big, fabsf(sc[b][r]));
        power[r] = (float)__builtin_amdgcn_frexp_expf(big);
      }
#pragma unroll
      for (int i = 0; i < HT; ++i) {
        float top = -__builtin_inff();
        S[i] *= c_log2;
        if (masked) {
          uint32_t mine = live;
          if constexpr (TREE) {
            if (draft >= 0) mine &= lds_get<uint32_t>(lds_address(s.sees) + ((draft & 1) * kHeads + head + 16 * i) * 4);
          }
          mine >>= 8 * quad + 4 * key_half;
#pragma unroll
          for (int r = 0; r < 4; ++r) S[i][r] = mine & (1u << r) ? S[i][r] : -__builtin_inff();
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) top = fmaxf(top, S[i][r] + power[r]);
        top = max_quads(top);
        if (quad == 0) lds_put(at_top + (tile & 1) * kHeads * 8 + 16 * i * 8 + 4 * key_half, top);
      }
    };
    barrier_keep_loads();
    if constexpr (TREE) first_keys(0);
    logits(0);
#pragma unroll 1
    for (int tile = 0; tile <= tiles; ++tile) {   // softmax of `tile`, logits of the next one
      barrier_keep_loads();
      const int buf = tile & 1;
      bool moved = false;
      f32x2 both[HT];                             // both halves' waves come to the same reference
#pragma unroll
      for (int i = 0; i < HT; ++i) both[i] = lds_get<f32x2>(at_top + buf * kHeads * 8 + 16 * i * 8);
      if constexpr (TREE) first_keys(tile + 1);
#pragma unroll
      for (int i = 0; i < HT; ++i) {
        const float top = fmaxf(both[i].x, both[i].y);
        const bool move = top > m[i] + 15.0f;
        const float nm = move ? top - 8.0f : m[i];
        const float fall = move ? m[i] - nm : 0.0f, al = near_power(fall);
        m[i] = nm;
        l[i] = l[i] * far_power(fall) * al;       // (1% of the time; a branch around the far power costs as much)
        const float base = nm == -__builtin_inff() ? 0.0f : nm;
        f32x4 p;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          p[r] = __builtin_amdgcn_exp2f(S[i][r] - base);
          l[i] += p[r];
        }
        const uint32_t pw = opaque(pwrite + buf * (uint32_t)sizeof(s.p[0]) + 16 * i * kTileKeys * (kTwo ? 4 : 2));
        if constexpr (kTwo) {
          lds_put(pw, p);
        } else {
#pragma unroll
          for (int b = 0; b < kLatentGroups; ++b) {
            f16x4 w;
#pragma unroll
            for (int r = 0; r < 4; ++r) w[r] = (_Float16)(p[r] * sc[b][r]);
            lds_put(pw + b * kHeads * kTileKeys * 2, w);
          }
        }
        moved |= move;
        if (quad == 0 && key_half == 0) s.alpha[buf][head + 16 * i] = al;
      }
      moved = __any(moved);
      if (lane == 0 && key_half == 0) s.moved[buf][wave] = moved;
      logits(tile + 1);
    }
#pragma unroll
    for (int i = 0; i < HT; ++i) l[i] = sum_quads(l[i]);
  }

  // every second wave needs every head's l and m
  float* ml = reinterpret_cast<float*>(s.p);
  barrier_keep_loads();
  if (!second && quad == 0) {
#pragma unroll
    for (int i = 0; i < HT; ++i) {
      const int head = head0 + 16 * i + col;
      ml[head] = m[i];
      ml[(1 + key_half) * kHeads + head] = l[i];
    }
  }
  barrier_keep_loads();
  float inv[HT];
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    const float lh = ml[kHeads + 32 * h + col32] + ml[2 * kHeads + 32 * h + col32];
    inv[h] = lh != 0.0f ? 1.0f / lh : 0.0f;
    const int head = hb * kHeads + 32 * h + col32;
    if (wave == 0 && half == 0 && head < a.heads) {
      const float lse2 = lh != 0.0f ? ml[32 * h + col32] + log2f(lh) : -__builtin_inff();
      if (splits > 1) a.part_lse[((size_t)(set - a.whole) * a.heads + head) * splits + split] = lse2;
      else if (a.lse) a.lse[(size_t)set * a.heads + head] = lse2 * kLn2;
    }
  }
  if (splits > 1) {   // this split's own result in 32 bits, joined by k_attend_join
    float* po = a.part_o + ((size_t)(set - a.whole) * a.heads * splits + split) * kLatent;
    store_heads<float>(s.ring[0], o, inv, hb * kHeads, a.heads, [&](int head, int ch, const vec4u v) {
      *reinterpret_cast<vec4u*>(po + (size_t)head * splits * kLatent + ch) = v;
    });
  } else {
    uint16_t* out = static_cast<uint16_t*>(a.out) + set * a.out_set_stride;
    const bool aligned = a.out_aligned;
    using Out = std::conditional_t<std::is_same_v<Q8, bf16x8>, __bf16, _Float16>;
    store_heads<Out>(s.ring[0], o, inv, hb * kHeads, a.heads, [&](int head, int ch, const vec4u v) {
      uint16_t* p = out + ch;
      if constexpr (TREE) {
        const int node = (int)a.by_heads.div(head);
        p += node * a.out_node_stride + (head - node * (int)a.by_heads.d) * a.out_head_stride;
      } else {
        p += head * a.out_head_stride;
      }
      if (aligned) {
        *reinterpret_cast<vec4u*>(p) = v;
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
      }
    });
  }
}

// Joins the splits of one (set, head): o = sum_s w_s o_s / sum_s w_s with
// w_s = 2^(lse_s - max lse). Bound by the latency of its reads, not their bytes:
// a workgroup reads as many splits at a time as its threads cover, whose sums
// meet in LDS, and the first of them while it finds the largest lse (16 sets, 32
// heads, 16 splits of 128 channels: 10.2 us with 32 threads that read one split
// after another, 4.2 us so).
template <typename Q8>
__global__ __launch_bounds__(kJoinThreads) void k_attend_join(GroupDev g, AttendDev a, int width) {
  constexpr int kJoinWaves = kJoinThreads / kWave;
  __shared__ int ok;
  __shared__ float s_w[kAttendMaxSplits];
  __shared__ float s_red[kJoinWaves];
  __shared__ f32x4 s_acc[kJoinThreads];
  const ReaderState state = reader_state(g);
  const size_t row = blockIdx.x;
  // `per` threads read a split's row; thread group `at` takes splits at, at + groups, ..
  const int per = width / 4, groups = kJoinThreads / per;
  const int at = threadIdx.x / per, c = 4 * (threadIdx.x % per);
  const float* po = a.part_o + row * a.splits * width + c;
  constexpr int kAhead = 4;                       // on their way while the weights are computed
  f32x4 first[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (at + u * groups < a.splits) first[u] = *reinterpret_cast<const f32x4*>(po + (size_t)(at + u * groups) * width);
  if (threadIdx.x == 0) ok = reader_ready(g, state, a.want_flag);
  const float* lse = a.part_lse + row * a.splits;
  float top = -__builtin_inff();
  for (int i = threadIdx.x; i < a.splits; i += kJoinThreads) top = fmaxf(top, s_w[i] = lse[i]);
  for (int d = kWave / 2; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
  if (lane_id() == 0) s_red[threadIdx.x / kWave] = top;
  barrier_keep_loads();
  if (!ok) return;
#pragma unroll
  for (int w = 0; w < kJoinWaves; ++w) top = fmaxf(top, s_red[w]);
  const float base = top == -__builtin_inff() ? 0.0f : top;
  f32x4 acc{};
  float sum = 0.0f;                               // of the group's splits
  auto add = [&](int i, const f32x4& v) {
    const float w = exp2f(s_w[i] - base);
    sum += w;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += w * v[e];
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (at + u * groups < a.splits) add(at + u * groups, first[u]);
#pragma unroll 4
  for (int i = at + kAhead * groups; i < a.splits; i += groups)
    add(i, *reinterpret_cast<const f32x4*>(po + (size_t)i * width));
  s_acc[threadIdx.x] = acc;
  __syncthreads();                                // every weight was read: s_w holds the groups' sums from here
  if (c == 0) s_w[at] = sum;
  __syncthreads();
  if (at != 0) return;
  for (int j = 1; j < groups; ++j) {
    const f32x4 v = s_acc[threadIdx.x + j * per];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += v[e];
    sum += s_w[j];
  }
  const int set = (int)(row / a.heads), at_head = (int)(row % a.heads);
  const int node = (int)a.by_heads.div(at_head), head = at_head - node * (int)a.by_heads.d;
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = acc[e] * inv;
  store4<Q8>(static_cast<uint16_t*>(a.out) + set * a.out_set_stride + node * a.out_node_stride + head * a.out_head_stride + c, v,
             a.out_aligned);
  if (threadIdx.x == 0 && a.lse) a.lse[row] = sum != 0.0f ? (top + log2f(sum)) * kLn2 : -__builtin_inff();
}

// The join of few splits of many rows, as a tree's are (46848 rows of 64 channels in 2
// splits: 54 us with a workgroup a row as above, about 12 us so): width / 4 threads a row.
template <typename Q8>
__global__ __launch_bounds__(kJoinThreads) void k_tree_join(GroupDev g, AttendDev a, int width, int rows) {
  const ReaderState state = reader_state(g);
  const int per = width / 4;
  const int row = blockIdx.x * (kJoinThreads / per) + threadIdx.x / per, c = threadIdx.x % per * 4;
  if (row >= rows) return;
  const float* lse = a.part_lse + (size_t)row * a.splits;
  const float* po = a.part_o + (size_t)row * a.splits * width + c;
  float w[kFewSplits], top = -__builtin_inff();
  f32x4 v[kFewSplits];
#pragma unroll
  for (int i = 0; i < kFewSplits; ++i) {
    if (i >= a.splits) break;
    w[i] = lse[i];
    v[i] = *reinterpret_cast<const f32x4*>(po + (size_t)i * width);
  }
  if (state.status || state.flag != a.want_flag) return;       // the attention said so
#pragma unroll
  for (int i = 0; i < kFewSplits; ++i) {
    if (i >= a.splits) break;
    top = fmaxf(top, w[i]);
  }
  const float base = top == -__builtin_inff() ? 0.0f : top;
  f32x4 acc{};
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kFewSplits; ++i) {
    if (i >= a.splits) break;
    const float x = exp2f(w[i] - base);
    sum += x;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(x, v[i][e], acc[e]);
  }
  const int set = row / a.heads, at_head = row % a.heads;
  const int node = (int)a.by_heads.div(at_head), head = at_head - node * (int)a.by_heads.d;
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  const float out[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
  store4<Q8>(static_cast<uint16_t*>(a.out) + set * a.out_set_stride + node * a.out_node_stride + head * a.out_head_stride + c, out,
             a.out_aligned);
  if (c == 0 && a.lse) a.lse[row] = sum != 0.0f ? (top + log2f(sum)) * kLn2 : -__builtin_inff();
}

// How a call's heads and keys are split over workgroups (one per compute unit at
// a time): 32 or 64 heads each, and the number of splits, with the least estimated
// time in us. A workgroup takes 0.85 us (32 heads) or 1.2 us (64) per tile and 14
// or 20 us for its start and end (lookups, q, results). With more than one split
// the join costs a launch, on the host too (7; 4 on the device), a part for each
// row and one for each split of a row. Measured, kernel + join, us:
//   sets x heads, keys   32 heads a workgroup, splits         64 heads, splits
//   1 x 16, 2048         8: 19   16: 16   32: 16   64: 15
//   4 x 16, 256          1: 14   2: 16    4: 13    8: 13
//   4 x 64, 2048         8: 22   16: 20   32: 22              8: 29   16: 26   32: 27
//   16 x 128, 2048       1: 63   2: 45    4: 36               4: 45   8: 37
//   64 x 128, 2048       1: 73   2: 95                        1: 101  2: 79
//   64 x 64, 700         1: 29   2: 32                        1: 42   2: 40
//   160 x 64, 2048       1: 132  3: 141                       1: 101  3: 114
AttendPlan plan_attend_latent(int n_sets, int k, int heads) {
  AttendPlan best{};
  const int tiles = (k + kTileKeys - 1) / kTileKeys;
  const int least = std::max(1, (k + kAttendKeys - 1) / kAttendKeys);
  const double rows = (double)n_sets * heads;
  double best_cost = 0;
  for (const int wg_heads : {32, 64}) {
    const int head_blocks = (heads + wg_heads - 1) / wg_heads;
    if (wg_heads == 64 && head_blocks == (heads + 31) / 32) break;   // the same workgroups, half empty
    const long long base = (long long)n_sets * head_blocks;
    const double tile_us = wg_heads == 32 ? 0.85 : 1.2, start_us = wg_heads == 32 ? 14.0 : 20.0;
    for (int want = least; want <= std::max(least, std::min(tiles, kComputeUnits)); ++want) {
      const int per = std::max(1, (tiles + want - 1) / want);   // tiles per split
      const int splits = std::max(1, (tiles + per - 1) / per);
      if (splits != want && want != least) continue;            // the same split as a smaller one
      double cost = (double)((base * splits + kComputeUnits - 1) / kComputeUnits) * (per * tile_us + start_us);
      if (splits > 1) cost += 7 + 9e-4 * rows + 2e-4 * rows * splits;
      if (best.splits == 0 || cost < best_cost) {
        best_cost = cost;
        best = {splits, per * kTileKeys, head_blocks};
      }
    }
  }
  return best;
}

// The same for a tree, where sets that fill the compute units evenly stay whole and the
// others are split, so that the last round of workgroups is a short one and the join
// has the rest alone. A tile is taken for 1.25 us here (64 rows; 0.9 for 32), a start and end
// for 15; with 1.6 and 1.1, which a tile with weights in two parts is nearer to, 18 calls of
// 1 to 257 sets took the same time to 2% but for 4 sets x 128 rows x 256 keys (22.3 us so, 23.5).
// Measured, all sets the same way and so, us a call: 24 sets x 1024 rows x 2048 keys 238,
// 206; 33 x 1024 x 1024 200, 162; 70 x 256 x 1024 133, 100.
AttendPlan plan_tree_latent(int n_sets, int tiles, int rows) {
  static_assert(kTileTokens == kTileKeys, "a tree's tiles are those of the kernel");
  AttendPlan best{};
  constexpr int kMostTiles = kItemKeys<true> / kTileKeys;
  double best_cost = 0;
  for (const int wg_rows : {32, 64}) {
    const int blocks = (rows + wg_rows - 1) / wg_rows;
    if (wg_rows == 64 && blocks == (rows + 31) / 32) break;        // the same workgroups, half empty
    const double tile_us = wg_rows == 32 ? 0.9 : 1.25, start_us = 15.0;
    const int rounds = (int)((long long)n_sets * blocks / kComputeUnits);   // full ones
    for (const int whole : {0, tiles <= kMostTiles ? (int)((long long)rounds * kComputeUnits / blocks) : 0}) {
      if (whole == n_sets) continue;                               // as no split at all
      const long long base = (long long)(n_sets - whole) * blocks;
      const int least = (tiles + kMostTiles - 1) / kMostTiles;
      for (int want = std::max(1, least); want <= std::max(std::max(1, least), std::min(tiles, kComputeUnits)); ++want) {
        const int per = std::max(1, (tiles + want - 1) / want), splits = std::max(1, (tiles + per - 1) / per);
        if (splits != want && want != least) continue;             // the same split as a smaller one
        double cost = (whole ? rounds : 0) * (tiles * tile_us + start_us) +
                      (double)((base * splits + kComputeUnits - 1) / kComputeUnits) * (per * tile_us + start_us);
        if (splits > 1) cost += 7 + (n_sets - whole) * (double)rows * (9e-4 + 2e-4 * splits);
        if (best.splits == 0 || cost < best_cost) {
          best_cost = cost;
          best = {splits, per * kTileKeys, blocks, 0, splits > 1 ? whole : 0};
        }
      }
    }
  }
  return best;
}

template <typename Q8, bool TREE>
static hipError_t launch_latent(const GroupDev& g, const AttendDev& a, int n_sets, hipStream_t s) {
  const int blocks = (a.whole + (n_sets - a.whole) * a.splits) * a.head_blocks;
  if (a.head_blocks == (a.heads + 31) / 32) k_attend_latent<Q8, 1, 5, TREE><<<blocks, kWaves * kWave, 0, s>>>(g, a);
  else k_attend_latent<Q8, 2, 5, TREE><<<blocks, kWaves * kWave, 0, s>>>(g, a);
  return hipGetLastError();
}

hipError_t launch_attend_latent(const GroupDev& g, const AttendDev& a, int type, int n_sets, hipStream_t s) {
  return type == ULA_BF16 ? launch_latent<bf16x8, false>(g, a, n_sets, s) : launch_latent<f16x8, false>(g, a, n_sets, s);
}

hipError_t launch_tree_latent(const GroupDev& g, const AttendDev& a, int type, int n_sets, hipStream_t s) {
  return type == ULA_BF16 ? launch_latent<bf16x8, true>(g, a, n_sets, s) : launch_latent<f16x8, true>(g, a, n_sets, s);
}

hipError_t launch_attend_join(const GroupDev& g, const AttendDev& a, int type, int n_sets, int width, hipStream_t s) {
  const int blocks = n_sets * a.heads;
  if (a.nodes && a.splits <= kFewSplits) {
    const int per = kJoinThreads / (width / 4), few = (blocks + per - 1) / per;
    if (type == ULA_BF16) k_tree_join<bf16x8><<<few, kJoinThreads, 0, s>>>(g, a, width, blocks);
    else k_tree_join<f16x8><<<few, kJoinThreads, 0, s>>>(g, a, width, blocks);
    return hipGetLastError();
  }
  if (type == ULA_BF16) k_attend_join<bf16x8><<<blocks, kJoinThreads, 0, s>>>(g, a, width);
  else k_attend_join<f16x8><<<blocks, kJoinThreads, 0, s>>>(g, a, width);
  return hipGetLastError();
}

}  // namespace ula
