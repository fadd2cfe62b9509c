// The two row formats that the attention kernels read and the row writer writes,
// and the wave-level pieces those kernels share.
//
// UlaCache summary (paper-daily.com), section 4: the KV cache is held in FP8;
// section 1: the latent representation is shared by every query head. The
// residency kernels move rows as opaque bytes; only the kernels that include
// this file look inside.
//
//   latent  512 e4m3 channels | 64 bf16 rotary channels | 4 fp32 scales (one per
//           128 channels): 656 bytes. key = [latent, rotary], value = latent.
//   heads   keys e4m3 [kv_heads][block][dim] | values, the same | key scales fp32
//           [kv_heads] | value scales fp32 [kv_heads] | int32 tokens in the
//           block | zeros up to a multiple of 16 bytes.
#pragma once

#include "device_util.h"

namespace ula {

constexpr int kLatent = 512;
constexpr int kScaleGroup = 128;
constexpr int kLatentGroups = kLatent / kScaleGroup;
constexpr int kRope = 64;
constexpr int kRopeAt = kLatent;                       // byte offsets inside a latent row
constexpr int kLatentScaleAt = kLatent + 2 * kRope;
constexpr int kLatentRow = kLatentScaleAt + 4 * kLatentGroups;
static_assert(kLatentRow == 656, "latent row bytes");
constexpr float kE4m3Max = 448.0f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kAttendKeys = 2048;                      // most keys one latent work item takes
constexpr int kAttendMaxSplits = 1024;             // parts of a row that the join takes
constexpr int kJoinThreads = 256;

// Device arguments of an attention call.
struct AttendDev {
  const int32_t* sel;
  const void* q;
  void* out;
  float* lse;              // nullable
  float* part_o;           // [n_sets][heads][splits][width] when splits > 1
  float* part_lse;         // [n_sets][heads][splits], base 2
  long long q_set_stride, q_head_stride, out_set_stride, out_head_stride;   // elements
  long long want_flag;
  float scale_log2;        // scale x log2(e)
  int32_t k, heads, layer, n_res;
  int32_t splits, split_keys, head_blocks;
  int32_t q_aligned, out_aligned;   // 16-byte vector accesses are possible
  int32_t kv_heads, block_shift;    // heads rows
};

// Rotary positions: pair i turns by pos[axis] x turns[i] turns; the axis is 0 for
// i < end0, 1 for i < end1, else 2.
constexpr int kMostPairs = 128;
struct RotaryDev {
  double turns[kMostPairs];
  int32_t axes, end0, end1, interleaved;
};

// Device arguments of the row writer: a and b are the latent and rotary channels
// of latent rows, the keys and values of heads rows.
struct PackDev {
  const void* a;
  const void* b;
  const int32_t* positions;   // nullable
  const int32_t* count;       // nullable (heads rows)
  uint8_t* rows;
  long long a_stride[4], b_stride[4];   // elements: entry, layer, token, head
  int32_t n, layers, latent, aligned;
  int32_t kv_heads, head_dim, block_tokens, row_bytes;
};

struct RotateDev {
  const void* x;
  void* out;
  const int32_t* positions;
  long long x_stride[2], out_stride[2];   // elements: token, head
  int32_t n, heads, dim, inverse, aligned;
  int32_t tokens_per_block, heads_per_block;
};

hipError_t launch_pack(const PackDev& a, const RotaryDev& rot, int type, hipStream_t s);
long long pack_heads_blocks(const PackDev& a);   // workgroups of heads rows, of either side
long long plan_rotate(RotateDev* a);   // fills the workgroup's part in; how many there are
hipError_t launch_rotate(const RotateDev& a, const RotaryDev& rot, int type, hipStream_t s);

struct AttendPlan {
  int32_t splits, split_keys, head_blocks;
};

AttendPlan plan_attend_latent(int n_sets, int k, int heads);
AttendPlan plan_attend_heads(int n_sets, int tokens, int heads, int kv_heads);

hipError_t launch_attend_latent(const GroupDev& g, const AttendDev& a, int type, int n_sets, hipStream_t s);
hipError_t launch_attend_heads(const GroupDev& g, const AttendDev& a, int type, int n_sets, int head_dim,
                               hipStream_t s);
hipError_t launch_attend_join(const GroupDev& g, const AttendDev& a, int type, int n_sets, int width, hipStream_t s);

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// Eight e4m3 codes (low byte first) as bf16 or fp16: exact, both hold every e4m3
// value, so the scales can wait until the products are in 32 bits.
template <typename V8>
__device__ __forceinline__ V8 widen8(uint32_t lo, uint32_t hi) {
  V8 v;
  if constexpr (__is_same(V8, bf16x8)) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    v = V8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    v = V8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
  return v;
}

// D += A B with A 32 x 16, B 16 x 32: lane l holds row (column) l % 32 and the
// eight k from 8 (l / 32); D's column is l % 32, its register r the row
// 8 (r / 4) + 4 (l / 32) + r % 4.
__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
// The same with 16 x 32 and 32 x 16: lane l holds row (column) l % 16 and the
// eight k from 8 (l / 16); D's register r is row 4 (l / 16) + r.
__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// LDS addresses as 32-bit numbers: the compiler folds a constant added to one
// into the instruction's offset.
template <typename T>
__device__ __forceinline__ uint32_t lds_address(const T& x) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)&x;
}
template <typename T>
__device__ __forceinline__ T lds_get(uint32_t addr) {
  return *(const __attribute__((address_space(3))) T*)(uintptr_t)addr;
}

template <typename T>
__device__ __forceinline__ void lds_put(uint32_t addr, T v) {
  *(__attribute__((address_space(3))) T*)(uintptr_t)addr = v;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __builtin_inff() ? a : 0.0f;   // false for NaN too
}

// Four values as e4m3 codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

// A lane's value and that of the lane 32 away (16 away), in either order.
__device__ __forceinline__ float2 swap_halves(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t p = r[0], q = r[1];
  return make_float2(__builtin_bit_cast(float, p), __builtin_bit_cast(float, q));
}
__device__ __forceinline__ float2 swap_quads(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t p = r[0], q = r[1];
  return make_float2(__builtin_bit_cast(float, p), __builtin_bit_cast(float, q));
}
// Maximum (sum) over the lanes that share lane % 32, or lane % 16.
__device__ __forceinline__ float max_halves(float x) {
  const float2 v = swap_halves(x);
  return fmaxf(v.x, v.y);
}
__device__ __forceinline__ float sum_halves(float x) {
  const float2 v = swap_halves(x);
  return v.x + v.y;
}
__device__ __forceinline__ float max_quads(float x) {
  const float2 v = swap_quads(x);
  return max_halves(fmaxf(v.x, v.y));
}
__device__ __forceinline__ float sum_quads(float x) {
  const float2 v = swap_quads(x);
  return sum_halves(v.x + v.y);
}

// Transposing LDS read: 16 lanes name 8 rows of 16 bytes (lane pair 2r, 2r + 1
// the halves of row r); lane i receives byte i of rows 0..7.
__device__ __forceinline__ i32x2 lds_read_transposed(uint32_t addr) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)(uintptr_t)addr);
}

// Eight consecutive 16-bit elements from p (at least 2-byte aligned).
template <typename V8, bool ALIGNED16>
__device__ __forceinline__ V8 load8(const uint16_t* p) {
  if constexpr (ALIGNED16) {
    return *reinterpret_cast<const V8*>(p);
  } else {
    union { V8 v; uint16_t u[8]; } x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.u[i] = p[i];
    return x.v;
  }
}

// Four consecutive results as 16-bit values at p.
template <typename V8>
__device__ __forceinline__ void store4(uint16_t* p, const float* v, bool aligned8) {
  union { uint16_t u[4]; uint2 w; } x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (__is_same(V8, bf16x8)) x.u[e] = __builtin_bit_cast(uint16_t, (__bf16)v[e]);
    else x.u[e] = __builtin_bit_cast(uint16_t, (_Float16)v[e]);
  }
  if (aligned8) {
    *reinterpret_cast<uint2*>(p) = x.w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = x.u[e];
  }
}

// Entry r of a selection and of the step's resolved selection, as loaded: apart
// from their use, so that several lookups' loads are in flight at once.
struct Lookup {
  uint2 res;
  int32_t la;
};
__device__ __forceinline__ Lookup look_up(const GroupDev& g, const int32_t* __restrict__ sel, int r, int n_res) {
  return {r < n_res ? g.res[r] : make_uint2(kAbsent, kAbsent), sel[r]};
}

// Its GPU slot: from the resolved selection where that names the same address,
// else through the mapping table. kAbsent for padding and for an address that is
// not on the GPU (err says why).
__device__ __forceinline__ uint32_t slot_of(const GroupDev& g, const Lookup& at, int n_res, int& err) {
  const int32_t la = at.la;
  if (la == -1) return kAbsent;
  uint32_t slot = kAbsent;
  if (at.res.x == (uint32_t)la) {
    slot = at.res.y;
    if ((slot & kHostBit) && slot != kAbsent && (int32_t)(slot & ~kHostBit) < n_res) {
      const uint2 first = g.res[slot & ~kHostBit];   // a repeated miss
      slot = first.x == (uint32_t)la ? first.y : kAbsent;
    }
  }
  if (slot & kHostBit) {
    if (la < 0 || la >= g.N) {
      err = ULA_ERANGE;
      return kAbsent;
    }
    slot = g.map[la];
    if (slot & kHostBit) {
      err = ULA_ENOTRESIDENT;
      return kAbsent;
    }
  }
  return slot;
}

// Whether a reader of step want_flag's rows may go on (one thread's answer): the
// group has no latched error and its completion counter is at that step. The two
// loads are apart from the answer, as a lookup's are.
struct ReaderState {
  int status;
  long long flag;
};
__device__ __forceinline__ ReaderState reader_state(const GroupDev& g) {
  return {status_of(g.ctr), __hip_atomic_load(&g.ctr->flag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)};
}
__device__ __forceinline__ bool reader_ready(const GroupDev& g, const ReaderState& at, long long want_flag) {
  if (at.status) return false;
  if (at.flag == want_flag) return true;
  latch_gather(g.ctr, ULA_ENOTRESIDENT);
  return false;
}

}  // namespace ula
