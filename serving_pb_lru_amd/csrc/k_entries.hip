// Copies of entries under new addresses (fork) and entries under new addresses
// without a copy (rename).
//
// UlaCache summary (paper-daily.com), section 2: the engine names entries by
// logical address only and the library places them, so a copy is placed as an
// append is, and a change of address changes the mapping table and the owner
// words alone; section 1: in a shared pool the space of one request serves the
// others.
//
// An entry's rows are in its GPU slot, in its host slot, or, if the last step
// evicted it and its write-back has not run, in that step's staging buffer; the
// copies read them where they are.
#include <algorithm>

#include "device_util.h"

namespace ula {

// Where the rows of the entry at `loc` (its mapping table word) are now.
__device__ __forceinline__ const uint8_t* rows_at(const GroupDev& g, uint32_t loc, uint32_t staged_step) {
  if (!(loc & kHostBit)) return g.pool + (size_t)loc * g.slot_bytes;
  const uint32_t h = loc & ~kHostBit;
  const unsigned long long st = g.hs_stage[h];
  if (staged_step != 0 && (uint32_t)(st >> 32) == staged_step) return g.evict_rows + (size_t)(uint32_t)st * g.slot_bytes;
  return g.host + (size_t)h * g.slot_bytes;
}

// Entry i of the chunk (source address src0 + i) into the place chosen for it
// (app_dst[i]: a free slot, so never one that is read here), published as
// address dst0 + i. One read and one write of every row; four pieces per lane in
// flight. The loads of a location are the same for a row's 16-byte pieces and
// hit the caches. (Pieces are counted in 32 bits: a configuration's max_append
// has fewer than 2^31, and a step of the loop is at most 2^23.)
__global__ __launch_bounds__(256) void k_fork_place(GroupDev g, int32_t src0, int32_t dst0, int32_t n,
                                                    FastDiv per_slot) {
  if (status_of(g.ctr)) return;
  const uint32_t staged = g.ctr->wb_step;
  const uint32_t chunks = (uint32_t)g.slot_bytes / 16u;
  const uint32_t total = (uint32_t)n * chunks;
  const uint32_t stride = gridDim.x * blockDim.x;
  constexpr int U = 4;
  for (uint32_t base = blockIdx.x * blockDim.x + threadIdx.x; base < total; base += U * stride) {
    vec4u v[U];
    uint32_t i[U], d[U];
    bool some[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t idx = base + u * stride;
      some[u] = false;
      if (idx < total) {
        i[u] = per_slot.div(idx);
        const uint32_t loc = g.map[src0 + (int32_t)i[u]];
        d[u] = g.app_dst[i[u]];
        if (loc == kAbsent) {             // the host checked this: an inconsistent state
          latch(g.ctr, ULA_ESTATE);
        } else {
          v[u] = reinterpret_cast<const vec4u*>(rows_at(g, loc, staged))[idx - i[u] * chunks];
          some[u] = true;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (some[u]) place_piece(g, d[u], base + u * stride - i[u] * chunks, dst0 + (int32_t)i[u], v[u]);
  }
}

// The chunk's rows and destination addresses into the append's staging buffers
// (for placements whose append moves GPU entries, among them sources, away).
__global__ __launch_bounds__(256) void k_fork_collect(GroupDev g, int32_t src0, int32_t dst0, int32_t n,
                                                      FastDiv per_slot) {
  if (status_of(g.ctr)) return;
  const uint32_t staged = g.ctr->wb_step;
  const uint32_t chunks = (uint32_t)g.slot_bytes / 16u;
  const uint32_t total = (uint32_t)n * chunks;
  for (uint32_t idx = blockIdx.x * blockDim.x + threadIdx.x; idx < total; idx += gridDim.x * blockDim.x) {
    const uint32_t i = per_slot.div(idx), c = idx - i * chunks;
    const uint32_t loc = g.map[src0 + (int32_t)i];
    if (c == 0) g.app_la[i] = dst0 + (int32_t)i;
    if (loc == kAbsent) {
      latch(g.ctr, ULA_ESTATE);
      continue;
    }
    reinterpret_cast<vec4u*>(g.app_rows)[idx] = reinterpret_cast<const vec4u*>(rows_at(g, loc, staged))[c];
  }
}

// Entry `loc` at its new address.
__device__ __forceinline__ void put_renamed(const GroupDev& g, uint32_t loc, int32_t la) {
  if (loc == kAbsent) {            // the host checked this: an inconsistent state
    latch(g.ctr, ULA_ESTATE);
    return;
  }
  g.map[la] = loc;
  if (loc & kHostBit) g.hown[loc & ~kHostBit] = la;
  else g.gown[loc] = la;
}

// Rename of a chunk: every location is taken out of the table before any is put
// back, since the two address ranges may overlap. Up to kRenameSmall entries in
// one workgroup, whose barrier lies between; more in two launches. (257 entries
// forked, renamed, gathered and released: 49 us with two launches and the list of
// addresses that a release of one run no longer copies, 42 us so.)
constexpr int kRenameThreads = 1024, kRenameEach = 4, kRenameSmall = kRenameThreads * kRenameEach;

__global__ __launch_bounds__(kRenameThreads) void k_rename_small(GroupDev g, int32_t src0, int32_t dst0, int32_t n) {
  if (block_failed(g.ctr)) return;
  uint32_t loc[kRenameEach];
#pragma unroll
  for (int j = 0; j < kRenameEach; ++j) {
    const int i = j * kRenameThreads + (int)threadIdx.x;
    if (i < n) loc[j] = g.map[src0 + i];
  }
#pragma unroll
  for (int j = 0; j < kRenameEach; ++j) {
    const int i = j * kRenameThreads + (int)threadIdx.x;
    if (i < n) g.map[src0 + i] = kAbsent;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kRenameEach; ++j) {
    const int i = j * kRenameThreads + (int)threadIdx.x;
    if (i < n) put_renamed(g, loc[j], dst0 + i);
  }
}

__global__ __launch_bounds__(256) void k_rename_take(GroupDev g, int32_t src0, int32_t n) {
  if (status_of(g.ctr)) return;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
    g.app_dst[i] = g.map[src0 + i];
    g.map[src0 + i] = kAbsent;
  }
}

__global__ __launch_bounds__(256) void k_rename_put(GroupDev g, int32_t dst0, int32_t n) {
  if (status_of(g.ctr)) return;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x)
    put_renamed(g, g.app_dst[i], dst0 + i);
}

static int grid_of(size_t work, size_t per_block, int cap) {
  return (int)std::max<size_t>(1, std::min<size_t>((work + per_block - 1) / per_block, (size_t)cap));
}

hipError_t launch_fork_place(const GroupDev& g, int32_t src0, int32_t dst0, int32_t n, hipStream_t s) {
  const uint32_t chunks = (uint32_t)g.slot_bytes / 16u;
  k_fork_place<<<grid_of((size_t)n * chunks, 4 * 256, 8192), 256, 0, s>>>(g, src0, dst0, n, FastDiv(chunks));
  return hipGetLastError();
}

hipError_t launch_fork_collect(const GroupDev& g, int32_t src0, int32_t dst0, int32_t n, hipStream_t s) {
  const uint32_t chunks = (uint32_t)g.slot_bytes / 16u;
  k_fork_collect<<<grid_of((size_t)n * chunks, 256, 4096), 256, 0, s>>>(g, src0, dst0, n, FastDiv(chunks));
  return hipGetLastError();
}

hipError_t launch_rename(const GroupDev& g, int32_t src0, int32_t dst0, int32_t n, hipStream_t s) {
  if (n <= kRenameSmall) {
    k_rename_small<<<1, kRenameThreads, 0, s>>>(g, src0, dst0, n);
    return hipGetLastError();
  }
  const int blocks = grid_of(n, 256, 1024);
  k_rename_take<<<blocks, 256, 0, s>>>(g, src0, n);
  k_rename_put<<<blocks, 256, 0, s>>>(g, dst0, n);
  return hipGetLastError();
}

}  // namespace ula
