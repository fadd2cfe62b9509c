// Sizes and device arguments of the selection of entries of least score (k_lightest.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ula {

constexpr int kLightSpan = 8192;          // addresses that one workgroup takes by itself
constexpr int kLightChunks = 64;          // most chunks of a longer range
constexpr int kLightBins = 2048;
constexpr int kLightRanges = 256;         // ranges of a launch, passed by value

// Chunks of a range (0: one workgroup has the whole of it), and their size.
__host__ __device__ constexpr int light_chunks(int length) {
  return length <= kLightSpan ? 0 : (length - 1) / kLightSpan + 1 < kLightChunks ? (length - 1) / kLightSpan + 1 : kLightChunks;
}
__host__ __device__ constexpr int light_chunk_size(int length) {
  const int chunks = light_chunks(length);
  return chunks ? (length - 1) / chunks + 1 : length;
}

struct LightRange {
  int32_t first, length, count;
};
struct LightRanges {
  int32_t n, first_range;                 // first_range: the number of range[0] among the call's
  LightRange range[kLightRanges];
};
// What a chunk of a long range tells the others.
struct alignas(32) LightChunkEnd {
  int32_t bin, need, before, within;      // of the range: the bin of its end, entries taken, in bins before, in the bin
  int32_t below, listed;                  // of the chunk: entries in bins before, in the bin
  int32_t unused[2];
};
struct LightDev {
  long long* scores;
  int32_t* out;                           // [ranges][most]
  uint32_t* bins;                         // long ranges: [chunks of all of them][kLightBins]
  LightChunkEnd* ends;                    // [chunks of all of them]
  unsigned long long* list;               // [addresses of all of them]
  int32_t most, mark;
};

hipError_t launch_lightest(const LightDev& a, const LightRanges& r, hipStream_t s);

}  // namespace ula
