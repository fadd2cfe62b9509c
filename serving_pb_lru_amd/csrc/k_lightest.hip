// The entries of least score in ranges of addresses: what an eviction by accumulated
// attention weight gives up.
//
// Of each range the n addresses with the least (score, address), in ascending order
// of address; entries of negative score are not there. A radix selection finds the
// last of them, T, and how many entries with T's score go with it:
//   - first by the score's magnitude: 64 scores below 64, then five bits behind the
//     leading one, so that scores which span many powers of two spread over the
//     2048 bins (the top bits of a whole number would all be 0);
//   - then, among the entries of the bin that holds T, by 11 bits at a time, until
//     the bin is taken whole or its scores are equal.
// A range of up to kLightSpan addresses is one workgroup's: its scores are read once,
// into LDS. A longer one is split into chunks, in three launches: each chunk's bins;
// each chunk's entries of T's bin, side by side; T from those (every workgroup for
// itself: they are few) and the chunk's part of the result, whose place follows from
// the bins and the lists of the chunks before it. Bound by its launches: the scores
// are read twice or three times, from the caches after the first.
#include <algorithm>

#include "device_util.h"
#include "lightest.h"

namespace ula {

constexpr int kLightThreads = 1024;
constexpr int kLightWaves = kLightThreads / kWave;
constexpr int kAtOnce = 8;                           // entries of a thread in one step
constexpr unsigned long long kNotThere = ~0ull;      // an entry of negative score

__device__ __forceinline__ int bin_of(unsigned long long key) {
  if (key < 64) return (int)key;
  const int e = 63 - __builtin_clzll(key);           // 6..62
  return 64 + (e - 6) * 32 + (int)(key >> (e - 5) & 31);
}
// Bits of a key that its bin leaves open.
__device__ __forceinline__ int open_bits(int bin) { return bin < 64 ? 0 : (bin - 64) / 32 + 1; }
static_assert(64 + (62 - 6) * 32 + 31 < kLightBins, "every score has a bin");

struct LightLds {
  uint32_t hist[kLightBins];
  int counts[kAtOnce * kLightWaves + 1];
  int waves[kLightWaves + 1];
  int bin, before, within;
};

// The bin in which the `need`-th (from 1) of the counted entries lies: bin, the
// entries in bins before it, and its own. need is at most the sum.
__device__ __forceinline__ void find_bin(LightLds& s, int need) {
  __syncthreads();
  constexpr int kPer = kLightBins / kLightThreads;
  int mine = 0, c[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) mine += c[i] = (int)s.hist[threadIdx.x * kPer + i];
  int total;
  int at = block_exclusive_sum<kLightThreads>(mine, s.waves, total);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (at < need && need <= at + c[i]) {
      s.bin = threadIdx.x * kPer + i;
      s.before = at;
      s.within = c[i];
    }
    at += c[i];
  }
  __syncthreads();
}

__device__ __forceinline__ void clear_bins(LightLds& s) {
  __syncthreads();
  for (int i = threadIdx.x; i < kLightBins; i += kLightThreads) s.hist[i] = 0;
  __syncthreads();
}

// Where the taken entries end: all keys below `key`, and the first `ties` with it.
struct LightEnd {
  unsigned long long key;
  int ties;
};

// The end of the `need` least of the `within` keys in magnitude bin `bin`; each(f) calls
// f(key) for this thread's part of them, and maybe for keys of other bins and kNotThere.
template <typename F>
__device__ __forceinline__ LightEnd end_within(LightLds& s, int bin, int within, int need, F each) {
  int open = open_bits(bin);
  // keys of the bin so far: those with key >> open == prefix
  unsigned long long prefix = bin < 64 ? (unsigned long long)bin : (32ull | (unsigned)((bin - 64) & 31));
  while (open > 0 && need < within) {
    const int digit = min(open, 11);
    clear_bins(s);
    each([&](unsigned long long key) {
      if (key != kNotThere && key >> open == prefix)
        atomicAdd(&s.hist[(key >> (open - digit)) & ((1u << digit) - 1)], 1u);
    });
    find_bin(s, need);
    need -= s.before;
    within = s.within;
    open -= digit;
    prefix = prefix << digit | (unsigned)s.bin;
    __syncthreads();
  }
  // the whole bin, or `need` of equal keys
  if (need == within) return {((prefix + 1) << open) - 1, 0x7FFFFFFF};
  return {prefix, need};
}

// Writes the entries of this workgroup's part (keys(i), i < count, in order of address)
// that lie before `end` to out, the first of them at place `at`; `tie` entries with the
// end's key lie before this part. Their scores become -1 if marks is given. A thread
// takes kAtOnce entries a workgroup apart; their waves' counts are summed up together.
template <typename F>
__device__ __forceinline__ void write_out(LightLds& s, const LightEnd& end, int count, int at, int tie, int most, int address,
                                          int32_t* out, long long* marks, F keys) {
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  for (int base = 0; base < count; base += kAtOnce * kLightThreads) {
    unsigned long long key[kAtOnce];
    int rank[kAtOnce];                                 // among the wave's: below the end, and << 16 with its key
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = base + u * kLightThreads + threadIdx.x;
      key[u] = i < count ? keys(i) : kNotThere;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const unsigned long long below = __ballot(key[u] < end.key), same = __ballot(key[u] == end.key);
      rank[u] = rank_below(below) | rank_below(same) << 16;
      if (lane == 0) s.counts[u * kLightWaves + wave] = __popcll(below) | __popcll(same) << 16;
    }
    __syncthreads();
    if (wave == 0) {                                   // at most 8192 of either: no carry into the high half
      constexpr int kEach = kAtOnce * kLightWaves / kWave;
      int c[kEach], sum = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) sum += c[i] = s.counts[lane * kEach + i];
      int before = wave_inclusive_sum(sum) - sum;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        s.counts[lane * kEach + i] = before;
        before += c[i];
      }
      if (lane == kWave - 1) s.counts[kAtOnce * kLightWaves] = before;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int mine = s.counts[u * kLightWaves + wave] + rank[u];
      const int nth_same = tie + (mine >> 16);
      const int place = at + (mine & 0xFFFF) + min(nth_same, end.ties) - min(tie, end.ties);
      const int i = base + u * kLightThreads + threadIdx.x;
      if ((key[u] < end.key || (key[u] == end.key && nth_same < end.ties)) && place < most) {
        out[place] = address + i;
        if (marks) marks[i] = -1;
      }
    }
    const int all = s.counts[kAtOnce * kLightWaves];
    at += (all & 0xFFFF) + min(tie + (all >> 16), end.ties) - min(tie, end.ties);
    tie += all >> 16;
    __syncthreads();
  }
}

__global__ __launch_bounds__(kLightThreads) void k_lightest(LightDev a, LightRanges r) {
  __shared__ unsigned long long s_key[kLightSpan];
  __shared__ LightLds s;
  const LightRange at = r.range[blockIdx.x];
  if (at.length > kLightSpan) return;                  // k_light_bins and the others
  long long* scores = a.scores + at.first;
  int32_t* out = a.out + (long long)(r.first_range + blockIdx.x) * a.most;
  for (int i = threadIdx.x; i < kLightBins; i += kLightThreads) s.hist[i] = 0;
  __syncthreads();
  int mine = 0;
  for (int i = threadIdx.x; i < at.length; i += kLightThreads) {
    const long long v = scores[i];
    s_key[i] = v < 0 ? kNotThere : (unsigned long long)v;
    if (v >= 0) {
      atomicAdd(&s.hist[bin_of(v)], 1u);
      ++mine;
    }
  }
  int there;
  block_exclusive_sum<kLightThreads>(mine, s.waves, there);
  const int need = min(at.count, there);
  LightEnd end{0, 0};
  if (need > 0) {
    find_bin(s, need);
    const int bin = s.bin, before = s.before, within = s.within;
    end = end_within(s, bin, within, need - before, [&](auto f) {
      for (int i = threadIdx.x; i < at.length; i += kLightThreads) f(s_key[i]);
    });
  }
  __syncthreads();
  if (need > 0)
    write_out(s, end, at.length, 0, 0, a.most, at.first, out, a.mark ? scores : nullptr, [&](int i) { return s_key[i]; });
  for (int i = need + threadIdx.x; i < a.most; i += kLightThreads) out[i] = -1;
}

// The chunk of a long range that a workgroup has.
struct LightChunk {
  LightRange at;
  int range, chunk, chunks, first, count;              // first: of the range's addresses
  uint32_t* bins;                                      // of the range's first chunk
  LightChunkEnd* ends;                                 // the same
  unsigned long long* list;                            // of the range
};
__device__ __forceinline__ LightChunk light_chunk(const LightDev& a, const LightRanges& r) {
  LightChunk c;
  int i = 0, block = blockIdx.x;
  long long lists = 0;
  for (; i < r.n - 1; ++i) {                           // few ranges are long
    const int n = light_chunks(r.range[i].length);
    if (block < n) break;
    block -= n;
    if (n) lists += r.range[i].length;
  }
  c.at = r.range[i];
  c.range = r.first_range + i;
  c.chunk = block;
  c.chunks = light_chunks(c.at.length);
  const int per = light_chunk_size(c.at.length);
  c.first = block * per;
  c.count = max(0, min(per, c.at.length - c.first));
  c.bins = a.bins + (size_t)(blockIdx.x - block) * kLightBins;
  c.ends = a.ends + (blockIdx.x - block);
  c.list = a.list + lists;
  return c;
}

__global__ __launch_bounds__(kLightThreads) void k_light_bins(LightDev a, LightRanges r) {
  __shared__ uint32_t hist[kLightBins];
  const LightChunk c = light_chunk(a, r);
  for (int i = threadIdx.x; i < kLightBins; i += kLightThreads) hist[i] = 0;
  __syncthreads();
  const long long* scores = a.scores + c.at.first + c.first;
#pragma unroll 4
  for (int i = threadIdx.x; i < c.count; i += kLightThreads) {
    const long long v = scores[i];
    if (v >= 0) atomicAdd(&hist[bin_of(v)], 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kLightBins; i += kLightThreads) c.bins[(size_t)c.chunk * kLightBins + i] = hist[i];
}

// Where the range's end lies, from the bins of its chunks added up, and what the chunk
// has before and in that bin; its entries of that bin to the list, from the place of
// the chunk's first address on, in any order: only how many they are is looked at.
__global__ __launch_bounds__(kLightThreads) void k_light_list(LightDev a, LightRanges r) {
  __shared__ LightLds s;
  __shared__ int s_listed;
  const LightChunk c = light_chunk(a, r);
  const long long* scores = a.scores + c.at.first + c.first;
  long long ahead[kAtOnce];                            // on their way meanwhile
#pragma unroll
  for (int u = 0; u < kAtOnce; ++u) {
    const int i = u * kLightThreads + threadIdx.x;
    ahead[u] = i < c.count ? scores[i] : -1;
  }
  constexpr int kPer = kLightBins / kLightThreads;
  static_assert(kPer == 2, "two bins of a thread in one load");
  const uint2* bins = reinterpret_cast<const uint2*>(c.bins) + threadIdx.x;
  const uint2 own = bins[(size_t)c.chunk * kLightThreads];
  uint2 sum = make_uint2(0, 0);
#pragma unroll 8
  for (int k = 0; k < c.chunks; ++k) {
    const uint2 v = bins[(size_t)k * kLightThreads];
    sum.x += v.x;
    sum.y += v.y;
  }
  if (threadIdx.x == 0) s_listed = 0;
  s.hist[2 * threadIdx.x] = sum.x;
  s.hist[2 * threadIdx.x + 1] = sum.y;
  int there;
  block_exclusive_sum<kLightThreads>((int)(sum.x + sum.y), s.waves, there);
  const int need = min(c.at.count, there);
  if (need > 0) find_bin(s, need);
  const int bin = need > 0 ? s.bin : 0;
  int below = 0;
  if (need > 0) {
    const int b = 2 * threadIdx.x;
    block_exclusive_sum<kLightThreads>((b < bin ? (int)own.x : 0) + (b + 1 < bin ? (int)own.y : 0), s.waves, below);
  }
  if (threadIdx.x == bin / 2)
    c.ends[c.chunk] = {bin, need, s.before, s.within, below, need > 0 ? (int)(bin % 2 ? own.y : own.x) : 0, 0, 0};
  if (need == 0) return;
  auto list = [&](long long v) {
    if (v >= 0 && bin_of(v) == bin) c.list[c.first + atomicAdd(&s_listed, 1)] = (unsigned long long)v;
  };
#pragma unroll
  for (int u = 0; u < kAtOnce; ++u) list(ahead[u]);
  for (int i = kAtOnce * kLightThreads + threadIdx.x; i < c.count; i += kLightThreads) list(scores[i]);
}

// The list's entries are read into LDS where that holds them, and looked at there.
__global__ __launch_bounds__(kLightThreads) void k_light_out(LightDev a, LightRanges r) {
  __shared__ LightLds s;
  __shared__ unsigned long long s_key[kLightSpan];
  // of each chunk: entries in the list and before it in those of the chunks before, in bins before its bin
  __shared__ int s_count[kLightChunks], s_from[kLightChunks], s_below[kLightChunks];
  const LightChunk c = light_chunk(a, r);
  int32_t* out = a.out + (long long)c.range * a.most;
  const LightChunkEnd in = c.ends[c.chunk];
  if (threadIdx.x < kWave) {
    static_assert(kLightChunks == kWave, "a lane for each chunk");
    const bool any = (int)threadIdx.x < c.chunks;
    const int listed = any ? c.ends[threadIdx.x].listed : 0;
    s_count[threadIdx.x] = listed;
    s_below[threadIdx.x] = any ? c.ends[threadIdx.x].below : 0;
    s_from[threadIdx.x] = wave_inclusive_sum(listed) - listed;
  }
  if (c.chunk == 0)
    for (int i = in.need + threadIdx.x; i < a.most; i += kLightThreads) out[i] = -1;
  if (in.need == 0) return;
  __syncthreads();
  const int per = light_chunk_size(c.at.length);
  const bool held = in.within <= kLightSpan;           // the list, in LDS
  // each(f, n) calls f(key) for this thread's part of the first n chunks' lists
  auto listed = [&](int n, auto f) {
    if (held) {
      const int all = n < c.chunks ? s_from[n] : in.within;
      for (int i = threadIdx.x; i < all; i += kLightThreads) f(s_key[i]);
    } else {
      for (int k = threadIdx.x / kWave; k < n; k += kLightWaves)
        for (int i = lane_id(); i < s_count[k]; i += kWave) f(c.list[(size_t)k * per + i]);
    }
  };
  if (held) {
    for (int k = threadIdx.x / kWave; k < c.chunks; k += kLightWaves)
      for (int i = lane_id(); i < s_count[k]; i += kWave) s_key[s_from[k] + i] = c.list[(size_t)k * per + i];
    __syncthreads();
  }
  const LightEnd end = end_within(s, in.bin, in.within, in.need - in.before, [&](auto f) { listed(c.chunks, f); });
  __syncthreads();
  // entries taken in the chunks before this one: whole bins, and the listed ones before the end
  int below = 0, same = 0;
  listed(c.chunk, [&](unsigned long long key) {
    below += key < end.key;
    same += key == end.key;
  });
  if (threadIdx.x < (unsigned)c.chunk) below += s_below[threadIdx.x];
  int at, tie;
  block_exclusive_sum<kLightThreads>(below, s.waves, at);
  block_exclusive_sum<kLightThreads>(same, s.waves, tie);
  at += min(tie, end.ties);
  long long* scores = a.scores + c.at.first + c.first;
  write_out(s, end, c.count, at, tie, a.most, c.at.first + c.first, out, a.mark ? scores : nullptr, [&](int i) {
    const long long v = scores[i];
    return v < 0 ? kNotThere : (unsigned long long)v;
  });
}

hipError_t launch_lightest(const LightDev& a, const LightRanges& r, hipStream_t s) {
  int blocks = 0, small = 0;
  for (int i = 0; i < r.n; ++i) {
    const int chunks = light_chunks(r.range[i].length);
    blocks += chunks;
    small += chunks == 0;
  }
  if (small) k_lightest<<<r.n, kLightThreads, 0, s>>>(a, r);
  if (blocks) {
    k_light_bins<<<blocks, kLightThreads, 0, s>>>(a, r);
    k_light_list<<<blocks, kLightThreads, 0, s>>>(a, r);
    k_light_out<<<blocks, kLightThreads, 0, s>>>(a, r);
  }
  return hipGetLastError();
}

}  // namespace ula
