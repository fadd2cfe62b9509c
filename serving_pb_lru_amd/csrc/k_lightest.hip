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
// end's key lie before this part. Their scores become -1 if marks is given.
template <typename F>
__device__ __forceinline__ int write_out(LightLds& s, const LightEnd& end, int count, int at, int tie, int most, int address,
                                         int32_t* out, long long* marks, F keys) {
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  for (int base = 0; base < count; base += kLightThreads) {
    const int i = base + threadIdx.x;
    const unsigned long long key = i < count ? keys(i) : kNotThere;
    const bool equal = key == end.key;
    // both ranks in one sum: taken below the end in the low half, equal ones in the high half
    const unsigned long long below = __ballot(key < end.key), same = __ballot(equal);
    if (lane == 0) s.waves[wave] = __popcll(below) | __popcll(same) << 16;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kLightWaves; ++w) {
      if (w == wave) before = all;
      all += s.waves[w];
    }
    const int rank_same = tie + (before >> 16) + rank_below(same);
    const int taken_same = min(rank_same, end.ties) - min(tie, end.ties);   // equal ones taken before this entry
    const int place = at + (before & 0xFFFF) + rank_below(below) + taken_same;
    if ((key < end.key || (equal && rank_same < end.ties)) && place < most) {
      out[place] = address + i;
      if (marks) marks[i] = -1;
    }
    at += (all & 0xFFFF) + min(tie + (all >> 16), end.ties) - min(tie, end.ties);
    tie += all >> 16;
    __syncthreads();
  }
  return at;
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
  c.list = a.list + lists;
  return c;
}

__global__ __launch_bounds__(kLightThreads) void k_light_bins(LightDev a, LightRanges r) {
  __shared__ uint32_t hist[kLightBins];
  const LightChunk c = light_chunk(a, r);
  for (int i = threadIdx.x; i < kLightBins; i += kLightThreads) hist[i] = 0;
  __syncthreads();
  const long long* scores = a.scores + c.at.first + c.first;
  for (int i = threadIdx.x; i < c.count; i += kLightThreads) {
    const long long v = scores[i];
    if (v >= 0) atomicAdd(&hist[bin_of(v)], 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kLightBins; i += kLightThreads) c.bins[(size_t)c.chunk * kLightBins + i] = hist[i];
}

// The bin of the last entry taken, of a whole range: the bins of its chunks added up.
// Returns how many are taken (0: none, and no bin).
__device__ __forceinline__ int range_bin(LightLds& s, const LightChunk& c) {
  constexpr int kPer = kLightBins / kLightThreads;
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = threadIdx.x * kPer + i;
    uint32_t sum = 0;
    for (int k = 0; k < c.chunks; ++k) sum += c.bins[(size_t)k * kLightBins + b];
    s.hist[b] = sum;
    mine += (int)sum;
  }
  int there;
  block_exclusive_sum<kLightThreads>(mine, s.waves, there);
  const int need = min(c.at.count, there);
  if (need > 0) find_bin(s, need);
  return need;
}

// The chunk's entries of that bin to the list, from the place of the chunk's first address on.
__global__ __launch_bounds__(kLightThreads) void k_light_list(LightDev a, LightRanges r) {
  __shared__ LightLds s;
  const LightChunk c = light_chunk(a, r);
  if (range_bin(s, c) == 0) return;
  const int bin = s.bin;
  const long long* scores = a.scores + c.at.first + c.first;
  int at = 0;
  for (int base = 0; base < c.count; base += kLightThreads) {
    const int i = base + threadIdx.x;
    const long long v = i < c.count ? scores[i] : -1;
    const bool in = v >= 0 && bin_of(v) == bin;
    int total;
    const int place = block_exclusive_sum<kLightThreads>(in, s.waves, total);
    if (in) c.list[c.first + at + place] = (unsigned long long)v;
    at += total;
  }
}

__global__ __launch_bounds__(kLightThreads) void k_light_out(LightDev a, LightRanges r) {
  __shared__ LightLds s;
  __shared__ int s_count[kLightChunks], s_below[kLightChunks];   // of each chunk: entries in the list, in bins before its bin
  const LightChunk c = light_chunk(a, r);
  int32_t* out = a.out + (long long)c.range * a.most;
  const int need = range_bin(s, c);
  if (c.chunk == 0)
    for (int i = need + threadIdx.x; i < a.most; i += kLightThreads) out[i] = -1;
  if (need == 0) return;
  const int bin = s.bin, before = s.before, within = s.within;
  // a wave for each chunk's bins before the end's
  for (int k = threadIdx.x / kWave; k < c.chunks; k += kLightWaves) {
    const uint32_t* bins = c.bins + (size_t)k * kLightBins;
    int below = 0;
    if (k < c.chunk)
      for (int b = lane_id(); b < bin; b += kWave) below += (int)bins[b];
    below = wave_sum(below);
    if (lane_id() == 0) {
      s_below[k] = below;
      s_count[k] = (int)bins[bin];
    }
  }
  const int per = light_chunk_size(c.at.length);
  const LightEnd end = end_within(s, bin, within, need - before, [&](auto f) {
    for (int k = threadIdx.x / kWave; k < c.chunks; k += kLightWaves)
      for (int i = lane_id(); i < s_count[k]; i += kWave) f(c.list[(size_t)k * per + i]);
  });
  __syncthreads();
  // entries taken in the chunks before this one: whole bins, and the listed ones before the end
  int below = 0, same = 0;
  for (int k = threadIdx.x / kWave; k < c.chunk; k += kLightWaves)
    for (int i = lane_id(); i < s_count[k]; i += kWave) {
      const unsigned long long key = c.list[(size_t)k * per + i];
      below += key < end.key;
      same += key == end.key;
    }
  int at, tie;
  block_exclusive_sum<kLightThreads>(below, s.waves, at);
  block_exclusive_sum<kLightThreads>(same, s.waves, tie);
  for (int k = 0; k < c.chunk; ++k) at += s_below[k];
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
