// Eviction of whole pages by accumulated attention weight.
//
// One workgroup per sequence.  The pages between the first `sink` and the last
// `recent` compete by a key that orders as their mass does.  A radix select
// from the highest bit in which the keys differ finds a key T and a number of
// ties: the pages above T stay, and the first `ties` of key T.  Its rounds of a
// 256-bin count end as soon as whole bins stay.  Then one pass in page order
// moves kept and dropped pages to the front of their outputs.
//
// Bound by its own chain of waits: one load, one barrier a round (each wave
// finds the bin by itself, each round has bins of its own) and one for every
// 1024 pages that move.  64 sequences of 1024 pages: 5.9 us; with rounds from
// the top bit down, two scans a round and keys read again 9.8 us.
#include "ops_device.h"
#include "ops_launch.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kPer = 4;  // pages of a thread, one behind the other
constexpr int kChunk = kThreads * kPer;

// Order-preserving bits of a float (-0 as 0); NaN above everything.
__device__ __forceinline__ uint32_t key_of(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// Sum over the lanes up to this one.
__device__ __forceinline__ int wave_scan(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int y = __shfl_up(v, off, kWave);
    if (lane >= off) v += y;
  }
  return v;
}

__global__ __launch_bounds__(kThreads) void evict_kernel(EvictArgs a) {
  __shared__ __align__(16) int s_bins[4][256];
  __shared__ uint32_t s_min[kWaves], s_max[kWaves];
  __shared__ int s_scan[2][kWaves];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const size_t row = static_cast<size_t>(b) * a.max_pages;
  const float* mass = a.mass + row;
  const int* table = a.table + row;
  // the first chunk's pages, whatever the length turns out to be
  float m0[kPer];
  int id0[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = kPer * tid + j;
    m0[j] = i < a.max_pages ? mass[i] : 0.f;
    id0[j] = i < a.max_pages ? table[i] : -1;
  }
  const int len = a.lens[b];
  const bool fits = len >= 0 && len <= a.max_pages * kPage;
  const int n = fits ? (len + kPage - 1) / kPage : a.max_pages;
  const int drop = fits ? max(n - a.keep, 0) : 0;
  // pages [lo, hi) compete; hi - lo - drop of them stay
  const int lo = min(a.sink, n), hi = max(n - a.recent, lo);
  uint32_t T = 0xffffffffu;  // nothing stays: no key is above, no tie wanted
  int ties = 0;              // pages of key T that stay, lowest first
  int want = hi - lo - drop;
  if (drop > 0 && want > 0) {
#pragma unroll
    for (int r = 0; r < 4; ++r) s_bins[r][tid] = 0;
    // f(key) of every competing page of this thread
    const auto each = [&](auto f) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = kPer * tid + j;
        if (i >= lo && i < hi) f(key_of(m0[j]));
      }
      for (int i = max(lo, kChunk) + tid; i < hi; i += kThreads) f(key_of(mass[i]));
    };
    uint32_t least = 0xffffffffu, most = 0;
    each([&](uint32_t k) {
      least = min(least, k);
      most = max(most, k);
    });
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      least = min(least, static_cast<uint32_t>(__shfl_xor(static_cast<int>(least), off, kWave)));
      most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), off, kWave)));
    }
    if (lane == 0) {
      s_min[wave] = least;
      s_max[wave] = most;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      least = min(least, s_min[w]);
      most = max(most, s_max[w]);
    }
    // bits above `left` are known: the same in all keys that are still in
    int left = least == most ? 0 : 32 - __clz(static_cast<int>(least ^ most));
    T = left == 32 ? 0 : most >> left << left;
    ties = want;
    for (int r = 0; left > 0; ++r) {
      const int shift = max(left - 8, 0);
      const uint32_t digits = (1u << (left - shift)) - 1u;
      each([&](uint32_t k) {
        if (left == 32 || (k ^ T) >> left == 0) atomicAdd(&s_bins[r][k >> shift & digits], 1);
      });
      __syncthreads();
      // lane l has bins 255 - 4 l and the three below, the largest first
      const int4 q = *reinterpret_cast<const int4*>(&s_bins[r][252 - 4 * lane]);
      const int upto = wave_scan(q.x + q.y + q.z + q.w);
      const int w1 = upto - q.x, w2 = w1 - q.y, w3 = w2 - q.z, w4 = w3 - q.w;
      const bool here = w4 < want && want <= upto;
      const int bin = want <= w3 ? 3 : want <= w2 ? 2 : want <= w1 ? 1 : 0;
      const int above = bin == 3 ? w4 : bin == 2 ? w3 : bin == 1 ? w2 : w1;
      const int in_bin = bin == 3 ? q.w : bin == 2 ? q.z : bin == 1 ? q.y : q.x;
      const int from = __ffsll(static_cast<unsigned long long>(__ballot(here))) - 1;
      T |= static_cast<uint32_t>(__shfl(252 - 4 * lane + bin, from, kWave)) << shift;
      want -= __shfl(above, from, kWave);
      ties = want;
      left = shift;
      if (want == __shfl(in_bin, from, kWave)) {
        // the bin stays as a whole: T its lowest key, with all of its ties
        ties = INT32_MAX;
        break;
      }
    }
  }
  int kept = 0, gone = 0, seen = 0;  // so far; seen: pages of key T
  for (int i0 = 0, turn = 0; i0 < n; i0 += kChunk, turn ^= 1) {
    float m[kPer];
    int id[kPer];
    bool in[kPer], rival[kPer], tie[kPer];
    int mine = 0;  // pages that stay without a tie, and ties * 2^16
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = i0 + kPer * tid + j;
      in[j] = i < n;
      m[j] = i0 == 0 ? m0[j] : in[j] ? mass[i] : 0.f;
      id[j] = i0 == 0 ? id0[j] : in[j] ? table[i] : -1;
      rival[j] = in[j] && drop > 0 && i >= lo && i < hi;
      const uint32_t k = key_of(m[j]);
      tie[j] = rival[j] && k == T;
      rival[j] = rival[j] && k <= T;
      mine += tie[j] ? 0x10000 : in[j] && !rival[j] ? 1 : 0;
    }
    const int upto = wave_scan(mine);
    if (lane == 63) s_scan[turn][wave] = upto;
    // every read of this chunk is done behind this, so the outputs may be the
    // inputs: a page never moves back
    __syncthreads();
    int before = upto - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int x = s_scan[turn][w];
      before += w < wave ? x : 0;
      all += x;
    }
    int tied = seen + (before >> 16);
    int at = kept + (before & 0xffff) + max(min(tied, ties) - min(seen, ties), 0);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = i0 + kPer * tid + j;
      const bool keep = in[j] && (!rival[j] || (tie[j] && tied < ties));
      tied += tie[j];
      if (keep) {
        a.out_table[row + at] = id[j];
        a.out_mass[row + at] = m[j];
      } else if (in[j]) {
        a.freed[row + i - at] = id[j];
      }
      at += keep;
    }
    const int now = (all & 0xffff) + min(seen + (all >> 16), ties) - min(seen, ties);
    seen += all >> 16;
    kept += now;
    gone += min(kChunk, n - i0) - now;
  }
  for (int i = kept + tid; i < a.max_pages; i += kThreads) {
    a.out_table[row + i] = -1;
    a.out_mass[row + i] = 0.f;
  }
  for (int i = gone + tid; i < a.max_pages; i += kThreads) a.freed[row + i] = -1;
  if (tid == 0) {
    a.out_lens[b] = len - kPage * gone;
    a.n_freed[b] = gone;
  }
}

}  // namespace

hipError_t launch_evict(const EvictArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(evict_kernel, dim3(a.B), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
