// Eviction of whole pages by accumulated attention weight.
//
// One workgroup per sequence.  The pages between the first `sink` and the last
// `recent` compete by a key that orders as their mass does; a radix select
// (four rounds of a 256-bin count, most significant byte first) finds the key
// T of the last page that stays and how many pages of key T do; then one pass
// in page order moves kept and dropped pages to the front of their outputs.
#include "ops_device.h"
#include "ops_launch.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// Order-preserving bits of a float (-0 as 0); NaN above everything.
__device__ __forceinline__ uint32_t key_of(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// Sum over the threads before this one, and over all (in *total); every
// thread calls it, *s has kWaves ints.
__device__ __forceinline__ int scan(int v, int* s, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int y = __shfl_up(x, off, kWave);
    if (lane >= off) x += y;
  }
  __syncthreads();  // the last scan's readers are done
  if (lane == 63) s[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? s[w] : 0;
    all += s[w];
  }
  *total = all;
  return before + x - v;
}

__global__ __launch_bounds__(kThreads) void evict_kernel(EvictArgs a) {
  __shared__ int s_scan[kWaves];
  __shared__ int s_bins[256];
  __shared__ int s_pick[2];
  const int b = blockIdx.x, tid = threadIdx.x;
  const size_t row = static_cast<size_t>(b) * a.max_pages;
  const int len = a.lens[b];
  const bool fits = len >= 0 && len <= a.max_pages * kPage;
  const int n = fits ? (len + kPage - 1) / kPage : a.max_pages;
  const int drop = fits ? max(n - a.keep, 0) : 0;
  // pages [lo, hi) compete; stay of them do
  const int lo = min(a.sink, n), hi = max(n - a.recent, lo);
  const int stay = hi - lo - drop;
  uint32_t T = 0;
  int ties = 0;  // pages of key T that stay, lowest first
  if (drop > 0) {
    uint32_t mask = 0;
    int want = stay;  // rank (from the largest) of the last page that stays
    if (want == 0) {
      T = 0xffffffffu;  // nothing stays: keys above T none, none of key T
    } else {
      for (int shift = 24; shift >= 0; shift -= 8) {
        s_bins[tid] = 0;
        __syncthreads();
        for (int i = lo + tid; i < hi; i += kThreads) {
          const uint32_t k = key_of(a.mass[row + i]);
          if ((k & mask) == T) atomicAdd(&s_bins[k >> shift & 255], 1);
        }
        __syncthreads();
        // thread tid has bin 255 - tid: bins from the largest down
        int all;
        const int mine = s_bins[255 - tid];
        const int before = scan(mine, s_scan, &all);
        if (before < want && want <= before + mine) {
          s_pick[0] = 255 - tid;
          s_pick[1] = want - before;
        }
        __syncthreads();
        T |= static_cast<uint32_t>(s_pick[0]) << shift;
        want = s_pick[1];
        mask |= 0xffu << shift;
      }
      ties = want;
    }
  }
  int kept = 0, gone = 0, seen = 0;  // so far; seen: pages of key T
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    const bool in = i < n, rival = in && drop > 0 && i >= lo && i < hi;
    const float mass = in ? a.mass[row + i] : 0.f;
    const int id = in ? a.table[row + i] : -1;
    const uint32_t k = key_of(mass);
    int total;
    const bool tie = rival && k == T;
    const int tie_rank = seen + scan(tie, s_scan, &total);
    seen += total;
    const bool keep = in && (!rival || (tie ? tie_rank < ties : k > T));
    const int at = kept + scan(keep, s_scan, &total);
    kept += total;
    const int nin = min(kThreads, n - i0);
    // every read of this round is done (scan's barriers), so the outputs may
    // be the inputs: a page never moves back
    if (keep) {
      a.out_table[row + at] = id;
      a.out_mass[row + at] = mass;
    } else if (in) {
      a.freed[row + gone + (i - i0) - (at - (kept - total))] = id;
    }
    gone += nin - total;
  }
  __syncthreads();
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
