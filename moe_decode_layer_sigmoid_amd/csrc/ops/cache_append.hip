// Append to the 8-bit paged cache: quantises the new tokens' K and V into
// their pages, one power-of-two scale per page, kv head and tensor.
//
// A workgroup owns one page, head and tensor of one sequence.  Its scale is
// the larger of what the page has (unless the page starts with a new token)
// and what the new tokens need; powers of two, so rescaling the page's
// earlier codes is a shift of their exponents and rounds only where a code
// becomes subnormal.
#include "ops_device.h"
#include "ops_launch.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Byte of token t, dimension d inside a page's K or V block.
__device__ __forceinline__ int byte_of(int kv, int D, int t, int d) {
  return kv == 0 ? ((d >> 4) * kPage + t) * 16 + (d & 15)
                 : (((t & 15) >> 2) * D + d) * 16 + (t >> 4) * 4 + (t & 3);
}

__global__ __launch_bounds__(kThreads) void append_kernel(CacheView c, const uint16_t* k,
                                                          int64_t k_stride, const uint16_t* v,
                                                          int64_t v_stride) {
  const int b = blockIdx.z, kv = blockIdx.y & 1, h = blockIdx.y >> 1;
  const Seq sq = seq_of(c, b);
  const int past = sq.len - sq.q;
  const int pi = past / kPage + blockIdx.x;
  const int t_lo = max(past - pi * kPage, 0), t_hi = min(sq.len - pi * kPage, kPage);
  if (sq.q == 0 || t_lo >= t_hi) return;  // uniform over the workgroup
  const int page = c.table[static_cast<size_t>(b) * c.max_pages + pi];
  if (page < 0 || page >= c.pages) return;
  const int D = c.D;
  const int64_t stride = kv ? v_stride : k_stride;
  // token t of the page is row q0 + (pi * 64 + t - past)
  const uint16_t* src = (kv ? v : k) + (static_cast<int64_t>(sq.q0) + pi * kPage - past) * stride +
                        static_cast<int64_t>(h) * D;
  const size_t blk = page_block(c, page, kv, h);
  uint8_t* dst = c.pool + blk * (static_cast<size_t>(kPage) * D);
  const int n = (t_hi - t_lo) * D;
  float amax = 0.f;
  for (int i = threadIdx.x; i < n; i += kThreads)
    amax = fmaxf(amax, finite_abs(bf16_to_f32(src[(t_lo + i / D) * stride + i % D])));
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, kWave));
  __shared__ float s_max[kThreads / kWave];
  if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = amax;
  const int old = static_cast<int>(c.scale[blk]) - 127;
  __syncthreads();  // also: every thread has read the old scale
  amax = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  int e = scale_exp(amax);
  if (t_lo > 0) e = max(e, old);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int t = t_lo + i / D, d = i % D;
    const float x = inf_to_nan(bf16_to_f32(src[t * stride + d])) * pow2f(-e);
    dst[byte_of(kv, D, t, d)] = static_cast<uint8_t>(to_fp8x4(x, x, x, x));
  }
  if (t_lo > 0 && e > old) {
    const float r = ldexpf(1.f, old - e);
    for (int i = threadIdx.x; i < t_lo * D; i += kThreads) {
      uint8_t* p = dst + byte_of(kv, D, i / D, i % D);
      float f[4];
      fp8x4_to_f32(*p, f);
      const float x = f[0] * r;
      *p = static_cast<uint8_t>(to_fp8x4(x, x, x, x));
    }
  }
  if (threadIdx.x == 0) c.scale[blk] = static_cast<uint8_t>(e + 127);
}

}  // namespace

hipError_t launch_append(const CacheView& c, const uint16_t* k, int64_t k_stride,
                         const uint16_t* v, int64_t v_stride, hipStream_t s) {
  // pages that max_q tokens can touch
  const dim3 grid((c.max_q + kPage - 2) / kPage + 1, 2 * c.Hkv, c.B);
  hipLaunchKernelGGL(append_kernel, grid, dim3(kThreads), 0, s, c, k, k_stride, v, v_stride);
  return hipGetLastError();
}

}  // namespace moe
