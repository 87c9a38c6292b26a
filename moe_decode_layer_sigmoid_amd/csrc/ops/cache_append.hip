// Append to the 8-bit paged cache: quantises the new tokens' K and V into
// their pages, one power-of-two scale per page, kv head and tensor.
//
// A workgroup owns one page, head and tensor of one sequence.  Its scale is
// the larger of what the page has (unless the page starts with a new token)
// and what the new tokens need; powers of two, so rescaling the page's
// earlier codes is a shift of their exponents and rounds only where a code
// becomes subnormal.
//
// 2 D threads, each with the 32 values that make two 16-byte units of the
// page: of K one token's 16 dimensions, twice; of V two dimensions' 16 tokens.
// So a page's new values are read once and held while their largest is found,
// and codes leave in units, in whole lines.  Measured for 8 sequences of 256
// new tokens, 8 heads of 128 (6.4 MB): 5.8 us, most of it the launch and one
// chain of loads; with one byte a thread and a second reading of the tokens
// 16.9 us.  One token a sequence is that chain alone, 4.3 us.
#include "ops_device.h"
#include "ops_launch.h"

namespace moe {
namespace {

// The lowest n bytes of a word, n in [0, 4].
__device__ __forceinline__ uint32_t bytes_below(int n) {
  return n == 4 ? 0xffffffffu : (1u << (8 * n)) - 1u;
}

// The bytes of `now` under the mask, elsewhere the old codes scaled by r.
__device__ __forceinline__ uint32_t keep_old(uint32_t now, uint32_t old, uint32_t mask, float r) {
  float f[4];
  fp8x4_to_f32(old, f);
  if (r != 1.f) old = to_fp8x4(f[0] * r, f[1] * r, f[2] * r, f[3] * r);
  return (now & mask) | (old & ~mask);
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s) {
  return to_fp8x4(inf_to_nan(a) * s, inf_to_nan(b) * s, inf_to_nan(c) * s, inf_to_nan(d) * s);
}

template <int D>
__global__ __launch_bounds__(2 * D) void append_kernel(CacheView c, const uint16_t* k,
                                                       int64_t k_stride, const uint16_t* v,
                                                       int64_t v_stride) {
  constexpr int kThreads = 2 * D, kWaves = kThreads / kWave;
  const int b = blockIdx.z, kv = blockIdx.y & 1, h = blockIdx.y >> 1, tid = threadIdx.x;
  const Seq sq = seq_of(c, b);
  const int past = sq.len - sq.q;
  const int pi = past / kPage + blockIdx.x;
  const int t_lo = max(past - pi * kPage, 0), t_hi = min(sq.len - pi * kPage, kPage);
  if (sq.q == 0 || t_lo >= t_hi) return;  // uniform over the workgroup
  const int page = c.table[static_cast<size_t>(b) * c.max_pages + pi];
  if (page < 0 || page >= c.pages) return;
  const int64_t stride = kv ? v_stride : k_stride;
  // token t of the page is row q0 + (pi * 64 + t - past)
  const uint16_t* src = (kv ? v : k) + (static_cast<int64_t>(sq.q0) + pi * kPage - past) * stride +
                        static_cast<int64_t>(h) * D;
  const size_t blk = page_block(c, page, kv, h);
  uint8_t* dst = c.pool + blk * (static_cast<size_t>(kPage) * D);
  const int old = static_cast<int>(c.scale[blk]) - 127;

  // K: dimensions 16 * (tid % (D / 16)) of tokens kt and kt + 32
  const int kd = tid % (D / 16), kt = tid / (D / 16);
  // V: dimensions vd and vd + 1 of tokens 16 g + vc + j, g and j below 4
  const int vd = tid % (D / 2) * 2, vc = tid / (D / 2) * 4;
  uint32_t x[16];
  uint4 had[2] = {};               // V's units as they are, where tokens are missing
  uint32_t fresh[4], past_end[4];  // V: bytes of new tokens, and behind the last
  bool any = false, all = true;
  if (kv == 0) {
    uint4 w[4] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = kt + 32 * i;
      if (t >= t_lo && t < t_hi) {
        const uint4* p = reinterpret_cast<const uint4*>(src + t * stride + kd * 16);
        w[2 * i] = p[0];
        w[2 * i + 1] = p[1];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = w[i].x;
      x[4 * i + 1] = w[i].y;
      x[4 * i + 2] = w[i].z;
      x[4 * i + 3] = w[i].w;
    }
  } else {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int a = min(max(t_lo - g * 16 - vc, 0), 4), z = min(max(t_hi - g * 16 - vc, 0), 4);
      fresh[g] = bytes_below(z) & ~bytes_below(a);
      past_end[g] = ~bytes_below(z);
      any |= fresh[g] != 0;
      all &= fresh[g] == 0xffffffffu;
    }
    if (any && !all) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        had[j] = *reinterpret_cast<const uint4*>(dst + (vc / 4 * D + vd + j) * 16);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int t = (i >> 2) * 16 + vc + (i & 3);
      x[i] = 0;
      if (t >= t_lo && t < t_hi)
        x[i] = *reinterpret_cast<const uint32_t*>(src + t * stride + vd);
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    amax = fmaxf(amax, fmaxf(finite_abs(bf16_lo(x[i])), finite_abs(bf16_hi(x[i]))));
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, kWave));
  __shared__ float s_max[kWaves];
  if ((tid & 63) == 0) s_max[tid >> 6] = amax;
  __syncthreads();  // also: every thread has read the old scale
#pragma unroll
  for (int i = 0; i < kWaves; ++i) amax = fmaxf(amax, s_max[i]);
  int e = scale_exp(amax);
  if (t_lo > 0) e = max(e, old);
  const float s = pow2f(-e);
  const bool rescale = t_lo > 0 && e > old;
  const float r = rescale ? ldexpf(1.f, old - e) : 1.f;

  if (kv == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = kt + 32 * i;
      uint4* unit = reinterpret_cast<uint4*>(dst + (kd * kPage + t) * 16);
      if (t >= t_lo && t < t_hi) {
        const uint32_t* y = x + 8 * i;
        *unit = make_uint4(
            codes4(bf16_lo(y[0]), bf16_hi(y[0]), bf16_lo(y[1]), bf16_hi(y[1]), s),
            codes4(bf16_lo(y[2]), bf16_hi(y[2]), bf16_lo(y[3]), bf16_hi(y[3]), s),
            codes4(bf16_lo(y[4]), bf16_hi(y[4]), bf16_lo(y[5]), bf16_hi(y[5]), s),
            codes4(bf16_lo(y[6]), bf16_hi(y[6]), bf16_lo(y[7]), bf16_hi(y[7]), s));
      } else if (rescale && t < t_lo) {
        const uint4 o = *unit;
        *unit = make_uint4(keep_old(0, o.x, 0, r), keep_old(0, o.y, 0, r), keep_old(0, o.z, 0, r),
                           keep_old(0, o.w, 0, r));
      }
    }
  } else {
    if (any || rescale) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint4* unit = reinterpret_cast<uint4*>(dst + (vc / 4 * D + vd + j) * 16);
        const uint4 o = any ? had[j] : *unit;
        uint32_t n[4], q[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = j ? bf16_hi(x[4 * g + i]) : bf16_lo(x[4 * g + i]);
          n[g] = codes4(f[0], f[1], f[2], f[3], s);
          const uint32_t kept = keep_old(n[g], q[g], fresh[g], r);
          n[g] = (kept & ~past_end[g]) | (q[g] & past_end[g]);
        }
        *unit = make_uint4(n[0], n[1], n[2], n[3]);
      }
    }
  }
  if (tid == 0) c.scale[blk] = static_cast<uint8_t>(e + 127);
}

template <int D>
void launch(const CacheView& c, const uint16_t* k, int64_t k_stride, const uint16_t* v,
            int64_t v_stride, hipStream_t s) {
  // pages that max_q tokens can touch
  const dim3 grid((c.max_q + kPage - 2) / kPage + 1, 2 * c.Hkv, c.B);
  hipLaunchKernelGGL(append_kernel<D>, grid, dim3(2 * D), 0, s, c, k, k_stride, v, v_stride);
}

}  // namespace

hipError_t launch_append(const CacheView& c, const uint16_t* k, int64_t k_stride,
                         const uint16_t* v, int64_t v_stride, hipStream_t s) {
  switch (c.D) {
    case 64: launch<64>(c, k, k_stride, v, v_stride, s); break;
    case 128: launch<128>(c, k, k_stride, v, v_stride, s); break;
    case 192: launch<192>(c, k, k_stride, v, v_stride, s); break;
    case 256: launch<256>(c, k, k_stride, v, v_stride, s); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace moe
