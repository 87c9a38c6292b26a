// Activation quantiser: bf16 rows -> e4m3 codes with one power-of-two scale
// per row and 128 columns, optionally of the clamped SwiGLU of a gate and an
// up half.
//
// 16 lanes hold one block of 128, eight values each.
#include "ops_device.h"
#include "ops_launch.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <bool SWIGLU>
__device__ __forceinline__ double value64(float g, float u, float limit) {
  if (!SWIGLU) return g;
  if (g != g || u != u) return static_cast<double>(g) + static_cast<double>(u);  // NaN stays NaN
  const double gc = fmin(static_cast<double>(g), static_cast<double>(limit));
  const double uc = fmin(fmax(static_cast<double>(u), -static_cast<double>(limit)),
                         static_cast<double>(limit));
  return gc / (1.0 + exp(-gc)) * uc;
}

__device__ __forceinline__ void unpack8(const uint4& v, float* o) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = bf16_lo(w[i]);
    o[2 * i + 1] = bf16_hi(w[i]);
  }
}

template <bool SWIGLU>
__global__ __launch_bounds__(kThreads) void quant_kernel(const uint16_t* __restrict__ x,
                                                         int64_t x_stride, int64_t blocks, int K,
                                                         float limit, uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales) {
  const int64_t blk = static_cast<int64_t>(blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 4);
  if (blk >= blocks) return;  // uniform over the 16 lanes of a block
  const int KB = K / kBlock;
  const int64_t row = blk / KB;
  const int col = static_cast<int>(blk - row * KB) * kBlock + 8 * (threadIdx.x & 15);
  const uint16_t* p = x + row * x_stride + col;
  float g[8], u[8];
  unpack8(*reinterpret_cast<const uint4*>(p), g);
  if (SWIGLU) unpack8(*reinterpret_cast<const uint4*>(p + K), u);
  // the values in 64 bits for the SwiGLU, so that no border is missed
  double a[8];
  float amax = 0.f;
  double amax64 = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = value64<SWIGLU>(g[i], u[i], limit);
    const double m = fabs(a[i]);
    if (m <= 3.402823466e38) amax64 = fmax(amax64, m);
  }
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) amax64 = fmax(amax64, __shfl_xor(amax64, off, kWave));
  // rounding up keeps amax <= 448 * 2^e true in 64 bits
  amax = __double2float_ru(amax64);
  const int e = scale_exp(amax);
  const double inv = SWIGLU ? ldexp(1.0, -e) : 0.0;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    y[i] = SWIGLU ? inf_to_nan(static_cast<float>(a[i] * inv)) : inf_to_nan(g[i]) * pow2f(-e);
  const uint2 c = make_uint2(to_fp8x4(y[0], y[1], y[2], y[3]), to_fp8x4(y[4], y[5], y[6], y[7]));
  *reinterpret_cast<uint2*>(codes + row * K + col) = c;
  if ((threadIdx.x & 15) == 0) scales[blk] = static_cast<uint8_t>(e + 127);
}

}  // namespace

hipError_t launch_quant(const uint16_t* x, int64_t x_stride, int M, int K, float limit,
                        uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t blocks = static_cast<int64_t>(M) * (K / kBlock);
  const unsigned grid = static_cast<unsigned>((blocks + kThreads / 16 - 1) / (kThreads / 16));
  if (limit > 0.f)
    hipLaunchKernelGGL(quant_kernel<true>, dim3(grid), dim3(kThreads), 0, s, x, x_stride, blocks,
                       K, limit, codes, scales);
  else
    hipLaunchKernelGGL(quant_kernel<false>, dim3(grid), dim3(kThreads), 0, s, x, x_stride,
                       blocks, K, limit, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
