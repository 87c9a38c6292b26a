// Activation quantiser: bf16 rows -> e4m3 codes with one power-of-two scale
// per row and 128 columns, optionally of the clamped SwiGLU of a gate and an
// up half.
//
// 16 lanes hold one block of 128, eight values each.  Plain values are exact
// in fp32 all the way: x * 2^-e, then one rounding to a code.
//
// SwiGLU values are computed in fp32, off by less than 2^-20 of themselves
// (below), and the codes and the scale are those of 64 bits: where a value
// moved by 2^-20 either way has another code, or the block's largest another
// exponent, the block is computed again in 64 bits: about one block in 300.
// Measured at 4096 x 2048 (42 MB): 12.2 us, 3.4 TB/s; everywhere in 64 bits
// 20.0 us.  Bound by the vector unit (270 instructions a wave, 4 waves a row of
// 2048) about as much as by the bytes (8.6 us at a copy's rate); two blocks a
// thread, loaded together, 13.5 us, four 14.4.  Plain values, 4096 x 4096: 10.6
// us, 4.8 TB/s, a copy's rate.
#include "ops_device.h"
#include "ops_launch.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr float kUp = 1.f + 0x1p-20f, kDown = 1.f - 0x1p-20f;

// The clamped SwiGLU in 64 bits (NaN stays NaN).
__device__ __forceinline__ double swiglu64(float g, float u, float limit) {
  if (g != g || u != u) return static_cast<double>(g) + static_cast<double>(u);
  const double gc = fmin(static_cast<double>(g), static_cast<double>(limit));
  const double uc = fmin(fmax(static_cast<double>(u), -static_cast<double>(limit)),
                         static_cast<double>(limit));
  return gc / (1.0 + exp(-gc)) * uc;
}

// In fp32, for u and g that are no NaN, g >= -87.  e^-g = 2^(-g kH) (1 + g kC):
// kH is log2(e) in 16 bits, so that its product with a bf16 g is exact, and g kC
// what is left of the exponent, below 2^-11, with a square below 2^-22.  (A g
// cut to a limit of more bits is positive: e^-g counts for less than 1 there.)
// v_exp_f32 and v_rcp_f32 are off by 2^-23, the four other roundings by 2^-24,
// the square's half by 2^-23: 10 * 2^-24 in all.
__device__ __forceinline__ float swiglu32(float g, float u, float limit) {
  constexpr float kH = 47274.f / 32768.f, kC = -4.888495152e-06f;
  const float gc = fminf(g, limit), uc = __builtin_amdgcn_fmed3f(u, -limit, limit);
  const float e = __builtin_amdgcn_exp2f(gc * -kH);
  return gc * __builtin_amdgcn_rcpf(fmaf(e, fmaf(gc, kC, 1.f), 1.f)) * uc;
}

// v in fp32 rounded to odd (cut, the last bit set if anything was cut off), so
// that the rounding to a code that follows is that of v itself.
__device__ __forceinline__ float to_odd(double v) {
  const float f = __double2float_rz(v);
  return static_cast<double>(f) == v || v != v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

__device__ __forceinline__ void unpack8(const uint4& v, float* o) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = bf16_lo(w[i]);
    o[2 * i + 1] = bf16_hi(w[i]);
  }
}

// Largest of v over the 16 lanes of a block.
template <class V>
__device__ __forceinline__ V block_max(V v) {
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v = fmax(v, __shfl_xor(v, off, kWave));
  return v;
}

__device__ __forceinline__ uint2 codes8(const float* y, float s) {
  return make_uint2(to_fp8x4(y[0] * s, y[1] * s, y[2] * s, y[3] * s),
                    to_fp8x4(y[4] * s, y[5] * s, y[6] * s, y[7] * s));
}

template <bool SWIGLU>
__global__ __launch_bounds__(kThreads) void quant_kernel(const uint16_t* __restrict__ x,
                                                         int64_t x_stride, uint32_t blocks, int K,
                                                         float limit, uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales) {
  const uint32_t blk = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
  if (blk >= blocks) return;  // uniform over the 16 lanes of a block
  const uint32_t KB = static_cast<uint32_t>(K) / kBlock, row = blk / KB;
  const int col = static_cast<int>(blk - row * KB) * kBlock + 8 * (threadIdx.x & 15);
  const uint16_t* p = x + static_cast<int64_t>(row) * x_stride + col;
  float g[8], u[8], a[8];
  unpack8(*reinterpret_cast<const uint4*>(p), g);
  if (SWIGLU) unpack8(*reinterpret_cast<const uint4*>(p + K), u);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = SWIGLU ? swiglu32(g[i], u[i], limit) : inf_to_nan(g[i]);
    amax = fmaxf(amax, SWIGLU ? fabsf(a[i]) : finite_abs(g[i]));
  }
  amax = block_max(amax);
  int e = scale_exp(amax);
  uint2 c = codes8(a, SWIGLU ? pow2f(-e) * kUp : pow2f(-e));
  if (SWIGLU) {
    // The whole block again if one of its lanes is next to a border, has a
    // number that the fp32 form is not for, or all are so small that fp32's
    // least numbers count.  (Between equal codes lies no other.)
    const uint2 lo = codes8(a, pow2f(-e) * kDown);
    float gmin = g[0];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gmin = fminf(gmin, g[i]);
      nan |= __builtin_isunordered(g[i], u[i]);
    }
    const bool near = nan || c.x != lo.x || c.y != lo.y ||
                      scale_exp(amax * kUp) != scale_exp(amax * kDown) || amax < 0x1p-80f ||
                      gmin < -87.f;
    const uint64_t any = __ballot(near);
    if ((any >> (threadIdx.x & 48)) & 0xffffu) {
      double b[8], m = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b[i] = swiglu64(g[i], u[i], limit);
        const double v = fabs(b[i]);
        if (v <= 3.402823466e38) m = fmax(m, v);
      }
      m = block_max(m);
      // rounding up keeps m <= 448 * 2^e true or false as in 64 bits
      e = scale_exp(__double2float_ru(m));
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = inf_to_nan(to_odd(b[i] * ldexp(1.0, -e)));
      c = codes8(a, 1.f);
    }
  }
  *reinterpret_cast<uint2*>(codes + static_cast<int64_t>(row) * K + col) = c;
  if ((threadIdx.x & 15) == 0) scales[blk] = static_cast<uint8_t>(e + 127);
}

}  // namespace

hipError_t launch_quant(const uint16_t* x, int64_t x_stride, int M, int K, float limit,
                        uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t blocks = static_cast<int64_t>(M) * (K / kBlock);
  const unsigned grid = static_cast<unsigned>((blocks + kThreads / 16 - 1) / (kThreads / 16));
  if (limit > 0.f)
    hipLaunchKernelGGL(quant_kernel<true>, dim3(grid), dim3(kThreads), 0, s, x, x_stride,
                       static_cast<uint32_t>(blocks), K, limit, codes, scales);
  else
    hipLaunchKernelGGL(quant_kernel<false>, dim3(grid), dim3(kThreads), 0, s, x, x_stride,
                       static_cast<uint32_t>(blocks), K, limit, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
