// Block-scaled fp8 product y = (sx x) (sw w)^T on the gfx950 matrix cores.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 weight rows (operand A) by
// 16 activation rows (operand B) over one scale block of 128 columns: lane
// (g, c) = (l / 16, l % 16) holds 32 bytes of row c; both operands take the
// same bytes of a row, so the order of the columns inside the block does not
// matter.  D[4 g + i][c] is weight row 4 g + i, activation row c.
// The power-of-two scales go into the instruction; fp32 weight scales
// multiply its result.
//
// That instruction aligns the products of each eight consecutive columns to
// the largest of them and drops what lies more than 13 bits below (seen with
// one large and one small product at every distance); their sums and the
// accumulator are fp32.  The result is off by about 1.5e-5 of its size on
// normal data, a hundredth of what rounding it to bf16 costs, so bf16 outputs
// take it.  fp32 outputs take v_mfma_f32_16x16x32_bf16 on the exactly converted
// codes instead, whose products and sums are fp32 throughout, at half the rate.
#include "ops_device.h"
#include "ops_launch.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 127;  // e8m0 byte of 1

__device__ __forceinline__ i32x8_t load32(const uint8_t* p) {
  const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 16);
  return i32x8_t{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z),
                 static_cast<int>(a.w), static_cast<int>(b.x), static_cast<int>(b.y),
                 static_cast<int>(b.z), static_cast<int>(b.w)};
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Eight codes -> eight bf16 (exact).
__device__ __forceinline__ bf16x8_t codes_bf16(int w0, int w1) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One wave: 16 weight rows x 16 activation rows.
template <bool E8, bool F32>
__global__ __launch_bounds__(kThreads) void product_kernel(ProductArgs a) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int n0 = (blockIdx.x * (kThreads / kWave) + (threadIdx.x >> 6)) * 16;
  const int m0 = blockIdx.y * 16;
  if (n0 >= a.N) return;
  const int KB = a.K / kBlock;
  const int n = min(n0 + c, a.N - 1), m = min(m0 + c, a.M - 1);
  const uint8_t* wp = a.w + static_cast<size_t>(n) * a.K + 32 * g;
  const uint8_t* xp = a.x + static_cast<size_t>(m) * a.K + 32 * g;
  const uint8_t* xs = a.xs + static_cast<size_t>(m) * KB;
  const size_t ws0 = static_cast<size_t>(n0 / kBlock) * KB;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int kb = 0; kb < KB; ++kb) {
    const i32x8_t wf = load32(wp + kb * kBlock), xf = load32(xp + kb * kBlock);
    const int sx = xs[kb];
    if (F32) {
      f32x4_t d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(wf[2 * q], wf[2 * q + 1]),
                                                    codes_bf16(xf[2 * q], xf[2 * q + 1]), d, 0, 0, 0);
      const float sw = load_scale<E8>(a.ws, ws0 + kb) * e8m0_to_f32(sx);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(sw, d[i], acc[i]);
    } else if (E8) {
      const int sw = static_cast<const uint8_t*>(a.ws)[ws0 + kb];
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf, acc, 0, 0, 0, sw, 0, sx);
    } else {
      const float sw = static_cast<const float*>(a.ws)[ws0 + kb];
      const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
      const f32x4_t d =
          __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf, zero, 0, 0, 0, kUnit, 0, sx);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(sw, d[i], acc[i]);
    }
  }
  if (m0 + c >= a.M) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int nn = n0 + 4 * g + i;
    if (nn >= a.N) continue;
    const size_t o = static_cast<size_t>(m0 + c) * a.ld + nn;
    if (F32) static_cast<float*>(a.out)[o] = acc[i];
    else static_cast<uint16_t*>(a.out)[o] = static_cast<uint16_t>(f32_to_bf16(acc[i]));
  }
}

}  // namespace

hipError_t launch_product(const ProductArgs& a, hipStream_t s) {
  const dim3 grid((a.N + 63) / 64, (a.M + 15) / 16);
  auto* k = a.e8m0 ? (a.f32 ? product_kernel<true, true> : product_kernel<true, false>)
                   : (a.f32 ? product_kernel<false, true> : product_kernel<false, false>);
  hipLaunchKernelGGL(k, grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
