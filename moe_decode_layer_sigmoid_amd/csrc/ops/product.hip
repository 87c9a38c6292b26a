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
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "ops_device.h"
#include "ops_launch.h"

namespace moe {
namespace {

constexpr int kUnit = 127;  // e8m0 byte of 1

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

typedef __attribute__((address_space(3))) void lds_void_t;

__device__ __forceinline__ i32x8_t join32(const uint4& a, const uint4& b) {
  return i32x8_t{static_cast<int>(a.x), static_cast<int>(a.y), static_cast<int>(a.z),
                 static_cast<int>(a.w), static_cast<int>(b.x), static_cast<int>(b.y),
                 static_cast<int>(b.z), static_cast<int>(b.w)};
}

// Four consecutive outputs of row m from column n on.
template <bool F32>
__device__ __forceinline__ void store4(const ProductArgs& a, int m, int n, const f32x4_t& v) {
  if (m >= a.M) return;
  const size_t o = static_cast<size_t>(m) * a.ld + n;
  if (a.wide && n + 3 < a.N) {
    if (F32)
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + o) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) = make_uint2(
          f32_to_bf16(v[0]) | f32_to_bf16(v[1]) << 16, f32_to_bf16(v[2]) | f32_to_bf16(v[3]) << 16);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n + i >= a.N) break;
    if (F32) static_cast<float*>(a.out)[o + i] = v[i];
    else static_cast<uint16_t*>(a.out)[o + i] = static_cast<uint16_t>(f32_to_bf16(v[i]));
  }
}

// Tile of workgroup `id` of `tiles`: the workgroups of one XCD (every eighth)
// take neighbouring tiles, eight rows of tiles deep, so that its L2 holds the
// rows and columns they share.
__device__ __forceinline__ void tile_of(int id, int nt, int mt, int* n, int* m) {
  constexpr int kXcds = 8, kDeep = 8;
  const int tiles = nt * mt, full = tiles / kXcds * kXcds;
  const int t = id < full ? id % kXcds * (full / kXcds) + id / kXcds : id;
  const int group = t / (kDeep * nt), in = t - group * kDeep * nt;
  const int deep = min(kDeep, mt - group * kDeep);
  *m = group * kDeep + in % deep;
  *n = in / deep;
}

// Loads from base + off (per lane) to LDS address lds (uniform): sixteen bytes
// to lds + 16 lane, a byte (as a dword) or a dword to lds + 4 lane.  As
// instructions of their own and not the builtin, after which the compiler
// waits for the load before the next read of any LDS, also of another buffer
// (317 us instead of 271 at 8192 x 4096 x 6144, when this was the only
// difference; 196 with what came after): the kernel waits itself
// before the barrier that hands a buffer over.  m0, which they take the address
// from, is reserved to the compiler and cannot be named as overwritten; it
// sets m0 itself right before each instruction of its own that reads it.
#define MOE_LOAD_TO_LDS(name, op)                                                           \
  __device__ __forceinline__ void name(const uint8_t* base, uint32_t off, uint32_t lds) {   \
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\t" op " %1, %2"                             \
                 :                                                                          \
                 : "s"(lds), "v"(off), "s"(base)                                            \
                 : "memory");                                                               \
  }
MOE_LOAD_TO_LDS(load16_to_lds, "global_load_lds_dwordx4")
MOE_LOAD_TO_LDS(load4_to_lds, "global_load_lds_dword")
MOE_LOAD_TO_LDS(load1_to_lds, "global_load_lds_ubyte")
#undef MOE_LOAD_TO_LDS

__device__ __forceinline__ uint32_t lds_address(unsigned char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void_t*)p));
}

// Waits until at most N of the wave's loads are on their way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Shape of a tile: WN x WM waves of NT x MT tiles of 16 weight rows x 16
// activation rows, ST buffers of one block of 128 columns.
template <int WN_, int WM_, int NT_, int MT_, int ST_>
struct Tile {
  static constexpr int WN = WN_, WM = WM_, NT = NT_, MT = MT_, ST = ST_;
  static constexpr int kWaves = WN * WM, kThreads = 64 * kWaves;
  static constexpr int TN = 16 * WN * NT, TM = 16 * WM * MT;
  static constexpr int kPieces = (TN + TM) / 8;                  // load instructions of a round
  static constexpr int kLoads = (kPieces + kWaves - 1) / kWaves; // of a wave; the last may repeat
  static constexpr int kCodes = (TN + TM) * kBlock;              // bytes of a round's codes
  static constexpr int kScaleX = (TM + 63) / 64;                 // waves that bring x's scales
  static constexpr int kNB = TN > kBlock ? TN / kBlock : 1;      // weight scales of a round
  static constexpr int kStage = kCodes + 256 * (kScaleX + 1);
  static constexpr int kLds = ST * kStage;
  static_assert((ST - 2) * (kLoads + 1) < 64, "the wait counts to 63");
  static_assert(kBlock % (16 * NT) == 0, "a wave's weight rows share a scale");
  static_assert(kWaves > kScaleX, "a wave for each 64 activation scales, one for the weights'");
};

// y = (scales) x w^T for one tile and one part of the columns.
//
// A round is one block of 128 columns: its codes go straight to LDS, eight
// lanes per 128-byte row piece, into the buffer that was read ST - 1 rounds
// ago, and are taken ST - 1 rounds later.  Piece p of row r lies at slot
// p ^ (r / 2 % 8), which spreads the sixteen lanes that read one piece of
// sixteen rows over the banks.
//
// With splits > 1 the tile's columns are shared out over that many
// workgroups; each leaves its sums in `part` and the last to finish adds them
// in order.
template <class T, bool E8, bool F32, bool SPLIT>
__global__ __launch_bounds__(T::kThreads) void product_kernel(ProductArgs a) {
  constexpr int NT = T::NT, MT = T::MT, TN = T::TN, TM = T::TM;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  __shared__ int s_last;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wn = wave / T::WM, wm = wave - wn * T::WM;
  const int splits = SPLIT ? a.splits : 1;
  const int id = blockIdx.x / splits, split = blockIdx.x - id * splits;
  int tn, tm;
  tile_of(id, (a.N + TN - 1) / TN, (a.M + TM - 1) / TM, &tn, &tm);
  const int n0 = tn * TN, m0 = tm * TM;
  const int KB = a.K / kBlock;
  // KB and the splits are at most 512
  const int k_lo = SPLIT ? KB * split / splits : 0;
  const int k_hi = SPLIT ? KB * (split + 1) / splits : KB;

  // load instruction i of the wave: rows 8 j .. 8 j + 7 of the round, weight
  // rows first
  const uint8_t* wbase = a.w + static_cast<size_t>(n0) * a.K;
  const uint8_t* xbase = a.x + static_cast<size_t>(m0) * a.K;
  uint32_t src[T::kLoads];
#pragma unroll
  for (int i = 0; i < T::kLoads; ++i) {
    const int j = min(T::kLoads * wave + i, T::kPieces - 1);
    const int r = 8 * j + (lane >> 3);
    const int piece = (lane & 7) ^ ((r >> 1) & 7);
    const int row = j < TN / 8 ? min(r, a.N - 1 - n0) : min(r - TN, a.M - 1 - m0);
    src[i] = static_cast<uint32_t>(row) * static_cast<uint32_t>(a.K) + 16 * piece;
  }
  // scales: wave w < kScaleX brings those of activation rows 64 w + lane, the
  // others the weight blocks' (one of them would do; all issue as many loads)
  const bool scale_w = wave >= T::kScaleX;
  const uint8_t* sbase = scale_w ? static_cast<const uint8_t*>(a.ws) +
                                       static_cast<size_t>(n0 / kBlock) * KB * (E8 ? 1 : 4)
                                 : a.xs + static_cast<size_t>(m0) * KB;
  const int srow = scale_w ? min(min(lane, T::kNB - 1), (a.N - 1) / kBlock - n0 / kBlock)
                           : min(64 * wave + lane, a.M - 1 - m0);
  const uint32_t soff = static_cast<uint32_t>(srow * KB) * (scale_w && !E8 ? 4 : 1);
  const uint32_t lds0 = lds_address(smem);
  auto stage_codes = [&](int kb, uint32_t to) {
    const uint8_t *wk = wbase + kb * kBlock, *xk = xbase + kb * kBlock;
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) {
      const int j = min(T::kLoads * wave + i, T::kPieces - 1);
      load16_to_lds(j < TN / 8 ? wk : xk, src[i], to + 1024 * j);
    }
  };
  auto stage_scales = [&](int kb, uint32_t to) {
    const uint32_t st = to + T::kCodes + 256 * (scale_w ? T::kScaleX : wave);
    if (scale_w && !E8) load4_to_lds(sbase + 4 * kb, soff, st);
    else load1_to_lds(sbase + kb, soff, st);
  };
  constexpr int kPerRound = T::kLoads + 1;

  f32x4_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int s = 0; s < T::ST - 1; ++s)
    if (k_lo + s < k_hi) {
      stage_scales(k_lo + s, lds0 + s * T::kStage);
      stage_codes(k_lo + s, lds0 + s * T::kStage);
    }
  if (k_lo + T::ST - 2 < k_hi) wait_loads<(T::ST - 2) * kPerRound>();
  else wait_loads<0>();
  __syncthreads();
  // the lane's 32 bytes of row c of a 16-row tile: pieces 2 g and 2 g + 1
  const int o0 = 128 * c + 16 * ((2 * g) ^ (c >> 1)), o1 = 128 * c + 16 * ((2 * g + 1) ^ (c >> 1));
  // One round on buffer `buf`; with MORE, round kb + ST - 1's loads into the
  // buffer that was read last are issued behind this round's first reads
  // (which they would hold up while the memory unit takes them).  No branch
  // stands in a round: the compiler would sink the products behind it, and so
  // behind the wait at the round's end.
  auto round = [&](auto more, int kb, int buf) {
    constexpr bool MORE = decltype(more)::value;
    const uint32_t to = lds0 + (buf == 0 ? T::ST - 1 : buf - 1) * T::kStage;
    if (MORE) stage_scales(kb + T::ST - 1, to);
    const unsigned char* wst = smem + buf * T::kStage + wn * NT * 2048;
    const unsigned char* xst = smem + buf * T::kStage + TN * kBlock + wm * MT * 2048;
    const uint32_t* sst = reinterpret_cast<const uint32_t*>(smem + buf * T::kStage + T::kCodes);
    int sx[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) sx[t] = sst[(wm * MT + t) * 16 + c];
    const uint32_t sw32 = sst[64 * T::kScaleX + wn * NT * 16 / kBlock];
    const float sw = __uint_as_float(sw32);
    i32x8_t xf[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
      xf[t] = join32(*reinterpret_cast<const uint4*>(xst + 2048 * t + o0),
                     *reinterpret_cast<const uint4*>(xst + 2048 * t + o1));
    if (F32) {
      if (MORE) stage_codes(kb + T::ST - 1, to);
      float s[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) s[t] = (E8 ? e8m0_to_f32(sw32) : sw) * e8m0_to_f32(sx[t]);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const i32x8_t wf = join32(*reinterpret_cast<const uint4*>(wst + 2048 * i + o0),
                                  *reinterpret_cast<const uint4*>(wst + 2048 * i + o1));
        f32x4_t d[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) d[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bf16x8_t wq = codes_bf16(wf[2 * q], wf[2 * q + 1]);
#pragma unroll
          for (int t = 0; t < MT; ++t)
            d[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                wq, codes_bf16(xf[t][2 * q], xf[t][2 * q + 1]), d[t], 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][t][e] = fmaf(s[t], d[t][e], acc[i][t][e]);
      }
    } else {
      const int sw_byte = E8 ? static_cast<int>(sw32) : kUnit;
      f32x4_t d[2][MT];
      uint4 wa[2], wb[2];
      wa[0] = *reinterpret_cast<const uint4*>(wst + o0);
      wb[0] = *reinterpret_cast<const uint4*>(wst + o1);
      if (MORE) stage_codes(kb + T::ST - 1, to);
#pragma unroll
      for (int i = 0; i <= NT; ++i) {
        // row i's products, and beside them the sums of row i - 1 (VALU) and
        // the operand of row i + 1 (LDS)
        if (i + 1 < NT) {
          wa[(i + 1) & 1] = *reinterpret_cast<const uint4*>(wst + 2048 * (i + 1) + o0);
          wb[(i + 1) & 1] = *reinterpret_cast<const uint4*>(wst + 2048 * (i + 1) + o1);
        }
        const i32x8_t wf = join32(wa[i & 1], wb[i & 1]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if (i < NT) {
            if (E8) {
              acc[i][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                  wf, xf[t], acc[i][t], 0, 0, 0, sw_byte, 0, sx[t]);
            } else {
              const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
              d[i & 1][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                  wf, xf[t], zero, 0, 0, 0, sw_byte, 0, sx[t]);
            }
          }
          if (!E8 && i > 0)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i - 1][t][e] = fmaf(sw, d[(i - 1) & 1][t][e], acc[i - 1][t][e]);
        }
        if (i + 1 < NT) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
          if (!E8) __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // this wave's part of the next round is in LDS, then every other wave's;
    // and all have read this round's
    wait_loads<MORE ? (T::ST - 2) * kPerRound : 0>();
    __syncthreads();
  };
  int buf = 0, kb = k_lo;
  for (; kb < k_hi - (T::ST - 1); ++kb) {
    round(std::true_type{}, kb, buf);
    buf = buf == T::ST - 1 ? 0 : buf + 1;
  }
  for (; kb < k_hi; ++kb) {
    round(std::false_type{}, kb, buf);
    buf = buf == T::ST - 1 ? 0 : buf + 1;
  }

  if (SPLIT) {
    // hand in (write-through stores, then the count); parts of rows past M
    // are left out
    f32x4_t* part = reinterpret_cast<f32x4_t*>(a.part) +
                    static_cast<size_t>(id) * splits * (NT * MT * T::kThreads) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (m0 + (wm * MT + t) * 16 + c < a.M)
          st_f32x4<true>(reinterpret_cast<float*>(
                             part + (static_cast<size_t>(split) * NT * MT + i * MT + t) * T::kThreads),
                         make_float4(acc[i][t][0], acc[i][t][1], acc[i][t][2], acc[i][t][3]));
    wait_memory();
    __syncthreads();
    if (threadIdx.x == 0) {
      s_last = __hip_atomic_fetch_add(a.count + id, 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) ==
               static_cast<uint32_t>(splits) - 1;
      if (s_last)
        __hip_atomic_store(a.count + id, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!s_last) return;
    // Plain loads: nobody has read these lines in this launch before they
    // were written through.
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < MT; ++t)
          if (m0 + (wm * MT + t) * 16 + c < a.M)
            acc[i][t] += part[(static_cast<size_t>(s) * NT * MT + i * MT + t) * T::kThreads];
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t)
      store4<F32>(a, m0 + (wm * MT + t) * 16 + c, n0 + (wn * NT + i) * 16 + 4 * g, acc[i][t]);
}

template <class T, bool SPLIT>
hipError_t launch_tile(const ProductArgs& a, hipStream_t s) {
  auto* k = a.e8m0 ? (a.f32 ? product_kernel<T, true, true, SPLIT>
                            : product_kernel<T, true, false, SPLIT>)
                   : (a.f32 ? product_kernel<T, false, true, SPLIT>
                            : product_kernel<T, false, false, SPLIT>);
  const unsigned tiles =
      static_cast<unsigned>((a.N + T::TN - 1) / T::TN) * ((a.M + T::TM - 1) / T::TM);
  hipLaunchKernelGGL(k, dim3(tiles * a.splits), dim3(T::kThreads), T::kLds, s, a);
  return hipGetLastError();
}

// Sixteen bytes per lane to dst (uniform) + 16 lane, not kept in the caches.
__device__ __forceinline__ void load16_once(const uint8_t* p, unsigned char* dst) {
  constexpr unsigned kCpolNT = 2;
  __builtin_amdgcn_global_load_lds(p, (lds_void_t*)dst, 16, 0, kCpolNT);
}

// Up to 16 activation rows: 16 weight rows per workgroup, whose sixteen waves
// share out the columns, so that no round of one waits for another's.  A wave
// asks for two blocks of its columns at once (weights straight to its own LDS
// area, each byte once; activations, which every workgroup reads, from the L2
// to registers), waits and multiplies; the waves' sums are added in LDS.
// Bound by the weights' bytes and by one trip to memory: 7.1 us at 1 x 6144 x
// 4096, a streaming read of the weights 3.6.  Measured there: eight waves of four
// blocks 7.6, four of eight 7.3, the tile kernel in two parts 9.2.
constexpr int kRowsWaves = 16, kRowsBlocks = 2;

template <bool E8, bool F32>
__global__ __launch_bounds__(64 * kRowsWaves) void product_rows_kernel(ProductArgs a) {
  constexpr int U = kRowsBlocks;
  constexpr int kArea = U * 2048;  // bytes of a wave's blocks, and then of its sums
  __shared__ __attribute__((aligned(16))) unsigned char smem[kRowsWaves * kArea];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int n0 = blockIdx.x * 16;
  const int KB = a.K / kBlock;
  const int k_lo = KB * wave / kRowsWaves, k_hi = KB * (wave + 1) / kRowsWaves;
  unsigned char* area = smem + wave * kArea;
  const uint8_t* wrow[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 8 * i + (lane >> 3);
    wrow[i] = a.w + static_cast<size_t>(min(n0 + r, a.N - 1)) * a.K +
              16 * ((lane & 7) ^ ((r >> 1) & 7));
  }
  const size_t m = min(c, a.M - 1);
  const uint8_t* xp = a.x + m * a.K + 32 * g;
  const uint8_t* xs = a.xs + m * KB;
  const size_t ws0 = static_cast<size_t>(n0 / kBlock) * KB;
  const int o0 = 128 * c + 16 * ((2 * g) ^ (c >> 1)), o1 = 128 * c + 16 * ((2 * g + 1) ^ (c >> 1));
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  f32x4_t acc = zero;
  for (int k0 = k_lo; k0 < k_hi; k0 += U) {
    // blocks past the end: the last one again, not taken below
    i32x8_t xf[U];
    int sx[U];
    uint32_t sw32[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(k0 + u, k_hi - 1);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        load16_once(wrow[i] + kb * kBlock, area + (2 * u + i) * 1024);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(k0 + u, k_hi - 1);
      xf[u] = join32(*reinterpret_cast<const uint4*>(xp + kb * kBlock),
                     *reinterpret_cast<const uint4*>(xp + kb * kBlock + 16));
      sx[u] = xs[kb];
      sw32[u] = E8 ? static_cast<const uint8_t*>(a.ws)[ws0 + kb]
                   : static_cast<const uint32_t*>(a.ws)[ws0 + kb];
    }
    // the weights are in LDS (the compiler need not wait for them by itself)
    wait_memory();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u >= k_hi) break;  // uniform over the wave
      const unsigned char* st = area + u * 2048;
      const i32x8_t wf = join32(*reinterpret_cast<const uint4*>(st + o0),
                                *reinterpret_cast<const uint4*>(st + o1));
      const float sw = __uint_as_float(sw32[u]);
      if (F32) {
        f32x4_t d = zero;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(wf[2 * q], wf[2 * q + 1]),
                                                      codes_bf16(xf[u][2 * q], xf[u][2 * q + 1]),
                                                      d, 0, 0, 0);
        const float s = (E8 ? e8m0_to_f32(sw32[u]) : sw) * e8m0_to_f32(sx[u]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fmaf(s, d[e], acc[e]);
      } else if (E8) {
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            wf, xf[u], acc, 0, 0, 0, static_cast<int>(sw32[u]), 0, sx[u]);
      } else {
        const f32x4_t d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            wf, xf[u], zero, 0, 0, 0, kUnit, 0, sx[u]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fmaf(sw, d[e], acc[e]);
      }
    }
  }
  __syncthreads();  // every wave's blocks are read: the area takes the sums
  f32x4_t* sums = reinterpret_cast<f32x4_t*>(smem);
  sums[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave > 0) return;
  for (int w = 1; w < kRowsWaves; ++w) acc += sums[w * 64 + lane];
  store4<F32>(a, c, n0 + 4 * g, acc);
}

hipError_t launch_rows(const ProductArgs& a, hipStream_t s) {
  auto* k = a.e8m0 ? (a.f32 ? product_rows_kernel<true, true> : product_rows_kernel<true, false>)
                   : (a.f32 ? product_rows_kernel<false, true> : product_rows_kernel<false, false>);
  hipLaunchKernelGGL(k, dim3((a.N + 15) / 16), dim3(64 * kRowsWaves), 0, s, a);
  return hipGetLastError();
}

// fp32 outputs of many rows and columns: a 64 x 64 tile per workgroup, its
// columns' blocks dealt out over eight waves, each of which takes the whole tile.
// So a code is converted once for four matrix instructions (two in the tile
// kernel's waves of 32 x 32, where conversions set the time), and no wave waits
// for another before the end.  A wave's block goes to its own LDS area, from
// there to registers, and the next block is on its way while this one is
// multiplied.  The waves' sums are added in LDS, in order.  Bound by the wave's
// own sequence of LDS reads, conversions and products, about 2.3 us a block of
// eight waves.  Measured against the tile kernel: 333 x 5003 x 6144 35 us (40),
// 64 x 16000 x 6144 27.9 (33.9), 128 x 8000 x 4096 15.7 (19.8); where its tiles
// leave a last round of CUs empty, the tile kernel stays (600 x 4096 x 4096 36.3,
// this one 39.5; 4096 x 4096 x 4096 111, 203).
constexpr int kDealWaves = 8, kDealTile = 64;

template <bool E8>
__global__ __launch_bounds__(64 * kDealWaves) void product_deal_kernel(ProductArgs a) {
  constexpr int T = kDealTile / 16;
  constexpr int kArea = 2 * kDealTile * kBlock;  // bytes of a wave's block, and of its sums
  constexpr int kLoads = kArea / 1024;
  static_assert(kArea == kDealTile * kDealTile * 4, "the sums take the areas");
  __shared__ __attribute__((aligned(16))) unsigned char smem[kDealWaves * kArea];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  int tn, tm;
  tile_of(blockIdx.x, (a.N + kDealTile - 1) / kDealTile, (a.M + kDealTile - 1) / kDealTile, &tn,
          &tm);
  const int n0 = tn * kDealTile, m0 = tm * kDealTile;
  const int KB = a.K / kBlock;
  const uint8_t* wbase = a.w + static_cast<size_t>(n0) * a.K;
  const uint8_t* xbase = a.x + static_cast<size_t>(m0) * a.K;
  const uint8_t* sbase = a.xs + static_cast<size_t>(m0) * KB;
  const size_t ws0 = static_cast<size_t>(n0 / kBlock) * KB;
  unsigned char* area = smem + wave * kArea;
  const uint32_t lds0 = lds_address(area);
  // load j: rows 8 j .. 8 j + 7, weight rows first, swizzled as in the tile kernel
  uint32_t src[kLoads], soff[T];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r = 8 * j + (lane >> 3), piece = (lane & 7) ^ ((r >> 1) & 7);
    const int row = j < kLoads / 2 ? min(r, a.N - 1 - n0) : min(r - kDealTile, a.M - 1 - m0);
    src[j] = static_cast<uint32_t>(row) * static_cast<uint32_t>(a.K) + 16 * piece;
  }
#pragma unroll
  for (int t = 0; t < T; ++t)
    soff[t] = static_cast<uint32_t>(min(16 * t + c, a.M - 1 - m0)) * KB;
  const int o0 = 128 * c + 16 * ((2 * g) ^ (c >> 1)), o1 = 128 * c + 16 * ((2 * g + 1) ^ (c >> 1));
  f32x4_t acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  int sx[T];
  uint32_t sw = 0;
  auto load_block = [&](int kb) {
#pragma unroll
    for (int t = 0; t < T; ++t) sx[t] = sbase[soff[t] + kb];
    sw = E8 ? static_cast<const uint8_t*>(a.ws)[ws0 + kb]
            : static_cast<const uint32_t*>(a.ws)[ws0 + kb];
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      load16_to_lds((j < kLoads / 2 ? wbase : xbase) + kb * kBlock, src[j], lds0 + 1024 * j);
  };
  load_block(wave);  // K has a block for every wave
  for (int kb = wave; kb < KB; kb += kDealWaves) {
    wait_loads<0>();
    float s[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
      s[t] = (E8 ? e8m0_to_f32(sw) : __uint_as_float(sw)) * e8m0_to_f32(sx[t]);
    uint4 w[T][2];
    bf16x8_t xq[T][4];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const unsigned char* p = area + (T + t) * 2048;
      const uint4 x0 = *reinterpret_cast<const uint4*>(p + o0);
      const uint4 x1 = *reinterpret_cast<const uint4*>(p + o1);
      xq[t][0] = codes_bf16(x0.x, x0.y);
      xq[t][1] = codes_bf16(x0.z, x0.w);
      xq[t][2] = codes_bf16(x1.x, x1.y);
      xq[t][3] = codes_bf16(x1.z, x1.w);
    }
#pragma unroll
    for (int i = 0; i < T; ++i) {
      w[i][0] = *reinterpret_cast<const uint4*>(area + i * 2048 + o0);
      w[i][1] = *reinterpret_cast<const uint4*>(area + i * 2048 + o1);
    }
    // every read of the area is done before the next block goes there
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    // past the end: this block again, so that no branch stands around the loads
    load_block(kb + kDealWaves < KB ? kb + kDealWaves : kb);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < T; ++i) {
      bf16x8_t wq[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        wq[2 * h] = codes_bf16(w[i][h].x, w[i][h].y);
        wq[2 * h + 1] = codes_bf16(w[i][h].z, w[i][h].w);
      }
      f32x4_t d[T];
#pragma unroll
      for (int t = 0; t < T; ++t) d[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int t = 0; t < T; ++t)
          d[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wq[q], xq[t][q], d[t], 0, 0, 0);
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][t][e] = fmaf(s[t], d[t][e], acc[i][t][e]);
    }
  }
  wait_loads<0>();  // the last loads, before the area takes the sums
  f32x4_t* mine = reinterpret_cast<f32x4_t*>(area) + lane;
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int t = 0; t < T; ++t) mine[(i * T + t) * 64] = acc[i][t];
  __syncthreads();
  const f32x4_t* sums = reinterpret_cast<const f32x4_t*>(smem) + lane;
  constexpr int kEach = T * T / kDealWaves;  // 16 x 16 tiles of a wave
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int p = wave * kEach + j, i = p / T, t = p % T;
    f32x4_t v = sums[p * 64];
    for (int k = 1; k < kDealWaves; ++k) v += sums[(k * T * T + p) * 64];
    store4<true>(a, m0 + 16 * t + c, n0 + 16 * i + 4 * g, v);
  }
}

hipError_t launch_deal(const ProductArgs& a, hipStream_t s) {
  const unsigned tiles = static_cast<unsigned>((a.N + kDealTile - 1) / kDealTile) *
                         ((a.M + kDealTile - 1) / kDealTile);
  hipLaunchKernelGGL(a.e8m0 ? product_deal_kernel<true> : product_deal_kernel<false>, dim3(tiles),
                     dim3(64 * kDealWaves), 0, s, a);
  return hipGetLastError();
}

// The shapes, and what a round of one costs in 10 ns, alone on its CU and per
// workgroup of a CU that has several (measured at K = 6144 and 1024, N = 128
// to 8192, 1 to 4096 rows, codes past the Infinity Cache).
using Tile64x32 = Tile<4, 1, 1, 2, 4>;
using Tile64 = Tile<2, 2, 2, 2, 4>;
using Tile128 = Tile<4, 2, 2, 4, 4>;
using Tile256 = Tile<2, 4, 8, 4, 2>;
struct Shape {
  int tn, tm;
  int alone, shared;          // bf16 outputs
  int alone_f32, shared_f32;  // fp32 outputs
};
constexpr Shape kShapes[] = {{Tile64x32::TN, Tile64x32::TM, 36, 20, 41, 26},
                             {Tile64::TN, Tile64::TM, 42, 26, 57, 40},
                             {Tile128::TN, Tile128::TM, 80, 80, 116, 116},
                             {Tile256::TN, Tile256::TM, 208, 208, 360, 360}};
constexpr int kRowsShape = 4;  // product_rows_kernel
constexpr int kDealShape = 5;  // product_deal_kernel
constexpr int kDealStep = 240, kDealFixed = 340;  // of it, in 10 ns
constexpr int kCus = 256;
// Splits only where all parts run at once: at most two workgroups per CU.
constexpr int kMaxParts = 2 * kCus;

struct Choice {
  int shape, splits;
  size_t tiles;
};

// The shape and the splits with the least estimated time: rounds times a
// round's cost, and for splits a join of about 0.6 us per split and 8 ns per
// part.  Measured against the alternatives at N = 4096, K = 6144: 16 rows 10.0
// us (rows kernel; 64 x 32 tiles in two parts 11.8), 64 rows 13.2 (64 x 32, two
// parts; whole 17.9), 333 rows 24.1 (64 x 64; 64 x 32 27.5), 1000 rows 39.6
// (128 x 128; 64 x 64 49.8), 4096 rows 106 (256 x 256; 128 x 128 153).
Choice choose(int M, int N, int K, bool f32) {
  // up to 16 rows: the rows kernel, unless its re-reading of x by every 16
  // weight rows outweighs the join (8192 weight rows: 16.3 us, split tiles 12.3)
  if (M <= 16 && (M <= 4 || N <= 6144)) return {kRowsShape, 1, 0};
  const int KB = K / kBlock;
  Choice best{0, 1, 0};
  int64_t least = INT64_MAX;
  for (int i = 0; i < kRowsShape; ++i) {
    const Shape& s = kShapes[i];
    const int64_t tiles = static_cast<int64_t>((N + s.tn - 1) / s.tn) * ((M + s.tm - 1) / s.tm);
    for (int splits = 1; splits <= (i < 2 ? 4 : 1); splits *= 2) {
      const int64_t parts = tiles * splits;
      if (splits > 1 && (parts > kMaxParts || KB < 2 * splits)) break;
      const int64_t per_cu = (parts + kCus - 1) / kCus;
      const int64_t round = f32 ? std::max<int64_t>(s.alone_f32, s.shared_f32 * per_cu)
                                : std::max<int64_t>(s.alone, s.shared * per_cu);
      const int64_t cost =
          (KB + splits - 1) / splits * round + (splits > 1 ? 60 * splits + parts * 4 / 5 : 0);
      if (cost < least) {
        least = cost;
        best = {i, splits, static_cast<size_t>(tiles)};
      }
    }
  }
  if (f32 && M > 32 && KB >= kDealWaves) {
    // the dealing kernel: rounds of one workgroup per CU, each some setting up
    // and joining and a step for every eight blocks (up to 32 rows waste half its
    // tile: 20 x 16000 x 4096 15.8 us, else 14.1)
    const int64_t tiles = static_cast<int64_t>((N + kDealTile - 1) / kDealTile) *
                          ((M + kDealTile - 1) / kDealTile);
    const int64_t cost = (tiles + kCus - 1) / kCus *
                         ((KB + kDealWaves - 1) / kDealWaves * kDealStep + kDealFixed);
    if (cost < least) best = {kDealShape, 1, static_cast<size_t>(tiles)};
  }
  return best;
}

// Bytes of a choice's counts and parts.
size_t parts_bytes(const Choice& c) {
  if (c.splits == 1) return 0;
  return kMaxParts * sizeof(uint32_t) +
         c.tiles * c.splits * kShapes[c.shape].tn * kShapes[c.shape].tm * sizeof(float);
}

template <class T, bool SPLIT>
hipError_t allow_lds() {
  const void* k[] = {reinterpret_cast<const void*>(product_kernel<T, true, true, SPLIT>),
                     reinterpret_cast<const void*>(product_kernel<T, true, false, SPLIT>),
                     reinterpret_cast<const void*>(product_kernel<T, false, true, SPLIT>),
                     reinterpret_cast<const void*>(product_kernel<T, false, false, SPLIT>)};
  for (const void* f : k) {
    const hipError_t e =
        hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t product_workspace(int max_rows, int N, int K, bool f32) {
  size_t most = 0;
  // the choice depends on the rows only through the rows kernel's limits and
  // through multiples of 32; no splits above kMaxParts tiles of 32 rows
  for (int M = 1; M <= max_rows && M <= 32 * kMaxParts + 1; M += M <= 32 ? 1 : 32)
    most = std::max(most, parts_bytes(choose(M, N, K, f32)));
  return most;
}

hipError_t product_prepare() {
  hipError_t e = allow_lds<Tile64x32, false>();
  if (e == hipSuccess) e = allow_lds<Tile64x32, true>();
  if (e == hipSuccess) e = allow_lds<Tile64, false>();
  if (e == hipSuccess) e = allow_lds<Tile64, true>();
  if (e == hipSuccess) e = allow_lds<Tile128, false>();
  if (e == hipSuccess) e = allow_lds<Tile256, false>();
  return e;
}

hipError_t launch_product(const ProductArgs& a0, void* ws, size_t ws_bytes, hipStream_t s) {
  ProductArgs a = a0;
  const Choice c = choose(a.M, a.N, a.K, a.f32);
  a.splits = parts_bytes(c) <= ws_bytes ? c.splits : 1;
  a.count = static_cast<uint32_t*>(ws);
  a.part = reinterpret_cast<float*>(a.count + kMaxParts);
  switch (c.shape) {
    case kRowsShape: return launch_rows(a, s);
    case kDealShape: return launch_deal(a, s);
    case 0: return a.splits > 1 ? launch_tile<Tile64x32, true>(a, s) : launch_tile<Tile64x32, false>(a, s);
    case 1: return a.splits > 1 ? launch_tile<Tile64, true>(a, s) : launch_tile<Tile64, false>(a, s);
    case 2: return launch_tile<Tile128, false>(a, s);
    default: return launch_tile<Tile256, false>(a, s);
  }
}

}  // namespace moe

