// Attention of a step's new tokens over the 8-bit paged cache.
//
// The q_b new tokens of a sequence and the G query heads of a kv head are
// its rows: row r = j G + i is token j, head i of the group.  A wave takes
// whole pages of 64 tokens and 16 rows:
//   S^T = K Q^T   v_mfma_f32_16x16x32_bf16, four tiles of 16 tokens: lane
//                 (g, c) = (l / 16, l % 16) gets S of tokens 16 s + 4 g + i
//                 (i < 4) and row c
//   O^T += V^T P^T  v_mfma_f32_16x16x32_f16: lane (g, c)'s 16 probabilities
//                 are its operand as they are, and V is stored so that a
//                 lane's 16 bytes are the same tokens of dimension c.
// Codes become bf16 / f16 exactly; the page's scale multiplies the scores (K)
// and the page's contribution (V) in fp32.  P goes in as f16: at most 1, off
// by at most 2^-12 of itself or 2^-25.  The softmax is kept as a running
// maximum and sum in fp32, in base 2; waves are joined at the end.
#include <algorithm>

#include "ops_device.h"
#include "ops_launch.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kRows = 16;
constexpr int kTeams = kThreads / 16;  // sixteen threads that hold one row
constexpr int kXcds = 8;
// Workgroups of a launch: one per CU.  Measured at one sequence of 131000
// tokens, 8 kv heads of 128: 50.6 us; two per CU 57.5 (the same bytes from
// twice as many places at once, and twice the parts to join), one of 512
// threads 52.7.
constexpr int kWantGroups = 256;

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ bf16x8_t codes_bf16(uint32_t w0, uint32_t w1) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ f16x8_t codes_f16(uint32_t w0, uint32_t w1) {
  const f16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, false);
  const f16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, true);
  const f16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, false);
  const f16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, true);
  return f16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 0xff in the bytes of w that are NaN codes.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  // (b & 0x7f) + 1 has bit 7 set only for 0x7f
  const uint32_t m = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return (m >> 7) * 0xffu;
}

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// Sixteen bytes; NT: not kept in the caches.
template <bool NT>
__device__ __forceinline__ uint4 load16(const uint8_t* p) {
  const u32x4_t* q = reinterpret_cast<const u32x4_t*>(p);
  return __builtin_bit_cast(uint4, NT ? __builtin_nontemporal_load(q) : *q);
}

// Maximum / sum over the four lane groups that share row c.
__device__ __forceinline__ float groups_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float groups_sum(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

// Least pages of a worker's share: one for each wave.
constexpr int kMinChunk = kWaves;

// Exclusive prefix over the sequences of the pages that row tile `rt` reads,
// in pref[0 .. B] (LDS).  Every thread calls it.
__device__ __forceinline__ void page_prefix(const AttendArgs& a, int rt, int* pref, int* tmp) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int carry = 0;
  for (int b0 = 0; b0 < a.c.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < a.c.B) {
      const Seq sq = seq_of(a.c, b);
      if (rt * kRows < sq.q * a.G) n = (sq.len + kPage - 1) / kPage;
    }
    int x = n;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int y = __shfl_up(x, off, kWave);
      if (lane >= off) x += y;
    }
    if (lane == 63) tmp[wave] = x;
    __syncthreads();
    int before = carry, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      before += w < wave ? tmp[w] : 0;
      all += tmp[w];
    }
    if (b < a.c.B) pref[b + 1] = before + x;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) pref[0] = 0;
  __syncthreads();
}

// Writes dimensions 4 q + 64 i .. + 3 of an output row, o scaled by inv.
template <int ND>
__device__ __forceinline__ void store_row(uint16_t* op, int q, const f32x4_t (&o)[ND], float inv) {
#pragma unroll
  for (int i = 0; i < ND; ++i)
    *reinterpret_cast<uint2*>(op + 4 * q + 64 * i) =
        make_uint2(f32_to_bf16(o[i][0] * inv) | f32_to_bf16(o[i][1] * inv) << 16,
                   f32_to_bf16(o[i][2] * inv) | f32_to_bf16(o[i][3] * inv) << 16);
}

// Workers: workgroup (w, y) has kv head y % Hkv and row tile y / Hkv and takes
// the pages [w chunk, (w + 1) chunk) of all sequences' pages laid end to end,
// so that every worker reads the same amount whatever the lengths are.  A
// sequence that lies in one worker is finished there; the parts of one that
// does not go to slots w + b (unique: along the pages either w or b grows)
// and the last worker to hand in joins them in order.
// head_dim = 64 ND; ONCE: one row tile, so that no other workgroup reads the
// same codes and the loads need not stay in the caches.
template <int ND, bool MASS, bool ONCE>
__global__ __launch_bounds__(kThreads, ND <= 2 ? 2 : 1) void attend_kernel(AttendArgs a) {
  constexpr int D = 64 * ND;
  constexpr int kJoin = ND <= 2 ? 8 : 4;  // parts that a thread loads at once
  __shared__ __attribute__((aligned(16))) float s_o[kWaves][kRows][D + 4];
  auto& s_j = *reinterpret_cast<float(*)[kTeams][D + 4]>(s_o);
  static_assert(kTeams <= kWaves * kRows, "a row of s_o per team");
  __shared__ float s_m[kWaves][kRows], s_l[kWaves][kRows];
  __shared__ int s_pref[kMaxBatch + 1];
  __shared__ int s_tmp[kWaves];
  __shared__ int s_b, s_last;
  const int h = blockIdx.y % a.c.Hkv, rt = blockIdx.y / a.c.Hkv, r0 = rt * kRows;
  const int tid = threadIdx.x;
  page_prefix(a, rt, s_pref, s_tmp);
  const int N = s_pref[a.c.B];
  const int chunk = max((N + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x),
                        kMinChunk);
  const int w_lo = blockIdx.x * chunk, w_hi = min(w_lo + chunk, N);
  if (w_lo >= w_hi) return;  // uniform over the workgroup
  for (int b = tid; b < a.c.B; b += kThreads)
    if (s_pref[b] <= w_lo && w_lo < s_pref[b + 1]) s_b = b;
  __syncthreads();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, g = lane >> 4, c = lane & 15;
  const size_t block_bytes = static_cast<size_t>(kPage) * D;
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};

  for (int at = w_lo, b = s_b; at < w_hi; ++b) {
    const int first = s_pref[b], n_pages = s_pref[b + 1] - first;
    if (n_pages == 0) continue;
    const Seq sq = seq_of(a.c, b);
    const int rows = sq.q * a.G;
    const int r = min(r0 + c, rows - 1);
    const int j = r / a.G;
    const int lim = sq.len - sq.q + j + 1;            // tokens that row c sees
    const int lim_lo = sq.len - sq.q + r0 / a.G + 1;  // that every row of the tile sees
    const int32_t* table = a.c.table + static_cast<size_t>(b) * a.c.max_pages;
    const int p_lo = at - first, p_hi = min(w_hi - first, n_pages);

    // Q operands: chunk q covers dimensions 64 (q / 2) + 16 g + 8 (q % 2) .. + 7
    bf16x8_t qf[2 * ND];
    {
      const uint16_t* qp = a.q + static_cast<int64_t>(sq.q0 + j) * a.q_stride +
                           (static_cast<int64_t>(h) * a.G + r - j * a.G) * D + 16 * g;
#pragma unroll
      for (int i = 0; i < 2 * ND; ++i)
        qf[i] = __builtin_bit_cast(
            bf16x8_t, *reinterpret_cast<const uint4*>(qp + 64 * (i >> 1) + 8 * (i & 1)));
    }
    f32x4_t acc[4 * ND];
#pragma unroll
    for (int t = 0; t < 4 * ND; ++t) acc[t] = zero;
    float m = neg_inf(), l = 0.f;  // l: this lane's tokens only

    // A page's operands and scales.  Each register is loaded with the next
    // page's bytes as soon as the matrix instruction has taken this page's, so
    // a whole page per wave is in flight at any time.
    uint4 kw[4 * ND], vw[4 * ND];
    uint32_t ks8, vs8;
    bool bad;
    size_t kb, vb;
    const uint8_t *kp, *vp;
    auto find_page = [&](int id) {
      bad = id < 0 || id >= a.c.pages;
      const int page = bad ? 0 : id;
      kb = page_block(a.c, page, 0, h);
      vb = page_block(a.c, page, 1, h);
      kp = a.c.pool + kb * block_bytes + (g * kPage + c) * 16;
      vp = a.c.pool + vb * block_bytes + (g * D + c) * 16;
    };
    auto load_k = [&](int s) {
#pragma unroll
      for (int i = 0; i < ND; ++i)
        kw[s * ND + i] = load16<ONCE>(kp + (i * 4 * kPage + 16 * s) * 16);
    };
    auto load_v = [&](int t) { vw[t] = load16<ONCE>(vp + t * 256); };
    for (int p0 = p_lo + wave; p0 < p_hi; p0 += kWave * kWaves) {
      // lane i holds the id of the wave's i-th page from here on: no load of an
      // id, and no wait for one, stands between the pages' loads
      const int ids = table[min(p0 + kWaves * lane, p_hi - 1)];
      const int count = min(kWave, (p_hi - p0 + kWaves - 1) / kWaves);
      find_page(__builtin_amdgcn_readlane(ids, 0));
      // In the order of the loop's loads: a wait is for the oldest loads, and
      // the compiler allows for both ways into the loop.
      ks8 = a.c.scale[kb];
      vs8 = a.c.scale[vb];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        load_k(s);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int t = 0; t < 4 * ND; ++t) {
        load_v(t);
        __builtin_amdgcn_sched_barrier(0);
      }
      for (int i = 0; i < count; ++i) {
        const int pi = p0 + i * kWaves;
        const float vs = e8m0_to_f32(vs8);
        const float ks = bad ? __uint_as_float(0x7fc00000u) : a.scale_log2 * e8m0_to_f32(ks8);
        // past the end: the last page again, so that no branch stands around
        // the loads (the waits below would then be for all of them)
        find_page(__builtin_amdgcn_readlane(ids, min(i + 1, count - 1)));
        ks8 = a.c.scale[kb];
        vs8 = a.c.scale[vb];
        __builtin_amdgcn_sched_barrier(0);
        f32x4_t sc[4];
#pragma unroll
        for (int s2 = 0; s2 < 4; s2 += 2) {
          // two tiles at a time: two independent chains of products
          sc[s2] = sc[s2 + 1] = zero;
#pragma unroll
          for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int s = s2; s < s2 + 2; ++s) {
              const uint4 w = kw[s * ND + i];
              sc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(w.x, w.y), qf[2 * i],
                                                              sc[s], 0, 0, 0);
              sc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(w.z, w.w),
                                                              qf[2 * i + 1], sc[s], 0, 0, 0);
            }
          load_k(s2);
          load_k(s2 + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
        const bool edge = pi * kPage + kPage > lim_lo;  // some row does not see all of the page
#pragma unroll
        for (int s = 0; s < 4; ++s) sc[s] *= ks;
        if (edge) {
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (pi * kPage + 16 * s + 4 * g + i >= lim) sc[s][i] = neg_inf();
          // A NaN code of V reaches only the rows that see it: 0 * NaN would
          // reach all.  Such places (rare) are cleared, and counted under the
          // rows' masks: a row that sees one is NaN from here on.
          uint32_t bits = 0;
#pragma unroll
          for (int t = 0; t < 4 * ND; ++t)
            bits |= nan_bytes(vw[t].x) | nan_bytes(vw[t].y) | nan_bytes(vw[t].z) |
                    nan_bytes(vw[t].w);
          if (__any(bits != 0)) {
            f16x8_t seen[2];
#pragma unroll
            for (int q = 0; q < 16; ++q)
              seen[q >> 3][q & 7] = static_cast<_Float16>(
                  pi * kPage + 16 * (q >> 2) + 4 * g + (q & 3) < lim ? 1.f : 0.f);
#pragma unroll
            for (int t = 0; t < 4 * ND; ++t) {
              const uint4 nb = make_uint4(nan_bytes(vw[t].x), nan_bytes(vw[t].y),
                                          nan_bytes(vw[t].z), nan_bytes(vw[t].w));
              vw[t] = make_uint4(vw[t].x & ~nb.x, vw[t].y & ~nb.y, vw[t].z & ~nb.z,
                                 vw[t].w & ~nb.w);
              constexpr uint32_t kOne = 0x38383838u;  // codes of 1
              f32x4_t n = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                  codes_f16(nb.x & kOne, nb.y & kOne), seen[0], zero, 0, 0, 0);
              n = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(nb.z & kOne, nb.w & kOne),
                                                         seen[1], n, 0, 0, 0);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n[i] > 0.f) acc[t][i] = __uint_as_float(0x7fc00000u);
            }
          }
        }
        float pm = neg_inf();
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) pm = fmaxf(pm, sc[s][i]);
        const float mn = fmaxf(m, groups_max(pm));
        const float ref = mn == neg_inf() ? 0.f : mn;
        const float alpha = exp2_(m - ref);
        float ps = 0.f;
        f16x8_t pf[2];
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = exp2_(sc[s][i] - ref);
            ps += p;
            pf[s >> 1][4 * (s & 1) + i] = static_cast<_Float16>(p);
          }
        l = l * alpha + ps;
        m = mn;
        if (MASS) {
          const float sum = groups_sum(ps);
          if (g == 0)
            a.rec[((static_cast<size_t>(b) * a.c.max_pages + pi) * a.c.Hkv + h) * a.max_rows + r0 +
                  c] = ref + __log2f(sum);
        }
#pragma unroll
        for (int t2 = 0; t2 < 4 * ND; t2 += 2) {
#pragma unroll
          for (int t = t2; t < t2 + 2; ++t) {
            const uint4 w = vw[t];
            f32x4_t o =
                __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(w.x, w.y), pf[0], zero, 0, 0, 0);
            o = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(w.z, w.w), pf[1], o, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(o[i], vs, acc[t][i] * alpha);
          }
          load_v(t2);
          load_v(t2 + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    l = groups_sum(l);
    // join the waves: dimension 16 t + 4 g + i of row c
    __syncthreads();  // the last segment's readers are done
#pragma unroll
    for (int t = 0; t < 4 * ND; ++t)
      *reinterpret_cast<f32x4_t*>(&s_o[wave][c][16 * t + 4 * g]) = acc[t];
    if (g == 0) {
      s_m[wave][c] = m;
      s_l[wave][c] = l;
    }
    __syncthreads();
    // A team of sixteen threads holds a row: thread q dimensions 4 q + 64 i.
    // The row's waves (here) or parts (below) are split over the teams that
    // the tile's rows leave: rv teams side by side take rows 0 .. rv - 1.
    const int valid = min(kRows, rows - r0);
    const int rv = valid > 8 ? 16 : valid > 4 ? 8 : valid > 2 ? 4 : valid > 1 ? 2 : 1;
    const int team = tid >> 4, q = tid & 15, row = team & (rv - 1), grp = team / rv;
    float mx = s_m[0][row];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mx = fmaxf(mx, s_m[w][row]);
    const float ref = mx == neg_inf() ? 0.f : mx;  // a part may see no token
    float sum = 0.f;
    f32x4_t o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) o[i] = zero;
    if (grp == 0 && row < valid) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = exp2_(s_m[w][row] - ref);
        sum += s_l[w][row] * f;
#pragma unroll
        for (int i = 0; i < ND; ++i)
          o[i] += *reinterpret_cast<const f32x4_t*>(&s_o[w][row][4 * q + 64 * i]) * f;
      }
    }
    const bool mine = grp == 0 && row < valid;
    const int out_j = (r0 + row) / a.G;
    uint16_t* op = a.out + static_cast<int64_t>(sq.q0 + out_j) * a.out_stride +
                   (static_cast<int64_t>(h) * a.G + r0 + row - out_j * a.G) * D;
    float* lse = a.lse + (static_cast<size_t>(b) * a.c.Hkv + h) * a.max_rows + r0 + row;
    if (p_hi - p_lo == n_pages) {
      if (mine) {
        store_row<ND>(op, q, o, 1.f / sum);
        if (MASS && q == 0) *lse = mx + __log2f(sum);
      }
    } else {
      // hand in: slots w0 + b .. w1 + b are the sequence's parts
      const int w0 = first / chunk, w1 = (first + n_pages - 1) / chunk, parts = w1 - w0 + 1;
      const size_t slot0 =
          static_cast<size_t>(blockIdx.y) * (gridDim.x + a.c.B) + w0 + b;  // part 0
      const size_t slot = slot0 + (blockIdx.x - w0);
      if (mine) {
        float* po = a.part_o + (slot * kRows + row) * D + 4 * q;
#pragma unroll
        for (int i = 0; i < ND; ++i)
          st_f32x4<true>(po + 64 * i, make_float4(o[i][0], o[i][1], o[i][2], o[i][3]));
        if (q == 0) {
          st_f32<true>(a.part_ml + (slot * kRows + row) * 2, mx);
          st_f32<true>(a.part_ml + (slot * kRows + row) * 2 + 1, sum);
        }
      }
      wait_memory();
      __syncthreads();
      uint32_t* cnt = a.count + static_cast<size_t>(blockIdx.y) * a.c.B + b;
      if (tid == 0)
        s_last = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                 static_cast<uint32_t>(parts) - 1;
      __syncthreads();
      if (s_last) {
        if (tid == 0) __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        // Plain loads: no workgroup has read a slot's lines in this launch
        // before they were written through.
        const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + slot0 * kRows;
        // Each team takes every step-th part of its row, a part's weight and
        // values loaded together (one trip to memory), in a running softmax.
        const int step = kTeams / rv;  // teams per row
        float top = neg_inf(), total = 0.f;
#pragma unroll
        for (int i = 0; i < ND; ++i) o[i] = zero;
        if (row < valid) {
          const float* base = a.part_o + (slot0 * kRows + row) * D + 4 * q;
          for (int p0 = grp; p0 < parts; p0 += kJoin * step) {
            float2 x[kJoin];
            float4 y[kJoin][ND];
#pragma unroll
            for (int k = 0; k < kJoin; ++k) {
              const int p = min(p0 + k * step, parts - 1);  // past the end: not used
              x[k] = ml[p * kRows + row];
#pragma unroll
              for (int i = 0; i < ND; ++i)
                y[k][i] = *reinterpret_cast<const float4*>(base + static_cast<size_t>(p) * kRows * D +
                                                           64 * i);
            }
            const float old = top;
#pragma unroll
            for (int k = 0; k < kJoin; ++k) top = fmaxf(top, x[k].x);
            const float r = top == neg_inf() ? 0.f : top;
            const float alpha = exp2_(old - r);
            total *= alpha;
#pragma unroll
            for (int i = 0; i < ND; ++i) o[i] *= alpha;
#pragma unroll
            for (int k = 0; k < kJoin; ++k) {
              if (p0 + k * step >= parts) break;
              const float w = exp2_(x[k].x - r);
              total += x[k].y * w;
#pragma unroll
              for (int i = 0; i < ND; ++i)
                o[i] += f32x4_t{y[k][i].x, y[k][i].y, y[k][i].z, y[k][i].w} * w;
            }
          }
        }
        // the row's teams in order
        if (row < valid) {
#pragma unroll
          for (int i = 0; i < ND; ++i)
            *reinterpret_cast<f32x4_t*>(&s_j[team][4 * q + 64 * i]) = o[i];
          if (q == 0) {
            s_j[team][D] = total;
            s_j[team][D + 1] = top;
          }
        }
        __syncthreads();
        if (mine) {
          for (int k = 1; k < step; ++k) top = fmaxf(top, s_j[k * rv + row][D + 1]);
          total = 0.f;
#pragma unroll
          for (int i = 0; i < ND; ++i) o[i] = zero;
          for (int k = 0; k < step; ++k) {
            const float* x = s_j[k * rv + row];
            const float w = exp2_(x[D + 1] - top);
#pragma unroll
            for (int i = 0; i < ND; ++i)
              o[i] += *reinterpret_cast<const f32x4_t*>(x + 4 * q + 64 * i) * w;
            total += x[D] * w;
          }
          store_row<ND>(op, q, o, 1.f / total);
          if (MASS && q == 0) *lse = top + __log2f(total);
        }
      }
    }
    at = first + p_hi;
  }
}

// mass_out of one page per thread: its share of every row, heads then rows in
// order.
__global__ __launch_bounds__(kThreads) void mass_kernel(AttendArgs a) {
  const int b = blockIdx.y, p = blockIdx.x * kThreads + threadIdx.x;
  const int32_t q0 = a.c.q_start[b], q1 = a.c.q_start[b + 1], len = a.c.lens[b];
  const Seq sq = seq_of(a.c, b);
  if (sq.q == 0 && !(q0 >= 0 && q0 == q1 && q1 <= a.c.T && len >= 0 &&
                     len <= a.c.max_pages * kPage))
    return;  // a sequence whose numbers do not fit
  if (p * kPage >= len) return;
  const size_t at = static_cast<size_t>(b) * a.c.max_pages + p;
  float sum = 0.f;
  for (int h = 0; h < a.c.Hkv; ++h) {
    const float* rec = a.rec + (at * a.c.Hkv + h) * a.max_rows;
    const float* lse = a.lse + (static_cast<size_t>(b) * a.c.Hkv + h) * a.max_rows;
    for (int r = 0; r < sq.q * a.G; ++r) sum += exp2_(rec[r] - lse[r]);
  }
  a.mass_out[at] = (a.mass_in ? a.mass_in[at] : 0.f) + sum;
}

template <int ND>
hipError_t launch(const AttendArgs& a, hipStream_t s) {
  const dim3 grid(a.workers, a.c.Hkv * (a.max_rows / kRows));
  const bool once = a.max_rows == kRows;
  auto* k = a.mass_out ? (once ? attend_kernel<ND, true, true> : attend_kernel<ND, true, false>)
                       : (once ? attend_kernel<ND, false, true> : attend_kernel<ND, false, false>);
  hipLaunchKernelGGL(k, grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Enough workgroups for two per CU, of no fewer than kMinChunk pages each, a
// multiple of the XCDs (a worker's row tiles then read its pages from one L2).
int attend_workers(int Hkv, int max_rows, int max_batch, int max_pages) {
  const int64_t y = static_cast<int64_t>(Hkv) * (max_rows / kRows);
  const int64_t pages = static_cast<int64_t>(max_batch) * max_pages;
  int64_t w = (kWantGroups + y - 1) / y;
  w = std::min(w, (pages + kMinChunk - 1) / kMinChunk);
  return static_cast<int>((w + kXcds - 1) / kXcds * kXcds);
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t s) {
  const hipError_t e = a.c.D == 64    ? launch<1>(a, s)
                       : a.c.D == 128 ? launch<2>(a, s)
                       : a.c.D == 192 ? launch<3>(a, s)
                                      : launch<4>(a, s);
  if (e != hipSuccess || !a.mass_out) return e;
  hipLaunchKernelGGL(mass_kernel, dim3((a.c.max_pages + kThreads - 1) / kThreads, a.c.B),
                     dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
