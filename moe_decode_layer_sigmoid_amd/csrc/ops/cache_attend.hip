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
// maximum and sum in fp32, in base 2; waves are joined at the end of a
// sequence, workers by the last of them.
//
// Bound by the cache's bytes where it is long: 131000 tokens of 8 kv heads of
// 128 (268 MB) in 48.5 us, of which the pages take 38 (7.0 TB/s), the way to the
// first page 3, the parts' joining 5; 64 sequences of up to 8192 tokens with the
// mass 72.5 us (5.1 TB/s).  Short sequences are bound by that chain of waits.
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
// Workgroups of a launch: one per CU.  Measured with one, one and a half, two
// per CU (the same bytes from more places at once, and more parts to join): one
// sequence of 131000 tokens, 8 kv heads of 128, 48.9, 57.8, 53.8 us; 8 of 16000,
// 8 kv heads of 64, 13.8, 14.3, 13.7 us; of 256, 33.0, 44.3, 42.0 us.
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

// Least share of a worker: a page for each wave.  Measured with 4, 8, 16: one
// sequence of 1000 tokens 9.3, 10.4, 10.3 us, of 4000 10.8, 11.4, 13.2 us.
constexpr int kMinChunk = kWaves;

// What a sequence costs a worker beside its pages, in pages: its waves joined,
// its output or part written.  Measured with 0, 4, 8, 12: 32 sequences of up to
// 2100 tokens, 2 kv heads of 64, 14.1, 12.3, 9.8, 9.7 us; 64 of up to 8192
// tokens, 8 kv heads of 128, 73.9, 72.5, 72.5, 73.0 us.
constexpr int kSeqCost = 8;

// The sequences' numbers, and the exclusive prefix of what row tile `rt` has
// to do for them (pages, and kSeqCost for any), in LDS.
struct Seqs {
  int pref[kMaxBatch + 1], q0[kMaxBatch], q[kMaxBatch], len[kMaxBatch];
  int tmp[kWaves];
};

// Every thread calls it.
__device__ __forceinline__ void read_seqs(const AttendArgs& a, int rt, Seqs& s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int carry = 0;
  if (threadIdx.x == 0) s.pref[0] = 0;
  for (int b0 = 0; b0 < a.c.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < a.c.B) {
      const Seq sq = seq_of(a.c, b);
      if (rt * kRows < sq.q * a.G) n = (sq.len + kPage - 1) / kPage + kSeqCost;
      s.q0[b] = sq.q0;
      s.q[b] = sq.q;
      s.len[b] = sq.len;
    }
    int x = n;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int y = __shfl_up(x, off, kWave);
      if (lane >= off) x += y;
    }
    if (lane == 63) s.tmp[wave] = x;
    __syncthreads();
    int before = carry, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      before += w < wave ? s.tmp[w] : 0;
      all += s.tmp[w];
    }
    if (b < a.c.B) s.pref[b + 1] = before + x;
    carry += all;
    __syncthreads();
  }
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Pages that a wave goes through between two fetches of page ids (a lane
// stays free for the id that comes after them).
constexpr int kBatch = kWave - 1;

// A worker's way through its pages, in batches: wave w's are p + w + 4 i of
// sequence b, i < kBatch, below hi.
struct Batch {
  int b, n_pages, lo, hi, p;  // [lo, hi): the worker's pages of b
  bool opens;                 // the first of its sequence
};

// The first batch of the first sequence from b on that has pages in [at, w_hi),
// or `none`.
__device__ __forceinline__ Batch open_batch(const Seqs& s, int B, int at, int b, int w_hi,
                                            Batch none) {
  for (; b < B; ++b) {
    const int first = uniform(s.pref[b]), n = uniform(s.pref[b + 1]) - first - kSeqCost;
    if (first >= w_hi) break;
    if (first + n <= at || n <= 0) continue;  // n < 0: no pages
    const int lo = max(at - first, 0);
    return Batch{b, n, lo, min(w_hi - first, n), lo, true};
  }
  return none;
}

// The batch behind x; behind the worker's last one its last page again (the
// loads that run ahead need something to load).
__device__ __forceinline__ Batch next_batch(const Seqs& s, int B, Batch x, int w_hi) {
  Batch more = x;
  more.opens = false;
  if (x.p + kBatch * kWaves < x.hi) {
    more.p += kBatch * kWaves;
    return more;
  }
  more.p = x.hi - 1;
  return open_batch(s, B, 0, x.b + 1, w_hi, more);
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
// the part [w chunk, (w + 1) chunk) of all sequences' pages (and costs) laid end
// to end, so that all workers have the same to do whatever the lengths are.  A
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
  __shared__ Seqs s_seq;
  __shared__ int s_b, s_last[2];
  const int h = blockIdx.y % a.c.Hkv, rt = blockIdx.y / a.c.Hkv, r0 = rt * kRows;
  const int tid = threadIdx.x;
  read_seqs(a, rt, s_seq);
  const int N = uniform(s_seq.pref[a.c.B]);
  const int chunk = max((N + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x),
                        kMinChunk);
  const int w_lo = blockIdx.x * chunk, w_hi = min(w_lo + chunk, N);
  if (w_lo >= w_hi) return;  // uniform over the workgroup
  for (int b = tid; b < a.c.B; b += kThreads)
    if (s_seq.pref[b] <= w_lo && w_lo < s_seq.pref[b + 1]) s_b = b;
  __syncthreads();
  const int wave = uniform(tid >> 6);
  const int lane = tid & 63, g = lane >> 4, c = lane & 15;
  const size_t block_bytes = static_cast<size_t>(kPage) * D;
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};

  // Q operands of a sequence: chunk q covers dimensions 64 (q / 2) + 16 g +
  // 8 (q % 2) .. + 7
  auto load_q = [&](int b, u32x4_t(&q)[2 * ND]) {
    const int r = min(r0 + c, s_seq.q[b] * a.G - 1), j = r / a.G;
    const uint16_t* qp = a.q + static_cast<int64_t>(s_seq.q0[b] + j) * a.q_stride +
                         (static_cast<int64_t>(h) * a.G + r - j * a.G) * D + 16 * g;
#pragma unroll
    for (int i = 0; i < 2 * ND; ++i)
      q[i] = *reinterpret_cast<const u32x4_t*>(qp + 64 * (i >> 1) + 8 * (i & 1));
  };
  // A wave without pages goes through the worker's last page with all of it
  // masked: then every batch has the same shape.
  auto pages_of_wave = [&](const Batch& x) {
    return uniform(max(min((x.hi - x.p - wave + kWaves - 1) / kWaves, kBatch), 1));
  };
  // Lane i holds the id of the wave's i-th page of batch x, the lanes behind
  // those that of its first page of the next batch: no load of an id, and no
  // wait for one, stands between the pages' loads.
  auto load_ids = [&](const Batch& x, const Batch& next) {
    const bool in = lane < pages_of_wave(x);
    const int b = in ? x.b : next.b;
    const int p = in ? min(x.p + wave + kWaves * lane, x.hi - 1) : min(next.p + wave, next.hi - 1);
    return a.c.table[static_cast<size_t>(b) * a.c.max_pages + p];
  };
  Batch cur = open_batch(s_seq, a.c.B, w_lo, uniform(s_b), w_hi, Batch{});
  if (!cur.opens) return;  // uniform over the workgroup
  Batch nxt = next_batch(s_seq, a.c.B, cur, w_hi);
  // ids and Q operands, and those of the batch that follows
  int ids, idn = load_ids(cur, nxt);
  u32x4_t qf[2 * ND], qn[2 * ND];
  load_q(cur.b, qn);

  // A page's operands and scales.  Each register is loaded with the next
  // page's bytes as soon as the matrix instruction has taken this page's, so
  // a whole page per wave is in flight at any time, also from one sequence to
  // the next.
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
  // In the order of the loop's loads: a wait is for the oldest loads, and the
  // compiler allows for every way into the loop.
  auto load_page = [&](int id) {
    find_page(id);
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
  };
  load_page(__builtin_amdgcn_readlane(idn, 0));

  f32x4_t acc[4 * ND];
  float m = 0.f, l = 0.f;  // l: this lane's tokens only
  int lim = 0, lim_lo = 0;
  int handed = 0, handed_b0 = 0, handed_b1 = 0;  // sequences whose parts this worker writes

  // A team of sixteen threads holds a row: thread q dimensions 4 q + 64 i.  The
  // row's parts are split over the teams that the tile's rows leave: rv teams
  // side by side take rows 0 .. rv - 1, step of them each row.
  const int q = tid & 15;
  struct Place {
    int valid, rv, step, row, grp;
    bool mine;
  };
  auto place = [&](int b) {
    Place x;
    x.valid = min(kRows, uniform(s_seq.q[b]) * a.G - r0);
    x.rv = x.valid > 8 ? 16 : x.valid > 4 ? 8 : x.valid > 2 ? 4 : x.valid > 1 ? 2 : 1;
    x.step = kTeams / x.rv;
    x.row = (tid >> 4) & (x.rv - 1);
    x.grp = (tid >> 4) / x.rv;
    x.mine = x.grp == 0 && x.row < x.valid;
    return x;
  };
  auto out_row = [&](int b, int row) {
    const int j = (r0 + row) / a.G;
    return a.out + static_cast<int64_t>(s_seq.q0[b] + j) * a.out_stride +
           (static_cast<int64_t>(h) * a.G + r0 + row - j * a.G) * D;
  };
  auto lse_of = [&](int b, int row) {
    return a.lse + (static_cast<size_t>(b) * a.c.Hkv + h) * a.max_rows + r0 + row;
  };
  // sequence b's parts: workers first .. last, in slots w + b
  auto first_worker = [&](int b) { return s_seq.pref[b] / chunk; };
  auto last_worker = [&](int b) { return (s_seq.pref[b + 1] - kSeqCost - 1) / chunk; };
  const size_t slots = static_cast<size_t>(blockIdx.y) * (gridDim.x + a.c.B);
  auto counter = [&](int b) { return a.count + static_cast<size_t>(blockIdx.y) * a.c.B + b; };
  for (;;) {
    const int b = cur.b;
    // Waits for what the batch before began with, and so stays out of the page
    // loop.
    ids = idn;
    asm volatile("" : "+v"(ids));
#pragma unroll
    for (int i = 0; i < 2 * ND; ++i) {
      qf[i] = qn[i];
      asm volatile("" : "+v"(qf[i]));
    }
    const Batch nn = next_batch(s_seq, a.c.B, nxt, w_hi);
    idn = load_ids(nxt, nn);
    load_q(nxt.b, qn);
    __builtin_amdgcn_sched_barrier(0);
    if (cur.opens) {
      const int rows = uniform(s_seq.q[b]) * a.G;
      const int past = uniform(s_seq.len[b] - s_seq.q[b]);
      lim = past + min(r0 + c, rows - 1) / a.G + 1;  // tokens that row c sees
      lim_lo = past + r0 / a.G + 1;                  // that every row of the tile sees
#pragma unroll
      for (int t = 0; t < 4 * ND; ++t) acc[t] = zero;
      m = neg_inf();
      l = 0.f;
    }
    const int count = pages_of_wave(cur);
    int i = 0;
    do {
      const int pi = cur.p + wave + i * kWaves;
      const bool real = pi < cur.hi;
      const int t0 = real ? pi * kPage : INT32_MAX - kPage;  // its first token
      const float vs = real ? e8m0_to_f32(vs8) : 0.f;
      const float ks = bad ? __uint_as_float(0x7fc00000u) : a.scale_log2 * e8m0_to_f32(ks8);
      find_page(__builtin_amdgcn_readlane(ids, i + 1));
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
            sc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                codes_bf16(w.x, w.y), __builtin_bit_cast(bf16x8_t, qf[2 * i]), sc[s], 0, 0, 0);
            sc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                codes_bf16(w.z, w.w), __builtin_bit_cast(bf16x8_t, qf[2 * i + 1]), sc[s], 0, 0, 0);
          }
        load_k(s2);
        load_k(s2 + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      const bool edge = t0 + kPage > lim_lo;  // some row does not see all of the page
#pragma unroll
      for (int s = 0; s < 4; ++s) sc[s] *= ks;
      if (edge) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t0 + 16 * s + 4 * g + i >= lim) sc[s][i] = neg_inf();
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
                t0 + 16 * (q >> 2) + 4 * g + (q & 3) < lim ? 1.f : 0.f);
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
        if (g == 0 && real)
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
    } while (++i < count);
    if (cur.p + kBatch * kWaves >= cur.hi) {  // the last batch of the sequence here
      l = groups_sum(l);
      // join the waves: dimension 16 t + 4 g + i of row c
      __syncthreads();  // the last sequence's readers are done
#pragma unroll
      for (int t = 0; t < 4 * ND; ++t)
        *reinterpret_cast<f32x4_t*>(&s_o[wave][c][16 * t + 4 * g]) = acc[t];
      if (g == 0) {
        s_m[wave][c] = m;
        s_l[wave][c] = l;
      }
      __syncthreads();
      const Place at = place(b);
      float mx = s_m[0][at.row];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) mx = fmaxf(mx, s_m[w][at.row]);
      const float ref = mx == neg_inf() ? 0.f : mx;  // a part may see no token
      float sum = 0.f;
      f32x4_t o[ND];
#pragma unroll
      for (int i = 0; i < ND; ++i) o[i] = zero;
      if (at.mine) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float f = exp2_(s_m[w][at.row] - ref);
          sum += s_l[w][at.row] * f;
#pragma unroll
          for (int i = 0; i < ND; ++i)
            o[i] += *reinterpret_cast<const f32x4_t*>(&s_o[w][at.row][4 * q + 64 * i]) * f;
        }
      }
      if (cur.hi - cur.lo == cur.n_pages) {
        if (at.mine) {
          store_row<ND>(out_row(b, at.row), q, o, 1.f / sum);
          if (MASS && q == 0) *lse_of(b, at.row) = mx + __log2f(sum);
        }
      } else {
        // A part: the sequence began before this worker's pages or goes on
        // behind them, so there are at most two.  Handed in at the end.
        if (at.mine) {
          const size_t slot = slots + blockIdx.x + b;
          float* po = a.part_o + (slot * kRows + at.row) * D + 4 * q;
#pragma unroll
          for (int i = 0; i < ND; ++i)
            st_f32x4<true>(po + 64 * i, make_float4(o[i][0], o[i][1], o[i][2], o[i][3]));
          if (q == 0) {
            st_f32<true>(a.part_ml + (slot * kRows + at.row) * 2, mx);
            st_f32<true>(a.part_ml + (slot * kRows + at.row) * 2 + 1, sum);
          }
        }
        if (handed == 0) handed_b0 = b;
        handed_b1 = b;
        ++handed;
      }
      if (!nxt.opens) break;
    }
    cur = nxt;
    nxt = nn;
  }
  if (handed == 0) return;

  // Parts are counted per sequence; the last worker to hand in joins them.
  wait_memory();
  __syncthreads();
  if (tid < handed) {
    const int b = tid ? handed_b1 : handed_b0;
    s_last[tid] = __hip_atomic_fetch_add(counter(b), 1u, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT) ==
                  static_cast<uint32_t>(last_worker(b) - first_worker(b));
  }
  __syncthreads();
  for (int k = 0; k < handed; ++k) {
    if (!s_last[k]) continue;  // uniform over the workgroup
    const int b = k ? handed_b1 : handed_b0;
    if (tid == 0) __hip_atomic_store(counter(b), 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const Place at = place(b);
    const int w0 = uniform(first_worker(b)), parts = uniform(last_worker(b)) - w0 + 1;
    const size_t slot0 = slots + w0 + b;
    // Plain loads: no workgroup has read a slot's lines in this launch before
    // they were written through.
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + slot0 * kRows;
    // Each team takes every step-th part of its row, a part's weight and
    // values loaded together (one trip to memory), in a running softmax.
    float top = neg_inf(), total = 0.f;
    f32x4_t o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) o[i] = zero;
    if (at.row < at.valid) {
      const float* base = a.part_o + (slot0 * kRows + at.row) * D + 4 * q;
      for (int p0 = at.grp; p0 < parts; p0 += kJoin * at.step) {
        float2 x[kJoin];
        float4 y[kJoin][ND];
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
          const int p = min(p0 + j * at.step, parts - 1);  // past the end: not used
          x[j] = ml[p * kRows + at.row];
#pragma unroll
          for (int i = 0; i < ND; ++i)
            y[j][i] = *reinterpret_cast<const float4*>(base + static_cast<size_t>(p) * kRows * D +
                                                       64 * i);
        }
        const float old = top;
#pragma unroll
        for (int j = 0; j < kJoin; ++j) top = fmaxf(top, x[j].x);
        const float r = top == neg_inf() ? 0.f : top;
        const float alpha = exp2_(old - r);
        total *= alpha;
#pragma unroll
        for (int i = 0; i < ND; ++i) o[i] *= alpha;
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
          // selects, no branch: the compiler would load behind it
          const bool in = p0 + j * at.step < parts;
          const float w = exp2_(x[j].x - r);
          total += in ? x[j].y * w : 0.f;
#pragma unroll
          for (int i = 0; i < ND; ++i)
            o[i] += in ? f32x4_t{y[j][i].x, y[j][i].y, y[j][i].z, y[j][i].w} * w : zero;
        }
      }
    }
    // the row's teams in order
    __syncthreads();  // the last readers of s_o are done
    if (at.row < at.valid) {
#pragma unroll
      for (int i = 0; i < ND; ++i)
        *reinterpret_cast<f32x4_t*>(&s_j[tid >> 4][4 * q + 64 * i]) = o[i];
      if (q == 0) {
        s_j[tid >> 4][D] = total;
        s_j[tid >> 4][D + 1] = top;
      }
    }
    __syncthreads();
    if (at.mine) {
      for (int j = 1; j < at.step; ++j) top = fmaxf(top, s_j[j * at.rv + at.row][D + 1]);
      total = 0.f;
#pragma unroll
      for (int i = 0; i < ND; ++i) o[i] = zero;
      for (int j = 0; j < at.step; ++j) {
        const float* x = s_j[j * at.rv + at.row];
        const float w = exp2_(x[D + 1] - top);
#pragma unroll
        for (int i = 0; i < ND; ++i)
          o[i] += *reinterpret_cast<const f32x4_t*>(x + 4 * q + 64 * i) * w;
        total += x[D] * w;
      }
      store_row<ND>(out_row(b, at.row), q, o, 1.f / total);
      if (MASS && q == 0) *lse_of(b, at.row) = top + __log2f(total);
    }
  }
}

// mass_out: sixteen threads per page take its share of the rows of all heads,
// in turn, and add their sums in a fixed order.
constexpr int kMassPages = kThreads / 16;

__global__ __launch_bounds__(kThreads) void mass_kernel(AttendArgs a) {
  const int b = blockIdx.y, i = threadIdx.x & 15;
  const int p = blockIdx.x * kMassPages + (threadIdx.x >> 4);
  const int32_t q0 = a.c.q_start[b], q1 = a.c.q_start[b + 1], len = a.c.lens[b];
  const Seq sq = seq_of(a.c, b);
  if (sq.q == 0 && !(q0 >= 0 && q0 == q1 && q1 <= a.c.T && len >= 0 &&
                     len <= a.c.max_pages * kPage))
    return;  // a sequence whose numbers do not fit
  if (p >= a.c.max_pages || p * kPage >= len) return;  // uniform over the sixteen
  const size_t at = static_cast<size_t>(b) * a.c.max_pages + p;
  const unsigned rows = sq.q * a.G, n = rows * a.c.Hkv;
  float sum = 0.f;
  for (unsigned x = i; x < n; x += 16) {
    const unsigned h = x / rows, r = x - h * rows;
    sum += exp2_(a.rec[(at * a.c.Hkv + h) * a.max_rows + r] -
                 a.lse[(static_cast<size_t>(b) * a.c.Hkv + h) * a.max_rows + r]);
  }
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor(sum, off, kWave);
  if (i == 0) a.mass_out[at] = (a.mass_in ? a.mass_in[at] : 0.f) + sum;
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

// Enough workgroups for one per CU, of no fewer than kMinChunk pages each; a
// multiple of the XCDs (a worker's row tiles then read its pages from one L2)
// unless that fills the CUs worse: heads of more than 128 leave room for one
// workgroup per CU, others for two.  Measured at 16 sequences of 4096 tokens, 5
// new ones, 8 query heads on each of 8 kv heads of 192 (24 tiles): 10 workers
// 27.5 us, 16 in two turns 43.5; 3 of 3096, 10 new, of 256 (40 tiles): 6 workers
// 23.4, 8 in two turns 32.4.
int attend_workers(int Hkv, int max_rows, int max_batch, int max_pages, int D) {
  const int64_t y = static_cast<int64_t>(Hkv) * (max_rows / kRows);
  const int64_t pages = static_cast<int64_t>(max_batch) * max_pages;
  const int64_t least = std::min((kWantGroups + y - 1) / y, (pages + kMinChunk - 1) / kMinChunk);
  const int64_t w = (least + kXcds - 1) / kXcds * kXcds;
  const int64_t room = D <= 128 ? 2 * kWantGroups : kWantGroups;
  const int64_t fit = room / y;  // that run at once
  const int64_t turns = (y * w + room - 1) / room;
  // a worker's share of the pages, times the turns
  return static_cast<int>(turns > 1 && fit > 0 && w < turns * fit ? fit : w);
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t s) {
  const hipError_t e = a.c.D == 64    ? launch<1>(a, s)
                       : a.c.D == 128 ? launch<2>(a, s)
                       : a.c.D == 192 ? launch<3>(a, s)
                                      : launch<4>(a, s);
  if (e != hipSuccess || !a.mass_out) return e;
  hipLaunchKernelGGL(mass_kernel, dim3((a.c.max_pages + kMassPages - 1) / kMassPages, a.c.B),
                     dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
