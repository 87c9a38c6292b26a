// Launch interfaces of the operators beside the MoE layer (moe_decode_ops.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_decode_ops.h"

namespace moe {

constexpr int kPage = MOE_DECODE_PAGE_TOKENS;
constexpr int kMaxBatch = 1024;

// ---- quantiser ----------------------------------------------------------------
hipError_t launch_quant(const uint16_t* x, int64_t x_stride, int M, int K, float limit,
                        uint8_t* codes, uint8_t* scales, hipStream_t s);

// ---- product ------------------------------------------------------------------
struct ProductArgs {
  const uint8_t* x;   // [M, K]
  const uint8_t* xs;  // [M, K/128]
  const uint8_t* w;   // [N, K]
  const void* ws;     // [ceil(N/128), K/128]
  void* out;
  int64_t ld;
  int M, N, K;
  bool e8m0, f32;
  bool wide;  // four outputs may be stored at once
  // (set by launch_product)
  int splits;       // workgroups that share out a tile's columns
  float* part;      // [tiles][splits] tiles of sums
  uint32_t* count;  // [tiles] parts handed in; 0 between runs
};
// Bytes that products of up to max_rows rows need, zeroed before the first.
size_t product_workspace(int max_rows, int N, int K, bool f32);
// Once per device (current), before the first launch.
hipError_t product_prepare();
hipError_t launch_product(const ProductArgs& a, void* ws, size_t ws_bytes, hipStream_t s);

// ---- cache --------------------------------------------------------------------
// The cache as the kernels see it.
struct CacheView {
  uint8_t* pool;
  uint8_t* scale;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* q_start;
  int pages, Hkv, D, max_pages, max_q, B, T;
};

// New tokens [q0, q0 + q) and length of sequence b; q = 0 for a sequence
// whose numbers do not fit.
struct Seq {
  int q0, q, len;
};
__device__ __forceinline__ Seq seq_of(const CacheView& c, int b) {
  const int q0 = c.q_start[b], q1 = c.q_start[b + 1], len = c.lens[b];
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= c.T && q1 - q0 <= c.max_q && len >= q1 - q0 &&
                  len <= c.max_pages * kPage;
  return ok ? Seq{q0, q1 - q0, len} : Seq{0, 0, 0};
}

// Codes of K (kv = 0) or V (1) of a page and head.
__device__ __forceinline__ size_t page_block(const CacheView& c, int page, int kv, int h) {
  return (static_cast<size_t>(page) * 2 + kv) * c.Hkv + h;
}

hipError_t launch_append(const CacheView& c, const uint16_t* k, int64_t k_stride,
                         const uint16_t* v, int64_t v_stride, hipStream_t s);

struct AttendArgs {
  CacheView c;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  int64_t out_stride;
  float scale_log2;  // sm_scale * log2(e)
  int G;             // heads per kv head
  int max_rows;      // rows of a sequence and kv head, padded to 16
  const float* mass_in;
  float* mass_out;
  float* rec;  // [B][max_pages][Hkv][max_rows]: log2 of a page's share of each row
  float* lse;  // [B][Hkv][max_rows]
  // workgroups per kv head and row tile, and what they hand to each other
  int workers;
  float* part_o;    // [y][workers + B][16][D]
  float* part_ml;   // [y][workers + B][16][2]: maximum, sum
  uint32_t* count;  // [y][B] parts handed in; 0 between runs
};
// Workgroups per kv head and row tile.
int attend_workers(int Hkv, int max_rows, int max_batch, int max_pages, int D);
hipError_t launch_attend(const AttendArgs& a, hipStream_t s);

struct EvictArgs {
  const int32_t *table, *lens;
  const float* mass;
  int32_t *out_table, *out_lens, *freed, *n_freed;
  float* out_mass;
  int B, max_pages, keep, sink, recent;
};
hipError_t launch_evict(const EvictArgs& a, hipStream_t s);

}  // namespace moe
