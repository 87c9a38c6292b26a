// C ABI of the operators beside the MoE layer: checks, plans, runs.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "device_common.h"
#include "moe_decode_ops.h"
#include "ops_launch.h"

struct moe_decode_product_plan_s {
  moe_decode_product_desc desc;
  int device;
  void* ws;
  size_t ws_bytes;
};

struct moe_decode_cache_plan_s {
  moe_decode_cache_desc desc;
  int device;
  void* ws;
  size_t ws_bytes;
};

namespace {

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// The current device for the length of a call.
class DeviceScope {
 public:
  explicit DeviceScope(int device) {
    if (hipGetDevice(&prev_) != hipSuccess) return;
    ok_ = prev_ == device || hipSetDevice(device) == hipSuccess;
    changed_ = ok_ && prev_ != device;
  }
  ~DeviceScope() {
    if (changed_) (void)hipSetDevice(prev_);
  }
  bool ok() const { return ok_; }

 private:
  int prev_ = -1;
  bool ok_ = false, changed_ = false;
};

// Checks the device and allocates a zeroed workspace on it (bytes > 0).
int plan_workspace(int device, size_t bytes, void** ws) {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) != hipSuccess || device < 0 || device >= ndev)
    return MOE_DECODE_ERR_INVALID_ARG;
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, device) != hipSuccess) return MOE_DECODE_ERR_HIP;
  if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) return MOE_DECODE_ERR_UNSUPPORTED;
  DeviceScope dev(device);
  if (!dev.ok()) return MOE_DECODE_ERR_HIP;
  *ws = nullptr;
  if (bytes == 0) return MOE_DECODE_OK;
  if (hipMalloc(ws, bytes) != hipSuccess) {
    *ws = nullptr;
    return MOE_DECODE_ERR_NO_MEMORY;
  }
  if (hipMemset(*ws, 0, bytes) != hipSuccess || hipDeviceSynchronize() != hipSuccess) {
    (void)hipFree(*ws);
    *ws = nullptr;
    return MOE_DECODE_ERR_HIP;
  }
  return MOE_DECODE_OK;
}

void free_workspace(int device, void* ws) {
  if (!ws) return;
  DeviceScope dev(device);
  (void)hipDeviceSynchronize();  // no launch of the plan may still use it
  (void)hipFree(ws);
}

int status(hipError_t e) { return e == hipSuccess ? MOE_DECODE_OK : MOE_DECODE_ERR_HIP; }

constexpr int32_t kMaxRows = 1 << 20, kMaxK = 65536;

int max_rows_of(const moe_decode_cache_desc& d) {
  const int rows = d.max_q * (d.heads / d.kv_heads);
  return (rows + 15) / 16 * 16;
}

// The attention's workspace, laid out from `base` (nullptr: only its size).
size_t cache_layout(const moe_decode_cache_desc& d, char* base, moe::AttendArgs* a) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? base + off : nullptr;
    off += align256(bytes);
    return p;
  };
  const size_t rows = max_rows_of(d), heads = d.kv_heads, B = d.max_batch;
  const size_t mass = d.with_mass ? 1 : 0;
  char* lse = take(mass * B * heads * rows * 4);
  char* rec = take(mass * B * d.max_pages * heads * rows * 4);
  const size_t y = heads * (rows / 16);
  const size_t workers = moe::attend_workers(d.kv_heads, static_cast<int>(rows), d.max_batch,
                                             d.max_pages, d.head_dim);
  char* part_o = take(y * (workers + B) * 16 * d.head_dim * 4);
  char* part_ml = take(y * (workers + B) * 16 * 2 * 4);
  char* count = take(y * B * 4);
  if (a) {
    a->workers = static_cast<int>(workers);
    a->part_o = reinterpret_cast<float*>(part_o);
    a->part_ml = reinterpret_cast<float*>(part_ml);
    a->count = reinterpret_cast<uint32_t*>(count);
    a->lse = reinterpret_cast<float*>(lse);
    a->rec = reinterpret_cast<float*>(rec);
  }
  return off;
}

bool cache_ok(const moe_decode_cache& c) {
  return c.pool && c.pool_scale && c.page_table && c.seq_lens && c.q_start &&
         aligned(c.pool, 16) && aligned(c.page_table, 4) && aligned(c.seq_lens, 4) &&
         aligned(c.q_start, 4);
}

bool run_sizes_ok(const moe_decode_cache_desc& d, int32_t B, int32_t T) {
  return B >= 0 && B <= d.max_batch && T >= 0;
}

// Rows of `heads` heads, `stride` elements apart.
bool rows_ok(const void* p, int64_t stride, int heads, int D, int align_elems) {
  return p && aligned(p, 2 * align_elems) && stride >= static_cast<int64_t>(heads) * D &&
         stride % align_elems == 0 && stride <= (int64_t{1} << 31);
}

moe::CacheView view(const moe_decode_cache_desc& d, const moe_decode_cache& c, int32_t B,
                    int32_t T) {
  return moe::CacheView{static_cast<uint8_t*>(c.pool),
                        static_cast<uint8_t*>(c.pool_scale),
                        c.page_table,
                        c.seq_lens,
                        c.q_start,
                        d.pages,
                        d.kv_heads,
                        d.head_dim,
                        d.max_pages,
                        d.max_q,
                        B,
                        T};
}

}  // namespace

extern "C" {

// ---- quantiser ------------------------------------------------------------------

int moe_decode_quant(const void* x, int64_t x_stride, int32_t M, int32_t K, float limit,
                     void* codes, void* scales, void* stream) {
  if (!x || !codes || !scales || M < 0 || K <= 0 || !(limit >= 0.f && limit <= 1e18f))
    return MOE_DECODE_ERR_INVALID_ARG;
  const int64_t cols = limit > 0.f ? 2 * static_cast<int64_t>(K) : K;
  if (!aligned(x, 16) || !aligned(codes, 8) || x_stride < cols || x_stride % 8)
    return MOE_DECODE_ERR_INVALID_ARG;
  // a launch has fewer than 2^32 threads, one for eight values (and room)
  if (K % moe::kBlock || K > kMaxK || M > kMaxRows || x_stride > (int64_t{1} << 31) ||
      static_cast<int64_t>(M) * K > int64_t{1} << 34)
    return MOE_DECODE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_DECODE_OK;
  return status(moe::launch_quant(static_cast<const uint16_t*>(x), x_stride, M, K, limit,
                                  static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                                  static_cast<hipStream_t>(stream)));
}

// ---- product --------------------------------------------------------------------

int moe_decode_product_desc_check(const moe_decode_product_desc* d) {
  if (!d || d->n <= 0 || d->k <= 0 || d->max_rows <= 0) return MOE_DECODE_ERR_INVALID_ARG;
  if (d->scale_fmt != MOE_DECODE_SCALE_FP32 && d->scale_fmt != MOE_DECODE_SCALE_E8M0)
    return MOE_DECODE_ERR_INVALID_ARG;
  if (d->out_fmt != MOE_DECODE_OUT_BF16 && d->out_fmt != MOE_DECODE_OUT_FP32)
    return MOE_DECODE_ERR_INVALID_ARG;
  if (d->k % moe::kBlock || d->k > kMaxK || d->n > kMaxRows || d->max_rows > kMaxRows)
    return MOE_DECODE_ERR_UNSUPPORTED;
  return MOE_DECODE_OK;
}

int moe_decode_product_args_check(const moe_decode_product_desc* d,
                                  const moe_decode_product_args* a, int32_t M) {
  const int rc = moe_decode_product_desc_check(d);
  if (rc) return rc;
  if (!a || M < 0 || M > d->max_rows) return MOE_DECODE_ERR_INVALID_ARG;
  if (!a->codes || !a->scales || !a->w || !a->w_scale || !a->out)
    return MOE_DECODE_ERR_INVALID_ARG;
  if (!aligned(a->codes, 16) || !aligned(a->w, 16)) return MOE_DECODE_ERR_INVALID_ARG;
  if (d->scale_fmt == MOE_DECODE_SCALE_FP32 && !aligned(a->w_scale, 4))
    return MOE_DECODE_ERR_INVALID_ARG;
  if (!aligned(a->out, d->out_fmt == MOE_DECODE_OUT_FP32 ? 4 : 2))
    return MOE_DECODE_ERR_INVALID_ARG;
  if (a->out_stride < d->n || a->out_stride > (int64_t{1} << 31))
    return MOE_DECODE_ERR_INVALID_ARG;
  return MOE_DECODE_OK;
}

int moe_decode_product_plan(const moe_decode_product_desc* d, int device,
                            moe_decode_product_plan_t* out) {
  if (!out) return MOE_DECODE_ERR_INVALID_ARG;
  *out = nullptr;
  int rc = moe_decode_product_desc_check(d);
  if (rc) return rc;
  void* ws = nullptr;
  const size_t bytes = moe::product_workspace(d->max_rows, d->n, d->k,
                                              d->out_fmt == MOE_DECODE_OUT_FP32);
  rc = plan_workspace(device, bytes, &ws);
  if (rc) return rc;
  {
    DeviceScope dev(device);
    if (!dev.ok() || moe::product_prepare() != hipSuccess) {
      free_workspace(device, ws);
      return MOE_DECODE_ERR_HIP;
    }
  }
  auto* p = new (std::nothrow) moe_decode_product_plan_s{*d, device, ws, bytes};
  if (!p) {
    free_workspace(device, ws);
    return MOE_DECODE_ERR_NO_MEMORY;
  }
  *out = p;
  return MOE_DECODE_OK;
}

int moe_decode_product_run(moe_decode_product_plan_t p, const moe_decode_product_args* a,
                           int32_t M, void* stream) {
  if (!p) return MOE_DECODE_ERR_INVALID_ARG;
  const int rc = moe_decode_product_args_check(&p->desc, a, M);
  if (rc || M == 0) return rc;
  DeviceScope dev(p->device);
  if (!dev.ok()) return MOE_DECODE_ERR_HIP;
  moe::ProductArgs k{};
  k.x = static_cast<const uint8_t*>(a->codes);
  k.xs = static_cast<const uint8_t*>(a->scales);
  k.w = static_cast<const uint8_t*>(a->w);
  k.ws = a->w_scale;
  k.out = a->out;
  k.ld = a->out_stride;
  k.M = M;
  k.N = p->desc.n;
  k.K = p->desc.k;
  k.e8m0 = p->desc.scale_fmt == MOE_DECODE_SCALE_E8M0;
  k.f32 = p->desc.out_fmt == MOE_DECODE_OUT_FP32;
  const int elem = k.f32 ? 4 : 2;
  k.wide = aligned(k.out, 4 * elem) && k.ld % 4 == 0;
  return status(moe::launch_product(k, p->ws, p->ws_bytes, static_cast<hipStream_t>(stream)));
}

int moe_decode_product_destroy(moe_decode_product_plan_t p) {
  if (!p) return MOE_DECODE_OK;
  free_workspace(p->device, p->ws);
  delete p;
  return MOE_DECODE_OK;
}

size_t moe_decode_product_workspace_bytes(moe_decode_product_plan_t p) {
  return p ? p->ws_bytes : 0;
}

// ---- cache ----------------------------------------------------------------------

int moe_decode_cache_desc_check(const moe_decode_cache_desc* d) {
  if (!d || d->heads <= 0 || d->kv_heads <= 0 || d->head_dim <= 0 || d->pages <= 0 ||
      d->max_batch <= 0 || d->max_pages <= 0 || d->max_q <= 0)
    return MOE_DECODE_ERR_INVALID_ARG;
  if (d->with_mass != 0 && d->with_mass != 1) return MOE_DECODE_ERR_INVALID_ARG;
  if (d->head_dim % 64 || d->head_dim > 256 || d->heads % d->kv_heads ||
      d->heads / d->kv_heads > 16 || d->kv_heads > 128 || d->max_batch > moe::kMaxBatch ||
      d->max_pages > 16384 || d->max_q > 256 || d->pages > (1 << 24))
    return MOE_DECODE_ERR_UNSUPPORTED;
  return MOE_DECODE_OK;
}

int moe_decode_append_check(const moe_decode_cache_desc* d, const moe_decode_append_args* a,
                            int32_t B, int32_t T) {
  const int rc = moe_decode_cache_desc_check(d);
  if (rc) return rc;
  if (!a || !run_sizes_ok(*d, B, T) || !cache_ok(a->cache) ||
      !rows_ok(a->k, a->k_stride, d->kv_heads, d->head_dim, 8) ||
      !rows_ok(a->v, a->v_stride, d->kv_heads, d->head_dim, 8))
    return MOE_DECODE_ERR_INVALID_ARG;
  return MOE_DECODE_OK;
}

int moe_decode_attend_check(const moe_decode_cache_desc* d, const moe_decode_attend_args* a,
                            int32_t B, int32_t T) {
  const int rc = moe_decode_cache_desc_check(d);
  if (rc) return rc;
  if (!a || !run_sizes_ok(*d, B, T) || !cache_ok(a->cache) ||
      !rows_ok(a->q, a->q_stride, d->heads, d->head_dim, 8) ||
      !rows_ok(a->out, a->out_stride, d->heads, d->head_dim, 4))
    return MOE_DECODE_ERR_INVALID_ARG;
  if (a->out == a->q || !std::isfinite(a->sm_scale)) return MOE_DECODE_ERR_INVALID_ARG;
  if ((a->mass_out && !d->with_mass) || (a->mass_in && !a->mass_out) ||
      !aligned(a->mass_in, 4) || !aligned(a->mass_out, 4))
    return MOE_DECODE_ERR_INVALID_ARG;
  return MOE_DECODE_OK;
}

int moe_decode_evict_check(const moe_decode_cache_desc* d, const moe_decode_evict_args* a,
                           int32_t B) {
  const int rc = moe_decode_cache_desc_check(d);
  if (rc) return rc;
  if (!a || !run_sizes_ok(*d, B, 0)) return MOE_DECODE_ERR_INVALID_ARG;
  const void* req[] = {a->page_table, a->seq_lens, a->mass,  a->out_table,
                       a->out_lens,   a->out_mass, a->freed, a->n_freed};
  for (const void* p : req)
    if (!p || !aligned(p, 4)) return MOE_DECODE_ERR_INVALID_ARG;
  // freed and n_freed are nothing else
  for (int i = 0; i < 6; ++i)
    if (req[i] == a->freed || req[i] == a->n_freed) return MOE_DECODE_ERR_INVALID_ARG;
  if (a->freed == a->n_freed) return MOE_DECODE_ERR_INVALID_ARG;
  if (a->recent < 1 || a->sink < 0 || a->keep < 1 ||
      static_cast<int64_t>(a->sink) + a->recent > a->keep)
    return MOE_DECODE_ERR_INVALID_ARG;
  return MOE_DECODE_OK;
}

int moe_decode_cache_plan(const moe_decode_cache_desc* d, int device,
                          moe_decode_cache_plan_t* out) {
  if (!out) return MOE_DECODE_ERR_INVALID_ARG;
  *out = nullptr;
  int rc = moe_decode_cache_desc_check(d);
  if (rc) return rc;
  void* ws = nullptr;
  const size_t bytes = cache_layout(*d, nullptr, nullptr);
  rc = plan_workspace(device, bytes, &ws);
  if (rc) return rc;
  auto* p = new (std::nothrow) moe_decode_cache_plan_s{*d, device, ws, bytes};
  if (!p) {
    free_workspace(device, ws);
    return MOE_DECODE_ERR_NO_MEMORY;
  }
  *out = p;
  return MOE_DECODE_OK;
}

int moe_decode_cache_destroy(moe_decode_cache_plan_t p) {
  if (!p) return MOE_DECODE_OK;
  free_workspace(p->device, p->ws);
  delete p;
  return MOE_DECODE_OK;
}

size_t moe_decode_cache_workspace_bytes(moe_decode_cache_plan_t p) { return p ? p->ws_bytes : 0; }

int moe_decode_cache_append(moe_decode_cache_plan_t p, const moe_decode_append_args* a,
                            int32_t B, int32_t T, void* stream) {
  if (!p) return MOE_DECODE_ERR_INVALID_ARG;
  const int rc = moe_decode_append_check(&p->desc, a, B, T);
  if (rc || B == 0 || T == 0) return rc;
  DeviceScope dev(p->device);
  if (!dev.ok()) return MOE_DECODE_ERR_HIP;
  return status(moe::launch_append(view(p->desc, a->cache, B, T),
                                   static_cast<const uint16_t*>(a->k), a->k_stride,
                                   static_cast<const uint16_t*>(a->v), a->v_stride,
                                   static_cast<hipStream_t>(stream)));
}

int moe_decode_cache_attend(moe_decode_cache_plan_t p, const moe_decode_attend_args* a,
                            int32_t B, int32_t T, void* stream) {
  if (!p) return MOE_DECODE_ERR_INVALID_ARG;
  const int rc = moe_decode_attend_check(&p->desc, a, B, T);
  if (rc || B == 0) return rc;
  DeviceScope dev(p->device);
  if (!dev.ok()) return MOE_DECODE_ERR_HIP;
  moe::AttendArgs k{};
  cache_layout(p->desc, static_cast<char*>(p->ws), &k);
  k.c = view(p->desc, a->cache, B, T);
  k.q = static_cast<const uint16_t*>(a->q);
  k.q_stride = a->q_stride;
  k.out = static_cast<uint16_t*>(a->out);
  k.out_stride = a->out_stride;
  k.scale_log2 = a->sm_scale * 1.44269504088896340736f;
  k.G = p->desc.heads / p->desc.kv_heads;
  k.max_rows = max_rows_of(p->desc);
  k.mass_in = a->mass_in;
  k.mass_out = a->mass_out;
  return status(moe::launch_attend(k, static_cast<hipStream_t>(stream)));
}

int moe_decode_cache_evict(moe_decode_cache_plan_t p, const moe_decode_evict_args* a, int32_t B,
                           void* stream) {
  if (!p) return MOE_DECODE_ERR_INVALID_ARG;
  const int rc = moe_decode_evict_check(&p->desc, a, B);
  if (rc || B == 0) return rc;
  DeviceScope dev(p->device);
  if (!dev.ok()) return MOE_DECODE_ERR_HIP;
  moe::EvictArgs k{};
  k.table = a->page_table;
  k.lens = a->seq_lens;
  k.mass = a->mass;
  k.out_table = a->out_table;
  k.out_lens = a->out_lens;
  k.out_mass = a->out_mass;
  k.freed = a->freed;
  k.n_freed = a->n_freed;
  k.B = B;
  k.max_pages = p->desc.max_pages;
  k.keep = a->keep;
  k.sink = a->sink;
  k.recent = a->recent;
  return status(moe::launch_evict(k, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
