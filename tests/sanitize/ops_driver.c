/*
 * Calls the host-side part of include/moe_decode_ops.h for a build with
 * AddressSanitizer and UndefinedBehaviorSanitizer on the host code: checks at
 * the largest and smallest numbers a caller can pass, and each entry point's
 * rejection of a null plan, all before any device is touched.
 */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "moe_decode_ops.h"

static int bad = 0;
#define EXPECT(expr, want)                                                        \
  do {                                                                            \
    int got_ = (expr);                                                            \
    if (got_ != (want)) {                                                         \
      printf("FAIL %s:%d: %s = %d, want %d\n", __FILE__, __LINE__, #expr, got_,   \
             (int)(want));                                                        \
      bad = 1;                                                                    \
    }                                                                             \
  } while (0)
#define OK MOE_DECODE_OK
#define BAD MOE_DECODE_ERR_INVALID_ARG
#define UNS MOE_DECODE_ERR_UNSUPPORTED

int main(void) {
  char* p = (char*)(uintptr_t)0x10000; /* an aligned address; never read */
  const int32_t edge[] = {INT32_MIN, -1, 0, 1, 127, 128, 65536, 1 << 20, 1 << 24, INT32_MAX};
  const int n = sizeof edge / sizeof edge[0];
  int i, j, k;

  EXPECT(moe_decode_quant(p, INT64_MAX - 7, 1, 128, 0.f, p, p, NULL), UNS);
  EXPECT(moe_decode_quant(p, INT64_MIN, 1, 128, 0.f, p, p, NULL), BAD);
  EXPECT(moe_decode_quant(p, INT32_MAX, INT32_MAX, INT32_MAX, 7.f, p, p, NULL), BAD);
  EXPECT(moe_decode_quant(p, 128, 0, 128, 0.f, p, p, NULL), OK);
  EXPECT(moe_decode_quant(NULL, 128, 1, 128, 0.f, p, p, NULL), BAD);

  for (i = 0; i < n; ++i)
    for (j = 0; j < n; ++j)
      for (k = 0; k < n; ++k) {
        moe_decode_product_desc d;
        moe_decode_product_args a;
        int rc, rc2;
        memset(&d, 0, sizeof d);
        memset(&a, 0, sizeof a);
        d.n = edge[i];
        d.k = edge[j];
        d.max_rows = edge[k];
        rc = moe_decode_product_desc_check(&d);
        if (rc != OK && rc != BAD && rc != UNS) EXPECT(rc, OK);
        a.codes = a.scales = a.w = a.w_scale = p;
        a.out = p;
        a.out_stride = INT64_MAX;
        rc2 = moe_decode_product_args_check(&d, &a, edge[k]);
        if (rc != OK) EXPECT(rc2 == OK, 0);
      }

  for (i = 0; i < n; ++i)
    for (j = 0; j < n; ++j)
      for (k = 0; k < n; ++k) {
        moe_decode_cache_desc d;
        moe_decode_append_args a;
        moe_decode_attend_args t;
        moe_decode_evict_args e;
        int rc;
        memset(&d, 0, sizeof d);
        memset(&a, 0, sizeof a);
        memset(&t, 0, sizeof t);
        memset(&e, 0, sizeof e);
        d.heads = edge[i];
        d.kv_heads = edge[j];
        d.head_dim = 128;
        d.pages = d.max_pages = edge[k];
        d.max_batch = d.max_q = 1;
        d.with_mass = 1;
        rc = moe_decode_cache_desc_check(&d);
        if (rc != OK && rc != BAD && rc != UNS) EXPECT(rc, OK);
        a.cache.pool = a.cache.pool_scale = p;
        a.cache.page_table = a.cache.seq_lens = a.cache.q_start = (const int32_t*)p;
        a.k = a.v = p;
        a.k_stride = a.v_stride = INT64_MAX - 7;
        t.cache = a.cache;
        t.q = p;
        t.out = p + 64;
        t.q_stride = t.out_stride = INT64_MIN;
        e.page_table = e.seq_lens = (const int32_t*)p;
        e.mass = (const float*)p;
        e.out_table = e.out_lens = e.freed = e.n_freed = (int32_t*)p;
        e.out_mass = (float*)p;
        e.keep = edge[i];
        e.sink = edge[j];
        e.recent = edge[k];
        if (rc != OK) EXPECT(moe_decode_append_check(&d, &a, 1, edge[k]) == OK, 0);
        EXPECT(moe_decode_attend_check(&d, &t, 1, edge[k]) == OK, 0);
        moe_decode_evict_check(&d, &e, 1);
        (void)moe_decode_append_check(&d, &a, edge[i], edge[j]);
      }

  EXPECT(moe_decode_product_desc_check(NULL), BAD);
  EXPECT(moe_decode_cache_desc_check(NULL), BAD);
  EXPECT(moe_decode_product_run(NULL, NULL, 1, NULL), BAD);
  EXPECT(moe_decode_cache_append(NULL, NULL, 1, 1, NULL), BAD);
  EXPECT(moe_decode_cache_attend(NULL, NULL, 1, 1, NULL), BAD);
  EXPECT(moe_decode_cache_evict(NULL, NULL, 1, NULL), BAD);
  EXPECT(moe_decode_product_destroy(NULL), OK);
  EXPECT(moe_decode_cache_destroy(NULL), OK);
  EXPECT((int)moe_decode_product_workspace_bytes(NULL), 0);
  EXPECT((int)moe_decode_cache_workspace_bytes(NULL), 0);
  if (!bad) printf("ops checks: ok\n");
  return bad;
}
