// Argument validation of the norm and of the packed serving step's operators, built with the host
// sanitizers: every call is rejected, or has nothing to do, before any HIP call.  Sizes at the ends
// of the integer types are among them, where a count held in too few bits would overflow.
#include <limits.h>
#include <math.h>
#include <stdio.h>

#include "bcq.h"

static int failures = 0;

static void expect(const char *what, long long got, long long want) {
  if (got == want) return;
  printf("FAIL %s: %lld, expected %lld\n", what, got, want);
  ++failures;
}

alignas(64) static char memory[64];

static bcq_kv_cache cache(int32_t batch, int32_t heads, int32_t page, int32_t num_pages,
                          int32_t max_pages) {
  uint8_t *p = reinterpret_cast<uint8_t *>(memory);
  const int32_t *t = reinterpret_cast<const int32_t *>(memory);
  return bcq_kv_cache{batch, heads, 128, page, num_pages, max_pages, p, p, p, t, t};
}

int main() {
  void *x = memory;
  int8_t *c = reinterpret_cast<int8_t *>(memory);
  float *f = reinterpret_cast<float *>(memory);
  int32_t *n = reinterpret_cast<int32_t *>(memory);
  int64_t *w = reinterpret_cast<int64_t *>(memory);
  const int32_t ends[] = {INT_MIN, INT_MIN + 1, -1, 0, INT_MAX - 15, INT_MAX};
  const bcq_kv_cache ok = cache(2, 2, 64, 8, 4);

  for (int32_t v : ends) {
    expect("norm K",
           bcq_rms_norm(x, 64, x, 64, x, 1e-5, 2, v, BCQ_F16, x, 64, x, 64, c, 64, f, nullptr),
           BCQ_ERR_INVALID_ARG);
    if (v != 0)
      expect("norm T",
             bcq_rms_norm(x, 64, x, 64, x, 1e-5, v, 64, BCQ_F16, x, 64, x, 64, c, 64, f, nullptr),
             BCQ_ERR_INVALID_ARG);
    if (v < 64) {
      for (int i = 0; i < 5; ++i)
        expect("norm leading dimension",
               bcq_rms_norm(x, i == 0 ? v : 64, x, i == 1 ? v : 64, x, 1e-5, 2, 64, BCQ_F16, x,
                            i == 2 ? v : 64, x, i == 3 ? v : 64, c, i == 4 ? v : 64, f, nullptr),
               BCQ_ERR_INVALID_ARG);
    }
    bcq_kv_cache bad[] = {cache(v, 2, 64, 8, 4), cache(2, v, 64, 8, 4), cache(2, 2, v, 8, 4),
                          cache(2, 2, 64, 8, v)};
    for (int i = 0; i < 4; ++i) {
      const bcq_status want = i == 2 ? BCQ_ERR_UNSUPPORTED : BCQ_ERR_INVALID_ARG;
      expect("append slots cache",
             bcq_kv_append_slots(&bad[i], 1, w, x, 1, 1, x, 1, 1, BCQ_F16, nullptr), want);
      expect("reserve cache",
             bcq_kv_reserve(&bad[i], n, n, 0, n, n, 1, n, n, n, n, n, w, n, x, SIZE_MAX, nullptr),
             want);
      expect("attend cache",
             bcq_kv_attend_packed(&bad[i], x, 1, 4, 1, 1, n, 1, 0, x, 1, 1, BCQ_F16, 1.f, x,
                                  SIZE_MAX, nullptr),
             want);
      expect("reserve workspace", bcq_kv_reserve_workspace_bytes(&bad[i]), 0);
      expect("attend workspace", bcq_kv_packed_workspace_bytes(&bad[i], 1, 4, 1, 0), 0);
    }
    if (v != 0) {
      expect("read slots T",
             bcq_kv_read_slots(&ok, v, w, x, INT64_MAX, INT64_MIN, x, 1, 1, BCQ_F32, nullptr),
             BCQ_ERR_INVALID_ARG);
      expect("reserve T",
             bcq_kv_reserve(&ok, n, n, 0, n, n, v, n, n, n, n, n, w, n, x, SIZE_MAX, nullptr),
             BCQ_ERR_INVALID_ARG);
      expect("reserve shared",
             bcq_kv_reserve(&ok, n, n, v, n, n, 1, n, n, n, n, n, w, n, x, SIZE_MAX, nullptr),
             BCQ_ERR_INVALID_ARG);
      expect("attend T",
             bcq_kv_attend_packed(&ok, x, v, 4, 1, 1, n, 1, 0, x, 1, 1, BCQ_F16, 1.f, x, SIZE_MAX,
                                  nullptr),
             BCQ_ERR_INVALID_ARG);
      expect("attend shared", bcq_kv_packed_workspace_bytes(&ok, 1, 4, 1, v), 0);
    }
    expect("attend heads", bcq_kv_packed_workspace_bytes(&ok, 1, v, 1, 0), 0);
    if (v <= 0) expect("attend max_n", bcq_kv_packed_workspace_bytes(&ok, 1, 4, v, 0), 0);
  }
  expect("attend max_n past T", bcq_kv_packed_workspace_bytes(&ok, 3, 4, INT_MAX, 0),
         bcq_kv_packed_workspace_bytes(&ok, 3, 4, 3, 0));

  // nothing to do
  expect("no rows",
         bcq_rms_norm(nullptr, 64, nullptr, 64, nullptr, 1e-5, 0, 64, BCQ_F16, nullptr, 64, nullptr,
                      64, nullptr, 64, nullptr, nullptr),
         BCQ_OK);
  expect("no slots",
         bcq_kv_append_slots(&ok, 0, nullptr, nullptr, 1, 1, nullptr, 1, 1, BCQ_F16, nullptr),
         BCQ_OK);
  expect("no queries",
         bcq_kv_attend_packed(&ok, nullptr, 0, 4, 1, 1, nullptr, 0, 0, nullptr, 1, 1, BCQ_F16, 1.f,
                              nullptr, 0, nullptr),
         BCQ_OK);

  // values and counts at their limits
  for (double eps : {0., -1., (double)INFINITY, (double)NAN, 1e300, 1e-300})
    expect("eps",
           bcq_rms_norm(x, 64, x, 64, x, eps, 2, 64, BCQ_F16, x, 64, x, 64, c, 64, f, nullptr),
           BCQ_ERR_INVALID_ARG);
  for (float scale : {INFINITY, -INFINITY, NAN})
    expect("scale",
           bcq_kv_attend_packed(&ok, x, 1, 4, 1, 1, n, 1, 0, x, 1, 1, BCQ_F16, scale, x, SIZE_MAX,
                                nullptr),
           BCQ_ERR_INVALID_ARG);
  // the most of everything at once: sizes that stay in their types, or a refusal
  const bcq_kv_cache wide = cache(1 << 12, 8, 256, INT_MAX, 1 << 10);
  if (bcq_kv_reserve_workspace_bytes(&wide) < (size_t)1 << 24)
    expect("pages of a wide cache", 0, 1);
  expect("vectors of a wide cache",
         bcq_kv_append_slots(&wide, 1 << 24, w, x, 1, 1, x, 1, 1, BCQ_F16, nullptr),
         BCQ_ERR_INVALID_ARG);
  if (bcq_kv_packed_workspace_bytes(&wide, 1 << 22, 64, 1 << 22, 1) < (size_t)1 << 36)
    expect("rows of a wide cache", 0, 1);
  const bcq_kv_cache deep = cache(2, 1, 256, INT_MAX, 1 << 16);
  for (int32_t heads : {1, 16, 1 << 16})
    for (int32_t T : {1, 1 << 12, 1 << 24})
      for (int32_t shared : {0, 1 << 16})
        bcq_kv_packed_workspace_bytes(&deep, T, heads, T, shared);
  expect("more rows than are counted",
         bcq_kv_packed_workspace_bytes(&deep, 1 << 22, 64, 1 << 22, 0), 0);
  const bcq_kv_cache many = cache((1 << 12) + 1, 2, 64, 8, 4);
  expect("more sequences than are planned", bcq_kv_packed_workspace_bytes(&many, 1, 4, 1, 0), 0);

  printf("%d failures\n", failures);
  return failures;
}
