// Argument validation of the low-bit serving operators, built with the host sanitizers: every
// call is rejected, or has nothing to do, before any HIP call.  Sizes at the ends of the integer
// types are among them, where a count held in too few bits would overflow.
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
  const int32_t ends[] = {INT_MIN, INT_MIN + 1, -1, 0, INT_MAX - 15, INT_MAX};

  for (int32_t v : ends) {
    expect("int workspace T", bcq_int_workspace_bytes(v, 64, 64), 0);
    expect("int workspace M", bcq_int_workspace_bytes(64, v, 64), 0);
    expect("int workspace K", bcq_int_workspace_bytes(64, 64, v), 0);
    expect("quantize K", bcq_int_quantize(x, BCQ_F16, 2, v, 64, c, 64, f, nullptr),
           BCQ_ERR_INVALID_ARG);
    expect("linear M",
           bcq_int_linear(x, 2, 64, c, f, v, 64, 64, nullptr, x, 64, BCQ_F16, x, SIZE_MAX, nullptr),
           BCQ_ERR_INVALID_ARG);
    expect("gemm K",
           bcq_int_gemm(c, f, 2, 64, c, f, 64, v, 64, nullptr, x, 64, BCQ_F16, x, SIZE_MAX, nullptr),
           BCQ_ERR_INVALID_ARG);
    if (v != 0) {
      expect("quantize rows", bcq_int_quantize(x, BCQ_F16, v, 64, 64, c, 64, f, nullptr),
             BCQ_ERR_INVALID_ARG);
      expect("linear T",
             bcq_int_linear(x, v, 64, c, f, 64, 64, 64, nullptr, x, 64, BCQ_F16, x, SIZE_MAX,
                            nullptr),
             BCQ_ERR_INVALID_ARG);
    }
    if (v < 64) {
      expect("quantize ldx", bcq_int_quantize(x, BCQ_F16, 2, 64, v, c, 64, f, nullptr),
             BCQ_ERR_INVALID_ARG);
      expect("linear ldy",
             bcq_int_linear(x, 2, 64, c, f, 64, 64, 64, nullptr, x, v, BCQ_F16, x, SIZE_MAX,
                            nullptr),
             BCQ_ERR_INVALID_ARG);
    }
    bcq_kv_cache bad[] = {cache(v, 2, 64, 8, 4), cache(2, v, 64, 8, 4), cache(2, 2, v, 8, 4),
                          cache(2, 2, 64, 8, v)};
    for (int i = 0; i < 4; ++i) {
      const bcq_status want = i == 2 ? BCQ_ERR_UNSUPPORTED : BCQ_ERR_INVALID_ARG;
      expect("append cache",
             bcq_kv_append(&bad[i], 1, x, 1, 1, 1, x, 1, 1, 1, BCQ_F16, nullptr, nullptr, nullptr,
                           nullptr),
             want);
      expect("attend cache",
             bcq_kv_attend(&bad[i], x, 1, 4, 1, 1, 1, x, 1, 1, 1, BCQ_F16, 1.f, f, x, SIZE_MAX,
                           nullptr),
             want);
      expect("evict cache",
             bcq_kv_evict(&bad[i], 16, 4, f, n, n, f, n, x, SIZE_MAX, nullptr), want);
      expect("kv workspace", bcq_kv_workspace_bytes(&bad[i], 1, 4, 1), 0);
      expect("evict workspace", bcq_kv_evict_workspace_bytes(&bad[i], 16), 0);
    }
    bcq_kv_cache ok = cache(2, 2, 64, 8, 4);
    if (v != 0) {
      expect("read n",
             bcq_kv_read(&ok, v, x, INT64_MAX, INT64_MIN, 1, x, 1, 1, 1, BCQ_F32, nullptr),
             BCQ_ERR_INVALID_ARG);
      expect("attend n",
             bcq_kv_attend(&ok, x, v, 4, 1, 1, 1, x, 1, 1, 1, BCQ_F16, 1.f, f, x, SIZE_MAX, nullptr),
             BCQ_ERR_INVALID_ARG);
    }
    expect("attend heads", bcq_kv_workspace_bytes(&ok, 1, v, 1), 0);
    if (v <= 0)
      expect("keep", bcq_kv_evict(&ok, v, 0, f, n, n, f, n, x, SIZE_MAX, nullptr),
             BCQ_ERR_INVALID_ARG);
    if (v != 0)
      expect("recent", bcq_kv_evict(&ok, 16, v, f, n, n, f, n, x, SIZE_MAX, nullptr),
             BCQ_ERR_INVALID_ARG);
  }

  // nothing to do
  expect("no rows", bcq_int_quantize(nullptr, BCQ_F16, 0, 64, 64, nullptr, 64, nullptr, nullptr),
         BCQ_OK);
  expect("no tokens",
         bcq_int_linear(nullptr, 0, 64, c, f, 64, 64, 64, nullptr, nullptr, 64, BCQ_F16, nullptr, 0,
                        nullptr),
         BCQ_OK);
  bcq_kv_cache ok = cache(2, 2, 64, 8, 4);
  expect("no vectors",
         bcq_kv_append(&ok, 0, nullptr, 1, 1, 1, nullptr, 1, 1, 1, BCQ_F16, nullptr, nullptr,
                       nullptr, nullptr),
         BCQ_OK);
  expect("no queries",
         bcq_kv_attend(&ok, nullptr, 0, 4, 1, 1, 1, nullptr, 1, 1, 1, BCQ_F16, 1.f, nullptr,
                       nullptr, 0, nullptr),
         BCQ_OK);

  // scales and counts at their limits
  expect("scale inf",
         bcq_kv_attend(&ok, x, 1, 4, 1, 1, 1, x, 1, 1, 1, BCQ_F16, INFINITY, nullptr, x, SIZE_MAX,
                       nullptr),
         BCQ_ERR_INVALID_ARG);
  const bcq_kv_cache huge = cache(1 << 16, 1 << 12, 256, INT_MAX, 1 << 16);
  expect("rows of a huge cache", bcq_kv_evict_workspace_bytes(&huge, 1 << 23), 0);
  expect("scores of a huge cache", bcq_kv_workspace_bytes(&huge, 1, 1 << 12, 1), 0);
  const bcq_kv_cache wide = cache(1 << 12, 8, 256, INT_MAX, 1 << 10);
  expect("vectors of a wide cache",
         bcq_kv_append(&wide, 1 << 24, x, 1, 1, 1, x, 1, 1, 1, BCQ_F16, nullptr, nullptr, nullptr,
                       nullptr),
         BCQ_ERR_INVALID_ARG);
  expect("rows of a wide cache", bcq_kv_workspace_bytes(&wide, 1 << 24, 1 << 12, 1), 0);
  if (bcq_kv_evict_workspace_bytes(&wide, 1 << 17) < (size_t)1 << 34)
    expect("moves of a wide cache", 0, 1);
  if (bcq_kv_workspace_bytes(&wide, 1, 64, 1) < (size_t)1 << 38)
    expect("scores of a wide cache", 0, 1);
  if (bcq_int_workspace_bytes(1 << 20, (1 << 24) - 1, 131071) < (size_t)1 << 37)
    expect("codes of the largest product", 0, 1);

  printf("%d failures\n", failures);
  return failures;
}
