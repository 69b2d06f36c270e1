// serve_api.hip -- the C entry points of the low-bit serving operators:
// argument validation on the host, then the launches.  As in bcq_api.hip every
// check runs before any HIP call.
#include <math.h>
#include <stdint.h>

#include "serve_internal.h"

namespace {

constexpr int32_t kMaxTokens = 1 << 20;
// Work items of a launch are counted in 32 bits: what these limits and those
// below let through stays under 2^24 workgroups of 256.
constexpr int32_t kMaxRows = (1 << 24) - 1;
constexpr int32_t kMaxIntK = 131071;  // 128 * 128 * K stays below 2^31

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t dtype_size(bcq_dtype d) { return d == BCQ_F16 ? 2 : 4; }
bool dtype_valid(bcq_dtype d) { return d == BCQ_F16 || d == BCQ_F32; }
bcq_status hip_status(hipError_t e) { return e == hipSuccess ? BCQ_OK : BCQ_ERR_HIP; }

#define BCQ_TRY(expr)            \
  do {                           \
    bcq_status s_ = (expr);      \
    if (s_ != BCQ_OK) return s_; \
  } while (0)

// Where a linear call keeps the tokens' codes and scales and the K slices' sums.
struct IntWorkspace {
  size_t scales, partial, bytes;
};
IntWorkspace int_workspace(int32_t T, int32_t M, int32_t K) {
  IntWorkspace w;
  w.scales = ((size_t)T * bcq::pad16(K) + 255) / 256 * 256;
  w.partial = w.scales + ((size_t)T * 4 + 255) / 256 * 256;
  w.bytes = w.partial + bcq::int_partial_bytes(T, M, K);
  return w;
}

bcq_status check_int_shape(int32_t T, int32_t M, int32_t K) {
  if (T < 0 || T > kMaxTokens || M < 1 || M > kMaxRows || K < 1 || K > kMaxIntK)
    return BCQ_ERR_INVALID_ARG;
  return BCQ_OK;
}

// The weights and the output, shared by the two products.
bcq_status check_int_product(const int8_t *W, const float *w_scales, int32_t T, int32_t M,
                             int32_t K, int32_t ldw, const void *bias, const void *Y, int32_t ldy,
                             bcq_dtype dtype) {
  BCQ_TRY(check_int_shape(T, M, K));
  if (!dtype_valid(dtype)) return BCQ_ERR_INVALID_ARG;
  if (W == nullptr || w_scales == nullptr || (Y == nullptr && T > 0)) return BCQ_ERR_INVALID_ARG;
  if (ldw < bcq::pad16(K) || ldy < M) return BCQ_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype);
  if (!aligned(W, 16) || ldw % 16 != 0 || !aligned(w_scales, 4) || !aligned(Y, es) ||
      !aligned(bias, es))
    return BCQ_ERR_ALIGNMENT;
  return BCQ_OK;
}

bcq_status check_cache(const bcq_kv_cache *c) {
  if (c == nullptr || c->k_codes == nullptr || c->v_codes == nullptr || c->scales == nullptr ||
      c->page_table == nullptr || c->lens == nullptr)
    return BCQ_ERR_INVALID_ARG;
  if (c->batch < 1 || c->batch > (1 << 16) || c->heads < 1 || c->heads > (1 << 12) ||
      c->num_pages < 1 || c->max_pages < 1)
    return BCQ_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return BCQ_ERR_UNSUPPORTED;
  const int32_t p = c->page_tokens;
  if (p < 16 || p > 256 || (p & (p - 1)) != 0) return BCQ_ERR_UNSUPPORTED;
  if ((int64_t)c->max_pages * p > BCQ_KV_MAX_TOKENS) return BCQ_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)c->batch * c->heads;
  if (rows >= 1 << 22 || rows * c->max_pages * p > (int64_t)1 << 33) return BCQ_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->scales, 16) ||
      !aligned(c->page_table, 4) || !aligned(c->lens, 4))
    return BCQ_ERR_ALIGNMENT;
  return BCQ_OK;
}

bcq::KvView view(const bcq_kv_cache *c) {
  bcq::KvView v;
  v.k = c->k_codes;
  v.v = c->v_codes;
  v.scales = static_cast<uint16_t *>(c->scales);
  v.table = c->page_table;
  v.lens = c->lens;
  v.B = c->batch;
  v.H = c->heads;
  v.page_log = 0;
  while ((1 << v.page_log) < c->page_tokens) ++v.page_log;
  v.num_pages = c->num_pages;
  v.max_pages = c->max_pages;
  return v;
}

int32_t room(const bcq_kv_cache *c) { return c->max_pages * c->page_tokens; }

// K and V of n new tokens, read or written.
bcq_status check_vectors(const bcq_kv_cache *c, int32_t n, const void *k, const void *v,
                         bcq_dtype dtype) {
  BCQ_TRY(check_cache(c));
  if (!dtype_valid(dtype) || n < 0 || n > BCQ_KV_MAX_TOKENS) return BCQ_ERR_INVALID_ARG;
  // a work item takes four channels of K or V, of up to six tokens more than n
  if ((int64_t)c->batch * c->heads * ((int64_t)n + 6) * c->head_dim >= ((int64_t)1 << 33) - 512)
    return BCQ_ERR_INVALID_ARG;
  if (n > 0 && (k == nullptr || v == nullptr)) return BCQ_ERR_INVALID_ARG;
  if (!aligned(k, dtype_size(dtype)) || !aligned(v, dtype_size(dtype))) return BCQ_ERR_ALIGNMENT;
  return BCQ_OK;
}

bcq_status check_attend(const bcq_kv_cache *c, int32_t n, int32_t q_heads) {
  BCQ_TRY(check_cache(c));
  if (n < 0 || n > BCQ_KV_MAX_TOKENS) return BCQ_ERR_INVALID_ARG;
  if (q_heads < 1 || q_heads > (1 << 16) || q_heads % c->heads != 0) return BCQ_ERR_INVALID_ARG;
  // rows are counted in 32 bits
  if ((int64_t)n * q_heads > 1 << 28 || (int64_t)c->batch * n * q_heads > (int64_t)1 << 29)
    return BCQ_ERR_INVALID_ARG;
  return BCQ_OK;
}

}  // namespace

extern "C" {

size_t bcq_int_workspace_bytes(int32_t T, int32_t M, int32_t K) {
  if (check_int_shape(T, M, K) != BCQ_OK || T == 0) return 0;
  return int_workspace(T, M, K).bytes;
}

bcq_status bcq_int_quantize(const void *X, bcq_dtype dtype, int32_t rows, int32_t K, int32_t ldx,
                            int8_t *codes, int32_t ldc, float *scales, hipStream_t stream) {
  if (!dtype_valid(dtype) || rows < 0 || rows > kMaxRows || K < 1 || K > kMaxIntK)
    return BCQ_ERR_INVALID_ARG;
  if (rows == 0) return BCQ_OK;
  if (X == nullptr || codes == nullptr || scales == nullptr) return BCQ_ERR_INVALID_ARG;
  if (ldx < K || ldc < bcq::pad16(K)) return BCQ_ERR_INVALID_ARG;
  if (!aligned(X, 16) || ((size_t)ldx * dtype_size(dtype)) % 16 != 0 || !aligned(codes, 16) ||
      ldc % 16 != 0 || !aligned(scales, 4))
    return BCQ_ERR_ALIGNMENT;
  return hip_status(bcq::launch_int_quantize(X, dtype, rows, K, ldx, codes, ldc, scales, stream));
}

bcq_status bcq_int_gemm(const int8_t *A, const float *a_scales, int32_t T, int32_t lda,
                        const int8_t *W, const float *w_scales, int32_t M, int32_t K, int32_t ldw,
                        const void *bias, void *Y, int32_t ldy, bcq_dtype dtype, void *workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  BCQ_TRY(check_int_product(W, w_scales, T, M, K, ldw, bias, Y, ldy, dtype));
  if (T == 0) return BCQ_OK;
  if (A == nullptr || a_scales == nullptr || lda < bcq::pad16(K)) return BCQ_ERR_INVALID_ARG;
  if (!aligned(A, 16) || lda % 16 != 0 || !aligned(a_scales, 4)) return BCQ_ERR_ALIGNMENT;
  const IntWorkspace w = int_workspace(T, M, K);
  if (workspace == nullptr || workspace_bytes < w.bytes) return BCQ_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return BCQ_ERR_ALIGNMENT;
  const bcq::IntProduct p{A, a_scales, W, w_scales, bias, Y, T, M, K, lda, ldw, ldy};
  return hip_status(bcq::launch_int_gemm(
      p, dtype, reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + w.partial), stream));
}

bcq_status bcq_int_linear(const void *X, int32_t T, int32_t ldx, const int8_t *W,
                          const float *w_scales, int32_t M, int32_t K, int32_t ldw,
                          const void *bias, void *Y, int32_t ldy, bcq_dtype dtype,
                          void *workspace, size_t workspace_bytes, hipStream_t stream) {
  BCQ_TRY(check_int_product(W, w_scales, T, M, K, ldw, bias, Y, ldy, dtype));
  if (T == 0) return BCQ_OK;
  if (X == nullptr || ldx < K) return BCQ_ERR_INVALID_ARG;
  if (!aligned(X, 16) || ((size_t)ldx * dtype_size(dtype)) % 16 != 0) return BCQ_ERR_ALIGNMENT;
  const IntWorkspace w = int_workspace(T, M, K);
  if (workspace == nullptr || workspace_bytes < w.bytes) return BCQ_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return BCQ_ERR_ALIGNMENT;
  char *ws = static_cast<char *>(workspace);
  int8_t *codes = reinterpret_cast<int8_t *>(ws);
  float *scales = reinterpret_cast<float *>(ws + w.scales);
  const int32_t lda = (int32_t)bcq::pad16(K);
  const bcq::IntProduct p{codes, scales, W, w_scales, bias, Y, T, M, K, lda, ldw, ldy};
  if (bcq::int_fused_ok(T, K)) return hip_status(bcq::launch_int_fused(p, X, ldx, dtype, stream));
  hipError_t e = bcq::launch_int_quantize(X, dtype, T, K, ldx, codes, lda, scales, stream);
  if (e != hipSuccess) return BCQ_ERR_HIP;
  return hip_status(
      bcq::launch_int_gemm(p, dtype, reinterpret_cast<int32_t *>(ws + w.partial), stream));
}

bcq_status bcq_kv_append(const bcq_kv_cache *cache, int32_t n, const void *K, int64_t k_batch,
                         int64_t k_token, int64_t k_head, const void *V, int64_t v_batch,
                         int64_t v_token, int64_t v_head, bcq_dtype dtype,
                         const int32_t *positions, float *weights, int32_t *pos,
                         hipStream_t stream) {
  BCQ_TRY(check_vectors(cache, n, K, V, dtype));
  if (!aligned(positions, 4) || !aligned(weights, 4) || !aligned(pos, 4)) return BCQ_ERR_ALIGNMENT;
  if (n == 0) return BCQ_OK;
  return hip_status(bcq::launch_kv_append(view(cache), cache->head_dim, n, K,
                                          {k_batch, k_token, k_head}, V,
                                          {v_batch, v_token, v_head}, dtype, positions, weights,
                                          pos, stream));
}

bcq_status bcq_kv_read(const bcq_kv_cache *cache, int32_t n, void *K, int64_t k_batch,
                       int64_t k_token, int64_t k_head, void *V, int64_t v_batch,
                       int64_t v_token, int64_t v_head, bcq_dtype dtype, hipStream_t stream) {
  BCQ_TRY(check_vectors(cache, n, K, V, dtype));
  if (n == 0) return BCQ_OK;
  return hip_status(bcq::launch_kv_read(view(cache), cache->head_dim, n, K,
                                        {k_batch, k_token, k_head}, V,
                                        {v_batch, v_token, v_head}, dtype, stream));
}

size_t bcq_kv_workspace_bytes(const bcq_kv_cache *cache, int32_t n, int32_t q_heads,
                              int32_t with_weights) {
  if (check_attend(cache, n, q_heads) != BCQ_OK || n == 0) return 0;
  return bcq::attend_plan(cache->batch, cache->heads, cache->head_dim, room(cache), n, q_heads,
                          with_weights != 0)
      .bytes;
}

bcq_status bcq_kv_attend(const bcq_kv_cache *cache, const void *Q, int32_t n, int32_t q_heads,
                         int64_t q_batch, int64_t q_token, int64_t q_head, void *O,
                         int64_t o_batch, int64_t o_token, int64_t o_head, bcq_dtype dtype,
                         float scale, float *weights, void *workspace, size_t workspace_bytes,
                         hipStream_t stream) {
  BCQ_TRY(check_attend(cache, n, q_heads));
  if (!dtype_valid(dtype) || !isfinite(scale)) return BCQ_ERR_INVALID_ARG;
  if (n == 0) return BCQ_OK;
  if (Q == nullptr || O == nullptr) return BCQ_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype);
  if (!aligned(Q, es) || !aligned(O, es) || !aligned(weights, 4)) return BCQ_ERR_ALIGNMENT;
  const size_t need = bcq_kv_workspace_bytes(cache, n, q_heads, weights != nullptr);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return BCQ_ERR_INVALID_ARG;
  if (need > 0 && !aligned(workspace, 16)) return BCQ_ERR_ALIGNMENT;
  bcq::AttendArgs a{};
  a.c = view(cache);
  a.q = Q;
  a.out = O;
  a.qs = {q_batch, q_token, q_head};
  a.os = {o_batch, o_token, o_head};
  a.n = n;
  a.G = q_heads / cache->heads;
  a.q_wide = aligned(Q, 16) && (q_batch * es) % 16 == 0 && (q_token * es) % 16 == 0 &&
             (q_head * es) % 16 == 0;
  a.weights = weights;
  a.ws = workspace;
  return hip_status(bcq::launch_kv_attend(a, scale, cache->head_dim, dtype, stream));
}

size_t bcq_kv_evict_workspace_bytes(const bcq_kv_cache *cache, int32_t keep) {
  if (check_cache(cache) != BCQ_OK || keep < 1) return 0;
  return bcq::evict_workspace_bytes(cache->batch, cache->heads, room(cache), keep);
}

bcq_status bcq_kv_evict(const bcq_kv_cache *cache, int32_t keep, int32_t recent,
                        const float *weights, const int32_t *pos, int32_t *lens_out,
                        float *weights_out, int32_t *pos_out, void *workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  BCQ_TRY(check_cache(cache));
  if (keep < 1 || recent < 0 || recent > keep) return BCQ_ERR_INVALID_ARG;
  if (weights == nullptr || pos == nullptr || lens_out == nullptr || weights_out == nullptr ||
      pos_out == nullptr)
    return BCQ_ERR_INVALID_ARG;
  if (!aligned(weights, 4) || !aligned(pos, 4) || !aligned(lens_out, 4) ||
      !aligned(weights_out, 4) || !aligned(pos_out, 4))
    return BCQ_ERR_ALIGNMENT;
  const size_t need = bcq_kv_evict_workspace_bytes(cache, keep);
  if (workspace == nullptr || workspace_bytes < need) return BCQ_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return BCQ_ERR_ALIGNMENT;
  return hip_status(bcq::launch_kv_evict(view(cache), cache->head_dim, keep, recent, weights, pos,
                                         lens_out, weights_out, pos_out, workspace, stream));
}

}  // extern "C"
