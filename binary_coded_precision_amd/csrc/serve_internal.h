// serve_internal.h -- declarations shared by the low-bit serving operators
// (8-bit integer products, the norm before them, and the 4-bit key/value cache).
// Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bcq.h"

namespace bcq {

// ---- 8-bit integer products (int_gemm.hip) ----

inline int64_t pad16(int64_t k) { return (k + 15) / 16 * 16; }

hipError_t launch_int_quantize(const void *X, bcq_dtype dt, int rows, int K, int ldx,
                               int8_t *codes, int ldc, float *scales, hipStream_t s);
struct IntProduct {
  const int8_t *a;       // [T][lda] token codes, zero from K to the next multiple of 16
  const float *a_scale;  // [T]
  const int8_t *w;       // [M][ldw]
  const float *w_scale;  // [M]
  const void *bias;      // [M] of the output type, or null
  void *y;               // [T][ldy]
  int T, M, K, lda, ldw, ldy;
};
// int32 partial sums of the K slices, 0 when K is not split.
size_t int_partial_bytes(int T, int M, int K);
hipError_t launch_int_gemm(const IntProduct &p, bcq_dtype dt, int32_t *partial, hipStream_t s);
// Few tokens: one launch quantizes the tokens and multiplies (see int_gemm.hip).
bool int_fused_ok(int T, int K);
hipError_t launch_int_fused(const IntProduct &p, const void *X, int ldx, bcq_dtype dt,
                            hipStream_t s);

// ---- norm (norm.hip) ----

struct NormArgs {
  const void *x, *residual, *gamma;  // residual may be null
  void *h, *y;                       // may be null; h may be x or residual
  int8_t *codes;                     // may be null, then scales is too
  float *scales;
  int64_t ldx, ldr, ldh, ldy, ldc;
  int K;
  double eps;
};
hipError_t launch_rms_norm(const NormArgs &a, int T, bcq_dtype dt, hipStream_t s);

// ---- 4-bit key/value cache ----

// The cache as the kernels see it: page_tokens = 1 << page_log.
struct KvView {
  uint8_t *k, *v;
  uint16_t *scales;
  const int32_t *table;
  const int32_t *lens;
  int B, H, page_log, num_pages, max_pages;
  __host__ __device__ int room() const { return max_pages << page_log; }
};

struct KvStrides {
  int64_t batch, token, head;  // elements
};

hipError_t launch_kv_append(const KvView &c, int D, int n, const void *k, KvStrides ks,
                            const void *v, KvStrides vs, bcq_dtype dt, const int32_t *positions,
                            float *weights, int32_t *pos, hipStream_t s);
hipError_t launch_kv_read(const KvView &c, int D, int n, void *k, KvStrides ks, void *v,
                          KvStrides vs, bcq_dtype dt, hipStream_t s);

// The same for n packed tokens, each in a slot (a place among all the pages'
// tokens); those in no page's are not there.
hipError_t launch_kv_append_slots(const KvView &c, int D, int n, const int64_t *slots,
                                  const void *k, KvStrides ks, const void *v, KvStrides vs,
                                  bcq_dtype dt, hipStream_t s);
hipError_t launch_kv_read_slots(const KvView &c, int D, int n, const int64_t *slots, void *k,
                                KvStrides ks, void *v, KvStrides vs, bcq_dtype dt, hipStream_t s);

// Pages given and taken back (kv_reserve.hip); see bcq_kv_reserve.
struct ReserveCall {
  const int32_t *new_tokens, *release, *free_pages, *free_count;
  int32_t *lens_out, *table_out, *free_out, *count_out, *starts, *positions;
  int64_t *slots;
  int shared_pages, T;
};
size_t reserve_workspace_bytes(int B, int max_pages);
hipError_t launch_kv_reserve(const KvView &c, const ReserveCall &r, void *ws, hipStream_t s);

// How a call of the attention is laid out; host arithmetic on shapes only, so
// that the workspace's size and the launch agree.
struct AttendPlan {
  int ct;          // 16-row tiles a wave holds
  int wt;          // waves of a workgroup that share its rows and take turns over the tokens
  int row_blocks;  // workgroups over a cached head's rows
  int splits;      // workgroups over the tokens
  bool scores;     // the weights are summed from stored scores, not from recomputed ones
  size_t off_o, off_scores, bytes;  // workspace: (m, l) pairs, then outputs, then scores
};
AttendPlan attend_plan(int B, int H, int D, int room, int n, int q_heads, bool weights);

struct AttendArgs {
  KvView c;
  const void *q;
  void *out;
  KvStrides qs, os;
  int n, G;          // queries of a sequence; query heads of a cached head
  bool q_wide;       // 8 channels of q can be read at once
  float unit;        // the softmax's scale times log2(e)
  float code_unit;   // that times 2^20, in fp16 calls
  float *weights;    // [B][H][room] or null
  void *ws;
};
// unit and code_unit of `call` are filled in from the softmax's scale.
hipError_t launch_kv_attend(const AttendArgs &call, float scale, int D, bcq_dtype dt,
                            hipStream_t s);

// Attention of packed tokens (kv_packed.hip); see bcq_kv_attend_packed.
struct PackedCall {
  KvView c;
  const void *q;
  void *out;
  KvStrides qs, os;  // token and head
  const int32_t *starts;
  int T, q_heads, max_n, shared;  // shared: tokens of the shared pages
  bool q_wide;                    // 8 channels of q can be read at once
  void *ws;
};
// 0 where the call has more rows than are counted.
size_t packed_workspace_bytes(int B, int H, int D, int room, int T, int q_heads, int max_n,
                              bool shared);
hipError_t launch_kv_attend_packed(const PackedCall &call, float scale, int D, bcq_dtype dt,
                                   hipStream_t s);

size_t evict_workspace_bytes(int B, int H, int room, int keep);
hipError_t launch_kv_evict(const KvView &c, int D, int keep, int recent, const float *weights,
                           const int32_t *pos, int32_t *lens_out, float *weights_out,
                           int32_t *pos_out, void *ws, hipStream_t s);

// ---- device helpers of the cache's kernels ----

// Length of sequence b, held to what its table has room for.
__device__ __forceinline__ int kv_len(const KvView &c, int b) {
  const int L = c.lens[b];
  return L < 0 ? 0 : (L > c.room() ? c.room() : L);
}

// Token index within all the pages of cached head h for slot `tok` of sequence
// b (an index times D/2 is the byte of its K codes, times 8 that of its
// scales), or -1 where the table's entry names no page.
__device__ __forceinline__ int64_t kv_token(const KvView &c, int b, int h, int tok) {
  const int page = c.table[(int64_t)b * c.max_pages + (tok >> c.page_log)];
  if ((unsigned)page >= (unsigned)c.num_pages) return -1;
  return (((int64_t)page * c.H + h) << c.page_log) + (tok & ((1 << c.page_log) - 1));
}

}  // namespace bcq
