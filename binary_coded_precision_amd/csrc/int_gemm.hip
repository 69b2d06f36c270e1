// int_gemm.hip -- the 8-bit integer linear layer (bcq_int_quantize,
// bcq_int_gemm, bcq_int_linear).
//
//   code = rint(x / s),  s = max|x| * (1/127) for each token (row of X)
//   y[t][m] = (sum_k a[t][k] w[m][k]) * (a_scale[t] * w_scale[m]) + bias[m]
//
// The sum is exact in int32 (K <= 131071), so neither the order of K nor a
// split of it changes a result; the scales are applied once, in fp32.
#include "serve_internal.h"

namespace bcq {
namespace {

typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int16v __attribute__((ext_vector_type(16)));

// 16 bytes of nothing for the chunks past the end of K.
__device__ const uint4 kZeros = {0, 0, 0, 0};

__device__ __forceinline__ float nan_max(float a, float b) { return (a > b || a != a) ? a : b; }

// 8 consecutive elements from a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void load8(float (&x)[8], const T *p) {
  if constexpr (sizeof(T) == 2) {
    typedef _Float16 half8 __attribute__((ext_vector_type(8)));
    const half8 h = *reinterpret_cast<const half8 *>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)h[e];
  } else {
    const float4 a = reinterpret_cast<const float4 *>(p)[0];
    const float4 b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}

// Elements k..k+7 of a row of K, zeros past its end; nothing past K is read.
template <typename T>
__device__ __forceinline__ void load_row8(float (&x)[8], const T *row, int k, int K) {
  if (k + 8 <= K) {
    load8(x, row + k);
  } else if (k >= K) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = k + e < K ? (float)row[k + e] : 0.f;
  }
}

// Codes of eight elements.  The quotient's neighbour x * (1/s), at most 5e-5 off
// it, rounds to the same integer unless it lies that close to a half; only then
// is the division done.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s) {
  const bool some = s > 0.f && s < INFINITY;
  const float inv = some ? 1.f / s : 0.f;
  float q[8];
  bool near = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = x[e] * inv;
    q[e] = rintf(y);
    near |= !(fabsf(y - q[e]) < 0.4999f);
  }
  if (__builtin_expect(near, 0) && some) {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = rintf(x[e] / s);
  }
  uint32_t c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    c[e] = some ? (uint32_t)(int)fminf(fmaxf(q[e], -127.f), 127.f) & 255u : 0u;
  return make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
                    c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
}

// A row's scale; NaN for a row that holds an infinity or NaN (its codes are 0),
// so that its products are NaN.
__device__ __forceinline__ float row_scale(float top) {
  return top < INFINITY ? top * (1.f / 127.f) : NAN;
}

// One workgroup a row.  Rows of up to 2048 N elements are held in registers
// between the two passes, longer ones (N = 0) read again from the caches.  Bound
// by memory and, at a row a workgroup, by the two passes' latency: 4096 rows of
// 4096 fp16 take 16.7 us (50 MB, 3.0 TB/s), in fp32 25.6 us (84 MB, 3.3 TB/s); a
// wave a row, four rows a workgroup, took 20.6 us in fp16.
template <typename T, int N>
__global__ __launch_bounds__(256) void quantize_kernel(const T *X, int K, int ldx, int8_t *codes,
                                                       int ldc, float *scales) {
  __shared__ float red[4];
  const T *x = X + (int64_t)blockIdx.x * ldx;
  const int tid = threadIdx.x;
  float v[N > 0 ? N : 1][8], top = 0.f;
  if constexpr (N > 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) load_row8(v[n], x, (n * 256 + tid) * 8, K);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = nan_max(top, fabsf(v[n][e]));
  } else {
    for (int k = tid * 8; k < K; k += 256 * 8) {
      load_row8(v[0], x, k, K);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = nan_max(top, fabsf(v[0][e]));
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = nan_max(top, __shfl_xor(top, d));
  if ((tid & 63) == 0) red[tid >> 6] = top;
  __syncthreads();
  top = nan_max(nan_max(red[0], red[1]), nan_max(red[2], red[3]));
  const float s = row_scale(top);
  if (tid == 0) scales[blockIdx.x] = s;
  int8_t *c = codes + (int64_t)blockIdx.x * ldc;
  const int end = (K + 15) / 16 * 16;  // zeros up to the next 16 bytes
  if constexpr (N > 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int k = (n * 256 + tid) * 8;
      if (k < end) *reinterpret_cast<uint2 *>(c + k) = codes8(v[n], s);
    }
  } else {
    for (int k = tid * 8; k < end; k += 256 * 8) {
      load_row8(v[0], x, k, K);
      *reinterpret_cast<uint2 *>(c + k) = codes8(v[0], s);
    }
  }
}

template <typename T>
struct __attribute__((aligned(4 * sizeof(T)))) Four {
  T x[4];
};

// Four outputs of token t from row m on: their scales and biases, from their exact sums.
struct RowFactors {
  float scale[4], bias[4];
};
template <typename T>
__device__ __forceinline__ RowFactors row_factors(const IntProduct &p, int m) {
  RowFactors f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int mm = min(m + e, p.M - 1);
    f.scale[e] = p.w_scale[mm];
    f.bias[e] = p.bias != nullptr ? (float)static_cast<const T *>(p.bias)[mm] : 0.f;
  }
  return f;
}
template <typename T>
__device__ __forceinline__ Four<T> finish(const RowFactors &f, float a_scale, const int (&acc)[4]) {
  Four<T> y;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    y.x[e] = (T)fmaf((float)acc[e], a_scale * f.scale[e], f.bias[e]);
  return y;
}
template <typename T>
__device__ __forceinline__ void store_y(const IntProduct &p, int t, int m, const Four<T> &v) {
  T *y = static_cast<T *>(p.y) + (int64_t)t * p.ldy + m;
  if (m + 4 <= p.M && ((uintptr_t)y & (4 * sizeof(T) - 1)) == 0) {
    *reinterpret_cast<Four<T> *>(y) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m + e < p.M) y[e] = v.x[e];
  }
}

// Sums of rows m..m+3 of one token of a slice.
__device__ __forceinline__ void store_sums(int32_t *token, int m, int M, int4v s) {
  int32_t *o = token + m;
  if (m + 4 <= M && (M & 3) == 0) {
    *reinterpret_cast<int4v *>(o) = s;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m + e < M) o[e] = s[e];
  }
}

// ---- few tokens: one launch
//
// 16 rows of W a workgroup, its four waves taking turns over K in steps of 128
// bytes; W goes from memory to the matrix operands without passing through
// shared memory, and a wave has up to eight steps (16 KB) in flight, asked for
// before the tokens are quantized.  Every workgroup quantizes the tokens for
// itself: T * K is at most kFusedElements, a fraction of a microsecond, where a
// launch of its own costs several.  One token by 4096 x 4096 (16.8 MB) takes
// 8.3 us, the chain from a token's first load to its codes among them; reading the
// weights alone would take 3.3 us.
//
// Up to two tokens: each one more costs every workgroup 1.7 us of loads, extremes
// and codes one after the other, and the two launches of the way below cost 3 (us
// in a graph, by 4096 x 4096: one token 8.0 against 11.2, two 9.6 against 11.8,
// three 11.5 each, four 12.8 against 11.8; eight by 4096 x 1024 11.5 against 6.3).
constexpr int kFusedTokens = 2, kFusedElements = 16384;
constexpr int kFusedDepth = 8;  // steps in flight

template <typename T>
__global__ __launch_bounds__(256) void fused_kernel(IntProduct p, const T *X, int ldx) {
  extern __shared__ __align__(16) int8_t xs[];  // [T][row]
  __shared__ float red[kFusedTokens][4];
  __shared__ int4v part[4][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int m0 = blockIdx.x * 16;
  const int K16 = (p.K + 15) / 16 * 16, steps = (p.K + 127) / 128;
  const int row = steps * 128 + 16;  // 16 past a multiple of 128: rows start in other banks
  const int8_t *w = p.w + (int64_t)min(m0 + r, p.M - 1) * p.ldw + g * 32;

  // the first elements of the first token, ahead of the flood of weights
  constexpr int kHeld = 2;
  float held[kHeld][8];
#pragma unroll
  for (int n = 0; n < kHeld; ++n) load_row8(held[n], X, (n * 256 + tid) * 8, p.K);
  int4v wf[kFusedDepth][2];
  auto fetch = [&](int4v(&f)[2], int step) {
    const int k = step * 128 + g * 32;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      f[e] = k + 16 * e < K16 ? *reinterpret_cast<const int4v *>(w + (int64_t)step * 128 + 16 * e)
                              : int4v{0, 0, 0, 0};
  };
#pragma unroll
  for (int d = 0; d < kFusedDepth; ++d)
    if (wave + 4 * d < steps) fetch(wf[d], wave + 4 * d);

  auto values = [&](float(&v)[8], int t, int n) {
    if (t == 0 && n < kHeld) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = n == 0 ? held[0][e] : held[1][e];
    } else {
      load_row8(v, X + (int64_t)t * ldx, (n * 256 + tid) * 8, p.K);
    }
  };
  const int parts = (p.K + 2047) / 2048;
  for (int t = 0; t < p.T; ++t) {
    float v[8], top = 0.f;
    for (int n = 0; n < parts; ++n) {
      values(v, t, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = nan_max(top, fabsf(v[e]));
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = nan_max(top, __shfl_xor(top, d));
    if (lane == 0) red[t][wave] = top;
  }
  __syncthreads();
  for (int t = 0; t < p.T; ++t) {
    const float s =
        row_scale(nan_max(nan_max(red[t][0], red[t][1]), nan_max(red[t][2], red[t][3])));
    float v[8];
    for (int n = 0; n < parts; ++n) {
      const int k = (n * 256 + tid) * 8;
      if (k >= steps * 128) break;
      values(v, t, n);
      *reinterpret_cast<uint2 *>(xs + t * row + k) = codes8(v, s);
    }
  }
  __syncthreads();

  int4v acc = {0, 0, 0, 0};
  const int8_t *xr = xs + min(r, p.T - 1) * row + g * 32;
  for (int step = wave; step < steps; step += 4 * kFusedDepth) {
#pragma unroll
    for (int d = 0; d < kFusedDepth; ++d) {
      const int st = step + 4 * d;
      if (st < steps) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
              wf[d][e], *reinterpret_cast<const int4v *>(xr + st * 128 + 16 * e), acc, 0, 0, 0);
        if (st + 4 * kFusedDepth < steps) fetch(wf[d], st + 4 * kFusedDepth);
      }
    }
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave == 0 && r < p.T) {
    int sum[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      sum[e] = part[0][lane][e] + part[1][lane][e] + part[2][lane][e] + part[3][lane][e];
    const float s =
        row_scale(nan_max(nan_max(red[r][0], red[r][1]), nan_max(red[r][2], red[r][3])));
    const int m = m0 + 4 * g;
    if (m < p.M) store_y<T>(p, r, m, finish<T>(row_factors<T>(p, m), s, sum));
  }
}

// ---- up to 64 tokens
//
// Bound by reading W once.  32 rows of W by all the tokens a workgroup; its four
// waves share a step's four products of 32 bytes of K between them, one each, and
// add up at the end.  Shared memory holds a ring of kRing steps that memory fills
// directly, so that a compute unit's two or three workgroups have 30 KB of W and
// more in flight; a step waits for its own loads only (loads return in order),
// and loads past the end of K come from 16 bytes of zeros, which keeps the count
// the same.  37 tokens by 14336 x 4096 (58.7 MB) take 15.0 us, 3.9 TB/s.
constexpr int kRing = 5;

template <typename T, int BT, bool SPLIT>
__global__ __launch_bounds__(256) void few_kernel(IntProduct p, int tiles_m, int slice_steps,
                                                  int32_t *partial) {
  constexpr int BM = 32, kT = BT / 32;
  constexpr int kLoads = (BM + BT) / 8 / 4;  // of 1 KB, a wave and step
  constexpr int kStage = (BM + BT) * 128;
  __shared__ __align__(16) int8_t lds[kRing][kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slice = SPLIT ? blockIdx.x / tiles_m : 0;
  const int m0 = (blockIdx.x - slice * tiles_m) * BM;
  const int K16 = (p.K + 15) / 16 * 16, all = (p.K + 127) / 128;
  const int first = SPLIT ? slice * slice_steps : 0;
  const int steps = SPLIT ? min(all - first, slice_steps) : all;

  const int8_t *src[kLoads];
  int chunk[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int row = (wave * kLoads + j) * 8 + (lane >> 3);
    chunk[j] = ((lane & 7) ^ (row & 7)) * 16;
    src[j] = row < BM ? p.w + (int64_t)min(m0 + row, p.M - 1) * p.ldw
                      : p.a + (int64_t)min(row - BM, p.T - 1) * p.lda;
  }
  auto stage = [&](int step) {
    int8_t *to = lds[step % kRing];
    const int k = (first + step) * 128;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const void *from = step < steps && k + chunk[j] < K16 ? (const void *)(src[j] + k + chunk[j])
                                            : (const void *)&kZeros;
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void *)from,
          (__attribute__((address_space(3))) void *)(to + (wave * kLoads + j) * 1024), 16, 0, 0);
    }
  };
#pragma unroll
  for (int s = 0; s < kRing - 1; ++s) stage(s);

  const int r = lane & 31, hi = lane >> 5;
  const int at = ((wave * 2 + hi) ^ (r & 7)) * 16;
  int16v acc[kT];
#pragma unroll
  for (int j = 0; j < kT; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[j][e] = 0;
  for (int step = 0; step < steps; ++step) {
    // this step's loads are the oldest kLoads of (kRing - 1) * kLoads
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kRing - 2) * kLoads) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    stage(step + kRing - 1);  // over the step before, which every wave has read
    const int8_t *from = lds[step % kRing];
    const int4v wf = *reinterpret_cast<const int4v *>(from + r * 128 + at);
#pragma unroll
    for (int j = 0; j < kT; ++j)
      acc[j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
          wf, *reinterpret_cast<const int4v *>(from + (BM + j * 32 + r) * 128 + at), acc[j], 0, 0,
          0);
    // reads are done before the barrier that lets the next load overwrite them
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();

  // the waves' sums: wave w adds up and writes rows 8w..8w+7 of every token
  int *part = reinterpret_cast<int *>(&lds[0][0]);  // [wave][token tile][row / 4][token][4]
#pragma unroll
  for (int j = 0; j < kT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<int4v *>(part + (((wave * kT + j) * 8 + 2 * q + hi) * 32 + r) * 4) =
          int4v{acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
  __syncthreads();
  const int m = m0 + 8 * wave + 4 * hi;
  if (m >= p.M) return;
  RowFactors f;
  if constexpr (!SPLIT) f = row_factors<T>(p, m);
#pragma unroll
  for (int j = 0; j < kT; ++j) {
    const int t = j * 32 + r;
    if (t >= p.T) continue;
    int4v s = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w)
      s += *reinterpret_cast<const int4v *>(
          part + (((w * kT + j) * 8 + 2 * wave + hi) * 32 + r) * 4);
    if constexpr (SPLIT) {
      store_sums(partial + ((int64_t)slice * p.T + t) * p.M, m, p.M, s);
    } else {
      const int sum[4] = {s[0], s[1], s[2], s[3]};
      store_y<T>(p, t, m, finish<T>(f, p.a_scale[t], sum));
    }
  }
}

// ---- tiles
//
// BM rows of W by BT tokens a workgroup, 128 bytes of K a step, two stages in
// shared memory that memory fills directly.  A row's eight 16-byte chunks lie in
// the order chunk ^ (row mod 8), so that the eight lanes that share a cycle of a
// 16-byte read are in different banks; the order is made by which chunk each
// lane asks memory for.
//
// A step is four products of 32 bytes.  Their operands are read one product
// ahead, and the barrier stands before the last of them: its operands are in
// registers by then, so it runs while the next step's first are read and the
// stage just finished is asked for again, a whole step ahead of its use.
//
// 4096 tokens by 14336 x 4096: the 768 whole tiles of 256 take 232 us, 1.78
// POP/s; at K = 14336 they reach 2.1 POP/s, the rate of a library's largest
// product, so what a shorter K loses is the start and the 128 KB of outputs at
// the end of each tile, which nothing overlaps (one workgroup fills a compute
// unit's shared memory).
constexpr int kStep = 128;

template <int BM, int BT, int WM, int WT>
struct TileShape {
  static constexpr int kRows = BM / WM, kTokens = BT / WT;    // of a wave
  static constexpr int kM = kRows / 32, kT = kTokens / 32;    // its 32x32 tiles
  static constexpr int kLoads = (BM + BT) / 8 / (WM * WT);    // of 1 KB, a wave and stage
  static constexpr int kStageBytes = (BM + BT) * kStep;
  static constexpr int kOutStride = kRows * 2 + 16;           // of a token's fp16 outputs
};

template <typename T, int BM, int BT, int WM, int WT, bool SPLIT>
__global__ __launch_bounds__(WM *WT * 64, BM * BT <= 128 * 128 ? 2 : 1) void tile_kernel(
    IntProduct p, int begin, int count, int tiles, int tiles_t, int slice_steps,
    int32_t *partial) {
  using S = TileShape<BM, BT, WM, WT>;
  __shared__ __align__(16) int8_t lds[2][S::kStageBytes];
  __shared__ __align__(16) float row_scales[BM], row_bias[BM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // workgroups go to the 8 XCDs in turn: each XCD gets a run of tiles that
  // shares rows of W
  const int per = (count + 7) / 8;
  const int nth = (int)(blockIdx.x % 8) * per + (int)blockIdx.x / 8;
  if (nth >= count) return;
  const int slice = (begin + nth) / tiles, tile = (begin + nth) % tiles;
  const int m0 = tile / tiles_t * BM, t0 = tile % tiles_t * BT;
  if (t0 >= p.T) return;  // the second half of a last tile
  const int K16 = (p.K + 15) / 16 * 16;
  const int steps = (p.K + kStep - 1) / kStep;
  const int first = slice * slice_steps, last = min(steps, first + slice_steps);

  // the chunks this lane brings in: load j covers stage rows 8j..8j+7, W's first
  const int8_t *src[S::kLoads];
  int chunk[S::kLoads];
#pragma unroll
  for (int j = 0; j < S::kLoads; ++j) {
    const int row = (wave * S::kLoads + j) * 8 + (lane >> 3);
    chunk[j] = ((lane & 7) ^ (row & 7)) * 16;
    src[j] = row < BM ? p.w + (int64_t)min(m0 + row, p.M - 1) * p.ldw
                      : p.a + (int64_t)min(t0 + row - BM, p.T - 1) * p.lda;
  }
  auto stage = [&](int buf, int step) {
    const int k = step * kStep;
#pragma unroll
    for (int j = 0; j < S::kLoads; ++j) {
      const void *from = k + chunk[j] < K16 ? (const void *)(src[j] + k + chunk[j])
                                            : (const void *)&kZeros;
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void *)from,
          (__attribute__((address_space(3))) void *)(&lds[buf][(wave * S::kLoads + j) * 1024]), 16,
          0, 0);
    }
  };

  int16v acc[S::kM][S::kT];
#pragma unroll
  for (int i = 0; i < S::kM; ++i)
#pragma unroll
    for (int j = 0; j < S::kT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  const int wm = wave / WT * S::kRows, wt = wave % WT * S::kTokens;
  const int r = lane & 31, hi = lane >> 5;
  int4v wf[2][S::kM], af[2][S::kT];
  auto operands = [&](int buf, int ks, int into) {
    const int at = ((ks * 2 + hi) ^ (r & 7)) * 16;
#pragma unroll
    for (int i = 0; i < S::kM; ++i)
      wf[into][i] = *reinterpret_cast<const int4v *>(&lds[buf][(wm + i * 32 + r) * kStep + at]);
#pragma unroll
    for (int j = 0; j < S::kT; ++j)
      af[into][j] =
          *reinterpret_cast<const int4v *>(&lds[buf][(BM + wt + j * 32 + r) * kStep + at]);
  };
  auto multiply = [&](int from) {
#pragma unroll
    for (int i = 0; i < S::kM; ++i)
#pragma unroll
      for (int j = 0; j < S::kT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[from][i], af[from][j], acc[i][j], 0,
                                                          0, 0);
  };
  // all of this wave's loads have landed and its reads are done, then all waves'
  auto meet = [&]() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
  };
  if (first < last) {
    stage(0, first);
    meet();
    if (first + 1 < last) stage(1, first + 1);
    operands(0, 0, 0);
  }
  for (int step = first; step < last; ++step) {
    const int buf = (step - first) & 1;
#pragma unroll
    for (int ks = 0; ks < 3; ++ks) {
      operands(buf, ks + 1, (ks + 1) & 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(ks & 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    meet();
    if (step + 2 < last) stage(buf, step + 2);
    if (step + 1 < last) operands(buf ^ 1, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    multiply(1);
    __builtin_amdgcn_sched_barrier(0);
  }

  if constexpr (SPLIT) {
#pragma unroll
    for (int j = 0; j < S::kT; ++j) {
      const int t = t0 + wt + j * 32 + r;
      if (t >= p.T) continue;
#pragma unroll
      for (int i = 0; i < S::kM; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int m = m0 + wm + i * 32 + 8 * q + 4 * hi;
          store_sums(partial + ((int64_t)slice * p.T + t) * p.M, m, p.M,
                     int4v{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                           acc[i][j][4 * q + 3]});
        }
    }
    return;
  }
  float a_scale[S::kT];
#pragma unroll
  for (int j = 0; j < S::kT; ++j) a_scale[j] = p.a_scale[min(t0 + wt + j * 32 + r, p.T - 1)];
  // fp16 outputs that can be written 16 bytes at a time turn in shared memory,
  // each wave its own: a lane holds 4 rows of one token, a write wants 8
  const bool turn = sizeof(T) == 2 && ((uintptr_t)p.y & 15) == 0 && p.ldy % 8 == 0;
  int8_t *out = &lds[0][0] + wave * (S::kOutStride * 32);
  if (tid < BM) {
    const int m = min(m0 + tid, p.M - 1);
    row_scales[tid] = p.w_scale[m];
    row_bias[tid] = p.bias != nullptr ? (float)static_cast<const T *>(p.bias)[m] : 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < S::kT; ++j) {
    const int t = t0 + wt + j * 32 + r;
    asm volatile("" ::: "memory");  // the factors are read again, not kept in registers
#pragma unroll
    for (int i = 0; i < S::kM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = i * 32 + 8 * q + 4 * hi, m = m0 + wm + row;
        int sum[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = acc[i][j][4 * q + e];
        RowFactors f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f.scale[e] = row_scales[wm + row + e];
          f.bias[e] = row_bias[wm + row + e];
        }
        const Four<T> y = finish<T>(f, a_scale[j], sum);
        if (turn)
          *reinterpret_cast<Four<T> *>(out + r * S::kOutStride + row * 2) = y;
        else if (t < p.T && m < p.M)
          store_y<T>(p, t, m, y);
      }
    if (turn) {
      constexpr int kPer = S::kRows / 8;  // 16-byte pieces of a token
#pragma unroll
      for (int k = 0; k < 32 * kPer / 64; ++k) {
        const int piece = k * 64 + lane, tt = t0 + wt + j * 32 + piece / kPer;
        const int row = piece % kPer * 8, m = m0 + wm + row;
        const int8_t *from = out + piece / kPer * S::kOutStride + row * 2;
        T *y = static_cast<T *>(p.y) + (int64_t)tt * p.ldy + m;
        if (tt < p.T && m + 8 <= p.M) {
          *reinterpret_cast<int4v *>(y) = *reinterpret_cast<const int4v *>(from);
        } else if (tt < p.T) {
          for (int e = 0; e < 8; ++e)
            if (m + e < p.M) y[e] = reinterpret_cast<const T *>(from)[e];
        }
      }
    }
  }
}

// Sums the slices of K, 4 outputs a thread.
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(IntProduct p, int slices,
                                                   const int32_t *partial) {
  const int quads = (p.M + 3) / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)quads * p.T) return;
  const int t = (int)(id / quads), m = (int)(id % quads) * 4;
  int sum[4] = {0, 0, 0, 0};
  for (int s = 0; s < slices; ++s) {
    const int32_t *o = partial + ((int64_t)s * p.T + t) * p.M + m;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m + e < p.M) sum[e] += o[e];
  }
  store_y<T>(p, t, m, finish<T>(row_factors<T>(p, m), p.a_scale[t], sum));
}

// The tile and the split of K for a product.  A tile of side b costs each compute
// unit b * b over what it reaches of the largest one's rate (measured at
// 4096 x 4096 x 14336 on 256 compute units: 2118, 1669 and 1128 TOP/s with 256,
// 128 and 64), and the compute unit with the most tiles ends last.  Where even
// the small tiles leave compute units idle K is split, never under eight steps.
// Up to kFewTokens tokens go through the ring instead (side 32 or 64, their
// number rounded up).
//
// Where the tiles of 256 fill the compute units a few times and at most half of
// them once more, those last tiles go in halves (256 x 128, 0.88 of the rate) to
// all of them, in a launch of their own: 4096 tokens by 14336 x 4096, 896 tiles,
// take 252 us so and 269 in whole tiles (without the quantizer, one set of inputs).
constexpr int kFewTokens = 64;
constexpr int kUnits = 256;
struct TilePlan {
  int side, tiles_m, tiles_t, slices, slice_steps;
  int halves;  // of the last tiles of 256: in two halves each
  bool few;
};
TilePlan tile_plan(int T, int M, int K) {
  TilePlan q{};
  const int steps = (K + kStep - 1) / kStep;
  auto split = [&](int64_t want) {
    int64_t slices = want / ((int64_t)q.tiles_m * q.tiles_t);
    slices = slices > steps / 8 ? steps / 8 : slices;
    slices = slices < 1 ? 1 : slices;
    q.slice_steps = (int)((steps + slices - 1) / slices);
    q.slices = (steps + q.slice_steps - 1) / q.slice_steps;
  };
  if (T <= kFewTokens) {
    q.few = true;
    q.side = T <= 32 ? 32 : 64;
    q.tiles_m = (M + 31) / 32;
    q.tiles_t = 1;
    split(256);
    return q;
  }
  double best = 0;
  const int sides[3] = {256, 128, 64};
  const double rate[3] = {1.0, 0.79, 0.53};
  for (int i = 0; i < 3; ++i) {
    const int b = sides[i];
    const int64_t tiles = (int64_t)((M + b - 1) / b) * ((T + b - 1) / b);
    const int64_t over = tiles % kUnits;
    const bool halved = b == 256 && tiles > kUnits && over > 0 && over <= kUnits / 2;
    const double rounds = (double)(tiles / kUnits) + (over == 0 ? 0 : halved ? 0.6 : 1);
    const double cost = rounds * b * b / rate[i];
    if (i == 0 || cost < best) {
      best = cost;
      q.side = b;
      q.halves = halved ? (int)over * 2 : 0;
    }
  }
  const int b = q.side;
  q.tiles_m = (M + b - 1) / b;
  q.tiles_t = (T + b - 1) / b;
  split(b > 64 ? 0 : 512);
  return q;
}

// Tiles begin .. begin + count of the grid of BM by BT tiles.
template <typename T, int BM, int BT, int WM, int WT, bool SPLIT>
void run_tiles(const IntProduct &p, const TilePlan &q, int tiles_t, int begin, int count,
               int32_t *partial, hipStream_t s) {
  tile_kernel<T, BM, BT, WM, WT, SPLIT><<<(count + 7) / 8 * 8, WM * WT * 64, 0, s>>>(
      p, begin, count, q.tiles_m * tiles_t, tiles_t, q.slice_steps, partial);
}

template <typename T>
hipError_t gemm_type(const IntProduct &p, int32_t *partial, hipStream_t s) {
  const TilePlan q = tile_plan(p.T, p.M, p.K);
  const int tiles = q.tiles_m * q.tiles_t;
  if (q.few) {
    const unsigned grid = (unsigned)q.tiles_m * q.slices;
    if (q.side == 32 && q.slices == 1)
      few_kernel<T, 32, false><<<grid, 256, 0, s>>>(p, q.tiles_m, q.slice_steps, partial);
    else if (q.side == 32)
      few_kernel<T, 32, true><<<grid, 256, 0, s>>>(p, q.tiles_m, q.slice_steps, partial);
    else if (q.slices == 1)
      few_kernel<T, 64, false><<<grid, 256, 0, s>>>(p, q.tiles_m, q.slice_steps, partial);
    else
      few_kernel<T, 64, true><<<grid, 256, 0, s>>>(p, q.tiles_m, q.slice_steps, partial);
  } else if (q.side == 256) {
    run_tiles<T, 256, 256, 4, 2, false>(p, q, q.tiles_t, 0, tiles - q.halves / 2, partial, s);
    if (q.halves > 0) {
      hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      run_tiles<T, 256, 128, 4, 2, false>(p, q, 2 * q.tiles_t, 2 * tiles - q.halves, q.halves,
                                          partial, s);
    }
  } else if (q.side == 128) {
    run_tiles<T, 128, 128, 2, 2, false>(p, q, q.tiles_t, 0, tiles, partial, s);
  } else if (q.slices == 1) {
    run_tiles<T, 64, 64, 2, 2, false>(p, q, q.tiles_t, 0, tiles, partial, s);
  } else {
    run_tiles<T, 64, 64, 2, 2, true>(p, q, q.tiles_t, 0, tiles * q.slices, partial, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || q.slices == 1) return e;
  const int64_t quads = (int64_t)((p.M + 3) / 4) * p.T;
  join_kernel<T><<<(unsigned)((quads + 255) / 256), 256, 0, s>>>(p, q.slices, partial);
  return hipGetLastError();
}

template <typename T>
hipError_t fused_type(const IntProduct &p, const void *X, int ldx, hipStream_t s) {
  const size_t lds = (size_t)p.T * ((p.K + 127) / 128 * 128 + 16);
  fused_kernel<T><<<(p.M + 15) / 16, 256, lds, s>>>(p, static_cast<const T *>(X), ldx);
  return hipGetLastError();
}

}  // namespace

template <typename T>
static hipError_t quantize_type(const void *X, int rows, int K, int ldx, int8_t *codes, int ldc,
                                float *scales, hipStream_t s) {
  const T *x = static_cast<const T *>(X);
  if (K <= 2048)
    quantize_kernel<T, 1><<<rows, 256, 0, s>>>(x, K, ldx, codes, ldc, scales);
  else if (K <= 4096)
    quantize_kernel<T, 2><<<rows, 256, 0, s>>>(x, K, ldx, codes, ldc, scales);
  else if (K <= 8192)
    quantize_kernel<T, 4><<<rows, 256, 0, s>>>(x, K, ldx, codes, ldc, scales);
  else
    quantize_kernel<T, 0><<<rows, 256, 0, s>>>(x, K, ldx, codes, ldc, scales);
  return hipGetLastError();
}
hipError_t launch_int_quantize(const void *X, bcq_dtype dt, int rows, int K, int ldx,
                               int8_t *codes, int ldc, float *scales, hipStream_t s) {
  return dt == BCQ_F16 ? quantize_type<_Float16>(X, rows, K, ldx, codes, ldc, scales, s)
                       : quantize_type<float>(X, rows, K, ldx, codes, ldc, scales, s);
}

size_t int_partial_bytes(int T, int M, int K) {
  const TilePlan q = tile_plan(T, M, K);
  return q.slices > 1 ? (size_t)q.slices * T * M * sizeof(int32_t) : 0;
}

hipError_t launch_int_gemm(const IntProduct &p, bcq_dtype dt, int32_t *partial, hipStream_t s) {
  return dt == BCQ_F16 ? gemm_type<_Float16>(p, partial, s) : gemm_type<float>(p, partial, s);
}

bool int_fused_ok(int T, int K) {
  return T <= kFusedTokens && (int64_t)T * K <= kFusedElements;
}

hipError_t launch_int_fused(const IntProduct &p, const void *X, int ldx, bcq_dtype dt,
                            hipStream_t s) {
  return dt == BCQ_F16 ? fused_type<_Float16>(p, X, ldx, s) : fused_type<float>(p, X, ldx, s);
}

}  // namespace bcq
