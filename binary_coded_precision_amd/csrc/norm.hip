// norm.hip -- residual addition, root-mean-square norm and rounding to 8 bits of
// each token's row (bcq_rms_norm).
//
//   h = round(x + residual)                      to the call's type
//   y = (h * inv) * gamma,  inv = 1 / sqrt(mean(h^2) + eps)
//   scale = max|y| * (1/127),  code = rint(y / scale)
//
// The squares are summed in fp64: they stay in range for every fp32 row, and
// inv, rounded once to fp32, does not depend on the order of the sum but for a
// sum within 1e-15 of a rounding's border.  The two products and the quotient
// are single operations in fp32, so that codes are a function of h and inv.
#include "row_codes.h"
#include "serve_internal.h"

namespace bcq {
namespace {

template <typename T>
__device__ __forceinline__ void store_row8(T *row, const float (&x)[8], int k, int K) {
  if (k + 8 <= K) {
    if constexpr (sizeof(T) == 2) {
      typedef _Float16 half8 __attribute__((ext_vector_type(8)));
      half8 h;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = (_Float16)x[e];
      *reinterpret_cast<half8 *>(row + k) = h;
    } else {
      reinterpret_cast<float4 *>(row + k)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4 *>(row + k)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e < K) row[k + e] = (T)x[e];
  }
}

// Sum and maximum over a workgroup's threads.  `red` is not in use by what was
// called before with another one.
template <int THREADS>
__device__ __forceinline__ double sum_all(double x, double *red) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  if constexpr (THREADS == 64) return x;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) x += red[w];
  return x;
}
template <int THREADS>
__device__ __forceinline__ float max_all(float x, float *red) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = nan_max(x, __shfl_xor(x, d));
  if constexpr (THREADS == 64) return x;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) x = nan_max(x, red[w]);
  return x;
}

// h of 8 elements from where they are found: the sum, rounded to T.
template <typename T>
__device__ __forceinline__ void load_h(float (&h)[8], const T *x, const T *r, int k, int K) {
  load_row8(h, x, k, K);
  if (r != nullptr) {
    float b[8];
    load_row8(b, r, k, K);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = (float)(T)(h[e] + b[e]);
  }
}

template <typename T>
__device__ __forceinline__ void scale_row8(float (&y)[8], const float (&h)[8], float inv,
                                           const T *gamma, int k, int K) {
  float g[8];
  load_row8(g, gamma, k, K);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = (h[e] * inv) * g[e];
}

// A row by THREADS threads.  Rows of up to 8 N THREADS elements are held in registers;
// longer ones (N = 0) are read again from the caches for each of three passes.
//
// Bound by the bytes of x, the residual, h, y and codes, each passed once: 4096 x 4096 in
// fp16 with h and codes (118 MB) 28.8 us, 4.1 TB/s; 30000 x 512 25 us, 4.3 TB/s.  Few
// rows are bound by one pass's latency, 2.6 us for one of 4096.
//
// Rows of up to 512 elements are a wave's, four to a workgroup: as fast as a workgroup a
// row for one row (4.0 us), 25 us rather than 59 for 30000 rows of 512, which are bound
// by workgroups started.  Rows of up to 1024 too from 4096 of them on (30000 x 1024 41 us,
// not 68; 1024 rows take the same, one row 4.6 us, not 3.9).  With more than that in a
// wave's registers, or longer rows, more threads are better (1 x 2048: 4.3 us, by one
// wave 6.8).  Longer rows than 2048 are 512 threads' where there is at most one for each
// compute unit (1 x 8192 5.6 us, by 256 threads 7.0), else 256 threads', which leave room
// for more rows (8192 x 4096 41 us, by 512 threads 49).
template <typename T, int N, int THREADS>
__device__ __forceinline__ void norm_row(const NormArgs &a, int64_t row, double *red_sum,
                                         float *red_max) {
  const int tid = threadIdx.x % THREADS, K = a.K;
  const T *x = static_cast<const T *>(a.x) + row * a.ldx;
  const T *r = a.residual == nullptr ? nullptr
                                     : static_cast<const T *>(a.residual) + row * a.ldr;
  const T *gamma = static_cast<const T *>(a.gamma);
  T *h_out = a.h == nullptr ? nullptr : static_cast<T *>(a.h) + row * a.ldh;
  T *y_out = a.y == nullptr ? nullptr : static_cast<T *>(a.y) + row * a.ldy;
  int8_t *codes = a.codes == nullptr ? nullptr : a.codes + row * a.ldc;
  constexpr int STEP = THREADS * 8;
  const int end = codes == nullptr ? K : (K + 15) / 16 * 16;  // codes' zeros behind K

  float v[N > 0 ? N : 1][8];
  double sum = 0.;
  if constexpr (N > 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) load_h<T>(v[n], x, r, n * STEP + tid * 8, K);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fma((double)v[n][e], (double)v[n][e], sum);
    if (h_out != nullptr)
#pragma unroll
      for (int n = 0; n < N; ++n) store_row8<T>(h_out, v[n], n * STEP + tid * 8, K);
  } else {
    for (int k = tid * 8; k < K; k += STEP) {
      load_h<T>(v[0], x, r, k, K);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fma((double)v[0][e], (double)v[0][e], sum);
      if (h_out != nullptr) store_row8<T>(h_out, v[0], k, K);
    }
    // x or the residual may be what h has just replaced; a thread reads what it wrote
    if (h_out != nullptr) x = h_out, r = nullptr;
  }
  sum = sum_all<THREADS>(sum, red_sum);
  const float inv = (float)(1. / sqrt(sum / K + a.eps));
  if (y_out == nullptr && codes == nullptr) return;

  float top = 0.f;
  if constexpr (N > 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int k = n * STEP + tid * 8;
      scale_row8<T>(v[n], v[n], inv, gamma, k, K);
      if (y_out != nullptr) store_row8<T>(y_out, v[n], k, K);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = nan_max(top, k + e < K ? fabsf(v[n][e]) : 0.f);
    }
  } else {
    for (int k = tid * 8; k < K; k += STEP) {
      load_h<T>(v[0], x, r, k, K);
      scale_row8<T>(v[0], v[0], inv, gamma, k, K);
      if (y_out != nullptr) store_row8<T>(y_out, v[0], k, K);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = nan_max(top, k + e < K ? fabsf(v[0][e]) : 0.f);
    }
  }
  if (codes == nullptr) return;
  const float s = row_scale(max_all<THREADS>(top, red_max));
  if (tid == 0) a.scales[row] = s;
  if constexpr (N > 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int k = n * STEP + tid * 8;
      if (k < end) *reinterpret_cast<uint2 *>(codes + k) = codes8(v[n], s);
    }
  } else {
    for (int k = tid * 8; k < end; k += STEP) {
      load_h<T>(v[0], x, r, k, K);
      scale_row8<T>(v[0], v[0], inv, gamma, k, K);
      *reinterpret_cast<uint2 *>(codes + k) = codes8(v[0], s);
    }
  }
}

template <typename T, int N, int THREADS>
__global__ __launch_bounds__(THREADS == 64 ? 256 : THREADS) void norm_kernel(NormArgs a, int rows) {
  __shared__ double red_sum[THREADS / 64];
  __shared__ float red_max[THREADS / 64];
  if constexpr (THREADS == 64) {
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row < rows) norm_row<T, N, THREADS>(a, row, nullptr, nullptr);
  } else if constexpr (THREADS <= 512) {
    norm_row<T, N, THREADS>(a, blockIdx.x, red_sum, red_max);
  } else {
    // a launch's work items are counted in 32 bits: more rows take turns
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
      norm_row<T, N, THREADS>(a, row, red_sum, red_max);
      __syncthreads();  // the sums are written again
    }
  }
}

template <typename T>
hipError_t norm_type(const NormArgs &a, int rows, hipStream_t s) {
  constexpr int kMostRows = (1 << 22) - 1;  // of 1024 threads
  const int turns = rows < kMostRows ? rows : kMostRows;
  const bool few = rows <= 256;
  const int quads = (int)(((int64_t)rows + 3) / 4);
  if (a.K <= 512)
    norm_kernel<T, 1, 64><<<quads, 256, 0, s>>>(a, rows);
  else if (a.K <= 1024 && rows >= 4096)
    norm_kernel<T, 2, 64><<<quads, 256, 0, s>>>(a, rows);
  else if (a.K <= 2048)
    norm_kernel<T, 1, 256><<<rows, 256, 0, s>>>(a, rows);
  else if (a.K <= 4096 && few)
    norm_kernel<T, 1, 512><<<rows, 512, 0, s>>>(a, rows);
  else if (a.K <= 8192 && few)
    norm_kernel<T, 2, 512><<<rows, 512, 0, s>>>(a, rows);
  else if (a.K <= 4096)
    norm_kernel<T, 2, 256><<<rows, 256, 0, s>>>(a, rows);
  else if (a.K <= 8192)
    norm_kernel<T, 4, 256><<<rows, 256, 0, s>>>(a, rows);
  else if (a.K <= 16384)
    norm_kernel<T, 2, 1024><<<turns, 1024, 0, s>>>(a, rows);
  else
    norm_kernel<T, 0, 1024><<<turns, 1024, 0, s>>>(a, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs &a, int T, bcq_dtype dt, hipStream_t s) {
  return dt == BCQ_F16 ? norm_type<_Float16>(a, T, s) : norm_type<float>(a, T, s);
}

}  // namespace bcq
