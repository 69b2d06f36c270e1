// row_codes.h -- a row rounded to 8 bits with one scale, as the integer products
// read it (shared by int_gemm.hip and norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bcq {

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

}  // namespace bcq
