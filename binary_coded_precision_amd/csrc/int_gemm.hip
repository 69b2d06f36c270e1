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
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = k + e < K ? (float)row[k + e] : 0.f;
  }
}

__device__ __forceinline__ uint32_t code_of(float x, float s) {
  const float q = s > 0.f && s < INFINITY ? rintf(x / s) : 0.f;
  return (uint32_t)(int)fminf(fmaxf(q, -127.f), 127.f) & 255u;
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s) {
  uint2 c = {0, 0};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c.x |= code_of(x[e], s) << (8 * e);
    c.y |= code_of(x[4 + e], s) << (8 * e);
  }
  return c;
}

// A row's scale; NaN for a row that holds an infinity or NaN (its codes are 0),
// so that its products are NaN.
__device__ __forceinline__ float row_scale(float top) {
  return top < INFINITY ? top * (1.f / 127.f) : NAN;
}

// One workgroup a row, read twice (the second time from the caches).
template <typename T>
__global__ __launch_bounds__(256) void quantize_kernel(const T *X, int K, int ldx, int8_t *codes,
                                                       int ldc, float *scales) {
  __shared__ float red[4];
  const T *x = X + (int64_t)blockIdx.x * ldx;
  const int tid = threadIdx.x;
  float v[8], top = 0.f;
  for (int k = tid * 8; k < K; k += 256 * 8) {
    load_row8(v, x, k, K);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = nan_max(top, fabsf(v[e]));
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
  for (int k = tid * 8; k < end; k += 256 * 8) {
    load_row8(v, x, k, K);
    *reinterpret_cast<uint2 *>(c + k) = codes8(v, s);
  }
}

template <typename T>
__device__ __forceinline__ void store_y(const IntProduct &p, int t, int m, const float (&v)[4]) {
  T *y = static_cast<T *>(p.y) + (int64_t)t * p.ldy + m;
  if (m + 4 <= p.M && ((uintptr_t)y & (4 * sizeof(T) - 1)) == 0) {
    struct __attribute__((aligned(4 * sizeof(T)))) V4 {
      T x[4];
    } o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o.x[e] = (T)v[e];
    *reinterpret_cast<V4 *>(y) = o;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m + e < p.M) y[e] = (T)v[e];
  }
}

// Outputs (t, m..m+3) from their exact sums.
template <typename T>
__device__ __forceinline__ void finish(const IntProduct &p, int t, int m, float a_scale,
                                       const int (&acc)[4]) {
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int mm = min(m + e, p.M - 1);
    v[e] = (float)acc[e] * (a_scale * p.w_scale[mm]);
    if (p.bias != nullptr) v[e] += (float)static_cast<const T *>(p.bias)[mm];
  }
  store_y<T>(p, t, m, v);
}

// ---- few tokens: one launch
//
// 16 rows of W a workgroup, its four waves taking turns over K in steps of 128
// bytes; W goes from memory to the matrix operands without passing through
// shared memory, eight loads of 16 bytes a lane in flight, the first of them
// asked for before the tokens are quantized.  Every workgroup quantizes the
// tokens for itself: T * K is at most kFusedElements, a fraction of a
// microsecond, where a launch of its own costs several.
constexpr int kFusedTokens = 16, kFusedElements = 16384;
constexpr int kFusedDepth = 4;  // steps in flight

template <typename T>
__global__ __launch_bounds__(256) void fused_kernel(IntProduct p, const T *X, int ldx) {
  extern __shared__ __align__(16) int8_t xs[];  // [T][row]
  __shared__ float red[kFusedTokens][4];
  __shared__ int4v part[4][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int m0 = blockIdx.x * 16;
  const int K16 = (p.K + 15) / 16 * 16, steps = (p.K + 127) / 128;
  const int row = steps * 128 + 16;  // 16 past a multiple of 128: rows start in other banks
  const int8_t *w = p.w + (int64_t)min(m0 + r, p.M - 1) * p.ldw + g * 32;

  int4v wf[kFusedDepth][2];
  auto fetch = [&](int4v(&f)[2], int step) {
    const int k = step * 128 + g * 32;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      f[e] = k + 16 * e < K16 && step < steps
                 ? *reinterpret_cast<const int4v *>(w + (int64_t)step * 128 + 16 * e)
                 : int4v{0, 0, 0, 0};
  };
#pragma unroll
  for (int d = 0; d < kFusedDepth; ++d) fetch(wf[d], wave + 4 * d);

  for (int t = 0; t < p.T; ++t) {
    float v[8], top = 0.f;
    for (int k = tid * 8; k < p.K; k += 256 * 8) {
      load_row8(v, X + (int64_t)t * ldx, k, p.K);
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
    for (int k = tid * 8; k < steps * 128; k += 256 * 8) {
      load_row8(v, X + (int64_t)t * ldx, k, p.K);
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
        fetch(wf[d], st + 4 * kFusedDepth);
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
    if (m0 + 4 * g < p.M) finish<T>(p, r, m0 + 4 * g, s, sum);
  }
}

// ---- tiles
//
// BM rows of W by BT tokens a workgroup of four waves, 128 bytes of K a step,
// two stages in shared memory that memory fills directly.  A row's eight
// 16-byte chunks lie in the order chunk ^ (row mod 8), so that the eight lanes
// that share a cycle of a 16-byte read are in different banks; the order is
// made by which chunk each lane asks memory for.
constexpr int kStep = 128;

template <int BM, int BT, int WM, int WT>
struct TileShape {
  static constexpr int kThreads = WM * WT * 64;
  static constexpr int kM = BM / WM / 32, kT = BT / WT / 32;  // 32x32 tiles of a wave
  static constexpr int kLoads = (BM + BT) / 8 / (WM * WT);    // of 1 KB, a wave and stage
  static constexpr int kStageBytes = (BM + BT) * kStep;
};

template <typename T, int BM, int BT, int WM, int WT, bool SPLIT>
__global__ __launch_bounds__(WM *WT * 64) void tile_kernel(IntProduct p, int tiles_m, int tiles_t,
                                                           int slices, int slice_steps,
                                                           int32_t *partial) {
  using S = TileShape<BM, BT, WM, WT>;
  __shared__ __align__(16) int8_t lds[2][S::kStageBytes];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // workgroups go to the 8 XCDs in turn: each XCD gets a run of tiles that
  // shares rows of W
  const int tiles = tiles_m * tiles_t;
  const int per = (tiles * slices + 7) / 8;
  const int id = (int)(blockIdx.x % 8) * per + (int)blockIdx.x / 8;
  if (id >= tiles * slices) return;
  const int slice = id / tiles, tile = id % tiles;
  const int m0 = tile / tiles_t * BM, t0 = tile % tiles_t * BT;
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

  const int wm = wave / WT * (BM / WM), wt = wave % WT * (BT / WT);
  const int r = lane & 31, hi = lane >> 5;
  if (first < last) stage(0, first);
  for (int step = first; step < last; ++step) {
    const int buf = (step - first) & 1;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (step + 1 < last) stage(buf ^ 1, step + 1);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      int4v wf[S::kM], af[S::kT];
      const int at = ((ks * 2 + hi) ^ (r & 7)) * 16;
#pragma unroll
      for (int i = 0; i < S::kM; ++i)
        wf[i] = *reinterpret_cast<const int4v *>(&lds[buf][(wm + i * 32 + r) * kStep + at]);
#pragma unroll
      for (int j = 0; j < S::kT; ++j)
        af[j] = *reinterpret_cast<const int4v *>(&lds[buf][(BM + wt + j * 32 + r) * kStep + at]);
#pragma unroll
      for (int i = 0; i < S::kM; ++i)
#pragma unroll
        for (int j = 0; j < S::kT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[i], af[j], acc[i][j], 0, 0, 0);
    }
  }

#pragma unroll
  for (int j = 0; j < S::kT; ++j) {
    const int t = t0 + wt + j * 32 + r;
    if (t >= p.T) continue;
    const float s = SPLIT ? 0.f : p.a_scale[t];
#pragma unroll
    for (int i = 0; i < S::kM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int m = m0 + wm + i * 32 + 8 * q + 4 * hi;
        if (m >= p.M) continue;
        int sum[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = acc[i][j][4 * q + e];
        if constexpr (SPLIT) {
          int32_t *o = partial + ((int64_t)slice * p.T + t) * p.M + m;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (m + e < p.M) o[e] = sum[e];
        } else {
          finish<T>(p, t, m, s, sum);
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
  finish<T>(p, t, m, p.a_scale[t], sum);
}

// The tile and the split of K for a product: the large tile once it fills the
// 256 compute units, else the small one, with K split until the card is full
// (never under four steps a slice).
struct TilePlan {
  bool large;
  int tiles_m, tiles_t, slices, slice_steps;
};
TilePlan tile_plan(int T, int M, int K) {
  TilePlan q;
  auto tiles = [&](int b) { return (int64_t)((M + b - 1) / b) * ((T + b - 1) / b); };
  q.large = tiles(128) >= 256;
  const int b = q.large ? 128 : 64;
  q.tiles_m = (M + b - 1) / b;
  q.tiles_t = (T + b - 1) / b;
  const int steps = (K + kStep - 1) / kStep;
  int slices = q.large ? 1 : (int)(512 / tiles(b));
  const int most = steps / 4;
  slices = slices > most ? most : slices;
  slices = slices < 1 ? 1 : slices;
  q.slice_steps = (steps + slices - 1) / slices;
  q.slices = (steps + q.slice_steps - 1) / q.slice_steps;
  return q;
}

template <typename T, int B, bool SPLIT>
void run_tiles(const IntProduct &p, const TilePlan &q, int32_t *partial, hipStream_t s) {
  const unsigned grid = (unsigned)(((int64_t)q.tiles_m * q.tiles_t * q.slices + 7) / 8 * 8);
  tile_kernel<T, B, B, 2, 2, SPLIT><<<grid, 256, 0, s>>>(p, q.tiles_m, q.tiles_t, q.slices,
                                                         q.slice_steps, partial);
}

template <typename T>
hipError_t gemm_type(const IntProduct &p, int32_t *partial, hipStream_t s) {
  const TilePlan q = tile_plan(p.T, p.M, p.K);
  if (q.large)
    run_tiles<T, 128, false>(p, q, partial, s);
  else if (q.slices == 1)
    run_tiles<T, 64, false>(p, q, partial, s);
  else
    run_tiles<T, 64, true>(p, q, partial, s);
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

hipError_t launch_int_quantize(const void *X, bcq_dtype dt, int rows, int K, int ldx,
                               int8_t *codes, int ldc, float *scales, hipStream_t s) {
  if (dt == BCQ_F16)
    quantize_kernel<<<rows, 256, 0, s>>>((const _Float16 *)X, K, ldx, codes, ldc, scales);
  else
    quantize_kernel<<<rows, 256, 0, s>>>((const float *)X, K, ldx, codes, ldc, scales);
  return hipGetLastError();
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
