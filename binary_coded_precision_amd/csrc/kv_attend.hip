// kv_attend.hip -- attention over the 4-bit key/value cache (bcq_kv_attend).
//
// For a query row q (one of the n queries of one of the G query heads that
// share a cached head) and the cached vectors k_t = kz_t + ks_t * ck_t and
// v_t = vz_t + vs_t * cv_t with codes c in 0..15:
//
//   s_t = scale * (ks_t * (q . ck_t) + kz_t * sum(q))        (in log2 units here)
//   out = sum_t p_t v_t / sum_t p_t,  p_t = 2^(s_t - m)
//       = (sum_t (p_t vs_t) (cv_t - 8) + sum_t p_t (vz_t + 8 vs_t)) / sum_t p_t
//
// so both products run on the codes themselves, which fp16 holds exactly, and
// each token's four factors enter in fp32 afterwards.  A code c of K sits in an
// operand as the fp16 with bit pattern c, the subnormal c * 2^-24 (the matrix
// cores keep subnormal inputs), which takes one AND for two codes; codes masked
// four bits up are 16c * 2^-24, and the queries of those channels carry 1/16.
// Codes of V are centred: an average over many tokens is small against its
// terms, and what the terms' roundings leave would otherwise be multiplied by
// the 7.5 that the codes have in common (measured over 1023 tokens: 8e-4 of the
// output's norm without centring, 3e-4 with it, of which 2e-4 is the output's
// rounding).
//
// Roundings below 32 bits, for fp16 calls: p_t * vs_t, once, to fp16, relative
// to the row's largest (below).  It is as large as the output's own rounding.
// For fp32 calls the queries (after a power of two for each row) and p_t * vs_t
// are each held as the sum of two fp16, 22 bits.
//
// The reference m of a row's exponentials is a maximum over s_t + log2(vs_t)
// (log2 to a tenth, from the fp16's bits) rather than over s_t: then p_t * vs_t
// stays within fp16's normal range around its largest whatever the scales of V
// are, and sum p_t in fp32 has room for the difference.  m is raised, and what
// is summed so far rescaled, only when a tile exceeds it by more than 2^8, so
// the lanes of a row rarely have to agree.
//
// Layout: S^T = K Q^T with 16 tokens as a tile's rows and 16 query rows as its
// columns leaves a lane with 4 consecutive tokens of one query row; two such
// tiles are, without moving anything between lanes, the right operand of
// O^T = V^T P^T over 32 tokens.  The cache keeps V in blocks of 4 tokens so
// that a lane reads the left operand's nibbles (4 tokens of its channels) in
// one load; K needs one load of D/8 bytes a lane for 16 tokens.  No shared
// memory is used in the loop and no barrier: the waves of a workgroup either
// take turns over the tokens (few rows) or hold different rows.
#include "serve_internal.h"

namespace bcq {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr float kNegInf = -INFINITY;
// A tile may exceed a row's reference by this many powers of two before what is
// summed is rescaled: p_t * vs_t then stays below 2^10 in fp16.
constexpr float kSlack = 8.f;
constexpr float kCodeScale = 16777216.f;  // 2^24: a code's subnormal back to the code

struct Ws {
  float2 *ml;     // [splits][BH][R]: reference and sum of a row's exponentials
  float *o;       // [splits][BH][R][D]: outputs before the division
  float *scores;  // [BH][R][room], log2 units, -inf where masked
};

union Frag {
  uint32_t w[4];
  half8 h;
};

// One 16-token tile as a lane holds it.
template <int D>
struct Tile {
  uint32_t k[D / 32];  // its quarter of one token's K codes
  uint32_t v[D / 32];  // 4 tokens' codes of its D/16 channels
  uint4 m[2];          // the 4 tokens' factors
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&dst)[N], const uint8_t *src) {
  if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2 *>(src);
    dst[0] = x.x, dst[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 x = reinterpret_cast<const uint4 *>(src)[i];
      dst[4 * i] = x.x, dst[4 * i + 1] = x.y, dst[4 * i + 2] = x.z, dst[4 * i + 3] = x.w;
    }
  }
}

template <int D>
__device__ __forceinline__ void load_tile(Tile<D> &t, const KvView &c, int b, int h, int tok,
                                          int lane) {
  const int r = lane & 15, g = lane >> 4;
  const int page = __builtin_amdgcn_readfirstlane(
      c.table[(int64_t)b * c.max_pages + (tok >> c.page_log)]);
  // an entry that names no page is never followed
  const int safe = (unsigned)page < (unsigned)c.num_pages ? page : 0;
  const int64_t at = (((int64_t)safe * c.H + h) << c.page_log) + (tok & ((1 << c.page_log) - 1));
  load_words(t.k, c.k + at * (D / 2) + r * (D / 2) + g * (D / 8));
  load_words(t.v, c.v + at * (D / 2) + g * (2 * D) + r * (D / 8));
  const uint4 *m = reinterpret_cast<const uint4 *>(c.scales + at * 4) + g * 2;
  t.m[0] = m[0];
  t.m[1] = m[1];
}

__device__ __forceinline__ float half_bits(uint32_t w) {
  union {
    uint16_t u;
    _Float16 h;
  } x;
  x.u = (uint16_t)w;
  return (float)x.h;
}

// A token's factors: K scale and zero in log2 units, V scale and the value of
// its code 8, and the
// rough log2 of the V scale (its fp16 bits over 1024, exact at powers of two).
struct Factors {
  float ks, kz, vs, vz, lv;
};
__device__ __forceinline__ Factors factors(uint32_t kw, uint32_t vw, float scale_log2) {
  Factors f;
  f.ks = half_bits(kw) * (scale_log2 * kCodeScale);
  f.kz = half_bits(kw >> 16) * scale_log2;
  f.vs = half_bits(vw);
  f.vz = half_bits(vw >> 16) + 8.f * f.vs;
  f.lv = (float)(vw & 0x7fffu) * (1.f / 1024.f) - 15.f;
  return f;
}
template <int D>
__device__ __forceinline__ Factors factors(const Tile<D> &t, int i, float scale_log2) {
  const uint4 m = t.m[i >> 1];
  return (i & 1) ? factors(m.z, m.w, scale_log2) : factors(m.x, m.y, scale_log2);
}

// Left operand of S^T for word w of the tile: channels 8w..8w+7 of the lane's
// quarter in the order 0 4 1 5 2 6 3 7, the odd ones sixteenfold.
template <int D>
__device__ __forceinline__ half8 k_frag(const Tile<D> &t, int w) {
  const uint32_t lo = t.k[w], hi = lo >> 8;
  Frag f;
  f.w[0] = lo & 0x000f000fu;
  f.w[1] = lo & 0x00f000f0u;
  f.w[2] = hi & 0x000f000fu;
  f.w[3] = hi & 0x00f000f0u;
  return f.h;
}

// Codes less 8 of two tokens: the nibbles N (of a 16-bit unit's lower two) of
// both halves of a word.  A nibble in a mantissa under the exponent of 2^10, or
// of 2^6 for one four bits up, is 1024 + c or 64 + c; the subtraction is exact.
template <int N>
__device__ __forceinline__ half2v centred(uint32_t w) {
  union {
    uint32_t u;
    half2v h;
  } x;
  x.u = N ? (w & 0x00f000f0u) | 0x54005400u : (w & 0x000f000fu) | 0x64006400u;
  const _Float16 base = N ? (_Float16)72.f : (_Float16)1032.f;
  return x.h - half2v{base, base};
}

// Right operand of S^T: a query row's channels in k_frag's order.
__device__ __forceinline__ half8 q_order(const float (&x)[8]) {
  half8 f;
  f[0] = (_Float16)x[0], f[1] = (_Float16)x[4];
  f[2] = (_Float16)(x[1] * 0.0625f), f[3] = (_Float16)(x[5] * 0.0625f);
  f[4] = (_Float16)x[2], f[5] = (_Float16)x[6];
  f[6] = (_Float16)(x[3] * 0.0625f), f[7] = (_Float16)(x[7] * 0.0625f);
  return f;
}

__device__ __forceinline__ float group_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float group_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// A lane's queries: its column's row of each of CT tiles, channels of its
// quarter.  F32 holds each as two fp16 after dividing the row by `row_scale`.
template <int D, int CT, bool F32>
struct Queries {
  half8 hi[CT][D / 32];
  half8 lo[F32 ? CT : 1][F32 ? D / 32 : 1];
  float sum[CT];
  float row_scale[F32 ? CT : 1];
};

template <int D, int CT, bool F32>
__device__ __forceinline__ void load_queries(Queries<D, CT, F32> &Q, const AttendArgs &a, int b,
                                             int h, int row0, int R, int lane) {
  const int g = lane >> 4;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int row = row0 + ct * 16 + (lane & 15);
    float x[D / 32][8];
    if (row < R) {
      const int i = row / a.G, hq = h * a.G + row % a.G;
      const int64_t at = b * a.qs.batch + i * a.qs.token + hq * a.qs.head + g * (D / 4);
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[w][e] = F32 ? static_cast<const float *>(a.q)[at + w * 8 + e]
                        : (float)static_cast<const _Float16 *>(a.q)[at + w * 8 + e];
    } else {
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[w][e] = 0.f;
    }
    float sum = 0.f, top = 0.f;
#pragma unroll
    for (int w = 0; w < D / 32; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum += x[w][e];
        top = fmaxf(top, fabsf(x[w][e]));
      }
    Q.sum[ct] = group_sum(sum);
    if constexpr (F32) {
      top = group_max(top);
      const int e2 = (top > 0.f && top < INFINITY) ? ilogbf(top) : 0;
      Q.row_scale[ct] = ldexpf(1.f, e2);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        float y[8], rest[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = ldexpf(x[w][e], -e2);
        Q.hi[ct][w] = q_order(y);
        // what the first fp16 leaves, taken at the scale it was rounded at
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float f = (e & 1) ? 0.0625f : 1.f, inv = (e & 1) ? 16.f : 1.f;
          rest[e] = y[e] - (float)(_Float16)(y[e] * f) * inv;
        }
        Q.lo[ct][w] = q_order(rest);
      }
    } else {
#pragma unroll
      for (int w = 0; w < D / 32; ++w) Q.hi[ct][w] = q_order(x[w]);
    }
  }
}

// q . c (times 2^-24) of one 16-token tile for the lane's column and 4 tokens.
template <int D, int CT, bool F32>
__device__ __forceinline__ void tile_scores(float4v (&S)[CT], const Tile<D> &t,
                                            const Queries<D, CT, F32> &Q) {
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) S[ct] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    const half8 kf = k_frag<D>(t, w);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      S[ct] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, Q.hi[ct][w], S[ct], 0, 0, 0);
      if constexpr (F32)
        S[ct] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, Q.lo[ct][w], S[ct], 0, 0, 0);
    }
  }
  if constexpr (F32) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[ct][i] *= Q.row_scale[ct];
  }
}

// What a wave has summed for its rows.
template <int D, int CT>
struct Sums {
  float4v o[CT][D / 16];  // block 4h + j: channels 64h + 4 * (4g + reg) + j
  float m[CT], l[CT], z[CT];
};

template <int D, int CT, bool F32, bool MASK, bool STORE>
__device__ __forceinline__ void step(Sums<D, CT> &A, const Tile<D> (&T)[2],
                                     const Queries<D, CT, F32> &Q, const AttendArgs &a, int t,
                                     const int (&last)[CT], int len, float *const (&sc)[CT],
                                     int lane) {
  const int g = lane >> 4;
  float4v S[2][CT];
#pragma unroll
  for (int s = 0; s < 2; ++s) tile_scores<D, CT, F32>(S[s], T[s], Q);

  float top[CT];
  bool raise = false;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) top[ct] = kNegInf;
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Factors f = factors<D>(T[s], i, a.scale_log2);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        float x = S[s][ct][i] * f.ks + Q.sum[ct] * f.kz;
        if (MASK && t + 16 * s + 4 * g + i > last[ct]) x = kNegInf;
        S[s][ct][i] = x;
        top[ct] = fmaxf(top[ct], x + f.lv);
      }
    }
  if constexpr (STORE) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        if (sc[ct] != nullptr && t + 16 * s < len)
          *reinterpret_cast<float4v *>(sc[ct] + t + 16 * s + 4 * g) = S[s][ct];
  }
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) raise |= top[ct] > A.m[ct] + kSlack;
  if (__any(raise)) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      // each row by its own scores, so that no row depends on its neighbours
      const float t = group_max(top[ct]);
      const float m = t > A.m[ct] + kSlack ? t : A.m[ct];
      const float f = m == A.m[ct] ? 1.f : exp2f(A.m[ct] - m);
      A.m[ct] = m;
      A.l[ct] *= f;
      A.z[ct] *= f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) A.o[ct][d][i] *= f;
    }
  }
  half8 P[CT], Plo[F32 ? CT : 1];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Factors f = factors<D>(T[s], i, a.scale_log2);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const bool hidden = MASK && t + 16 * s + 4 * g + i > last[ct];
        // a masked token's factors may hold anything, NaN included
        const float p = hidden ? 0.f : __builtin_amdgcn_exp2f(S[s][ct][i] - A.m[ct]);
        A.l[ct] += p;
        A.z[ct] += hidden ? 0.f : p * f.vz;
        const float pv = hidden ? 0.f : p * f.vs;
        P[ct][4 * s + i] = (_Float16)pv;
        if constexpr (F32) Plo[ct][4 * s + i] = (_Float16)(pv - (float)(_Float16)pv);
      }
    }
#pragma unroll
  for (int hh = 0; hh < D / 64; ++hh) {
    half8 vf[4];  // by the channel's place in its four
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = T[e >> 1].v[2 * hh + (e & 1)], w8 = w >> 8;
      const half2v x[4] = {centred<0>(w), centred<1>(w), centred<0>(w8), centred<1>(w8)};
#pragma unroll
      for (int j = 0; j < 4; ++j) vf[j][2 * e] = x[j][0], vf[j][2 * e + 1] = x[j][1];
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4v &o = A.o[ct][4 * hh + j];
        o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[j], P[ct], o, 0, 0, 0);
        if constexpr (F32) o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[j], Plo[ct], o, 0, 0, 0);
      }
  }
}

__device__ __forceinline__ void store_out(const AttendArgs &a, int64_t at, float x, bool f32) {
  if (f32)
    static_cast<float *>(a.out)[at] = x;
  else
    static_cast<_Float16 *>(a.out)[at] = (_Float16)x;
}

__device__ __forceinline__ int64_t out_at(const AttendArgs &a, int b, int h, int row) {
  return b * a.os.batch + (row / a.G) * a.os.token + (int64_t)(h * a.G + row % a.G) * a.os.head;
}

// Grid: BH x splits x row_blocks workgroups, the cached head fastest (those of
// one head are 8 apart whenever BH is a multiple of 8, so they share an XCD's
// L2), the last rows first (they see the most tokens).
template <int D, int CT, int WT, bool F32, bool STORE>
__global__ __launch_bounds__(256) void attend_kernel(AttendArgs a, int splits, int row_blocks,
                                                     Ws ws) {
  constexpr int WR = 4 / WT;
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WT, wt = wave % WT;
  const int BH = a.c.B * a.c.H, R = a.n * a.G;
  const int bh = blockIdx.x % BH, rest = blockIdx.x / BH;
  const int split = rest % splits, rb = row_blocks - 1 - rest / splits;
  const int b = bh / a.c.H, h = bh % a.c.H;
  const int L = kv_len(a.c, b);
  const int row0 = (rb * WR + wr) * CT * 16;

  // tokens of these rows and of this split
  int tile_end = 0, tile_begin = 0, free_end = 0;
  if (row0 < R) {
    const int end_row = min(row0 + CT * 16, R) - 1;
    const int tiles = (max(0, L - a.n + end_row / a.G + 1) + 31) / 32;
    const int chunk = (tiles + splits - 1) / splits;
    tile_begin = split * chunk;
    tile_end = min(tiles, tile_begin + chunk);
    free_end = max(0, L - a.n + row0 / a.G + 1) / 32;  // tiles before it need no mask
  }

  Queries<D, CT, F32> Q;
  load_queries<D, CT, F32>(Q, a, b, h, row0, R, lane);
  Sums<D, CT> A;
  int last[CT];
  float *sc[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int row = row0 + ct * 16 + (lane & 15);
    last[ct] = L - a.n + min(row, R - 1) / a.G;
    sc[ct] = STORE && row < R ? ws.scores + ((int64_t)bh * R + row) * a.c.room() : nullptr;
    A.m[ct] = kNegInf;
    A.l[ct] = A.z[ct] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) A.o[ct][d] = float4v{0.f, 0.f, 0.f, 0.f};
  }

  int tile = tile_begin + wt;
  Tile<D> cur[2], nxt[2];
  auto load = [&](Tile<D>(&T)[2], int ti) {
    const int t = ti * 32;
    load_tile<D>(T[0], a.c, b, h, t, lane);
    load_tile<D>(T[1], a.c, b, h, t + 16 < L ? t + 16 : t, lane);
  };
  if (tile < tile_end) load(cur, tile);
  while (tile < tile_end) {
    const int next = tile + WT;
    load(nxt, next < tile_end ? next : tile);
    if (tile < free_end)
      step<D, CT, F32, false, STORE>(A, cur, Q, a, tile * 32, last, L, sc, lane);
    else
      step<D, CT, F32, true, STORE>(A, cur, Q, a, tile * 32, last, L, sc, lane);
    cur[0] = nxt[0];
    cur[1] = nxt[1];
    tile = next;
  }

  // a row's sums over its four lanes; the zeros added to the outputs
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    A.l[ct] = group_sum(A.l[ct]);
    A.z[ct] = group_sum(A.z[ct]);
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        A.o[ct][d][i] += A.z[ct];
  }

  if constexpr (WT > 1) {
    // the waves' rows are the same: join them in shared memory
    constexpr int N = CT * 16;
    __shared__ float so[WT][N][D + 4];
    __shared__ float sm[WT][N], sl[WT][N];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int col = ct * 16 + (lane & 15);
      if (g == 0) {
        sm[wt][col] = A.m[ct];
        sl[wt][col] = A.l[ct];
      }
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float4v x;
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = A.o[ct][4 * hh + j][i];
          *reinterpret_cast<float4v *>(&so[wt][col][64 * hh + 16 * g + 4 * i]) = x;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < N * D; e += 256) {
      const int col = e / D, d = e % D, row = row0 + col;
      if (row >= R) break;
      float m = sm[0][col], l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 1; w < WT; ++w) m = fmaxf(m, sm[w][col]);
#pragma unroll
      for (int w = 0; w < WT; ++w) {
        const float f = m == kNegInf ? 0.f : exp2f(sm[w][col] - m);
        l += f * sl[w][col];
        o += f * so[w][col][d];
      }
      if (splits == 1)
        store_out(a, out_at(a, b, h, row) + d, l == 0.f ? 0.f : o / l, F32);
      else
        ws.o[(((int64_t)split * BH + bh) * R + row) * D + d] = o;
      if (d == 0 && ws.ml != nullptr)
        ws.ml[((int64_t)split * BH + bh) * R + row] = make_float2(m, l);
    }
  } else {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int row = row0 + ct * 16 + (lane & 15);
      if (row >= R) continue;
      const int64_t part = ((int64_t)split * BH + bh) * R + row;
      if (g == 0 && ws.ml != nullptr) ws.ml[part] = make_float2(A.m[ct], A.l[ct]);
      const int64_t at = out_at(a, b, h, row);
      const float inv = A.l[ct] == 0.f ? 0.f : 1.f / A.l[ct];
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = 64 * hh + 16 * g + 4 * i + j;
            const float x = A.o[ct][4 * hh + j][i];
            if (splits == 1)
              store_out(a, at + d, A.l[ct] == 0.f ? 0.f : x * inv, F32);
            else
              ws.o[part * D + d] = x;
          }
    }
  }
}

// log2 of a row's sum of exponentials over all splits; +inf for a row that
// sees nothing, so that its probabilities come out as zero.
__device__ __forceinline__ float row_lse(const Ws &ws, int splits, int64_t stride, int64_t row) {
  float m = kNegInf;
  for (int s = 0; s < splits; ++s) m = fmaxf(m, ws.ml[s * stride + row].x);
  if (m == kNegInf) return INFINITY;
  float l = 0.f;
  for (int s = 0; s < splits; ++s) {
    const float2 x = ws.ml[s * stride + row];
    l += x.y * exp2f(x.x - m);
  }
  return m + log2f(l);
}

// Joins the splits (blocks [0, join)), one thread a channel, and adds the
// rows' probabilities to the weights from the stored scores (the other blocks,
// 1024 tokens each).
constexpr int kSumTokens = 1024;
template <int D>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs a, int splits, int join, bool f32,
                                                   Ws ws) {
  const int BH = a.c.B * a.c.H, R = a.n * a.G;
  const int64_t rows = (int64_t)BH * R;
  if ((int)blockIdx.x < join) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = e / D;
    const int d = e % D;
    if (row >= rows) return;
    float m = kNegInf;
    for (int s = 0; s < splits; ++s) m = fmaxf(m, ws.ml[s * rows + row].x);
    float l = 0.f, o = 0.f;
    if (m != kNegInf)
      for (int s = 0; s < splits; ++s) {
        const float2 x = ws.ml[s * rows + row];
        const float f = exp2f(x.x - m);
        l += f * x.y;
        o += f * ws.o[(s * rows + row) * D + d];
      }
    const int bh = (int)(row / R), r = (int)(row % R);
    store_out(a, out_at(a, bh / a.c.H, bh % a.c.H, r) + d, l == 0.f ? 0.f : o / l, f32);
    return;
  }
  __shared__ float lse[32];
  const int blk = blockIdx.x - join, bh = blk % BH;
  const int t = blk / BH * kSumTokens + threadIdx.x * 4;
  const int L = kv_len(a.c, bh / a.c.H);
  if (blk / BH * kSumTokens >= L) return;
  if ((int)threadIdx.x < R) lse[threadIdx.x] = row_lse(ws, splits, rows, (int64_t)bh * R + threadIdx.x);
  __syncthreads();
  if (t >= L) return;
  float4v sum = {0.f, 0.f, 0.f, 0.f};
  for (int r = 0; r < R; ++r) {
    const int seen = L - a.n + r / a.G;
    // tiles past the last token a row sees were not visited: nothing is stored
    if (t / 32 * 32 > seen) continue;
    const float4v s =
        *reinterpret_cast<const float4v *>(ws.scores + ((int64_t)bh * R + r) * a.c.room() + t);
    const float e = lse[r];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += t + i > seen ? 0.f : exp2f(s[i] - e);
  }
  float *w = a.weights + (int64_t)bh * a.c.room() + t;
  for (int i = 0; i < 4 && t + i < L; ++i) w[i] += sum[i];
}

// The weights of many rows: 32 tokens a workgroup, whose waves take turns over
// the row tiles and recompute the scores from the K codes; the sums stay in
// registers, so no atomics and a fixed order.
template <int D, bool F32>
__global__ __launch_bounds__(256) void weights_kernel(AttendArgs a, int splits, Ws ws) {
  __shared__ float part[4][32];
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int BH = a.c.B * a.c.H, R = a.n * a.G;
  const int64_t rows = (int64_t)BH * R;
  const int bh = blockIdx.x % BH, t = blockIdx.x / BH * 32;
  const int b = bh / a.c.H, h = bh % a.c.H;
  const int L = kv_len(a.c, b);
  if (t >= L) return;
  Tile<D> T[2];
  load_tile<D>(T[0], a.c, b, h, t, lane);
  load_tile<D>(T[1], a.c, b, h, t + 16 < L ? t + 16 : t, lane);
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  // the first query that sees token t
  const int first = max(0, t - (L - a.n)) * a.G / 16;
  for (int rt = first + wave; rt * 16 < R; rt += 4) {
    Queries<D, 1, F32> Q;
    load_queries<D, 1, F32>(Q, a, b, h, rt * 16, R, lane);
    const int row = rt * 16 + (lane & 15);
    const float lse = row < R ? row_lse(ws, splits, rows, (int64_t)bh * R + row) : INFINITY;
    const int last = row < R ? L - a.n + row / a.G : -1;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float4v S[1];
      tile_scores<D, 1, F32>(S, T[s], Q);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Factors f = factors<D>(T[s], i, a.scale_log2);
        const float x = S[0][i] * f.ks + Q.sum[0] * f.kz;
        sum[4 * s + i] +=
            t + 16 * s + 4 * g + i > last ? 0.f : __builtin_amdgcn_exp2f(x - lse);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int k = 1; k < 16; k <<= 1) sum[i] += __shfl_xor(sum[i], k);
    if ((lane & 15) == 0) part[wave][16 * (i >> 2) + 4 * g + (i & 3)] = sum[i];
  }
  __syncthreads();
  if (threadIdx.x < 32 && t + (int)threadIdx.x < L) {
    const int i = threadIdx.x;
    a.weights[(int64_t)bh * a.c.room() + t + i] +=
        part[0][i] + part[1][i] + (part[2][i] + part[3][i]);
  }
}

template <int D, int CT, int WT, bool F32>
void launch_attend(const AttendArgs &a, const AttendPlan &p, const Ws &ws, hipStream_t s) {
  const unsigned grid = (unsigned)a.c.B * a.c.H * p.splits * p.row_blocks;
  if constexpr (WT > 1) {
    if (p.scores) {
      attend_kernel<D, CT, WT, F32, true><<<grid, 256, 0, s>>>(a, p.splits, p.row_blocks, ws);
      return;
    }
  }
  attend_kernel<D, CT, WT, F32, false><<<grid, 256, 0, s>>>(a, p.splits, p.row_blocks, ws);
}

template <int D, bool F32>
hipError_t launch_dim(const AttendArgs &a, hipStream_t s) {
  const int BH = a.c.B * a.c.H, R = a.n * a.G, room = a.c.room();
  const AttendPlan p = attend_plan(a.c.B, a.c.H, D, room, a.n, a.G * a.c.H, a.weights != nullptr);
  char *w = static_cast<char *>(a.ws);
  Ws ws{};
  if (p.splits > 1 || a.weights != nullptr) ws.ml = reinterpret_cast<float2 *>(w);
  if (p.splits > 1) ws.o = reinterpret_cast<float *>(w + p.off_o);
  if (p.scores) ws.scores = reinterpret_cast<float *>(w + p.off_scores);
  if (p.wt == 4) {
    if (p.ct == 1)
      launch_attend<D, 1, 4, F32>(a, p, ws, s);
    else if constexpr (D <= 128)
      launch_attend<D, 2, 4, F32>(a, p, ws, s);
  } else {
    launch_attend<D, D <= 128 ? 2 : 1, 1, F32>(a, p, ws, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.splits > 1 || p.scores) {
    const int join = p.splits > 1 ? (int)(((int64_t)BH * R * D + 255) / 256) : 0;
    const int sums = p.scores ? BH * ((room + kSumTokens - 1) / kSumTokens) : 0;
    join_kernel<D><<<join + sums, 256, 0, s>>>(a, p.splits, join, F32, ws);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.weights != nullptr && !p.scores) {
    weights_kernel<D, F32><<<BH * ((room + 31) / 32), 256, 0, s>>>(a, p.splits, ws);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

AttendPlan attend_plan(int B, int H, int D, int room, int n, int q_heads, bool weights) {
  AttendPlan p{};
  const int64_t R = (int64_t)n * (q_heads / H), BH = (int64_t)B * H;
  // Up to 16 rows (32 up to 128 channels) a workgroup holds them all and its
  // waves share the tokens; more rows are spread over the waves.
  p.ct = D <= 128 && R > 16 ? 2 : 1;
  p.wt = R <= 16 * p.ct ? 4 : 1;
  const int block = p.ct * 16 * (4 / p.wt);
  p.row_blocks = (int)((R + block - 1) / block);
  const int64_t units = BH * p.row_blocks;
  // Enough workgroups for 256 compute units, none with less than one step of
  // 32 tokens a wave.
  const int64_t want = p.wt == 4 ? 1024 : 512, least = p.wt == 4 ? 128 : 256;
  int64_t splits = (want + units - 1) / units;
  const int64_t most = (room + least - 1) / least;
  splits = splits > most ? most : splits;
  p.splits = (int)(splits < 1 ? 1 : splits);
  p.scores = weights && p.wt == 4;
  const size_t rows = (size_t)(BH * R);
  size_t at = 0;
  if (p.splits > 1 || weights) at += rows * p.splits * sizeof(float2);
  at = (at + 255) / 256 * 256;
  p.off_o = at;
  if (p.splits > 1) at += rows * p.splits * D * sizeof(float);
  at = (at + 255) / 256 * 256;
  p.off_scores = at;
  if (p.scores) at += rows * (size_t)room * sizeof(float);
  p.bytes = at;
  return p;
}

hipError_t launch_kv_attend(const AttendArgs &a, int D, bcq_dtype dt, hipStream_t s) {
  if (dt == BCQ_F32)
    return D == 64    ? launch_dim<64, true>(a, s)
           : D == 128 ? launch_dim<128, true>(a, s)
                      : launch_dim<256, true>(a, s);
  return D == 64    ? launch_dim<64, false>(a, s)
         : D == 128 ? launch_dim<128, false>(a, s)
                    : launch_dim<256, false>(a, s);
}

}  // namespace bcq
