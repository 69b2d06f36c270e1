// kv_tiles.h -- the steps of attention over the 4-bit key/value cache that its kernels
// share (kv_attend.hip, kv_packed.hip): 32 tokens against a wave's query rows.
//
// For a query row q (one of the n queries of one of the G query heads that
// share a cached head) and the cached vectors k_t = kz_t + ks_t * ck_t and
// v_t = vz_t + vs_t * cv_t with codes c in 0..15:
//
//   s_t = scale * (ks_t * (q . ck_t) + kz_t * sum(q))        (in log2 units here)
//   out = sum_t p_t v_t / sum_t p_t,  p_t = 2^(s_t - m)
//       = (sum_t (p_t vs_t) (cv_t - 7.5) + sum_t p_t (vz_t + 7.5 vs_t)) / sum_t p_t
//
// so both products run on the codes themselves, which fp16 holds exactly, and
// each token's four factors enter in fp32 afterwards.  A code c of K sits in an
// operand as the fp16 with bit pattern 16c, the subnormal c * 2^-20 (the matrix
// cores keep subnormal inputs), which takes a shift and an AND for two codes, and
// the queries of fp16 calls are the other operand as they are.
// Codes of V are centred: an average over many tokens is small against its
// terms, and what the terms' roundings leave would otherwise be multiplied by
// the 7.5 that the codes have in common, which the matrix cores' sums, cut off
// downwards at each addition (below), would show.
//
// Roundings below 32 bits: p_t * vs_t is held as the sum of two fp16, 22 bits
// relative to the row's largest (below), and for fp32 calls the queries are too
// (after a power of two for each row).  One fp16 for p_t * vs_t would add an error
// as large as an fp16 output's own rounding: 3.0e-4 to 3.4e-4 of the output's norm
// in all, against 2.1e-4 (and 2 x 2048 queries over 6001 and 4501 tokens would
// take 400 us, not 460).  As the matrix cores cut off
// what they add to a running sum, 1e-7 of it each time and always downwards
// (measured), fp32 calls start every product at zero and sum in ordinary fp32.
//
// The reference m of a row's exponentials is a maximum over s_t + log2(vs_t)
// (log2 to a tenth, from the fp16's bits) rather than over s_t: then p_t * vs_t
// stays within fp16's normal range around its largest whatever the scales of V
// are, and sum p_t in fp32 has room for the difference.  m is raised, and what
// is summed so far rescaled, only when a tile exceeds it by more than 2^6, so
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
#pragma once

#include <float.h>

#include "serve_internal.h"

namespace bcq {
namespace kv {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr float kNegInf = -INFINITY;
// A tile may exceed a row's reference by this many powers of two before what is
// summed is rescaled, and terms are held larger by kLift powers of two than that
// reference says: p_t * vs_t is about 2^9 at a row's largest and stays below 2^15.1
// in fp16, and what fp32 calls keep of its rounding is above fp16's smallest.
constexpr float kSlack = 6.f, kLift = 9.f;
constexpr float kRaise = 15.f + kLift;  // 15: the exponent's bias in the V scale's bits
constexpr int kCodeLog = 20;
constexpr float kCodeScale = 1 << kCodeLog;  // a code's subnormal back to the code

union Frag {
  uint32_t w[4];
  half2v p[4];
  half8 h;
};

// Two 16-token tiles as a lane holds them.
template <int D>
struct Tiles {
  uint32_t k[2][D / 32];  // its quarter of one token's K codes
  uint32_t v[2][D / 32];  // 4 tokens' codes of its D/16 channels
  uint32_t m[2][8];       // the 4 tokens' factors: (K scale, zero), (V scale, zero) each
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

// Where the two tiles of tokens t..t+31 lie.  The second is the first again where
// the sequence ends before it; an entry that names no page is never followed.
// The table is read through the scalar cache: as a vector load it would return
// behind the tiles asked for before it.
struct Where {
  int64_t at[2];
};
typedef const __attribute__((address_space(4))) int32_t *ScalarInts;
__device__ __forceinline__ Where where(const KvView &c, int b, int h, int t, int len) {
  const ScalarInts table = (ScalarInts)(uintptr_t)(c.table + (int64_t)b * c.max_pages);
  Where w;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int tok = __builtin_amdgcn_readfirstlane(t + 16 * s < len ? t + 16 * s : t);
    const int page = table[tok >> c.page_log];
    const int safe = (unsigned)page < (unsigned)c.num_pages ? page : 0;
    w.at[s] = (((int64_t)safe * c.H + h) << c.page_log) + (tok & ((1 << c.page_log) - 1));
  }
  return w;
}
template <int D>
__device__ __forceinline__ void load_k(Tiles<D> &t, const KvView &c, const Where &w, int lane) {
  const int off = (lane & 15) * (D / 2) + (lane >> 4) * (D / 8);
#pragma unroll
  for (int s = 0; s < 2; ++s) load_words(t.k[s], c.k + w.at[s] * (D / 2) + off);
}
template <int D>
__device__ __forceinline__ void load_v(Tiles<D> &t, const KvView &c, const Where &w, int lane) {
  const int off = (lane >> 4) * (2 * D) + (lane & 15) * (D / 8);
#pragma unroll
  for (int s = 0; s < 2; ++s) load_words(t.v[s], c.v + w.at[s] * (D / 2) + off);
}
template <int D>
__device__ __forceinline__ void load_m(Tiles<D> &t, const KvView &c, const Where &w, int lane) {
#pragma unroll
  for (int s = 0; s < 2; ++s)
    load_words(t.m[s],
               reinterpret_cast<const uint8_t *>(c.scales) + w.at[s] * 8 + (lane >> 4) * 32);
}

__device__ __forceinline__ half2v pair_of(uint32_t w) {
  union {
    uint32_t u;
    half2v h;
  } x;
  x.u = w;
  return x.h;
}

// Left operand of S^T for word w of a tile: channels 8w..8w+7 of the lane's
// quarter in the order 0 4 1 5 2 6 3 7.  All four bits up: with half of them as
// the subnormals c * 2^-24, which saves two of these shifts (448 against 456 us
// at 2 x 2048 queries over 6001 and 4501 tokens), their queries would have to carry 1/16,
// which fp16 does not hold of queries below 2^-10, and the matrix cores keep
// fewer bits of a product with a smaller subnormal (measured: 1e-6 of a sum of 32
// products with c * 2^-24, 2e-8 with c * 2^-20).
__device__ __forceinline__ half8 code_frag(uint32_t x) {
  Frag f;
  f.w[0] = (x << 4) & 0x00f000f0u;
  f.w[1] = x & 0x00f000f0u;
  f.w[2] = (x >> 4) & 0x00f000f0u;
  f.w[3] = (x >> 8) & 0x00f000f0u;
  return f.h;
}
template <int D>
__device__ __forceinline__ half8 k_frag(const Tiles<D> &t, int s, int w) {
  return code_frag(t.k[s][w]);
}

// (code - 7.5) / 512 of two tokens, the low (N = 0) or high nibbles of the bytes
// at the bottom of a word's halves: as subnormals c * 2^-24 or 16c * 2^-24, which
// one exact multiply-add takes to the centred value.
template <int N>
__device__ __forceinline__ half2v centred(uint32_t w) {
  const half2v x = pair_of(w & (N ? 0x00f000f0u : 0x000f000fu));
  const _Float16 up = (_Float16)(N ? 2048.f : 32768.f), mid = (_Float16)(-7.5f / 512.f);
  return __builtin_elementwise_fma(x, half2v{up, up}, half2v{mid, mid});
}
constexpr float kCentreScale = 512.f;

// Right operand of S^T: a query row's channels in k_frag's order.
__device__ __forceinline__ half8 q_order(const float (&x)[8]) {
  half8 f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = (_Float16)x[e];
    f[2 * e + 1] = (_Float16)x[e + 4];
  }
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
// quarter.  F32 holds each as two fp16 after taking a power of two out of the row.
template <int D, int CT, bool F32>
struct Queries {
  half8 hi[CT][D / 32];
  half8 lo[F32 ? CT : 1][F32 ? D / 32 : 1];
  float sum[CT];              // of the row, in the scores' unit
  float unit[F32 ? CT : 1];  // of a product with the codes, in the scores'
};

// The queries as they lie in memory: their loads can be under way long before
// what converts them.
template <int D, int CT, bool F32>
struct RawQueries {
  float4v f[F32 ? CT : 1][F32 ? D / 16 : 1];
  half8 h[F32 ? 1 : CT][F32 ? 1 : D / 32];
};
// The lane's row of tile ct: element `at` of q and on, 8 channels at once where
// `wide` says that they can be read so.
template <int D, int CT, bool F32>
__device__ __forceinline__ void fetch_query(RawQueries<D, CT, F32> &raw, int ct, const void *base,
                                            int64_t at, bool wide) {
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    if constexpr (F32) {
      const float *q = static_cast<const float *>(base) + at + w * 8;
      if (wide) {
        raw.f[ct][2 * w] = reinterpret_cast<const float4v *>(q)[0];
        raw.f[ct][2 * w + 1] = reinterpret_cast<const float4v *>(q)[1];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) raw.f[ct][2 * w + (e >> 2)][e & 3] = q[e];
      }
    } else {
      const _Float16 *q = static_cast<const _Float16 *>(base) + at + w * 8;
      if (wide) {
        raw.h[ct][w] = *reinterpret_cast<const half8 *>(q);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) raw.h[ct][w][e] = q[e];
      }
    }
  }
}

// Rows past R become zeros: a tile's spare columns.
template <int D, int CT, bool F32>
__device__ __forceinline__ void load_queries(Queries<D, CT, F32> &Q,
                                             const RawQueries<D, CT, F32> &raw, float unit,
                                             int row0, int R, int lane) {
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int row = row0 + ct * 16 + (lane & 15);
    float x[D / 32][8];
#pragma unroll
    for (int w = 0; w < D / 32; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (F32)
          x[w][e] = raw.f[ct][2 * w + (e >> 2)][e & 3];
        else
          x[w][e] = (float)raw.h[ct][w][e];
        if (row >= R) x[w][e] = 0.f;
      }
    float sum = 0.f;
    if constexpr (F32) {
      float top = 0.f;
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[w][e]));
      top = group_max(top);
      // the largest to 2^10..2^11: what the first fp16 leaves stays a normal one
      const int e2 = (top > 0.f && top < INFINITY) ? ilogbf(top) - 10 : 0;
      // scores are finite up to here, and rows of this size have nothing but their
      // largest left long before
      constexpr float kMost = 0x1p100f;
      Q.unit[ct] = fminf(fmaxf(ldexpf(unit, e2 + kCodeLog), -kMost), kMost);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        float y[8], rest[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] = ldexpf(x[w][e], -e2);
          sum += y[e];
          rest[e] = y[e] - (float)(_Float16)y[e];
        }
        Q.hi[ct][w] = q_order(y);
        Q.lo[ct][w] = q_order(rest);
      }
      Q.sum[ct] = group_sum(sum) * (Q.unit[ct] * (1.f / kCodeScale));
    } else {
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += x[w][e];
        Q.hi[ct][w] = q_order(x[w]);
      }
      Q.sum[ct] = group_sum(sum) * unit;
    }
  }
}

// q . c of one 16-token tile for the lane's column and 4 tokens: times 2^-20, in
// fp32 calls times the scores' unit.
template <int D, int CT, bool F32>
__device__ __forceinline__ void tile_scores(float4v (&S)[CT], const Tiles<D> &t, int s,
                                            const Queries<D, CT, F32> &Q) {
  const float4v zero = {0.f, 0.f, 0.f, 0.f};
  float4v low[F32 ? CT : 1];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    S[ct] = zero;
    if constexpr (F32) low[ct] = zero;
  }
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    const half8 kf = k_frag<D>(t, s, w);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      if constexpr (F32) {
        low[ct] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, Q.lo[ct][w], low[ct], 0, 0, 0);
        S[ct] += __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, Q.hi[ct][w], zero, 0, 0, 0);
      } else {
        S[ct] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, Q.hi[ct][w], S[ct], 0, 0, 0);
      }
    }
  }
  if constexpr (F32) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) S[ct] = (S[ct] + low[ct]) * Q.unit[ct];
  }
}

// What a wave has summed for its rows.
template <int D, int CT>
struct Sums {
  float4v o[CT][D / 16];  // block 4h + j: channels 64h + 4 * (4g + reg) + j
  float m[CT], l[CT], z[CT];
};

// A score in log2 units, rounded as such: ks * (q . c) + kz * sum(q).  What goes
// into an exponential is then a difference of two such numbers, which is exact
// where it matters; scale * score - reference in one multiply-add would leave
// the rounding of a large reference in it.
template <bool F32>
__device__ __forceinline__ float score(float qc, float sum, uint32_t m, float code_unit) {
  const half2v f = pair_of(m);
  return fmaf(qc, F32 ? (float)f[0] : (float)f[0] * code_unit, sum * (float)f[1]);
}

template <int D, int CT, bool F32>
__device__ __forceinline__ void scores(float4v (&S)[2][CT], const Tiles<D> &T,
                                       const Queries<D, CT, F32> &Q, float code_unit) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    tile_scores<D, CT, F32>(S[s], T, s, Q);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        S[s][ct][i] = score<F32>(S[s][ct][i], Q.sum[ct], T.m[s][2 * i], code_unit);
  }
}

__device__ __forceinline__ bool not_finite(uint32_t w) {
  return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
}

// Scores of the tokens past each row's last to -inf.  Factors of V that are not
// finite would reach hidden rows as 0 * NaN: they become 0, and what a row that
// does see them has summed of the zeros NaN, which its output is made with; its
// probabilities do not depend on V.
template <int D, int CT>
__device__ __forceinline__ void mask_scores(float4v (&S)[2][CT], Tiles<D> &T, Sums<D, CT> &A,
                                            int t, const int (&last)[CT]) {
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // opaque here, so that the compiler leaves the test in this branch
      asm volatile("" : "+v"(T.m[s][2 * i + 1]));
      const bool bad = not_finite(T.m[s][2 * i + 1]);
      T.m[s][2 * i + 1] = bad ? 0u : T.m[s][2 * i + 1];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const bool hidden = t + 16 * s + i > last[ct];
        S[s][ct][i] = hidden ? kNegInf : S[s][ct][i];
        A.z[ct] = bad && !hidden ? NAN : A.z[ct];
      }
    }
}

// log2 of an fp16 from its bits, to a tenth, plus 15 (the exponent's bias).
__device__ __forceinline__ float rough_log2(uint32_t half) { return (float)half * (1.f / 1024.f); }

__device__ __forceinline__ ushort2v pair16(uint32_t w) {
  union {
    uint32_t u;
    ushort2v h;
  } x;
  x.u = w;
  return x.h;
}

__device__ __forceinline__ half2v cut(float a, float b) {
  return __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_pkrtz(a, b));
}

// Raises the reference of the row of tile ct where its largest term z asks for it (each
// row by its own scores, so that no row depends on its neighbours) and rescales; `high`
// is the largest score of the lane.
template <int D, int CT>
__device__ __forceinline__ void raise_row(Sums<D, CT> &A, int ct, float z, float high) {
  float m = z > A.m[ct] + (kRaise + kSlack) ? z - kRaise : A.m[ct];
  // Scores so large that such sums are rounded to units and more: the largest
  // itself is the reference.  Terms are then at most the V scales.
  const bool vast = fabsf(z) >= 0x1p22f && fabsf(z) < INFINITY;
  if (__any(vast)) {
    const float most = group_max(high);
    m = vast ? fmaxf(A.m[ct], most) : m;
  }
  const float f = m == A.m[ct] ? 1.f : exp2f(A.m[ct] - m);
  A.m[ct] = m;
  A.l[ct] *= f;
  A.z[ct] *= f;
#pragma unroll
  for (int d = 0; d < D / 16; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) A.o[ct][d][i] *= f;
}

// The softmax's step over 32 tokens: raises the rows' references, rescales, adds
// to their sums and leaves probability times V scale in P, what that rounds off in
// Plo.
template <int D, int CT>
__device__ __forceinline__ void softmax_tiles(Sums<D, CT> &A, Frag (&P)[CT], Frag (&Plo)[CT],
                                              const float4v (&S)[2][CT], const Tiles<D> &T) {
  // The tile's largest score and largest V scale together bound its terms; only
  // where that asks for it are the terms themselves looked at.
  ushort2v scales = pair16(T.m[0][1]);
  float high[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) high[ct] = S[0][ct][0];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      scales = __builtin_elementwise_max(scales, pair16(T.m[s][2 * i + 1]));
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) high[ct] = fmaxf(high[ct], S[s][ct][i]);
    }
  const float room = kRaise + kSlack - rough_log2((uint32_t)scales[0]);
  bool raise = false;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) raise |= high[ct] - A.m[ct] > room;
  if (__any(raise)) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      float top = kNegInf;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = fmaxf(top, S[s][ct][i] + rough_log2(T.m[s][2 * i + 1] & 0xffffu));
      raise_row(A, ct, group_max(top), high[ct]);
    }
  }
  // a row that has seen nothing yet has no reference; its terms are 2^-inf
  float m[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) m[ct] = fmaxf(A.m[ct], -3.0e38f);
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      half2v f[2];
      float mid[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f[j] = pair_of(T.m[s][2 * (i + j) + 1]);
        mid[j] = fmaf(7.5f, (float)f[j][0], (float)f[j][1]);
      }
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        float pv[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float p = __builtin_amdgcn_exp2f(S[s][ct][i + j] - m[ct]);
          A.l[ct] += p;
          A.z[ct] = fmaf(p, mid[j], A.z[ct]);
          pv[j] = p * (float)f[j][0];
        }
        // in pairs, cut off rather than rounded: what is left goes to Plo either way
        const half2v part = cut(pv[0], pv[1]);
        P[ct].p[2 * s + (i >> 1)] = part;
        Plo[ct].p[2 * s + (i >> 1)] = cut(pv[0] - (float)part[0], pv[1] - (float)part[1]);
      }
    }
}

// Channels 64hh .. 64hh + 63 of the outputs, from 32 tokens' V by the channel's place in
// its four.
template <int D, int CT, bool F32>
__device__ __forceinline__ void add_block(Sums<D, CT> &A, const Frag (&P)[CT],
                                          const Frag (&Plo)[CT], const half8 (&vf)[4], int hh) {
  if constexpr (F32) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4v x = {0.f, 0.f, 0.f, 0.f};
        x = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[j], Plo[ct].h, x, 0, 0, 0);
        A.o[ct][4 * hh + j] += __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[j], P[ct].h, x, 0, 0, 0);
      }
  } else {
    // no product waits for the one before it
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float4v &o = A.o[ct][4 * hh + j];
          const half8 p = part ? P[ct].h : Plo[ct].h;
          o = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[j], p, o, 0, 0, 0);
        }
  }
}

template <int D, int CT, bool F32>
__device__ __forceinline__ void add_values(Sums<D, CT> &A, const Frag (&P)[CT],
                                           const Frag (&Plo)[CT], const Tiles<D> &T) {
#pragma unroll
  for (int hh = 0; hh < D / 64; ++hh) {
    half8 vf[4];  // by the channel's place in its four
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = T.v[e >> 1][2 * hh + (e & 1)], w8 = w >> 8;
      const half2v x[4] = {centred<0>(w), centred<1>(w), centred<0>(w8), centred<1>(w8)};
#pragma unroll
      for (int j = 0; j < 4; ++j) vf[j][2 * e] = x[j][0], vf[j][2 * e + 1] = x[j][1];
    }
    add_block<D, CT, F32>(A, P, Plo, vf, hh);
  }
}

}  // namespace kv
}  // namespace bcq
