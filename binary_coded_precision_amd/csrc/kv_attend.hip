// kv_attend.hip -- attention over the 4-bit key/value cache (bcq_kv_attend); the
// mathematics and a wave's steps are in kv_tiles.h.
#include <algorithm>

#include "kv_tiles.h"

namespace bcq {
namespace {

using namespace kv;

struct Ws {
  float2 *ml;     // [splits][BH][R]: reference and sum of a row's exponentials; joined,
                  // [BH][R], for the weights of many rows
  float *o;       // [splits][BH][R][D]: outputs before the division
  float *scores;  // [BH][R][room], log2 units, -inf where masked
};

template <int D, int CT, bool F32>
__device__ __forceinline__ void fetch_queries(RawQueries<D, CT, F32> &raw, const AttendArgs &a,
                                              int b, int h, int row0, int R, int lane) {
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int row = min(row0 + ct * 16 + (lane & 15), R - 1);
    const int i = row / a.G, hq = h * a.G + row - i * a.G;
    const int64_t at = b * a.qs.batch + i * a.qs.token + hq * a.qs.head + (lane >> 4) * (D / 4);
    fetch_query<D, CT, F32>(raw, ct, a.q, at, a.q_wide);
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

// Waves a SIMD that the registers are held to: with few rows the loads' latency
// is what counts, and 4 waves (128 registers) hide more of it than 3.  The others
// need 113 to 256 registers, two waves at least.
constexpr int least_waves(int D, int CT, int WT, bool f32) {
  return WT == 4 && CT == 1 && D <= 128 && !f32 ? 4 : 2;
}

// The sequence of a given rank by length, the longest first (by index past 64
// sequences).
__device__ __forceinline__ int by_length(const KvView &c, int rank, int lane) {
  if (c.B == 1 || c.B > 64) return rank;
  const int mine = lane < c.B ? c.lens[lane] : INT32_MIN;
  int at = 0;
  for (int j = 0; j < c.B; ++j) {
    const int other = __builtin_amdgcn_readlane(mine, j);
    at += other > mine || (other == mine && j < lane);
  }
  return __builtin_ctzll(__ballot(lane < c.B && at == rank));
}

// Grid: BH x splits x row_blocks workgroups, the cached head fastest (those of
// one head are 8 apart whenever their number is a multiple of 8, so they share an
// XCD's L2).  WT waves take turns over the tokens of a workgroup's rows, and
// splits of a sequence start at different sequences, so that the compute unit
// that gets the same place of every split does not get one long sequence's share
// each time.  Or WR waves have rows of their own: then the sequences come by length
// and their last rows, which see the most tokens, first, as workgroups are handed
// out in order and the longest should not be left for last (2048 queries of
// two sequences over 6001 and 4501 tokens, on two workgroups a compute unit: 15%
// more in turns than by length).
//
// With few rows it is bound by the cache's bytes: 32 sequences of 4224 to 8192
// tokens, 8 cached heads of 128 channels (216 MB, and 25 MB of scores written)
// take 58 us, 4.2 TB/s.
// With many rows by the instructions that unpack codes and form probabilities:
// 2 x 2048 queries of 32 heads over 6001 and 4501 tokens take 460 us;
// their products alone would take 247 us at a library's fp16 rate.
template <int D, int CT, int WT, int WR, bool F32, bool STORE>
__global__ __launch_bounds__(64 * WT * WR, least_waves(D, CT, WT, F32)) void attend_kernel(
    AttendArgs a, int splits, int row_blocks, Ws ws) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / WT, wt = wave % WT;
  const int BH = a.c.B * a.c.H, R = a.n * a.G;
  const int h = blockIdx.x % a.c.H, rest = blockIdx.x / a.c.H;
  int b, split, rb;
  if constexpr (WT > 1) {
    split = rest / a.c.B % splits;
    rb = rest / a.c.B / splits;
    b = (rest % a.c.B + split * ((a.c.B + splits - 1) / splits)) % a.c.B;
  } else {
    const int rank = rest / (splits * row_blocks), at = rest - rank * splits * row_blocks;
    rb = row_blocks - 1 - at / splits;
    split = at % splits;
    b = __builtin_amdgcn_readfirstlane(by_length(a.c, rank, lane));
  }
  const int bh = b * a.c.H + h;
  const int row0 = (rb * WR + wr) * CT * 16;
  RawQueries<D, CT, F32> raw;
  fetch_queries<D, CT, F32>(raw, a, b, h, row0, R, lane);
  const int L = kv_len(a.c, b);

  // tokens of these rows and of this split
  int tile_end = 0, tile = 0, free_end = 0;
  if (row0 < R) {
    const int end_row = min(row0 + CT * 16, R) - 1;
    const int tiles = (max(0, L - a.n + end_row / a.G + 1) + 31) / 32;
    const int chunk = (tiles + splits - 1) / splits;
    tile = split * chunk + wt;
    tile_end = min(tiles, split * chunk + chunk);
    free_end = max(0, L - a.n + row0 / a.G + 1) / 32;  // tiles before it need no mask
  }
  Tiles<D> T;
  if (tile < tile_end) {
    const Where w = where(a.c, b, h, tile * 32, L);
    load_k(T, a.c, w, lane);
    load_m(T, a.c, w, lane);
    load_v(T, a.c, w, lane);
  }

  Queries<D, CT, F32> Q;
  load_queries<D, CT, F32>(Q, raw, a.unit, row0, R, lane);
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

  // the next tiles are asked for as soon as the registers of these are free, and
  // the place of those after them is looked up a step earlier still
  auto place_of = [&](int ti) { return where(a.c, b, h, (ti < tile_end ? ti : tile) * 32, L); };
  Where ahead{};
  if (tile < tile_end) ahead = place_of(tile + WT);
  while (tile < tile_end) {
    const int next = tile + WT;
    const Where w = ahead;
    ahead = place_of(next + WT);
    float4v S[2][CT];
    scores<D, CT, F32>(S, T, Q, a.code_unit);
    load_k(T, a.c, w, lane);
    if (tile >= free_end) mask_scores<D, CT>(S, T, A, tile * 32 + 4 * g, last);
    if constexpr (STORE) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          if (sc[ct] != nullptr && tile * 32 + 16 * s < L)
            *reinterpret_cast<float4v *>(sc[ct] + tile * 32 + 16 * s + 4 * g) = S[s][ct];
    }
    Frag P[CT], Plo[CT];
    softmax_tiles<D, CT>(A, P, Plo, S, T);
    load_m(T, a.c, w, lane);
    add_values<D, CT, F32>(A, P, Plo, T);
    load_v(T, a.c, w, lane);
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
        A.o[ct][d][i] = fmaf(A.o[ct][d][i], kCentreScale, A.z[ct]);
  }

  if constexpr (WT > 1) {
    // the waves' rows are the same: they meet in shared memory, then a wave joins
    // a row
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
      if (row0 + col < R)
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
    for (int col = wave; col < N && row0 + col < R; col += WT) {
      const int row = row0 + col;
      const float mw = lane < WT ? sm[lane][col] : kNegInf;
      float m = mw;
#pragma unroll
      for (int d = 1; d < WT; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
      const float f = mw == kNegInf ? 0.f : exp2f(mw - m);
      float l = lane < WT ? f * sl[lane][col] : 0.f;
#pragma unroll
      for (int d = 1; d < WT; d <<= 1) l += __shfl_xor(l, d);
      m = __shfl(m, 0);
      l = __shfl(l, 0);
      const int64_t part = ((int64_t)split * BH + bh) * R + row;
      const int64_t at = out_at(a, b, h, row);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < WT; ++w) o += __shfl(f, w) * so[w][col][c * 64 + lane];
        if (splits == 1)
          store_out(a, at + c * 64 + lane, l == 0.f ? 0.f : o / l, F32);
        else
          ws.o[part * D + c * 64 + lane] = o;
      }
      if (lane == 0 && ws.ml != nullptr) ws.ml[part] = make_float2(m, l);
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

constexpr int kMaxSplits = 64;  // one a lane where they are joined
// Tokens whose terms a wave sums in one go: what the matrix cores cut off at each
// addition grows with them.  Values that are all alike, the worst for it, come out
// 1.00 times as far off as fp16's rounding takes them over 2^16 tokens, up to
// 1.26 times over 2^17 and 2.6 over 2^20.
constexpr int64_t kMostTokens = 1 << 16;

// Splits of one row over the lanes of a wave: each split's factor against the
// row's largest reference (0 for lanes past them), the sum of exponentials, and
// that reference.
struct RowJoin {
  float f, l, m;
};
__device__ __forceinline__ RowJoin join_row(const Ws &ws, int splits, int64_t stride, int64_t row,
                                            int lane) {
  const float2 x =
      lane < splits ? ws.ml[lane * stride + row] : make_float2(kNegInf, 0.f);
  RowJoin j;
  j.m = x.x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) j.m = fmaxf(j.m, __shfl_xor(j.m, d));
  j.f = x.x == kNegInf ? 0.f : exp2f(x.x - j.m);
  j.l = x.y * j.f;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) j.l += __shfl_xor(j.l, d);
  return j;
}
// What a row's probabilities are made of: 2^(score - m) * inv, all zero for a row
// that sees nothing.  One number, m + log2(sum), would be rounded to a unit and
// more where scores are large.
__device__ __forceinline__ float2 normal_of(float m, float l) {
  return m == kNegInf ? make_float2(INFINITY, 0.f) : make_float2(m, 1.f / l);
}

// Joins the splits (blocks [0, join)), a wave a row, and adds the rows'
// probabilities to the weights from the stored scores (the other blocks, 1024
// tokens each).  Bound by reading both: 1024 rows and the weights of 8 heads of
// 32 sequences of 4224 to 8192 tokens (38 MB and the outputs) take 9.1 us.
constexpr int kSumTokens = 1024;
template <int D>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs a, int splits, int join, bool f32,
                                                   Ws ws) {
  const int BH = a.c.B * a.c.H, R = a.n * a.G;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t rows = (int64_t)BH * R;
  if ((int)blockIdx.x < join) {
    const int64_t row = (int64_t)blockIdx.x * 4 + wave;
    if (row >= rows) return;
    // the first splits' outputs are on their way while the factors are worked out
    constexpr int kAhead = 8;
    float early[kAhead][D / 64];
#pragma unroll
    for (int s = 0; s < kAhead; ++s)
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        early[s][c] = ws.o[(min(s, splits - 1) * rows + row) * D + c * 64 + lane];
    const RowJoin j = join_row(ws, splits, rows, row, lane);
    const int bh = (int)(row / R), r = (int)(row % R);
    const int64_t at = out_at(a, bh / a.c.H, bh % a.c.H, r);
    float o[D / 64] = {};
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const float f = s < splits ? __shfl(j.f, s) : 0.f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) o[c] += f * early[s][c];
    }
    for (int s0 = kAhead; s0 < splits; s0 += 4) {  // four splits' reads in flight
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int s = min(s0 + k, splits - 1);
        const float f = s0 + k < splits ? __shfl(j.f, s) : 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          o[c] += f * ws.o[(s * rows + row) * D + c * 64 + lane];
      }
    }
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store_out(a, at + c * 64 + lane, j.l == 0.f ? 0.f : o[c] / j.l, f32);
    // where no block of this launch reads it, for the weights formed afterwards
    if (lane == 0 && ws.scores == nullptr) ws.ml[row] = make_float2(j.m, j.l);
    return;
  }
  __shared__ float2 normal[32];
  const int blk = blockIdx.x - join, bh = blk % BH;
  const int t = blk / BH * kSumTokens + threadIdx.x * 4;
  const int L = kv_len(a.c, bh / a.c.H);
  if (blk / BH * kSumTokens >= L) return;
  // four rows' scores at a time in flight, the first of them and the weights while
  // the sums of exponentials are worked out (t is in the row for every thread:
  // rows have room for multiples of 16, this block's first token is one of them)
  const int tt = min(t, (L - 1) & ~3);
  auto fetch = [&](float4v(&s)[4], int r0) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      s[k] = *reinterpret_cast<const float4v *>(
          ws.scores + ((int64_t)bh * R + min(r0 + k, R - 1)) * a.c.room() + tt);
  };
  float4v s[4];
  fetch(s, 0);
  float4v *w = reinterpret_cast<float4v *>(a.weights + (int64_t)bh * a.c.room() + tt);
  const bool wide = ((uintptr_t)a.weights & 15) == 0 && t + 4 <= L;
  float4v was = {0.f, 0.f, 0.f, 0.f};
  if (wide) was = *w;
  for (int r = wave; r < R; r += 4) {
    const RowJoin j = join_row(ws, splits, rows, (int64_t)bh * R + r, lane);
    if (lane == 0) normal[r] = normal_of(j.m, j.l);
  }
  __syncthreads();
  if (t >= L) return;
  float4v sum = {0.f, 0.f, 0.f, 0.f};
  for (int r0 = 0; r0 < R; r0 += 4) {
    float4v next[4];
    if (r0 + 4 < R) fetch(next, r0 + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = min(r0 + k, R - 1);
      // nothing is stored in tiles past the last token that a row sees
      const int seen = r0 + k < R ? L - a.n + r / a.G : -1;
      const float2 e = normal[r];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float with = fmaf(__builtin_amdgcn_exp2f(s[k][i] - e.x), e.y, sum[i]);
        sum[i] = t + i > seen ? sum[i] : with;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = next[k];
  }
  if (wide) {
    *w = was + sum;
  } else {
    float *one = a.weights + (int64_t)bh * a.c.room() + t;
    for (int i = 0; i < 4 && t + i < L; ++i) one[i] += sum[i];
  }
}

// The weights of many rows: 32 TN tokens a workgroup, whose waves take turns over
// the row tiles and form the scores again from the K codes; the sums stay in
// registers, so no atomics and a fixed order.  A row tile's queries and factors
// cost more to bring in than 32 tokens' scores: they are asked for a tile ahead,
// and TN is 2, what the registers hold as unpacked codes up to 128 channels, where
// that leaves two workgroups for each compute unit.  2 x 2048 queries of 32 heads
// over 6001 and 4501 tokens (128 channels, 8 cached heads): 413 us; 462 without
// the tile ahead, 589 with TN = 1.  At 4 x 1000 over 1000 (64 channels) 27 us, 28
// with TN = 1 or 4.
template <int D, bool F32, int TN>
__global__ __launch_bounds__(256) void weights_kernel(AttendArgs a, Ws ws) {
  __shared__ float part[4][32 * TN];
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int BH = a.c.B * a.c.H, R = a.n * a.G;
  const int bh = blockIdx.x % BH, stride = gridDim.x / BH * 32 * TN;
  const int b = bh / a.c.H, h = bh % a.c.H;
  const int L = kv_len(a.c, b);
  for (int t = blockIdx.x / BH * 32 * TN; t < L; t += stride) {
    Tiles<D> T[TN];
#pragma unroll
    for (int k = 0; k < TN; ++k) {
      // tiles past the last token are the first one again, and not written
      const Where at = where(a.c, b, h, t + 32 * k < L ? t + 32 * k : t, L);
      load_k(T[k], a.c, at, lane);
      load_m(T[k], a.c, at, lane);
    }
    float sum[TN][8];
#pragma unroll
    for (int k = 0; k < TN; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[k][i] = 0.f;
    // the first query that sees token t
    const int first = max(0, t - (L - a.n)) * a.G / 16;
    // a row tile's queries and factors are asked for while the one before is summed
    RawQueries<D, 1, F32> raw;
    float2 ml{};
    auto ask = [&](int rt) {
      fetch_queries<D, 1, F32>(raw, a, b, h, rt * 16, R, lane);
      ml = ws.ml[(int64_t)bh * R + min(rt * 16 + (lane & 15), R - 1)];
    };
    if ((first + wave) * 16 < R) ask(first + wave);
    for (int rt = first + wave; rt * 16 < R; rt += 4) {
      Queries<D, 1, F32> Q;
      load_queries<D, 1, F32>(Q, raw, a.unit, rt * 16, R, lane);
      const int row = rt * 16 + (lane & 15);
      const int last = row < R ? L - a.n + row / a.G : -1;
      const float2 normal = normal_of(ml.x, ml.y);
      if ((rt + 4) * 16 < R) ask(rt + 4);
#pragma unroll
      for (int k = 0; k < TN; ++k)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float4v S[1];
          tile_scores<D, 1, F32>(S, T[k], s, Q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = score<F32>(S[0][i], Q.sum[0], T[k].m[s][2 * i], a.code_unit);
            float &to = sum[k][4 * s + i];
            const float with = fmaf(__builtin_amdgcn_exp2f(x - normal.x), normal.y, to);
            to = t + 32 * k + 16 * s + 4 * g + i > last ? to : with;
          }
        }
    }
#pragma unroll
    for (int k = 0; k < TN; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x = sum[k][i];
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) x += __shfl_xor(x, d);
        if ((lane & 15) == 0) part[wave][32 * k + 16 * (i >> 2) + 4 * g + (i & 3)] = x;
      }
    __syncthreads();
    if (threadIdx.x < 32 * TN && t + (int)threadIdx.x < L) {
      const int i = threadIdx.x;
      a.weights[(int64_t)bh * a.c.room() + t + i] +=
          part[0][i] + part[1][i] + (part[2][i] + part[3][i]);
    }
    __syncthreads();  // part is written again
  }
}

// Workgroups of 256 in a launch, whose work items are counted in 32 bits.
constexpr int kMaxGroups = (1 << 24) - 1;

// Tiles of rows that a wave holds when the waves have rows of their own.
constexpr int many_rows_ct(int D) { return D <= 128 ? 2 : 1; }

template <int D, int CT, int WT, int WR, bool F32>
void launch_attend(const AttendArgs &a, const AttendPlan &p, const Ws &ws, hipStream_t s) {
  const unsigned grid = (unsigned)a.c.B * a.c.H * p.splits * p.row_blocks;
  const int threads = 64 * WT * WR;
  if constexpr (WT > 1) {
    if (p.scores) {
      attend_kernel<D, CT, WT, WR, F32, true>
          <<<grid, threads, 0, s>>>(a, p.splits, p.row_blocks, ws);
      return;
    }
  }
  attend_kernel<D, CT, WT, WR, F32, false>
      <<<grid, threads, 0, s>>>(a, p.splits, p.row_blocks, ws);
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
  if (p.wt == 1)
    launch_attend<D, many_rows_ct(D), 1, 4, F32>(a, p, ws, s);
  else if (p.ct == 2) {
    if constexpr (D <= 128) launch_attend<D, 2, 4, 1, F32>(a, p, ws, s);
  } else {
    launch_attend<D, 1, 4, 1, F32>(a, p, ws, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.splits > 1 || p.scores) {
    const int join = p.splits > 1 ? (int)(((int64_t)BH * R + 3) / 4) : 0;
    const int sums = p.scores ? BH * ((room + kSumTokens - 1) / kSumTokens) : 0;
    join_kernel<D><<<join + sums, 256, 0, s>>>(a, p.splits, join, F32, ws);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.weights != nullptr && !p.scores) {
    // a launch's work items are counted in 32 bits: longer rows take turns
    constexpr int kTiles = D <= 128 ? 2 : 1;
    const int wide = (room + 32 * kTiles - 1) / (32 * kTiles), narrow = (room + 31) / 32;
    if ((int64_t)BH * wide >= 512)
      weights_kernel<D, F32, kTiles>
          <<<BH * std::min(wide, kMaxGroups / BH), 256, 0, s>>>(a, ws);
    else
      weights_kernel<D, F32, 1><<<BH * narrow, 256, 0, s>>>(a, ws);
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
  if (p.wt == 1) p.ct = many_rows_ct(D);
  const int block = p.ct * 16 * (p.wt == 1 ? 4 : 1);
  p.row_blocks = (int)((R + block - 1) / block);
  const int64_t units = BH * p.row_blocks;
  // Enough workgroups for 256 compute units, none with less than one step of
  // 32 tokens a wave, and no wave with more than kMostTokens unless there are more
  // rows than one launch can join.
  const int64_t want = p.wt == 4 ? 1024 : 512, least = p.wt == 4 ? 128 : 256;
  const int64_t most = (room + least - 1) / least;
  const int64_t few = (room + kMostTokens * p.wt - 1) / (kMostTokens * p.wt);
  int64_t splits = std::max(std::min((want + units - 1) / units, most), few);
  splits = std::min<int64_t>({splits, kMaxSplits, kMaxGroups / units});
  p.splits = BH * R > 4 * (int64_t)kMaxGroups ? 1 : (int)splits;
  p.scores = weights && p.wt != 1;
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

hipError_t launch_kv_attend(const AttendArgs &call, float scale, int D, bcq_dtype dt,
                            hipStream_t s) {
  // fp16 calls: up to 2^80 the scores of any queries and factors are finite, and a
  // scale that large already leaves nothing of any but the largest, whose
  // distance to the next is at least 2^-48 before it.  fp32 calls: see load_queries.
  AttendArgs a = call;
  if (dt == BCQ_F16) scale = fminf(fmaxf(scale, -0x1p80f), 0x1p80f);
  a.unit = fminf(fmaxf(scale * 1.44269504088896340736f, -FLT_MAX), FLT_MAX);
  a.code_unit = dt == BCQ_F16 ? a.unit * kCodeScale : 0.f;
  if (dt == BCQ_F32)
    return D == 64    ? launch_dim<64, true>(a, s)
           : D == 128 ? launch_dim<128, true>(a, s)
                      : launch_dim<256, true>(a, s);
  return D == 64    ? launch_dim<64, false>(a, s)
         : D == 128 ? launch_dim<128, false>(a, s)
                    : launch_dim<256, false>(a, s);
}

}  // namespace bcq
