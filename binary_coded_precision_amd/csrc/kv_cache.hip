// kv_cache.hip -- what fills, reads back and shrinks the 4-bit key/value cache
// (bcq_kv_append, bcq_kv_read, bcq_kv_evict).
//
// A vector of D channels (one token's K or V of one cached head) is
// zero + scale * code: zero = fp16(min), scale = fp16((max - min) * (1/15)),
// code = rint((x - zero) / scale) held to 0..15, each step rounded to fp32 (the
// constant too), so the codes are a function of the inputs alone.
#include "serve_internal.h"

namespace bcq {
namespace {

struct __attribute__((aligned(8))) Half4 {
  _Float16 x[4];
};

// D/4 lanes hold a vector, 4 consecutive channels each.  Lane i's two bytes of
// codes are bytes 2i, 2i+1 of a K row; in a block of 4 tokens of V they are one
// 16-bit unit: row i % 16, channel block i / 16.
template <int D>
__device__ __forceinline__ int64_t k_byte(int64_t token, int i) {
  return token * (D / 2) + i * 2;
}
template <int D>
__device__ __forceinline__ int64_t v_byte(int64_t token, int i) {
  return (token & ~(int64_t)3) * (D / 2) + (i & 15) * (D / 8) + (i >> 4) * 8 + (token & 3) * 2;
}

// NaN wins, as a vector holding one cannot be represented.
__device__ __forceinline__ float nan_min(float a, float b) { return (a < b || a != a) ? a : b; }
__device__ __forceinline__ float nan_max(float a, float b) { return (a > b || a != a) ? a : b; }

template <typename T, bool VEC>
__device__ __forceinline__ void load4(float (&x)[4], const T *p) {
  if constexpr (VEC && sizeof(T) == 2) {
    const Half4 h = *reinterpret_cast<const Half4 *>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (float)h.x[e];
  } else if constexpr (VEC) {
    const float4 f = *reinterpret_cast<const float4 *>(p);
    x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (float)p[e];
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store4(T *p, const float (&x)[4]) {
  if constexpr (VEC && sizeof(T) == 2) {
    Half4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h.x[e] = (_Float16)x[e];
    *reinterpret_cast<Half4 *>(p) = h;
  } else if constexpr (VEC) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = (T)x[e];
  }
}

// Vector `vec` of a call over n tokens: K and V of (sequence, token, head), V last.
struct Place {
  int b, i, h, slot;
  bool v;
};
__device__ __forceinline__ Place place(const KvView &c, int n, uint32_t vec) {
  Place p;
  p.v = vec & 1;
  const uint32_t at = (vec >> 1) / (uint32_t)c.H;
  p.h = (int)((vec >> 1) - at * (uint32_t)c.H);
  p.b = (int)(at / (uint32_t)n);
  p.i = (int)(at - (uint32_t)p.b * (uint32_t)n);
  p.slot = kv_len(c, p.b) - n + p.i;
  return p;
}

// Bound by the bytes of the vectors read; every lane converts what it loads,
// the extremes meet in D/4 lanes and no shared memory is needed.
template <int D, typename T, bool VEC>
__global__ __launch_bounds__(256) void append_kernel(KvView c, int n, const T *k, KvStrides ks,
                                                     const T *v, KvStrides vs,
                                                     const int32_t *positions, float *weights,
                                                     int32_t *pos, uint32_t vecs) {
  constexpr int L = D / 4;
  const uint32_t vec = blockIdx.x * (256 / L) + threadIdx.x / L;
  const int i = threadIdx.x % L;
  if (vec >= vecs) return;  // whole groups of L lanes leave together
  const Place p = place(c, n, vec);
  const KvStrides st = p.v ? vs : ks;
  const T *src = (p.v ? v : k) + p.b * st.batch + p.i * st.token + p.h * st.head + i * 4;
  float x[4];
  load4<T, VEC>(x, src);
  float lo = nan_min(nan_min(x[0], x[1]), nan_min(x[2], x[3]));
  float hi = nan_max(nan_max(x[0], x[1]), nan_max(x[2], x[3]));
#pragma unroll
  for (int d = 1; d < L; d <<= 1) {
    lo = nan_min(lo, __shfl_xor(lo, d));
    hi = nan_max(hi, __shfl_xor(hi, d));
  }
  float step = (hi - lo) * (1.f / 15.f);
  asm volatile("" : "+v"(step));  // rounded to fp32 first: one instruction could do both at once
  const _Float16 zh = (_Float16)lo, sh = (_Float16)step;
  const float zero = (float)zh, scale = (float)sh;
  uint32_t word = 0;
  // the quotient's neighbour y * (1 / scale) is less than 1e-5 off it and rounds
  // to the same integer unless it lies that close to a half
  const float inv = scale > 0.f ? 1.f / scale : 0.f;
  float q[4];
  bool near = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float y = (x[e] - zero) * inv;
    q[e] = rintf(y);
    near |= !(fabsf(y - q[e]) < 0.4999f);
  }
  if (__builtin_expect(near, 0) && scale > 0.f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = rintf((x[e] - zero) / scale);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    word |= (scale > 0.f ? (uint32_t)fminf(fmaxf(q[e], 0.f), 15.f) : 0u) << (4 * e);
  if (p.slot < 0) return;
  const int64_t token = kv_token(c, p.b, p.h, p.slot);
  if (token < 0) return;
  *reinterpret_cast<uint16_t *>(p.v ? c.v + v_byte<D>(token, i) : c.k + k_byte<D>(token, i)) =
      (uint16_t)word;
  if (i == 0) {
    union {
      _Float16 h[2];
      uint32_t u;
    } m;
    m.h[0] = sh;
    m.h[1] = zh;
    *reinterpret_cast<uint32_t *>(c.scales + token * 4 + (p.v ? 2 : 0)) = m.u;
    if (!p.v) {
      const int64_t at = ((int64_t)p.b * c.H + p.h) * c.room() + p.slot;
      if (weights != nullptr) weights[at] = 0.f;
      if (pos != nullptr)
        pos[at] = positions != nullptr ? positions[(int64_t)p.b * n + p.i] : p.slot;
    }
  }
}

template <int D, typename T, bool VEC>
__global__ __launch_bounds__(256) void read_kernel(KvView c, int n, T *k, KvStrides ks, T *v,
                                                   KvStrides vs, uint32_t vecs) {
  constexpr int L = D / 4;
  const uint32_t vec = blockIdx.x * (256 / L) + threadIdx.x / L;
  const int i = threadIdx.x % L;
  if (vec >= vecs) return;
  const Place p = place(c, n, vec);
  const KvStrides st = p.v ? vs : ks;
  T *dst = (p.v ? v : k) + p.b * st.batch + p.i * st.token + p.h * st.head + i * 4;
  const int64_t token = p.slot < 0 ? -1 : kv_token(c, p.b, p.h, p.slot);
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (token >= 0) {
    const uint32_t word = *reinterpret_cast<const uint16_t *>(
        p.v ? c.v + v_byte<D>(token, i) : c.k + k_byte<D>(token, i));
    union {
      uint32_t u;
      _Float16 h[2];
    } m;
    m.u = *reinterpret_cast<const uint32_t *>(c.scales + token * 4 + (p.v ? 2 : 0));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = (float)m.h[1] + (float)m.h[0] * (float)((word >> (4 * e)) & 15u);
  }
  store4<T, VEC>(dst, x);
}

bool vec_ok(const void *p, KvStrides s, size_t size) {
  return (uintptr_t)p % (4 * size) == 0 && s.batch % 4 == 0 && s.token % 4 == 0 &&
         s.head % 4 == 0;
}

template <int D, typename T>
hipError_t append_dim(const KvView &c, int n, const void *k, KvStrides ks, const void *v,
                      KvStrides vs, const int32_t *positions, float *weights, int32_t *pos,
                      hipStream_t s) {
  const uint32_t vecs = (uint32_t)c.B * n * c.H * 2, per = 256 / (D / 4);
  const uint32_t grid = (vecs + per - 1) / per;
  if (vec_ok(k, ks, sizeof(T)) && vec_ok(v, vs, sizeof(T)))
    append_kernel<D, T, true><<<grid, 256, 0, s>>>(c, n, (const T *)k, ks, (const T *)v, vs,
                                                   positions, weights, pos, vecs);
  else
    append_kernel<D, T, false><<<grid, 256, 0, s>>>(c, n, (const T *)k, ks, (const T *)v, vs,
                                                    positions, weights, pos, vecs);
  return hipGetLastError();
}

template <int D, typename T>
hipError_t read_dim(const KvView &c, int n, void *k, KvStrides ks, void *v, KvStrides vs,
                    hipStream_t s) {
  const uint32_t vecs = (uint32_t)c.B * n * c.H * 2, per = 256 / (D / 4);
  const uint32_t grid = (vecs + per - 1) / per;
  if (vec_ok(k, ks, sizeof(T)) && vec_ok(v, vs, sizeof(T)))
    read_kernel<D, T, true><<<grid, 256, 0, s>>>(c, n, (T *)k, ks, (T *)v, vs, vecs);
  else
    read_kernel<D, T, false><<<grid, 256, 0, s>>>(c, n, (T *)k, ks, (T *)v, vs, vecs);
  return hipGetLastError();
}

// ---- eviction
//
// Each (sequence, cached head) keeps its own tokens: the `recent` newest by
// position, then those of the largest accumulated weight, the lower slot first
// among equals.  Kept tokens already in front stay where they are and the i-th
// evicted slot in front takes the i-th kept token from behind, so that what
// moves is the least possible and no move reads what another writes.

// Order of a slot: recent tokens above every weight, NaN below every weight.
__device__ __forceinline__ uint32_t order_of(float w, bool late) {
  if (late) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kEvictThreads = 1024, kEvictWaves = kEvictThreads / 64;
constexpr int kCopies = 16;  // of the histogram, so that lanes rarely meet in a counter

struct EvictArgs {
  KvView c;
  int keep, recent;
  const float *weights;
  const int32_t *pos;
  int32_t *lens_out;
  float *weights_out;
  int32_t *pos_out;
  int32_t *count;  // [BH] moves
  int2 *moves;     // [BH][most]: (from, to)
  int most;
};

// Set bits of a ballot below the lane.
__device__ __forceinline__ uint32_t below(uint64_t ballot) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(ballot >> 32),
                                   __builtin_amdgcn_mbcnt_lo((uint32_t)ballot, 0));
}

// One workgroup a row.  A wave has 256 Q slots in a row, a thread the orders of 4 Q
// of them in registers, slot 256 q + 4 lane + e of the wave's, so that reads are
// wide and coalesced; rows with room for more than the workgroup holds (ONCE is
// false) go through all steps in rounds, which read weights and positions again.
// A radix select over the orders, eight bits a pass, finds the last one kept and
// ends early where a whole bin is; ballots then number what moves in slot order.
template <int Q, bool ONCE>
__global__ __launch_bounds__(kEvictThreads) void select_kernel(EvictArgs a) {
  constexpr int kRound = 4 * Q * kEvictThreads;
  __shared__ uint32_t hist[256 * kCopies];
  __shared__ uint32_t total[256];
  __shared__ int tmp[kEvictWaves];
  __shared__ uint32_t sums[3][kEvictWaves];
  __shared__ uint32_t picked, above, inside;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = blockIdx.x, b = row / a.c.H;
  const int64_t at = (int64_t)row * a.c.room();
  const int L = kv_len(a.c, b), m = min(L, a.keep);
  const int end = ONCE ? 1 : L;  // of the rounds' first slots
  const float *w = a.weights + at;
  const int32_t *pos = a.pos + at;
  const int first = wave * 256 * Q + lane * 4;  // of the thread's slots, in a round

  // Rows start at multiples of 16 slots and end at one, so a read of 4 from a
  // multiple of 4 below L stays in its row.
  int newest = INT32_MIN;
  for (int s0 = first; s0 < end + first; s0 += kRound) {
    int4 v[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (s0 + 256 * q < L) v[q] = *reinterpret_cast<const int4 *>(pos + s0 + 256 * q);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int s = s0 + 256 * q;
      if (s < L) newest = max(newest, v[q].x);
      if (s + 1 < L) newest = max(newest, v[q].y);
      if (s + 2 < L) newest = max(newest, v[q].z);
      if (s + 3 < L) newest = max(newest, v[q].w);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) newest = max(newest, __shfl_xor(newest, d));
  if (lane == 0) tmp[wave] = newest;
  for (int i = tid; i < 256 * kCopies; i += kEvictThreads) hist[i] = 0;
  __syncthreads();
  for (int i = 0; i < kEvictWaves; ++i) newest = max(newest, tmp[i]);
  const int64_t late_from = (int64_t)newest - a.recent;

  // The orders of the round whose slots start at s0 for this thread.  On the
  // way what is in front goes to the output; what is evicted of it is
  // overwritten by the moves.
  uint32_t key[Q][4];
  auto orders = [&](int s0, bool write) {
    float4 x[Q];
    int4 y[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (s0 + 256 * q < L) {
        x[q] = *reinterpret_cast<const float4 *>(w + s0 + 256 * q);
        y[q] = *reinterpret_cast<const int4 *>(pos + s0 + 256 * q);
      }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float xs[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
      const int32_t ys[4] = {y[q].x, y[q].y, y[q].z, y[q].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int s = s0 + 256 * q + e;
        key[q][e] = order_of(xs[e], ys[e] > late_from);
        if (write && s < m) {
          a.weights_out[at + s] = xs[e];
          a.pos_out[at + s] = ys[e];
        }
      }
    }
  };
  const bool apart = a.weights_out != a.weights || a.pos_out != a.pos;
  if (ONCE)
    orders(first, apart);
  else if (apart)
    for (int s0 = first; s0 < end + first; s0 += kRound) orders(s0, true);
  if (L <= a.keep) {
    if (tid == 0) a.count[row] = 0;
    return;
  }

  uint32_t prefix = 0;
  int left = m;  // still to be taken among the slots whose order starts with prefix
  int shift = 24;
  for (;; shift -= 8) {
    for (int s0 = first; s0 < end + first; s0 += kRound) {
      if (!ONCE) orders(s0, false);
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t k = key[q][e];
          if (s0 + 256 * q + e < L &&
              (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))))
            atomicAdd(&hist[((k >> shift) & 255u) * kCopies + (lane & (kCopies - 1))], 1u);
        }
    }
    __syncthreads();
    {
      // 4 threads a bin, which also clear the counters for the next pass
      uint4 *h = reinterpret_cast<uint4 *>(hist) + tid;
      const uint4 x = *h;
      uint32_t t = x.x + x.y + x.z + x.w;
      *h = make_uint4(0, 0, 0, 0);
      t += __shfl_xor(t, 1);
      t += __shfl_xor(t, 2);
      if ((tid & 3) == 0) total[tid >> 2] = t;
    }
    __syncthreads();
    if (wave == 0) {
      // lane l sums bins 4l..4l+3; the bin where the count from the top passes `left`
      uint32_t t[4], sum = 0;
      for (int i = 0; i < 4; ++i) sum += t[i] = total[lane * 4 + i];
      uint32_t up = sum;  // of this lane's bins and all above
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_down(up, d);
        if (lane + d < 64) up += o;
      }
      uint32_t over = up - sum;
      for (int i = 3; i >= 0; --i) {
        if (over < (uint32_t)left && over + t[i] >= (uint32_t)left) {
          picked = lane * 4 + i;
          above = over;
          inside = t[i];
        }
        over += t[i];
      }
    }
    __syncthreads();
    prefix |= picked << shift;
    left -= (int)above;
    if (shift == 0 || (int)inside == left) break;
  }

  // kept: every order above prefix's leading bits, and the first `left` slots at them
  const uint32_t edge = prefix >> shift;
  int2 *mv = a.moves + (int64_t)row * a.most;
  uint32_t ties = 0, holes = 0, fills = 0;  // before this round
  for (int s0 = first; s0 < end + first; s0 += kRound) {
    if (!ONCE) orders(s0, false);
    uint32_t n = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        n += __popcll(__ballot(s0 + 256 * q + e < L && (key[q][e] >> shift) == edge));
    if (lane == 0) sums[0][wave] = n;
    __syncthreads();
    uint32_t tie = ties;
    for (int i = 0; i < kEvictWaves; ++i) {
      const uint32_t x = sums[0][i];
      tie += i < wave ? x : 0;
      ties += x;
    }
    uint32_t hole = 0, fill = 0;  // 4 bits a q
    uint32_t n_holes = 0, n_fills = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      uint64_t eq[4];
      uint32_t before = tie;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        eq[e] = __ballot(s0 + 256 * q + e < L && (key[q][e] >> shift) == edge);
        before += below(eq[e]);
        tie += __popcll(eq[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int s = s0 + 256 * q + e;
        const uint32_t k = key[q][e] >> shift;
        const bool same = k == edge;
        const bool kept = s < L && (k > edge || (same && before < (uint32_t)left));
        before += s < L && same;
        const bool ho = s < m && !kept, fi = s >= m && kept;
        hole |= (uint32_t)ho << (4 * q + e);
        fill |= (uint32_t)fi << (4 * q + e);
        n_holes += __popcll(__ballot(ho));
        n_fills += __popcll(__ballot(fi));
      }
    }
    if (lane == 0) {
      sums[1][wave] = n_holes;
      sums[2][wave] = n_fills;
    }
    __syncthreads();
    uint32_t at_hole = holes, at_fill = fills;
    for (int i = 0; i < kEvictWaves; ++i) {
      const uint32_t x = sums[1][i], y = sums[2][i];
      at_hole += i < wave ? x : 0;
      at_fill += i < wave ? y : 0;
      holes += x;
      fills += y;
    }
    if (n_holes + n_fills > 0) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        uint32_t h = at_hole, f = at_fill;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t hb = __ballot(hole >> (4 * q + e) & 1);
          const uint64_t fb = __ballot(fill >> (4 * q + e) & 1);
          h += below(hb);
          f += below(fb);
          at_hole += __popcll(hb);
          at_fill += __popcll(fb);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int s = s0 + 256 * q + e;
          if (hole >> (4 * q + e) & 1) mv[h++].y = s;
          if (fill >> (4 * q + e) & 1) mv[f++].x = s;
        }
      }
    }
  }
  if (tid == 0) a.count[row] = (int)holes;
}

// D/4 lanes a group of moves: four in a row, whose loads are all in flight before
// the first is stored (they go to neighbouring slots, mostly).  A stride of the
// grid over the row's moves, so that the host need not know their number.
constexpr int kMoves = 4;
template <int D>
__global__ __launch_bounds__(256) void move_kernel(EvictArgs a) {
  constexpr int L = D / 4;
  const int row = blockIdx.x, b = row / a.c.H, h = row % a.c.H;
  const int i = threadIdx.x % L;
  if (h == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    // the only place that reads lens after the selection, so it may be lens_out
    const int len = kv_len(a.c, b);
    a.lens_out[b] = min(len, a.keep);
  }
  const int64_t at = (int64_t)row * a.c.room();
  const int count = a.count[row];
  const int2 *moves = a.moves + (int64_t)row * a.most;
  const int group = blockIdx.y * (256 / L) + threadIdx.x / L;
  for (int k0 = group * kMoves; k0 < count; k0 += gridDim.y * (256 / L) * kMoves) {
    int2 mv[kMoves];
    int64_t from[kMoves], to[kMoves];
#pragma unroll
    for (int k = 0; k < kMoves; ++k) mv[k] = moves[min(k0 + k, count - 1)];
#pragma unroll
    for (int k = 0; k < kMoves; ++k) {
      from[k] = kv_token(a.c, b, h, mv[k].x);
      to[k] = kv_token(a.c, b, h, mv[k].y);
      if (to[k] < 0) from[k] = -1;
    }
    uint16_t ck[kMoves], cv[kMoves];
    uint2 cs[kMoves];
    float cw[kMoves];
    int32_t cp[kMoves];
#pragma unroll
    for (int k = 0; k < kMoves; ++k) {
      const int64_t t = max(from[k], (int64_t)0);
      ck[k] = *reinterpret_cast<const uint16_t *>(a.c.k + k_byte<D>(t, i));
      cv[k] = *reinterpret_cast<const uint16_t *>(a.c.v + v_byte<D>(t, i));
      cs[k] = *reinterpret_cast<const uint2 *>(a.c.scales + t * 4);
      cw[k] = a.weights[at + mv[k].x];
      cp[k] = a.pos[at + mv[k].x];
    }
#pragma unroll
    for (int k = 0; k < kMoves; ++k) {
      if (k0 + k >= count) break;
      if (from[k] >= 0) {
        *reinterpret_cast<uint16_t *>(a.c.k + k_byte<D>(to[k], i)) = ck[k];
        *reinterpret_cast<uint16_t *>(a.c.v + v_byte<D>(to[k], i)) = cv[k];
        if (i == 0) *reinterpret_cast<uint2 *>(a.c.scales + to[k] * 4) = cs[k];
      }
      if (i == 0) {
        a.weights_out[at + mv[k].y] = cw[k];
        a.pos_out[at + mv[k].y] = cp[k];
      }
    }
  }
}

int most_moves(int room, int keep) { return keep < room - keep ? keep : room - keep; }

}  // namespace

hipError_t launch_kv_append(const KvView &c, int D, int n, const void *k, KvStrides ks,
                            const void *v, KvStrides vs, bcq_dtype dt, const int32_t *positions,
                            float *weights, int32_t *pos, hipStream_t s) {
#define BCQ_DIM(D_)                                                                            \
  return dt == BCQ_F16                                                                         \
             ? append_dim<D_, _Float16>(c, n, k, ks, v, vs, positions, weights, pos, s)        \
             : append_dim<D_, float>(c, n, k, ks, v, vs, positions, weights, pos, s)
  if (D == 64) BCQ_DIM(64);
  if (D == 128) BCQ_DIM(128);
  BCQ_DIM(256);
#undef BCQ_DIM
}

hipError_t launch_kv_read(const KvView &c, int D, int n, void *k, KvStrides ks, void *v,
                          KvStrides vs, bcq_dtype dt, hipStream_t s) {
#define BCQ_DIM(D_)                                                  \
  return dt == BCQ_F16 ? read_dim<D_, _Float16>(c, n, k, ks, v, vs, s) \
                       : read_dim<D_, float>(c, n, k, ks, v, vs, s)
  if (D == 64) BCQ_DIM(64);
  if (D == 128) BCQ_DIM(128);
  BCQ_DIM(256);
#undef BCQ_DIM
}

size_t evict_workspace_bytes(int B, int H, int room, int keep) {
  if (keep >= room) return (size_t)B * H * 8;
  return (size_t)B * H * (8 + (size_t)most_moves(room, keep) * sizeof(int2));
}

hipError_t launch_kv_evict(const KvView &c, int D, int keep, int recent, const float *weights,
                           const int32_t *pos, int32_t *lens_out, float *weights_out,
                           int32_t *pos_out, void *ws, hipStream_t s) {
  const int BH = c.B * c.H, room = c.room();
  EvictArgs a{c, keep, recent, weights, pos, lens_out, weights_out, pos_out, nullptr, nullptr, 0};
  a.most = keep < room ? most_moves(room, keep) : 0;
  a.moves = static_cast<int2 *>(ws);
  a.count = reinterpret_cast<int32_t *>(a.moves + (size_t)BH * a.most);
  if (room <= 4 * kEvictThreads)
    select_kernel<1, true><<<BH, kEvictThreads, 0, s>>>(a);
  else if (room <= 32 * kEvictThreads)
    select_kernel<8, true><<<BH, kEvictThreads, 0, s>>>(a);
  else
    select_kernel<4, false><<<BH, kEvictThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int per = 256 / (D / 4) * kMoves;
  // about 4096 workgroups in all: enough to fill the card several times over
  const int most_chunks = BH >= 4096 ? 1 : 4096 / BH;
  int chunks = (a.most + per - 1) / per;
  chunks = chunks < 1 ? 1 : (chunks > most_chunks ? most_chunks : chunks);
  const dim3 grid(BH, chunks);
  if (D == 64)
    move_kernel<64><<<grid, 256, 0, s>>>(a);
  else if (D == 128)
    move_kernel<128><<<grid, 256, 0, s>>>(a);
  else
    move_kernel<256><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace bcq
