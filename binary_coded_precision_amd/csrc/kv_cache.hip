// kv_cache.hip -- what fills, reads back and shrinks the 4-bit key/value cache
// (bcq_kv_append, bcq_kv_read, the same by slots, bcq_kv_evict).
//
// A vector of D channels (one token's K or V of one cached head) is
// zero + scale * code: zero = fp16(min), scale = fp16((max - min) * (1/15)),
// code = rint((x - zero) / scale) held to 0..15, each step rounded to fp32 (the
// constant too), so the codes are a function of the inputs alone.  Where either
// factor is not finite the scale becomes NaN: an infinite zero beside a finite
// scale would be read as an infinity, and as a score of -inf hide the token.
#include <type_traits>

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

// Vector `vec` of a call over n tokens of every sequence.  Four tokens that share a
// block of V are neighbours, K before V, then heads: a block is written (and
// read) by one wave or two of one workgroup.  A call of n tokens has quads_of(n)
// quads a sequence, the first and last of which may be partly or wholly outside.
struct Place {
  int b, i, h, slot;
  bool v, in;
};
__host__ __device__ __forceinline__ uint32_t quads_of(int n) { return ((uint32_t)n + 6) / 4; }
__device__ __forceinline__ Place place(const KvView &c, int n, uint32_t vec) {
  Place p;
  const uint32_t quads = n == 1 ? 1 : quads_of(n);
  const uint32_t t = n == 1 ? 0 : vec & 3, head = n == 1 ? vec : vec >> 2;
  p.v = head & 1;
  const uint32_t quad = (head >> 1) / (uint32_t)c.H;
  p.h = (int)((head >> 1) - quad * (uint32_t)c.H);
  p.b = (int)(quad / quads);
  const int first = kv_len(c, p.b) - n;  // slot of token 0
  p.i = (int)(quad - (uint32_t)p.b * quads) * 4 + (int)t - (n == 1 ? 0 : first & 3);
  p.slot = first + p.i;
  p.in = p.i >= 0 && p.i < n;
  return p;
}
__host__ __forceinline__ uint32_t vectors_of(const KvView &c, int n) {
  return (uint32_t)c.B * c.H * 2 * (n == 1 ? 1 : quads_of(n) * 4);
}

// Instructions weigh as much as bytes here.  The extremes take 16 where compares and
// selects that order NaN and zeros took 74, which made 8192 packed tokens of 8 heads of
// 128 channels in fp16 20.5 us rather than 12.4; those are for the vectors that need them.
//
// A vector's 4 channels of this lane as codes (bits 4e of `word`) and the vector's
// scale and zero, the same in all its D/4 lanes.
struct Coded {
  uint32_t word;
  _Float16 scale, zero;
};
// Of 16 lanes, the value N lanes further on, the first behind the last.
template <int N>
__device__ __forceinline__ float rotated(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x130 - N, 0xf, 0xf, false));
}
template <int N>
__device__ __forceinline__ void ordered_extremes(float &lo, float &hi) {
  lo = nan_min(lo, rotated<N>(lo));
  hi = nan_max(hi, rotated<N>(hi));
}
template <int N>
__device__ __forceinline__ void extremes(float &lo, float &hi) {
  lo = __builtin_elementwise_minimum(lo, rotated<N>(lo));
  hi = __builtin_elementwise_maximum(hi, rotated<N>(hi));
}
template <int D>
__device__ __forceinline__ Coded code_vector(const float (&x)[4]) {
  const auto least = [](float a, float b) { return __builtin_elementwise_minimum(a, b); };
  const auto largest = [](float a, float b) { return __builtin_elementwise_maximum(a, b); };
  float lo = least(least(x[0], x[1]), least(x[2], x[3]));
  float hi = largest(largest(x[0], x[1]), largest(x[2], x[3]));
  extremes<1>(lo, hi);
  extremes<2>(lo, hi);
  extremes<4>(lo, hi);
  extremes<8>(lo, hi);
#pragma unroll
  for (int d = 16; d < D / 4; d <<= 1) {
    lo = least(lo, __shfl_xor(lo, d));
    hi = largest(hi, __shfl_xor(hi, d));
  }
  // Which of zeros of both signs, and of NaN, is stored depends on the order: there it is
  // that of a butterfly for lane 0, which stores it, the later one winning.
  if (__builtin_expect(__any(!(fabsf(lo) > 0.f)), 0)) {
    lo = nan_min(nan_min(x[0], x[1]), nan_min(x[2], x[3]));
    hi = nan_max(nan_max(x[0], x[1]), nan_max(x[2], x[3]));
    ordered_extremes<1>(lo, hi);
    ordered_extremes<2>(lo, hi);
    ordered_extremes<4>(lo, hi);
    ordered_extremes<8>(lo, hi);
#pragma unroll
    for (int d = 16; d < D / 4; d <<= 1) {
      lo = nan_min(lo, __shfl_xor(lo, d));
      hi = nan_max(hi, __shfl_xor(hi, d));
    }
  }
  float step = (hi - lo) * (1.f / 15.f);
  asm volatile("" : "+v"(step));  // rounded to fp32 first: one instruction could do both at once
  const _Float16 zh = (_Float16)lo, near_step = (_Float16)step;
  const float zero = (float)zh;
  const bool good = (float)near_step < INFINITY && fabsf(zero) < INFINITY;
  const _Float16 sh = good ? near_step : (_Float16)NAN;
  const float scale = (float)sh;
  // the quotient's neighbour y * rcp(scale) is less than 1e-5 off it and rounds
  // to the same integer unless it lies that close to a half
  const float inv = __builtin_amdgcn_rcpf(scale);
  float q[4], off[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float y = (x[e] - zero) * inv;
    q[e] = rintf(y);
    off[e] = fabsf(y - q[e]);
  }
  const bool near = !(fmaxf(fmaxf(off[0], off[1]), fmaxf(off[2], off[3])) < 0.4999f);
  if (__builtin_expect(near, 0)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = rintf((x[e] - zero) / scale);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] = __builtin_amdgcn_fmed3f(q[e], 0.f, 15.f);
  // whole numbers below 2^16, so their sum in fp32 is exact
  const float all = fmaf(q[3], 4096.f, fmaf(q[2], 256.f, fmaf(q[1], 16.f, q[0])));
  const uint32_t word = scale > 0.f ? (uint32_t)all : 0u;
  return {word, sh, zh};
}
// Stored as K or V of cached token `token` (lane i of the vector's).
template <int D>
__device__ __forceinline__ void put_vector(const KvView &c, const Coded &x, int64_t token, bool v,
                                           int i) {
  *reinterpret_cast<uint16_t *>(v ? c.v + v_byte<D>(token, i) : c.k + k_byte<D>(token, i)) =
      (uint16_t)x.word;
  if (i == 0) {
    union {
      _Float16 h[2];
      uint32_t u;
    } m;
    m.h[0] = x.scale;
    m.h[1] = x.zero;
    *reinterpret_cast<uint32_t *>(c.scales + token * 4 + (v ? 2 : 0)) = m.u;
  }
}
// The values of cached token `token`, zeros where it is negative.
template <int D, typename T, bool VEC>
__device__ __forceinline__ void get_vector(const KvView &c, T *dst, int64_t token, bool v, int i) {
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (token >= 0) {
    const uint32_t word = *reinterpret_cast<const uint16_t *>(v ? c.v + v_byte<D>(token, i)
                                                                : c.k + k_byte<D>(token, i));
    union {
      uint32_t u;
      _Float16 h[2];
    } m;
    m.u = *reinterpret_cast<const uint32_t *>(c.scales + token * 4 + (v ? 2 : 0));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = (float)m.h[1] + (float)m.h[0] * (float)((word >> (4 * e)) & 15u);
  }
  store4<T, VEC>(dst, x);
}

// Bound by the bytes of the vectors read; every lane converts what it loads,
// the extremes meet in D/4 lanes and no shared memory is needed.  2 x 4099 tokens
// of 8 heads of 64 channels in fp32, slices of one projection (33.6 MB read, 4.6
// MB written): 14.2 us, 2.7 TB/s.
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
  if (!p.in) return;
  const KvStrides st = p.v ? vs : ks;
  float values[4];
  load4<T, VEC>(values, (p.v ? v : k) + p.b * st.batch + p.i * st.token + p.h * st.head + i * 4);
  const Coded x = code_vector<D>(values);
  if (p.slot < 0) return;
  const int64_t token = kv_token(c, p.b, p.h, p.slot);
  if (token < 0) return;
  put_vector<D>(c, x, token, p.v, i);
  if (i == 0 && !p.v) {
    const int64_t at = ((int64_t)p.b * c.H + p.h) * c.room() + p.slot;
    if (weights != nullptr) weights[at] = 0.f;
    if (pos != nullptr)
      pos[at] = positions != nullptr ? positions[(int64_t)p.b * n + p.i] : p.slot;
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
  if (!p.in) return;
  const KvStrides st = p.v ? vs : ks;
  const int64_t token = p.slot < 0 ? -1 : kv_token(c, p.b, p.h, p.slot);
  get_vector<D, T, VEC>(c, (p.v ? v : k) + p.b * st.batch + p.i * st.token + p.h * st.head + i * 4,
                        token, p.v, i);
}

// Packed tokens, each with its slot among all the pages: a workgroup has a head's K and
// V of 1024 / D tokens that follow each other, D/4 lanes a token, so that what is
// written of a block of V mostly comes from one wave.  Places are formed once a
// workgroup, but for the token within it (each lane's own cost as much as the
// conversion), and K and V are both on their way at once.  Bound by bytes: 32768 tokens
// of 8 heads of 128 in fp16 38 us appended (170 MB, 4.4 TB/s), 34 read; 6567 of 64 in
// fp32 11.4 and 11.0 (4.3 TB/s).  Few tokens are one pass's latency: 4 us for 1063.
template <int D>
struct PackedPlace {
  static constexpr int L = D / 4, PER = 256 / L;
  int64_t t0;  // the workgroup's first token
  int h, i, j, last;
  // workgroups past the last token have none
  __device__ __forceinline__ PackedPlace(int n) {
    h = blockIdx.x;
    i = threadIdx.x % L;
    t0 = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * PER;
    last = (int)min((int64_t)PER, n - t0) - 1;
    j = min((int)threadIdx.x / L, last);
  }
  __device__ __forceinline__ bool mine() const { return (int)threadIdx.x / L <= last; }
  __device__ __forceinline__ int64_t at(const KvStrides &s) const {
    return t0 * s.token + (int64_t)h * s.head + (int64_t)j * s.token + i * 4;
  }
};
// Index of a slot's token within all the pages of cached head h, as kv_token, or -1
// for a slot that no page has.
__device__ __forceinline__ int64_t slot_token(const KvView &c, int64_t slot, int h) {
  const int64_t page = slot >> c.page_log;
  if ((uint64_t)page >= (uint64_t)c.num_pages) return -1;
  const int64_t rows = (int64_t)((uint64_t)(uint32_t)page * (uint32_t)c.H + (uint32_t)h);
  return (rows << c.page_log) + ((int)slot & ((1 << c.page_log) - 1));
}

template <int D, typename T, bool VEC>
__global__ __launch_bounds__(256) void append_slots_kernel(KvView c, int n, const int64_t *slots,
                                                           const T *k, KvStrides ks, const T *v,
                                                           KvStrides vs) {
  const PackedPlace<D> p(n);
  if (p.last < 0) return;
  const int64_t slot = slots[p.t0 + p.j];
  float x[4], y[4];
  load4<T, VEC>(x, k + p.at(ks));
  load4<T, VEC>(y, v + p.at(vs));
  const Coded kc = code_vector<D>(x), vc = code_vector<D>(y);
  const int64_t token = slot_token(c, slot, p.h);
  if (token < 0 || !p.mine()) return;
  put_vector<D>(c, kc, token, false, p.i);
  put_vector<D>(c, vc, token, true, p.i);
}

template <int D, typename T, bool VEC>
__global__ __launch_bounds__(256) void read_slots_kernel(KvView c, int n, const int64_t *slots,
                                                         T *k, KvStrides ks, T *v,
                                                         KvStrides vs) {
  const PackedPlace<D> p(n);
  if (p.last < 0 || !p.mine()) return;
  const int64_t token = slot_token(c, slots[p.t0 + p.j], p.h);
  get_vector<D, T, VEC>(c, k + p.at(ks), token, false, p.i);
  get_vector<D, T, VEC>(c, v + p.at(vs), token, true, p.i);
}

bool vec_ok(const void *p, KvStrides s, size_t size) {
  return (uintptr_t)p % (4 * size) == 0 && s.batch % 4 == 0 && s.token % 4 == 0 &&
         s.head % 4 == 0;
}

template <int D, typename T>
hipError_t append_dim(const KvView &c, int n, const void *k, KvStrides ks, const void *v,
                      KvStrides vs, const int32_t *positions, float *weights, int32_t *pos,
                      hipStream_t s) {
  const uint32_t vecs = vectors_of(c, n), per = 256 / (D / 4);
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
  const uint32_t vecs = vectors_of(c, n), per = 256 / (D / 4);
  const uint32_t grid = (vecs + per - 1) / per;
  if (vec_ok(k, ks, sizeof(T)) && vec_ok(v, vs, sizeof(T)))
    read_kernel<D, T, true><<<grid, 256, 0, s>>>(c, n, (T *)k, ks, (T *)v, vs, vecs);
  else
    read_kernel<D, T, false><<<grid, 256, 0, s>>>(c, n, (T *)k, ks, (T *)v, vs, vecs);
  return hipGetLastError();
}

template <int D, typename T, typename K>
hipError_t slots_dim(const KvView &c, int n, const int64_t *slots, K *k, KvStrides ks, K *v,
                     KvStrides vs, hipStream_t s) {
  const uint32_t groups = ((uint32_t)n + PackedPlace<D>::PER - 1) / PackedPlace<D>::PER;
  const uint32_t deep = (groups + 65534) / 65535;  // a grid's limit but for x
  const dim3 grid(c.H, (groups + deep - 1) / deep, deep);
  const bool vec = vec_ok(k, ks, sizeof(T)) && vec_ok(v, vs, sizeof(T));
  if constexpr (std::is_const<K>::value) {
    if (vec)
      append_slots_kernel<D, T, true><<<grid, 256, 0, s>>>(c, n, slots, (const T *)k, ks,
                                                           (const T *)v, vs);
    else
      append_slots_kernel<D, T, false><<<grid, 256, 0, s>>>(c, n, slots, (const T *)k, ks,
                                                            (const T *)v, vs);
  } else {
    if (vec)
      read_slots_kernel<D, T, true><<<grid, 256, 0, s>>>(c, n, slots, (T *)k, ks, (T *)v, vs);
    else
      read_slots_kernel<D, T, false><<<grid, 256, 0, s>>>(c, n, slots, (T *)k, ks, (T *)v, vs);
  }
  return hipGetLastError();
}
template <typename K>
hipError_t launch_slots(const KvView &c, int D, int n, const int64_t *slots, K *k, KvStrides ks,
                        K *v, KvStrides vs, bcq_dtype dt, hipStream_t s) {
  if (dt == BCQ_F16)
    return D == 64    ? slots_dim<64, _Float16>(c, n, slots, k, ks, v, vs, s)
           : D == 128 ? slots_dim<128, _Float16>(c, n, slots, k, ks, v, vs, s)
                      : slots_dim<256, _Float16>(c, n, slots, k, ks, v, vs, s);
  return D == 64    ? slots_dim<64, float>(c, n, slots, k, ks, v, vs, s)
         : D == 128 ? slots_dim<128, float>(c, n, slots, k, ks, v, vs, s)
                    : slots_dim<256, float>(c, n, slots, k, ks, v, vs, s);
}

// ---- eviction
//
// Each (sequence, cached head) keeps its own tokens: the `recent` newest by
// position, then those of the largest accumulated weight, the lower slot first
// among equals.  Kept tokens already in front stay where they are and the i-th
// evicted slot in front takes the i-th kept token from behind, so that what
// moves is the least possible and no move reads what another writes.

constexpr uint32_t kLate = 0xffffffffu;  // above every weight's order

// Order of a slot: recent tokens above every weight, NaN below every weight.
__device__ __forceinline__ uint32_t order_of(float w, bool late) {
  if (late) return kLate;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kEvictThreads = 1024, kEvictWaves = kEvictThreads / 64;
constexpr int kDigit = 12, kBins = 1 << kDigit;
constexpr int kList = 2048;  // slots left that are listed and further passes go over
constexpr int kRank = 256;   // slots left that are ranked against each other
// Evicted slots that are looked for one by one: each costs 2.3 us where the select
// costs 5 (rows of 2049: one 8.7 us against 12.2, two 11.4 against 11.5, four 15.7
// against 11.3; rows of 30001: two 18.5 against 19.7, four 25.4 against 21.5).
constexpr int kFew = 2;
// Moves that the selecting workgroup makes itself, by the most there can be (rows
// of up to 2048 + that many, 32 and 256 rows, in a graph): with 64 10 and 11.6 us
// against 11.4 and 14.0 for a launch of their own, with 128 12.1 and 14.5 against 11.6
// and 16.8, with 256 15.4 and 20.3 against 12.0 and 21.2.
constexpr int kInPlace = 64;

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

// A slot's rank value: its order, then the lower slot; no two are alike.
__device__ __forceinline__ uint64_t rank_of(uint32_t order, int slot) {
  return (uint64_t)order << 32 | (0xffffffffu - (uint32_t)slot);
}

// Moves [k0, k0 + N) of a row of `count`, D/4 lanes (lane i of them): all loads are
// in flight before the first is stored.  What is read lies in slots that no
// move writes.
template <int D, int N>
__device__ __forceinline__ void move_tokens(const EvictArgs &a, int row, const int2 *moves, int k0,
                                            int count, int i) {
  const int b = row / a.c.H, h = row % a.c.H;
  const int64_t at = (int64_t)row * a.c.room();
  int2 mv[N];
  int64_t from[N], to[N];
#pragma unroll
  for (int k = 0; k < N; ++k) mv[k] = moves[min(k0 + k, count - 1)];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    from[k] = kv_token(a.c, b, h, mv[k].x);
    to[k] = kv_token(a.c, b, h, mv[k].y);
    if (to[k] < 0) from[k] = -1;
  }
  uint16_t ck[N], cv[N];
  uint2 cs[N];
  float cw[N];
  int32_t cp[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int64_t t = max(from[k], (int64_t)0);
    ck[k] = *reinterpret_cast<const uint16_t *>(a.c.k + k_byte<D>(t, i));
    cv[k] = *reinterpret_cast<const uint16_t *>(a.c.v + v_byte<D>(t, i));
    cs[k] = *reinterpret_cast<const uint2 *>(a.c.scales + t * 4);
    cw[k] = a.weights[at + mv[k].x];
    cp[k] = a.pos[at + mv[k].x];
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
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

// Element i, of 4 bytes, of a row's array: a scalar base and 32 bits of offset.
template <typename T, typename B>
__device__ __forceinline__ T *nth(B *base, uint32_t i) {
  using Byte = std::conditional_t<std::is_const_v<B>, const char, char>;
  return reinterpret_cast<T *>(reinterpret_cast<Byte *>(base) + (uint32_t)(4 * i));
}

// One workgroup a row.  A wave has 256 Q slots in a row, a thread the orders of 4 Q
// of them in registers, slot 256 q + 4 lane + e of the wave's, so that reads are
// wide and coalesced; rows with room for more than the workgroup holds (ONCE is
// false) go through all steps in rounds, which read weights and positions again.
//
// The row's smallest kept rank value is found, and ballots then number what
// moves in slot order.  Up to kFew evicted slots (a decode loop's step) are found
// as so many minima.  Otherwise a radix select takes 12 bits a pass of the
// orders' distances from the smallest, until a bin is kept whole or holds at most
// kRank slots, which are ranked against each other; once at most kList slots are
// left they are listed and the list is gone over, so that one count over all
// slots and one listing are the rule.  (With the orders' own bits as digits, 8
// bins an octave, a bin of 32768 softmax sums held a thousand slots and a second
// count followed.)
// One compute unit's vector ALUs bound it (an operation on each of 32768 slots
// takes 0.2 us), hence few operations a slot and pass: slots past L have a rank
// below all others instead of a test, and blocks without a match are left after
// one ballot.  32 rows of 32768 slots, 4096 kept: 24 us, then 21 us of moves.
//
// D > 0: there are at most kInPlace moves, made here; lens_out is then not lens.
template <int Q, bool ONCE, int D>
__global__ __launch_bounds__(kEvictThreads) void select_kernel(EvictArgs a) {
  constexpr int kRound = 4 * Q * kEvictThreads;
  __shared__ __align__(16) uint32_t hist[kBins];
  __shared__ uint32_t list_high[kList], list_low[kList];
  __shared__ uint64_t cand[kRank];
  __shared__ uint64_t least[kEvictWaves];
  __shared__ int tmp[kEvictWaves];
  __shared__ uint32_t sums[2][kEvictWaves];
  __shared__ uint32_t picked, above, inside, listed, ranked;
  __shared__ uint64_t edge_at;
  __shared__ int few_count;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = blockIdx.x, b = row / a.c.H;
  const int64_t at = (int64_t)row * a.c.room();
  const int L = kv_len(a.c, b), m = min(L, a.keep);
  const int end = ONCE ? 1 : L;  // of the rounds' first slots
  const float *w = a.weights + at;
  const int32_t *pos = a.pos + at;
  float *w_out = a.weights_out + at;
  int32_t *pos_out = a.pos_out + at;
  // A wave's first slot in a round, its blocks of 256, and the thread's in a block
  const int first = wave * 256 * Q, mine = lane * 4;
  if (D > 0 && tid == 0 && row % a.c.H == 0) a.lens_out[b] = m;

  // Rows start at multiples of 16 slots and end at one: reads of 4 slots past L
  // come from the row's last 4 or those at L.  Blocks past L are not read.
  float4 wv[Q];
  int4 pv[Q];
  auto read = [&](int s0, bool both) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (s0 + 256 * q < L) {
        const int s = min(s0 + 256 * q + mine, a.c.room() - 4);
        pv[q] = *nth<const int4>(pos, s);
        if (both) wv[q] = *nth<const float4>(w, s);
      }
  };
  int newest = INT32_MIN;
  for (int s0 = first; s0 < end + first; s0 += kRound) {
    read(s0, ONCE);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (s0 + 256 * q + 256 <= L) {
        newest = max(newest, max(max(pv[q].x, pv[q].y), max(pv[q].z, pv[q].w)));
      } else if (s0 + 256 * q < L) {
        const int s = s0 + 256 * q + mine;
        if (s < L) newest = max(newest, pv[q].x);
        if (s + 1 < L) newest = max(newest, pv[q].y);
        if (s + 2 < L) newest = max(newest, pv[q].z);
        if (s + 3 < L) newest = max(newest, pv[q].w);
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) newest = max(newest, __shfl_xor(newest, d));
  if (lane == 0) tmp[wave] = newest;
  reinterpret_cast<uint4 *>(hist)[tid] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  for (int i = 0; i < kEvictWaves; ++i) newest = max(newest, tmp[i]);
  // newest is at least every position, so their distance fits 32 bits
  auto is_late = [&](int32_t p) { return (uint32_t)newest - (uint32_t)p < (uint32_t)a.recent; };

  // The orders of the round whose slots start at s0 for this wave, 0 past L: as
  // rank values those are below every other, so that nothing else asks for L.  On
  // the way what is in front goes to the output; what is evicted of it is
  // overwritten by the moves.
  uint32_t key[Q][4];
  const bool apart = a.weights_out != a.weights || a.pos_out != a.pos;
  const bool wide = (((uintptr_t)a.weights_out | (uintptr_t)a.pos_out) & 15) == 0;
  auto orders = [&](int s0, bool write) {
    if (!ONCE) read(s0, true);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int block = s0 + 256 * q;
      if (block >= L) {
#pragma unroll
        for (int e = 0; e < 4; ++e) key[q][e] = 0;
        continue;
      }
      const float xs[4] = {wv[q].x, wv[q].y, wv[q].z, wv[q].w};
      const int32_t ys[4] = {pv[q].x, pv[q].y, pv[q].z, pv[q].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) key[q][e] = order_of(xs[e], is_late(ys[e]));
      const int s = block + mine;
      if (block + 256 > L) {
#pragma unroll
        for (int e = 0; e < 4; ++e) key[q][e] = s + e < L ? key[q][e] : 0;
      }
      if (!write || block >= m) continue;
      if (s + 3 < m && wide) {
        *nth<float4>(w_out, s) = wv[q];
        *nth<int4>(pos_out, s) = pv[q];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (s + e < m) {
            *nth<float>(w_out, s + e) = xs[e];
            *nth<int32_t>(pos_out, s + e) = ys[e];
          }
      }
    }
  };
  if (ONCE)
    orders(first, apart);
  else if (apart)
    for (int s0 = first; s0 < end + first; s0 += kRound) orders(s0, true);
  if (L <= a.keep) {
    if (tid == 0) a.count[row] = 0;
    return;
  }
  int2 *mv = a.moves + (int64_t)row * a.most;
  const int evicted = L - m;

  // ---- the smallest rank value kept
  uint64_t edge = 0;  // kept: rank values from here on
  uint32_t base = 0, late = kLate;
  auto distances = [&] {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) key[q][e] = min(max(key[q][e], base) - base, late);
  };
  if (evicted <= kFew) {
    edge = rank_of(0, L - 1);  // above those past L
    uint32_t out = 0;  // evicted slots behind m, by their distance from it
    int front[kFew], fronts = 0;
    for (int n = 0; n < evicted; ++n) {
      uint64_t low = ~0ull;
      for (int s0 = first; s0 < end + first; s0 += kRound) {
        if (!ONCE) orders(s0, false);
        uint32_t l = 0xffffffffu - (uint32_t)(s0 + mine);
        if (Q > 1) asm volatile("" : "+v"(l));  // or 4 Q rank values would be kept
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t v = (uint64_t)key[q][e] << 32 | (l - 256 * q - e);
            if (v >= edge && v < low) low = v;
          }
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint64_t o = __shfl_xor(low, d);
        low = o < low ? o : low;
      }
      __syncthreads();
      if (lane == 0) least[wave] = low;
      __syncthreads();
      for (int i = 0; i < kEvictWaves; ++i) low = least[i] < low ? least[i] : low;
      edge = low + 1;
      const int s = (int)(0xffffffffu - (uint32_t)low);
      if (s >= m)
        out |= 1u << (s - m);
      else if (tid == 0) {
        int k = fronts++;  // into place among the lower ones
        for (; k > 0 && front[k - 1] > s; --k) front[k] = front[k - 1];
        front[k] = s;
      }
    }
    if (tid == 0) {
      for (int k = 0, s = 0; k < fronts; ++k, ++s) {
        while (out >> s & 1) ++s;
        mv[k] = make_int2(m + s, front[k]);
      }
      a.count[row] = few_count = fronts;
    }
    if constexpr (D > 0) {
      __syncthreads();
      for (int k = tid / (D / 4); k < few_count; k += kEvictThreads / (D / 4))
        move_tokens<D, 1>(a, row, mv, k, few_count, tid % (D / 4));
    }
    return;
  } else {
    // Orders as their distance from the smallest one (late ones one past the
    // largest, NaN 0): the first digit then tells apart weights of a few octaves,
    // whatever those are.
    uint32_t lo = 0xffffffffu, hi = 0;  // the smallest less 1, the largest plus 1
    for (int s0 = first; s0 < end + first; s0 += kRound) {
      if (!ONCE) orders(s0, false);
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo = min(lo, key[q][e] - 1);
          hi = max(hi, key[q][e] + 1);
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      lo = min(lo, (uint32_t)__shfl_xor((int)lo, d));
      hi = max(hi, (uint32_t)__shfl_xor((int)hi, d));
    }
    if (lane == 0) {
      sums[0][wave] = lo;
      sums[1][wave] = hi;
    }
    __syncthreads();
    for (int i = 0; i < kEvictWaves; ++i) {
      lo = min(lo, sums[0][i]);
      hi = max(hi, sums[1][i]);
    }
    base = lo < hi ? lo : 0;  // none but late ones and NaN
    late = lo < hi ? hi - lo : 1;
    __syncthreads();
    if (ONCE) distances();

    uint32_t left = m;     // still to be taken among the values that start with edge
    bool in_list = false;  // those are in `list`
    // Whether a rank value, in halves, starts with edge from bit `from` up.
    auto starts = [&](int from) {
      const uint64_t bits = ~0ull << from;
      const uint32_t high = (uint32_t)(edge >> 32), low = (uint32_t)edge;
      const uint32_t of_high = (uint32_t)(bits >> 32), of_low = (uint32_t)bits;
      return [=](uint32_t k, uint32_t l) {
        return (((k ^ high) & of_high) | ((l ^ low) & of_low)) == 0;
      };
    };
    // Visits what does, of those listed or of all slots; a block without any is
    // left at once.
    auto match_listed = [&](int from, auto &&visit) {
      const auto is = starts(from);
      for (int i = tid; i < (int)listed; i += kEvictThreads) {
        const uint32_t k = list_high[i], l = list_low[i];
        if (is(k, l)) visit(k, l);
      }
    };
    auto match = [&](int from, auto &&visit) {
      const auto is = starts(from);
      for (int s0 = first; s0 < end + first; s0 += kRound) {
        if (!ONCE) {
          orders(s0, false);
          distances();
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int block = s0 + 256 * q;
          if (block >= L) break;
          const uint32_t l = 0xffffffffu - (uint32_t)(block + mine);
          bool any = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) any |= is(key[q][e], l - e);
          if (__ballot(any) == 0) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (is(key[q][e], l - e)) visit(key[q][e], l - e);
        }
      }
    };
    // Digits from the highest bit that is set in any.  Five end it at the latest:
    // from bit 8 down a bin has at most kRank values, all distinct.
    const int top = 32 - __clz((int)late);  // late is at least 1
    int from = 32 + max(top, kDigit), shift = from - kDigit;
    for (int s0 = first; s0 < end + first; s0 += kRound) {
      if (!ONCE) {
        orders(s0, false);
        distances();
      }
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if (s0 + 256 * q >= L) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) atomicAdd(&hist[key[q][e] >> (shift - 32)], 1u);
      }
    }
    for (;;) {
      __syncthreads();
      {
        // from the top: thread t has bins 4 (1023 - t) .. + 3, and clears them
        uint4 *h = reinterpret_cast<uint4 *>(hist) + (kEvictThreads - 1 - tid);
        const uint4 x = *h;
        *h = make_uint4(0, 0, 0, 0);
        const uint32_t t[4] = {x.w, x.z, x.y, x.x};
        const uint32_t sum = t[0] + t[1] + t[2] + t[3];
        uint32_t up = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const uint32_t o = __shfl_up(up, d);
          if (lane >= d) up += o;
        }
        if (lane == 63) sums[0][wave] = up;
        if (tid == 0) ranked = 0;
        if (tid == 0 && !in_list) listed = 0;
        __syncthreads();
        uint32_t over = up - sum;
        for (int i = 0; i < wave; ++i) over += sums[0][i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (over < left && over + t[i] >= left) {
            picked = 4 * (kEvictThreads - 1 - tid) + 3 - i;
            above = over;
            inside = t[i];
          }
          over += t[i];
        }
      }
      __syncthreads();
      edge |= (uint64_t)picked << shift;
      left -= above;
      if (inside == left) break;
      if (inside <= kList && !in_list) {
        match(shift, [&](uint32_t k, uint32_t l) {
          const uint32_t i = atomicAdd(&listed, 1u);
          list_high[i] = k;
          list_low[i] = l;
        });
        __syncthreads();
        in_list = true;
      }
      if (inside <= kRank) {
        // the left-th from the top of what starts with edge is the last kept
        match_listed(shift, [&](uint32_t k, uint32_t l) {
          cand[atomicAdd(&ranked, 1u)] = (uint64_t)k << 32 | l;
        });
        __syncthreads();
        const uint32_t n = ranked;
        if (tid < (int)n) {
          const uint64_t v = cand[tid];
          uint32_t higher = 0;
          for (uint32_t i = 0; i < n; ++i) higher += cand[i] > v;
          if (higher == left - 1) edge_at = v;
        }
        __syncthreads();
        edge = edge_at;
        break;
      }
      from = shift;
      shift = max(shift - kDigit, 0);
      auto count = [&](uint32_t k, uint32_t l) {
        const uint32_t digit =
            shift >= 32 ? k >> (shift - 32) : __builtin_amdgcn_alignbit(k, l, shift);
        atomicAdd(&hist[digit & ((1u << (from - shift)) - 1)], 1u);
      };
      if (in_list)
        match_listed(from, count);
      else
        match(from, count);
    }
  }

  // ---- what moves, in slot order
  const uint32_t edge_key = (uint32_t)(edge >> 32);
  const int edge_slot = (int)min(0xffffffffu - (uint32_t)edge, 0x7fffffffu);
  uint32_t holes = 0, fills = 0;  // before this round
  for (int s0 = first; s0 < end + first; s0 += kRound) {
    if (!ONCE) {
      orders(s0, false);
      distances();
    }
    // 4 bits a q: evicted in front of m, kept behind it
    uint32_t hole = 0, fill = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int s = s0 + 256 * q + mine;
      uint32_t kept = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        kept |= (uint32_t)(key[q][e] >= (s + e <= edge_slot ? edge_key : edge_key + 1)) << e;
      const uint32_t front = (1u << max(0, min(m - s, 4))) - 1;
      hole |= (front & ~kept) << (4 * q);
      fill |= (kept & ~front) << (4 * q);
    }
    uint32_t both = __popc(hole) | __popc(fill) << 16;  // at most 256 Q each in a wave
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) both += __shfl_xor((int)both, d);
    const uint32_t n_holes = both & 0xffff, n_fills = both >> 16;
    __syncthreads();
    if (lane == 0) {
      sums[0][wave] = n_holes;
      sums[1][wave] = n_fills;
    }
    __syncthreads();
    uint32_t at_hole = holes, at_fill = fills;
    for (int i = 0; i < kEvictWaves; ++i) {
      const uint32_t x = sums[0][i], y = sums[1][i];
      at_hole += i < wave ? x : 0;
      at_fill += i < wave ? y : 0;
      holes += x;
      fills += y;
    }
    auto number = [&](uint32_t bits, uint32_t place, bool to) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if (__ballot(bits >> (4 * q) & 15) == 0) continue;
        uint32_t n = place;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t x = __ballot(bits >> (4 * q + e) & 1);
          n += below(x);
          place += __popcll(x);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (bits >> (4 * q + e) & 1) {
            *nth<int32_t>(mv, 2 * n + to) = s0 + 256 * q + mine + e;
            ++n;
          }
      }
    };
    if (n_holes > 0) number(hole, at_hole, true);
    if (n_fills > 0) number(fill, at_fill, false);
  }
  if (tid == 0) a.count[row] = (int)holes;
  if constexpr (D > 0) {
    __syncthreads();  // the moves are this workgroup's own writes
    const int count = (int)holes;
    constexpr int kLanes = D / 4;
    for (int k = tid / kLanes; k < count; k += kEvictThreads / kLanes)
      move_tokens<D, 1>(a, row, mv, k, count, tid % kLanes);
  }
}

// D/4 lanes a group of moves: four in a row (they go to neighbouring slots,
// mostly).  A stride of the grid over the row's moves, so that the host need not
// know their number.  Bound by the sectors that the scattered pairs of V's bytes
// touch (a token's are 2 of every 8): 32 rows of about 3500 moves take 20.6 us.
constexpr int kMoves = 4;
template <int D>
__global__ __launch_bounds__(256) void move_kernel(EvictArgs a) {
  constexpr int L = D / 4;
  const int row = blockIdx.x, b = row / a.c.H;
  if (row % a.c.H == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    // the only place that reads lens after the selection, so it may be lens_out
    const int len = kv_len(a.c, b);
    a.lens_out[b] = min(len, a.keep);
  }
  const int count = a.count[row];
  const int2 *moves = a.moves + (int64_t)row * a.most;
  const int group = blockIdx.y * (256 / L) + threadIdx.x / L;
  for (int k0 = group * kMoves; k0 < count; k0 += gridDim.y * (256 / L) * kMoves)
    move_tokens<D, kMoves>(a, row, moves, k0, count, threadIdx.x % L);
}

template <int D>
hipError_t evict_dim(const EvictArgs &a, hipStream_t s) {
  const int BH = a.c.B * a.c.H, room = a.c.room();
  const bool once = room <= 32 * kEvictThreads, small = room <= 4 * kEvictThreads;
  if (a.most <= kInPlace && once && a.lens_out != a.c.lens) {
    if (small)
      select_kernel<1, true, D><<<BH, kEvictThreads, 0, s>>>(a);
    else
      select_kernel<8, true, D><<<BH, kEvictThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  if (small)
    select_kernel<1, true, 0><<<BH, kEvictThreads, 0, s>>>(a);
  else if (once)
    select_kernel<8, true, 0><<<BH, kEvictThreads, 0, s>>>(a);
  else
    select_kernel<2, false, 0><<<BH, kEvictThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int per = 256 / (D / 4) * kMoves;
  // about 4096 workgroups in all: enough to fill the card several times over
  const int most_chunks = BH >= 4096 ? 1 : 4096 / BH;
  int chunks = (a.most + per - 1) / per;
  chunks = chunks < 1 ? 1 : (chunks > most_chunks ? most_chunks : chunks);
  move_kernel<D><<<dim3(BH, chunks), 256, 0, s>>>(a);
  return hipGetLastError();
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

hipError_t launch_kv_append_slots(const KvView &c, int D, int n, const int64_t *slots,
                                  const void *k, KvStrides ks, const void *v, KvStrides vs,
                                  bcq_dtype dt, hipStream_t s) {
  return launch_slots(c, D, n, slots, k, ks, v, vs, dt, s);
}
hipError_t launch_kv_read_slots(const KvView &c, int D, int n, const int64_t *slots, void *k,
                                KvStrides ks, void *v, KvStrides vs, bcq_dtype dt,
                                hipStream_t s) {
  return launch_slots(c, D, n, slots, k, ks, v, vs, dt, s);
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
  return D == 64 ? evict_dim<64>(a, s) : D == 128 ? evict_dim<128>(a, s) : evict_dim<256>(a, s);
}

}  // namespace bcq
