// kv_packed.hip -- attention of packed tokens, sequences with unlike numbers of them,
// over the 4-bit key/value cache (bcq_kv_attend_packed); the mathematics and a
// wave's steps are in kv_tiles.h.
//
// What a call has to do is known on the device only (starts, lengths), so a first
// kernel of one workgroup cuts it into items, one a workgroup and cached head:
//
//  - A sequence's rows (its tokens, times the query heads of a cached head) are
//    blocks of up to four waves' rows.  Where one wave or two hold them all, the
//    waves share the tokens instead.
//  - Its tokens are cut into `ns` shares, so that all items together are about as
//    many as the card holds and none is longer than the others' average asks for.
//  - Rows of sequences with few of them (decode steps, drafted tokens) all meet the
//    shared pages together, as the rows of one sequence: those pages are read
//    once, and up to 128 rows share the unpacking of their codes.  The sequences'
//    own items then start behind the shared pages.  Sequences with many rows gain
//    nothing from that and read the shared pages as their own.
//
// Shares leave sums and outputs before the division, which a last kernel joins; what
// has one share only is written at once.
#include <algorithm>

#include "kv_tiles.h"

namespace bcq {
namespace {

using namespace kv;

constexpr int kThreads = 256, kWaves = 4;
constexpr int kMaxShares = 64;  // of a row, one a lane where they are joined
// Workgroups that a call is cut into when there is enough to do: two a compute unit,
// as many as their registers leave room for.
constexpr int kTarget = 512;
constexpr int kLeastSteps = 1;
constexpr int kMaxGroups = (1 << 24) - 1;  // of 256 work items in a launch
constexpr int kMostParts = 1 << 30;        // partial rows of a cached head
constexpr int kMostSteps = 2048;  // of 32 tokens, that a wave sums in one go (kv_attend.hip)

// Rows of a wave in a block of many rows, tiles of 16 of them.
constexpr int wave_tiles(int D) { return D <= 128 ? 2 : 1; }
constexpr int wave_rows(int D) { return 16 * wave_tiles(D); }
// Rows up to which blocks have 16 and their waves share the tokens.
constexpr int kFewRows = 32;
struct Shape {
  int blocks, waves;  // waves that share a block's tokens
};
template <int U>
__host__ __device__ constexpr Shape shape_of(int rows) {
  return rows <= kFewRows ? Shape{(rows + 15) / 16, 4} : Shape{(rows + 4 * U - 1) / (4 * U), 1};
}

struct PlanHead {
  int items;       // in use
  int base;        // tokens that sequences with few rows leave to the shared items
  int few;         // such rows
  int few_shares;  // of the shared pages
  int few_at;      // their partial rows
  int split;       // rows of the sequences of many rows that are to be joined
  int splits;      // such sequences
};
// A sequence's share of work: rows [128 block ..) of it, share `share` of `shares`.
// seq -1: the shared pages, n tokens of the list.
struct Item {
  int seq, block, share, shares;
  int start, n, len, part;  // part: the first of its partial rows, -1 where there is one share
};
struct FewToken {
  int token, last;  // packed token; last slot it sees
  int part;         // partial rows of its heads in its sequence's own shares, or -1
  int rows_shares;  // rows of the sequence << 8 | own shares
};
struct SplitSeq {
  int row, seq;  // rows before it; the sequence
  int start, n, part, shares;
};

struct PackedArgs {
  KvView c;
  const void *q;
  void *out;
  int64_t q_token, q_head, o_token, o_head;
  const int32_t *starts;
  int T, G, max_n, shared;  // shared: tokens of the shared pages
  bool q_wide;
  float unit, code_unit;
  PlanHead *head;
  Item *items;
  FewToken *few;
  SplitSeq *splits;
  float2 *ml;  // [H][part_cap]
  float *o;    // [H][part_cap][D]
  int item_cap, few_cap, part_cap;
};

struct Seq {
  int start, n, len, rows, blocks, steps;
  bool few;
};
// U: rows of a wave; base: tokens that sequences with few rows do not walk.
template <int U>
__device__ __forceinline__ Seq seq_of(const PackedArgs &a, int b, int base) {
  Seq q{};
  if (b >= a.c.B) return q;
  const int s0 = min(max(a.starts[b], 0), a.T), s1 = min(max(a.starts[b + 1], 0), a.T);
  q.start = s0;
  q.n = min(max(s1 - s0, 0), a.max_n);
  q.len = kv_len(a.c, b);
  q.rows = q.n * a.G;
  q.few = q.n > 0 && q.rows <= 2 * U;
  const Shape shape = shape_of<U>(q.rows);
  q.blocks = shape.blocks;
  const int tiles = (max(0, q.len - (q.few ? base : 0)) + 31) / 32;
  q.steps = (tiles + shape.waves - 1) / shape.waves;
  return q;
}

__device__ __forceinline__ int capped(int a, int b) { return min(a + b, 1 << 30); }
// Inclusive sum over the workgroup and the sum of all, each up to 2^30.
__device__ __forceinline__ int2 scan(int x, int *part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x = capped(x, y);
  }
  if (lane == 63) part[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int y = part[w];
    if (w < wave) before = capped(before, y);
    all = capped(all, y);
  }
  __syncthreads();
  return make_int2(capped(x, before), all);
}
__device__ __forceinline__ float sum_of(float x, float *part) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  x = (part[0] + part[1]) + (part[2] + part[3]);
  __syncthreads();
  return x;
}

__device__ __forceinline__ int shares_of(int steps, int chunk, int most) {
  return min(max((steps + chunk - 1) / chunk, 1), most);
}

template <int U>
__global__ __launch_bounds__(kThreads) void plan_kernel(PackedArgs a) {
  __shared__ int part[kWaves];
  __shared__ float partf[kWaves];
  __shared__ int offset[BCQ_KV_PACKED_MAX_BATCH + 1];  // of a sequence's items, in order
  __shared__ uint16_t order[BCQ_KV_PACKED_MAX_BATCH];
  const int tid = threadIdx.x, B = a.c.B;
  // tokens of sequences with few rows
  int seqs = 0, tokens = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const Seq q = seq_of<U>(a, b0 + tid, 0);
    seqs += scan(q.few, part).y;
    tokens = capped(tokens, scan(q.few ? q.n : 0, part).y);
  }
  PlanHead h{};
  const bool together = a.shared > 0 && seqs > 1 && tokens <= a.few_cap;
  h.base = together ? a.shared : 0;
  tokens = min(tokens, a.few_cap);
  h.few = tokens * a.G;
  // the shared items' shape, as a sequence's
  int few_blocks = 0, few_steps = 0;
  if (together) {
    const Shape shape = shape_of<U>(h.few);
    few_blocks = shape.blocks;
    few_steps = ((a.shared + 31) / 32 + shape.waves - 1) / shape.waves;
  }
  float cost = 0.f;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const Seq q = seq_of<U>(a, b0 + tid, h.base);
    cost += sum_of((float)q.blocks * (float)q.steps, partf);
  }
  cost += (float)few_blocks * (float)few_steps;
  const int chunk = max(
      kLeastSteps, (int)fminf(ceilf(cost * (float)a.c.H * (1.f / kTarget)), (float)kMostSteps));
  const int most = together ? kMaxShares / 2 : kMaxShares;
  int used = 0;  // partial rows
  if (together) {
    h.few_shares = shares_of(few_steps, chunk, most);
    if ((int64_t)h.few_shares * h.few > a.part_cap) h.few_shares = 0;
    used = h.few_shares * h.few;
  }
  int items = few_blocks * h.few_shares;
  const int few_items = items;
  // the longest sequences' items first, as workgroups are handed out in order
  if (B <= kThreads) {
    const Seq q = seq_of<U>(a, tid, h.base);
    offset[tid] = tid < B ? q.steps : -1;
    __syncthreads();
    int rank = 0;
    for (int j = 0; j < B; ++j) rank += offset[j] > q.steps || (offset[j] == q.steps && j < tid);
    if (tid < B) order[rank] = (uint16_t)tid;
  } else {
    for (int b = tid; b < B; b += kThreads) order[b] = (uint16_t)b;
  }
  __syncthreads();
  int few_before = 0, split = 0, splits = 0;
  for (int r0 = 0; r0 < B; r0 += kThreads) {
    const int r = r0 + tid, b = r < B ? order[r] : B;
    const Seq q = seq_of<U>(a, b, h.base);
    const bool joined = together && q.few;
    int shares = q.blocks == 0 ? 0 : shares_of(q.steps, chunk, most);
    if (joined && q.steps == 0) shares = 0;
    const bool parts = shares > 1 || (joined && shares > 0);
    const int rows = parts ? (int)min((int64_t)q.rows * shares, (int64_t)1 << 30) : 0;
    const int2 pr = scan(rows, part);
    const int at = capped(used, pr.x) - rows;
    if (parts && capped(used, pr.x) > a.part_cap) shares = 0;  // starts that are none
    const int2 it = scan((int)min((int64_t)q.blocks * shares, (int64_t)1 << 30), part);
    const int2 fw = scan(q.few ? q.n : 0, part);
    const bool many = shares > 1 && !q.few;
    const int2 sr = scan(many ? q.rows : 0, part), sn = scan(many, part);
    if (r < B) {
      offset[r] = capped(items, it.x) - q.blocks * shares;
      // an item's description, for those who write the items
      a.items[a.item_cap + b] =
          Item{b, q.blocks, 0, shares, q.start, q.n, q.len, parts && shares > 0 ? at : -1};
      if (q.few)
        for (int i = 0; i < q.n; ++i) {
          const int k = few_before + fw.x - q.n + i;
          if (k < a.few_cap)
            a.few[k] = FewToken{q.start + i, q.len - q.n + i,
                                parts && shares > 0 ? at + i * a.G : -1, q.rows << 8 | shares};
        }
      if (many)
        a.splits[splits + sn.x - 1] =
            SplitSeq{split + sr.x - q.rows, b, q.start, q.n, at, shares};
    }
    used = capped(used, pr.y);
    items = capped(items, it.y);
    few_before = capped(few_before, fw.y);
    split = capped(split, sr.y);
    splits += sn.y;
  }
  h.items = min(items, a.item_cap);
  h.split = split;
  h.splits = splits;
  if (tid == 0) *a.head = h;
  __syncthreads();
  for (int i = tid; i < h.items; i += kThreads) {
    Item x;
    if (i < few_items) {
      // shares of one block are neighbours
      x = Item{-1, i / h.few_shares, i % h.few_shares, h.few_shares, 0, tokens, a.shared, 0};
    } else {
      int r = 0;
      for (int step = 1 << (31 - __clz(B)); step > 0; step >>= 1)
        if (r + step < B && offset[r + step] <= i) r += step;
      x = a.items[a.item_cap + order[r]];
      const int j = i - offset[r];
      x.block = x.block - 1 - j / x.shares;  // the last rows, which see the most, first
      x.share = j % x.shares;
    }
    a.items[i] = x;
  }
}

__device__ __forceinline__ void store_out(const PackedArgs &a, int64_t at, float x, bool f32) {
  if (f32)
    static_cast<float *>(a.out)[at] = x;
  else
    static_cast<_Float16 *>(a.out)[at] = (_Float16)x;
}

// Waves of the same rows meet here.
template <int D>
struct Meet {
  float o[kWaves][16][D + 4];
  float m[kWaves][16], l[kWaves][16];
};
// The rows of a wave: the last slot that each lane's sees, and the wave's first and last.
template <int CT>
struct Rows {
  int last[CT], high, low;
};
template <int D, int CT, bool F32>
__device__ __forceinline__ Rows<CT> rows_of(const PackedArgs &a, const Item &x, int h, int row0,
                                            int lane, RawQueries<D, CT, F32> &raw) {
  const int R = x.n * a.G;
  Rows<CT> r;
  int high = -1, low = INT32_MAX;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int row = min(row0 + ct * 16 + (lane & 15), R - 1);
    const int i = row / a.G;
    int64_t token = x.start + i;
    r.last[ct] = x.len - x.n + i;
    if (x.seq < 0) {
      const FewToken t = a.few[i];
      token = t.token;
      r.last[ct] = min(t.last, x.len - 1);
    }
    const int64_t at =
        token * a.q_token + (int64_t)(h * a.G + row - i * a.G) * a.q_head + (lane >> 4) * (D / 4);
    fetch_query<D, CT, F32>(raw, ct, a.q, at, a.q_wide);
    high = max(high, r.last[ct]);
    low = min(low, r.last[ct]);
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    high = max(high, __shfl_xor(high, d));
    low = min(low, __shfl_xor(low, d));
  }
  r.high = __builtin_amdgcn_readfirstlane(high);
  r.low = __builtin_amdgcn_readfirstlane(low);
  return r;
}
template <int D, int CT>
__device__ __forceinline__ void clear(Sums<D, CT> &A) {
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    A.m[ct] = kNegInf;
    A.l[ct] = A.z[ct] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) A.o[ct][d] = float4v{0.f, 0.f, 0.f, 0.f};
  }
}

// An item of few rows: 16 of them, four waves share the tokens.
template <int D, bool F32>
__device__ __forceinline__ void run_few(const PackedArgs &a, const Item &x, int base, int h,
                                        Meet<D> &meet) {
  int lane = threadIdx.x & 63;
  // opaque, so that nothing formed from it is kept in registers from item to item
  asm volatile("" : "+v"(lane));
  const int g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool shared = x.seq < 0;
  const int R = x.n * a.G, L = x.len, b = shared ? 0 : x.seq;
  const int row0 = x.block * 16, t0 = shared ? 0 : base;

  RawQueries<D, 1, F32> raw;
  const Rows<1> rows = rows_of<D, 1, F32>(a, x, h, row0, lane, raw);
  // tiles of 32 tokens of these rows and of this share, in whole rounds of the waves
  const int tiles = (max(0, rows.high + 1 - t0) + 31) / 32;
  const int rounds = (tiles + kWaves - 1) / kWaves;
  const int chunk = (rounds + x.shares - 1) / x.shares * kWaves;
  int tile = x.share * chunk + wave;
  const int tile_end = min(tiles, x.share * chunk + chunk);
  const int free_end = max(0, rows.low + 1 - t0) / 32;  // tiles before it need no mask
  Tiles<D> T;
  if (tile < tile_end) {
    const Where w = where(a.c, b, h, t0 + tile * 32, L);
    load_k(T, a.c, w, lane);
    load_m(T, a.c, w, lane);
    load_v(T, a.c, w, lane);
  }
  Queries<D, 1, F32> Q;
  load_queries<D, 1, F32>(Q, raw, a.unit, row0, R, lane);
  Sums<D, 1> A;
  clear(A);
  // the next tiles are asked for as soon as the registers of these are free, and
  // the place of those after them is looked up a step earlier still
  auto place_of = [&](int ti) {
    return where(a.c, b, h, t0 + (ti < tile_end ? ti : tile) * 32, L);
  };
  Where ahead{};
  if (tile < tile_end) ahead = place_of(tile + kWaves);
  while (tile < tile_end) {
    const int next = tile + kWaves;
    const Where w = ahead;
    ahead = place_of(next + kWaves);
    float4v S[2][1];
    scores<D, 1, F32>(S, T, Q, a.code_unit);
    load_k(T, a.c, w, lane);
    if (tile >= free_end) mask_scores<D, 1>(S, T, A, t0 + tile * 32 + 4 * g, rows.last);
    Frag P[1], Plo[1];
    softmax_tiles<D, 1>(A, P, Plo, S, T);
    load_m(T, a.c, w, lane);
    add_values<D, 1, F32>(A, P, Plo, T);
    load_v(T, a.c, w, lane);
    tile = next;
  }

  // the waves' rows are the same: they meet in shared memory, then a wave joins a row
  A.l[0] = group_sum(A.l[0]);
  A.z[0] = group_sum(A.z[0]);
  const int col = lane & 15;
  if (g == 0) {
    meet.m[wave][col] = A.m[0];
    meet.l[wave][col] = A.l[0];
  }
  if (row0 + col < R)
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float4v v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(A.o[0][4 * hh + j][i], kCentreScale, A.z[0]);
        *reinterpret_cast<float4v *>(&meet.o[wave][col][64 * hh + 16 * g + 4 * i]) = v;
      }
  __syncthreads();
  const int64_t part0 = (int64_t)h * a.part_cap + x.part + (int64_t)x.share * R;
  for (int c = wave; c < 16 && row0 + c < R; c += kWaves) {
    const int row = row0 + c;
    const float mw = lane < kWaves ? meet.m[lane][c] : kNegInf;
    float m = mw;
#pragma unroll
    for (int d = 1; d < kWaves; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float f = mw == kNegInf ? 0.f : exp2f(mw - m);
    float l = lane < kWaves ? f * meet.l[lane][c] : 0.f;
#pragma unroll
    for (int d = 1; d < kWaves; d <<= 1) l += __shfl_xor(l, d);
    m = __shfl(m, 0);
    l = __shfl(l, 0);
    const int i = row / a.G;
    const int64_t at = (x.start + i) * a.o_token + (int64_t)(h * a.G + row - i * a.G) * a.o_head;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) o += __shfl(f, w) * meet.o[w][c][e * 64 + lane];
      if (x.part < 0)
        store_out(a, at + e * 64 + lane, l == 0.f ? 0.f : o / l, F32);
      else
        a.o[(part0 + row) * D + e * 64 + lane] = o;
    }
    if (lane == 0 && x.part >= 0) a.ml[part0 + row] = make_float2(m, l);
  }
}

// An item of many rows: every wave has rows of its own.
template <int D, bool F32>
__device__ __forceinline__ void run_many(const PackedArgs &a, const Item &x, int base, int h) {
  constexpr int CT = wave_tiles(D), U = wave_rows(D);
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // as in run_few
  const int g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool shared = x.seq < 0;
  const int R = x.n * a.G, L = x.len, b = shared ? 0 : x.seq;
  const int row0 = (x.block * kWaves + wave) * U;
  if (row0 >= R) return;
  const int t0 = shared || R > 2 * U ? 0 : base;

  RawQueries<D, CT, F32> raw;
  const Rows<CT> rows = rows_of<D, CT, F32>(a, x, h, row0, lane, raw);
  // tiles of 32 tokens of the wave's rows and of this share
  const int tiles = (max(0, rows.high + 1 - t0) + 31) / 32;
  const int chunk = (tiles + x.shares - 1) / x.shares;
  int tile = x.share * chunk;
  const int tile_end = min(tiles, tile + chunk);
  const int free_end = max(0, rows.low + 1 - t0) / 32;
  Tiles<D> T;
  if (tile < tile_end) {
    const Where w = where(a.c, b, h, t0 + tile * 32, L);
    load_k(T, a.c, w, lane);
    load_m(T, a.c, w, lane);
    load_v(T, a.c, w, lane);
  }
  Queries<D, CT, F32> Q;
  load_queries<D, CT, F32>(Q, raw, a.unit, row0, R, lane);
  Sums<D, CT> A;
  clear(A);
  auto place_of = [&](int ti) {
    return where(a.c, b, h, t0 + (ti < tile_end ? ti : tile) * 32, L);
  };
  Where ahead{};
  if (tile < tile_end) ahead = place_of(tile + 1);
  for (; tile < tile_end; ++tile) {
    const Where w = ahead;
    ahead = place_of(tile + 2);
    float4v S[2][CT];
    scores<D, CT, F32>(S, T, Q, a.code_unit);
    load_k(T, a.c, w, lane);
    if (tile >= free_end) mask_scores<D, CT>(S, T, A, t0 + tile * 32 + 4 * g, rows.last);
    Frag P[CT], Plo[CT];
    softmax_tiles<D, CT>(A, P, Plo, S, T);
    load_m(T, a.c, w, lane);
    add_values<D, CT, F32>(A, P, Plo, T);
    load_v(T, a.c, w, lane);
  }

  asm volatile("" : "+v"(lane));  // nothing of the outputs' places is kept over the loop
  const int64_t part0 = (int64_t)h * a.part_cap + x.part + (int64_t)x.share * R;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    // a row's sums over its four lanes; the zeros added to the outputs
    A.l[ct] = group_sum(A.l[ct]);
    A.z[ct] = group_sum(A.z[ct]);
    const int row = row0 + ct * 16 + (lane & 15);
    if (row >= R) continue;
    if (g == 0 && x.part >= 0) a.ml[part0 + row] = make_float2(A.m[ct], A.l[ct]);
    const int i = row / a.G;
    const int64_t at = (x.start + i) * a.o_token + (int64_t)(h * a.G + row - i * a.G) * a.o_head;
    const float inv = A.l[ct] == 0.f ? 0.f : 1.f / A.l[ct];
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 64 * hh + 16 * g + 4 * i;
        float4v v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(A.o[ct][4 * hh + j][i], kCentreScale, A.z[ct]);
        if (x.part >= 0) {
          *reinterpret_cast<float4v *>(&a.o[(part0 + row) * D + d]) = v;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            store_out(a, at + d + j, A.l[ct] == 0.f ? 0.f : v[j] * inv, F32);
        }
      }
  }
}

template <int D, bool F32>
__global__ __launch_bounds__(kThreads, 2) void packed_kernel(PackedArgs a) {
  __shared__ Meet<D> meet;
  const int h = blockIdx.x % a.c.H, items = a.head->items, base = a.head->base;
  // a launch has a workgroup for each item but where their number passes its limit
  for (int i = blockIdx.x / a.c.H; i < items; i += gridDim.x / a.c.H) {
    const Item x = a.items[i];
    if (x.n * a.G <= kFewRows)
      run_few<D, F32>(a, x, base, h, meet);
    else
      run_many<D, F32>(a, x, base, h);
    __syncthreads();  // meet is written again
  }
}

// Joins the shares of one row: own ones [own, + stride, ..), then the shared pages'.
template <int D, bool F32>
__device__ __forceinline__ void join_row(const PackedArgs &a, int64_t own, int64_t stride,
                                         int shares, int64_t few, int64_t few_stride,
                                         int few_shares, int64_t out, int lane) {
  const int all = shares + few_shares;
  const auto place = [&](int s) {
    return s < shares ? own + s * stride : few + (s - shares) * few_stride;
  };
  const float2 x = lane < all ? a.ml[place(lane)] : make_float2(kNegInf, 0.f);
  float m = x.x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float f = x.x == kNegInf ? 0.f : exp2f(x.x - m);
  float l = x.y * f;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
  float o[D / 64] = {};
  for (int s0 = 0; s0 < all; s0 += 4) {  // four shares' reads in flight
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = min(s0 + k, all - 1);
      const float fs = s0 + k < all ? __shfl(f, s) : 0.f;
      const float *from = a.o + place(s) * D;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const float v = from[c * 64 + lane];
        o[c] += s0 + k < all ? fs * v : 0.f;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    store_out(a, out + c * 64 + lane, l == 0.f ? 0.f : o[c] / l, F32);
}

// A wave a row: blocks [0, few_blocks) for the rows of sequences with few of them, the
// others for what is split of those with many.
template <int D, bool F32>
__global__ __launch_bounds__(kThreads) void join_kernel(PackedArgs a, int few_blocks) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const PlanHead h = *a.head;
  const int Hq = a.G * a.c.H;
  if ((int)blockIdx.x < few_blocks) {
    const int64_t r = (int64_t)blockIdx.x * kWaves + wave;
    const int k = (int)(r / Hq), hq = (int)(r % Hq);
    if (k * a.G >= h.few) return;
    const FewToken t = a.few[k];
    if (t.part < 0 && h.base == 0) return;
    const int g = hq % a.G;
    const int64_t at = (int64_t)(hq / a.G) * a.part_cap;
    join_row<D, F32>(a, at + t.part + g, t.rows_shares >> 8, t.part < 0 ? 0 : t.rows_shares & 255,
                     at + k * a.G + g, h.few, h.base > 0 ? h.few_shares : 0,
                     t.token * a.o_token + hq * a.o_head, lane);
    return;
  }
  const int64_t stride = (int64_t)(gridDim.x - few_blocks) * kWaves;
  for (int64_t r = (int64_t)(blockIdx.x - few_blocks) * kWaves + wave;
       r < (int64_t)h.split * a.c.H; r += stride) {
    const int row = (int)(r / a.c.H), head = (int)(r % a.c.H);
    int j = 0;
    for (int step = 1 << (31 - __clz(h.splits)); step > 0; step >>= 1)
      if (j + step < h.splits && a.splits[j + step].row <= row) j += step;
    const SplitSeq s = a.splits[j];
    const int mine = row - s.row, i = mine / a.G, hq = head * a.G + mine - i * a.G;
    join_row<D, F32>(a, (int64_t)head * a.part_cap + s.part + mine, (int64_t)s.n * a.G, s.shares,
                     0, 0, 0, (s.start + i) * a.o_token + hq * a.o_head, lane);
  }
}

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

// How many items, tokens and partial rows a call can have.  With C the blocks' steps
// in all, shares have at least C H / kTarget steps, so that the sum of steps / share
// over the blocks is at most kTarget / H, and a block has at most one share more than
// that; or, where kMostSteps is less, a block has at most `past`.
struct PackedPlan {
  int item_cap, few_cap;
  int64_t part_cap;
  size_t off_items, off_few, off_splits, off_ml, off_o, bytes;
};
PackedPlan packed_plan(int B, int H, int D, int room, int T, int q_heads, int max_n,
                       bool shared) {
  const int64_t G = q_heads / H, U = wave_rows(D), block = 4 * U;
  const int64_t seqs = std::min(B, T), rows = (int64_t)T * G;
  const int64_t few = std::min<int64_t>(T, seqs * (2 * U / G));
  const int64_t blocks = rows / block + 2 * seqs;  // two of up to kFewRows rows
  const int64_t few_blocks = shared ? few * G / block + 2 : 0;
  const int64_t target = kTarget / H + 1, past = room / (32 * kMostSteps) + 1;
  PackedPlan p;
  p.item_cap = (int)std::min<int64_t>(target + (blocks + few_blocks) * past, 1 << 30);
  p.few_cap = (int)std::max<int64_t>(few, 1);
  // rows of all the shares: a block's has at most `most`; blocks with one share have
  // none but those that meet the shared pages
  const int64_t most = std::min<int64_t>((int64_t)max_n * G <= kFewRows ? 16 : block,
                                         (int64_t)max_n * G);
  const int64_t own = std::min(target * most + rows, 2 * target * most + (shared ? few * G : 0));
  const int64_t met =
      shared ? target * std::min<int64_t>(few * G <= kFewRows ? 16 : block, few * G) + few * G : 0;
  p.part_cap = past == 1 ? own + met
                         : std::max(own, rows * past) + std::max(met, shared ? few * G * past : 0);
  size_t at = 256;
  p.off_items = at;
  at += pad256((size_t)(p.item_cap + B) * sizeof(Item));
  p.off_few = at;
  at += pad256((size_t)p.few_cap * sizeof(FewToken));
  p.off_splits = at;
  at += pad256((size_t)B * sizeof(SplitSeq));
  p.off_ml = at;
  at += pad256((size_t)H * p.part_cap * sizeof(float2));
  p.off_o = at;
  at += (size_t)H * p.part_cap * D * sizeof(float);
  p.bytes = p.part_cap < kMostParts ? at : 0;
  return p;
}

template <int D, bool F32>
hipError_t launch_dim(PackedArgs a, int q_heads, void *ws, hipStream_t s) {
  const PackedPlan p =
      packed_plan(a.c.B, a.c.H, D, a.c.room(), a.T, q_heads, a.max_n, a.shared > 0);
  char *w = static_cast<char *>(ws);
  a.head = reinterpret_cast<PlanHead *>(w);
  a.items = reinterpret_cast<Item *>(w + p.off_items);
  a.few = reinterpret_cast<FewToken *>(w + p.off_few);
  a.splits = reinterpret_cast<SplitSeq *>(w + p.off_splits);
  a.ml = reinterpret_cast<float2 *>(w + p.off_ml);
  a.o = reinterpret_cast<float *>(w + p.off_o);
  a.item_cap = p.item_cap, a.few_cap = p.few_cap, a.part_cap = (int)p.part_cap;
  plan_kernel<wave_rows(D)><<<1, kThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  packed_kernel<D, F32><<<(unsigned)std::min(p.item_cap, kMaxGroups / a.c.H) * a.c.H, kThreads, 0,
                          s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int few_blocks = (int)(((int64_t)p.few_cap * q_heads + kWaves - 1) / kWaves);
  const int many_blocks = (int64_t)a.max_n * a.G > 2 * wave_rows(D) ? 1024 : 0;
  join_kernel<D, F32><<<few_blocks + many_blocks, kThreads, 0, s>>>(a, few_blocks);
  return hipGetLastError();
}

}  // namespace

size_t packed_workspace_bytes(int B, int H, int D, int room, int T, int q_heads, int max_n,
                              bool shared) {
  return packed_plan(B, H, D, room, T, q_heads, max_n, shared).bytes;
}

hipError_t launch_kv_attend_packed(const PackedCall &r, float scale, int D, bcq_dtype dt,
                                   hipStream_t s) {
  PackedArgs a{};
  a.c = r.c;
  a.q = r.q, a.out = r.out;
  a.q_token = r.qs.token, a.q_head = r.qs.head, a.o_token = r.os.token, a.o_head = r.os.head;
  a.starts = r.starts;
  a.T = r.T, a.G = r.q_heads / r.c.H, a.max_n = r.max_n, a.shared = r.shared;
  a.q_wide = r.q_wide;
  // the same limits as in launch_kv_attend, for the same reasons
  if (dt == BCQ_F16) scale = fminf(fmaxf(scale, -0x1p80f), 0x1p80f);
  a.unit = fminf(fmaxf(scale * 1.44269504088896340736f, -FLT_MAX), FLT_MAX);
  a.code_unit = dt == BCQ_F16 ? a.unit * kCodeScale : 0.f;
  if (dt == BCQ_F32)
    return D == 64    ? launch_dim<64, true>(a, r.q_heads, r.ws, s)
           : D == 128 ? launch_dim<128, true>(a, r.q_heads, r.ws, s)
                      : launch_dim<256, true>(a, r.q_heads, r.ws, s);
  return D == 64    ? launch_dim<64, false>(a, r.q_heads, r.ws, s)
         : D == 128 ? launch_dim<128, false>(a, r.q_heads, r.ws, s)
                    : launch_dim<256, false>(a, r.q_heads, r.ws, s);
}

}  // namespace bcq
