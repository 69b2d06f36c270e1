// kv_packed.hip -- attention of packed tokens, sequences with unlike numbers of them,
// over the 4-bit key/value cache (bcq_kv_attend_packed); the mathematics and a
// wave's steps are in kv_tiles.h.
//
// What a call has to do is known on the device only (starts, lengths).  It is cut into
// items, one for a workgroup and cached head:
//
//  - A sequence's rows (its tokens, times the query heads of a cached head) are
//    blocks of four waves' rows.  Where they are few, a block has 16 and its waves
//    share the tokens instead.
//  - Its tokens are cut into shares, so that all items together are about as many as
//    the card holds and none is much longer than the others.
//  - Rows of sequences with few of them (decode steps, drafted tokens) all meet the
//    shared pages together, as the rows of one sequence: those pages are read
//    from memory once, and 32 rows (a wave's; 16 of 256 channels, or where there are
//    few) share the unpacking of their codes.  A block's other waves, and other
//    blocks, unpack them again, from the caches.  The sequences'
//    own items then start behind the shared pages.  Sequences with many rows gain
//    nothing from that and read the shared pages as their own.
//
// Shares leave sums and outputs before the division, which a last kernel joins; what
// has one share only is written at once.
//
// Up to 64 sequences every wave works all that out by itself, a sequence a lane (a
// kernel for it took 6 us of a small call's 18); for more a first kernel writes it down.
#include <algorithm>

#include "kv_tiles.h"
#include "lane_sums.h"

namespace bcq {
namespace {

using namespace kv;

constexpr int kThreads = 256, kWaves = 4;
constexpr int kMaxShares = 64;  // of a row, one a lane where they are joined
// Workgroups that a call is cut into when there is enough to do: two a compute unit,
// as many as their registers leave room for.
constexpr int kTarget = 512;
constexpr int kUnits = kTarget / 2;
constexpr int kNearTurn = kUnits / 5;
constexpr int kMaxGroups = (1 << 24) - 1;  // of 256 work items in a launch
constexpr int kMostParts = 1 << 30;        // partial rows of a cached head
constexpr int kMostSteps = 2048;  // of 32 tokens, that a wave sums in one go (kv_attend.hip)

// Rows of a wave in a block of many rows, tiles of 16 of them.
constexpr int wave_tiles(int D) { return D <= 128 ? 2 : 1; }
constexpr int wave_rows(int D) { return 16 * wave_tiles(D); }
// Rows up to which blocks have 16 and their waves share the tokens.  Four waves with rows of
// their own would leave two or three idle up to 64 rows of 128, but split blocks of 16
// unpack the codes again for each: past two of them that costs more.  Blocks of 32 with
// shared tokens took 42 us for 16 x 8 drafted tokens over 3000, two of 16 take 32.
constexpr int kFewRows = 32;
struct Shape {
  int blocks, waves, weight;  // waves that share a block's tokens; weight of a step
};
template <int U>
__host__ __device__ constexpr Shape shape_of(int rows) {
  return rows <= kFewRows ? Shape{(rows + 15) / 16, 4, 2}
                          : Shape{(rows + 4 * U - 1) / (4 * U), 1, 1 + U / 16};
}

struct PlanHead {
  int items;       // in use, the shared pages' first
  int few_items;   // those
  int base;        // tokens that sequences with few rows leave to the shared items
  int few;         // such sequences' tokens
  int few_shares;  // of the shared pages
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
  int row;  // rows before it
  int start, n, part, shares;
};
// What a row of the shared items needs to know of its token.
struct Listed {
  int token, last;
};
constexpr int kListed = 130;  // tokens that a block's rows belong to, at most

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
  int start, n, len, rows, blocks, steps, weight;
  bool few;
};
// U: rows of a wave.
template <int U>
__device__ __forceinline__ Seq seq_of(const PackedArgs &a, int start, int end, int len) {
  Seq q{};
  q.start = min(max(start, 0), a.T);
  q.n = min(max(min(max(end, 0), a.T) - q.start, 0), a.max_n);
  q.len = len;
  q.rows = q.n * a.G;
  q.few = q.n > 0 && q.rows <= 2 * U;
  return q;
}
template <int U>
__device__ __forceinline__ Seq seq_at(const PackedArgs &a, int b) {
  if (b >= a.c.B) return Seq{};
  return seq_of<U>(a, a.starts[b], a.starts[b + 1], kv_len(a.c, b));
}
// Blocks and their steps, of 32 tokens for each wave; base: tokens that sequences with few
// rows do not walk.
template <int U>
__device__ __forceinline__ void shape(Seq &q, int base) {
  const Shape s = shape_of<U>(q.rows);
  const int tiles = (max(0, q.len - (q.few ? base : 0)) + 31) / 32;
  q.blocks = s.blocks;
  q.steps = (tiles + s.waves - 1) / s.waves;
  q.weight = s.weight;
}

__device__ __forceinline__ int product(int a, int b) {
  return (int)min((int64_t)a * b, (int64_t)1 << 30);
}

// What a sequence's blocks take, in half steps of few rows; an item's start and end are
// worth kStart of them.  Two kernels work out the same plan: no two operations of it
// become one, which the compiler could do in one of them alone.
constexpr int kStart = 8;
__device__ __forceinline__ float weight_of(int blocks, int steps, int weight) {
#pragma clang fp contract(off)
  return (float)blocks * ((float)steps * (float)weight + (float)kStart);
}
// Lengths are cut by chunk: the steps' weight that a share should have.
__device__ __forceinline__ int chunk_of(const PackedArgs &a, float cost) {
#pragma clang fp contract(off)
  return max(1, (int)fminf(ceilf(cost * (float)a.c.H * (1.f / kTarget)), (float)(1 << 24)));
}
// A share of 128 rows costs its partial rows too, written and read again: with all the
// compute units at it some 0.03 of a step (half of that for rows of half the work).  N
// shares of c steps, W = N c in all, take c + 0.03 N steps, least for c = sqrt(0.03 W);
// 0.02 a unit of weight is what measured best.  It counts where the card is not full
// without: a prompt's 225 tokens in 40 heads 24 us, cut for 512 workgroups 31; 30 tokens
// of five in 28 heads of 256 channels 17 and 21.5.
template <int U>
__device__ __forceinline__ int wide_chunk_of(const PackedArgs &a, int chunk, float cost) {
#pragma clang fp contract(off)
  constexpr float kPart = 0.06f * (1 + U / 16);
  return max(chunk, (int)sqrtf(kPart * (float)a.c.H * cost));
}
__device__ __forceinline__ int shares_of(int steps, int weight, int chunk, int most) {
  const int by_chunk = (steps * weight + chunk - 1) / chunk;
  return min(max(max(by_chunk, (steps + kMostSteps - 1) / kMostSteps), 1), most);
}

// What the whole call is: the first part of a plan, from the sums over the sequences.
template <int U>
struct Whole {
  PlanHead h{};
  bool together;
  int few_blocks = 0, few_steps = 0, few_weight = 0, chunk, wide_chunk, most, used = 0;

  // sequences with few rows, and their tokens
  __device__ __forceinline__ Whole(const PackedArgs &a, int seqs, int tokens) {
    together = a.shared > 0 && seqs > 1 && tokens <= a.few_cap;
    h.base = together ? a.shared : 0;
    h.few = min(tokens, a.few_cap);
    if (together) {
      const Shape shape = shape_of<U>(h.few * a.G);
      few_blocks = shape.blocks;
      few_steps = ((a.shared + 31) / 32 + shape.waves - 1) / shape.waves;
      few_weight = shape.weight;
    }
    most = together ? kMaxShares / 2 : kMaxShares;
  }
  // the weight of all the sequences' own steps
  __device__ __forceinline__ void divide(const PackedArgs &a, float cost, float wide_cost) {
#pragma clang fp contract(off)
    const bool wide_few = h.few * a.G > kFewRows;
    const float few_cost = weight_of(few_blocks, few_steps, few_weight);
    chunk = chunk_of(a, cost + few_cost);
    wide_chunk = wide_chunk_of<U>(a, chunk, wide_cost + (wide_few ? few_cost : 0.f));
    if (!together) return;
    h.few_shares = shares_of(few_steps, few_weight, wide_few ? wide_chunk : chunk, most);
    // The shared items are much alike and start first, one on each compute unit, then a
    // second: with a second on half of the units the others would wait for those.  So
    // whole turns of them, the sequences' own items beside the last.  At 25 sizes (20 to 128
    // decode steps behind 4096 to 32768 tokens, 2 to 32 cached heads of 64 to 256 channels)
    // that is as fast as what the weights say or faster (11% less time at the median of the 20
    // sizes where the two differ): 64 behind 16384 tokens 56 us with 256 items rather than 384 in 63, 32 of 64
    // heads behind 8192 tokens 40 us with 256 rather than 272 in 50.  What lacks a fifth of a
    // turn is made a whole one (480 items: 80 us, with one turn 80); two fifths are too much
    // (128 decode steps, 416 items: 87 us, with two turns 94).
    const int wide = few_blocks * a.c.H, turns = (h.few_shares * wide + kNearTurn) / kUnits;
    if (h.few_shares * wide >= kUnits)
      h.few_shares = min(max(max(turns * kUnits / wide, 1),
                             (few_steps + kMostSteps - 1) / kMostSteps), most);
    if ((int64_t)h.few_shares * h.few * a.G > a.part_cap) h.few_shares = 0;
    used = h.few_shares * h.few * a.G;
    h.few_items = few_blocks * h.few_shares;
  }
  // shares of a sequence's blocks, and the partial rows that they leave
  __device__ __forceinline__ int shares(const Seq &q) const {
    if (q.blocks == 0 || (together && q.few && q.steps == 0)) return 0;
    return shares_of(q.steps, q.weight, q.rows > kFewRows ? wide_chunk : chunk, most);
  }
  __device__ __forceinline__ int rows(const Seq &q, int shares) const {
    return shares > 1 || (together && q.few) ? product(q.rows, shares) : 0;
  }
  // shares of one block are neighbours
  static __device__ __forceinline__ Item few_item(const PackedArgs &a, const PlanHead &h, int i) {
    return Item{-1, i / h.few_shares, i % h.few_shares, h.few_shares, 0, h.few, a.shared, 0};
  }
};
// Item j of a sequence: the last rows, which see the most, first.
__device__ __forceinline__ void pick(Item &x, int blocks, int j) {
  x.block = blocks - 1 - j / x.shares;
  x.share = j % x.shares;
}

// ---- up to 64 sequences, one a lane

struct LanePlan {
  PlanHead h;
  Seq q;  // the lane's sequence
  int shares, part, item, few, split;  // partial rows, items, few tokens, split rows before it
  bool many;                           // its rows are split ones
};
template <int U>
__device__ __forceinline__ LanePlan lane_plan(const PackedArgs &a, int lane) {
  LanePlan p;
  p.q = seq_at<U>(a, lane);
  const int few = lane_scan(p.q.few ? p.q.n : 0);
  Whole<U> whole(a, __popcll(__ballot(p.q.few)), last_lane(few));
  shape<U>(p.q, whole.h.base);
  const float weight = weight_of(p.q.blocks, p.q.steps, p.q.weight);
  whole.divide(a, lane_sum(weight), lane_sum(p.q.rows > kFewRows ? weight : 0.f));
  p.shares = whole.shares(p.q);
  const int rows = whole.rows(p.q, p.shares), end = capped(whole.used, lane_scan(rows));
  if (rows > 0 && end > a.part_cap) p.shares = 0;  // starts that are none
  p.part = rows > 0 && p.shares > 0 ? end - rows : -1;
  p.few = few - (p.q.few ? p.q.n : 0);
  p.many = p.shares > 1 && !p.q.few;
  const int split = lane_scan(p.many ? p.q.rows : 0), items = product(p.q.blocks, p.shares);
  p.split = split - (p.many ? p.q.rows : 0);
  const int total = lane_scan(items);
  p.item = total - items;
  if (__ballot(p.q.n > 0 && !p.q.few)) {
    // the longest sequences' items first, as workgroups are handed out in order
    p.item = 0;
    for (int j = 0; j < a.c.B; ++j) {
      const int steps = __builtin_amdgcn_readlane(p.q.steps, j);
      const int theirs = __builtin_amdgcn_readlane(items, j);
      const bool before = steps > p.q.steps || (steps == p.q.steps && j < lane);
      p.item = capped(p.item, before ? theirs : 0);
    }
  }
  p.item = capped(p.item, whole.h.few_items);
  p.h = whole.h;
  p.h.items = min(capped(last_lane(total), whole.h.few_items), a.item_cap);
  p.h.split = last_lane(split);
  return p;
}
// Item i, below p.h.items (one without rows where it is nobody's).
template <int U>
__device__ __forceinline__ Item lane_item(const PackedArgs &a, const LanePlan &p, int i) {
  if (i < p.h.few_items) return Whole<U>::few_item(a, p.h, i);
  const int items = product(p.q.blocks, p.shares);
  const uint64_t whose = __ballot(i >= p.item && i - p.item < items);
  if (whose == 0) return Item{};
  const int b = __builtin_ctzll(whose);
  const auto of = [&](int x) { return __builtin_amdgcn_readlane(x, b); };
  Item x{b, 0, 0, of(p.shares), of(p.q.start), of(p.q.n), of(p.q.len), of(p.part)};
  pick(x, of(p.q.blocks), i - of(p.item));
  return x;
}

// ---- more sequences

__device__ __forceinline__ float sum_of(float x, float *part) {
#pragma clang fp contract(off)
  x = lane_sum(x);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  x = (part[0] + part[1]) + (part[2] + part[3]);
  __syncthreads();
  return x;
}

template <int U>
__global__ __launch_bounds__(kThreads) void plan_kernel(PackedArgs a) {
  __shared__ int part[kWaves];
  __shared__ float partf[kWaves];
  __shared__ int offset[BCQ_KV_PACKED_MAX_BATCH];  // of a sequence's items
  const int tid = threadIdx.x, B = a.c.B;
  int seqs = 0, tokens = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const Seq q = seq_at<U>(a, b0 + tid);
    seqs += block_scan<kWaves>(q.few, part).y;
    tokens = capped(tokens, block_scan<kWaves>(q.few ? q.n : 0, part).y);
  }
  Whole<U> whole(a, seqs, tokens);
  float cost = 0.f, wide_cost = 0.f;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    Seq q = seq_at<U>(a, b0 + tid);
    shape<U>(q, whole.h.base);
    const float weight = weight_of(q.blocks, q.steps, q.weight);
    cost += sum_of(weight, partf);
    wide_cost += sum_of(q.rows > kFewRows ? weight : 0.f, partf);
  }
  whole.divide(a, cost, wide_cost);
  int used = whole.used, items = whole.h.few_items, few_before = 0, split = 0, splits = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + tid;
    Seq q = seq_at<U>(a, b);
    shape<U>(q, whole.h.base);
    int shares = whole.shares(q);
    const int rows = whole.rows(q, shares);
    const int2 pr = block_scan<kWaves>(rows, part);
    const int end = capped(used, pr.x);
    if (rows > 0 && end > a.part_cap) shares = 0;  // starts that are none
    const int at = rows > 0 && shares > 0 ? end - rows : -1, mine = product(q.blocks, shares);
    const int2 it = block_scan<kWaves>(mine, part), fw = block_scan<kWaves>(q.few ? q.n : 0, part);
    const bool many = shares > 1 && !q.few;
    const int2 sr = block_scan<kWaves>(many ? q.rows : 0, part);
    const int2 sn = block_scan<kWaves>(many, part);
    if (b < B) {
      offset[b] = capped(items, it.x) - mine;
      // an item's description, for those who write the items
      a.items[a.item_cap + b] = Item{b, q.blocks, 0, shares, q.start, q.n, q.len, at};
      if (q.few)
        for (int i = 0; i < q.n; ++i) {
          const int k = few_before + fw.x - q.n + i;
          if (k < a.few_cap)
            a.few[k] = FewToken{q.start + i, q.len - q.n + i, at < 0 ? -1 : at + i * a.G,
                                q.rows << 8 | shares};
        }
      if (many)
        a.splits[splits + sn.x - 1] = SplitSeq{split + sr.x - q.rows, q.start, q.n, at, shares};
    }
    used = capped(used, pr.y);
    items = capped(items, it.y);
    few_before = capped(few_before, fw.y);
    split = capped(split, sr.y);
    splits += sn.y;
  }
  PlanHead h = whole.h;
  h.items = min(items, a.item_cap);
  h.split = split;
  h.splits = splits;
  if (tid == 0) *a.head = h;
  __syncthreads();
  for (int i = tid; i < h.items; i += kThreads) {
    Item x;
    if (i < h.few_items) {
      x = whole.few_item(a, h, i);
    } else {
      int b = 0;
      for (int step = 1 << (31 - __clz(B)); step > 0; step >>= 1)
        if (b + step < B && offset[b + step] <= i) b += step;
      x = a.items[a.item_cap + b];
      pick(x, x.block, i - offset[b]);
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

// ---- a wave's step over 32 tokens
//
// As in kv_tiles.h, with the reference taken off inside a score's own sum: d = s - ref
// comes out of fma(q . c, ks, fma(kz, sum(q), -ref)), one operation a score less, and the
// factors enter as the fp16 that they are.  For references up to 2^18 that rounds no
// more than s itself would be; a row past that has ref 0 and `rest` taken off
// afterwards.
struct Ref {
  float ref, rest;  // their sum is the reference; rest is -inf where there is none yet
};
__device__ __forceinline__ Ref ref_of(float m) {
  return fabsf(m) < 0x1p18f ? Ref{m, 0.f} : Ref{0.f, m};
}

template <int D, int CT, bool F32>
__device__ __forceinline__ void step_scores(float4v (&S)[2][CT], const Tiles<D> &T,
                                            const Queries<D, CT, F32> &Q, const Sums<D, CT> &A,
                                            float code_unit) {
  float minus[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) minus[ct] = -ref_of(A.m[ct]).ref;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    tile_scores<D, CT, F32>(S[s], T, s, Q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const half2v f = pair_of(T.m[s][2 * i]);
      const float ks = F32 ? 0.f : fmaf((float)f[0], code_unit, 0.f);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const float t = fmaf((float)f[1], Q.sum[ct], minus[ct]);
        S[s][ct][i] = F32 ? fmaf((float)f[0], S[s][ct][i], t) : fmaf(S[s][ct][i], ks, t);
      }
    }
  }
}

template <int D, int CT>
__device__ __forceinline__ void step_softmax(Sums<D, CT> &A, Frag (&P)[CT], Frag (&Plo)[CT],
                                             float4v (&S)[2][CT], const Tiles<D> &T) {
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
  bool raise = false, rests = false;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const float rest = ref_of(A.m[ct]).rest;
    raise |= high[ct] - rest > room;
    rests |= rest != 0.f;
  }
  if (__any(raise || rests)) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const Ref was = ref_of(A.m[ct]);
      float top = kNegInf;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = fmaxf(top, S[s][ct][i] + rough_log2(T.m[s][2 * i + 1] & 0xffffu));
      raise_row(A, ct, group_max(top) + was.ref, high[ct] + was.ref);
      const Ref now = ref_of(A.m[ct]);
      // from the old reference to the new one; a row that has seen nothing has -inf
      // only, and no reference
      const float by = was.ref - now.ref - (now.rest > kNegInf ? now.rest : 0.f);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[s][ct][i] += by;
    }
  }
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
        float p[2], pv[2], rest[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          p[j] = __builtin_amdgcn_exp2f(S[s][ct][i + j]);
          A.l[ct] += p[j];
          A.z[ct] = fmaf(p[j], mid[j], A.z[ct]);
          pv[j] = fmaf((float)f[j][0], p[j], 0.f);
        }
        // cut off rather than rounded: what is left goes to Plo either way
        const half2v part = kv::cut(pv[0], pv[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) rest[j] = fmaf((float)f[j][0], p[j], -(float)part[j]);
        P[ct].p[2 * s + (i >> 1)] = part;
        Plo[ct].p[2 * s + (i >> 1)] = kv::cut(rest[0], rest[1]);
      }
    }
}

// Waves of the same rows meet here.
template <int D>
struct Meet {
  float o[kWaves][16][D + 4];
  float m[kWaves][16], l[kWaves][16];
};
// The first token of the list that a shared item's rows belong to.
template <int D>
__device__ __forceinline__ int listed_from(const PackedArgs &a, const Item &x) {
  return x.block * (x.n * a.G <= kFewRows ? 16 : kWaves * wave_rows(D)) / a.G;
}
// The rows of a wave: the last slot that each lane's sees, and the wave's first and last.
template <int CT>
struct Rows {
  int last[CT], high, low;
};
template <int D, int CT, bool F32>
__device__ __forceinline__ Rows<CT> rows_of(const PackedArgs &a, const Item &x,
                                            const Listed *list, int h, int row0, int lane,
                                            RawQueries<D, CT, F32> &raw) {
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
      const Listed t = list[i - listed_from<D>(a, x)];
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

// An item of few rows: 16 of them, four waves share the tokens.  A step is bound by its
// loads: 32 decode steps over 8192 to 4224 tokens of 8 heads of 128 channels (216 MB) take
// 65 us, 3.3 TB/s; 50 us where a call finds them in the last cache.
template <int D, bool F32>
__device__ __forceinline__ void run_few(const PackedArgs &a, const Item &x, const Listed *list,
                                        int base, int h, Meet<D> &meet) {
  int lane = threadIdx.x & 63;
  // opaque, so that nothing formed from it is kept in registers from item to item
  asm volatile("" : "+v"(lane));
  const int g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool shared = x.seq < 0;
  const int R = x.n * a.G, L = x.len, b = shared ? 0 : x.seq;
  const int row0 = x.block * 16, t0 = shared ? 0 : base;

  RawQueries<D, 1, F32> raw;
  const Rows<1> rows = rows_of<D, 1, F32>(a, x, list, h, row0, lane, raw);
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
    step_scores<D, 1, F32>(S, T, Q, A, a.code_unit);
    load_k(T, a.c, w, lane);
    if (tile >= free_end) mask_scores<D, 1>(S, T, A, t0 + tile * 32 + 4 * g, rows.last);
    Frag P[1], Plo[1];
    step_softmax<D, 1>(A, P, Plo, S, T);
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

// An item of many rows: every wave has rows of its own, 32 (16 of 256 channels, as many as
// its registers hold); waves past the last row have nothing to do.  Bound by instructions:
// a step of 32 rows over 32 tokens of 128 channels has 48 matrix instructions and 340
// others, of which unpacking is a third (fp32 calls 64 and 530: queries in two parts, and
// every product summed outside the matrix cores).  Six prompts of 2334 to 4001 tokens, 443
// us at the rate of a large matrix product, take 806 us; the vector ALUs are at work for 86%
// of that, the matrix cores for 40%, and the probabilities' second fp16 is 16 of the 48.
template <int D, bool F32>
__device__ __forceinline__ void run_many(const PackedArgs &a, const Item &x, const Listed *list,
                                         int base, int h) {
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
  const Rows<CT> rows = rows_of<D, CT, F32>(a, x, list, h, row0, lane, raw);
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
    step_scores<D, CT, F32>(S, T, Q, A, a.code_unit);
    load_k(T, a.c, w, lane);
    if (tile >= free_end) mask_scores<D, CT>(S, T, A, t0 + tile * 32 + 4 * g, rows.last);
    Frag P[CT], Plo[CT];
    step_softmax<D, CT>(A, P, Plo, S, T);
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
__device__ __forceinline__ void run(const PackedArgs &a, const Item &x, const Listed *list,
                                    int base, int h, Meet<D> &meet) {
  if (x.n * a.G <= kFewRows)
    run_few<D, F32>(a, x, list, base, h, meet);
  else
    run_many<D, F32>(a, x, list, base, h);
}

// SMALL: up to 64 sequences, and a workgroup for each item that there can be.  The smallest
// calls are a chain of latencies: lengths, pages, codes, then partial rows (8.8 us, and
// 4.4 for the join).
template <int D, bool F32, bool SMALL>
__global__ __launch_bounds__(kThreads, 2) void packed_kernel(PackedArgs a) {
  __shared__ Meet<D> meet;
  __shared__ Listed list[kListed];
  const int h = blockIdx.x % a.c.H, tid = threadIdx.x;
  if constexpr (SMALL) {
    const LanePlan p = lane_plan<wave_rows(D)>(a, tid & 63);
    const int i = blockIdx.x / a.c.H;
    if (i >= p.h.items) return;
    const Item x = lane_item<wave_rows(D)>(a, p, i);
    if (x.n == 0) return;
    if (x.seq < 0) {
      const int from = listed_from<D>(a, x);
      if (tid < 64 && p.q.few)
        for (int j = max(0, from - p.few); j < p.q.n && p.few + j < from + kListed; ++j)
          list[p.few + j - from] = Listed{p.q.start + j, p.q.len - p.q.n + j};
      __syncthreads();
    }
    run<D, F32>(a, x, list, p.h.base, h, meet);
  } else {
    // a launch has a workgroup for each item but where their number passes its limit
    const PlanHead head = *a.head;
    for (int i = blockIdx.x / a.c.H; i < head.items; i += gridDim.x / a.c.H) {
      const Item x = a.items[i];
      if (x.seq < 0) {
        const int k = listed_from<D>(a, x) + tid;
        if (tid < kListed && k < head.few) list[tid] = Listed{a.few[k].token, a.few[k].last};
        __syncthreads();
      }
      run<D, F32>(a, x, list, head.base, h, meet);
      __syncthreads();  // the shared memory is written again
    }
  }
}

// Joins the shares of ROWS rows, which have the same number of them: own ones [own, +
// stride, ..), then the shared pages'.
template <int ROWS>
struct JoinRows {
  int64_t own[ROWS], few[ROWS], out[ROWS];
  int live;  // of them; the others are not stored
};
template <int D, bool F32, int ROWS>
__device__ __forceinline__ void join_rows(const PackedArgs &a, const JoinRows<ROWS> &j,
                                          int64_t stride, int shares, int64_t few_stride,
                                          int few_shares, int lane) {
  const int all = shares + few_shares;
  const auto place = [&](int k, int s) {
    return s < shares ? j.own[k] + s * stride : j.few[k] + (s - shares) * few_stride;
  };
  float2 x[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k)
    x[k] = lane < all ? a.ml[place(k, lane)] : make_float2(kNegInf, 0.f);
  float f[ROWS], l[ROWS], o[ROWS][D / 64] = {};
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    float m = x[k].x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    f[k] = x[k].x == kNegInf ? 0.f : exp2f(x[k].x - m);
    l[k] = x[k].y * f[k];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) l[k] += __shfl_xor(l[k], d);
  }
  for (int s0 = 0; s0 < all; s0 += 4) {  // four shares' reads in flight
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int s = min(s0 + t, all - 1);
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const float fs = s0 + t < all ? __shfl(f[k], s) : 0.f;
        const float *from = a.o + place(k, s) * D;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const float v = from[c * 64 + lane];
          o[k][c] += s0 + t < all ? fs * v : 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    if (k >= j.live) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store_out(a, j.out[k] + c * 64 + lane, l[k] == 0.f ? 0.f : o[k][c] / l[k], F32);
  }
}

// A wave a row at a time, those of sequences with few of them first, then what is split of
// those with many.  Every wave works the plan out, so there are no more than the card
// holds at once: 31 decode steps beside a prompt's 1024 tokens 206 us (1024 workgroups
// 210, 4096 207, 8192 210).
constexpr int kJoins = 2048;
template <int D, bool F32, bool SMALL>
__global__ __launch_bounds__(kThreads) void join_kernel(PackedArgs a) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  LanePlan p;
  PlanHead h;
  if constexpr (SMALL) {
    p = lane_plan<wave_rows(D)>(a, lane);
    h = p.h;
  } else {
    h = *a.head;
  }
  const int Hq = a.G * a.c.H;
  // a split row of two cached heads at a time, so that twice as many reads are on their way:
  // a prompt's 2252 tokens 62 us, one at a time 67
  const int halves = (a.c.H + 1) / 2;
  const int64_t few = (int64_t)h.few * Hq, all = few + (int64_t)h.split * halves;
  for (int64_t r = (int64_t)blockIdx.x * kWaves + wave; r < all;
       r += (int64_t)gridDim.x * kWaves) {
    if (r < few) {
      const int k = (int)(r / Hq), hq = (int)(r % Hq), g = hq % a.G;
      FewToken t;
      if constexpr (SMALL) {
        const uint64_t whose = __ballot(p.q.few && k >= p.few && k - p.few < p.q.n);
        if (whose == 0) continue;
        const int b = __builtin_ctzll(whose);
        const auto of = [&](int x) { return __builtin_amdgcn_readlane(x, b); };
        const int i = k - of(p.few), part = of(p.part);
        t = FewToken{of(p.q.start) + i, 0, part < 0 ? -1 : part + i * a.G,
                     of(p.q.rows) << 8 | of(p.shares)};
      } else {
        t = a.few[k];
      }
      if (t.part < 0 && h.base == 0) continue;
      const int64_t at = (int64_t)(hq / a.G) * a.part_cap;
      const JoinRows<1> rows{
          {at + t.part + g}, {at + k * a.G + g}, {t.token * a.o_token + hq * a.o_head}, 1};
      join_rows<D, F32, 1>(a, rows, t.rows_shares >> 8, t.part < 0 ? 0 : t.rows_shares & 255,
                           h.few * a.G, h.base > 0 ? h.few_shares : 0, lane);
      continue;
    }
    const int row = (int)((r - few) / halves), head = (int)((r - few) % halves);
    SplitSeq s;
    if constexpr (SMALL) {
      const uint64_t whose = __ballot(p.many && row >= p.split && row - p.split < p.q.rows);
      if (whose == 0) return;
      const int b = __builtin_ctzll(whose);
      const auto of = [&](int x) { return __builtin_amdgcn_readlane(x, b); };
      s = SplitSeq{of(p.split), of(p.q.start), of(p.q.n), of(p.part), of(p.shares)};
    } else {
      int j = 0;
      for (int step = 1 << (31 - __clz(h.splits)); step > 0; step >>= 1)
        if (j + step < h.splits && a.splits[j + step].row <= row) j += step;
      s = a.splits[j];
    }
    const int mine = row - s.row, i = mine / a.G, next = min(head + halves, a.c.H - 1);
    JoinRows<2> rows{{}, {}, {}, head + halves < a.c.H ? 2 : 1};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int at = k == 0 ? head : next;
      rows.own[k] = (int64_t)at * a.part_cap + s.part + mine;
      rows.out[k] = (s.start + i) * a.o_token + (int64_t)(at * a.G + mine - i * a.G) * a.o_head;
    }
    join_rows<D, F32, 2>(a, rows, (int64_t)s.n * a.G, s.shares, 0, 0, lane);
  }
}

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

// How many items, tokens and partial rows a call can have.  With C the blocks' steps
// in all, shares have at least C H / kTarget steps, so that the sum of steps / share
// over the blocks is at most kTarget / H (and kNearTurn / H for the shared pages'), and a
// block has at most one share more than that; where kMostSteps cuts a block further, it
// has at most `past` besides.
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
  const int64_t target = (kTarget + kNearTurn) / H + 1, past = room / (32 * kMostSteps) + 1;
  PackedPlan p;
  const int64_t cuts = past == 1 ? 1 : past + 1;  // of a block, but for the target's
  p.item_cap = (int)std::min<int64_t>(target + (blocks + few_blocks) * cuts, 1 << 30);
  p.few_cap = (int)std::max<int64_t>(few, 1);
  // rows of all the shares: a block's has at most `most`; blocks with one share have
  // none but those that meet the shared pages
  const int64_t most = std::min<int64_t>((int64_t)max_n * G <= kFewRows ? 16 : block,
                                         (int64_t)max_n * G);
  const int64_t own = std::min(target * most + rows, 2 * target * most + (shared ? few * G : 0));
  const int64_t met =
      shared ? target * std::min<int64_t>(few * G <= kFewRows ? 16 : block, few * G) + few * G : 0;
  p.part_cap = own + met + (past == 1 ? 0 : (rows + (shared ? few * G : 0)) * past);
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
  const int joins = (int)std::min<int64_t>(((int64_t)a.T * q_heads + kWaves - 1) / kWaves, kJoins);
  const int most = kMaxGroups / a.c.H;
  if (a.c.B <= 64 && p.item_cap <= most) {
    packed_kernel<D, F32, true><<<(unsigned)p.item_cap * a.c.H, kThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    join_kernel<D, F32, true><<<joins, kThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  plan_kernel<wave_rows(D)><<<1, kThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  packed_kernel<D, F32, false>
      <<<(unsigned)std::min(p.item_cap, most) * a.c.H, kThreads, 0, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  join_kernel<D, F32, false><<<joins, kThreads, 0, s>>>(a);
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
