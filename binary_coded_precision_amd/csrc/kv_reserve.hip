// kv_reserve.hip -- pages of the key/value cache given to a step's new tokens and
// taken back from sequences that ended (bcq_kv_reserve).
//
// All of it is sums over the sequences in their order: the pages that come back go
// on top of the stack of free ones one sequence after another, and a request gets
// its pages from the top if those asked for up to and with it do not pass what is
// there.  So three prefix sums (pages back; pages and tokens asked for; tokens
// given) decide everything, and what is left is copying: every page, token and
// table entry then finds its source by itself.
#include <algorithm>

#include "lane_sums.h"
#include "serve_internal.h"

namespace bcq {
namespace {

// Tokens up to which one workgroup does everything, for up to 64 and up to 256 sequences.  A
// second launch costs 3 us or so, and one workgroup comes to little.  64 sequences with 64,
// 4096, 8192 tokens: 3.9, 6.8, 10.1 us, two launches 6.9, 9.2, 9.0; 200 with 200, 4096: 5.8,
// 22, two launches 7.4, 7.4.
// A place of a stack that is copied counts a quarter: 64 sequences with 64 tokens and 8000,
// 16000, 24000, 32000 places 5.1, 6.1, 7.1, 8.1 us, two launches 7.1.  Entries of tables that
// are copied have 16 lanes a sequence in either form: up to 64 sequences they count nothing (64
// full tables of 128, 256, 512 pages 5.3, 6.7, 9.5 us, two launches 8.3, 9.6, 12.1; one of 8192
// pages 70 and 74).  Past that the one workgroup, of 256 threads, has a few sequences' copies
// one behind the other; there an entry counts a quarter (100 sequences with 17 entries 6.9 us,
// two launches 7.2; 200 with 5 entries 9.2 and 7.6; 70 with 21 entries, the worst, are given two
// launches, 7.2, where one workgroup takes 6.2).
constexpr int64_t kAloneSmall = 6144, kAlone = 512;
// Sequences whose starts, or pages, a workgroup looks up in shared memory.
constexpr int kStarts = 4096;

struct Given {
  int32_t len, first, need, base;  // cached before; pages before; new pages; those before them
};
struct Head {
  int32_t count, top;  // free pages before, with those that came back
  int32_t left, tokens;
};

struct ReserveArgs {
  KvView c;
  const int32_t *want, *release, *free_in, *count_in;
  int32_t *lens_out, *table_out, *free_out, *count_out, *starts, *positions;
  int64_t *slots;
  int shared, T;
  // workspace
  Head *head;
  Given *given;     // [B]
  int *back;        // [B] pages that come back before a sequence's
  int32_t *staged;  // [B * max_pages] pages that came back, in their order on the stack
};

struct Sequence {
  int len, back, want, first, need;
  bool fits;
};
__device__ __forceinline__ Sequence sequence(const ReserveArgs &a, int b) {
  Sequence q{};
  if (b >= a.c.B) return q;
  const int log = a.c.page_log, room = a.c.room(), ahead = a.shared << log;
  const auto pages = [&](int n) { return max((n + (1 << log) - 1) >> log, a.shared); };
  const int len = max(kv_len(a.c, b), ahead);
  const bool gone = a.release != nullptr && a.release[b] != 0;
  q.back = gone ? pages(len) - a.shared : 0;
  q.len = gone ? ahead : len;
  const int want = max(a.want[b], 0);
  q.fits = want <= room - q.len;
  q.want = q.fits ? want : 0;
  q.first = pages(q.len);
  q.need = pages(q.len + q.want) - q.first;
  return q;
}

// A page of the stack as it is with those that came back.
__device__ __forceinline__ int32_t stack_at(const ReserveArgs &a, const Head &h, int i) {
  return i < h.count ? a.free_in[i] : a.staged[i - h.count];
}
// Entry e of sequence b's table, e below its pages after the call.
__device__ __forceinline__ int32_t page_at(const ReserveArgs &a, const Head &h, const Given &g,
                                           int b, int e) {
  return e < g.first ? a.c.table[(int64_t)b * a.c.max_pages + e]
                     : stack_at(a, h, h.top - 1 - (g.base + e - g.first));
}

// The sequence that packed token i belongs to (or page i of those that came back), i below
// all of them: the last one that starts at i or before.
template <typename S>
__device__ __forceinline__ int owner(const S &starts, int B, int i) {
  int b = 0;
  for (int step = 1 << (31 - __clz(B)); step > 0; step >>= 1)
    if (b + step < B && starts[b + step] <= i) b += step;
  return b;
}

// What is left once all sequences are `given` theirs, by `threads` threads of which this
// is number t: table entries (16 lanes a sequence; only the new ones where the
// table is updated in place), tokens, and the stack where it is not the one read.
template <typename S, typename G>
__device__ __forceinline__ void fill(const ReserveArgs &a, const Head &h, const S &starts,
                                     const G &given, int64_t t, int64_t threads) {
  const int log = a.c.page_log;
  const bool in_place = a.table_out == a.c.table;
  for (int64_t b = t >> 4; b < a.c.B; b += threads >> 4) {
    const Given g = given[b];
    for (int e = (in_place ? g.first : 0) + (int)(t & 15); e < g.first + g.need; e += 16)
      a.table_out[b * a.c.max_pages + e] = page_at(a, h, g, (int)b, e);
  }
  for (int64_t i = t; i < a.T; i += threads) {
    int32_t position = -1;
    int64_t slot = -1;
    if (i < h.tokens) {
      const int b = owner(starts, a.c.B, (int)i);
      const Given g = given[b];
      position = g.len + (int)(i - starts[b]);
      slot = ((int64_t)page_at(a, h, g, b, position >> log) << log) +
             (position & ((1 << log) - 1));
    }
    a.positions[i] = position;
    a.slots[i] = slot;
  }
  if (a.free_out != a.free_in)
    for (int64_t i = t; i < min(h.count, h.left); i += threads) a.free_out[i] = a.free_in[i];
}

// The pages that came back, `total` of them, sequence b's behind `before[b]` others.
template <typename S>
__device__ __forceinline__ void take_back(const ReserveArgs &a, const Head &h, const S &before,
                                          int total, int t, int threads) {
  for (int i = t; i < total; i += threads) {
    const int b = owner(before, a.c.B, i);
    const int32_t page = a.c.table[(int64_t)b * a.c.max_pages + a.shared + i - before[b]];
    a.staged[i] = page;
    if (h.count + i < h.left) a.free_out[h.count + i] = page;
  }
}

// Up to 64 sequences and little to copy: every wave works the sums out by itself, a
// sequence a lane, and the waves share the copying.  64 decoding requests: 3.6 us
// where the general kernel took 7.7.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void small_kernel(ReserveArgs a) {
  __shared__ int starts[65];
  __shared__ Given given[64];
  __shared__ int back[64];
  const int tid = threadIdx.x, lane = tid & 63, B = a.c.B;
  const Sequence q = sequence(a, lane);
  Head h;
  h.count = min(max(a.count_in[0], 0), a.c.num_pages);
  const int returned = lane_scan(q.back);
  h.top = min(capped(h.count, last_lane(returned)), a.c.num_pages);
  const int need = lane_scan(q.need), want = lane_scan(q.want);
  const bool granted = want <= a.T && (q.need == 0 || need <= h.top);
  const int n = granted ? q.want : 0, ends = lane_scan(n);
  // those granted pages are the first that asked for some
  const uint64_t some = __ballot(granted && q.need > 0);
  h.left = h.top - (some == 0 ? 0 : __builtin_amdgcn_readlane(need, 63 - __builtin_clzll(some)));
  h.tokens = last_lane(ends);
  if (tid < 64) {
    starts[lane + 1] = ends;
    given[lane] = Given{q.len, q.first, granted ? q.need : 0, need - q.need};
    back[lane] = returned - q.back;
    if (lane == 0) starts[0] = 0;
  }
  __syncthreads();  // what is updated in place has been read
  if (tid < B) {
    a.lens_out[lane] = q.len + n;
    a.starts[lane + 1] = ends;
    if (lane == 0) {
      a.starts[0] = 0;
      a.count_out[0] = h.left;
    }
  }
  if (last_lane(returned) > 0) {
    take_back(a, h, back, last_lane(returned), tid, THREADS);
    __syncthreads();
  }
  fill(a, h, starts, given, tid, THREADS);
}

// One workgroup: the sums, then the pages that came back.  Where the rest is little it is
// done here too (ALL).
template <bool ALL, int THREADS>
__global__ __launch_bounds__(THREADS) void reserve_kernel(ReserveArgs a) {
  constexpr int WAVES = THREADS / 64;
  __shared__ int part[WAVES];
  __shared__ int most;
  __shared__ int before[kStarts];
  const int tid = threadIdx.x, B = a.c.B;
  Head h;
  h.count = min(max(a.count_in[0], 0), a.c.num_pages);
  int back = 0;
  if (a.release != nullptr)
    for (int b0 = 0; b0 < B; b0 += THREADS) {
      const int n = sequence(a, b0 + tid).back;
      const int2 x = block_scan<WAVES>(n, part);
      if (b0 + tid < B) {
        a.back[b0 + tid] = back + x.x - n;
        if (b0 + tid < kStarts) before[b0 + tid] = back + x.x - n;
      }
      back += x.y;
    }
  h.top = min(capped(h.count, back), a.c.num_pages);
  if (tid == 0) most = 0, a.starts[0] = 0;
  __syncthreads();
  int needed = 0, wanted = 0, tokens = 0;
  for (int b0 = 0; b0 < B; b0 += THREADS) {
    const int b = b0 + tid;
    const Sequence q = sequence(a, b);
    const int2 need = block_scan<WAVES>(q.need, part), want = block_scan<WAVES>(q.want, part);
    const int with = capped(needed, need.x);
    const bool granted = capped(wanted, want.x) <= a.T && (q.need == 0 || with <= h.top);
    const int n = granted ? q.want : 0;
    const int2 given = block_scan<WAVES>(n, part);
    if (b < B) {
      a.starts[b + 1] = tokens + given.x;
      a.given[b] = Given{q.len, q.first, granted ? q.need : 0, with - q.need};
      a.lens_out[b] = q.len + n;
      if (granted && q.need > 0) atomicMax(&most, with);
    }
    needed = capped(needed, need.y);
    wanted = capped(wanted, want.y);
    tokens += given.y;
  }
  __syncthreads();
  h.left = h.top - most;
  h.tokens = tokens;
  if (tid == 0) {
    *a.head = h;
    a.count_out[0] = h.left;
  }
  if (back > 0 && B <= kStarts)
    take_back(a, h, before, back, tid, THREADS);
  else if (back > 0)
    take_back(a, h, a.back, back, tid, THREADS);
  if constexpr (ALL) {
    __syncthreads();
    fill(a, h, a.starts, a.given, tid, THREADS);
  }
}

// A thread an entry, token and place.  Bound by the latency of a few loads one behind the
// other: 200 sequences with 28000 new tokens take 5 us.
__global__ __launch_bounds__(256) void fill_kernel(ReserveArgs a) {
  constexpr int kGiven = 1024;
  __shared__ int starts[kStarts];
  __shared__ Given given[kGiven];
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x, threads = (int64_t)gridDim.x * 256;
  const Head h = *a.head;
  if (a.c.B <= kGiven) {
    for (int b = threadIdx.x; b < a.c.B; b += 256) {
      starts[b] = a.starts[b];
      given[b] = a.given[b];
    }
    __syncthreads();
    fill(a, h, starts, given, t, threads);
  } else if (a.c.B <= kStarts) {
    for (int b = threadIdx.x; b < a.c.B; b += 256) starts[b] = a.starts[b];
    __syncthreads();
    fill(a, h, starts, a.given, t, threads);
  } else {
    fill(a, h, a.starts, a.given, t, threads);
  }
}

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t reserve_workspace_bytes(int B, int max_pages) {
  return 256 + pad256((size_t)B * sizeof(Given)) + pad256((size_t)B * sizeof(int)) +
         (size_t)B * max_pages * 4;
}

hipError_t launch_kv_reserve(const KvView &c, const ReserveCall &r, void *ws, hipStream_t s) {
  ReserveArgs a{};
  a.c = c;
  a.want = r.new_tokens, a.release = r.release, a.free_in = r.free_pages;
  a.count_in = r.free_count;
  a.lens_out = r.lens_out, a.table_out = r.table_out, a.free_out = r.free_out;
  a.count_out = r.count_out, a.starts = r.starts, a.positions = r.positions, a.slots = r.slots;
  a.shared = r.shared_pages, a.T = r.T;
  char *w = static_cast<char *>(ws);
  a.head = reinterpret_cast<Head *>(w);
  w += 256;
  a.given = reinterpret_cast<Given *>(w);
  w += pad256((size_t)c.B * sizeof(Given));
  a.back = reinterpret_cast<int *>(w);
  w += pad256((size_t)c.B * sizeof(int));
  a.staged = reinterpret_cast<int32_t *>(w);
  const int64_t places = a.free_out != a.free_in ? c.num_pages : 0;
  const int64_t copies =
      (a.table_out != c.table ? (int64_t)c.B * c.max_pages : c.B) + r.T + places;
  if (c.B <= 64 && r.T + places / 4 <= kAloneSmall) {
    small_kernel<1024><<<1, 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  if (c.B <= 256 && r.T + (copies - r.T) / 4 <= kAlone) {
    reserve_kernel<true, 256><<<1, 256, 0, s>>>(a);
    return hipGetLastError();
  }
  // many threads for the pages that come back
  reserve_kernel<false, 1024><<<1, 1024, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  fill_kernel<<<(unsigned)std::min<int64_t>((copies + 255) / 256, 2048), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace bcq
