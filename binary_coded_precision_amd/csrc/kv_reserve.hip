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

#include "serve_internal.h"

namespace bcq {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kMost = 1 << 30;  // sums stop here
// Entries, tokens and stack places up to which one workgroup does everything.
constexpr int64_t kAlone = 16384;

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
  int2 *back;       // [B] pages that come back: those before them, their number
  int32_t *staged;  // [B * max_pages] pages that came back, in their order on the stack
};

__device__ __forceinline__ int capped(int a, int b) { return min(a + b, kMost); }

// Inclusive sum of x over the workgroup's threads and the sum of all; x and the sums
// up to kMost.  `part` is free to be written.
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

// What is left once `given` and `head` are known, by `threads` threads of which this
// is number t: table entries (16 lanes a sequence; only the new ones where the
// table is updated in place), tokens, and the stack where it is not the one read.
__device__ __forceinline__ void fill(const ReserveArgs &a, const Head &h, int64_t t,
                                     int64_t threads) {
  const int log = a.c.page_log;
  const bool in_place = a.table_out == a.c.table;
  for (int64_t b = t >> 4; b < a.c.B; b += threads >> 4) {
    const Given g = a.given[b];
    for (int e = (in_place ? g.first : 0) + (int)(t & 15); e < g.first + g.need; e += 16)
      a.table_out[b * a.c.max_pages + e] = page_at(a, h, g, (int)b, e);
  }
  for (int64_t i = t; i < a.T; i += threads) {
    int32_t position = -1;
    int64_t slot = -1;
    if (i < h.tokens) {
      int b = 0;  // the last sequence that starts at i or before: the one with tokens there
      for (int step = 1 << (31 - __clz(a.c.B)); step > 0; step >>= 1)
        if (b + step < a.c.B && a.starts[b + step] <= i) b += step;
      const Given g = a.given[b];
      position = g.len + (int)(i - a.starts[b]);
      slot = ((int64_t)page_at(a, h, g, b, position >> log) << log) +
             (position & ((1 << log) - 1));
    }
    a.positions[i] = position;
    a.slots[i] = slot;
  }
  if (a.free_out != a.free_in)
    for (int64_t i = t; i < min(h.count, h.left); i += threads) a.free_out[i] = a.free_in[i];
}

// One workgroup: the sums, then the pages that came back, 16 lanes a sequence.  Where
// the rest is little it is done here too (ALL).
template <bool ALL>
__global__ __launch_bounds__(kThreads) void reserve_kernel(ReserveArgs a) {
  __shared__ int part[kWaves];
  __shared__ int most;
  const int tid = threadIdx.x, B = a.c.B;
  Head h;
  h.count = min(max(a.count_in[0], 0), a.c.num_pages);
  int back = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int n = sequence(a, b0 + tid).back;
    const int2 x = scan(n, part);
    if (b0 + tid < B) a.back[b0 + tid] = make_int2(back + x.x - n, n);
    back += x.y;
  }
  h.top = min(capped(h.count, back), a.c.num_pages);
  if (tid == 0) most = 0, a.starts[0] = 0;
  __syncthreads();
  int needed = 0, wanted = 0, tokens = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + tid;
    const Sequence q = sequence(a, b);
    const int2 need = scan(q.need, part), want = scan(q.want, part);
    const int with = capped(needed, need.x);
    const bool granted = capped(wanted, want.x) <= a.T && (q.need == 0 || with <= h.top);
    const int n = granted ? q.want : 0;
    const int2 given = scan(n, part);
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
  if (back > 0)
    for (int b = tid >> 4; b < B; b += kThreads >> 4) {
      const int2 x = a.back[b];
      for (int j = tid & 15; j < x.y; j += 16) {
        const int32_t page = a.c.table[(int64_t)b * a.c.max_pages + a.shared + j];
        a.staged[x.x + j] = page;
        if (h.count + x.x + j < h.left) a.free_out[h.count + x.x + j] = page;
      }
    }
  if constexpr (ALL) {
    __syncthreads();
    fill(a, h, tid, kThreads);
  }
}

__global__ __launch_bounds__(256) void fill_kernel(ReserveArgs a) {
  fill(a, *a.head, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t reserve_workspace_bytes(int B, int max_pages) {
  return 256 + pad256((size_t)B * sizeof(Given)) + pad256((size_t)B * sizeof(int2)) +
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
  a.back = reinterpret_cast<int2 *>(w);
  w += pad256((size_t)c.B * sizeof(int2));
  a.staged = reinterpret_cast<int32_t *>(w);
  const int64_t copies = (a.table_out != c.table ? (int64_t)c.B * c.max_pages : c.B) + r.T +
                         (a.free_out != a.free_in ? c.num_pages : 0);
  if (copies <= kAlone) {
    reserve_kernel<true><<<1, kThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  reserve_kernel<false><<<1, kThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  fill_kernel<<<(unsigned)std::min<int64_t>((copies + 255) / 256, 2048), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace bcq
