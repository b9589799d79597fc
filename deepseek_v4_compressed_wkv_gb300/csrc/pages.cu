// The page table of paged caches (see include/csa.h): sequences that grow, fork, end, and are packed
// together, and the copying of a cache's pages that follows.
//
// All of it is exact integer work whose results do not depend on timing: pages are handed out lowest
// first, in the sequences' order, by prefix sums over the use counts; counts change by atomic additions
// only.  Nothing is kept besides the counts (no list of free pages that could disagree with them).
//
// One CTA or one cluster does a step, in phases between barriers; each warp owns a contiguous range of
// pages and one of sequences, leaves its sums where all can read them, and finds its place by adding up the
// sums of the warps before it.  A step is a chain of trips to memory, about 0.7 us each; launches of their own
// would add 2 us a phase.  A CTA alone has its sums and the sequences' heirs in shared memory and cheaper barriers; a cluster
// has more warps for the sequences' rows and reads the counts faster.  us in a graph, one CTA and clusters of 4 and 8:
// fork of 8 sequences 5.6, 8.5 and 8.9, of 128 of up to 35 pages 11.3, 10.7 and 11.0; extension of 128 2.7, 4.4 and 4.8;
// packing of 1000 pages 4.4, 8.0 and 8.4, of 16384 with 128 sequences 20.7, 11.5 and 11.9.
#include <cstdlib>

#include "layer_ops.h"
#include "tc_common.cuh"

namespace csa {
namespace {

using namespace tcx;

constexpr int kThreads = 1024;
constexpr int kMostCtas = 8;
constexpr int kMostWarps = kMostCtas * kThreads / 32;
constexpr int kOutOfPages = 1, kBadArgument = 2, kBadPage = 4;  // bits of the status word

struct PagesParams {
  csa_pages t;
  const int32_t* in;  // more or parent
  int32_t* first;
  int32_t *src, *dst, *count;
  int moves;             // entries of src and dst
  int ctas;
  // the workspace's parts
  int32_t *sum0, *sum1;  // [kMostWarps] each
  int32_t* list;         // [pages] free pages, or the movers' ranks
  int32_t *heirs, *keep; // [sequences] each
  int32_t* len;          // [sequences] the parents' entries
  int32_t* rows;         // [sequences][max_pages] the parents' pages
#ifdef CSA_DEBUG_BOUNDS
  int less;              // the test of the checks: extents that much shorter
#endif
};

// This warp's place among the step's, and the barrier between phases.  kOne: a CTA alone.
constexpr int kFewSequences = 1024;  // of a CTA alone: their heirs are in shared memory
template <bool kOne>
struct Team {
  int w, warps, lane;
  __device__ explicit Team(int ctas) {
    w = (kOne ? 0 : (int)cluster_rank()) * (kThreads / 32) + (int)(threadIdx.x >> 5);
    warps = (kOne ? 1 : ctas) * (kThreads / 32);
    lane = threadIdx.x & 31;
  }
  __device__ void sync() const {
    if constexpr (kOne) {
      __syncthreads();
    } else {
      cluster_arrive();
      cluster_wait();
    }
  }
  // what warps leave one another: in shared memory, or in global memory past the SMs' own caches
  static __device__ int load(const int32_t* p) { return kOne ? *reinterpret_cast<const volatile int32_t*>(p) : __ldcg(p); }
  static __device__ void store(int32_t* p, int v) {
    if constexpr (kOne) *reinterpret_cast<volatile int32_t*>(p) = v; else __stcg(p, v);
  }
  __device__ int2 range(int n) const {  // of n things
    const long long a = (long long)n * w / warps, b = (long long)n * (w + 1) / warps;
    return make_int2((int)a, (int)b);
  }
  __device__ void leave(int32_t* sums, int v) const {  // v: each lane's part
    v = __reduce_add_sync(0xffffffffu, v);
    if (lane == 0) store(sums + w, v);
  }
  __device__ int2 add_up(const int32_t* sums) const {  // the warps' before this one, all
    int a = 0, b = 0;
    for (int i = lane; i < warps; i += 32) {
      const int v = load(sums + i);
      b += v;
      if (i < w) a += v;
    }
    return make_int2(__reduce_add_sync(0xffffffffu, a), __reduce_add_sync(0xffffffffu, b));
  }
};
__device__ __forceinline__ int lane_scan(int v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}
__device__ __forceinline__ int pages_for(long long entries, int page_size) { return (int)((entries + page_size - 1) / page_size); }
__device__ __forceinline__ void raise(const PagesParams& P, int bits) {
  if (P.t.status) atomicOr(P.t.status, bits);
}
// Whether element i of an array of n may be written: the bounds-checked build's check (bit 8 of the status word).
#ifdef CSA_DEBUG_BOUNDS
__device__ __forceinline__ bool inside(const PagesParams& P, long long i, long long n) {
  if (i >= 0 && i < n - P.less) return true;
  raise(P, 8);
  return false;
}
#else
__device__ __forceinline__ bool inside(const PagesParams&, long long, long long) { return true; }
#endif
__device__ __forceinline__ long long slots(const PagesParams& P) { return (long long)P.t.sequences * P.t.max_pages; }

// Entries of sequence b; a number that its pages cannot hold raises the flag and is taken as none.
__device__ __forceinline__ int entries_of(const PagesParams& P, int b, bool tell) {
  const int n = __ldcg(P.t.lens + b);
  if (n >= 0 && n <= (long long)P.t.max_pages * P.t.page_size) return n;
  if (tell) raise(P, kBadArgument);
  return 0;
}
// A row of n pages, a warp's: load(j) of eight slots a lane before use(j, v) of any, since for the compiler what is stored
// might be what the next load reads (us, 32 rows of 4096 pages, one slot at a time, four and eight: fork 81, 39 and 33, extension
// 41, 19 and 15, packing of half of them 129, 60 and 54).  load has no branch, and may be asked for the last slot again.
constexpr int kRowAhead = 8;
template <class Load, class Use>
__device__ __forceinline__ void over_row(int n, int lane, Load load, Use use) {
  if (n <= 32) {
    if (lane < n) use(lane, load(lane));
    return;
  }
  for (int j = lane; j < n; j += 32 * kRowAhead) {
    int v[kRowAhead];
#pragma unroll
    for (int k = 0; k < kRowAhead; ++k) v[k] = load(min(j + 32 * k, n - 1));
#pragma unroll
    for (int k = 0; k < kRowAhead; ++k)
      if (j + 32 * k < n) use(j + 32 * k, v[k]);
  }
}
__device__ __forceinline__ bool in_pool(const PagesParams& P, int page) { return page >= 0 && page < P.t.pages; }

__device__ __forceinline__ int count_pages(const PagesParams& P, int2 r, int lane, bool live) {
  int n = 0;
#pragma unroll 4
  for (int p = r.x + lane; p < r.y; p += 32) n += (__ldcg(P.t.refs + p) != 0) == live;
  return n;
}
constexpr int kPoolAhead = 4;  // (as rows)
// The lowest `most` free pages into the list, `at` of which lie before this warp's range.
__device__ __forceinline__ void list_free(const PagesParams& P, int2 r, int at, int most, int lane) {
  for (int p0 = r.x; p0 < r.y && at < most; p0 += 32 * kPoolAhead) {
    bool free[kPoolAhead];
#pragma unroll
    for (int k = 0; k < kPoolAhead; ++k) free[k] = p0 + 32 * k + lane < r.y && __ldcg(P.t.refs + p0 + 32 * k + lane) == 0;
#pragma unroll
    for (int k = 0; k < kPoolAhead && p0 + 32 * k < r.y; ++k) {
      const uint32_t who = __ballot_sync(0xffffffffu, free[k]);
      const int i = at + __popc(who & ((1u << lane) - 1));
      if (free[k] && i < most && inside(P, i, P.t.pages)) __stcg(P.list + i, p0 + 32 * k + lane);
      at += __popc(who);
    }
  }
}

// ---- each sequence gets pages for `more` new entries
__device__ __forceinline__ int pages_wanted(const PagesParams& P, int b, int& len, int& more, bool& ok) {
  len = __ldcg(P.t.lens + b);
  more = __ldcg(P.in + b);
  const long long top = (long long)P.t.max_pages * P.t.page_size;
  ok = len >= 0 && len <= top && more >= 0 && (long long)len + more <= top;
  return ok ? pages_for((long long)len + more, P.t.page_size) - pages_for(len, P.t.page_size) : 0;
}
template <bool kOne>
__global__ void __launch_bounds__(kThreads, 1) pages_extend_kernel(const __grid_constant__ PagesParams P) {
  __shared__ int32_t sums[2][kOne ? kThreads / 32 : 1];
  griddep_wait();
  griddep_launch_dependents();
  const Team<kOne> T(P.ctas);
  int32_t *const sum0 = kOne ? sums[0] : P.sum0, *const sum1 = kOne ? sums[1] : P.sum1;
  const int lane = T.lane;
  const int2 mine = T.range(P.t.pages), seqs = T.range(P.t.sequences);
  int want = 0, len, more;
  bool ok;
  for (int b = seqs.x + lane; b < seqs.y; b += 32) want += pages_wanted(P, b, len, more, ok);
  T.leave(sum0, count_pages(P, mine, lane, false));
  T.leave(sum1, want);
  T.sync();
  const int2 free = T.add_up(sum0), need = T.add_up(sum1);
  list_free(P, mine, free.x, min(free.y, need.y), lane);
  T.sync();
  int at = need.x;
  for (int b0 = seqs.x; b0 < seqs.y; b0 += 32) {
    const int b = b0 + lane;
    len = more = want = 0;
    ok = false;
    if (b < seqs.y) want = pages_wanted(P, b, len, more, ok);
    const int end = at + lane_scan(want, lane);  // pages wanted up to this sequence
    // in order until the pages run out: behind the first that cannot have its pages none is given any
    const bool served = ok && (want == 0 || end <= free.y);
    if (b < seqs.y) {
      if (!ok) raise(P, kBadArgument);
      if (ok && !served) raise(P, kOutOfPages);
      if (inside(P, b, P.t.sequences)) P.first[b] = served ? len : -1;
      if (served && inside(P, b, P.t.sequences)) P.t.lens[b] = len + more;
    }
    const int slot = (int)(((long long)len + P.t.page_size - 1) / P.t.page_size), n = served ? want : 0;
    const int here = min(32, seqs.y - b0);
    for (int i = 0; i < here; ++i) {
      const int ni = __shfl_sync(0xffffffffu, n, i), from = __shfl_sync(0xffffffffu, end - want, i), si = __shfl_sync(0xffffffffu, slot, i);
      int32_t* row = P.t.table + (long long)(b0 + i) * P.t.max_pages + si;
      over_row(ni, lane, [&](int j) { return __ldcg(P.list + from + j); }, [&](int j, int p) {
        if (inside(P, row - P.t.table + j, slots(P))) row[j] = p;
        if (inside(P, p, P.t.pages)) P.t.refs[p] = 1;
      });
    }
    at = __shfl_sync(0xffffffffu, end, 31);
  }
}

// ---- sequence i becomes a copy of what sequence parent[i] was.  Lanes look at 32 sequences at once; their rows
// are the whole warp's.
template <bool kOne>
__global__ void __launch_bounds__(kThreads, 1) pages_fork_kernel(const __grid_constant__ PagesParams P) {
  __shared__ int32_t sums[2][kOne ? kThreads / 32 : 1], few[2][kOne ? kFewSequences : 1];
  griddep_wait();
  griddep_launch_dependents();
  using Tm = Team<kOne>;
  const Tm T(P.ctas);
  const int lane = T.lane, S = P.t.sequences, width = P.t.max_pages, page_size = P.t.page_size;
  const int2 mine = T.range(P.t.pages), seqs = T.range(S);
  int32_t *const sum0 = kOne ? sums[0] : P.sum0, *const sum1 = kOne ? sums[1] : P.sum1;
  int32_t *const heirs = kOne ? few[0] : P.heirs, *const keep = kOne ? few[1] : P.keep;
  auto parent_of = [&](int i) {
    const int p = i < seqs.y ? __ldcg(P.in + i) : -1;
    return p < S ? p : -1;
  };
  for (int b = seqs.x + lane; b < seqs.y; b += 32) Tm::store(heirs + b, 0), Tm::store(keep + b, 0x7fffffff);
  T.sync();
  // who keeps a page that is not full: the sequence itself, else its lowest heir
  for (int i = seqs.x + lane; i < seqs.y; i += 32) {
    const int p = __ldcg(P.in + i);
    if (p >= S) raise(P, kBadArgument);
    if (p < 0 || p >= S) continue;
    atomicAdd(heirs + p, 1);
    atomicMin(keep + p, p == i ? -1 : i);
  }
  T.sync();
  // sequences without an heir give their pages back; every heir but the sequence itself takes down its
  // parent's pages, whose row may be written later
  int copies = 0;
  for (int i0 = seqs.x; i0 < seqs.y; i0 += 32) {
    const int i = i0 + lane, p = parent_of(i);
    const bool there = i < seqs.y;
    const int old = there ? entries_of(P, i, true) : 0, len = p >= 0 ? entries_of(P, p, false) : 0;
    const bool ends = there && Tm::load(heirs + i) == 0;
    if (p >= 0 && p != i && Tm::load(keep + p) != i && len % page_size != 0) ++copies;
    if (there && inside(P, i, S)) P.len[i] = len;
    const int here = min(32, seqs.y - i0);
    for (int x = 0; x < here; ++x) {
      const int px = __shfl_sync(0xffffffffu, p, x);
      const int used = __shfl_sync(0xffffffffu, ends ? pages_for(old, page_size) : 0, x);
      const int taken = __shfl_sync(0xffffffffu, p >= 0 && p != i ? pages_for(len, page_size) : 0, x);
      const int32_t* row = P.t.table + (long long)(i0 + x) * width;
      over_row(used, lane, [&](int j) { return row[j]; }, [&](int, int page) {
        if (in_pool(P, page))
          atomicAdd(P.t.refs + page, -1);
        else
          raise(P, kBadPage);
      });
      over_row(taken, lane, [&](int j) { return P.t.table[(long long)px * width + j]; }, [&](int j, int page) {
        const long long to = (long long)(i0 + x) * width + j;
        if (inside(P, to, slots(P))) P.rows[to] = page;
      });
    }
  }
  T.leave(sum1, copies);
  T.sync();
  T.leave(sum0, count_pages(P, mine, lane, false));
  T.sync();
  const int2 free = T.add_up(sum0), need = T.add_up(sum1);
  list_free(P, mine, free.x, min(free.y, need.y), lane);
  if (T.w == 0 && lane == 0) *P.count = min(free.y, need.y);
  T.sync();
  int at = need.x;
  for (int i0 = seqs.x; i0 < seqs.y; i0 += 32) {
    // (lens of parents may be written by now: their copies are read; what `keep` says stays)
    const int i = i0 + lane, p = parent_of(i);
    const bool change = i < seqs.y && p != i;  // (else nothing of its own changes: other heirs add their uses)
    const int had = change ? pages_for(entries_of(P, i, false), page_size) : 0;
    int len = change && p >= 0 ? P.len[i] : 0;
    const bool keeps = change && p >= 0 && Tm::load(keep + p) == i, copy = change && p >= 0 && !keeps && len % page_size != 0;
    const int full = len / page_size;
    const uint32_t who = __ballot_sync(0xffffffffu, copy);
    const int mine_at = at + __popc(who & ((1u << lane) - 1));
    at += __popc(who);
    int fresh = -1;
    if (copy) {
      if (mine_at < free.y) {
        fresh = __ldcg(P.list + mine_at);
        const int from = P.rows[(long long)i * width + full];
        if (!in_pool(P, from)) raise(P, kBadPage);  // (the copy leaves it out)
        if (inside(P, mine_at, P.moves)) P.src[mine_at] = from, P.dst[mine_at] = fresh;
        if (inside(P, fresh, P.t.pages)) P.t.refs[fresh] = 1;
      } else {  // no page left for the copy: it ends up empty
        raise(P, kOutOfPages);
        len = 0;
      }
    }
    if (change && inside(P, i, S)) P.t.lens[i] = len;
    const int used = pages_for(len, page_size);
    uint32_t todo = __ballot_sync(0xffffffffu, change && (used > 0 || had > 0));
    while (todo) {
      const int x = __ffs(todo) - 1;
      todo &= todo - 1;
      const int n = __shfl_sync(0xffffffffu, used, x), clear = __shfl_sync(0xffffffffu, had, x), last = __shfl_sync(0xffffffffu, full, x),
                page_x = __shfl_sync(0xffffffffu, fresh, x);
      const bool counted = !__shfl_sync(0xffffffffu, (int)keeps, x);
      int32_t* row = P.t.table + (long long)(i0 + x) * width;
      const int32_t* from = P.rows + (long long)(i0 + x) * width;
      over_row(n, lane, [&](int j) { return j == last && page_x >= 0 ? page_x : from[j]; }, [&](int j, int page) {
        if (!in_pool(P, page))
          raise(P, kBadPage);
        else if (counted && j < last)
          atomicAdd(P.t.refs + page, 1);
        if (inside(P, row - P.t.table + j, slots(P))) row[j] = page;
      });
      for (int j = n + lane; j < clear; j += 32)
        if (inside(P, row - P.t.table + j, slots(P))) row[j] = -1;
    }
  }
}

// ---- the pages in use become the first ones: the i-th in use behind their number goes to the i-th
// free one before it
template <bool kOne>
__global__ void __launch_bounds__(kThreads, 1) pages_compact_kernel(const __grid_constant__ PagesParams P) {
  __shared__ int32_t sums[2][kOne ? kThreads / 32 : 1];
  griddep_wait();
  griddep_launch_dependents();
  const Team<kOne> T(P.ctas);
  int32_t *const sum0 = kOne ? sums[0] : P.sum0, *const sum1 = kOne ? sums[1] : P.sum1;
  const int lane = T.lane, width = P.t.max_pages;
  const int2 mine = T.range(P.t.pages), seqs = T.range(P.t.sequences);
  T.leave(sum0, count_pages(P, mine, lane, true));
  T.sync();
  const int2 live = T.add_up(sum0);
  T.leave(sum1, count_pages(P, make_int2(mine.x, min(mine.y, live.y)), lane, false));
  T.sync();
  const int2 holes = T.add_up(sum1);  // as many as pages in use behind the border
  int hole = holes.x, mover = live.x - (live.y - holes.y);  // (pages in use before this range, less those that stay)
  for (int p0 = mine.x; p0 < mine.y; p0 += 32 * kPoolAhead) {
    bool uses[kPoolAhead];
#pragma unroll
    for (int k = 0; k < kPoolAhead; ++k) uses[k] = p0 + 32 * k + lane < mine.y && __ldcg(P.t.refs + p0 + 32 * k + lane) != 0;
#pragma unroll
    for (int k = 0; k < kPoolAhead && p0 + 32 * k < mine.y; ++k) {
      const int p = p0 + 32 * k + lane;
      const bool there = p < mine.y, used = uses[k], before = p < live.y;
      const uint32_t f = __ballot_sync(0xffffffffu, there && before && !used), u = __ballot_sync(0xffffffffu, used),
                     low = (1u << lane) - 1;
      if (there && before && !used && inside(P, hole + __popc(f & low), P.moves)) P.dst[hole + __popc(f & low)] = p;
      if (used && !before) {
        const int i = mover + __popc(u & low);
        if (inside(P, i, P.moves)) P.src[i] = p;
        if (inside(P, p, P.t.pages)) __stcg(P.list + p, i);
      }
      hole += __popc(f);
      mover += __popc(u);
    }
  }
  if (T.w == 0 && lane == 0) *P.count = holes.y;
  T.sync();
  const int2 moves = T.range(holes.y);
  for (int i = moves.x + lane; i < moves.y; i += 32) {
    const int a = __ldcg(P.src + i), b = __ldcg(P.dst + i);
    if (!inside(P, max(a, b), P.t.pages)) continue;
    P.t.refs[b] = P.t.refs[a];
    P.t.refs[a] = 0;
  }
  for (int s0 = seqs.x; s0 < seqs.y; s0 += 32) {
    const int all = s0 + lane < seqs.y ? pages_for(entries_of(P, s0 + lane, true), P.t.page_size) : 0;
    const int here = min(32, seqs.y - s0);
    for (int x = 0; x < here; ++x) {
      const int used = __shfl_sync(0xffffffffu, all, x);
      int32_t* row = P.t.table + (long long)(s0 + x) * width;
      // what a page that moves becomes; -1: it stays, -2: it is none
      auto where = [&](int j) {
        const int p = row[j], q = in_pool(P, p) ? p : 0;
        const int i = __ldcg(P.list + q);  // (of a page that no use is counted for: anything)
        const bool moves = i >= 0 && i < holes.y;
        const int a = __ldcg(P.src + (moves ? i : 0)), b = __ldcg(P.dst + (moves ? i : 0));  // (without branches)
        return q != p ? -2 : p < live.y ? -1 : moves && a == p ? b : -2;
      };
      over_row(used, lane, where, [&](int j, int p) {
        if (p == -2) raise(P, kBadPage);
        if (p >= 0 && inside(P, row - P.t.table + j, slots(P))) row[j] = p;
      });
    }
  }
}

// ---- copying of pages.  A page of each array is one range of bytes; warps take pieces of 2 KB of all the moves' pages in
// turn, so that few large pages and many small ones fill the GPU alike (pieces of 16 KB a CTA: pages of 16 fp4 entries of 512
// features 2.5 TB/s, now 6.2).
constexpr int kCopyThreads = 256, kCopyAhead = 4;
struct CopyParams {
  uint8_t* base[3];
  long long bytes[3];  // of a page; 0: no such array
  int unit[3];         // bytes moved at a time
  int pieces[3];
  const int32_t *src, *dst, *count;
  int n, per;          // most moves, pieces of a move
  long long pages;
  int* status;
#ifdef CSA_DEBUG_BOUNDS
  int less;
#endif
};
constexpr long long kPiece = 16 * 32 * kCopyAhead;  // bytes at most of a warp's turn

template <class U>
__device__ __forceinline__ void copy_piece(uint8_t* dst, const uint8_t* src, long long bytes) {
  const int n = (int)(bytes / (long long)sizeof(U));
  for (int i = threadIdx.x & 31; i < n; i += 32 * kCopyAhead) {
    U v[kCopyAhead];
#pragma unroll
    for (int j = 0; j < kCopyAhead; ++j)
      if (i + j * 32 < n) v[j] = reinterpret_cast<const U*>(src)[i + j * 32];
#pragma unroll
    for (int j = 0; j < kCopyAhead; ++j)
      if (i + j * 32 < n) reinterpret_cast<U*>(dst)[i + j * 32] = v[j];
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const int n = P.count ? min(max(*P.count, 0), P.n) : P.n;
  const int lane = threadIdx.x & 31, first = (blockIdx.x * kCopyThreads + threadIdx.x) / 32, warps = gridDim.x * (kCopyThreads / 32);
  const int moves = warps / P.per, pieces = warps - moves * P.per;  // from a warp's turn to its next
  int of = first % P.per;
  for (long long m = first / P.per; m < n; m += moves, of += pieces, m += of >= P.per, of -= of >= P.per ? P.per : 0) {
    int piece = of, a = 0;
    const long long from = P.src[m], to = P.dst[m];
    if (from < 0 || from >= P.pages || to < 0 || to >= P.pages) {
      if (P.status && lane == 0 && piece == 0) atomicOr(P.status, 4);
      continue;
    }
    if (from == to) continue;
    while (piece >= P.pieces[a]) piece -= P.pieces[a++];
#ifdef CSA_DEBUG_BOUNDS
    if (to >= P.pages - P.less) {
      if (P.status && lane == 0) atomicOr(P.status, 8);
      continue;
    }
#endif
    const long long at = piece * kPiece, bytes = min(kPiece, P.bytes[a] - at);
    uint8_t* d = P.base[a] + to * P.bytes[a] + at;
    const uint8_t* s = P.base[a] + from * P.bytes[a] + at;
    if (P.unit[a] == 16)
      copy_piece<uint4>(d, s, bytes);
    else if (P.unit[a] == 4)
      copy_piece<uint32_t>(d, s, bytes);
    else
      copy_piece<uint8_t>(d, s, bytes);
  }
}

cudaError_t launch_pages(void (*one)(PagesParams), void (*cluster)(PagesParams), int ctas, PagesParams P, cudaStream_t s) {
  int32_t* w = P.t.workspace;
  P.sum0 = w, P.sum1 = w + kMostWarps;
  P.heirs = w + 2 * kMostWarps, P.keep = P.heirs + P.t.sequences, P.len = P.keep + P.t.sequences;
  P.list = P.len + P.t.sequences;
  P.rows = P.list + P.t.pages;
  P.ctas = ctas;
#ifdef CSA_DEBUG_BOUNDS
  P.less = getenv("CSA_TEST_SHORT_EXTENTS") ? 1 : 0;
#endif
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, ctas > 1 ? cluster : one, P);
}

// CTAs of a step: one while its warps have few pages and few sequences' rows each, more as those grow (see above).
int ctas_for(const csa_pages& t, int few_pages, int few_sequences) {
  if (t.pages <= few_pages && t.sequences <= few_sequences) return 1;
  return t.pages <= 65536 ? 4 : kMostCtas;
}

}  // namespace

long long pages_workspace_ints(long long pages, long long sequences, long long max_pages) {
  return 2 * kMostWarps + 3 * sequences + pages + sequences * max_pages;
}

cudaError_t launch_pages_extend(const csa_pages& t, const int32_t* more, int32_t* first, cudaStream_t s) {
  PagesParams P{};
  P.t = t;
  P.in = more;
  P.first = first;
  return launch_pages(pages_extend_kernel<true>, pages_extend_kernel<false>, ctas_for(t, 16384, 1024), P, s);
}
cudaError_t launch_pages_fork(const csa_pages& t, const int32_t* parent, int32_t* src, int32_t* dst, int32_t* count, cudaStream_t s) {
  PagesParams P{};
  P.t = t;
  P.in = parent;
  P.src = src, P.dst = dst, P.count = count;
  P.moves = t.sequences;
  return launch_pages(pages_fork_kernel<true>, pages_fork_kernel<false>, ctas_for(t, 8192, 64), P, s);
}
cudaError_t launch_pages_compact(const csa_pages& t, int32_t* src, int32_t* dst, int32_t* count, cudaStream_t s) {
  PagesParams P{};
  P.t = t;
  P.src = src, P.dst = dst, P.count = count;
  P.moves = t.pages > 1 ? t.pages / 2 : 1;
  return launch_pages(pages_compact_kernel<true>, pages_compact_kernel<false>, ctas_for(t, 4096, 64), P, s);
}

cudaError_t launch_copy_pages(const csa_cache& c, const int32_t* src, const int32_t* dst, int n, const int32_t* count, int* status,
                              cudaStream_t s) {
  CopyParams P{};
  P.base[0] = reinterpret_cast<uint8_t*>(c.latent), P.base[1] = c.codes, P.base[2] = c.scales;
  const long long row[3] = {2LL * c.head_dim, c.head_dim / 2, c.head_dim / (c.fp4 == 2 ? 32 : 16)};
  for (int i = 0; i < 3; ++i) {
    P.bytes[i] = P.base[i] ? row[i] * c.page_size : 0;
    const uintptr_t u = (uintptr_t)P.base[i] | (uintptr_t)P.bytes[i];
    P.unit[i] = u % 16 == 0 ? 16 : u % 4 == 0 ? 4 : 1;
    P.pieces[i] = (int)((P.bytes[i] + kPiece - 1) / kPiece);
    P.per += P.pieces[i];
  }
  P.src = src, P.dst = dst, P.count = count;
  P.n = n;
  P.pages = c.pages;
  P.status = status;
#ifdef CSA_DEBUG_BOUNDS
  P.less = getenv("CSA_TEST_SHORT_EXTENTS") ? 1 : 0;
#endif
  const long long items = ((long long)n * P.per + kCopyThreads / 32 - 1) / (kCopyThreads / 32), most = 8LL * current_sm_count();
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < most ? items : most));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, copy_pages_kernel, P);
}

}  // namespace csa
