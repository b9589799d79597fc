// Attention over one shared key/value row per position (see include/csa.h): a prompt's tokens over
// their own rows with a window and sinks, or one new token a sequence over a paged cache.
//
// A sequence's queries are its N tokens' heads in order, [N * H][D]; an item is 64 of them (one
// token's at H = 64, four tokens' at H = 16, half a token's at H = 128), over the rows that any of
// its tokens sees: the sinks, then the window.  Those rows are taken 64 at a time:
//
//   S^T = C Q^T   [64 rows x 64 queries], features as the K dimension
//   P   = exp2(S^T * scale - m)           m: a reference for each query
//   O^T = O^T + C^T P                     [D features x 64 queries], rows as the K dimension
//
// Transposed, both products take the rows' tile as their A operand, once K-major (64 x D) and once
// M-major (D x 64): one copy in shared memory is key and value, which is what a shared row offers,
// and O^T takes D / 128 * 64 columns of tensor memory (256 of 512 at D = 512) where queries as rows
// would take all of it.  The scores come back with a row per TMEM lane in the matrix-fragment shape.
// The reference need not be the maximum: bf16 weights and f32 sums keep their relative precision as
// long as it is near.  It begins as the first row's score, and is only renewed (as the maximum so
// far, with O^T and l scaled) when a score passes it by 2^16; taking the maximum over rows costs
// shuffles and an exchange between the warps that most tiles need not pay.
//
// What bounds it (probes on GB300, cycles): a 64 x 64 x 16 MMA takes 32 and a 128 x 64 x 16 one 48
// (shared-memory reads of both operands at 128 bytes a cycle), so a tile of 64 rows at D = 512 costs
// 1024 + 768; its 64 KB arrive from HBM in 2510 (26 bytes a cycle and SM, 7.2 TB/s).  Decode over
// latents is therefore bound by HBM, over codes (18 KB a tile) by the MMAs' operand reads.  Rows
// come by 16-byte cp.async, which takes any page size and leaves hidden rows out (zeros) at the rate
// of tiled TMA boxes (760 cycles a tile from L2, against 8010 for four-row TMA gathers).
//
// Work is cut by tiles: the call's tiles, in item order, are divided evenly over the CTAs, so ragged
// lengths and few long sequences fill the GPU alike; an item cut by a CTA boundary leaves partial
// (m, l, O) pieces in the workspace, which a second kernel joins.  Where no item is longer than
// kJoinTiles tiles the boundaries are moved to item starts instead: the imbalance costs less than
// pieces and their join.
#include <atomic>
#include <cstdlib>

#include "layer_ops.h"
#include "tc_common.cuh"

namespace csa {
namespace {

using namespace tcx;

constexpr int kTile = 64;                      // rows of a tile
constexpr int kCols = 64;                      // queries of an item
constexpr int kChunkBytes = 8192;              // 64 rows x 64 features bf16: one column of swizzled atoms
constexpr int kPBytes = kTile * kCols * 2;     // one weights buffer
constexpr int kStageOut = 2048;                // a warp's staging of 32 queries x 32 features bf16
constexpr int kJoinTiles = 6;   // items longer than this are split
constexpr int kMinTiles = 4;    // a split call gives a CTA at least this many tiles
constexpr float kStep = 16.0f;  // base-2 steps a score may pass the reference by
constexpr float kFloor = -1e38f;  // a reference that any score passes
constexpr int kSpins = 1 << 16;   // polls of two barriers before the MMA warp waits for one of them
constexpr int kAuxBytes = 3584;   // barriers, flags, per-warp maxima and sums

struct AttnParams {
  AttnCall c;
  int H, D, window, sinks;
  int per, items;    // items of a sequence, of the call
  float scale_log2;  // scale * log2(e): scores in base-2 exponents
  int* flag;
  float4* part;      // pieces: [2 * grid][64 * D / 4] f32, in the order of the fragment loads
  float2* part_ml;   // (maximum, sum) of each piece and query [2 * grid][64]
  int2* record;      // per CTA: (item, pieces) of an item whose first piece it made, or (-1, 0)
  int stages;
  bool split;        // items may be cut (the join kernel follows); else they are drawn from `ticket`
  int* ticket;       // items drawn beyond each CTA's first; 0 between calls
#ifdef CSA_DEBUG_BOUNDS
  uint64_t wait_ns;  // the time-out test shortens the waits
  int test_stall;    // and leaves out each CTA's last tile
#endif
};

// ---- the rows an item sees
struct Seen {
  int b;                // sequence
  int f0, cols;         // first query, queries with an output (0: padding)
  int tlo, thi;         // positions of its first and last token (thi -1: a sequence without entries)
  int cnt;              // rows: row v is position v, or v + jump from the sinks on
  int jump;
};

__device__ __forceinline__ Seen seen_rows(const AttnParams& P, int item) {
  Seen s;
  s.b = item / P.per;
  s.f0 = (item - s.b * P.per) * kCols;
  if (P.c.paged) {
    const int top = P.c.max_pages * P.c.cache.page_size, n = __ldg(P.c.lens + s.b);
    s.cols = min(kCols, P.H - s.f0);
    s.tlo = s.thi = min(max(n, 0), top) - 1;
  } else {
    const int n = P.c.lens ? min(max(__ldg(P.c.lens + s.b), 0), P.c.N) : P.c.N;
    s.cols = max(0, min(kCols, n * P.H - s.f0));
    s.tlo = P.c.start + s.f0 / P.H;
    s.thi = P.c.start + (s.f0 + max(s.cols, 1) - 1) / P.H;
  }
  // every token from tlo on sees the rows after thi - most and the sinks at most
  const long long most = (long long)P.window + (s.thi - s.tlo) + P.sinks;
  const bool all = P.window == 0 || s.thi + 1 <= most;
  s.cnt = all ? s.thi + 1 : (int)most;
  s.jump = all ? 0 : s.thi + 1 - (int)most;
  return s;
}
__device__ __forceinline__ int tiles_of(const Seen& s) {
  return s.cols == 0 ? 0 : max(1, (s.cnt + kTile - 1) / kTile);  // a sequence without entries still has its output
}

// A run of tiles of one item, as the scheduling warp hands it to the others through a ring of slots.
struct __align__(16) Segment {
  Seen s;
  int item, t0, t1, tiles;  // tiles [t0, t1) of the item's; t1 0: no more segments
  int pad;
  long long index;          // tile t0's number among the call's tiles (split calls)
};
static_assert(sizeof(Segment) == 64, "a ring slot");
constexpr int kRing = 4;

// ---- tensor-core helpers
// Descriptors of 128-byte-swizzled tiles of 128-byte rows.  K-major: 8-row groups 1024 bytes apart.
// MN-major: groups of 8 K-rows 1024 bytes apart, 64-element columns `atom` bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t atom) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((atom >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
constexpr uint32_t kTransposed = (1u << 15) | (1u << 16);  // A and B MN-major

// 16 TMEM lanes x 64 columns in the matrix-fragment shape: r[4i + 2h + e] is lane l / 4 + 8h, column
// 8i + 2 (l % 4) + e.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x8.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// The same over 32 columns, not waiting.
__device__ __forceinline__ void tmem_ld_half(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
template <bool kTrans>
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  if constexpr (kTrans)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
  else
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// One poll of the phase of `parity`, not suspending while it is incomplete.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait for a barrier's phase.  The poll is inlined, what follows an incomplete one is not: the
// kernel's instructions have to stay in the SM's instruction caches (with every wait inlined, and the
// items' ranges worked out by every role, the kernel was 144 KB and ran at half its speed).
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t wait_ns) {
  return mbar_wait(bar, parity, abort_flag, wait_ns);
}
// A barrier of four warps (1: softmax, 2: epilogue); group_or gives every thread whether any passed
// true.
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool group_or(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return r != 0;
}
// One lane of a converged warp, the same at every call: what it alone issues stays in uniform
// registers (an MMA issued under `lane == 0` cost 70 to 126 cycles in descriptor moves, 32 this way).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Eight e2m1 codes (element 0 in the low nibble) times a scale (bf16x2) to eight bf16.  The bytes of
// a magnitude's bf16 pattern (0, .5, 1, 1.5, 2, 3, 4, 6) are looked up by byte permutation; products
// of 2 and 4 significant bits are exact in bf16.
__device__ __forceinline__ uint4 dequant8(uint32_t w, uint32_t scale2) {
  const uint32_t m0 = w & 0x77777777u, m1 = m0 >> 16;
  const uint32_t h0 = __byte_perm(0x3F3F3F00u, 0x40404040u, m0), h1 = __byte_perm(0x3F3F3F00u, 0x40404040u, m1);
  const uint32_t l0 = __byte_perm(0xC0800000u, 0xC0804000u, m0), l1 = __byte_perm(0xC0800000u, 0xC0804000u, m1);
  uint32_t v[4] = {__byte_perm(l0, h0, 0x5140), __byte_perm(l0, h0, 0x7362), __byte_perm(l1, h1, 0x5140),
                   __byte_perm(l1, h1, 0x7362)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the signs are bits 3 and 7 of byte i: to bits 15 and 31
    const uint32_t s = ((w >> (8 * i)) & 0x88u) * 0x01001000u;
    v[i] |= s & 0x80008000u;
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(scale2));
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// ---- the kernel's warps: 0-3 softmax (TMEM lane quarter = warp); with one CTA an SM 4-7 the
// epilogue, which reads O^T while the softmax warps go on with the next item (up to D = 192 two CTAs
// share an SM instead, whose softmax warps read their own O^T); then one that issues the MMAs, one
// for the queries' copies, and the rows' warps in two groups that take alternate tiles (one group's
// tile can be in flight while the other waits for its stage).
template <bool kFp4, int kCtas>
struct Roles {
  static constexpr bool kEpi = kCtas == 1;
  static constexpr int kMma = kEpi ? 8 : 4, kQ = kMma + 1, kRows = kMma + 2;
  static constexpr int kRowWarps = kCtas == 2 ? 2 : 4;
  static constexpr int kGroupWarps = kRowWarps / 2;
  static constexpr int kTileRows = kTile / kGroupWarps;  // rows of a tile a warp brings
  static constexpr int kThreads = 32 * (kRows + kRowWarps);
};

template <bool kFp4, int kCtas>
__global__ void __launch_bounds__(Roles<kFp4, kCtas>::kThreads, kCtas)
    attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ AttnParams P) {
  using R = Roles<kFp4, kCtas>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int D = P.D, chunks = D / 64;
  const uint32_t nst = P.stages;
  const int stage_bytes = chunks * kChunkBytes;
  uint8_t* sQ = smem;
  uint8_t* sC = sQ + chunks * kChunkBytes;
  uint8_t* sP = sC + nst * stage_bytes;  // two weights buffers
  uint8_t* sO = sP + 2 * kPBytes;        // the epilogue's staging, 2 KB a warp
  uint8_t* aux = sO + 4 * kStageOut;
  uint64_t* c_full = (uint64_t*)aux;  // [8] a stage's rows have landed
  uint64_t* c_empty = c_full + 8;     // [8] a stage's products are done
  uint64_t* s_full = c_empty + 8;     // [2] scores ready
  uint64_t* p_full = s_full + 2;      // [2] weights written, scores read
  uint64_t* pv_done = p_full + 2;     // [2] second product done: weights buffer free, O^T complete to it
  uint64_t* g_full = pv_done + 2;     // [4] a segment's slot is written
  uint64_t* g_empty = g_full + kRing; // [4] and has been read by every role
  uint64_t* q_full = g_empty + kRing;
  uint64_t* q_empty = q_full + 1;
  uint64_t* o_empty = q_empty + 1;    // O^T has been read
  uint64_t* l_full = o_empty + 1;     // the item's references and sums are in `fin`
  uint64_t* l_empty = l_full + 1;     // and have been read
  uint64_t* mma_done = l_empty + 1;   // clean-up after an abort
  uint32_t* tmem_slot = (uint32_t*)(mma_done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  Segment* ring = (Segment*)(aux + 384);
  long long* work = (long long*)(aux + 640);  // split calls: first item, tile, tiles, tile index, end, total, CTAs
  float* red = (float*)(aux + 704);   // [4][64] per-warp maxima; the scan's sums before
  float* fin = red + 256;             // [4][64] per-warp sums, [64] references
  float* inv = fin + 320;             // [64] 1 / sum
  int* colt = (int*)(inv + 64);       // [64] the queries' positions
  static_assert(704 + (256 + 320 + 64 + 64) * 4 <= kAuxBytes, "aux region");

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
#ifdef CSA_DEBUG_BOUNDS
  const uint64_t kWait = P.wait_ns;
#else
  constexpr uint64_t kWait = kWaitNs;
#endif
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_try_wait(bar, parity & 1) || wait_slow(bar, parity & 1, abort_flag, kWait);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      mbar_init(&c_full[s], R::kGroupWarps);
      mbar_init(&c_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&g_full[i], 1);
      mbar_init(&g_empty[i], R::kThreads / 32 - 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_empty, 4);
    mbar_init(l_full, 4);
    mbar_init(l_empty, 4);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_map(&map_q);
  }
  const uint32_t oc = (uint32_t)((D + 127) / 128) * kCols;  // columns of O^T; two score buffers follow
  const uint32_t tmem_cols = oc + 2 * kCols <= 256 ? 256 : 512;
  if (warp == R::kMma) tmem_alloc(tmem_slot, tmem_cols);
  griddep_launch_dependents();

  if (blockIdx.x == 0 && P.c.lens) {  // lengths out of range are taken as the nearest end
    const int most = P.c.paged ? P.c.max_pages * P.c.cache.page_size : P.c.N;
    for (int b = threadIdx.x; b < P.c.B; b += R::kThreads) {
      const int n = P.c.lens[b];
      if (n < 0 || n > most) atomicOr(P.flag, 1);
    }
  }
  if (P.split) {
    // ---- the CTA's share of the call's tiles: every CTA adds up the items' tiles (threads over
    // contiguous items) and finds its own first one
    const int per = (P.items + R::kThreads - 1) / R::kThreads, lo = min(P.items, per * (int)threadIdx.x),
              hi = min(P.items, lo + per);
    long long sum = 0;
    int top = 0;
#pragma unroll 1
    for (int i = lo; i < hi; ++i) {
      const int n = tiles_of(seen_rows(P, i));
      sum += n;
      top = max(top, n);
    }
    long long pre = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += y;
      top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    long long* ws = (long long*)red;  // [warp] sums, then [warp] maxima
    if (lane == 31) ws[warp] = pre, ws[32 + warp] = top;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < R::kThreads / 32; ++w) {
      if (w < warp) before += ws[w];
      total += ws[w];
      top = max(top, (int)ws[32 + w]);
    }
    pre += before - sum;  // tiles before this thread's items
    const bool cut = top > kJoinTiles;
    const long long ctas = cut ? min((long long)gridDim.x, max(1LL, total / kMinTiles)) : gridDim.x;
    const long long i = blockIdx.x;
    const long long a = i < ctas ? total * i / ctas : total, e = i < ctas ? total * (i + 1) / ctas : total;
    if (threadIdx.x == 0) work[0] = P.items, work[1] = 0, work[3] = work[4] = total, work[5] = total, work[6] = ctas;
    __syncthreads();
    // the boundary x: the item it falls in or, without cutting, the first item that starts from it on
    if ((a >= pre && a < pre + sum) || (e >= pre && e < pre + sum)) {
      long long at = pre;
#pragma unroll 1
      for (int item = lo; item < hi; ++item) {
        const int n = tiles_of(seen_rows(P, item));
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          const long long x = w ? e : a;
          if (x < at || x >= at + n) continue;
          const int tile = (int)(x - at);
          const bool move = !cut && tile > 0;
          if (w == 0) work[0] = item + move, work[1] = move ? 0 : tile;
          work[3 + w] = move ? at + n : x;
        }
        at += n;
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      work[2] = work[4] - work[3];
      P.record[blockIdx.x] = make_int2(-1, 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  // the next segment, for every role but the scheduling warp
  uint32_t seg = 0;  // segments read
  Segment g;
  auto next = [&]() {
    const uint32_t slot = seg % kRing;
    if (!wait(&g_full[slot], seg / kRing)) return false;
    g = ring[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&g_empty[slot]);
    ++seg;
    return g.t1 > 0;
  };

  // ---- an item's end, by the four warps that own O^T's lane quarters (w = warp % 4): the sums over
  // rows in `fin`, O^T (complete with tile kl) scaled to out, or left as a piece.  False after an abort.
  auto finish = [&](int w, int bar, uint32_t kl, int tid) -> bool {
    bool ok = !R::kEpi || wait(l_full, seg - 1);
    ok = ok && wait(&pv_done[kl & 1], kl >> 1);
    if (group_or(bar, !ok)) return false;
    tc_fence_after();
    const bool whole = g.t0 == 0 && g.t1 == g.tiles;
    // a piece: slot 0 of the CTA for its first segment's, 1 for its last's (an item's first piece)
    const int slot = 2 * blockIdx.x + (g.t0 == 0 ? 1 : 0);
    const long long orow = (long long)g.s.b * P.c.N * P.H + g.s.f0, rows = (long long)P.c.B * P.c.N * P.H;
    if (tid < kCols) {
      const float l = (fin[tid] + fin[64 + tid]) + (fin[128 + tid] + fin[192 + tid]), m = fin[256 + tid];
      if (whole) {
        float r, lg;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(l));
        asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(l));
        inv[tid] = l == 0.0f ? 0.0f : r;
        if (P.c.lse && tid < g.s.cols && in_bounds(orow + tid, rows, P.flag))
          P.c.lse[orow + tid] = l == 0.0f ? -INFINITY : (m + lg) * 0.693147180559945f;
      } else {
        P.part_ml[slot * kCols + tid] = make_float2(m, l);
      }
    }
    group_sync(bar);
    if (R::kEpi && lane == 0) mbar_arrive(l_empty);
    const uint32_t base = tmem + ((uint32_t)(32 * w) << 16);
    if (whole) {
      // steps of 32 queries x 16 or 32 features; the next step's loads run ahead of a step's stores
      uint8_t* stage = sO + w * kStageOut;
      const int u = lane & 3;
      uint32_t o[2][16];
      tmem_ld_half(base, o[0]);
      tmem_ld_half(base + (16u << 16), o[1]);
      const int steps = (chunks + 1) & ~1;
#pragma unroll 1
      for (int step = 0; step < steps; ++step) {
        const int x = step & ~1, c = step & 1;
        const bool full = x + 1 < chunks;  // 128 features: 32 a warp; else 64: 16
        float2 f[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) f[q] = *reinterpret_cast<const float2*>(inv + 32 * c + 8 * q + 2 * (lane & 3));
        tmem_ld_wait();
        // to [query][32 features] by transposed stores; 16-byte units swizzled against conflicts
#pragma unroll
        for (int i = 0; i < 4; i += 2)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int q = i + (j >> 1);
              v[j] = bf16x2(__uint_as_float(o[h][4 * q + 2 * (j & 1)]) * f[q].x,
                            __uint_as_float(o[h][4 * q + 2 * (j & 1) + 1]) * f[q].y);
            }
            const int r = 8 * (i + (lane >> 4)) + (lane & 7), uu = 2 * h + ((lane >> 3) & 1);
            stmatrix4<true>(smem_addr(stage) + r * 64 + ((uu ^ ((r >> 1) & 3)) << 4), v[0], v[1], v[2], v[3]);
          }
        if (step + 1 < steps) {
          const uint32_t at = base + 32 * (step + 1);  // 64 columns a block of 128 features
          tmem_ld_half(at, o[0]);
          tmem_ld_half(at + (16u << 16), o[1]);
        }
        __syncwarp();
        uint4 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (lane >> 2) + 8 * i;
          y[i] = *reinterpret_cast<const uint4*>(stage + r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
        }
        __syncwarp();
        uint16_t* dst = P.c.out + (orow + 32 * c + (lane >> 2)) * D + x * 64 + w * (full ? 32 : 16) + 8 * u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int q = 32 * c + (lane >> 2) + 8 * i;
          if ((full || u < 2) && q < g.s.cols && in_bounds(orow + q, rows, P.flag))
            *reinterpret_cast<uint4*>(dst + (size_t)(8 * i) * D) = y[i];
        }
      }
    } else {
      float4* dst = P.part + (size_t)slot * (kCols * D / 4) + w * 256 + lane;
#pragma unroll 1
      for (int x = 0; x < chunks; ++x) {  // half x % 2 of 16 lanes a warp of the block of 128 features
        uint32_t o[32];
        tmem_ld_frag(base + (x >> 1) * kCols + ((uint32_t)(16 * (x & 1)) << 16), o);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dst[(x * 32 + i) * 32] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                               __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
      }
      if (g.t0 == 0 && tid == 0) {
        // the item ends in the CTA whose share holds its last tile
        const long long end = g.index + g.tiles, total = work[5], ctas = work[6];
        long long j = (end * ctas - 1) / total;
        while (total * (j + 1) / ctas < end) ++j;
        while (total * j / ctas >= end) --j;
        P.record[blockIdx.x] = make_int2(g.item, (int)(j - blockIdx.x) + 1);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(o_empty);
    return true;
  };

  if (warp == R::kQ) {
    // ---- scheduling and queries (one lane).  A split call's segments are the CTA's share; otherwise
    // items are drawn one at a time, the CTA's first being its own number: SMs differ in speed and
    // padding in place.  The CTA that draws the last ticket sets the counter back.  A segment is
    // published one ahead of its queries' copy (64 rows of [B * N * H][D] from the item's first; rows past
    // its last are other sequences' or zeros: columns that nothing reads).
    if (lane == 0) {
      const bool split = P.split;
      int item = split ? (int)work[0] : blockIdx.x, tile = split ? (int)work[1] : 0, drawn = 0;
      long long left = split ? work[2] : 0, index = split ? work[3] : 0;
      uint32_t n = 0, loads = 0;
      bool end = false;
      auto draw = [&]() {
        const int t = atomicAdd(P.ticket, 1);
        if (t == P.items - 1) *P.ticket = 0;  // every CTA draws until it is past the last item
        return (int)gridDim.x + t;
      };
      if (!split) drawn = draw();
      int row = 0, bytes = 0;  // queries still to be copied: those of the segment published last
      for (;;) {
        Segment a;
        bool more = false;
        while (!end) {
          end = item >= P.items || (split && left <= 0);
          if (end) break;
          a.s = seen_rows(P, item);
          a.tiles = tiles_of(a.s);
          a.item = item;
          a.t0 = tile;
          a.t1 = split ? (int)min((long long)a.tiles, tile + left) : a.tiles;
          a.index = index;
          more = a.t1 > tile;
          left -= a.t1 - tile;
          index += a.t1 - tile;
          tile = 0;
          if (split) {
            ++item;
          } else {
            item = drawn;
            if (item < P.items) drawn = draw();
          }
          if (more) break;  // else padding
        }
        if (!more) a.t1 = 0;
        if (n >= kRing && !wait(&g_empty[n % kRing], n / kRing - 1)) break;
        ring[n % kRing] = a;
        mbar_arrive(&g_full[n % kRing]);
        const int next_row = more ? a.s.b * P.c.N * P.H + a.s.f0 : 0, next_bytes = more ? a.s.cols * D * 2 : 0;
        if (n == 0)
          row = next_row, bytes = next_bytes;  // the first segment's at once
        else if (more)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(P.c.q + (size_t)next_row * D), "r"(next_bytes)
                       : "memory");
        if (bytes > 0) {
          if (loads > 0 && !wait(q_empty, loads - 1)) break;
          mbar_arrive_expect_tx(q_full, chunks * kChunkBytes);
          for (int c = 0; c < chunks; ++c) tma_load_2d(sQ + c * kChunkBytes, &map_q, c * 64, row, q_full);
          ++loads;
        }
        row = next_row, bytes = n > 0 ? next_bytes : 0;
        ++n;
        if (!more) break;
      }
      // after an abort: the tickets up to the end are drawn all the same, the copies in flight land
      if (!split)
        while (*abort_flag && item < P.items) item = drawn, drawn = item < P.items ? draw() : item;
      if (*abort_flag && loads > 0) mbar_wait_bounded(q_full, (loads - 1) & 1);
    }
  } else if (R::kEpi && warp >= 4 && warp < 8) {
    uint32_t k = 0;
    while (next()) {
      k += g.t1 - g.t0;
      if (!finish(warp & 3, 2, k - 1, (int)threadIdx.x - 128)) break;
    }
  } else if (warp >= R::kRows) {
    // ---- rows: warp w of a group brings rows kTileRows * w .. of its group's tiles
    const int grp = (warp - R::kRows) / R::kGroupWarps, w = (warp - R::kRows) % R::kGroupWarps;
    const uint8_t* base = (const uint8_t*)(P.c.paged ? P.c.cache.latent : P.c.kv);
    // eight rows at a time, four lanes a row, such that the eight lanes of a quarter warp hit every bank
    // of the swizzled rows once: rows r and r + 4 side by side for 16-byte units, eight rows for units
    // that expand to 64 bytes
    const int r8 = kFp4 ? lane & 7 : (lane >> 3) + 4 * ((lane >> 2) & 1), u0 = kFp4 ? lane >> 3 : lane & 3;
    uint32_t k = 0;
    int pending = -1;  // a stage whose copies were issued and not yet handed over
    bool ok = true;
    // visible row v: the entry's row in the cache, or -1 past the last one (and for a page outside the
    // cache)
    auto entry = [&](int v) -> int {
      if (v >= g.s.cnt) return -1;
      const int j = v < P.sinks ? v : v + g.s.jump;
      if (!P.c.paged) return g.s.b * P.c.kv_rows + j;
      const int ps = P.c.cache.page_size, pg = (int)((uint32_t)j / (uint32_t)ps);
      const int page = __ldg(P.c.page_table + (long long)g.s.b * P.c.max_pages + pg);
      if (page >= 0 && page < P.c.cache.pages) return page * ps + (j - pg * ps);
      atomicOr(P.flag, 2);
      return -1;
    };
    auto hand_over = [&](int st) {  // this warp's rows have landed
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c_full[st]);
    };
    auto stage_free = [&](uint32_t st) {  // the whole warp's answer
      const bool yes = k < nst || wait(&c_empty[st], k / nst - 1);
      return __all_sync(0xffffffffu, yes) != 0;
    };
    while (ok && next()) {
#pragma unroll 1
      for (int t = g.t0; t < g.t1; ++t, ++k) {
        if ((int)(k & 1) != grp) continue;
        const uint32_t st = k % nst;
#ifdef CSA_DEBUG_BOUNDS
        if (P.test_stall && k == 0) break;  // test of the time-out path: a first tile never comes
#endif
        const uint32_t dst = smem_addr(sC) + st * stage_bytes;
        const int v0 = t * kTile + R::kTileRows * w + r8;
        constexpr int kGroups = R::kTileRows / 8;
        if constexpr (kFp4) {
          // codes, expanded into the bf16 operand: a lane takes 32 codes and two scales (half a chunk) of
          // its row at a time; the next eight rows' are on their way while eight are expanded
          const int upr = D / 32;
          uint4 code[4];
          uint32_t sc[4];
          auto load = [&](int i) {
            const int row = entry(v0 + 8 * i);
            const uint4* cp = reinterpret_cast<const uint4*>(P.c.cache.codes + (size_t)max(row, 0) * (D / 2)) + u0;
            const uint16_t* sp = reinterpret_cast<const uint16_t*>(P.c.cache.scales + (size_t)max(row, 0) * (D / 16)) + u0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool live = row >= 0 && u0 + 4 * j < upr;
              code[j] = live ? __ldg(cp + 4 * j) : make_uint4(0, 0, 0, 0);
              sc[j] = live ? __ldg(sp + 4 * j) : 0;
            }
          };
          load(0);
          if (!(ok = stage_free(st))) break;
#pragma unroll 1
          for (int i = 0; i < kGroups; ++i) {
            uint4 cur[4];
            uint32_t cs[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) cur[j] = code[j], cs[j] = sc[j];
            if (i + 1 < kGroups) load(i + 1);
            const uint32_t r = R::kTileRows * w + 8 * i + r8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t u = u0 + 4 * j;
              if (4 * j >= upr) break;
              if ((int)u >= upr) continue;
              const uint32_t at = dst + (u >> 1) * kChunkBytes + r * 128;
              const uint32_t word[4] = {cur[j].x, cur[j].y, cur[j].z, cur[j].w};
              const float s0 = e4m3_value(cs[j] & 255u), s1 = e4m3_value(cs[j] >> 8);
              const uint32_t s2[2] = {bf16x2(s0, s0), bf16x2(s1, s1)};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint4 d = dequant8(word[q], s2[q >> 1]);
                const uint32_t c = ((u & 1) * 4 + q) ^ (r & 7);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + c * 16), "r"(d.x), "r"(d.y), "r"(d.z),
                             "r"(d.w)
                             : "memory");
              }
            }
          }
          hand_over(st);
        } else {
          int row[kGroups];
#pragma unroll
          for (int i = 0; i < kGroups; ++i) row[i] = entry(v0 + 8 * i);
          if (pending >= 0 && k >= nst && !mbar_test(&c_empty[st], (k / nst - 1) & 1)) {
            cp_wait<0>();
            hand_over(pending);
            pending = -1;
          }
          if (!(ok = stage_free(st))) break;
#pragma unroll
          for (int i = 0; i < kGroups; ++i) {
            const uint32_t r = R::kTileRows * w + 8 * i + r8, bytes = row[i] < 0 ? 0u : 16u;
            const uint8_t* src = base + (size_t)max(row[i], 0) * (2 * D) + u0 * 16;
            const uint32_t lo = dst + r * 128 + ((u0 ^ (r & 7)) << 4), hi = lo ^ 64;
#pragma unroll 2
            for (int c = 0; c < chunks; ++c) {
              cp_async16(lo + c * kChunkBytes, src + c * 128, bytes);
              cp_async16(hi + c * kChunkBytes, src + c * 128 + 64, bytes);
            }
          }
          cp_commit();
          if (nst == 2) {
            cp_wait<0>();
            hand_over(st);
          } else {
            if (pending >= 0) {
              cp_wait<1>();
              hand_over(pending);
            }
            pending = st;
          }
        }
      }
    }
    if constexpr (!kFp4) {
      cp_wait<0>();
      if (pending >= 0) hand_over(pending);
    }
  } else if (warp == R::kMma) {
    // ---- MMAs: the whole warp runs the loop, one elected lane issues
    const bool leader = elect_one();
    const uint32_t idesc_s = idesc_bf16(64, kCols), idesc_o = idesc_bf16(128, kCols) | kTransposed,
                   idesc_o64 = idesc_bf16(64, kCols) | kTransposed;
    const uint32_t c0 = smem_addr(sC), p0 = smem_addr(sP);
    const uint64_t qd = sw128_desc(smem_addr(sQ), 16);
    uint32_t k = 0;  // tiles of earlier segments
    bool ok = true;
    while (ok && next()) {
      ok = __all_sync(0xffffffffu, wait(q_full, seg - 1));
      const uint32_t n = g.t1 - g.t0;
      uint32_t ns = 0, nv = 0;  // tiles whose scores, whose values have been issued
      while (ok && nv < n) {
        // a tile's scores go ahead of the values of the one before it, unless its rows are still on
        // their way when that one's weights are ready
        bool score = ns < n && ns <= nv + 1;
        if (score && ns > nv) {
          const uint32_t st = (k + ns) % nst;
          for (int spin = 0; score && !mbar_test(&c_full[st], ((k + ns) / nst) & 1); ++spin)
            score = spin < kSpins && !mbar_test(&p_full[(k + nv) & 1], ((k + nv) >> 1) & 1);
          score = __all_sync(0xffffffffu, score);
        }
        const uint32_t kk = __shfl_sync(0xffffffffu, k + (score ? ns : nv), 0), st = kk % nst, buf = kk & 1;
        if (score) {
          ok = wait(&c_full[st], kk / nst);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          const uint32_t d = tmem + oc + buf * kCols;
          uint64_t a = sw128_desc(c0 + st * stage_bytes, 16), b = qd;  // addresses in units of 16 bytes
#pragma unroll 1
          for (int x = 0; x < chunks; ++x, a += kChunkBytes / 16, b += kChunkBytes / 16)
            if (leader) {
#pragma unroll
              for (int y = 0; y < 4; ++y) mma_bf16(d, a + 2 * y, b + 2 * y, idesc_s, x | y ? 1u : 0u);
            }
          if (leader) {
            mma_commit(&s_full[buf]);
            if (ns + 1 == n) mma_commit(q_empty);
          }
          ++ns;
        } else {
          ok = wait(&p_full[buf], kk >> 1) && (nv > 0 || seg == 1 || wait(o_empty, seg - 2));
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          uint64_t a = sw128_desc(c0 + st * stage_bytes, kChunkBytes);
          const uint64_t b = sw128_desc(p0 + buf * kPBytes, kChunkBytes);
#pragma unroll 1
          for (int x = 0; x < chunks; x += 2, a += 2 * kChunkBytes / 16)
            if (leader) {
#pragma unroll
              for (int y = 0; y < 4; ++y)
                mma_bf16(tmem + (x >> 1) * kCols, a + 128 * y, b + 128 * y, x + 1 < chunks ? idesc_o : idesc_o64,
                         nv | y ? 1u : 0u);
            }
          if (leader) {
            mma_commit(&c_empty[st]);
            mma_commit(&pv_done[buf]);
          }
          ++nv;
        }
        __syncwarp();
      }
      k += n;
    }
  } else {
    // ---- softmax
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const int c2 = 2 * (lane & 3);
    const float sl = P.scale_log2;
    uint32_t k = 0;
    bool ok = true;
    while (ok && next()) {
      float m[16], l[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) l[i] = 0.0f;
      const bool several = g.s.tlo != g.s.thi;  // tokens: their rows differ
      if (several) {
        if (threadIdx.x < kCols) colt[threadIdx.x] = min(g.s.thi, P.c.start + (g.s.f0 + (int)threadIdx.x) / P.H);
        group_sync(1);
      }
#pragma unroll 1
      for (int t = g.t0; t < g.t1; ++t, ++k) {
        ok = wait(&s_full[k & 1], k >> 1);
        // the weights buffer is free once the tile two before has been used
        if (ok && k >= 2) ok = wait(&pv_done[k & 1], (k >> 1) - 1);
        tc_fence_after();
        uint32_t raw[32];
        tmem_ld_frag(tmem + oc + (k & 1) * kCols + lanes, raw);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(raw[i]);
        const int v0 = t * kTile, v1 = min(v0 + kTile, g.s.cnt), v = v0 + 16 * warp + (lane >> 2);
        if (t == g.t0 && several) {  // the first row may be hidden from some tokens
#pragma unroll
          for (int i = 0; i < 16; ++i) m[i] = kFloor;
        } else if (t == g.t0) {
          if (warp == 0 && lane < 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float2*>(red + 8 * i + c2) =
                  make_float2(fabsf(x[4 * i]) < INFINITY ? x[4 * i] * sl : kFloor,
                              fabsf(x[4 * i + 1]) < INFINITY ? x[4 * i + 1] * sl : kFloor);
          }
          group_sync(1);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 y = *reinterpret_cast<const float2*>(red + 8 * i + c2);
            m[2 * i] = y.x, m[2 * i + 1] = y.y;
          }
        }
        bool renew = !ok;
        uint32_t spoilt = 0;  // bits 0, 1: this thread's rows hold a NaN or infinity that a token must not see
        if (several) {
          // rows that only some of the item's tokens see
          const int first = max(v0, P.sinks);
          if ((v1 - 1 < P.sinks ? v1 - 1 : v1 - 1 + g.s.jump) > g.s.tlo ||
              (P.window && first < v1 && first + g.s.jump <= g.s.thi - P.window)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int vv = v + 8 * h, j = vv < P.sinks ? vv : vv + g.s.jump;
              const int low = P.window && vv >= P.sinks ? j + P.window : 0x7fffffff;  // hidden from there on
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int2 tc = *reinterpret_cast<const int2*>(colt + 8 * i + c2);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int tt = e ? tc.y : tc.x;
                  float& y = x[4 * i + 2 * h + e];
                  // a score of -inf is a row with an infinity: NaN for a token that sees it
                  if (j > tt || tt >= low) {
                    if (!(fabsf(y) < INFINITY)) spoilt |= 1u << h;
                    y = -INFINITY;
                  } else if (y == -INFINITY) {
                    y = __int_as_float(0x7fffffff);
                  }
                }
              }
              if (vv >= g.s.cnt) spoilt &= ~(1u << h);
            }
            renew = renew || spoilt;
          }
        }
        if (v0 + kTile > g.s.cnt) {  // rows past the last one
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (v >= g.s.cnt) x[4 * i] = x[4 * i + 1] = -INFINITY;
            if (v + 8 >= g.s.cnt) x[4 * i + 2] = x[4 * i + 3] = -INFINITY;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            renew = renew || fmaf(fmaxf(x[4 * i + e], x[4 * i + 2 + e]), sl, -m[2 * i + e]) > kStep;
        if (group_or(1, renew)) {
          if (group_or(1, !ok)) {
            ok = false;
            break;
          }
          if (several) {
            // a row that really holds a NaN or infinity is cleared: weight 0 times it is then 0
            spoilt |= __shfl_xor_sync(0xffffffffu, spoilt, 1);
            spoilt |= __shfl_xor_sync(0xffffffffu, spoilt, 2);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              uint8_t* at = sC + (k % nst) * stage_bytes + (16 * warp + (lane >> 2) + 8 * h) * 128 + (lane & 3) * 32;
              uint32_t bad = 0;
              if (spoilt >> h & 1)
#pragma unroll 1
                for (int c = 0; c < 8 * chunks; ++c) {
                  const uint32_t y = *reinterpret_cast<const uint32_t*>(at + (c >> 3) * kChunkBytes + (c & 7) * 4);
                  bad |= (y & 0x7F80u) == 0x7F80u || (y & 0x7F800000u) == 0x7F800000u;
                }
              bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
              bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
              if (bad)
#pragma unroll 1
                for (int c = 0; c < 8 * chunks; ++c)
                  *reinterpret_cast<uint32_t*>(at + (c >> 3) * kChunkBytes + (c & 7) * 4) = 0u;
            }
          }
          float f[16];
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float y = fmaxf(x[4 * i + e], x[4 * i + 2 + e]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
              f[2 * i + e] = y * sl;
            }
          if (lane < 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float2*>(red + warp * 64 + 8 * i + c2) = make_float2(f[2 * i], f[2 * i + 1]);
          }
          group_sync(1);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float2 y = make_float2(m[2 * i], m[2 * i + 1]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float2 z = *reinterpret_cast<const float2*>(red + w * 64 + 8 * i + c2);
              y.x = fmaxf(y.x, z.x), y.y = fmaxf(y.y, z.y);
            }
            f[2 * i] = ex2(m[2 * i] - y.x), f[2 * i + 1] = ex2(m[2 * i + 1] - y.y);
            l[2 * i] *= f[2 * i], l[2 * i + 1] *= f[2 * i + 1];
            m[2 * i] = y.x, m[2 * i + 1] = y.y;
          }
          if (t > g.t0) {
            ok = wait(&pv_done[(k & 1) ^ 1], (k - 1) >> 1);
            if (group_or(1, !ok)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int x2 = 0; x2 < chunks; ++x2) {  // half x2 % 2 of the block of 128 features
              const uint32_t at = tmem + (x2 >> 1) * kCols + lanes + ((uint32_t)(16 * (x2 & 1)) << 16);
              uint32_t o[32];
              tmem_ld_frag(at, o);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * f[2 * (i >> 2) + (i & 1)]);
              tmem_st_frag(at, o);
            }
          } else {
            group_sync(1);  // `red` has been read
          }
        }
        // weights [row][64 queries] as 128-byte swizzled rows; matrices of a store: rows 0-7 and 8-15 of
        // two groups of 8 queries
        const uint32_t at = smem_addr(sP) + (k & 1) * kPBytes + (16 * warp + (lane & 15)) * 128;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          uint32_t pk[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int q = i + (j >> 1), h = j & 1;
            const float p0 = ex2(fmaf(x[4 * q + 2 * h], sl, -m[2 * q])),
                        p1 = ex2(fmaf(x[4 * q + 2 * h + 1], sl, -m[2 * q + 1]));
            l[2 * q] += p0;
            l[2 * q + 1] += p1;
            pk[j] = bf16x2(p0, p1);
          }
          stmatrix4<false>(at + (((i + (lane >> 4)) ^ (lane & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
        }
        fence_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[k & 1]);
      }
      if (!ok) break;
      // the segment's end: sums over the warp's rows
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      if (R::kEpi && seg > 1) {
        ok = wait(l_empty, seg - 2);
        if (group_or(1, !ok)) {
          ok = false;
          break;
        }
      }
      if (lane < 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          *reinterpret_cast<float2*>(fin + warp * 64 + 8 * i + c2) = make_float2(l[2 * i], l[2 * i + 1]);
          if (warp == 0) *reinterpret_cast<float2*>(fin + 256 + 8 * i + c2) = make_float2(m[2 * i], m[2 * i + 1]);
        }
      }
      if constexpr (R::kEpi) {
        __syncwarp();
        if (lane == 0) mbar_arrive(l_full);
      } else {
        group_sync(1);
        ok = finish(warp, 1, k - 1, (int)threadIdx.x);
      }
    }
  }

  // ---- leave: after an abort, let the products already issued complete
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) atomicOr(P.flag, 4);
    if (warp == R::kMma && elect_one()) {  // the lane that issued them
      mma_commit(mma_done);
      mbar_wait_bounded(mma_done, 0);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == R::kMma) tmem_dealloc(tmem, tmem_cols);
}

// ---- pieces of split items joined: one CTA per record and 16 features (a warp's share of a fragment
// load), a thread per four values of a piece.
//   M = max m_p;  out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p
// The pieces are added in order by each of blockDim.y groups of threads and the groups' sums in order
// after that: the result does not depend on timing.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(1024) attention_join_kernel(const AttnParams P) {
  extern __shared__ float wgt[];  // [pieces][64]
  __shared__ float4 acc[4][kJoinThreads];
  __shared__ __align__(16) uint16_t tile[kCols][16];
  __shared__ float red[16][kCols], top[kCols], sum[kCols];
  griddep_wait();
  const int2 rec = P.record[blockIdx.x];
  if (rec.x < 0) return;
  const int n = rec.y, x = blockIdx.y >> 2, w = blockIdx.y & 3, i = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = threadIdx.y, groups = blockDim.y, q = 8 * i + 2 * (lane & 3);
  const Seen s = seen_rows(P, rec.x);
  auto slot = [&](int p) { return 2 * ((int)blockIdx.x + p) + (p == 0 ? 1 : 0); };
  {
    // the pieces' weights: thread rows over pieces, a query a thread
    const int tid = grp * kJoinThreads + threadIdx.x, qq = tid & 63, r0 = tid >> 6, nr = 4 * groups;
    float t = kFloor, z = 0.0f;
    for (int p = r0; p < n; p += nr) t = fmaxf(t, P.part_ml[slot(p) * kCols + qq].x);
    red[r0][qq] = t;
    __syncthreads();
    for (int r = 0; r < nr; ++r) t = fmaxf(t, red[r][qq]);
    __syncthreads();
    for (int p = r0; p < n; p += nr) {
      const float2 y = P.part_ml[slot(p) * kCols + qq];
      const float f = ex2(y.x - t);
      wgt[p * kCols + qq] = f;
      z = fmaf(y.y, f, z);
    }
    red[r0][qq] = z;
    __syncthreads();
    if (r0 == 0) {
      z = 0.0f;
      for (int r = 0; r < nr; ++r) z += red[r][qq];
      top[qq] = t, sum[qq] = z;
    }
    __syncthreads();
  }
  const float4* src = P.part + (x * 4 + w) * 256 + threadIdx.x;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int p = grp; p < n; p += groups) {
    const float4 o = src[(size_t)slot(p) * (kCols * P.D / 4)];
    const float2 f = *reinterpret_cast<const float2*>(wgt + p * kCols + q);
    a.x = fmaf(o.x, f.x, a.x), a.y = fmaf(o.y, f.y, a.y), a.z = fmaf(o.z, f.x, a.z), a.w = fmaf(o.w, f.y, a.w);
  }
  if (groups > 1) {
    acc[grp][threadIdx.x] = a;
    __syncthreads();
    if (grp == 0)
      for (int r = 1; r < groups; ++r) {
        const float4 o = acc[r][threadIdx.x];
        a.x += o.x, a.y += o.y, a.z += o.z, a.w += o.w;
      }
  }
  const long long orow = (long long)s.b * P.c.N * P.H + s.f0, rows = (long long)P.c.B * P.c.N * P.H;
  if (grp == 0) {
    const float i0 = sum[q] == 0.0f ? 0.0f : 1.0f / sum[q], i1 = sum[q + 1] == 0.0f ? 0.0f : 1.0f / sum[q + 1];
    tile[q][lane >> 2] = bf16_bits(a.x * i0), tile[q + 1][lane >> 2] = bf16_bits(a.y * i1);
    tile[q][8 + (lane >> 2)] = bf16_bits(a.z * i0), tile[q + 1][8 + (lane >> 2)] = bf16_bits(a.w * i1);
    if (P.c.lse && blockIdx.y == 0 && threadIdx.x < s.cols && in_bounds(orow + threadIdx.x, rows, P.flag)) {
      const float z = sum[threadIdx.x];
      P.c.lse[orow + threadIdx.x] = z == 0.0f ? -INFINITY : (top[threadIdx.x] + log2f(z)) * 0.693147180559945f;
    }
  }
  __syncthreads();
  // features 16 w of the last 64, else 32 w + 16 h of 128
  const int d = (x | 1) < P.D / 64 ? (x >> 1) * 128 + 32 * w + 16 * (x & 1) : x * 64 + 16 * w;
  const int r = threadIdx.x >> 1, u = threadIdx.x & 1;
  if (grp == 0 && r < s.cols && r < kCols && in_bounds(orow + r, rows, P.flag))
    *reinterpret_cast<uint4*>(P.c.out + (orow + r) * P.D + d + 8 * u) = *reinterpret_cast<const uint4*>(&tile[r][8 * u]);
}

// ---- host side
// Stages: as many tiles (a power of two, at most 8) as the shared memory takes: two CTAs an SM up
// to D = 192 over latents (their tensor memory is 256 columns), else one.
struct Shape {
  int ctas, stages, smem;
};
Shape attn_shape(int D, bool fp4) {
  Shape s;
  s.ctas = D <= 192 && !fp4 ? 2 : 1;
  const int chunk = D / 64 * kChunkBytes, rest = 2 * kPBytes + 4 * kStageOut + kAuxBytes + 1024;
  const int budget = (s.ctas == 2 ? 113 : 227) * 1024 - rest;
  s.stages = 8;
  while (s.stages > 2 && (s.stages + 1) * chunk > budget) s.stages /= 2;
  s.smem = (s.stages + 1) * chunk + rest;
  return s;
}
int attn_slots(int D) { return 2 * current_sm_count() * attn_shape(D, false).ctas; }

}  // namespace

size_t attention_workspace_bytes(int head_dim) {
  return (size_t)attn_slots(head_dim) * (kCols * (head_dim * sizeof(float) + sizeof(float2)) + sizeof(int2)) + 64;
}

cudaError_t launch_attention(csa_attention* a, const AttnCall& call, cudaStream_t s) {
  auto encode = get_encode();
  if (!encode) return cudaErrorNotSupported;
  const bool fp4 = call.paged && !call.cache.latent;
  const Shape sh = attn_shape(a->D, fp4);
  auto* kernel = fp4 ? attention_kernel<true, 1> : sh.ctas == 2 ? attention_kernel<false, 2> : attention_kernel<false, 1>;
  const int threads = fp4 ? Roles<true, 1>::kThreads : sh.ctas == 2 ? Roles<false, 2>::kThreads : Roles<false, 1>::kThreads;
  static std::atomic<unsigned long long> attr{0};
  cudaError_t e = once_per_device(attr, [] {
    const int most = 227 * 1024;
    cudaError_t r = cudaFuncSetAttribute(attention_kernel<true, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(attention_kernel<false, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(attention_kernel<false, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(attention_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
    return r;
  });
  if (e != cudaSuccess) return e;
  const int slots = attn_slots(a->D), most_ctas = current_sm_count() * sh.ctas;
  AttnParams P{};
  P.c = call;
  P.H = a->heads;
  P.D = a->D;
  P.window = a->window;
  P.sinks = a->sinks;
  P.per = (int)(((long long)call.N * a->heads + kCols - 1) / kCols);
  P.items = call.B * P.per;
  P.scale_log2 = (float)(a->scale * 1.4426950408889634);
  P.flag = a->dev_flag;
  P.part = (float4*)a->workspace;
  P.part_ml = (float2*)((float*)a->workspace + (size_t)slots * kCols * a->D);
  P.record = (int2*)(P.part_ml + (size_t)slots * kCols);
  P.ticket = (int*)(P.record + slots);
  P.stages = sh.stages;
#ifdef CSA_DEBUG_BOUNDS
  P.test_stall = getenv("CSA_TEST_STALL_LAST_STAGE") != nullptr;
  P.wait_ns = P.test_stall ? 200000000ull : kWaitNs;
#endif
  // the longest range of rows that this call can have decides whether items may be cut
  long long most = call.paged ? (long long)call.max_pages * call.cache.page_size : (long long)call.start + call.N;
  const long long window = (long long)a->window + a->sinks + kCols / a->heads;
  if (a->window && most > window) most = window;
  P.split = most > (long long)kJoinTiles * kTile;
  const long long longest = most > kTile ? (most + kTile - 1) / kTile : 1, tiles = P.items * longest;
  const long long shares = P.split ? tiles : P.items;
  const int grid = (int)(shares < most_ctas ? shares : most_ctas);
  CUtensorMap mq;
  {
    cuuint64_t dims[2] = {(cuuint64_t)a->D, (cuuint64_t)call.B * call.N * a->heads};
    cuuint64_t strides[1] = {(cuuint64_t)a->D * 2};
    cuuint32_t box[2] = {64, kCols};
    cuuint32_t es[2] = {1, 1};
    if (encode(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (void*)call.q, dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  kernel<<<grid, threads, sh.smem, s>>>(mq, P);
  a->launches += 1;
  if ((e = cudaGetLastError()) != cudaSuccess || !P.split) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, a->D / 16);
  // few items have many pieces each: four groups of threads share them
  cfg.blockDim = dim3(kJoinThreads, P.items * 8 <= grid ? 4 : 1);
  // an item's pieces: every CTA has at least kMinTiles tiles
  cfg.dynamicSmemBytes = kCols * sizeof(float) * (longest / kMinTiles + 2 < grid ? longest / kMinTiles + 2 : grid);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  a->launches += 1;
  return cudaLaunchKernelEx(&cfg, attention_join_kernel, P);
}

}  // namespace csa
