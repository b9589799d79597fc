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
// long as it is near.  It begins as 0, and is only renewed (as the tile's maximum, with O^T and l
// scaled) when a score passes it by 16 base-2 steps, or when a query's first scores are all below
// -64: taking the maximum over rows costs an exchange between the warps that most tiles need not pay.
// (Items of a single tile always pay it: with few rows the largest weight should be 1, which is exact.)
//
// What bounds it (probes on GB300, cycles): a 64 x 64 x 16 MMA takes 32 and a 128 x 64 x 16 one 48
// (shared-memory reads of both operands at 128 bytes a cycle), so a tile of 64 rows at D = 512 costs
// 1024 + 768; its 64 KB arrive from HBM in 2510 (26 bytes a cycle and SM, 7.2 TB/s) and from L2 in 700.
// A tile passes four stations one after the other, its copy, the scores (1100), the softmax (1200)
// and the values (900), and shared memory holds two tiles of 512 features beside the queries, so two
// tiles go through them at a time:
//   decode over latents  3200 cycles a tile, 0.78 of that rate while tiles stream; 128 sequences of up
//                        to 2048 entries, 64 heads of 512: 48.9 us in all (152 MB, 3.1 TB/s), of which 4
//                        pass before the first copy (lengths, shares, page table: one after the other),
//                        2.3 until it lands, 2.5 in the last pieces' stores and 8.5 in their join
//   decode over codes    3750 cycles a tile, 1900 of them the expansion of codes to bf16 (736 are its
//                        instructions' issue, the rest latencies with two of these warps a scheduler):
//                        50.1 us, 0.9 of it gained since by the hardware's conversion of the scales
//   a prompt's window    7400 cycles an item of two tiles: the epilogue reads O^T for 5000 of them, which
//                        the next item's values wait for block by block (there is no room for a second
//                        whole O^T at D = 512; two of its four blocks would fit, which is not built): 4096
//                        tokens, 64 heads of 512, window 128: 112.4 us (542 MB, 4.8 TB/s)
//   narrow heads         1250 cycles a tile at D = 128, the softmax alone: 2 x 1777 tokens, 16 heads, window
//                        512: 45.1 us (0.3 of it the look at rows whose scores pass f32's range)
// (times: a call in a graph of 16 or 64 of them over changing inputs)
//
// Measured and not taken: stages handed over by blocks of 128 features (decode 128 x 2048 1 % faster, a
// windowed prompt 2 to 8 % and codes 4 % slower); products over rows in steps that leave out a last
// tile's absent rows (1 % slower, 2 % faster for windows of 128 + 4); rows by four-row TMA gathers (8010
// cycles a tile; cp.async 760 from L2, any page size, absent rows as zeros); a second set of registers in
// the epilogue (spills: 112 -> 146 us); two tiles a softmax step with four score and weights buffers (D = 128:
// the same over long ranges, 56 -> 69 us for 4096 tokens with a window of 128).
//
// Work is cut by tiles: the call's tiles, in item order (and a tile's time for each item), are divided
// evenly over the CTAs, so ragged lengths and few long sequences fill the GPU alike; an item cut by a CTA
// boundary leaves partial (m, l, O) pieces in the workspace, which a second kernel joins.  Where cutting
// would cost more than it saves, items are whole: one a CTA, or a share's by their starts.  Without a
// tile's time for each item, CTAs with three items ended 4 us after those with one (decode 128 x 2048:
// 49.3 -> 47.6 us).
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
constexpr int kStageOut = 1024;                // a warp's staging of 16 queries x 32 features bf16
constexpr int kCutMany = 8;  // units (see units_of) that cutting items costs: their pieces and the join
constexpr int kCutFew = 3;   // and where the items are few
constexpr float kStep = 16.0f;  // base-2 steps a score may pass the reference by
constexpr float kLow = -64.0f;  // where the first scores are all lower, 0 is no reference for them
constexpr float kFloor = -3.402823466e38f;  // the maximum of no scores
// Base-2 scores from here on (either sign) have no digits behind the point, and x * scale - m, which is
// rounded once, would be off by half a step of the reference m, up to any power of two: as maxima they
// make the reference, and with it the result, NaN.  Below, that is a factor of 2^-32 to 2^32 common to all of a
// query's weights.
constexpr float kHuge = 1073741824.0f;
constexpr int kAuxBytes = 6144;   // barriers, flags, references and sums

// Division of 31-bit numbers by a number known to the host: with l = ceil(log2 d) and
// m = floor(2^(31 + l) / d) + 1, n / d = (m n) >> (31 + l) (Granlund and Montgomery, 1994).
struct Divisor {
  uint32_t d, m;
  int shift;
  Divisor(uint32_t by = 1) : d(by), shift(31) {
    while ((1u << (shift - 31)) < by) ++shift;
    m = (uint32_t)((1ull << shift) / by + 1);
  }
  __device__ __forceinline__ int of(int n) const { return (int)(((uint64_t)m * (uint32_t)n) >> shift); }
};

struct AttnParams {
  AttnCall c;
  int H, D, window, sinks;
  int per, items;    // items of a sequence, of the call
  Divisor by_per, by_heads, by_page;
  float scale_log2;  // scale * log2(e): scores in base-2 exponents
  int* flag;
  float4* part;      // pieces: [2 * grid][64 * D / 4] f32, in the order of the fragment loads
  float2* part_ml;   // (maximum, sum) of each piece and query [2 * grid][64]
  int2* record;      // per CTA: (item, pieces) of an item whose first piece it made, or (-1, 0); per
                     // item with few of them: (CTA of the first piece, pieces), or (-1, 0)
  int ctas;          // of the kernel that leaves pieces
  bool few;
  int log_stages;
  bool split;        // items may be cut (the join kernel follows); else they are drawn from `ticket`
  int* ticket;       // items drawn beyond each CTA's first; 0 between calls
#ifdef CSA_DEBUG_BOUNDS
  long long rows, slots;  // extents of the outputs and of the workspace's pieces (and records)
  uint64_t wait_ns;       // the time-out tests shorten the waits
  int test_stall;         // and leave out each CTA's first tile
  int test_late;          // or publish each CTA's first segment only once a wait for it has run out
#endif
};

// The bounds-checked build's checks of a store: to row `row` of the outputs, to element i of the pieces,
// their statistics or the records, `per` of which make a slot.
#ifdef CSA_DEBUG_BOUNDS
__device__ __forceinline__ bool in_rows(const AttnParams& P, long long row) { return in_bounds(row, P.rows, P.flag); }
__device__ __forceinline__ bool in_slots(const AttnParams& P, long long i, long long per) {
  return in_bounds(i, P.slots * per, P.flag);
}
#else
__device__ __forceinline__ bool in_rows(const AttnParams&, long long) { return true; }
__device__ __forceinline__ bool in_slots(const AttnParams&, long long, long long) { return true; }
#endif

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
  s.b = P.by_per.of(item);
  s.f0 = (item - s.b * P.per) * kCols;
  if (P.c.paged) {
    const int top = P.c.max_pages * P.c.cache.page_size, n = P.c.lens[s.b];
    s.cols = min(kCols, P.H - s.f0);
    s.tlo = s.thi = min(max(n, 0), top) - 1;
  } else {
    const int n = P.c.lens ? min(max(P.c.lens[s.b], 0), P.c.N) : P.c.N;
    s.cols = max(0, min(kCols, n * P.H - s.f0));
    s.tlo = P.c.start + P.by_heads.of(s.f0);
    s.thi = P.c.start + P.by_heads.of(s.f0 + max(s.cols, 1) - 1);
  }
  // every token from tlo on sees the rows after thi - most and the sinks at most
  const int most = P.window + (s.thi - s.tlo) + P.sinks;
  const bool all = P.window == 0 || s.thi + 1 <= most;
  s.cnt = all ? s.thi + 1 : most;
  s.jump = all ? 0 : s.thi + 1 - most;
  return s;
}
__device__ __forceinline__ int tiles_of(const Seen& s) {
  return s.cols == 0 ? 0 : max(1, (s.cnt + kTile - 1) / kTile);  // a sequence without entries still has its output
}

// What an item costs in a split call's shares, in tiles: a CTA takes about as long over changing to an
// item (its queries' copy, the epilogue) as over a tile.
__device__ __forceinline__ int units_of(int tiles) { return tiles == 0 ? 0 : tiles + 1; }

// A run of tiles of one item, as the scheduling warp hands it to the others through a ring of slots.
struct __align__(16) Segment {
  Seen s;
  int item, t0, t1, tiles;  // tiles [t0, t1) of the item's; t1 0: no more segments
  int index;                // units of the call before this segment (split calls)
};
static_assert(sizeof(Segment) == 48, "a ring slot");
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
// The same over 32 columns, not waiting.
__device__ __forceinline__ void tmem_ld_half(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_half(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
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
// A barrier of some warps (1: softmax, 2: epilogue); group_or gives every thread whether any passed
// true.
constexpr int kSoftWarps = 8;
template <int kWarps = kSoftWarps>
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(32 * kWarps) : "memory");
}
template <int kWarps = kSoftWarps>
__device__ __forceinline__ bool group_or(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id), "n"(32 * kWarps)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ uint64_t l2_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
      "%4}], [%5], %6;" ::"r"(smem_addr(dst)),
      "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
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

// Two e4m3 scales, the first in the low byte.  The caller's arrays may hold any byte: 0x7F and 0xFF are
// NaN, and make the entry's block NaN.
__device__ __forceinline__ float2 e4m3x2_values(uint32_t bytes) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)bytes, __NV_E4M3)));
}

// Eight e2m1 codes (element 0 in the low nibble) times a scale (bf16x2) to eight bf16.  The bytes of
// a magnitude's bf16 pattern (0, .5, 1, 1.5, 2, 3, 4, 6) are looked up by byte permutation; products
// of 2 and 4 significant bits are exact in bf16.
__device__ __forceinline__ uint4 dequant8(uint32_t w, uint32_t scale2) {
  const uint32_t m = w & 0x77777777u;
  uint32_t v[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // four codes each
    const uint32_t sel = m >> (16 * h), lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
    // high bytes with the codes' signs, bits 3 and 7 of the two bytes that hold them
    const uint32_t b = __byte_perm(w, 0u, h ? 0x3322 : 0x1100);
    const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel) | (((b & 0xFF00FF00u) | ((b << 4) & 0x00FF00FFu)) & 0x80808080u);
    v[2 * h] = __byte_perm(lo, hi, 0x5140);
    v[2 * h + 1] = __byte_perm(lo, hi, 0x7362);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(scale2));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// ---- the kernel's warps: 0-7 softmax (TMEM lane quarter = warp % 4, 32 of the 64 queries each); 8-15 the
// epilogue, which reads O^T while the softmax warps go on with the next item; then two that issue the
// MMAs (scores run up to two tiles ahead of values, also into the next item, without one loop having to
// look out for both), one that schedules and copies the queries, and the rows' warps: for latents two
// groups that take alternate tiles (one group's can be in flight while the other waits for its stage).
// One CTA an SM at every D: two of half the warps sharing an SM up to D = 192 (their softmax warps
// reading their own O^T) took 118 us where one took 66 (2 x 1777 tokens, D 128, window 512).
// Codes need more warps to expand them, which are half of the epilogue's, and all eight take a tile's
// rows together, eight rows each: expanding them takes 1900 cycles of a tile's 3750 (alternate tiles by
// four warps each: 52.3 us where this takes 49.0, 128 sequences of up to 2048 entries; a second set of
// registers for the next tile's codes: 50.1).
constexpr int kEpiWarp = 8;
constexpr int kAttnThreads = 32 * 23;
template <bool kFp4>
struct Roles {
  static constexpr int kEpiWarps = kFp4 ? 4 : 8;
  static constexpr int kMma = kEpiWarp + kEpiWarps, kVal = kMma + 1, kQ = kMma + 2, kRow = kMma + 3;
  static constexpr int kRowWarps = kAttnThreads / 32 - kRow;
  static constexpr int kRowGroup = kFp4 ? kRowWarps : kRowWarps / 2;                    // a group brings a tile
  static constexpr int kTileRows = kTile / kRowGroup;                                   // of which a warp these
};

template <bool kFp4>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_c,
                     const __grid_constant__ AttnParams P) {
  using R = Roles<kFp4>;
  constexpr int kEpiWarps = R::kEpiWarps, kMmaWarp = R::kMma, kValWarp = R::kVal, kQWarp = R::kQ, kRowWarp = R::kRow;
  constexpr int kRowWarps = R::kRowWarps, kRowGroup = R::kRowGroup, kTileRows = R::kTileRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int D = P.D, chunks = D / 64;
  const uint32_t lst = P.log_stages, nst = 1u << lst;  // stages: a power of two
  const int stage_bytes = chunks * kChunkBytes;
  uint8_t* sQ = smem;
  uint8_t* sC = sQ + chunks * kChunkBytes;
  uint8_t* sP = sC + nst * stage_bytes;  // two weights buffers
  uint8_t* sO = sP + 2 * kPBytes;        // the epilogue's staging, 1 KB a warp
  uint8_t* aux = sO + 8 * kStageOut;
  uint64_t* c_full = (uint64_t*)aux;  // [8] a stage's rows have landed
  uint64_t* c_empty = c_full + 8;     // [8] a stage's products are done
  uint64_t* s_full = c_empty + 8;     // [2] scores ready
  uint64_t* p_full = s_full + 2;      // [2] weights written, scores read
  uint64_t* pv_done = p_full + 2;     // [2] second product done: weights buffer free, O^T complete to it
  uint64_t* g_full = pv_done + 2;     // [4] a segment's slot is written
  uint64_t* g_empty = g_full + kRing; // [4] and has been read by every role
  uint64_t* q_full = g_empty + kRing;
  uint64_t* q_empty = q_full + 1;
  uint64_t* o_empty = q_empty + 1;    // [4] O^T's block of 128 features has been read
  uint64_t* l_full = o_empty + 4;     // the item's references and sums are in `fin`
  uint64_t* l_empty = l_full + 1;     // and have been read
  uint64_t* mma_done = l_empty + 1;   // clean-up after an abort
  uint32_t* tmem_slot = (uint32_t*)(mma_done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  Segment* ring = (Segment*)(aux + 384);
  int* work = (int*)(aux + 640);  // split calls: units of a share, shares with one more
  float* red = (float*)(aux + 704);   // [2][64] references, factors
  float* fin = red + 128;             // [16][64] sums over rows, [64] references
  float* inv = fin + 1088;            // [64] 1 / sum
  int* colt = (int*)(inv + 64);       // [64] the queries' positions
  static_assert(704 + (128 + 1088 + 64 + 64) * 4 <= kAuxBytes, "aux region");

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
      mbar_init(&c_full[s], kRowGroup);
      mbar_init(&c_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSoftWarps);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&g_full[i], 1);
      mbar_init(&g_empty[i], kAttnThreads / 32 - 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&o_empty[i], kEpiWarps);
    mbar_init(l_full, kSoftWarps);
    mbar_init(l_empty, kEpiWarps);
    mbar_init(mma_done, 2);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_map(&map_q);
  }
  const uint32_t oc = (uint32_t)((D + 127) / 128) * kCols;  // columns of O^T; two score buffers follow
  const uint32_t tmem_cols = oc + 2 * kCols <= 256 ? 256 : 512;
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, tmem_cols);
  griddep_wait();  // what the launches before this one wrote and read
  griddep_launch_dependents();

  if (blockIdx.x == 0 && P.c.lens) {  // lengths out of range are taken as the nearest end
    const int most = P.c.paged ? P.c.max_pages * P.c.cache.page_size : P.c.N;
    for (int b = threadIdx.x; b < P.c.B; b += kAttnThreads) {
      const int n = P.c.lens[b];
      if (n < 0 || n > most) atomicOr(P.flag, 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  // The next segment, for every role but the scheduling warp; false behind the last one and after an
  // abort.  The softmax's and the epilogue's warps meet at named barriers, which have no time limit, and
  // after an abort one of them may still find a slot written that another has given up on: they go on or
  // leave by their group's common decision (the epilogue's here, the softmax's at its first tile's barrier,
  // which costs it none), all others by the warp's own.
  uint32_t seg = 0;  // segments read
  Segment g;
  auto next = [&]() {
    const uint32_t slot = seg % kRing;
    const bool there = wait(&g_full[slot], seg / kRing);
    if (warp >= kEpiWarp && warp < kMmaWarp ? group_or<kEpiWarps>(2, !there) : !__all_sync(0xffffffffu, there)) {
      g.t1 = -1;
      return false;
    }
    g = ring[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&g_empty[slot]);
    ++seg;
    return g.t1 > 0;
  };

  // ---- an item's end, by the epilogue's warps, one or two of each of O^T's lane quarters (warp % 4; two
  // share its columns or halves): the sums over rows in `fin`, O^T (complete with tile kl) scaled to
  // out, or left as a piece.  A block of 128 features is given back to the MMAs as soon as it has
  // been read.  False after an abort.
  auto finish = [&](uint32_t kl, int tid) -> bool {
    constexpr int kTwo = kEpiWarps / 4;
    const int w = warp & 3, half = tid >> 7;
    bool ok = wait(l_full, seg - 1);
    const bool whole = g.t0 == 0 && g.t1 == g.tiles;
    // a piece: slot 0 of the CTA for its first segment's, 1 for its last's (an item's first piece)
    const int slot = 2 * blockIdx.x + (g.t0 == 0 ? 1 : 0);
    const long long orow = (long long)g.s.b * P.c.N * P.H + g.s.f0;
    if (ok && tid < kCols) {
      float l = 0.0f;
#pragma unroll 4
      for (int i = 0; i < 16; ++i) l += fin[64 * i + tid];
      const float m = fin[1024 + tid];
      if (whole) {
        float r, lg;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(l));
        asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(l));
        inv[tid] = l == 0.0f ? 0.0f : r;
        if (P.c.lse && tid < g.s.cols && in_rows(P, orow + tid))
          P.c.lse[orow + tid] = l == 0.0f ? -INFINITY : (m + lg) * 0.693147180559945f;
      } else if (in_slots(P, slot * kCols + tid, kCols)) {
        P.part_ml[slot * kCols + tid] = make_float2(l == 0.0f ? kFloor : m, l);  // (no row: no reference either)
      }
    }
    // (the sums are there before the last product over rows is done)
    ok = ok && wait(&pv_done[kl & 1], kl >> 1);
    if (group_or<kEpiWarps>(2, !ok)) return false;
    tc_fence_after();
    if (lane == 0) mbar_arrive(l_empty);
    auto give_back = [&](int block) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_empty[block]);
    };
    const uint32_t base = tmem + ((uint32_t)(32 * w) << 16);
    if (whole) {
      if (P.split && P.few && tid == 0 && in_slots(P, g.item, 1)) P.record[g.item] = make_int2(-1, 0);
      // steps of 32 queries x 32 features (16 of a last block of 64) a warp; the next step's loads run
      // ahead of a step's stores
      const int steps = (chunks + 1) & ~1;  // two of a block
      float2 f[4];
      auto factors = [&](int c) {
#pragma unroll
        for (int q = 0; q < 4; ++q) f[q] = *reinterpret_cast<const float2*>(inv + 32 * c + 8 * q + 2 * (lane & 3));
      };
      if (kTwo == 2) factors(half);
      // to [query][32 features] by transposed stores, 16 queries at a time; 16-byte units swizzled against
      // conflicts: row r of 64 bytes, unit u at u ^ (r / 2 % 4)
      uint8_t* const stage = sO + (warp & 7) * kStageOut;
      const int r = 8 * (lane >> 4) + (lane & 7);
      const uint32_t put = smem_addr(stage) + r * 64 + ((((lane >> 3) & 1) ^ ((r >> 1) & 3)) << 4);
      const uint8_t* const get = stage + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
      uint8_t* const to = reinterpret_cast<uint8_t*>(
          P.c.out + (orow + (kTwo == 2 ? 32 * half : 0) + (lane >> 2)) * D + 32 * w + 8 * (lane & 3));
      uint32_t o[2][16];
      tmem_ld_half(base + 32 * half, o[0]);
      tmem_ld_half(base + 32 * half + (16u << 16), o[1]);
#pragma unroll 1
      for (int step = half; step < steps; step += kTwo) {
        const int x = step & ~1, c = step & 1;
        const bool full = x + 1 < chunks;
        if (kTwo == 1) factors(c);
        tmem_ld_wait();
        uint32_t v[2][2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int q = 2 * i + (j >> 1);
              v[i][h][j] = bf16x2(__uint_as_float(o[h][4 * q + 2 * (j & 1)]) * f[q].x,
                                  __uint_as_float(o[h][4 * q + 2 * (j & 1) + 1]) * f[q].y);
            }
        if (kTwo == 2 || c == 1) give_back(step >> 1);
        if (step + kTwo < steps) {
          const uint32_t at = base + 32 * (step + kTwo);  // 64 columns a block of 128 features
          tmem_ld_half(at, o[0]);
          tmem_ld_half(at + (16u << 16), o[1]);
        }
        uint8_t* dst = to + (long long)(x * 128 + (full ? 0 : -32 * w)) + (kTwo == 1 ? 64 * D * c : 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            stmatrix4<true>(put ^ (h << 5), v[i][h][0], v[i][h][1], v[i][h][2], v[i][h][3]);
          __syncwarp();
          uint4 y[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) y[z] = *reinterpret_cast<const uint4*>(get + 512 * z);
          __syncwarp();
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int q = 32 * c + 16 * i + 8 * z + (lane >> 2);
            if ((full || (lane & 3) < 2) && q < g.s.cols && in_rows(P, orow + q))
              *reinterpret_cast<uint4*>(dst + (16 * i + 8 * z) * 2 * D) = y[z];
          }
        }
      }
    } else {
      float4* dst = P.part + (size_t)slot * (kCols * D / 4) + w * 256 + lane;
#pragma unroll 1
      for (int x = half; x < ((chunks + 1) & ~1); x += kTwo) {  // half x % 2 of 16 lanes a warp of a block
        if (x < chunks) {
        uint32_t o[32];
        tmem_ld_frag(base + (x >> 1) * kCols + ((uint32_t)(16 * (x & 1)) << 16), o);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (in_slots(P, (dst - P.part) + (x * 32 + i) * 32, kCols * D / 4)) dst[(x * 32 + i) * 32] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                               __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        }
        if (kTwo == 2 || (x & 1)) give_back(x >> 1);
      }
      if (g.t0 == 0 && tid == 0) {
        // the item ends in the CTA whose share holds its last tile
        const int last = g.index + g.tiles, each = work[0], more = work[1], wide = more * (each + 1);
        const int j = last < wide ? last / (each + 1) : more + (last - wide) / each;
        const int n = j - (int)blockIdx.x + 1;
        const int at = P.few ? g.item : (int)blockIdx.x;
        if (in_slots(P, at, 1)) P.record[at] = make_int2(P.few ? (int)blockIdx.x : g.item, n);
      }
    }
    return true;
  };

  if (warp == kQWarp) {
    int first_item = blockIdx.x, first_tile = 0, share = 0, first_index = 0;
    if (P.split) {
      // ---- the CTA's share of the call's units: every CTA's scheduling warp adds up the items' (lanes over
      // contiguous items; the other roles' instructions arrive meanwhile) and finds its first one
      const int per = (P.items + 31) / 32, lo = min(P.items, per * lane), hi = min(P.items, lo + per);
      int sum = 0, top = 0;  // (the host has made sure that the call's units fit)
#pragma unroll 1
      for (int i = lo; i < hi; ++i) {
        const int n = tiles_of(seen_rows(P, i));
        sum += units_of(n);
        top = max(top, n);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      int pre = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += y;
      }
      const int total = __shfl_sync(0xffffffffu, pre, 31);
      pre -= sum;
      // Items are cut where that saves more units than it costs.  Uncut, each has a CTA of its own or, where
      // they are more than the CTAs, a CTA has its rounds of equal items or at most one more than its share.
      // (64 heads of 512: 128 x 512 entries 22.8 us uncut and 33.8 us cut, 300 x 512 40.6 and 54; 128 sequences
      // of up to 1024 34.6 us cut and 48 us uncut.  Shares are four units at least, but two up to 64 CTAs: the
      // fewer pieces join faster, 1 x 32768 22.6 us against 24 us, the shorter shares matter where they are
      // few, 1 x 4096 14.9 us against 17 us.  At 64, 128, 256 and 512 features, 64 and 16 heads, each way forced,
      // in graphs: the rule's is the faster one or within 4 % of it for nine of eleven batches, 300 x 640 to 1 x
      // 32768; it errs for ragged ones of a few tiles an item: 128 of up to 1024 entries at 128 features 19.8 us
      // cut and 17.9 uncut, 40 of up to 700 at 512 features 27.1 us uncut and 20.9 cut.)
      int ctas = min((int)gridDim.x, max(1, max(min(64, total / 2), total / 4)));
      const int longest = units_of(top);
      const bool own = P.items <= (int)gridDim.x;
      const long long uncut = own ? longest
                              : total == (long long)P.items * longest
                                  ? (long long)((P.items - 1) / (int)gridDim.x + 1) * longest
                                  : (long long)total / (int)gridDim.x + longest;
      const bool cut = uncut > total / ctas + (P.few ? kCutFew : kCutMany);
      if (!cut) ctas = gridDim.x;
      // share i begins at each * i + min(i, more)
      const int each = total / ctas, more = total - each * ctas, i0 = min((int)blockIdx.x, ctas), i1 = min(i0 + 1, ctas);
      const int a = each * i0 + min(i0, more), e = each * i1 + min(i1, more);
      // a boundary x: the item it falls in or, without cutting, the first item that starts from it on
      // (scalars: an array of both would lie in local memory)
#pragma unroll 1
      for (int w = 0; w < 2; ++w) {
        const int x = w ? e : a;
        int item = P.items, tile = 0, start = total;
        if (x >= pre && x < pre + sum) {
          int at = pre;
          item = lo;
          int n = units_of(tiles_of(seen_rows(P, item)));
#pragma unroll 1
          while (x >= at + n) at += n, n = units_of(tiles_of(seen_rows(P, ++item)));
          // the unit of the change goes with the first tile
          tile = max(0, x - at - 1), start = tile ? x : at;
          if (!cut && tile > 0) ++item, tile = 0, start = at + n;
        }
        const uint32_t who = __ballot_sync(0xffffffffu, x >= pre && x < pre + sum);
        const int from = who ? __ffs(who) - 1 : 0;
        start = __shfl_sync(0xffffffffu, start, from);
        if (w == 0) {
          first_item = __shfl_sync(0xffffffffu, item, from), first_tile = __shfl_sync(0xffffffffu, tile, from);
          first_index = start;
        } else {
          share = start - first_index;
        }
      }
      if (own && !cut) {
        first_item = blockIdx.x, first_tile = 0;
        share = first_item < P.items ? units_of(tiles_of(seen_rows(P, first_item))) : 0;
      }
      if (lane == 0) {
        work[0] = each, work[1] = more;  // (read by whoever leaves an item's first piece)
        if (!P.few && in_slots(P, blockIdx.x, 1)) P.record[blockIdx.x] = make_int2(-1, 0);
      }
    }
    // ---- scheduling and queries (one lane).  A split call's segments are the CTA's share; otherwise
    // items are drawn one at a time from the last (a prompt's longest) on, the CTA's first by its own
    // number: SMs differ in speed, items in length and padding in place.  The CTA that draws the last
    // ticket sets the counter back.  A segment is
    // published one ahead of its queries' copy (64 rows of [B * N * H][D] from the item's first; rows past
    // its last are other sequences' or zeros: columns that nothing reads).
#ifdef CSA_DEBUG_BOUNDS
    if (P.test_late && lane == 0) {
      const uint64_t t0 = globaltimer();
      while (!*abort_flag && globaltimer() - t0 < 4 * kWait) {}
    }
    __syncwarp();
#endif
    if (lane == 0) {
      const bool split = P.split;
      int item = first_item, tile = first_tile, drawn = 0, left = share, index = first_index;
      uint32_t n = 0, loads = 0;
      bool end = false;
      auto draw = [&]() {
        const int t = atomicAdd(P.ticket, 1);
        if (t == P.items - 1) *P.ticket = 0;  // every CTA draws until it is past the last item
        return (int)gridDim.x + t;
      };
      auto advance = [&](const Segment& a) {
        const int units = a.t0 == 0 ? units_of(a.t1) : a.t1 - a.t0;
        left -= units;
        index += units;
        tile = 0;
        if (split) {
          ++item;
        } else {
          item = drawn;
          if (item < P.items) drawn = draw();
        }
      };
      if (!split) drawn = draw();
      int row = 0, bytes = 0;  // queries still to be copied: those of the segment published last
      for (;;) {
        Segment a;
        bool more = false;
        while (!end) {
          end = item >= P.items || (split && left <= 0);
          if (end) break;
          a.item = split ? item : P.items - 1 - item;
          a.s = seen_rows(P, a.item);
          a.tiles = tiles_of(a.s);
          a.t0 = tile;
          a.t1 = split ? min(a.tiles, tile == 0 ? left - 1 : tile + left) : a.tiles;
          a.index = index;
          more = a.t1 > tile;
          if (more) break;
          advance(a);  // padding
        }
        if (!more) a.t1 = 0;
        if (n >= kRing && !wait(&g_empty[n % kRing], n / kRing - 1)) break;
        ring[n % kRing] = a;
        mbar_arrive(&g_full[n % kRing]);
        if (more) advance(a);
        const int next_row = more ? a.s.b * P.c.N * P.H + a.s.f0 : 0, next_bytes = more ? a.s.cols * D * 2 : 0;
        if (n == 0) row = next_row, bytes = next_bytes;  // the first segment's at once
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
  } else if (warp >= kEpiWarp && warp < kMmaWarp) {
    uint32_t k = 0;
    while (next()) {
      k += g.t1 - g.t0;
      if (!finish(k - 1, (int)threadIdx.x - 256)) break;
    }
  } else if (warp >= kRowWarp) {
    // ---- rows: warp w of a group brings rows kTileRows * w .. of its group's tiles
    const int grp = (warp - kRowWarp) / kRowGroup, w = (warp - kRowWarp) % kRowGroup;
    const uint8_t* base = (const uint8_t*)(P.c.paged ? P.c.cache.latent : P.c.kv);
    // eight rows at a time, four lanes a row, such that the eight lanes of a quarter warp hit every bank
    // of the swizzled rows once: rows r and r + 4 side by side for 16-byte units, eight rows for units
    // that expand to 64 bytes
    const int r8 = kFp4 ? lane & 7 : (lane >> 3) + 4 * ((lane >> 2) & 1), u0 = kFp4 ? lane >> 3 : lane & 3;
    constexpr int kGroups = kTileRows / 8;  // (latents)
    // a cache's rows are read once by a call: they are not to drive pieces out of L2
    const uint64_t policy = P.c.paged ? l2_evict_first() : l2_evict_normal();
    uint32_t k = 0;
    int pending = -1;  // a stage whose copies were issued and not yet handed over
    bool ok = true;
    // visible row v: the entry's row in the cache, or -1 past the last one (and for a page outside the
    // cache)
    auto entry = [&](int v) -> int {
      if (v >= g.s.cnt) return -1;
      const int j = v < P.sinks ? v : v + g.s.jump;
      if (!P.c.paged) return g.s.b * P.c.kv_rows + j;
      const int ps = P.c.cache.page_size, pg = P.by_page.of(j);
      const int page = P.c.page_table[(long long)g.s.b * P.c.max_pages + pg];
      if (page >= 0 && page < P.c.cache.pages) return page * ps + (j - pg * ps);
      atomicOr(P.flag, 2);
      return -1;
    };
    auto hand_over = [&](int st) {  // this warp's rows have landed
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c_full[st]);
    };
    auto flush = [&]() {
      if (pending >= 0) {
        cp_wait<0>();
        hand_over(pending);
        pending = -1;
      }
    };
    auto stage_free = [&](uint32_t st) {  // the whole warp's answer
      if (!kFp4 && k >= nst && !__all_sync(0xffffffffu, mbar_test(&c_empty[st], ((k >> lst) - 1) & 1))) flush();
      return __all_sync(0xffffffffu, k < nst || wait(&c_empty[st], (k >> lst) - 1)) != 0;
    };
    while (ok) {
      if (!kFp4 && !__all_sync(0xffffffffu, mbar_test(&g_full[seg % kRing], (seg / kRing) & 1))) flush();
      if (!next()) break;
      // these warps are ahead of the others: they ask the segment's queries into L2 (as plain prefetches:
      // a bulk one holds up the tensor copies behind it)
      const uint8_t* qrow = (const uint8_t*)(P.c.q + ((size_t)g.s.b * P.c.N * P.H + g.s.f0) * D);
      for (int x = 128 * ((int)threadIdx.x - 32 * kRowWarp); x < g.s.cols * D * 2; x += 128 * 32 * kRowWarps)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(qrow + x));
      int e0 = 0, e1 = 0;  // lane l's entries l and l + 32 of the tile
      bool known = false;  // (found when the tile was looked ahead to)
#pragma unroll 1
      for (int t = g.t0; t < g.t1; ++t, ++k) {
        if (!kFp4 && (int)(k & 1) != grp) continue;
        const uint32_t st = k & (nst - 1);
#ifdef CSA_DEBUG_BOUNDS
        if (P.test_stall && k == 0) break;  // test of the time-out path: the first tile never comes
#endif
        const uint32_t dst = smem_addr(sC) + st * stage_bytes;
        if (!known) e0 = entry(t * kTile + lane), e1 = entry(t * kTile + 32 + lane);
        // The group's next tile: its entries, asked into L2 (a half by each warp of the group).  Two stages of
        // 64 KB a CTA are not enough bytes in flight for HBM's latency.
        auto look_ahead = [&](int next_t) {
          known = next_t < g.t1;
          if (!known) return;
          e0 = entry(next_t * kTile + lane), e1 = entry(next_t * kTile + 32 + lane);
          const int row = w == 0 ? e0 : w == 1 ? e1 : -1;
          const uint8_t* at = kFp4 ? P.c.cache.codes + (size_t)max(row, 0) * (D / 2) : base + (size_t)max(row, 0) * (2 * D);
          if (row >= 0)
            for (int x = 0; x < (kFp4 ? D / 2 : 2 * D); x += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + x));
          if (kFp4 && row >= 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(P.c.cache.scales + (size_t)row * (D / 16)));
        };
        if constexpr (kFp4) {
          // codes, expanded into the bf16 operand: a lane takes 32 codes and two scales (half a chunk) of
          // its row at a time; they are on their way while the stage's last products run
          const int upr = D / 32;
          uint4 code[4];
          uint32_t sc[4];
          const uint32_t r = kTileRows * w + r8;
          {
            const int a = __shfl_sync(0xffffffffu, e0, r & 31), b = __shfl_sync(0xffffffffu, e1, r & 31), rr = r < 32 ? a : b;
            const uint4* cp = reinterpret_cast<const uint4*>(P.c.cache.codes + (size_t)max(rr, 0) * (D / 2)) + u0;
            const uint16_t* sp = reinterpret_cast<const uint16_t*>(P.c.cache.scales + (size_t)max(rr, 0) * (D / 16)) + u0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool live = rr >= 0 && u0 + 4 * j < upr;
              code[j] = live ? cp[4 * j] : make_uint4(0, 0, 0, 0);
              sc[j] = live ? sp[4 * j] : 0;
            }
          }
          look_ahead(t + 1);
          if (!(ok = stage_free(st))) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t u = u0 + 4 * j;
            if (4 * j >= upr) break;
            if ((int)u >= upr) continue;
            const uint32_t at = dst + (u >> 1) * kChunkBytes + r * 128;
            const uint32_t word[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
            const float2 s = e4m3x2_values(sc[j]);
            const uint32_t s2[2] = {bf16x2(s.x, s.x), bf16x2(s.y, s.y)};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint4 d = dequant8(word[q], s2[q >> 1]);
              const uint32_t c = ((u & 1) * 4 + q) ^ (r & 7);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + c * 16), "r"(d.x), "r"(d.y), "r"(d.z),
                           "r"(d.w)
                           : "memory");
            }
          }
          hand_over(st);
        } else {
          const int e = __shfl_sync(0xffffffffu, e0, 0);
          const bool run = __all_sync(0xffffffffu, e0 >= 0 && e0 == e + lane && e1 == e + 32 + lane) != 0;
          if (!(ok = stage_free(st))) break;
          if (run) {
            // 64 consecutive rows: one tensor copy
            if (lane == 0) {
              if (w == 0) {
                mbar_arrive_expect_tx(&c_full[st], (uint32_t)stage_bytes);
                tma_load_3d_hint(sC + st * stage_bytes, &map_c, 0, e, 0, &c_full[st], policy);
              } else {
                mbar_arrive(&c_full[st]);
              }
            }
            look_ahead(t + 2);
            continue;
          }
#pragma unroll 1
          for (int i = 0; i < kGroups; ++i) {
            const int r = kTileRows * w + 8 * i + r8, ra = __shfl_sync(0xffffffffu, e0, r & 31),
                      rb = __shfl_sync(0xffffffffu, e1, r & 31), rr = r < 32 ? ra : rb;
            const uint32_t bytes = rr < 0 ? 0u : 16u;
            const uint8_t* src = base + (size_t)max(rr, 0) * (2 * D) + u0 * 16;
            const uint32_t lo = dst + r * 128 + ((u0 ^ (r & 7)) << 4), hi = lo ^ 64;
#pragma unroll 4
            for (int c = 0; c < chunks; ++c) {
              cp_async16(lo + c * kChunkBytes, src + c * 128, bytes);
              cp_async16(hi + c * kChunkBytes, src + c * 128 + 64, bytes);
            }
          }
          cp_commit();
          if (pending >= 0) {
            cp_wait<1>();
            hand_over(pending);
          }
          pending = (int)st;
          look_ahead(t + 2);
          if (nst == 2) flush();
        }
      }
    }
    if constexpr (!kFp4) {
      flush();
      // after an abort: the tensor copies in flight land (a stage's last use)
      if (*abort_flag && lane == 0 && w == 0)
        for (uint32_t i = k > nst ? k - nst : 0; i < k; ++i)
          if ((int)(i & 1) == grp) mbar_wait_bounded(&c_full[i & (nst - 1)], (i >> lst) & 1, 1000000);
    }
  } else if (warp == kMmaWarp) {
    // ---- scores: the whole warp runs the loop, one elected lane issues
    const bool leader = elect_one();
    const uint32_t idesc = idesc_bf16(64, kCols), c0 = smem_addr(sC);
    const uint64_t qd = sw128_desc(smem_addr(sQ), 16);
    uint32_t k = 0;
    bool ok = true;
    while (ok && next()) {
      ok = __all_sync(0xffffffffu, wait(q_full, seg - 1));
#pragma unroll 1
      for (int t = g.t0; ok && t < g.t1; ++t, ++k) {
        const uint32_t kk = __shfl_sync(0xffffffffu, k, 0), st = kk & (nst - 1), buf = kk & 1;
        // the buffer's scores of two tiles before have been read, and the rows have landed
        ok = (k < 2 || wait(&p_full[buf], (kk >> 1) - 1)) && wait(&c_full[st], kk >> lst);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint32_t d = tmem + oc + buf * kCols;
        uint64_t a = sw128_desc(c0 + st * stage_bytes, 16), b = qd;  // addresses in units of 16 bytes
#pragma unroll 1
        for (int x = 0; x < chunks; ++x, a += kChunkBytes / 16, b += kChunkBytes / 16)
          if (leader) {
#pragma unroll
            for (int y = 0; y < 4; ++y) mma_bf16(d, a + 2 * y, b + 2 * y, idesc, x | y ? 1u : 0u);
          }
        if (leader) {
          mma_commit(&s_full[buf]);
          if (t + 1 == g.t1) mma_commit(q_empty);
        }
        __syncwarp();
      }
    }
  } else if (warp == kValWarp) {
    // ---- values, likewise
    const bool leader = elect_one();
    const uint32_t idesc = idesc_bf16(128, kCols) | kTransposed, idesc64 = idesc_bf16(64, kCols) | kTransposed;
    const uint32_t c0 = smem_addr(sC), p0 = smem_addr(sP);
    uint32_t k = 0;
    bool ok = true;
    while (ok && next()) {
#pragma unroll 1
      for (int t = g.t0; ok && t < g.t1; ++t, ++k) {
        const uint32_t kk = __shfl_sync(0xffffffffu, k, 0), st = kk & (nst - 1), buf = kk & 1;
        if (!(ok = __all_sync(0xffffffffu, wait(&p_full[buf], kk >> 1)))) break;
        tc_fence_after();
        const bool begin = __shfl_sync(0xffffffffu, (int)(t == g.t0), 0);
        uint64_t a = sw128_desc(c0 + st * stage_bytes, kChunkBytes);
        const uint64_t b = sw128_desc(p0 + buf * kPBytes, kChunkBytes);
#pragma unroll 1
        for (int x = 0; x < chunks; x += 2, a += 2 * kChunkBytes / 16) {
          if (begin && seg > 1) {  // the item before has been read out of this block
            if (!(ok = __all_sync(0xffffffffu, wait(&o_empty[x >> 1], seg - 2)))) break;
            tc_fence_after();
          }
          if (leader) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              mma_bf16(tmem + (x >> 1) * kCols, a + 128 * y, b + 128 * y, x + 1 < chunks ? idesc : idesc64,
                       !begin || y ? 1u : 0u);
          }
        }
        if (!ok) break;
        if (leader) {
          mma_commit(&c_empty[st]);
          mma_commit(&pv_done[buf]);
        }
        __syncwarp();
      }
    }
  } else {
    // ---- softmax: a warp has 16 rows (its lane quarter's) of 32 queries (half `hq`)
    const int qt = warp & 3, hq = warp >> 2, c2 = 32 * hq + 2 * (lane & 3);  // columns c2 + 8 i + e
    const uint32_t lanes = (uint32_t)(32 * qt) << 16;
    const float sl = P.scale_log2;
    uint32_t k = 0;
    bool ok = true;
    for (;;) {
      if (!next()) {
        // the two barriers that a warp which has the segment comes to when its first tile has failed
        if (group_or(1, g.t1 < 0)) group_or(1, true);
        break;
      }
      float m[8], l[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = l[i] = 0.0f;
      const bool several = g.s.tlo != g.s.thi;  // tokens: their rows differ
      if (several) {  // (every warp of a half writes its 32 positions, the same ones: no barrier for them)
        const int f = 32 * hq + lane;
        colt[f] = min(g.s.thi, P.c.start + P.by_heads.of(g.s.f0 + f));
        __syncwarp();
      }
#pragma unroll 1
      for (int t = g.t0; t < g.t1; ++t, ++k) {
        ok = wait(&s_full[k & 1], k >> 1);
        // the weights buffer is free once the tile two before has been used
        if (ok && k >= 2) ok = wait(&pv_done[k & 1], (k >> 1) - 1);
        tc_fence_after();
        uint32_t raw[16];
        tmem_ld_half(tmem + oc + (k & 1) * kCols + 32 * hq + lanes, raw);
        tmem_ld_wait();
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(raw[i]);
        const int v0 = t * kTile, v1 = min(v0 + kTile, g.s.cnt), v = v0 + 16 * qt + (lane >> 2);
        bool renew = !ok || g.tiles == 1;
        uint32_t spoilt = 0;  // bits 0, 1: this thread's rows may hold a NaN or infinity that a token must not see
        if (several) {
          // rows that only some of the item's tokens see
          const int begin = max(v0, P.sinks);
          if ((v1 - 1 < P.sinks ? v1 - 1 : v1 - 1 + g.s.jump) > g.s.tlo ||
              (P.window && begin < v1 && begin + g.s.jump <= g.s.thi - P.window)) {
            int2 tc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) tc[i] = *reinterpret_cast<const int2*>(colt + 8 * i + c2);
            float odd = 0.0f;  // NaN if any score is not finite
#pragma unroll
            for (int i = 0; i < 16; ++i) odd = fmaf(x[i], 0.0f, odd);
            const bool rare = __any_sync(0xffffffffu, odd != 0.0f);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // a row is seen by the tokens of its position and the next `reach`
              const int vv = v + 8 * h, j = vv < P.sinks ? vv : vv + g.s.jump;
              const uint32_t reach = P.window && vv >= P.sinks ? P.window : 0x7fffffffu;
              if (rare) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  // (a token that sees such a row gets NaN from any other score)
                  const float y = x[4 * (i >> 1) + 2 * h + (i & 1)];
                  const bool sees = (uint32_t)((i & 1 ? tc[i >> 1].y : tc[i >> 1].x) - j) < reach;
                  if (sees ? y == -INFINITY : !(fabsf(y) < INFINITY)) spoilt |= 1u << h;
                }
                if (vv >= g.s.cnt) spoilt &= ~(1u << h);
              }
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if ((uint32_t)((i & 1 ? tc[i >> 1].y : tc[i >> 1].x) - j) >= reach) x[4 * (i >> 1) + 2 * h + (i & 1)] = -INFINITY;
            }
            renew = renew || spoilt;
          }
        }
        if (v0 + kTile > g.s.cnt) {  // rows past the last one
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (v >= g.s.cnt) x[4 * i] = x[4 * i + 1] = -INFINITY;
            if (v + 8 >= g.s.cnt) x[4 * i + 2] = x[4 * i + 3] = -INFINITY;
          }
        }
        // the largest step past a reference; on a first tile the largest score that is there and too low
        float past = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) past = fmaxf(past, fmaf(fmaxf(x[4 * i + e], x[4 * i + 2 + e]), sl, -m[2 * i + e]));
        renew = renew || past > kStep;
        if (t == g.t0 || (several && t == g.t0 + 1)) {  // (every token's first row is in the first two tiles)
          float low = INFINITY;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float y = fmaxf(x[4 * i + e], x[4 * i + 2 + e]) * sl;
              low = fminf(low, y > -INFINITY ? y : 0.0f);
            }
          renew = renew || low < kLow;
        }
        if (group_or(1, renew)) {
          if (group_or(1, !ok)) {
            ok = false;
            break;
          }
          if (several) {
            // a row that really holds a NaN or infinity is cleared: weight 0 times it is then 0.  For a token that
            // sees it, its score is NaN; -inf from a finite row is the weight 0.
            spoilt |= __shfl_xor_sync(0xffffffffu, spoilt, 1);
            spoilt |= __shfl_xor_sync(0xffffffffu, spoilt, 2);
            uint32_t cleared = 0;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              uint8_t* at = sC + (k & (nst - 1)) * stage_bytes + (16 * qt + (lane >> 2) + 8 * h) * 128 + (lane & 3) * 32;
              uint32_t bad = 0;
              if (spoilt >> h & 1)
#pragma unroll 1
                for (int c = 0; c < 8 * chunks; ++c) {
                  const uint32_t y = *reinterpret_cast<const volatile uint32_t*>(at + (c >> 3) * kChunkBytes + (c & 7) * 4);
                  bad |= (y & 0x7F80u) == 0x7F80u || (y & 0x7F800000u) == 0x7F800000u;
                }
              bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
              bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
              group_sync(1);  // (the other half's warp may look at the same row)
              if (bad)
#pragma unroll 1
                for (int c = 0; c < 8 * chunks; ++c)
                  *reinterpret_cast<volatile uint32_t*>(at + (c >> 3) * kChunkBytes + (c & 7) * 4) = 0u;
              cleared |= bad << h;
            }
            if (cleared) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int vv = v + 8 * h, j = vv < P.sinks ? vv : vv + g.s.jump;
                const uint32_t reach = P.window && vv >= P.sinks ? P.window : 0x7fffffffu;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if ((cleared >> h & 1) && (uint32_t)(colt[8 * (i >> 1) + c2 + (i & 1)] - j) < reach)
                    x[4 * (i >> 1) + 2 * h + (i & 1)] = __int_as_float(0x7fffffff);
              }
            }
          }
          // the queries' maxima over the tile, by way of the weights buffer (rows of 64): this thread's
          // two rows, then a query a thread over the 32 pairs of rows
          float* col = reinterpret_cast<float*>(sP + (k & 1) * kPBytes);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float2*>(col + (8 * qt + (lane >> 2)) * 64 + 8 * i + c2) =
                make_float2(fmaxf(x[4 * i], x[4 * i + 2]), fmaxf(x[4 * i + 1], x[4 * i + 3]));
          if (lane < 4 && qt == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(red + 8 * i + c2) = make_float2(m[2 * i], m[2 * i + 1]);
          }
          group_sync(1);
          if (threadIdx.x < kCols) {
            float y = kFloor;
#pragma unroll 4
            for (int i = 0; i < 32; ++i) y = fmaxf(y, col[i * 64 + threadIdx.x]);
            // only the queries that need it: what a query gives does not depend on the others'
            bool before = t > g.t0;  // it has seen a row of the segment
            if (before && several) {
              const int tt = colt[threadIdx.x], begin = g.t0 * kTile;
              const int v = begin < P.sinks ? begin : max(begin, P.window ? tt - P.window + 1 - g.s.jump : 0);
              before = v < v0 && (v < P.sinks ? v : v + g.s.jump) <= tt;
            }
            const float m0 = red[threadIdx.x], top = fabsf(y * sl) < kHuge ? y * sl : __int_as_float(0x7fffffff);
            const float m1 = y * sl - m0 > kStep || (!before && y > kFloor && (y * sl < kLow || g.tiles == 1)) ? top : m0;
            red[threadIdx.x] = m1;
            red[64 + threadIdx.x] = before ? ex2(m0 - m1) : 1.0f;
          }
          group_sync(1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 y = *reinterpret_cast<const float2*>(red + 8 * i + c2),
                         z = *reinterpret_cast<const float2*>(red + 64 + 8 * i + c2);
            m[2 * i] = y.x, m[2 * i + 1] = y.y;
            l[2 * i] *= z.x, l[2 * i + 1] *= z.y;
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
              const uint32_t at = tmem + (x2 >> 1) * kCols + 32 * hq + lanes + ((uint32_t)(16 * (x2 & 1)) << 16);
              uint32_t o[16];
              tmem_ld_half(at, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 z = *reinterpret_cast<const float2*>(red + 64 + 8 * i + c2);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  o[4 * i + 2 * h] = __float_as_uint(__uint_as_float(o[4 * i + 2 * h]) * z.x);
                  o[4 * i + 2 * h + 1] = __float_as_uint(__uint_as_float(o[4 * i + 2 * h + 1]) * z.y);
                }
              }
              tmem_st_half(at, o);
            }
          }
          group_sync(1);  // `red` has been read
        }
        // weights [row][64 queries] as 128-byte swizzled rows; matrices of a store: rows 0-7 and 8-15 of
        // two groups of 8 queries
        const uint32_t at = smem_addr(sP) + (k & 1) * kPBytes + (16 * qt + (lane & 15)) * 128;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
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
          stmatrix4<false>(at + (((4 * hq + i + (lane >> 4)) ^ (lane & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
        }
        fence_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[k & 1]);
      }
      if (!ok) break;
      // the segment's end: sums over rows, four lanes' of a warp left to the epilogue
#pragma unroll
      for (int i = 0; i < 8; ++i) l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
      if (seg > 1) {
        ok = wait(l_empty, seg - 2);
        if (group_or(1, !ok)) {
          ok = false;
          break;
        }
      }
      if (lane < 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float2*>(fin + (4 * qt + (lane >> 2)) * 64 + 8 * i + c2) = make_float2(l[2 * i], l[2 * i + 1]);
      } else if (qt == 0 && lane < 20) {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(fin + 1024 + 8 * i + c2) = make_float2(m[2 * i], m[2 * i + 1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(l_full);
    }
  }

  // ---- leave: after an abort, let the products already issued complete
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) atomicOr(P.flag, 4);
    if ((warp == kMmaWarp || warp == kValWarp) && elect_one()) {  // the lanes that issued them
      mma_commit(mma_done);
      mbar_wait_bounded(mma_done, 0);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, tmem_cols);
}

// ---- pieces of split items joined.
//   M = max m_p;  out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p
// A thread takes four values (two queries, features d and d + 8) of every kGroups-th piece, kReps times
// 16 features on; the groups' results are merged like pieces, in order: nothing depends on timing.
// Few items have many pieces each (16 groups, the item over D / 4 CTAs, read in one pass with a running
// maximum: 1 x 32768 entries 22.4 us; maxima first, with spilled registers, 23.2, 4 x 8192 28.5 and 32.2),
// many items a few (128 sequences of up to 2048 entries: 8.5 us for 36 MB of pieces, which lie in L2).
template <int kLanes, int kGroups, int kReps>
__global__ void __launch_bounds__(kLanes * kGroups, 1024 / (kLanes * kGroups)) attention_join_kernel(const __grid_constant__ AttnParams P) {
  __shared__ float4 acc[kGroups > 1 ? kGroups : 1][kLanes];
  __shared__ float4 ml[kGroups > 1 ? kGroups : 1][kLanes];
  __shared__ __align__(16) uint16_t tile[kLanes / 4][16];  // queries x 16 features
  griddep_wait();
  int2 rec = P.record[blockIdx.x];
  // (after a wait that ran out a record may be an earlier call's: no index comes from one that does not fit)
  if (kGroups == 1 ? rec.x >= P.items || rec.y > P.ctas - (int)blockIdx.x : rec.x < 0 || rec.y > P.ctas - rec.x) rec.x = -1;
  const int j0 = blockIdx.y * kLanes * kReps + threadIdx.x;  // of the piece's 16 D quads of values
  const int lane = threadIdx.x & 31, grp = threadIdx.y, qt = 8 * (threadIdx.x >> 5) + 2 * (lane & 3);
  const int q0 = 8 * ((j0 >> 5) & 7) - 8 * (int)(threadIdx.x >> 5), q = q0 + qt;  // the CTA's, the thread's first query
  const int most = (int)gridDim.x;  // (with one group of threads a CTA's records: the last CTA has no next)
  auto stats = [&](int slot) { return *reinterpret_cast<const float4*>(P.part_ml + slot * kCols + q); };
  auto quad = [&](int slot, int r) {
    return j0 + r * kLanes < 16 * P.D ? P.part[(size_t)slot * (kCols * P.D / 4) + j0 + r * kLanes] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  float4 y = make_float4(kFloor, 0.0f, kFloor, 0.0f);  // maximum and sum of both queries
  float4 a[kReps];
  Seen s;
  if constexpr (kGroups == 1) {
    // The first two pieces (a split item has them) are asked for before the record is known: one trip to
    // L2 instead of three.
    const int s0 = 2 * blockIdx.x + 1, s1 = 2 * min((int)blockIdx.x + 1, most - 1);
    const float4 z0 = stats(s0), z1 = stats(s1);
    float4 o0[kReps], o1[kReps];
#pragma unroll
    for (int r = 0; r < kReps; ++r) o0[r] = quad(s0, r), o1[r] = quad(s1, r);
    if (rec.x < 0) return;
    s = seen_rows(P, rec.x);
    y.x = fmaxf(z0.x, z1.x), y.z = fmaxf(z0.z, z1.z);
#pragma unroll 1
    for (int p = 2; p < rec.y; ++p) {
      const float4 z = stats(2 * (blockIdx.x + p));
      y.x = fmaxf(y.x, z.x), y.z = fmaxf(y.z, z.z);
    }
    const float f0 = ex2(z0.x - y.x), f1 = ex2(z0.z - y.z), g0 = ex2(z1.x - y.x), g1 = ex2(z1.z - y.z);
    y.y = fmaf(z1.y, g0, z0.y * f0), y.w = fmaf(z1.w, g1, z0.w * f1);
#pragma unroll
    for (int r = 0; r < kReps; ++r)
      a[r] = make_float4(fmaf(o1[r].x, g0, o0[r].x * f0), fmaf(o1[r].y, g1, o0[r].y * f1), fmaf(o1[r].z, g0, o0[r].z * f0),
                         fmaf(o1[r].w, g1, o0[r].w * f1));
#pragma unroll 1
    for (int p = 2; p < rec.y; ++p) {
      const int slot = 2 * (blockIdx.x + p);
      const float4 z = stats(slot);
      const float h0 = ex2(z.x - y.x), h1 = ex2(z.z - y.z);
      y.y = fmaf(z.y, h0, y.y), y.w = fmaf(z.w, h1, y.w);
#pragma unroll
      for (int r = 0; r < kReps; ++r) {
        const float4 o = quad(slot, r);
        a[r].x = fmaf(o.x, h0, a[r].x), a[r].y = fmaf(o.y, h1, a[r].y);
        a[r].z = fmaf(o.z, h0, a[r].z), a[r].w = fmaf(o.w, h1, a[r].w);
      }
    }
  } else {
    s = seen_rows(P, blockIdx.x);
    if (rec.x < 0 || s.cols == 0) return;
    auto slot = [&](int p) { return 2 * (rec.x + p) + (p == 0 ? 1 : 0); };
    a[0] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int p = grp; p < rec.y; p += 2 * kGroups) {  // two pieces at once; the sums are scaled as the maximum grows
      float4 z[2], o[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int pp = p + i * kGroups;
        const bool there = pp < rec.y;
        z[i] = there ? stats(slot(pp)) : make_float4(kFloor, 0.0f, kFloor, 0.0f);
        o[i] = there ? quad(slot(pp), 0) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      float2 top = make_float2(y.x, y.z);
#pragma unroll
      for (int i = 0; i < 2; ++i) top.x = fmaxf(top.x, z[i].x), top.y = fmaxf(top.y, z[i].z);
      const float k0 = ex2(y.x - top.x), k1 = ex2(y.z - top.y);
      y = make_float4(top.x, y.y * k0, top.y, y.w * k1);
      a[0] = make_float4(a[0].x * k0, a[0].y * k1, a[0].z * k0, a[0].w * k1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f0 = ex2(z[i].x - top.x), f1 = ex2(z[i].z - top.y);
        y.y = fmaf(z[i].y, f0, y.y), y.w = fmaf(z[i].w, f1, y.w);
        a[0].x = fmaf(o[i].x, f0, a[0].x), a[0].y = fmaf(o[i].y, f1, a[0].y);
        a[0].z = fmaf(o[i].z, f0, a[0].z), a[0].w = fmaf(o[i].w, f1, a[0].w);
      }
    }
  }
  if constexpr (kGroups > 1) {
    acc[grp][threadIdx.x] = a[0], ml[grp][threadIdx.x] = y;
    __syncthreads();
    if (grp == 0) {
      float2 top = make_float2(kFloor, kFloor);
#pragma unroll 4
      for (int i = 0; i < kGroups; ++i)
        top.x = fmaxf(top.x, ml[i][threadIdx.x].x), top.y = fmaxf(top.y, ml[i][threadIdx.x].z);
      y = make_float4(top.x, 0.0f, top.y, 0.0f), a[0] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int i = 0; i < kGroups; ++i) {
        const float4 z = ml[i][threadIdx.x], o = acc[i][threadIdx.x];
        const float f0 = ex2(z.x - top.x), f1 = ex2(z.z - top.y);
        y.y = fmaf(z.y, f0, y.y), y.w = fmaf(z.w, f1, y.w);
        a[0].x = fmaf(o.x, f0, a[0].x), a[0].y = fmaf(o.y, f1, a[0].y);
        a[0].z = fmaf(o.z, f0, a[0].z), a[0].w = fmaf(o.w, f1, a[0].w);
      }
    }
  }
  const long long orow = (long long)s.b * P.c.N * P.H + s.f0;
  const float i0 = y.y == 0.0f ? 0.0f : 1.0f / y.y, i1 = y.w == 0.0f ? 0.0f : 1.0f / y.w;
  if (grp == 0 && P.c.lse && j0 - threadIdx.x < 256 && lane < 4) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float t = e ? y.w : y.y;
      if (q + e < s.cols && in_rows(P, orow + q + e))
        P.c.lse[orow + q + e] = t == 0.0f ? -INFINITY : ((e ? y.z : y.x) + log2f(t)) * 0.693147180559945f;
    }
  }
#pragma unroll 1
  for (int r = 0; r < kReps; ++r) {
    const int at = (j0 + r * kLanes) >> 8, x = at >> 2, w = at & 3;  // the fragment load's half block and warp
    if (x >= P.D / 64) break;
    if (grp == 0) {
      float4 v = a[0];
#pragma unroll
      for (int i = 1; i < kReps; ++i)
        if (i == r) v = a[i];
      tile[qt][lane >> 2] = bf16_bits(v.x * i0), tile[qt + 1][lane >> 2] = bf16_bits(v.y * i1);
      tile[qt][8 + (lane >> 2)] = bf16_bits(v.z * i0), tile[qt + 1][8 + (lane >> 2)] = bf16_bits(v.w * i1);
    }
    __syncthreads();
    // features 16 w of the last 64, else 32 w + 16 (x % 2) of 128
    const int d = (x | 1) < P.D / 64 ? (x >> 1) * 128 + 32 * w + 16 * (x & 1) : x * 64 + 16 * w;
    const int t = threadIdx.x >> 1, u = threadIdx.x & 1;
    if (grp == 0 && t < kLanes / 4 && q0 + t < s.cols && in_rows(P, orow + q0 + t))
      *reinterpret_cast<uint4*>(P.c.out + (orow + q0 + t) * P.D + d + 8 * u) = *reinterpret_cast<const uint4*>(&tile[t][8 * u]);
    __syncthreads();
  }
}

// ---- host side
// Stages: as many tiles (a power of two, at most 8) as the shared memory takes.
struct Shape {
  int stages, smem;
};
Shape attn_shape(int D) {
  Shape s;
  const int chunk = D / 64 * kChunkBytes, rest = 2 * kPBytes + 8 * kStageOut + kAuxBytes + 1024;
  s.stages = 8;
  while (s.stages > 2 && (s.stages + 1) * chunk + rest > 227 * 1024) s.stages /= 2;
  s.smem = (s.stages + 1) * chunk + rest;
  return s;
}

}  // namespace

size_t attention_workspace_bytes(int head_dim) {
  return 2 * (size_t)current_sm_count() * (kCols * (head_dim * sizeof(float) + sizeof(float2)) + sizeof(int2)) + 64;
}

// Few items have many pieces each, and a join of their own (1 x 32768 entries 22.6 us, 4 x 8192 28 us
// against 36 us with the other; 9 x 2000 25 us against 35 us with this one).
static bool few_items(long long items, int sms) { return items * 32 <= sms; }

// The units (see units_of) that a call whose items may be cut can have at most; 0 where none is cut.
long long attention_units(const csa_attention* a, const AttnCall& call) {
  // the longest range of rows that this call can have decides whether items may be cut
  const long long items = call.B * (((long long)call.N * a->heads + kCols - 1) / kCols);
  long long most = call.paged ? (long long)call.max_pages * call.cache.page_size : (long long)call.start + call.N;
  const long long window = (long long)a->window + a->sinks + (kCols - 1) / a->heads + 1;
  if (a->window && most > window) most = window;
  // (a share is two units at least: shorter items than these are never cut; nor is a prompt with several
  // items a CTA, where drawing them, the longest first, balances as well: 700 tokens of 64 heads over
  // their own rows take 57 us drawn and 81 us cut, 200 tokens behind 2000 others 111 us drawn and 88 us cut)
  if (most <= ((few_items(items, a->sms) ? kCutFew : kCutMany) + 1) * (long long)kTile || (!call.paged && items >= 4LL * a->sms)) return 0;
  return items * ((most + kTile - 1) / kTile + 1);
}

cudaError_t launch_attention(csa_attention* a, const AttnCall& call, cudaStream_t s) {
  auto encode = get_encode();
  if (!encode) return cudaErrorNotSupported;
  const bool fp4 = call.paged && !call.cache.latent;
  const Shape sh = attn_shape(a->D);
  static std::atomic<unsigned long long> attr{0};
  cudaError_t e = once_per_device(attr, [] {
    const int most = 227 * 1024;
    cudaError_t r = cudaFuncSetAttribute(attention_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(attention_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return r;
  });
  if (e != cudaSuccess) return e;
  const int slots = 2 * a->sms;
  AttnParams P{};
  P.c = call;
  P.H = a->heads;
  P.D = a->D;
  // positions are below 2^30: a longer window is none, more sinks are all
  P.window = a->window < (1 << 30) ? a->window : 0;
  P.sinks = P.window == 0 ? 0 : a->sinks < (1 << 30) - 128 ? a->sinks : (1 << 30) - 128;
  P.per = (int)(((long long)call.N * a->heads + kCols - 1) / kCols);
  P.items = call.B * P.per;
  P.scale_log2 = (float)(a->scale * 1.4426950408889634);
  P.flag = a->dev_flag;
  P.part = (float4*)a->workspace;
  P.part_ml = (float2*)((float*)a->workspace + (size_t)slots * kCols * a->D);
  P.record = (int2*)(P.part_ml + (size_t)slots * kCols);
  P.ticket = (int*)(P.record + slots);
  while ((1 << P.log_stages) < sh.stages) ++P.log_stages;
  P.by_per = Divisor(P.per);
  P.by_heads = Divisor(P.H);
  P.by_page = Divisor(call.paged ? call.cache.page_size : 1);
#ifdef CSA_DEBUG_BOUNDS
  const char* shorter = getenv("CSA_TEST_SHORT_EXTENTS");  // the test of the checks: "rows" or "slots"
  P.rows = (long long)call.B * call.N * a->heads - (shorter && *shorter == 'r' ? 1 : 0);
  P.slots = shorter && *shorter == 's' ? 1 : slots;
  P.test_stall = getenv("CSA_TEST_STALL_LAST_STAGE") != nullptr;
  P.test_late = getenv("CSA_TEST_LATE_SEGMENT") != nullptr;
  P.wait_ns = P.test_stall || P.test_late ? 200000000ull : kWaitNs;
#endif
  const long long units = attention_units(a, call);
  P.split = units > 0;
  if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
  const long long shares = P.split ? units : P.items;
  const int grid = (int)(shares < a->sms ? shares : a->sms);
  P.ctas = grid;
  P.few = few_items(P.items, a->sms);
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
  CUtensorMap mc = mq;  // not used for codes
  if (!fp4) {
    // 64 consecutive rows, chunk by chunk of 64 features
    cuuint64_t dims[3] = {64, call.paged ? (cuuint64_t)call.cache.pages * call.cache.page_size
                                         : (cuuint64_t)call.B * call.kv_rows, (cuuint64_t)a->D / 64};
    cuuint64_t strides[2] = {(cuuint64_t)a->D * 2, 128};
    cuuint32_t box[3] = {64, kTile, (cuuint32_t)a->D / 64};
    cuuint32_t es[3] = {1, 1, 1};
    if (encode(&mc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, (void*)(call.paged ? call.cache.latent : call.kv), dims, strides,
               box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  a->launches += 1;
  e = launch_early(fp4 ? attention_kernel<true> : attention_kernel<false>, dim3(grid), dim3(kAttnThreads), sh.smem, s, mq, mc, P);
  if (e != cudaSuccess || !P.split) return e;
  a->launches += 1;
  return P.few ? launch_early(attention_join_kernel<64, 16, 1>, dim3(P.items, a->D / 4), dim3(64, 16), 0, s, P)
               : launch_early(attention_join_kernel<256, 1, 4>, dim3(grid, a->D / 64), dim3(256, 1), 0, s, P);
}

}  // namespace csa
