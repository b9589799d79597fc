// Attention over one shared key/value row per position (see include/csa.h): a prompt's tokens over
// their own rows with a window and sinks, or one new token a sequence over a paged cache.
//
// An item is one token's up to 64 query heads.  Its visible rows c_0, c_1, .. (the sinks, then the
// window; hidden rows are never loaded) are taken 64 at a time:
//
//   S^T = C Q^T   [64 rows x 64 heads], features as the K dimension
//   P   = exp2(S^T * scale - m)         m: the running maximum of each head
//   O^T = O^T + C^T P                   [D features x 64 heads], rows as the K dimension
//
// Transposed, both products keep the rows' tile as the A operand, once K-major (64 x D) and once
// M-major (D x 64): one copy in shared memory serves as key and as value, which is what a shared
// row offers, and O^T takes D / 128 * 64 columns of tensor memory (256 of 512 at D = 512) where O
// with heads as rows would take all of it for half a filled tile.  The scores come back with a
// row (key) per TMEM lane in the matrix-fragment shape, where the maximum over rows is three
// shuffles.  That maximum is only renewed (and O^T, l scaled) when a score passes it by 2^8:
// the weights then stay below 2^8 in bf16, whose relative precision does not depend on it.
//
// Work is cut by tiles: the call's tiles, in item order, are divided evenly over the CTAs, so ragged
// lengths and few long sequences fill the GPU alike; an item cut by a CTA boundary leaves partial
// (m, l, O) pieces in the workspace, which a second kernel joins.  Where no item is longer than
// kJoinTiles tiles the boundaries are moved to item starts instead: the imbalance costs less than
// pieces and their join.
#include <atomic>

#include "layer_ops.h"
#include "tc_common.cuh"

namespace csa {
namespace {

using namespace tcx;

constexpr int kTile = 64;                      // rows of a tile
constexpr int kHeads = 64;                     // heads of an item
constexpr int kChunkBytes = 8192;              // 64 rows x 64 features bf16: one column of swizzled atoms
constexpr int kPBytes = kTile * kHeads * 2;    // one weights buffer
constexpr int kSoftWarps = 4, kSoftThreads = 128;
constexpr int kMmaWarp = 4, kQWarp = 5, kProdWarp = 6;
constexpr int kJoinTiles = 6;   // items longer than this are split
constexpr int kMinTiles = 4;    // a split call gives a CTA at least this many tiles
constexpr float kStep = 8.0f;   // base-2 steps a score may pass the running maximum by
constexpr float kFloor = -1e38f;  // running maximum while no score was seen
constexpr int kSpins = 1 << 16;   // polls of two barriers before the MMA warp waits for one of them
constexpr int kAuxBytes = 3072;   // barriers, flags, per-warp maxima and sums

struct AttnParams {
  AttnCall c;
  int H, D, window, sinks, hblocks;
  long long toks;   // tokens: B * N
  float scale_log2;  // scale * log2(e): scores in base-2 exponents
  int* flag;
  float* part;       // pieces: [2 * grid][64][D] f32
  float2* part_ml;   // (maximum, sum) of each piece and head [2 * grid][64]
  int2* record;      // per CTA: (item, pieces) of an item whose first piece it made, or (-1, 0)
  int stages;
  uint32_t unit_magic;  // ceil(2^32 / (D / 32)): units of a row of codes
  bool split;        // items may be cut (the join kernel follows)
};

// ---- the rows a token sees
struct Seen {
  int b;          // sequence
  long long cnt;  // visible rows; row v of them is position v, or v + jump from the sinks on
  long long jump;
  bool skip;      // padding: no output
};

__device__ __forceinline__ Seen seen_rows(const AttnParams& P, long long tok) {
  Seen s;
  long long t;
  s.skip = false;
  if (P.c.paged) {
    s.b = (int)tok;
    const long long top = (long long)P.c.max_pages * P.c.cache.page_size, n = __ldg(P.c.lens + tok);
    t = (n < 0 ? 0 : n > top ? top : n) - 1;
  } else {
    const uint32_t b = (uint32_t)tok / (uint32_t)P.c.N, i = (uint32_t)tok - b * (uint32_t)P.c.N;
    s.b = (int)b;
    s.skip = P.c.lens && (int)i >= __ldg(P.c.lens + b);
    t = (long long)P.c.start + i;
  }
  const long long most = (long long)P.window + P.sinks;
  const bool all = P.window == 0 || t + 1 <= most;
  s.cnt = all ? t + 1 : most;
  s.jump = all ? 0 : t + 1 - most;
  return s;
}
__device__ __forceinline__ long long tiles_of(const Seen& s) {
  return s.skip ? 0 : s.cnt <= kTile ? 1 : (s.cnt + kTile - 1) / kTile;  // an empty item still has its output
}

// A CTA's work: `left` tiles from tile `tile` of item `item` on.  next() gives the next segment: a
// run of tiles of one item.
struct Segment {
  long long tok, t0, t1, tiles;
  int hb;
  Seen s;
};
struct Walk {
  long long tok, tile, left;
  int hb;
  __device__ __forceinline__ bool next(const AttnParams& P, Segment& g) {
    if (left <= 0) return false;
    for (;; ++tok, tile = 0, hb = 0) {  // over padding
      if (tok >= P.toks) return false;  // only if the lengths changed under the kernel
      g.s = seen_rows(P, tok);
      g.tiles = tiles_of(g.s);
      if (tile < g.tiles) break;
    }
    g.tok = tok, g.hb = hb, g.t0 = tile;
    g.t1 = min(g.tiles, tile + left);
    left -= g.t1 - tile;
    tile = 0;
    if (++hb == P.hblocks) hb = 0, ++tok;
    return true;
  }
};

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
// The softmax warps' barrier; or_ gives every thread whether any passed true.
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory"); }
__device__ __forceinline__ bool soft_or(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "n"(kSoftThreads)
      : "memory");
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

// ---- the kernel: warps 0-3 softmax and epilogue (TMEM lane quarter = warp), 4 MMA issue, 5 the
// queries' copies, 6.. the rows' copies, in two groups that take alternate tiles (so that one
// group's tile can be in flight while the other waits for its stage)
template <bool kFp4>
constexpr int prod_warps() {
  return kFp4 ? 8 : 4;
}
template <bool kFp4>
constexpr int attn_threads() {
  return (kProdWarp + prod_warps<kFp4>()) * 32;
}

template <bool kFp4, int kCtas>
__global__ void __launch_bounds__(attn_threads<kFp4>(), kCtas)
    attention_kernel(const __grid_constant__ CUtensorMap map_q, const AttnParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int D = P.D, chunks = D / 64, nst = P.stages;
  const int stage_bytes = chunks * kChunkBytes;
  uint8_t* sQ = smem;
  uint8_t* sC = sQ + chunks * kChunkBytes;
  uint8_t* sP = sC + nst * stage_bytes;  // two weights buffers; the epilogue's staging
  uint8_t* aux = sP + 2 * kPBytes;
  uint64_t* c_full = (uint64_t*)aux;  // [8] a stage's rows have landed
  uint64_t* c_empty = c_full + 8;     // [8] a stage's products are done
  uint64_t* s_full = c_empty + 8;     // [2] scores ready
  uint64_t* p_full = s_full + 2;      // [2] weights written, scores read
  uint64_t* pv_done = p_full + 2;     // [2] second product done: weights buffer free, O^T complete to it
  uint64_t* q_full = pv_done + 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* o_empty = q_empty + 1;    // O^T has been read
  uint64_t* mma_done = o_empty + 1;   // clean-up after an abort
  uint32_t* tmem_slot = (uint32_t*)(mma_done + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  int* q_loads = (int*)(tmem_slot + 2);
  long long* work = (long long*)(aux + 320);  // first token, first tile, tiles, first head block, tile index, total
  float* red = (float*)(aux + 512);           // [2][4][64] per-warp maxima, sums; the scan's sums before
  static_assert(512 + 2 * 4 * 64 * 4 <= kAuxBytes, "aux region");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kThreads = attn_threads<kFp4>();
  constexpr int kGroupWarps = prod_warps<kFp4>() / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      mbar_init(&c_full[s], kGroupWarps);
      mbar_init(&c_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSoftWarps);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_empty, kSoftWarps);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    *q_loads = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_map(&map_q);
  }
  const uint32_t oc = (uint32_t)((D + 127) / 128) * kHeads;  // columns of O^T; two score buffers follow
  const uint32_t tmem_cols = oc + 2 * kHeads <= 256 ? 256 : 512;
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, tmem_cols);
  griddep_launch_dependents();

  // ---- the CTA's share of the call's tiles: every CTA adds up the tokens' tiles (threads over
  // contiguous tokens) and finds its own first one
  {
    const long long per = (P.toks + kThreads - 1) / kThreads, lo = min(P.toks, per * threadIdx.x),
                    hi = min(P.toks, lo + per);
    long long sum = 0, top = 0;
    for (long long i = lo; i < hi; ++i) {
      const long long n = tiles_of(seen_rows(P, i));
      sum += n;
      top = max(top, n);
    }
    if (blockIdx.x == 0 && P.c.lens) {  // lengths out of range are taken as the nearest end
      const long long most = P.c.paged ? (long long)P.c.max_pages * P.c.cache.page_size : P.c.N;
      for (int b = threadIdx.x; b < P.c.B; b += kThreads) {
        const long long n = P.c.lens[b];
        if (n < 0 || n > most) atomicOr(P.flag, 1);
      }
    }
    long long pre = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += y;
      top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    long long* ws = (long long*)red;  // [warp] sums, then [warp] maxima
    if (lane == 31) ws[warp] = pre, ws[16 + warp] = top;
    if (threadIdx.x == 0) work[0] = P.toks, work[1] = 0, work[2] = 0, work[3] = 0, work[4] = 0;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += ws[w];
      total += ws[w];
      top = max(top, ws[16 + w]);
    }
    pre += before - sum;  // tokens' tiles before this thread's
    const int hbs = P.hblocks;
    total *= hbs;
    const bool cut = P.split && top > kJoinTiles;
    const long long ctas = cut ? min((long long)gridDim.x, max(1LL, total / kMinTiles)) : gridDim.x;
    const long long i = blockIdx.x;
    const long long a = i < ctas ? total * i / ctas : total, e = i < ctas ? total * (i + 1) / ctas : total;
    // the boundary x: the item it falls in and, without cutting, the start of the first item from it on
    auto locate = [&](long long x, bool first) {
      if (sum == 0 || x < pre * hbs || x >= (pre + sum) * hbs) return;
      long long at = pre * hbs;
      for (long long tok = lo; tok < hi; ++tok) {
        const long long n = tiles_of(seen_rows(P, tok));
        if (n == 0 || x >= at + n * hbs) {
          at += n * hbs;
          continue;
        }
        const int hb = (int)((x - at) / n);
        long long start = at + hb * n, tile = x - start;
        long long t = tok, h = hb;
        if (!cut && tile > 0) {
          start += n, tile = 0;
          if (++h == hbs) h = 0, ++t;
        }
        if (first)
          work[0] = t, work[1] = tile, work[3] = h, work[4] = start + tile;
        else
          work[5] = start + tile;
        return;
      }
    };
    if (threadIdx.x == 0) work[4] = work[5] = total;
    __syncthreads();
    locate(a, true);
    locate(e, false);
    __syncthreads();
    if (threadIdx.x == 0) {
      work[2] = work[5] - work[4];
      work[6] = total;
      work[7] = ctas;
      if (P.split) P.record[blockIdx.x] = make_int2(-1, 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk walk{work[0], work[1], work[2], (int)work[3]};
  Segment g;

  if (warp >= kProdWarp) {
    // ---- rows: warp w of a group takes rows kRows * w .. of its group's tiles
    constexpr int kRows = kTile / kGroupWarps;
    const int grp = (warp - kProdWarp) / kGroupWarps, w = (warp - kProdWarp) % kGroupWarps;
    const uint16_t* base = P.c.paged ? P.c.cache.latent : P.c.kv;
    uint32_t k = 0;
    int pending = -1;  // a stage whose copies were issued and not yet handed over
    bool ok = true;
    auto hand_over = [&](int st) {  // this thread's copies have landed
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c_full[st]);
    };
    while (ok && walk.next(P, g)) {
      for (long long t = g.t0; t < g.t1; ++t, ++k) {
        if ((int)(k & 1) != grp) continue;
        const int st = (int)(k % (uint32_t)nst);
        // lane r of the warp resolves its row r: the entry's row in the cache, or -1
        long long row = -1;
        const long long v = t * kTile + kRows * w + (lane % kRows);
        if (v < g.s.cnt) {
          const long long j = v < P.sinks ? v : v + g.s.jump;
          if (P.c.paged) {
            const uint32_t ps = (uint32_t)P.c.cache.page_size, pg = (uint32_t)j / ps;
            const int page = __ldg(P.c.page_table + (long long)g.s.b * P.c.max_pages + pg);
            if (page >= 0 && page < P.c.cache.pages)
              row = (long long)page * ps + ((uint32_t)j - pg * ps);
            else
              atomicOr(P.flag, 2);
          } else {
            row = (long long)g.s.b * P.c.kv_rows + j;
          }
        }
        const uint32_t dst = smem_addr(sC) + st * stage_bytes;
        if constexpr (kFp4) {
          // units of 32 codes and two scales; loaded before the stage is free
          uint4 code[8];
          uint32_t sc[8];
          const int upr = D / 32;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i >= chunks) break;
            const uint32_t x = lane + 32 * i, r = __umulhi(x, P.unit_magic), u = x - r * upr;
            const long long rr = __shfl_sync(0xffffffffu, row, (int)r);
            code[i] = make_uint4(0, 0, 0, 0);
            sc[i] = 0;
            if (rr >= 0) {
              code[i] = __ldg(reinterpret_cast<const uint4*>(P.c.cache.codes + rr * (D / 2)) + u);
              sc[i] = __ldg(reinterpret_cast<const uint16_t*>(P.c.cache.scales + rr * (D / 16)) + u);
            }
          }
          if (k >= (uint32_t)nst && !mbar_wait(&c_empty[st], ((k / nst) & 1) ^ 1, abort_flag)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i >= chunks) break;
            const uint32_t x = lane + 32 * i, rw = __umulhi(x, P.unit_magic), u = x - rw * upr, r = kRows * w + rw;
            const uint32_t at = dst + (u >> 1) * kChunkBytes + r * 128;
            const uint32_t word[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
            uint32_t s2[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float s = e4m3_value((sc[i] >> (8 * h)) & 255u);
              s2[h] = bf16x2(s, s);
            }
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
          if (k >= (uint32_t)nst) {
            const uint32_t par = ((k / nst) & 1) ^ 1;
            if (pending >= 0 && !mbar_test(&c_empty[st], par)) {
              cp_wait<0>();
              hand_over(pending);
              pending = -1;
            }
            if (!mbar_wait(&c_empty[st], par, abort_flag)) {
              ok = false;
              break;
            }
          }
          // 16-byte units of a row over the lanes (two or four narrow rows at a time)
          const int units = D / 8, lpr = min(32, units), rpi = units <= 16 ? 32 / units : 1;
          const int sub = rpi > 1 ? lane / lpr : 0, u0 = rpi > 1 ? lane % lpr : lane;
          for (int r0 = 0; r0 < kRows; r0 += rpi) {
            const int rw = r0 + sub, r = kRows * w + rw;
            const long long rr = __shfl_sync(0xffffffffu, row, rw);
            const uint8_t* src = (const uint8_t*)(base + (rr < 0 ? 0 : rr) * D);
            for (int u = u0; u < units; u += 32)
              cp_async16(dst + (u >> 3) * kChunkBytes + r * 128 + (((u & 7) ^ (r & 7)) << 4), src + u * 16,
                         rr < 0 ? 0u : 16u);
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
  } else if (warp == kQWarp) {
    // ---- queries: 64 rows of [tokens * H][D] from the item's first head (rows past its heads are
    // other tokens' or zeros: columns that nothing reads)
    if (lane == 0) {
      int n = 0;
      while (walk.next(P, g)) {
        if (n > 0 && !mbar_wait(q_empty, (n - 1) & 1, abort_flag)) break;
        mbar_arrive_expect_tx(q_full, chunks * kChunkBytes);
        const int row = (int)(g.tok * P.H + g.hb * kHeads);
        for (int c = 0; c < chunks; ++c) tma_load_2d(sQ + c * kChunkBytes, &map_q, c * 64, row, q_full);
        *q_loads = ++n;
      }
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      const uint32_t idesc_s = idesc_bf16(64, kHeads), idesc_o = idesc_bf16(128, kHeads) | kTransposed,
                     idesc_o64 = idesc_bf16(64, kHeads) | kTransposed;
      const uint32_t q0 = smem_addr(sQ), c0 = smem_addr(sC), p0 = smem_addr(sP);
      uint32_t k = 0, seg = 0;
      bool ok = true;
      auto scores = [&](uint32_t kk, bool last) {
        const int st = (int)(kk % (uint32_t)nst);
        if (!mbar_wait(&c_full[st], (kk / nst) & 1, abort_flag)) return false;
        tc_fence_after();
        const uint32_t d = tmem + oc + (kk & 1) * kHeads, c = c0 + st * stage_bytes;
        for (int x = 0; x < chunks; ++x)
          for (int y = 0; y < 4; ++y)
            mma_bf16(d, sw128_desc(c + x * kChunkBytes + y * 32, 16), sw128_desc(q0 + x * kChunkBytes + y * 32, 16),
                     idesc_s, x | y ? 1u : 0u);
        mma_commit(&s_full[kk & 1]);
        if (last) mma_commit(q_empty);
        return true;
      };
      auto values = [&](uint32_t kk, bool first) {
        if (!mbar_wait(&p_full[kk & 1], (kk >> 1) & 1, abort_flag)) return false;
        if (first && seg > 0 && !mbar_wait(o_empty, (seg - 1) & 1, abort_flag)) return false;
        tc_fence_after();
        const int st = (int)(kk % (uint32_t)nst);
        const uint32_t c = c0 + st * stage_bytes, p = p0 + (kk & 1) * kPBytes;
        for (int x = 0; x < chunks; x += 2)
          for (int y = 0; y < 4; ++y)
            mma_bf16(tmem + (x >> 1) * kHeads, sw128_desc(c + x * kChunkBytes + y * 2048, kChunkBytes),
                     sw128_desc(p + y * 2048, kChunkBytes), x + 1 < chunks ? idesc_o : idesc_o64, !first || y ? 1u : 0u);
        mma_commit(&c_empty[st]);
        mma_commit(&pv_done[kk & 1]);
        return true;
      };
      while (ok && walk.next(P, g)) {
        if (!(ok = mbar_wait(q_full, seg & 1, abort_flag))) break;
        const long long n = g.t1 - g.t0;
        ok = scores(k, n == 1);
        for (long long t = 0; ok && t < n; ++t, ++k) {
          // the next tile's scores go ahead of this tile's values, unless its rows are still on
          // their way when this tile's weights are ready
          bool ahead = t + 1 < n;
          for (int spin = 0; ahead && !mbar_test(&c_full[(k + 1) % (uint32_t)nst], ((k + 1) / nst) & 1); ++spin)
            ahead = spin < kSpins && !mbar_test(&p_full[k & 1], (k >> 1) & 1);
          if (ahead) ok = scores(k + 1, t + 2 == n);
          ok = ok && values(k, t == 0);
          if (!ahead && t + 1 < n) ok = ok && scores(k + 1, t + 2 == n);
        }
        ++seg;
      }
    }
  } else {
    // ---- softmax and epilogue
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const int c2 = 2 * (lane & 3);
    const float sl = P.scale_log2;
    uint32_t k = 0, seg = 0;
    long long index = work[4];  // tile index of the segment's first tile
    bool ok = true;
    while (ok && walk.next(P, g)) {
      float m[16], l[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) m[i] = kFloor, l[i] = 0.0f;
      for (long long t = g.t0; t < g.t1; ++t, ++k) {
        ok = mbar_wait(&s_full[k & 1], (k >> 1) & 1, abort_flag);
        // the weights buffer is free once the tile two before has been used
        if (ok && k >= 2) ok = mbar_wait(&pv_done[k & 1], ((k >> 1) & 1) ^ 1, abort_flag);
        tc_fence_after();
        uint32_t raw[32];
        tmem_ld_frag(tmem + oc + (k & 1) * kHeads + lanes, raw);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(raw[i]);
        if ((t + 1) * kTile > g.s.cnt) {  // rows past the last one
          const long long v = t * kTile + 16 * warp + (lane >> 2);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (v >= g.s.cnt) x[4 * i] = x[4 * i + 1] = -INFINITY;
            if (v + 8 >= g.s.cnt) x[4 * i + 2] = x[4 * i + 3] = -INFINITY;
          }
        }
        bool renew = t == g.t0 || !ok;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            renew = renew || fmaf(fmaxf(x[4 * i + e], x[4 * i + 2 + e]), sl, -m[2 * i + e]) > kStep;
        if (soft_or(renew)) {
          if (soft_or(!ok)) {
            ok = false;
            break;
          }
          float top[16];
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float y = fmaxf(x[4 * i + e], x[4 * i + 2 + e]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
              top[2 * i + e] = y * sl;
            }
          if (lane < 4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) red[warp * 64 + 8 * (i >> 1) + c2 + (i & 1)] = top[i];
          }
          soft_sync();
          float f[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float y = m[i];
#pragma unroll
            for (int w = 0; w < 4; ++w) y = fmaxf(y, red[w * 64 + 8 * (i >> 1) + c2 + (i & 1)]);
            f[i] = ex2(m[i] - y);
            l[i] *= f[i];
            m[i] = y;
          }
          if (t > g.t0) {
            ok = mbar_wait(&pv_done[(k & 1) ^ 1], ((k - 1) >> 1) & 1, abort_flag);
            if (soft_or(!ok)) {
              ok = false;
              break;
            }
            tc_fence_after();
            for (int x2 = 0; x2 < chunks; x2 += 2)
              for (int h = 0; h < (x2 + 1 < chunks ? 2 : 1); ++h) {
                const uint32_t at = tmem + (x2 >> 1) * kHeads + lanes + ((uint32_t)(16 * h) << 16);
                uint32_t o[32];
                tmem_ld_frag(at, o);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  o[i] = __float_as_uint(__uint_as_float(o[i]) * f[2 * (i >> 2) + (i & 1)]);
                tmem_st_frag(at, o);
              }
          } else {
            soft_sync();  // `red` has been read
          }
        }
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = ex2(fmaf(x[4 * i + 2 * h], sl, -m[2 * i])),
                        p1 = ex2(fmaf(x[4 * i + 2 * h + 1], sl, -m[2 * i + 1]));
            l[2 * i] += p0;
            l[2 * i + 1] += p1;
            pk[2 * i + h] = bf16x2(p0, p1);
          }
        {
          // weights [row][64 heads] as 128-byte swizzled rows; matrices of a store: rows 0-7 and 8-15
          // of two head groups of 8
          const int r = 16 * warp + (lane & 15), hg = lane >> 4;
          const uint32_t at = smem_addr(sP) + (k & 1) * kPBytes + r * 128;
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            stmatrix4<false>(at + (((i + hg) ^ (r & 7)) << 4), pk[2 * i], pk[2 * i + 1], pk[2 * i + 2], pk[2 * i + 3]);
        }
        fence_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[k & 1]);
      }
      if (!ok) break;
      // ---- the segment's end: sums over rows, then O^T
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      if (lane < 4) {
#pragma unroll
        for (int i = 0; i < 16; ++i) red[256 + warp * 64 + 8 * (i >> 1) + c2 + (i & 1)] = l[i];
      }
      const uint32_t kl = k - 1;
      ok = mbar_wait(&pv_done[kl & 1], (kl >> 1) & 1, abort_flag);
      if (soft_or(!ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        l[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) l[i] += red[256 + w * 64 + 8 * (i >> 1) + c2 + (i & 1)];
      }
      const bool whole = g.t0 == 0 && g.t1 == g.tiles;
      const int heads = min(kHeads, P.H - g.hb * kHeads);
      const long long orow = g.tok * P.H + g.hb * kHeads;  // the item's first row of out
      if (whole) {
        if (P.c.lse && warp == 0 && lane < 4) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int h = 8 * (i >> 1) + c2 + (i & 1);
            if (h < heads && in_bounds(orow + h, P.toks * P.H, P.flag))
              P.c.lse[orow + h] = l[i] == 0.0f ? -INFINITY : (m[i] + log2f(l[i])) * 0.693147180559945f;
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) l[i] = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
        for (int x2 = 0; x2 < chunks; x2 += 2) {
          const bool full = x2 + 1 < chunks;  // 128 features, else 64
          for (int h = 0; h < (full ? 2 : 1); ++h) {
            uint32_t o[32];
            tmem_ld_frag(tmem + (x2 >> 1) * kHeads + lanes + ((uint32_t)(16 * h) << 16), o);
            // staged as [head][128 features] (16-byte units swizzled by the head): transposed stores
            const int du = (full ? 4 * warp + 2 * h : 2 * warp) + ((lane >> 3) & 1);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              uint32_t v[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int q = i + (j >> 1);
                v[j] = bf16x2(__uint_as_float(o[4 * q + 2 * (j & 1)]) * l[2 * q],
                              __uint_as_float(o[4 * q + 2 * (j & 1) + 1]) * l[2 * q + 1]);
              }
              const int head = 8 * (i + (lane >> 4)) + (lane & 7);
              stmatrix4<true>(smem_addr(sP) + head * 256 + ((du ^ (head & 7)) << 4), v[0], v[1], v[2], v[3]);
            }
          }
          soft_sync();
          const int u = lane & 15;
          for (int h = 2 * warp + (lane >> 4); h < heads; h += 8)
            if ((full || u < 8) && in_bounds(orow + h, P.toks * P.H, P.flag))
              *reinterpret_cast<uint4*>(P.c.out + (orow + h) * D + x2 * 64 + u * 8) =
                  *reinterpret_cast<const uint4*>(sP + h * 256 + ((u ^ (h & 7)) << 4));
          soft_sync();
        }
      } else {
        // a piece: slot 0 of the CTA for its first segment's, 1 for its last's (a first piece)
        const int slot = 2 * blockIdx.x + (g.t0 == 0 ? 1 : 0);
        if (warp == 0 && lane < 4) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            P.part_ml[slot * kHeads + 8 * (i >> 1) + c2 + (i & 1)] = make_float2(m[i], l[i]);
        }
        float* dst = P.part + (size_t)slot * kHeads * D;
        for (int x2 = 0; x2 < chunks; x2 += 2) {
          const bool full = x2 + 1 < chunks;
          const int d = x2 * 64 + (full ? 32 * warp + lane : 16 * warp + lane);
          for (int hh = 0; hh < kHeads; hh += 32) {
            uint32_t o[32];
            tmem_ld32(tmem + (x2 >> 1) * kHeads + hh + lanes, o);
            if (full || lane < 16) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (hh + i < heads) dst[(size_t)(hh + i) * D + d] = __uint_as_float(o[i]);
            }
          }
        }
        if (g.t0 == 0 && threadIdx.x == 0) {
          // the item ends in the CTA whose share holds its last tile
          const long long end = index + g.tiles, total = work[6], ctas = work[7];
          long long j = (end * ctas - 1) / total;
          while (total * (j + 1) / ctas < end) ++j;
          while (total * j / ctas >= end) --j;
          P.record[blockIdx.x] = make_int2((int)(g.tok * P.hblocks + g.hb), (int)(j - blockIdx.x) + 1);
        }
        soft_sync();  // `red` has been read before the next segment writes it
      }
      index += g.t1 - g.t0;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty);
      ++seg;
    }
  }

  // ---- leave: after an abort, let the copies in flight land and the issued products complete
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) atomicOr(P.flag, 4);
    if (warp == kQWarp && lane == 0 && *q_loads > 0) mbar_wait_bounded(q_full, (*q_loads - 1) & 1);
    if (warp == kMmaWarp && lane == 0) {
      mma_commit(mma_done);
      mbar_wait_bounded(mma_done, 0);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, tmem_cols);
}

// ---- pieces of split items joined: one CTA per (record, head).
//   M = max m_p;  out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p
// The pieces are added in order by each of the CTA's thread rows (a row covers the D features) and
// the rows' sums in order after that: the result does not depend on timing.
constexpr int kJoinThreads = 256, kMaxPieces = 1024;
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const AttnParams P) {
  __shared__ float w[kMaxPieces];
  __shared__ float red[16];
  __shared__ float4 acc[kJoinThreads];
  griddep_wait();
  const int2 rec = P.record[blockIdx.x];
  const int n = rec.y, h = blockIdx.y;
  if (rec.x < 0) return;
  const long long tok = rec.x / P.hblocks;
  const int hb = rec.x % P.hblocks, head = hb * kHeads + h;
  if (head >= P.H) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto slot = [&](int p) { return 2 * ((int)blockIdx.x + p) + (p == 0 ? 1 : 0); };
  float top = kFloor;
  for (int p = threadIdx.x; p < n; p += kJoinThreads) top = fmaxf(top, P.part_ml[slot(p) * kHeads + h].x);
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) red[warp] = top;
  __syncthreads();
  for (int i = 0; i < kJoinThreads / 32; ++i) top = fmaxf(top, red[i]);
  float sum = 0.0f;
  for (int p = threadIdx.x; p < n; p += kJoinThreads) {
    const float2 ml = P.part_ml[slot(p) * kHeads + h];
    w[p] = ex2(ml.x - top);
    sum += ml.y * w[p];
  }
  sum = warp_sum(sum);
  if (lane == 0) red[8 + warp] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int i = 0; i < kJoinThreads / 32; ++i) sum += red[8 + i];
  const int quads = P.D / 4, rows = kJoinThreads / quads, q = threadIdx.x % quads, r = threadIdx.x / quads;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (r < rows) {
#pragma unroll 4
    for (int p = r; p < n; p += rows) {
      const float4 o = reinterpret_cast<const float4*>(P.part + ((size_t)slot(p) * kHeads + h) * P.D)[q];
      const float f = w[p];
      a.x = fmaf(o.x, f, a.x), a.y = fmaf(o.y, f, a.y), a.z = fmaf(o.z, f, a.z), a.w = fmaf(o.w, f, a.w);
    }
  }
  acc[threadIdx.x] = a;
  __syncthreads();
  if (r != 0) return;
  for (int i = 1; i < rows; ++i) {
    const float4 o = acc[i * quads + q];
    a.x += o.x, a.y += o.y, a.z += o.z, a.w += o.w;
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const long long orow = tok * P.H + head;
  if (in_bounds(orow, P.toks * P.H, P.flag)) {
    reinterpret_cast<uint2*>(P.c.out + orow * P.D)[q] = make_uint2(bf16x2(a.x * inv, a.y * inv), bf16x2(a.z * inv, a.w * inv));
    if (P.c.lse && q == 0) P.c.lse[orow] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
  }
}

// ---- host side
// Stages: as many tiles (a power of two, at most 8) as the shared memory takes: two CTAs an SM up
// to D = 192 (their tensor memory is 256 columns), else one.
struct Shape {
  int ctas, stages, smem;
};
Shape attn_shape(int D, bool fp4) {
  Shape s;
  s.ctas = D <= 192 && !fp4 ? 2 : 1;
  const int chunk = D / 64 * kChunkBytes, budget = (s.ctas == 2 ? 113 : 227) * 1024 - 1024 - kAuxBytes;
  s.stages = 8;
  while (s.stages > 2 && (s.stages + 1) * chunk + 2 * kPBytes > budget) s.stages /= 2;
  s.smem = (s.stages + 1) * chunk + 2 * kPBytes + kAuxBytes + 1024;
  return s;
}

}  // namespace

size_t attention_workspace_bytes(int head_dim) {
  const size_t slots = 2 * (size_t)current_sm_count() * attn_shape(head_dim, false).ctas;
  return slots * kHeads * (head_dim * sizeof(float) + sizeof(float2)) + slots * sizeof(int2);
}

cudaError_t launch_attention(csa_attention* a, const AttnCall& call, cudaStream_t s) {
  auto encode = get_encode();
  if (!encode) return cudaErrorNotSupported;
  const bool fp4 = call.paged && !call.cache.latent;
  const Shape sh = attn_shape(a->D, fp4);
  auto* kernel = fp4 ? attention_kernel<true, 1> : sh.ctas == 2 ? attention_kernel<false, 2> : attention_kernel<false, 1>;
  static std::atomic<unsigned long long> attr{0};
  cudaError_t e = once_per_device(attr, [] {
    const int most = 227 * 1024;
    cudaError_t r = cudaFuncSetAttribute(attention_kernel<true, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(attention_kernel<false, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(attention_kernel<false, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return r;
  });
  if (e != cudaSuccess) return e;
  const int sms = current_sm_count();
  const int slots = 2 * sms * attn_shape(a->D, false).ctas;
  AttnParams P{};
  P.c = call;
  P.H = a->heads;
  P.D = a->D;
  P.window = a->window;
  P.sinks = a->sinks;
  P.hblocks = (a->heads + kHeads - 1) / kHeads;
  P.toks = (long long)call.B * call.N;
  P.scale_log2 = (float)(a->scale * 1.4426950408889634);
  P.flag = a->dev_flag;
  P.part = (float*)a->workspace;
  P.part_ml = (float2*)(P.part + (size_t)slots * kHeads * a->D);
  P.record = (int2*)(P.part_ml + (size_t)slots * kHeads);
  P.stages = sh.stages;
  P.unit_magic = (uint32_t)((0x100000000ull + a->D / 32 - 1) / (a->D / 32));
  // the longest visible range that this call can have decides whether items may be cut
  long long most = call.paged ? (long long)call.max_pages * call.cache.page_size : (long long)call.start + call.N;
  if (a->window && most > (long long)a->window + a->sinks) most = (long long)a->window + a->sinks;
  P.split = most > (long long)kJoinTiles * kTile;
  const long long tiles = P.toks * P.hblocks * ((most + kTile - 1) / kTile > 0 ? (most + kTile - 1) / kTile : 1);
  const int grid = (int)(tiles < (long long)sms * sh.ctas ? tiles : (long long)sms * sh.ctas);
  CUtensorMap mq;
  {
    cuuint64_t dims[2] = {(cuuint64_t)a->D, (cuuint64_t)(P.toks * a->heads)};
    cuuint64_t strides[1] = {(cuuint64_t)a->D * 2};
    cuuint32_t box[2] = {64, kHeads};
    cuuint32_t es[2] = {1, 1};
    if (encode(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (void*)call.q, dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  kernel<<<grid, fp4 ? attn_threads<true>() : attn_threads<false>(), sh.smem, s>>>(mq, P);
  a->launches += 1;
  if ((e = cudaGetLastError()) != cudaSuccess || !P.split) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, a->heads < kHeads ? a->heads : kHeads);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  a->launches += 1;
  return cudaLaunchKernelEx(&cfg, attention_join_kernel, P);
}

}  // namespace csa
