// Matrix product of e4m3 values with f32 scales per 128 (see include/csa.h):
//
//   out[t][n] = sum_b a[t][b] * w[n / 128][b] * sum_{k of block b} Q[t][k] * W[n][k]
//
// The inner sums are exact products added by the tensor core; the outer ones, with the scales, are f32
// FMAs on what is read back from tensor memory block by block.
//
// linear_tile_kernel: a CTA takes 128 rows of W as the MMA's rows and NT tokens as its columns, so that
// few tokens cost few columns and a tile's 128 rows have one scale a block (128 tokens are the MMA's rows).  K is split over the CTAs of
// a cluster where there are few tiles: each adds its blocks up, and the partial sums are added through
// distributed shared memory in the order of the CTAs.  Else a CTA takes tile after tile.
//   1 token of 4096 to 512       3.7 to 4.1 us (bound by the launch and the chain copy, MMA, sums, cluster, store)
//   1 to 64 tokens to 32768      22.5 to 25 us (134 MB of W: 6.0 to 5.5 TB/s, 0.88 to 0.81 of a copy's rate)
//   128 tokens to 32768          27.4 us (5.2 TB/s: a block of 128 x 112 takes 650 cycles, 480 of them its 30 KB in and out
//                                of shared memory; HBM would need 620)
//   333 tokens of 4224 to 1000   7.9 us (96 CTAs of 8 blocks: the chain again)
#include <cstdlib>

#include "layer_ops.h"
#include "tc_common.cuh"

namespace csa {
namespace {

using namespace tcx;

constexpr int kBlock = 128;                    // features of a scale: bytes of a row in a stage
constexpr int kRowsN = 128;                    // rows of W in a tile, at most, and of a scale
constexpr int kWBytes = kRowsN * kBlock;       // a stage's W
constexpr int kSlots = 8;                      // ring of scale products
constexpr int kMostSplit = 8;                  // CTAs that share a tile's K
constexpr long long kMostItems = 0x7fff0000LL;  // tiles of a call: a CTA's stride further is an int still
constexpr int kSumRow = kRowsN + 4;             // a token's sums where CTAs add theirs up (banks)
constexpr int kFirstEpi = 3;                   // warps: copies, MMAs, scales, then the sums

// A time-out (4) or, in the bounds-checked build, a store outside the output (8), of any call on the device.
__device__ int linear_flag;

struct LinearParams {
  const float* a;  // [T][blocks]
  const float* w;  // [tiles of N][blocks]
  void* out;       // [T][N] bf16 or f32
  int T, N, blocks, f32;
  int split;    // CTAs of a cluster
  int columns;  // tiles of tokens
  int items;    // tiles of W x tokens
  int rows;     // of W in a tile
  int vec2;     // whether rows of a bf16 output are aligned for two values at a time
  int vec;      // whether rows of the output are aligned for four values at a time
  int vec16;    // or for 16 bytes
  int m_tiles, n_tiles;  // of pairs
  int half;              // blocks of the first of two pairs that share a tile
  int vec_scales;        // rows of scales are aligned for four at a time
  uint64_t wait_ns;
#ifdef CSA_DEBUG_BOUNDS
  long long extent;  // values of the output
  int test_stall;    // the time-out test: the last stage never comes
#endif
};

#ifdef CSA_DEBUG_BOUNDS
__device__ __forceinline__ bool in_out(const LinearParams& P, long long i) { return in_bounds(i, P.extent, &linear_flag); }
#else
__device__ __forceinline__ bool in_out(const LinearParams&, long long) { return true; }
#endif

// kind::f8f6f4 with e4m3 operands (format 0 of both), f32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(
          d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// K-major tile of 128-byte rows with 128-byte swizzle: 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1u << 46 |
         (uint64_t)2u << 61;
}
__device__ __forceinline__ float2 f32_pair(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }
// One lane of a converged warp, the same at every call: what it alone issues stays in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16 columns of a warp's 32 lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 64 columns.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, "
      "%40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, "
      "%63}, [%64];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), 
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), 
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), 
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), 
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), 
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), 
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), 
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}

// Four adjacent values n .. n + 3 of the output's row t.
__device__ __forceinline__ void store4(const LinearParams& P, long long t, int n, float4 v) {
  const long long at = t * P.N + n;
  if (P.vec && n + 3 < P.N) {
    if (!in_out(P, at + 3)) return;
    if (P.f32)
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(P.out) + at) = v;
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(P.out) + at) = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
    return;
  }
  const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < P.N && in_out(P, at + i)) {
      if (P.f32)
        reinterpret_cast<float*>(P.out)[at + i] = x[i];
      else
        reinterpret_cast<uint16_t*>(P.out)[at + i] = bf16_bits(x[i]);
    }
}

// 16 bytes (eight bf16 or four f32 values) from column n of the output's row t, whose rows are aligned for them.
__device__ __forceinline__ void store16(const LinearParams& P, long long t, int n, uint4 v) {
  const long long at = t * P.N + n;
  if (!in_out(P, at + (P.f32 ? 3 : 7))) return;
  if (P.f32)
    __stcs(reinterpret_cast<uint4*>(reinterpret_cast<float*>(P.out) + at), v);
  else
    __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(P.out) + at), v);
}

// A thread's sums of row n of W and kCols tokens from t on: two lanes exchange a value for stores of two
// bf16, so that a warp writes 64 bytes of two tokens' rows at a time.
template <int kCols>
__device__ __forceinline__ void store_columns(const LinearParams& P, const float2 (&acc)[kCols / 2], int t, int n, int lane) {
#pragma unroll
  for (int c = 0; c < kCols / 2; ++c) {
    const long long at = (long long)(t + 2 * c) * P.N + n;
    if (P.f32) {
      if (n < P.N && t + 2 * c < P.T && in_out(P, at)) reinterpret_cast<float*>(P.out)[at] = acc[c].x;
      if (n < P.N && t + 2 * c + 1 < P.T && in_out(P, at + P.N)) reinterpret_cast<float*>(P.out)[at + P.N] = acc[c].y;
    } else if (P.vec2) {
      const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? acc[c].x : acc[c].y, 1);
      const long long to = lane & 1 ? at + P.N - 1 : at;  // (an even lane the first token's, an odd one the second's)
      if ((n | 1) < P.N && t + 2 * c + (lane & 1) < P.T && in_out(P, to + 1))
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(P.out) + to) = lane & 1 ? bf16_pair(other, acc[c].y) : bf16_pair(acc[c].x, other);
    } else {
      if (n < P.N && t + 2 * c < P.T && in_out(P, at)) reinterpret_cast<uint16_t*>(P.out)[at] = bf16_bits(acc[c].x);
      if (n < P.N && t + 2 * c + 1 < P.T && in_out(P, at + P.N)) reinterpret_cast<uint16_t*>(P.out)[at + P.N] = bf16_bits(acc[c].y);
    }
  }
}

// A warp's staging to `rows` rows and `bytes` of each of an output whose rows are not aligned for 16 bytes: lanes take
// neighbouring values, so that a store is 64 bytes of one row or two (by 16 bytes a lane, value after value, us: 2000 tokens of
// 128 to 30001 256 -> 68, 4000 to 20002 335 -> 67).  U: two bytes of bf16 at a time, or four.
template <class U>
__device__ __forceinline__ void store_unaligned(uint8_t* out, long long pitch, const uint8_t* stage, int rows, int bytes, int lane) {
  constexpr int kAcross = 64 / (int)sizeof(U), kStep = 32 / kAcross, kAhead = 8;
  const int at = (int)sizeof(U) * (lane % kAcross), first = lane / kAcross;
  if (at >= bytes) return;
  for (int r0 = first; r0 < rows; r0 += kStep * kAhead) {
    U v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int r = (r0 + kStep * k) & 31;
      v[k] = *reinterpret_cast<const U*>(stage + r * 64 + (((at >> 4) ^ ((r >> 1) & 3)) << 4) + (at & 15));
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (r0 + kStep * k < rows) *reinterpret_cast<U*>(out + (r0 + kStep * k) * pitch + at) = v[k];
  }
}

// A thread's sums of token row0 + lane and kRowCols rows of W from n0 on (before `end`), to the output by way of shared memory: 64 bytes of
// each of 32 rows at a time, 16-byte units swizzled.  kOdd: rows may be unaligned for 16 bytes.
constexpr int kRowCols = 64;
constexpr int kRowStage = 2048;  // a warp's staging of 32 rows of 64 bytes
template <bool kOdd>
__device__ __forceinline__ void store_rows(const LinearParams& P, const float2 (&acc)[kRowCols / 2], uint8_t* stage, int row0, int n0, int end,
                                           int lane) {
  const int per = P.f32 ? 4 : 8, sw = (lane >> 1) & 3;
#pragma unroll
  for (int c = 0; c < kRowCols; c += 16) {
    if (P.f32) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 x = acc[c / 2 + 2 * u], y = acc[c / 2 + 2 * u + 1];
        *reinterpret_cast<float4*>(stage + lane * 64 + ((u ^ sw) << 4)) = make_float4(x.x, x.y, y.x, y.y);
      }
    } else {
      const int off = (c & 16) ? 2 : 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float2* x = acc + c / 2 + 4 * u;
        *reinterpret_cast<uint4*>(stage + lane * 64 + (((u + off) ^ sw) << 4)) =
            make_uint4(bf16_pair(x[0].x, x[0].y), bf16_pair(x[1].x, x[1].y), bf16_pair(x[2].x, x[2].y), bf16_pair(x[3].x, x[3].y));
      }
      if (!off) continue;
    }
    __syncwarp();
    const int col0 = n0 + (P.f32 ? c : c - 16);  // of this piece's columns
    if (kOdd && !P.vec16) {
      const int each = P.f32 ? 4 : 2, there = min(32, P.T - row0), bytes = (end - col0) * each;
#ifdef CSA_DEBUG_BOUNDS
      const bool whole = there <= 0 || bytes <= 0 || in_out(P, (long long)(row0 + there - 1) * P.N + min(end, col0 + 64 / each) - 1);
#else
      constexpr bool whole = true;
#endif
      uint8_t* const to = reinterpret_cast<uint8_t*>(P.out) + ((long long)row0 * P.N + col0) * each;
      // (in the bounds-checked build a piece that ends outside loses its last row)
      if (P.f32 || P.vec2)
        store_unaligned<uint32_t>(to, (long long)P.N * each, stage, there - !whole, bytes, lane);
      else
        store_unaligned<uint16_t>(to, (long long)P.N * each, stage, there - !whole, bytes, lane);
      __syncwarp();
      continue;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 8 * k + (lane >> 2), u = lane & 3;
      const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
      const int n = col0 + u * per;
      if (row0 + r < P.T && n < end) store16(P, row0 + r, n, v);
    }
    __syncwarp();
  }
}

template <int NT>
struct Tile {
  // up to 64 tokens two CTAs share an SM: what one's fill and end leave idle the other uses (with 128
  // there are not the registers for it)
  static constexpr int kCtas = NT == 128 ? 1 : 2;
  static constexpr int kGroups = NT == 128 ? 2 : 1;  // of four warps, which take 64 tokens at most
  static constexpr int kEpiWarps = 4 * kGroups, kThreads = 32 * (kFirstEpi + kEpiWarps);
  static constexpr int kCols = NT / kGroups;         // a thread's sums
  static constexpr int kStages = NT == 64 ? 4 : NT == 32 ? 5 : 6;
  static constexpr int kStageBytes = kWBytes + NT * kBlock;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kBuffers = 4;  // accumulators
  // 128 tokens are the MMA's rows: a thread of the sums has one token, and one factor a block where its 64 columns' would
  // be 16 loads from a shared memory that the copies and MMAs fill (128 tokens of 4096 to 32768 31.2 -> 27.7 us, of 512 to
  // 130000 24.4 -> 19.4)
  static constexpr bool kTokenRows = NT == 128;
  static constexpr int kColumns = NT * kBuffers < 32 ? 32 : NT * kBuffers;
  static constexpr int kStaging = kTokenRows ? kEpiWarps * kRowStage : 0;
  static constexpr int kScales = kTokenRows ? 2 : 1;  // of a token and block
  static constexpr int kSmem = kRing + kStaging + kScales * kSlots * NT * 4 + 512 + 1024;
  static_assert(kBuffers <= kStages, "see the commits");
  static_assert(NT * kSumRow * 4 <= kRing, "the partial sums take the ring's place");
  static_assert(!kTokenRows || kCols == kRowCols, "of store_rows");
};

template <int NT>
__global__ void __launch_bounds__(Tile<NT>::kThreads, Tile<NT>::kCtas)
    linear_tile_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ LinearParams P) {
  using C = Tile<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  float* scale = reinterpret_cast<float*>(smem + C::kRing + C::kStaging);  // [kSlots][NT]
  uint64_t* full = reinterpret_cast<uint64_t*>(scale + C::kScales * kSlots * NT);
  uint64_t* empty = full + C::kStages;
  uint64_t* t_empty = empty + C::kStages;
  uint64_t* s_full = t_empty + C::kBuffers;
  uint64_t* s_empty = s_full + kSlots;
  uint64_t* mma_done = s_empty + kSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < C::kBuffers; ++i) mbar_init(&t_empty[i], C::kEpiWarps);
    for (int i = 0; i < kSlots; ++i) mbar_init(&s_full[i], 1), mbar_init(&s_empty[i], C::kEpiWarps);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_map(&map_q);
    prefetch_map(&map_w);
  }
  if (warp == 1) tmem_alloc(tmem_slot, C::kColumns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  const int rank = P.split > 1 ? (int)cluster_rank() : 0;
  const int b0 = (int)((long long)P.blocks * rank / P.split), b1 = (int)((long long)P.blocks * (rank + 1) / P.split);
  const int steps = b1 - b0;
  // Items (tile of W, tokens), the CTAs of a tile's tokens side by side, so that its rows of W come from memory
  // once.  A CTA of its own takes item after item, the next one's copies and MMAs under way while it stores; a
  // cluster has one item.
  const int first_item = blockIdx.x / P.split, stride = gridDim.x / P.split;
  auto item_tile = [&](int item) { return item / P.columns; };
  const int rows = C::kTokenRows ? P.rows : kRowsN;  // of W in a tile
  auto item_token = [&](int item) { return (item - item / P.columns * P.columns) * NT; };
  const int first_col = warp < kFirstEpi ? 0 : C::kCols * ((warp - kFirstEpi) >> 2);
  int issued = 0;
  float2 acc[C::kCols / 2];  // (paired FMAs: two a lane and instruction)

  if (warp == 0) {
    // ---- copies
    if (lane == 0) {
      bool ok = true;
      for (int item = first_item; ok && item < P.items; item += stride) {
        const int n0 = item_tile(item) * rows, t0 = item_token(item);
        for (int i = 0; i < steps; ++i) {
          const int st = issued % C::kStages;
          if (issued >= C::kStages && !(ok = mbar_wait(&empty[st], (issued / C::kStages - 1) & 1, abort_flag, P.wait_ns))) break;
#ifdef CSA_DEBUG_BOUNDS
          if (P.test_stall && i + 1 == steps && item + stride >= P.items) {
            ok = false;
            break;
          }
#endif
          mbar_arrive_expect_tx(&full[st], (rows + NT) * kBlock);
          tma_load_2d(smem + st * C::kStageBytes, &map_w, (b0 + i) * kBlock, n0, &full[st]);
          tma_load_2d(smem + st * C::kStageBytes + kWBytes, &map_q, (b0 + i) * kBlock, t0, &full[st]);
          ++issued;
        }
      }
    }
  } else if (warp == 1) {
    // ---- MMAs: a block's accumulator of its own
    // the whole warp runs the loop and one elected lane issues (under `lane == 0` the descriptors' way to uniform
    // registers cost 100 cycles an MMA)
    constexpr uint32_t idesc = idesc_e4m3(kRowsN, NT);
    const uint32_t idesc_rows = idesc_e4m3(NT, P.rows);
    const bool leader = elect_one();
    const uint64_t first = sw128_desc(smem_addr(smem));
    int i = 0, st = 0, round = 0;
    bool ok = true;
    for (int item = first_item; ok && item < P.items; item += stride)
      for (int b = 0; b < steps; ++b, ++i) {
        const int buf = i % C::kBuffers;
        const uint32_t pe = (i / C::kBuffers - 1) & 1, pf = round & 1;
        const bool e0 = i < C::kBuffers || mbar_try_wait(&t_empty[buf], pe), f0 = mbar_try_wait(&full[st], pf);
        if (!__all_sync(0xffffffffu, e0 && f0)) {
          ok = (e0 || mbar_wait(&t_empty[buf], pe, abort_flag, P.wait_ns)) && (f0 || mbar_wait(&full[st], pf, abort_flag, P.wait_ns));
          if (!(ok = __all_sync(0xffffffffu, ok) != 0)) break;
        }
        tc_fence_after();
        if (leader) {
          const uint64_t x = first + (uint64_t)(st * (C::kStageBytes / 16)), y = x + kWBytes / 16;
#pragma unroll
          for (int k = 0; k < kBlock / 32; ++k) mma_e4m3(tmem + buf * NT, (C::kTokenRows ? y : x) + 2 * k, (C::kTokenRows ? x : y) + 2 * k, C::kTokenRows ? idesc_rows : idesc, k ? 1u : 0u);
          // one commit says that the stage is free and the accumulator there (a commit takes hundreds of cycles of
          // the tensor core's queue): a stage's next block waits for a buffer that the sums have read, so its
          // phase is never past what they wait for
          mma_commit(&empty[st]);
        }
        __syncwarp();
        if (++st == C::kStages) st = 0, ++round;
      }
  } else if (warp == 2) {
    // ---- scales: a[t][b] * w[tile][b] of each block, a lane per token, four blocks' loads at once
    constexpr int kPer = (NT + 31) / 32, kAhead = 4;
    bool ok = true;
    int n = 0;
    for (int item = first_item; ok && item < P.items; item += stride) {
      const int t0 = item_token(item);
      const int tile = item_tile(item) * rows / kRowsN;
      const float* w = P.w + (size_t)tile * P.blocks;
      const float* w2 = (tile + 1LL) * kRowsN < P.N ? w + P.blocks : w;  // (a tile of fewer rows may have two scales)
      for (int i = 0; ok && i < steps; i += kAhead) {
        float v[kAhead][kPer], sw[kAhead], sw2[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const bool there = i + j < steps;
          sw[j] = there ? w[b0 + i + j] : 0.0f;
          sw2[j] = C::kTokenRows && there ? w2[b0 + i + j] : 0.0f;
#pragma unroll
          for (int x = 0; x < kPer; ++x) {
            const int c = 32 * x + lane;
            v[j][x] = there && c < NT && t0 + c < P.T ? P.a[(size_t)(t0 + c) * P.blocks + b0 + i + j] : 0.0f;
          }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (!ok || i + j >= steps) break;
          const int s = n % kSlots;
          ok = n < kSlots || mbar_wait(&s_empty[s], (n / kSlots - 1) & 1, abort_flag, P.wait_ns);
          if (!(ok = __all_sync(0xffffffffu, ok) != 0)) break;
#pragma unroll
          for (int x = 0; x < kPer; ++x)
            if (32 * x + lane < NT) {
              scale[C::kScales * s * NT + 32 * x + lane] = v[j][x] * sw[j];
              if (C::kTokenRows) scale[(C::kScales * s + 1) * NT + 32 * x + lane] = v[j][x] * sw2[j];
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_full[s]);
          ++n;
        }
      }
    }
  } else {
    // ---- sums: a thread has a row of W and 64 tokens at most, or a token and 64 rows of W
    const int row = 32 * (warp & 3) + lane;
    const uint32_t base = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + first_col;
    int i = 0, st = 0, round = 0;
    bool ok = true;
    for (int item = first_item; ok && item < P.items; item += stride) {
#pragma unroll
      for (int c = 0; c < C::kCols / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
      const int n0 = item_tile(item) * rows, border = (n0 / kRowsN + 1) * kRowsN - n0 - first_col;  // of the second scale
      for (int b = 0; b < steps; ++b, ++i) {
        const int buf = i % C::kBuffers, s = i % kSlots;
        const uint32_t ps = (i / kSlots) & 1, pe = round & 1;
        const bool s0 = mbar_try_wait(&s_full[s], ps), e0 = mbar_try_wait(&empty[st], pe);
        if (!__all_sync(0xffffffffu, s0 && e0)) {
          ok = (s0 || mbar_wait(&s_full[s], ps, abort_flag, P.wait_ns)) && (e0 || mbar_wait(&empty[st], pe, abort_flag, P.wait_ns));
          if (!(ok = __all_sync(0xffffffffu, ok) != 0)) break;
        }
        if (++st == C::kStages) st = 0, ++round;
        tc_fence_after();
        if constexpr (C::kTokenRows) {
          const float fa = scale[2 * s * NT + row], fb = scale[(2 * s + 1) * NT + row];
          uint32_t r[kRowCols];
          tmem_ld64(base + buf * NT, r);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&t_empty[buf]);
            mbar_arrive(&s_empty[s]);
          }
#pragma unroll
          for (int k = 0; k < kRowCols; k += 2) {
            const float f = (k & ~15) < border ? fa : fb;  // (16 rows of W have one scale)
            acc[k / 2] = __ffma2_rn(f32_pair(r[k], r[k + 1]), make_float2(f, f), acc[k / 2]);
          }
          continue;
        }
        constexpr int kPart = C::kCols < 32 ? C::kCols : 32;
#pragma unroll
        for (int c = 0; c < C::kCols; c += kPart) {
          uint32_t r[kPart];
          if constexpr (kPart == 32)
            tmem_ld32(base + buf * NT + c, r);
          else
            tmem_ld16(base + buf * NT + c, r);
#pragma unroll
          for (int j = 0; j < kPart; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(scale + s * NT + first_col + c + j);
            float2& x = acc[(c + j) / 2];
            float2& y = acc[(c + j) / 2 + 1];
            x = __ffma2_rn(f32_pair(r[j], r[j + 1]), make_float2(f.x, f.y), x);
            y = __ffma2_rn(f32_pair(r[j + 2], r[j + 3]), make_float2(f.z, f.w), y);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&t_empty[buf]);
          mbar_arrive(&s_empty[s]);
        }
      }
      if (ok && P.split == 1) {
        if constexpr (C::kTokenRows)
          store_rows<true>(P, acc, smem + C::kRing + (warp - kFirstEpi) * kRowStage, item_token(item) + row - lane,
                     n0 + first_col, min(P.N, n0 + rows), lane);
        else
          store_columns<C::kCols>(P, acc, item_token(item) + first_col, n0 + row, lane);
      }
    }
  }

  // ---- every role has left its loop: the ring's copies have been used, or land now
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) atomicOr(&linear_flag, 4);
    drain_after_abort(warp == 0 && lane == 0, warp == 1 && elect_one(), full, C::kStages, issued, mma_done);
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kColumns);
  if (P.split == 1) return;
  // ---- the cluster's partial sums, each CTA's share of the tokens
  const int n0 = item_tile(first_item) * kRowsN, t0 = item_token(first_item);
  float* part = reinterpret_cast<float*>(smem);  // [NT][kSumRow]
  if (warp >= kFirstEpi) {
    const int r = 32 * (warp & 3) + lane;
    if constexpr (C::kTokenRows) {
#pragma unroll
      for (int c = 0; c < C::kCols; c += 4)
        *reinterpret_cast<float4*>(part + r * kSumRow + first_col + c) = make_float4(acc[c / 2].x, acc[c / 2].y, acc[c / 2 + 1].x, acc[c / 2 + 1].y);
    } else {
#pragma unroll
      for (int c = 0; c < C::kCols; ++c) part[(first_col + c) * kSumRow + r] = c & 1 ? acc[c / 2].y : acc[c / 2].x;
    }
  }
  const int c0 = NT * rank / P.split, c1 = NT * (rank + 1) / P.split;
  cluster_arrive();
  cluster_wait();
  for (int c = c0 + warp; c < c1; c += C::kThreads / 32) {
    if (t0 + c >= P.T) break;
    float4 v = make_float4(0, 0, 0, 0), x[kMostSplit];  // (all under way before the first is added)
#pragma unroll
    for (int j = 0; j < kMostSplit; ++j)
      if (j < P.split) x[j] = ld_cluster_f4(cluster_map(part + c * kSumRow + 4 * lane, j));
#pragma unroll
    for (int j = 0; j < kMostSplit; ++j)
      if (j < P.split) v = make_float4(v.x + x[j].x, v.y + x[j].y, v.z + x[j].z, v.w + x[j].w);
    if (n0 + 4 * lane < P.N) store4(P, t0 + c, n0 + 4 * lane, v);
  }
  cluster_arrive();  // no CTA leaves while its sums are read
  cluster_wait();
}

// ---------------------------------------------------------------------------------------
// linear_pair_kernel: two CTAs of a cluster share tiles of 256 tokens x 128 rows of W.  Tokens are the MMA's
// rows (M = 256: each CTA's 128 from its own shared memory), W's rows its columns (N = 128: each CTA
// brings half), so a stage of 128 features is 24 KB a CTA.  A thread of the epilogue has a token's 64 columns:
// the token's scale and the columns' one scale make one factor a block.  One pair an SM pair, tile after
// tile: the next tile's copies and MMAs run while a tile's sums are stored.  Few tiles of many blocks are shared by two pairs
// of a cluster of four CTAs, whose sums are added through distributed shared memory.
//
// What bounds it: every block's accumulator goes through the epilogue, and tensor memory holds four, 1024 cycles of
// MMAs.  From a block's issue to its buffer's reuse pass about 2000 (its MMAs 256, the commit to both CTAs 1100,
// the reading 80, the arrival from the other CTA 500 to 800), so a block takes 470 where its MMAs need 256: 4096
// tokens of 4096 to 32768 in 429 us, 2.56 PFLOP/s (1.36 of the bf16 rate; the power cap brings long runs to 480 us).
// Measured and not taken (us, the same product, when this took 441): tiles of 256 x 256 with two accumulators 526; the same by MMAs of
// one CTA with W's rows multicast to both, whose commits and arrivals stay in the SM, 470 (shared memory then takes in and
// gives out 96 KB a block); the warp that issues looking at four blocks' barriers at once 488.  And against 429:
// sixteen warps of 32 columns 456; half a block's columns asked for while the other half's are added up 504 (two loads of 32
// columns cost more than one of 64); without the additions 378, which is what a second set of registers could gain at most.
constexpr int kPairM = 256, kPairN = 128;
constexpr int kPairSplitBlocks = 28;  // of a tile that two pairs share, at least
constexpr int kPairBuffers = 512 / kPairN;
constexpr int kPairStages = 8, kPairStageBytes = kWBytes + kPairN / 2 * kBlock;
constexpr int kPairEpi = 8, kPairFirst = 3, kPairThreads = 32 * (kPairFirst + kPairEpi);
constexpr int kPairCols = kPairN / (kPairEpi / 4);  // a warp's columns
static_assert(kPairCols == kRowCols, "of store_rows");
constexpr int kPairScales = 4 * 128;                // products of scales: of four blocks, 128 tokens
constexpr int kPairSmem = kPairStages * kPairStageBytes + kPairEpi * kRowStage + 2 * kPairScales * 4 + 256 + 1024;

__device__ __forceinline__ void mma_e4m3_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(
          d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_addr(dst)),
      "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// An arrival that orders nothing in memory: the accumulator's values are in registers (tcgen05.wait::ld).  The
// releasing form takes thousands of cycles where 32 warps of two CTAs do it for every block: 4096 x 4096 to
// 32768 took 1230 us with it.
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The i-th tile of a pair: tokens fastest within groups of 16 tiles, so that the tiles that run at one time
// read few rows of either operand.
__device__ __forceinline__ int2 pair_tile(const LinearParams& P, int i) {
  const int group = 16 * P.n_tiles, g = i / group, left = min(16, P.m_tiles - 16 * g), r = i - g * group;
  return make_int2(16 * g + r % left, r / left);
}

// Four scales of a row from block b on; behind the last one anything.
__device__ __forceinline__ float4 scales4(const LinearParams& P, const float* row, int b) {
  const int last = P.blocks - 1;
  if (P.vec_scales) return *reinterpret_cast<const float4*>(row + min(b, last & ~3));
  return make_float4(row[min(b, last)], row[min(b + 1, last)], row[min(b + 2, last)], row[min(b + 3, last)]);
}

// A wait that looks at the barrier a while before it lets itself be suspended: a sum's warp that is woken reads its values
// later, and its buffer is in the way of the next MMAs (4096 tokens to 32768: 446 -> 429 us; the MMAs' warp too: 436; in linear_tile_kernel, whose
// sums have the SM's issue to share, 31.6 -> 32.2 us).
__device__ __forceinline__ bool mbar_wait_awake(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t wait_ns) {
  for (int i = 0; i < 256; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return mbar_wait(bar, parity, abort_flag, wait_ns);
}

// kTwo: two pairs a tile.  (A template, and the first tile found by each role: as a run-time choice, or with the first
// tile in a variable of all roles, 4096 tokens to 32768 took 6 % longer.)  kOdd: the output's rows are unaligned for 16 bytes (the
// code for both cost aligned ones 2 %).
template <bool kTwo, bool kOdd>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_w,
                       const __grid_constant__ LinearParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* staging = smem + kPairStages * kPairStageBytes;
  float* scale = reinterpret_cast<float*>(staging + kPairEpi * kRowStage);  // two groups of four blocks
  uint64_t* full = reinterpret_cast<uint64_t*>(scale + 2 * kPairScales);
  uint64_t* empty = full + kPairStages;
  uint64_t* t_empty = empty + kPairStages;
  uint64_t* s_full = t_empty + kPairBuffers;
  uint64_t* s_empty = s_full + 2;
  uint64_t* mma_done = s_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = kTwo ? (int)cluster_rank() & 1 : (int)cluster_rank();  // in the pair
  const int first_cta = kTwo ? (int)cluster_rank() & ~1 : 0;              // the pair's
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < kPairBuffers; ++i) mbar_init(&t_empty[i], 2 * kPairEpi);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kPairEpi);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_map(&map_q);
    prefetch_map(&map_w);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();  // both CTAs' barriers are there before either's copies complete on them
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  constexpr int kCtas = kTwo ? 4 : 2;
  const int pairs = gridDim.x / kCtas, tiles = P.m_tiles * P.n_tiles;
  const int b0 = kTwo && first_cta ? P.half : 0, own = kTwo ? (first_cta ? P.blocks : P.half) - b0 : 0;  // the pair's blocks
  auto steps = [&]() { return kTwo ? own : P.blocks; };
  int issued = 0;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      for (int t = blockIdx.x / kCtas; ok && t < tiles; t += pairs) {
        const int2 at = pair_tile(P, t);
        const int row = at.x * kPairM + 128 * rank, col = at.y * kPairN + kPairN / 2 * rank;
        for (int b = 0; b < steps(); ++b, ++issued) {
          const int st = issued % kPairStages;
          if (issued >= kPairStages && !(ok = mbar_wait(&empty[st], (issued / kPairStages - 1) & 1, abort_flag, P.wait_ns))) break;
#ifdef CSA_DEBUG_BOUNDS
          if (P.test_stall && b + 1 == steps() && t + pairs >= tiles) {
            ok = false;
            break;
          }
#endif
          uint8_t* dst = smem + st * kPairStageBytes;
          const uint32_t bar = cluster_map(&full[st], first_cta);  // which counts both CTAs' bytes
          if (leader) mbar_arrive_expect_tx(&full[st], 2 * kPairStageBytes);
          tma_load_2d_pair(dst, &map_q, (b0 + b) * kBlock, row, bar);
          tma_load_2d_pair(dst + kWBytes, &map_w, (b0 + b) * kBlock, col, bar);
        }
      }
    }
  } else if (warp == 1) {
    if (leader) {
      constexpr uint32_t idesc = idesc_e4m3(kPairM, kPairN);
      const bool one = elect_one();
      const uint64_t first = sw128_desc(smem_addr(smem));
      bool ok = true;
      int i = 0, st = 0, round = 0;
      for (int t = blockIdx.x / kCtas; ok && t < tiles; t += pairs)
        for (int b = 0; b < steps(); ++b, ++i) {
          const int buf = i % kPairBuffers;
          // (both polls under way at once: one behind the other they cost as much as a block's MMAs)
          const uint32_t pe = (i / kPairBuffers - 1) & 1, pf = round & 1;
          const bool e0 = i < kPairBuffers || mbar_try_wait_cluster(&t_empty[buf], pe), f0 = mbar_try_wait_cluster(&full[st], pf);
          if (!__all_sync(0xffffffffu, e0 && f0)) {
            ok = (e0 || mbar_wait<true>(&t_empty[buf], pe, abort_flag, P.wait_ns)) &&
                 (f0 || mbar_wait<true>(&full[st], pf, abort_flag, P.wait_ns));
            if (!(ok = __all_sync(0xffffffffu, ok) != 0)) break;
          }
          tc_fence_after();
          if (one) {
            const uint64_t a = first + (uint64_t)(st * (kPairStageBytes / 16)), w = a + kWBytes / 16;
#pragma unroll
            for (int k = 0; k < kBlock / 32; ++k) mma_e4m3_pair(tmem + buf * kPairN, a + 2 * k, w + 2 * k, idesc, k ? 1u : 0u);
            mma_commit_pair_multicast(&empty[st], 0x3 << first_cta);
          }
          __syncwarp();
          if (++st == kPairStages) st = 0, ++round;
        }
    }
  } else if (warp == 2) {
    // ---- scales: the products of a token's and the columns' scale, four blocks at a time (each of the epilogue's
    // threads reading its own token's took a fifth of the kernel's time: 32 lines a load)
    int group = 0;
    bool ok = true;
    for (int t = blockIdx.x / kCtas; ok && t < tiles; t += pairs) {
      const int2 at = pair_tile(P, t);
      static_assert(kPairN == kRowsN, "one scale a block for a tile's columns");
      const int row0 = at.x * kPairM + 128 * rank + lane;
      const float* w = P.w + (size_t)at.y * P.blocks;
      for (int b = 0; b < steps(); b += 4, ++group) {
        float4 v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = scales4(P, P.a + (size_t)min(row0 + 32 * x, P.T - 1) * P.blocks, b0 + b);
        const float4 u = scales4(P, w, b0 + b);
        ok = group < 2 || mbar_wait(&s_empty[group & 1], ((group >> 1) - 1) & 1, abort_flag, P.wait_ns);
        if (!(ok = __all_sync(0xffffffffu, ok) != 0)) break;
        float* to = scale + (group & 1) * kPairScales + lane;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          to[32 * x] = v[x].x * u.x, to[32 * x + 128] = v[x].y * u.y;
          to[32 * x + 256] = v[x].z * u.z, to[32 * x + 384] = v[x].w * u.w;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_full[group & 1]);
      }
    }
  } else {
    // ---- a warp has 32 tokens and 64 of the tile's columns
    const int quarter = warp & 3, col = kPairCols * ((warp - kPairFirst) >> 2);
    const uint32_t base = tmem + ((uint32_t)(32 * quarter) << 16) + col;
    uint8_t* stage = staging + (warp - kPairFirst) * kRowStage;
    const float* mine = scale + 32 * quarter + lane;
    const uint32_t freed = cluster_map(t_empty, first_cta);
    bool ok = true;
    int i = 0, st = 0, round = 0, group = 0;
    for (int t = blockIdx.x / kCtas; ok && t < tiles; t += pairs) {
      const int2 at = pair_tile(P, t);
      const int row0 = at.x * kPairM + 128 * rank + 32 * quarter, n0 = at.y * kPairN + col;
      float2 acc[kPairCols / 2];
#pragma unroll
      for (int c = 0; c < kPairCols / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
      for (int b = 0; b < steps(); ++b, ++i) {
        const int buf = i % kPairBuffers, j = b & 3;
        ok = j || mbar_wait_awake(&s_full[group & 1], (group >> 1) & 1, abort_flag, P.wait_ns);
        ok = ok && mbar_wait_awake(&empty[st], round & 1, abort_flag, P.wait_ns);
        if (!(ok = __all_sync(0xffffffffu, ok) != 0)) break;
        if (++st == kPairStages) st = 0, ++round;
        tc_fence_after();
        const float f = mine[(group & 1) * kPairScales + j * 128];
        const float2 f2 = make_float2(f, f);
        uint32_t r[kPairCols];
        tmem_ld64(base + buf * kPairN, r);
        // read: the buffer is free before the sums are done
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_relaxed(freed + 8 * buf);
#pragma unroll
        for (int k = 0; k < kPairCols; k += 2) acc[k / 2] = __ffma2_rn(f32_pair(r[k], r[k + 1]), f2, acc[k / 2]);
        if (j == 3 || b + 1 == steps()) {
          if (lane == 0) mbar_arrive(&s_empty[group & 1]);
          ++group;
        }
      }
      if (!ok) break;
      if constexpr (kTwo) {  // one tile: its part of the sums into the ring's place, which every copy and MMA has left
        float* const to = reinterpret_cast<float*>(smem) + (32 * quarter + lane) * kSumRow + col;
#pragma unroll
        for (int k = 0; k < kPairCols; k += 4)
          *reinterpret_cast<float4*>(to + k) = make_float4(acc[k / 2].x, acc[k / 2].y, acc[k / 2 + 1].x, acc[k / 2 + 1].y);
        break;
      }
      store_rows<kOdd>(P, acc, stage, row0, n0, P.N, lane);
    }
  }

  // ---- leave: as in the prefill's pairs (the leader's barriers count both CTAs' copies; what the other CTA
  // issued beyond what the leader expected is given time to land)
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (warp == 0 && lane == 0) {
      if (leader) {
        for (int t = max(0, issued - kPairStages); t < issued; ++t)
          mbar_wait_bounded(&full[t % kPairStages], (t / kPairStages) & 1);
      } else {
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 50000ull) __nanosleep(1000);
      }
    }
    if (warp == 1 && leader && elect_one()) {
      mma_commit_pair(mma_done);
      mbar_wait_bounded(mma_done, 0);
    }
    if (threadIdx.x == 0) atomicOr(&linear_flag, 4);
    tc_fence_before();
    __syncthreads();
  }
  cluster_arrive();
  cluster_wait();  // the leader's MMAs into this CTA's tensor memory and its arrivals here are over
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  if constexpr (kTwo) {
    // ---- both pairs' sums of half of this CTA's tokens, in the pairs' order
    const int2 at = pair_tile(P, blockIdx.x / kCtas);
    constexpr int kWarps = kPairThreads / 32, kRows = (64 + kWarps - 1) / kWarps;
    const float* const mine = reinterpret_cast<const float*>(smem) + 4 * lane;
    const int r0 = first_cta ? 64 : 0, t0 = at.x * kPairM + 128 * rank, n = at.y * kPairN + 4 * lane;
    float4 x[kRows][2];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (kWarps * i + warp < 64) x[i][p] = ld_cluster_f4(cluster_map(mine + (r0 + kWarps * i + warp) * kSumRow, 2 * p + rank));
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = kWarps * i + warp, t = t0 + r0 + r;
      if (r < 64 && t < P.T && n < P.N)
        store4(P, t, n, make_float4(x[i][0].x + x[i][1].x, x[i][0].y + x[i][1].y, x[i][0].z + x[i][1].z, x[i][0].w + x[i][1].w));
    }
    cluster_arrive();  // no CTA leaves while its sums are read
    cluster_wait();
  }
}

bool encode_rows(CUtensorMap* m, const void* base, long long rows, int K, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)K};
  cuuint32_t box[2] = {kBlock, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  return get_encode()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void*)base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters that the device runs at once: those of eight CTAs are fewer than its SMs would hold, since a cluster
// stays in one group of SMs (16 such clusters of 128 tokens took two rounds: 512 tokens of 4096 to 512 14.4 us, and 8.4 by
// clusters of four).  The runtime counts one CTA an SM where two fit; they do run (1 token of 8192 to 2048, 16 clusters of
// eight 6.7 us, of four 7.2).
long long clusters_at_once(std::atomic<int> (&known)[64], const void* kernel, int threads, int smem, int ctas) {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::atomic<int>& mine = known[dev & 63];  // one more than the number
  if (mine.load()) return mine.load() - 1;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
  mine.store(n + 1);
  return n;
}

template <int NT>
cudaError_t launch_tile(const uint8_t* q, const uint8_t* w, LinearParams P, cudaStream_t s) {
  const int K = P.blocks * kBlock;
  CUtensorMap mq, mw;
  const long long columns = (P.T + NT - 1) / NT;
  long long tiles = (P.N + kRowsN - 1) / kRowsN;
  // CTAs of a cluster: while they all fit at once, and a CTA keeps two blocks at least
  P.split = 1;
  static std::atomic<int> known[3][64];
  for (int i = 0; P.split < kMostSplit && P.blocks >= 4 * P.split &&
                  tiles * columns <= Tile<NT>::kCtas * clusters_at_once(known[i], (const void*)linear_tile_kernel<NT>, Tile<NT>::kThreads,
                                                                        Tile<NT>::kSmem, 2 * P.split);
       ++i)
    P.split *= 2;
  // 128 tokens: short sums over K rather by one CTA and fewer rows of W, since a cluster's sum costs 3 us (us, clusters and
  // fewer rows: 1024 features to 2048 5.8 and 4.9, to 8192 8.1 and 6.3; 2048 to 3000, by four, 7.6 and 7.4, to 8192, by two,
  // 9.3 and 8.1; 4096 to 6000, by two, 11.5 and 12.8).
  if (Tile<NT>::kTokenRows && (P.blocks <= 8 || (P.blocks <= 16 && P.split <= 4))) P.split = 1;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = P.split;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  // Where the last round of CTAs would be a part of one, tiles of fewer rows for as many rounds (128 tokens, us: of 4096 to
  // 20480 26.9 -> 23.9, to 32768 28.0 -> 27.4, of 7168 to 20000 41.1 -> 35.7); a multiple of 16, as the MMA's columns are.
  // (With W's rows as the MMA's rows a tile of fewer costs the same.)
  const int ctas = Tile<NT>::kCtas * current_sm_count();
  P.rows = kRowsN;
  if (Tile<NT>::kTokenRows && P.split == 1) {
    const long long most = (tiles * columns + ctas - 1) / ctas * ctas / columns, rows = ((P.N + most - 1) / most + 15) / 16 * 16;
    P.rows = (int)(rows > kRowsN ? kRowsN : rows < 32 ? 32 : rows);
    tiles = (P.N + P.rows - 1) / P.rows;
  }
  if (!encode_rows(&mq, q, P.T, K, NT) || !encode_rows(&mw, w, P.N, K, P.rows)) return cudaErrorInvalidValue;
  if (tiles * columns * P.split > kMostItems) return cudaErrorInvalidValue;
  P.columns = (int)columns;
  P.items = (int)(tiles * columns);
  cfg.gridDim = dim3((unsigned)(P.split > 1 ? P.items * P.split : P.items < ctas ? P.items : ctas));
  cfg.blockDim = dim3(Tile<NT>::kThreads);
  cfg.dynamicSmemBytes = Tile<NT>::kSmem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = P.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_tile_kernel<NT>, mq, mw, P);
}

cudaError_t launch_pair(const uint8_t* q, const uint8_t* w, LinearParams P, cudaStream_t s) {
  const int K = P.blocks * kBlock;
  CUtensorMap mq, mw;
  if (!encode_rows(&mq, q, P.T, K, 128) || !encode_rows(&mw, w, P.N, K, kPairN / 2)) return cudaErrorInvalidValue;
  const int sms = current_sm_count();
  P.m_tiles = (P.T + kPairM - 1) / kPairM;
  P.n_tiles = (P.N + kPairN - 1) / kPairN;
  const long long tiles = (long long)P.m_tiles * P.n_tiles;
  if (tiles > kMostItems) return cudaErrorInvalidValue;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  // Two pairs share a tile's blocks while all of them run at once and each has its part of the sum's time back (us with one
  // and with two, 256 tokens to 4096: 16384 features 34.1 and 22.8, 4096 11.7 and 10.8, 2048 8.0 and 8.7, 1024 6.1 and 7.4;
  // 512 tokens of 8192 to 2048 19.0 and 14.6).
  static std::atomic<int> known[64];
  P.split = P.blocks >= kPairSplitBlocks && tiles <= clusters_at_once(known, (const void*)linear_pair_kernel<true, false>, kPairThreads, kPairSmem, 4) ? 2 : 1;
  P.half = (P.blocks + 7) / 8 * 4;  // (a multiple of four: of scales that are read at once)
  at[1].val.clusterDim.x = 2 * P.split;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  const auto kernel = P.split == 2 ? linear_pair_kernel<true, false> : P.vec16 ? linear_pair_kernel<false, false> : linear_pair_kernel<false, true>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * P.split * (P.split == 2 || tiles < sms / 2 ? tiles : sms / 2)));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, mq, mw, P);
}

}  // namespace

// Pairs wherever the tiles of 128 x 128 could not each be split over four CTAs (us, pairs and tiles: 4096 tokens of 4096
// to 4096 60 and 113, 512 tokens 11.5 and 16.9, 256 tokens 10.8 and 13.3, 333 tokens of 4224 to 1000 11.4 and 8.3).
static bool use_pair(int T, int N) {
  return T > 128 && 4LL * ((T + 127) / 128) * ((N + 127) / 128) > current_sm_count();
}

cudaError_t launch_linear_q8(const uint8_t* q, const float* a, const uint8_t* w, const float* ws, int T, int N, int K, void* out,
                             bool f32, cudaStream_t s) {
  if (!get_encode()) return cudaErrorNotSupported;
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = once_per_device(attr, [] {  // (every kernel's at once: a later call may be captured)
    constexpr auto what = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t r = cudaFuncSetAttribute(linear_tile_kernel<16>, what, Tile<16>::kSmem);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(linear_tile_kernel<32>, what, Tile<32>::kSmem);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(linear_tile_kernel<64>, what, Tile<64>::kSmem);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(linear_tile_kernel<128>, what, Tile<128>::kSmem);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(linear_pair_kernel<false, false>, what, kPairSmem);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(linear_pair_kernel<false, true>, what, kPairSmem);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(linear_pair_kernel<true, false>, what, kPairSmem);
    return r;
  });
  if (e != cudaSuccess) return e;
  LinearParams P{};
  P.a = a;
  P.w = ws;
  P.out = out;
  P.T = T;
  P.N = N;
  P.blocks = K / kBlock;
  P.f32 = f32;
  P.vec = N % 4 == 0 && ((uintptr_t)out & (f32 ? 15 : 7)) == 0;
  P.vec_scales = P.blocks % 4 == 0 && (((uintptr_t)a | (uintptr_t)ws) & 15) == 0;
  P.vec2 = N % 2 == 0 && ((uintptr_t)out & 3) == 0;
  P.vec16 = (long long)N * (f32 ? 4 : 2) % 16 == 0 && ((uintptr_t)out & 15) == 0;
  P.wait_ns = kWaitNs;
#ifdef CSA_DEBUG_BOUNDS
  P.extent = (long long)T * N - (getenv("CSA_TEST_SHORT_EXTENTS") ? 1 : 0);
  P.test_stall = getenv("CSA_TEST_STALL_LAST_STAGE") != nullptr;
  if (P.test_stall) P.wait_ns = 200000000ull;
#endif
  if (use_pair(T, N)) return launch_pair(q, w, P, s);
  return T <= 16   ? launch_tile<16>(q, w, P, s)
         : T <= 32 ? launch_tile<32>(q, w, P, s)
         : T <= 64 ? launch_tile<64>(q, w, P, s)
                   : launch_tile<128>(q, w, P, s);
}

// Takes away the bits that were seen: a call on another stream may have raised one since, which is left to the next look.
// (The same bit raised again before it is taken away is reported by the look that had seen it.)
__global__ void clear_linear_flag_kernel(int seen) {
  griddep_wait();
  griddep_launch_dependents();
  atomicAnd(&linear_flag, ~seen);
}

// Reads and clears the device's flag behind the stream's work.
cudaError_t take_linear_flag(cudaStream_t s, int* flag) {
  *flag = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(flag, linear_flag, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess || !*flag) return e;
#ifdef CSA_DEBUG_BOUNDS
  // the test of this: a bit is raised between the look and the clearing
  if (const char* bits = getenv("CSA_TEST_RAISE_BEFORE_CLEARING")) {
    const int more = *flag | atoi(bits);
    e = cudaMemcpyToSymbolAsync(linear_flag, &more, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e != cudaSuccess) return e;
  }
#endif
  clear_linear_flag_kernel<<<1, 1, 0, s>>>(*flag);
  e = cudaGetLastError();
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace csa
