// The paged cache's write and the residual RMSNorm with an 8-bit output.
#include <cstdlib>

#include "layer_ops.h"
#include "tc_common.cuh"

namespace csa {
namespace {

using namespace tcx;

// ---------------------------------------------------------------------------------------
// Cache write: entry e = b * G + i of the call's rows to index first[b] + i of sequence b.
//
// Bytes are moved once; one warp per entry, each array's row as units of the widest type its
// addresses allow (a 512-wide latent is two 16-byte units a lane).  8 x 2048 latents of 512 features
// (33.6 MB) take 8.1 us in a graph of calls, which is also what a call costs its host; a decode step's 128
// entries 1.9 us, bound by the launch.  Entries and indices fit 32 bits: with 64-bit quotients the kernel
// ran twice as many instructions (10.2 us with them and without the early start).  Asking for the
// latent before its slot is looked up measured the same.

struct AppendParams {
  csa_cache cache;
  csa_out in;
  const int32_t* page_table;
  const int32_t* first;
  const uint8_t* mask;
  int* status;
  int B, G, max_pages;
  int lat_unit, code_unit, scale_unit;  // bytes moved at a time: 16, 8, 4, 2 or 1
  int lat_bytes, code_bytes, scale_bytes;
#ifdef CSA_DEBUG_BOUNDS
  long long rows;  // of the cache
#endif
};

template <class T>
__device__ __forceinline__ void copy_units(uint8_t* dst, const uint8_t* src, int bytes, int lane) {
  // (units loaded before the first store: the entries may be the cache's own memory as far as the compiler knows)
  constexpr int kAhead = 4;
  const int n = bytes / (int)sizeof(T);
  for (int i = lane; i < n; i += 32 * kAhead) {
    T v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + 32 * j < n) v[j] = reinterpret_cast<const T*>(src)[i + 32 * j];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + 32 * j < n) reinterpret_cast<T*>(dst)[i + 32 * j] = v[j];
  }
}

__device__ __forceinline__ void copy_row(uint8_t* dst, const uint8_t* src, int bytes, int unit, int lane) {
  if (unit == 16)
    copy_units<uint4>(dst, src, bytes, lane);
  else if (unit == 8)
    copy_units<uint2>(dst, src, bytes, lane);
  else if (unit == 4)
    copy_units<uint32_t>(dst, src, bytes, lane);
  else if (unit == 2)
    copy_units<uint16_t>(dst, src, bytes, lane);
  else
    copy_units<uint8_t>(dst, src, bytes, lane);
}

constexpr int kAppendWarps = 8;

__global__ void __launch_bounds__(kAppendWarps * 32) cache_append_kernel(const AppendParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t e = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);  // (B * G is below 2^31)
  if (e >= (uint32_t)P.B * (uint32_t)P.G) return;
  const uint32_t b = e / (uint32_t)P.G, i = e - b * (uint32_t)P.G;
  if (P.mask && !P.mask[b]) return;
  const long long index = (long long)P.first[b] + i;  // below 2^32
  const uint32_t j = (uint32_t)index, size = (uint32_t)P.cache.page_size, page = j / size;
  int bad = index < 0 ? 1 : page >= (uint32_t)P.max_pages ? 2 : 0;
  int p = 0;
  if (!bad) {
    p = P.page_table[(long long)b * P.max_pages + page];
    if (p < 0 || p >= P.cache.pages) bad = 4;
  }
  if (bad) {
    if (P.status && lane == 0) atomicOr(P.status, bad);
    return;
  }
  const long long row = (long long)p * size + (j - page * size);
#ifdef CSA_DEBUG_BOUNDS
  if (row < 0 || row >= P.rows) {  // (the status word, where the caller has one, stands in for a handle's flag)
    if (P.status && lane == 0) atomicOr(P.status, 8);
    return;
  }
#endif
  if (P.cache.latent)
    copy_row((uint8_t*)P.cache.latent + row * P.lat_bytes, (const uint8_t*)P.in.latent + (size_t)e * P.lat_bytes, P.lat_bytes,
             P.lat_unit, lane);
  if (P.cache.codes) {
    copy_row(P.cache.codes + row * P.code_bytes, P.in.codes + (size_t)e * P.code_bytes, P.code_bytes, P.code_unit, lane);
    copy_row(P.cache.scales + row * P.scale_bytes, P.in.scales + (size_t)e * P.scale_bytes, P.scale_bytes, P.scale_unit, lane);
  }
}

int common_unit(const void* a, const void* b, int bytes) {
  const uintptr_t u = (uintptr_t)a | (uintptr_t)b | (uintptr_t)bytes | 16;
  return (int)(u & (~u + 1));
}

// ---------------------------------------------------------------------------------------
// Residual addition, RMSNorm and e4m3 quantisation.
//
// One pass: a row is held in registers (8 features a thread and piece, piece i at feature
// 8 * (i * T + t), so that a block's scale is a maximum over 4 or 16 adjacent threads), its sum of
// squares and, with one scale per row, its maximum are reduced over the T threads, and every
// output is written from the registers.  The sum, the mean, the normalised values, the scales and
// the products with a scale's reciprocal are f32.
//
// 9 bytes a feature move through HBM, which bounds it: 16461 rows of 4096 with scales per 128 take
// 95 us (609 MB, 6.4 TB/s, 95 % of a copy's).  Every load of a thread is asked for before the first value is used:
// with each piece's residual stored before the next piece's loads, and eight divisions a piece, the
// same rows took 112 us.  Two pieces a thread: one (512 threads, two CTAs' worth of them waiting at
// each reduction) takes 134 us, four (a third of the warps) 114 us.  128 rows take 2.8 us in a graph of calls, bound by the launch.

struct NormParams {
  const uint16_t* x;
  const uint16_t* residual;
  const float* gain;
  uint16_t* residual_out;
  uint16_t* y;
  uint8_t* q;
  void* scales;
  long long rows;
  int dim;
  float eps;
#ifdef CSA_DEBUG_BOUNDS
  long long extent;  // rows that the outputs have
#endif
};

// The bounds-checked build's check of a store to element i of an output of `per` elements a row; the
// operator has no handle whose flag could be raised, so this build keeps one of its own.
#ifdef CSA_DEBUG_BOUNDS
__device__ int norm_flag;
__device__ __forceinline__ bool in_output(const NormParams& P, long long i, long long per) {
  return in_bounds(i, P.extent * per, &norm_flag);
}
#else
__device__ __forceinline__ bool in_output(const NormParams&, long long, long long) { return true; }
#endif

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
  return (uint32_t)bf16_bits(lo) | ((uint32_t)bf16_bits(hi) << 16);
}
// The maximum, NaN if either is (a row's NaN shows in its scale).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 448.0f * 1.17549435082228750797e-38f;  // 448 * 2^-126: the scale stays normal

// The power-of-two scale for amax: the smallest power of two >= max(amax, floor) / 448; *byte is its
// e8m0 encoding (255: NaN).
__device__ __forceinline__ float e4m3_pow2_scale(float amax, uint32_t* byte) {
  const float a = __fdiv_rn(max_nan(amax, kAmaxFloor), kE4m3Max);
  const uint32_t u = __float_as_uint(a);
  const uint32_t e = min((u >> 23) + ((u & 0x7FFFFFu) != 0u ? 1u : 0u), 255u);
  *byte = e;
  return e == 255u ? __int_as_float(0x7fffffff) : __uint_as_float(e << 23);
}

// A row's outputs are not read again here; its inputs are read once.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// BLOCK: features per scale (32, 128, 0 for the row).  PIECES: 8-feature pieces a thread.
template <int BLOCK, int PIECES>
__global__ void __launch_bounds__(1024) rmsnorm_q8_kernel(const NormParams P) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float red[2][32];
  const int T = blockDim.x, t = threadIdx.x, lane = t & 31, warp = threadIdx.y * (T >> 5) + (t >> 5);
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < P.rows;
  const long long base = row * P.dim;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 x[PIECES], r[PIECES];
  float4 g[PIECES][2];  // (asked for before the sum is known)
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int f = 8 * (i * T + t);
    const bool act = live && f < P.dim;
    x[i] = act ? load16(P.x + base + f) : zero;
    r[i] = act && P.residual ? load16(P.residual + base + f) : zero;
  }
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int f = 8 * (i * T + t);
    const bool act = live && f < P.dim;
    const float4* gp = reinterpret_cast<const float4*>(P.gain + f);
    g[i][0] = act ? gp[0] : make_float4(0, 0, 0, 0);
    g[i][1] = act ? gp[1] : make_float4(0, 0, 0, 0);
  }
  float s[PIECES][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, v[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s[i][2 * k] = bf_lo(w[k]) + bf_lo(v[k]);
      s[i][2 * k + 1] = bf_hi(w[k]) + bf_hi(v[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(s[i][k], s[i][k], ss);
  }
  if (P.residual_out) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int f = 8 * (i * T + t);
      if (live && f < P.dim && in_output(P, base + f, P.dim))
        __stcs(reinterpret_cast<uint4*>(P.residual_out + base + f),
               make_uint4(bf_pack(s[i][0], s[i][1]), bf_pack(s[i][2], s[i][3]), bf_pack(s[i][4], s[i][5]),
                          bf_pack(s[i][6], s[i][7])));
    }
  }
  ss = warp_sum(ss);
  if (T > 32) {
    if (lane == 0) red[0][warp] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int w = 0; w < (T >> 5); ++w) ss += red[0][threadIdx.y * (T >> 5) + w];
  }
  const float inv = 1.0f / sqrtf(ss / (float)P.dim + P.eps);
  float amax[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int f = 8 * (i * T + t);
    const float gk[8] = {g[i][0].x, g[i][0].y, g[i][0].z, g[i][0].w, g[i][1].x, g[i][1].y, g[i][1].z, g[i][1].w};
    amax[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      s[i][k] = s[i][k] * inv * gk[k];
      amax[i] = max_nan(amax[i], fabsf(s[i][k]));
    }
    if (P.y && live && f < P.dim && in_output(P, base + f, P.dim))
      __stcs(reinterpret_cast<uint4*>(P.y + base + f),
             make_uint4(bf_pack(s[i][0], s[i][1]), bf_pack(s[i][2], s[i][3]), bf_pack(s[i][4], s[i][5]),
                        bf_pack(s[i][6], s[i][7])));
  }
  if (BLOCK == 0) {
    float m = amax[0];
#pragma unroll
    for (int i = 1; i < PIECES; ++i) m = max_nan(m, amax[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (T > 32) {
      if (lane == 0) red[1][warp] = m;
      __syncthreads();
      for (int w = 0; w < (T >> 5); ++w) m = max_nan(m, red[1][threadIdx.y * (T >> 5) + w]);
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) amax[i] = m;
  }
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int f = 8 * (i * T + t);
    float a, m = amax[i];
    constexpr int kLanes = BLOCK / 8;  // adjacent threads of a block, in one warp and live together
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    uint32_t byte = 0;
    if (BLOCK == 32)
      a = e4m3_pow2_scale(m, &byte);
    else
      a = __fdiv_rn(max_nan(m, kAmaxFloor), kE4m3Max);
    if (!live || f >= P.dim) continue;
    if (BLOCK == 32) {
      if ((t & (kLanes - 1)) == 0 && in_output(P, row * (P.dim / 32) + f / 32, P.dim / 32))
        reinterpret_cast<uint8_t*>(P.scales)[row * (P.dim / 32) + f / 32] = (uint8_t)byte;
    } else if (BLOCK == 128) {
      if ((t & (kLanes - 1)) == 0 && in_output(P, row * (P.dim / 128) + f / 128, P.dim / 128))
        reinterpret_cast<float*>(P.scales)[row * (P.dim / 128) + f / 128] = a;
    } else if (f == 0 && in_output(P, row, 1)) {
      reinterpret_cast<float*>(P.scales)[row] = a;
    }
    // One reciprocal for the block's quotients: 2^-126 <= a <= 2^120, so it is a normal number.
    const float back = __frcp_rn(a);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = __nv_cvt_float2_to_fp8x2(make_float2(s[i][2 * k] * back, s[i][2 * k + 1] * back), __NV_SATFINITE, __NV_E4M3);
    if (in_output(P, base + f, P.dim))
      __stcs(reinterpret_cast<uint2*>(P.q + base + f), make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16)));
  }
}

template <int BLOCK>
cudaError_t launch_norm(const NormParams& P, cudaStream_t s) {
  // threads of a row: a warp up to 256 features, else two pieces a thread (1024 threads at 16384)
  const int units = P.dim / 8;
  const int pieces = units > 32 ? 2 : 1;
  const int T = (units + 32 * pieces - 1) / (32 * pieces) * 32;
  const int R = T >= 256 ? 1 : min(8, 256 / T);  // rows of a CTA
  const dim3 block(T, R), grid((unsigned)((P.rows + R - 1) / R));
  return launch_early(pieces == 1 ? rmsnorm_q8_kernel<BLOCK, 1> : rmsnorm_q8_kernel<BLOCK, 2>, grid, block, 0, s, P);
}

}  // namespace

cudaError_t launch_cache_append(const csa_cache& cache, const csa_out& in, int B, int G, const int32_t* page_table,
                                int max_pages, const int32_t* first, const uint8_t* mask, int* status, cudaStream_t s) {
  AppendParams P{};
  P.cache = cache;
  P.in = in;
  P.page_table = page_table;
  P.first = first;
  P.mask = mask;
  P.status = status;
  P.B = B;
  P.G = G;
  P.max_pages = max_pages;
#ifdef CSA_DEBUG_BOUNDS
  P.rows = cache.pages * cache.page_size - (getenv("CSA_TEST_SHORT_EXTENTS") ? 1 : 0);
#endif
  P.lat_bytes = cache.head_dim * 2;
  P.code_bytes = cache.head_dim / 2;
  P.scale_bytes = cache.head_dim / fp4_scale_block(cache.fp4);
  P.lat_unit = common_unit(cache.latent, in.latent, P.lat_bytes);
  P.code_unit = common_unit(cache.codes, in.codes, P.code_bytes);
  P.scale_unit = common_unit(cache.scales, in.scales, P.scale_bytes);
  const long long n = (long long)B * G;
  return launch_early(cache_append_kernel, dim3((unsigned)((n + kAppendWarps - 1) / kAppendWarps)), dim3(kAppendWarps * 32), 0, s, P);
}

cudaError_t launch_rmsnorm_residual_q8(const uint16_t* x, const uint16_t* residual, const float* gain, long long rows,
                                       int dim, float eps, int scale_block, uint16_t* residual_out, uint16_t* y,
                                       uint8_t* q, void* scales, cudaStream_t s) {
  NormParams P{x, residual, gain, residual_out, y, q, scales, rows, dim, eps};
#ifdef CSA_DEBUG_BOUNDS
  P.extent = rows - (getenv("CSA_TEST_SHORT_EXTENTS") ? 1 : 0);
#endif
  return scale_block == 32 ? launch_norm<32>(P, s) : scale_block == 128 ? launch_norm<128>(P, s) : launch_norm<0>(P, s);
}

#ifdef CSA_DEBUG_BOUNDS
// Reads and clears the flag behind the stream's work; 0 while the stream is captured.
cudaError_t take_norm_flag(cudaStream_t s, int* flag) {
  *flag = 0;
  cudaStreamCaptureStatus capture;
  cudaError_t e = cudaStreamIsCapturing(s, &capture);
  if (e != cudaSuccess || capture != cudaStreamCaptureStatusNone) return e;
  const int zero = 0;
  e = cudaMemcpyFromSymbolAsync(flag, norm_flag, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && *flag) e = cudaMemcpyToSymbolAsync(norm_flag, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}
#endif

}  // namespace csa
