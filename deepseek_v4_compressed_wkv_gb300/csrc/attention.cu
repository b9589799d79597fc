// Attention over one shared key/value row per position (see include/csa.h): a prompt's tokens over
// their own rows with a window and sinks, or one new token over a paged cache.
#include "layer_ops.h"

namespace csa {
namespace {

struct AttnParams {
  AttnCall c;
  int H, D, window, sinks;
  float scale_log2;  // scale * log2(e): scores in base-2 exponents
  int* flag;
};

// Value pair (features 2i, 2i + 1) of an entry's row.
__device__ __forceinline__ float2 entry_pair(const AttnParams& P, long long row, int i) {
  const uint16_t* kv = P.c.paged ? P.c.cache.latent : P.c.kv;
  if (kv) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(kv + row * P.D + 2 * i);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  const uint32_t c = P.c.cache.codes[row * (P.D / 2) + i];
  const float s = e4m3_value(P.c.cache.scales[row * (P.D / 16) + i / 8]);
  return make_float2(e2m1_value(c & 15u) * s, e2m1_value(c >> 4) * s);
}

// One CTA of four warps per (token, head): each warp takes every fourth visible row with a running
// maximum and sum, lanes over feature pairs; the warps' results are joined at the end.
__global__ void __launch_bounds__(128) attention_kernel(const AttnParams P) {
  __shared__ float sm[4], sl[4];
  __shared__ float2 so[4][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long item = blockIdx.x / P.H;
  const int h = blockIdx.x % P.H, b = (int)(item / P.c.N), i = (int)(item % P.c.N);
  long long t;  // position of the query
  if (P.c.paged) {
    const long long top = (long long)P.c.max_pages * P.c.cache.page_size;
    const long long n = P.c.lens[b], m = n < 0 ? 0 : n > top ? top : n;
    if (m != n && threadIdx.x == 0) atomicOr(P.flag, 1);
    t = m - 1;
  } else {
    if (P.c.lens) {
      const int n = P.c.lens[b];
      if ((n < 0 || n > P.c.N) && threadIdx.x == 0) atomicOr(P.flag, 1);
      if (i >= n) return;
    }
    t = (long long)P.c.start + i;
  }
  // visible rows in order: the sinks, then the window
  const bool all = P.window == 0 || t + 1 <= (long long)P.window + P.sinks;
  const long long cnt = all ? t + 1 : (long long)P.window + P.sinks;
  const uint32_t* q = reinterpret_cast<const uint32_t*>(P.c.q + ((size_t)item * P.H + h) * P.D);
  const int np = P.D / 64;  // pairs a lane
  float2 qv[8], o[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    o[k] = make_float2(0.0f, 0.0f);
    const uint32_t w = k < np ? q[k * 32 + lane] : 0u;
    qv[k] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  float m = -INFINITY, l = 0.0f;
  for (long long v = warp; v < cnt; v += 4) {
    const long long j = all || v < P.sinks ? v : v - P.sinks + (t + 1 - P.window);
    long long row;
    if (P.c.paged) {
      const int p = P.c.page_table[(long long)b * P.c.max_pages + j / P.c.cache.page_size];
      if (p < 0 || p >= P.c.cache.pages) {
        if (lane == 0) atomicOr(P.flag, 2);
        continue;
      }
      row = (long long)p * P.c.cache.page_size + j % P.c.cache.page_size;
    } else {
      row = (long long)b * P.c.kv_rows + j;
    }
    float2 kv[8];
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      kv[k] = make_float2(0.0f, 0.0f);
      if (k < np) kv[k] = entry_pair(P, row, k * 32 + lane);
      s = fmaf(qv[k].x, kv[k].x, fmaf(qv[k].y, kv[k].y, s));
    }
    s = warp_sum(s) * P.scale_log2;
    const float mn = fmaxf(m, s), r = m == -INFINITY ? 0.0f : exp2f(m - mn), p = exp2f(s - mn);
    l = l * r + p;
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = make_float2(fmaf(p, kv[k].x, o[k].x * r), fmaf(p, kv[k].y, o[k].y * r));
    m = mn;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < np) so[warp][k * 32 + lane] = o[k];
  __syncthreads();
  float top = -INFINITY, sum = 0.0f, f[4];
  for (int w = 0; w < 4; ++w) top = fmaxf(top, sm[w]);
  for (int w = 0; w < 4; ++w) {
    f[w] = sm[w] == -INFINITY ? 0.0f : exp2f(sm[w] - top);
    sum += sl[w] * f[w];
  }
  const size_t out = (size_t)item * P.H + h;
  if (P.c.lse && threadIdx.x == 0)
    P.c.lse[out] = cnt == 0 ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
  for (int i2 = threadIdx.x; i2 < P.D / 2; i2 += 128) {
    float x = 0.0f, y = 0.0f;
    for (int w = 0; w < 4; ++w) x = fmaf(so[w][i2].x, f[w], x), y = fmaf(so[w][i2].y, f[w], y);
    const float inv = cnt == 0 ? 0.0f : 1.0f / sum;
    reinterpret_cast<uint32_t*>(P.c.out + out * P.D)[i2] = (uint32_t)bf16_bits(x * inv) | ((uint32_t)bf16_bits(y * inv) << 16);
  }
}

}  // namespace

size_t attention_workspace_bytes(int) { return 256; }

cudaError_t launch_attention(csa_attention* a, const AttnCall& call, cudaStream_t s) {
  AttnParams P{call, a->heads, a->D, a->window, a->sinks, (float)(a->scale * 1.4426950408889634), a->dev_flag};
  attention_kernel<<<(unsigned)((long long)call.B * call.N * a->heads), 128, 0, s>>>(P);
  a->launches += 1;
  return cudaGetLastError();
}

}  // namespace csa
