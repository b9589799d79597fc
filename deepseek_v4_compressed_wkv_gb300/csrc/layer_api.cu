// C ABI of the operators around the compressor: argument checks and ownership.  Declared in
// include/csa.h.
#include <cmath>
#include <cstdio>
#include <new>

#include <nvtx3/nvToolsExt.h>

#include "layer_ops.h"

// Defined in api.cu: records the message returned by csa_last_error on this thread.
int csa_internal_fail(int code, const char* msg);

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

template <class... A>
int fail(int code, const char* fmt, A... a) {
  char buf[512];
  snprintf(buf, sizeof buf, fmt, a...);
  return csa_internal_fail(code, buf);
}
int fail(int code, const char* msg) { return csa_internal_fail(code, msg); }

int cuda_fail(cudaError_t e, const char* what) {
  return fail(CSA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

#define CSA_CUDA(call, what)                           \
  do {                                                 \
    cudaError_t e_ = (call);                           \
    if (e_ != cudaSuccess) return cuda_fail(e_, what); \
  } while (0)

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Checks the handle and that its device is the current one.
int check_handle(const csa_attention* a, const char* what) {
  if (!a) return fail(CSA_ERR_ARG, "%s: handle is NULL", what);
  int dev = -1;
  CSA_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev != a->device)
    return fail(CSA_ERR_ARG, "%s: the handle lives on device %d but device %d is current", what, a->device, dev);
  return CSA_OK;
}

int check_cache(const csa_cache* c, const char* what) {
  if (!c) return fail(CSA_ERR_ARG, "%s: cache is NULL", what);
  if (!c->latent && !c->codes) return fail(CSA_ERR_ARG, "%s: the cache has neither latent nor codes", what);
  if (!c->codes != !c->scales) return fail(CSA_ERR_ARG, "%s: codes and scales go together", what);
  if (c->codes && c->fp4 != 1 && c->fp4 != 2) return fail(CSA_ERR_ARG, "%s: fp4 %d must be 1 or 2", what, c->fp4);
  if (c->pages < 1 || c->pages > 0x7fffffffLL || c->page_size < 1)
    return fail(CSA_ERR_ARG, "%s: pages (%lld) must be in [1, 2^31) and page_size (%d) >= 1", what, (long long)c->pages,
                c->page_size);
  if (c->head_dim < 16 || c->head_dim > 512 || c->head_dim % (c->codes && c->fp4 == 2 ? 32 : 16))
    return fail(CSA_ERR_ARG, "%s: head_dim %d of the cache must be a multiple of %d in [16, 512]", what, c->head_dim,
                c->codes && c->fp4 == 2 ? 32 : 16);
  return CSA_OK;
}

// The steps' loops go up to 256 pages, slots or sequences past the last one before they end, as ints.
constexpr long long kMostPages = 0x7fffffffLL - 1023;

int check_pages(const csa_pages* t, const char* what) {
  if (!t) return fail(CSA_ERR_ARG, "%s: the page table is NULL", what);
  if (t->pages < 1 || t->sequences < 1 || t->max_pages < 1 || t->page_size < 1)
    return fail(CSA_ERR_ARG, "%s: pages (%d), sequences (%d), max_pages (%d) and page_size (%d) must be >= 1", what, t->pages,
                t->sequences, t->max_pages, t->page_size);
  if (t->pages > kMostPages || (long long)t->sequences * t->max_pages > kMostPages)
    return fail(CSA_ERR_ARG, "%s: pages and sequences * max_pages must be at most 2^31 - 1024", what);
  if ((long long)t->max_pages * t->page_size > 0x7fffffffLL)
    return fail(CSA_ERR_ARG, "%s: max_pages * page_size must be below 2^31", what);
  if (!t->refs || !t->table || !t->lens || !t->workspace)
    return fail(CSA_ERR_ARG, "%s: refs, table, lens and workspace are required", what);
  return CSA_OK;
}

}  // namespace

extern "C" {

int csa_cache_append(const csa_cache* cache, const csa_out* in, int B, int G, const int32_t* page_table, int max_pages,
                     const int32_t* first, const uint8_t* mask, int* status, csa_stream_t stream) {
  const char* what = "csa_cache_append";
  NvtxRange range(what);
  if (int rc = check_cache(cache, what)) return rc;
  if (B < 1 || G < 1 || (long long)B * G > 0x7fffffffLL)
    return fail(CSA_ERR_ARG, "%s: B (%d) and G (%d) must be >= 1 and B * G below 2^31", what, B, G);
  if (!in || (cache->latent && !in->latent) || (cache->codes && (!in->codes || !in->scales)))
    return fail(CSA_ERR_ARG, "%s: the entries lack an array that the cache has", what);
  if (max_pages < 1 || !page_table || !first) return fail(CSA_ERR_ARG, "%s: page_table and first are required", what);
  CSA_CUDA(csa::launch_cache_append(*cache, *in, B, G, page_table, max_pages, first, mask, status, (cudaStream_t)stream),
           "cache append launch");
  return CSA_OK;
}

int csa_attention_create(int heads, int head_dim, int window, int sinks, float scale, csa_attention** out) {
  if (!out) return fail(CSA_ERR_ARG, "csa_attention_create: out is NULL");
  *out = nullptr;
  if (heads < 1 || heads > 1024) return fail(CSA_ERR_ARG, "heads %d must be in [1, 1024]", heads);
  if (head_dim < 64 || head_dim > 512 || head_dim % 64)
    return fail(CSA_ERR_ARG, "head_dim %d must be a multiple of 64 in [64, 512]", head_dim);
  if (window < 0 || sinks < 0) return fail(CSA_ERR_ARG, "window (%d) and sinks (%d) must be >= 0", window, sinks);
  if (!(scale >= 0.0f) || std::isinf((float)(scale * 1.4426950408889634)))
    return fail(CSA_ERR_ARG, "scale must be >= 0 and, times log2(e), finite");
  auto* a = new (std::nothrow) csa_attention();
  if (!a) return fail(CSA_ERR_INTERNAL, "out of host memory");
  a->heads = heads;
  a->D = head_dim;
  a->window = window;
  a->sinks = window ? sinks : 0;
  a->scale = scale > 0.0f ? scale : (float)(1.0 / std::sqrt((double)head_dim));
  cudaError_t e = cudaGetDevice(&a->device);
  a->sms = csa::current_sm_count();
  if (e == cudaSuccess) e = cudaMalloc((void**)&a->dev_flag, sizeof(int));
  if (e == cudaSuccess) e = cudaMalloc((void**)&a->workspace, csa::attention_workspace_bytes(head_dim));
  if (e == cudaSuccess) e = cudaMemset(a->dev_flag, 0, sizeof(int));
  if (e == cudaSuccess) e = cudaMemset(a->workspace, 0, csa::attention_workspace_bytes(head_dim));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    cudaFree(a->dev_flag);
    cudaFree(a->workspace);
    delete a;
    return cuda_fail(e, "csa_attention_create");
  }
  *out = a;
  return CSA_OK;
}

int csa_attention_prefill(csa_attention* a, const uint16_t* q, const uint16_t* kv, int B, int N, int start_pos,
                          int kv_rows, const int32_t* lens, uint16_t* out, float* lse, csa_stream_t stream) {
  const char* what = "csa_attention_prefill";
  NvtxRange range(what);
  if (int rc = check_handle(a, what)) return rc;
  if (B < 1 || N < 1 || (long long)B * N * a->heads > 0x7fffffffLL)
    return fail(CSA_ERR_ARG, "%s: B (%d) and N (%d) must be >= 1 and B * N * heads below 2^31", what, B, N);
  if (start_pos < 0 || (long long)start_pos + N > 0x3fffffffLL)
    return fail(CSA_ERR_ARG, "%s: start_pos %d must be >= 0 and start_pos + N below 2^30", what, start_pos);
  if (kv_rows < start_pos + N)
    return fail(CSA_ERR_ARG, "%s: kv_rows %d must be at least start_pos + N = %d", what, kv_rows, start_pos + N);
  if ((long long)B * kv_rows > 0x7ffffffeLL)
    return fail(CSA_ERR_ARG, "%s: B * kv_rows must be below 2^31 - 1", what);
  if (!q || !kv || !out) return fail(CSA_ERR_ARG, "%s: q, kv and out are required", what);
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(out, 16))
    return fail(CSA_ERR_ARG, "%s: q, kv and out must be 16-byte aligned", what);
  csa::AttnCall c{};
  c.q = q;
  c.out = out;
  c.lse = lse;
  c.lens = lens;
  c.kv = kv;
  c.B = B;
  c.N = N;
  c.start = start_pos;
  c.kv_rows = kv_rows;
  if (csa::attention_units(a, c) > 0x7fffffffLL)
    return fail(CSA_ERR_ARG, "%s: too many tiles of 64 rows (items of 64 queries times rows / 64): 2^31 or more", what);
  CSA_CUDA(csa::launch_attention(a, c, (cudaStream_t)stream), "attention launch");
  return CSA_OK;
}

// A decode call's checks and launch; `more`: its groups of sequences that share entries, if any.
static int decode(csa_attention* a, const uint16_t* q, const csa_cache* cache, const int32_t* page_table, int max_pages,
                  const int32_t* lens, int B, const csa::AttnCall& more, uint16_t* out, float* lse, csa_stream_t stream,
                  const char* what) {
  if (int rc = check_handle(a, what)) return rc;
  if (int rc = check_cache(cache, what)) return rc;
  if (cache->head_dim != a->D)
    return fail(CSA_ERR_ARG, "%s: the cache holds %d features, the handle %d", what, cache->head_dim, a->D);
  if (!cache->latent && cache->fp4 != 1)
    return fail(CSA_ERR_ARG, "%s: codes must have e4m3 scales per 16 (fp4 = 1)", what);
  if (cache->pages > 0x7ffffffeLL / cache->page_size)
    return fail(CSA_ERR_ARG, "%s: the cache's entries must number less than 2^31 - 1", what);
  if (B < 1 || (long long)B * a->heads > 0x7fffffffLL) return fail(CSA_ERR_ARG, "%s: B (%d) must be >= 1", what, B);
  if (max_pages < 0 || (max_pages > 0 && !page_table))
    return fail(CSA_ERR_ARG, "%s: page_table is required", what);
  if ((long long)max_pages * cache->page_size > 0x3fffffffLL)
    return fail(CSA_ERR_ARG, "%s: max_pages * page_size must be below 2^30", what);
  if (!q || !lens || !out) return fail(CSA_ERR_ARG, "%s: q, lens and out are required", what);
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache->latent, 16) ||
      (!cache->latent && (!aligned(cache->codes, 16) || !aligned(cache->scales, 16))))
    return fail(CSA_ERR_ARG, "%s: q, out and the cache's arrays must be 16-byte aligned", what);
  csa::AttnCall c = more;
  c.q = q;
  if (c.part) {
    c.merged = out;
    c.merged_lse = lse;
    c.part_ml = (float2*)(c.part + 2LL * B * a->heads * a->D);
  } else {
    c.out = out;
    c.lse = lse;
  }
  c.lens = lens;
  c.cache = *cache;
  c.page_table = page_table;
  c.max_pages = max_pages;
  c.paged = true;
  c.B = B;
  c.N = 1;
  if (csa::attention_units(a, c) > 0x7fffffffLL)
    return fail(CSA_ERR_ARG, "%s: too many tiles of 64 rows (items of 64 queries times rows / 64): 2^31 or more", what);
  CSA_CUDA(csa::launch_attention(a, c, (cudaStream_t)stream), "attention launch");
  return CSA_OK;
}

int csa_attention_decode(csa_attention* a, const uint16_t* q, const csa_cache* cache, const int32_t* page_table,
                         int max_pages, const int32_t* lens, int B, uint16_t* out, float* lse, csa_stream_t stream) {
  const char* what = "csa_attention_decode";
  NvtxRange range(what);
  return decode(a, q, cache, page_table, max_pages, lens, B, csa::AttnCall{}, out, lse, stream, what);
}

int64_t csa_attention_shared_workspace(const csa_attention* a, int B, int G, int max_pages, int page_size) {
  if (!a) return fail(CSA_ERR_ARG, "handle is NULL");
  if (B < 1 || (long long)B * a->heads > 0x3fffffffLL || G < 1 || G > B)
    return fail(CSA_ERR_ARG, "csa_attention_shared_workspace: B (%d) must be >= 1, B * heads below 2^30, G (%d) in [1, B]", B, G);
  if (max_pages < 0 || page_size < 1 || (long long)max_pages * page_size > 0x3fffffffLL)
    return fail(CSA_ERR_ARG, "csa_attention_shared_workspace: max_pages * page_size must be in [0, 2^30)");
  return csa::shared_pays(a, B, G, (long long)max_pages * page_size) ? csa::shared_parts_bytes(B, a->heads, a->D) : 0;
}

int csa_attention_decode_shared(csa_attention* a, const uint16_t* q, const csa_cache* cache, const int32_t* page_table,
                                int max_pages, const int32_t* lens, int B, const int32_t* groups, const int32_t* shared, int G,
                                void* workspace, uint16_t* out, float* lse, csa_stream_t stream) {
  const char* what = "csa_attention_decode_shared";
  NvtxRange range(what);
  if (int rc = check_handle(a, what)) return rc;
  if (a->window) return fail(CSA_ERR_ARG, "%s: the handle has a window: only attention over all entries can share them", what);
  if (B < 1 || (long long)B * a->heads > 0x3fffffffLL)
    return fail(CSA_ERR_ARG, "%s: B (%d) must be >= 1 and B * heads below 2^30", what, B);
  if (G < 1 || G > B) return fail(CSA_ERR_ARG, "%s: G %d must be in [1, B]", what, G);
  if (!groups || !shared) return fail(CSA_ERR_ARG, "%s: groups and shared are required", what);
  if (int rc = check_cache(cache, what)) return rc;
  const bool pays = csa::shared_pays(a, B, G, (long long)(max_pages < 0 ? 0 : max_pages) * cache->page_size);
  if (pays && !workspace) return fail(CSA_ERR_ARG, "%s: workspace is required", what);
  if (!aligned(workspace, 16)) return fail(CSA_ERR_ARG, "%s: workspace must be 16-byte aligned", what);
  csa::AttnCall c{};
  c.groups = groups;
  c.shared = shared;
  c.G = G;
  c.part = pays ? (float*)workspace : nullptr;
  return decode(a, q, cache, page_table, max_pages, lens, B, c, out, lse, stream, what);
}

int csa_attention_status(csa_attention* a, csa_stream_t stream) {
  if (int rc = check_handle(a, "csa_attention_status")) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  int flag = 0;
  CSA_CUDA(cudaMemcpyAsync(&flag, a->dev_flag, sizeof(int), cudaMemcpyDeviceToHost, s), "read device flag");
  CSA_CUDA(cudaStreamSynchronize(s), "cudaStreamSynchronize");
  if (!flag) return CSA_OK;
  CSA_CUDA(cudaMemsetAsync(a->dev_flag, 0, sizeof(int), s), "clear device flag");
  return fail((flag & 4) ? CSA_ERR_TIMEOUT : CSA_ERR_DEVICE, "device flag 0x%x:%s%s%s%s", flag,
              (flag & 1) ? " a length out of range;" : "", (flag & 2) ? " a page outside the cache;" : "",
              (flag & 4) ? " wait budget exhausted;" : "", (flag & 8) ? " index out of bounds (bounds-checked build);" : "");
}

int64_t csa_attention_launches(const csa_attention* a) {
  if (!a) return fail(CSA_ERR_ARG, "handle is NULL");
  return a->launches;
}

void csa_attention_destroy(csa_attention* a) {
  if (!a) return;
  cudaDeviceSynchronize();
  cudaFree(a->dev_flag);
  cudaFree(a->workspace);
  delete a;
}

int csa_rmsnorm_residual_q8(const uint16_t* x, const uint16_t* residual, const float* gain, int64_t rows, int dim,
                            float eps, int scale_block, uint16_t* residual_out, uint16_t* y, uint8_t* q, void* scales,
                            csa_stream_t stream) {
  const char* what = "csa_rmsnorm_residual_q8";
  NvtxRange range(what);
  if (scale_block != 0 && scale_block != 32 && scale_block != 128)
    return fail(CSA_ERR_ARG, "%s: scale_block %d must be 0 (one scale per row), 32 or 128", what, scale_block);
  if (dim < 32 || dim > 16384 || dim % (scale_block == 128 ? 128 : 32))
    return fail(CSA_ERR_ARG, "%s: dim %d must be a multiple of %d, at most 16384", what, dim,
                scale_block == 128 ? 128 : 32);
  if (rows < 0 || rows > 0x7fffffffLL) return fail(CSA_ERR_ARG, "%s: rows must be in [0, 2^31)", what);
  if (!(eps >= 0.0f)) return fail(CSA_ERR_ARG, "%s: eps must be >= 0", what);
  if (rows == 0) return CSA_OK;  // nothing to do, nothing enqueued
  if (!x || !gain || !q || !scales) return fail(CSA_ERR_ARG, "%s: x, gain, q and scales are required", what);
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gain, 16) || !aligned(residual_out, 16) ||
      !aligned(y, 16) || !aligned(q, 16) || !aligned(scales, scale_block == 32 ? 1 : 4))
    return fail(CSA_ERR_ARG, "%s: the arrays must be 16-byte aligned", what);
  CSA_CUDA(csa::launch_rmsnorm_residual_q8(x, residual, gain, rows, dim, eps, scale_block, residual_out, y, q, scales,
                                           (cudaStream_t)stream),
           "rmsnorm launch");
#ifdef CSA_DEBUG_BOUNDS
  int flag = 0;
  CSA_CUDA(csa::take_norm_flag((cudaStream_t)stream, &flag), "rmsnorm bounds flag");
  if (flag) return fail(CSA_ERR_DEVICE, "%s: index out of bounds (bounds-checked build)", what);
#endif
  return CSA_OK;
}

int64_t csa_pages_workspace(int pages, int sequences, int max_pages) {
  if (pages < 1 || sequences < 1 || max_pages < 1 || pages > kMostPages || (long long)sequences * max_pages > kMostPages)
    return fail(CSA_ERR_ARG, "csa_pages_workspace: pages (%d), sequences (%d) and max_pages (%d) must be >= 1, pages and sequences * max_pages at most 2^31 - 1024",
                pages, sequences, max_pages);
  return csa::pages_workspace_ints(pages, sequences, max_pages);
}

int csa_pages_extend(const csa_pages* t, const int32_t* more, int32_t* first, csa_stream_t stream) {
  const char* what = "csa_pages_extend";
  NvtxRange range(what);
  if (int rc = check_pages(t, what)) return rc;
  if (!more || !first) return fail(CSA_ERR_ARG, "%s: more and first are required", what);
  CSA_CUDA(csa::launch_pages_extend(*t, more, first, (cudaStream_t)stream), "pages extend launch");
  return CSA_OK;
}

int csa_pages_fork(const csa_pages* t, const int32_t* parent, int32_t* src, int32_t* dst, int32_t* count, csa_stream_t stream) {
  const char* what = "csa_pages_fork";
  NvtxRange range(what);
  if (int rc = check_pages(t, what)) return rc;
  if (!parent || !src || !dst || !count) return fail(CSA_ERR_ARG, "%s: parent, src, dst and count are required", what);
  CSA_CUDA(csa::launch_pages_fork(*t, parent, src, dst, count, (cudaStream_t)stream), "pages fork launch");
  return CSA_OK;
}

int csa_pages_compact(const csa_pages* t, int32_t* src, int32_t* dst, int32_t* count, csa_stream_t stream) {
  const char* what = "csa_pages_compact";
  NvtxRange range(what);
  if (int rc = check_pages(t, what)) return rc;
  if (!src || !dst || !count) return fail(CSA_ERR_ARG, "%s: src, dst and count are required", what);
  CSA_CUDA(csa::launch_pages_compact(*t, src, dst, count, (cudaStream_t)stream), "pages compact launch");
  return CSA_OK;
}

int csa_cache_copy_pages(const csa_cache* cache, const int32_t* src, const int32_t* dst, int n, const int32_t* count, int* status,
                         csa_stream_t stream) {
  const char* what = "csa_cache_copy_pages";
  NvtxRange range(what);
  if (int rc = check_cache(cache, what)) return rc;
  if (n < 0) return fail(CSA_ERR_ARG, "%s: n %d must be >= 0", what, n);
  if (n == 0) return CSA_OK;  // nothing to do, nothing enqueued
  if (!src || !dst) return fail(CSA_ERR_ARG, "%s: src and dst are required", what);
  CSA_CUDA(csa::launch_copy_pages(*cache, src, dst, n, count, status, (cudaStream_t)stream), "page copy launch");
  return CSA_OK;
}

int csa_linear_q8(const uint8_t* q, const float* scales, const uint8_t* weight, const float* weight_scales, int64_t T, int N,
                  int K, void* out, int out_f32, csa_stream_t stream) {
  const char* what = "csa_linear_q8";
  NvtxRange range(what);
  if (K < 128 || K % 128) return fail(CSA_ERR_ARG, "%s: K %d must be a positive multiple of 128", what, K);
  if (N < 1 || N > 0x7fffff80) return fail(CSA_ERR_ARG, "%s: N %d must be in [1, 2^31 - 128]", what, N);
  if (T < 0 || T >= 1 << 22) return fail(CSA_ERR_ARG, "%s: T %lld must be in [0, 2^22)", what, (long long)T);
  if (out_f32 != 0 && out_f32 != 1) return fail(CSA_ERR_ARG, "%s: out_f32 %d must be 0 or 1", what, out_f32);
  if (T == 0) return CSA_OK;  // nothing to do, nothing enqueued
  if (((T + 15) / 16) * (((long long)N + 127) / 128) > 0x7fff0000LL / 8)
    return fail(CSA_ERR_ARG, "%s: too many tiles of 16 x 128 outputs: 2^28 or more", what);
  if (!q || !scales || !weight || !weight_scales || !out)
    return fail(CSA_ERR_ARG, "%s: q, scales, weight, weight_scales and out are required", what);
  if (!aligned(q, 16) || !aligned(weight, 16) || !aligned(scales, 4) || !aligned(weight_scales, 4) || !aligned(out, out_f32 ? 4 : 2))
    return fail(CSA_ERR_ARG, "%s: q and weight must be 16-byte aligned, the others by their type", what);
  CSA_CUDA(csa::launch_linear_q8(q, scales, weight, weight_scales, (int)T, N, K, out, out_f32 != 0, (cudaStream_t)stream),
           "linear launch");
  return CSA_OK;
}

int csa_linear_q8_status(csa_stream_t stream) {
  int flag = 0;
  CSA_CUDA(csa::take_linear_flag((cudaStream_t)stream, &flag), "linear flag");
  if (!flag) return CSA_OK;
  return fail((flag & 4) ? CSA_ERR_TIMEOUT : CSA_ERR_DEVICE, "device flag 0x%x:%s%s", flag, (flag & 4) ? " wait budget exhausted;" : "",
              (flag & 8) ? " index out of bounds (bounds-checked build);" : "");
}

}  // extern "C"
