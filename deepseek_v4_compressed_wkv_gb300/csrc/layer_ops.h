// Launchers of the operators around the compressor (host side, enqueue only).
#pragma once

#include <type_traits>

#include "csa_internal.cuh"

namespace csa {

// Arguments of one attention call.  Prefill: token i of sequence b is row b * N + i of q and out,
// at position start + i, over rows 0 .. start + i of kv [B][kv_rows][D].  Decode (page_table in
// use, N = 1): the token is at position lens[b] - 1 over the cache's entries.
struct AttnCall {
  const uint16_t* q;
  uint16_t* out;
  float* lse;           // may be null
  const int32_t* lens;  // decode: entries; prefill: tokens, may be null
  const uint16_t* kv;   // prefill's rows
  csa_cache cache;      // decode's entries
  const int32_t* page_table;
  int max_pages;
  bool paged;
  int B, N, start, kv_rows;
};

long long attention_units(const csa_attention* a, const AttnCall& call);  // above 2^31 - 1: too large a call
cudaError_t launch_attention(csa_attention* a, const AttnCall& call, cudaStream_t s);
size_t attention_workspace_bytes(int head_dim);

// Launches a kernel that may be set up while the launch before it in the stream ends (it waits for that
// one, griddep_wait, before it touches memory): 2 of the 10 us that a small kernel takes in a stream.
// Such a kernel lets its own successor be set up only behind its wait, so that a kernel that has
// started finds everything before its direct predecessor complete (the compressor's decode reads its
// weights, and then its state, before it waits).  What it reads may be written by that launch while it
// already runs: such a kernel takes it by ordinary loads behind its wait, never by the non-coherent path
// (__ldg), which is for data that does not change during the kernel's life.
template <class... Params>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                         const std::remove_cv_t<Params>&... params) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, params...);
}

cudaError_t launch_cache_append(const csa_cache& cache, const csa_out& in, int B, int G, const int32_t* page_table,
                                int max_pages, const int32_t* first, const uint8_t* mask, int* status, cudaStream_t s);

cudaError_t launch_rmsnorm_residual_q8(const uint16_t* x, const uint16_t* residual, const float* gain, long long rows,
                                       int dim, float eps, int scale_block, uint16_t* residual_out, uint16_t* y,
                                       uint8_t* q, void* scales, cudaStream_t s);
#ifdef CSA_DEBUG_BOUNDS
cudaError_t take_norm_flag(cudaStream_t s, int* flag);  // the norm's stores outside their outputs
#endif

}  // namespace csa

struct csa_attention {
  int heads, D, window, sinks, device, sms;
  float scale;
  int* dev_flag;       // device-side error flag
  uint8_t* workspace;  // partial results of split sequences
  long long launches;  // kernels enqueued so far
};
