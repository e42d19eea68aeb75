// Launch interface of the rotary / paged-cache kernels between the C entry
// points (paged_api.cu) and the kernels.  Not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tilemix {

constexpr int kStatusBadPages = 7;  // TILEMIX_ERR_BAD_PAGES

// Rows of 16-bit channels: a [T, heads, d] tensor with strides (elements).
struct RowTensor {
  uint16_t* p;
  int64_t st, sh;
};

// One launch of the rotary / append kernel.  The heads of all tensors count
// through: hq query heads, hk key heads, then hv value heads.
struct RopeArgs {
  RowTensor q, q_out;  // rotated q -> q_out (hq may be 0)
  RowTensor k, k_out;  // rotary call: rotated k -> k_out
  RowTensor v;         // append only
  const int32_t* positions;
  const double* freqs;  // nullptr: no rotation (append)
  float attn_factor;    // never 0
  float sign;           // +1, or -1 for the inverse rotation
  int total_tokens, hq, hk, hv, head_dim, rot_dim;
  int interleaved;
  // append: destination of k and v rows
  void* k_pages;
  void* v_pages;
  int64_t page_stride, token_stride, head_stride;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* cu_seqlens;
  const int32_t* kv_lens;
  int batch, num_pages, page_shift, max_pages;
  int32_t* status;
};

// mode: 0 rotary call, 1 append to 16-bit pages, 2 append to INT8 pages.
cudaError_t launch_rope(const RopeArgs& a, bool bf16, int mode,
                        cudaStream_t stream);

// Everything the paged attention kernels read; passed as a __grid_constant__
// parameter.
struct PagedArgs {
  CUtensorMap tm_k, tm_v;  // {d, page_size, hkv, num_pages}
  const uint16_t* q;
  int64_t q_st, q_sh;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* cu_seqlens;
  const int32_t* kv_lens;
  int batch, total_tokens, max_q_len, max_kv_len;
  int hq, hkv, group;  // group = hq / hkv
  int num_pages, page_shift, max_pages;
  int causal;
  float scale_log2;  // softmax scale * log2(e)
  int test_expire_wait;  // a first tile's barrier never completes
  uint16_t* out;
  float* lse;
  int32_t* status;
  // partial results (paged_common.cuh)
  float* part;
  int4* head;
};

struct PagedShape {
  int head_dim;
  bool bf16, int8;
};

// Keys that one copy of the step kernel's ring brings at most.
constexpr int paged_step_group(int head_dim, bool int8) {
  return head_dim == 128 && !int8 ? 16 : 32;
}

// Launches a kernel that may be scheduled while the one before it on the
// stream drains; it has to wait (pdl_wait) before it touches memory.
template <class... P, class... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                          cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The step kernel (16 packed rows a pass) and the chunk kernel (256); each has
// its own workspace size.
size_t paged_step_workspace_bytes(int head_dim);
size_t paged_chunk_workspace_bytes(int head_dim);

cudaError_t launch_paged_step(const PagedArgs& a, const PagedShape& s,
                              void* workspace, cudaStream_t stream);
cudaError_t launch_paged_chunk(const PagedArgs& a, const PagedShape& s,
                               void* workspace, cudaStream_t stream);

}  // namespace tilemix
