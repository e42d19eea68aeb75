// Device helpers of the paged attention kernels: problem geometry, the split
// of all key work over the grid, partial results.
#pragma once

#include <cuda_runtime.h>
#include <math_constants.h>

#include "internal.h"
#include "paged.h"

namespace tilemix {

// One sequence as the kernels see it.  Packed row r of the sequence and a KV
// head is query head r % group of new token r / group.
struct SeqGeom {
  int start, n, len;  // first token row, new tokens, keys
};

// Sequence b; n = 0 when it has no new tokens or fails a check (reported
// once per block that looks at it when `report`).
__device__ __forceinline__ SeqGeom seq_geom(const PagedArgs& p, int b,
                                            bool report) {
  const int start = p.cu_seqlens[b];
  const int end = p.cu_seqlens[b + 1];
  const int len = p.kv_lens[b];
  const bool bad =
      start < 0 || end < start || end > p.total_tokens || len < 0 ||
      end - start > p.max_q_len || len > p.max_kv_len ||
      len > (static_cast<long long>(p.max_pages) << p.page_shift);
  if (bad) {
    if (report) report_status(p.status, kStatusBadSeqlens);
    return SeqGeom{0, 0, 0};
  }
  return SeqGeom{start, end - start, len};
}

// Keys that new token i sees.
__device__ __forceinline__ int keys_of_token(const PagedArgs& p,
                                             const SeqGeom& g, int i) {
  return p.causal ? max(0, g.len - g.n + i + 1) : g.len;
}

}  // namespace tilemix
