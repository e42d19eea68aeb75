// Device helpers of the paged attention kernels: a block's part of the work,
// partial results and their merge.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "internal.h"
#include "paged.h"
#include "paged_line.cuh"
#include "ptx.cuh"

namespace tilemix {

// A block's part of the line: from its own start to the next block's.  Two
// warps find them; every thread gets both.  False: nothing to do.
template <class L>
__device__ __forceinline__ bool find_part(const PagedArgs& p, const L& line,
                                          int warp, int lane, Cursor& begin,
                                          Cursor& end) {
  __shared__ Cursor s_part[2];
  if (warp < 2) {
    const Cursor at = line.locate(p, blockIdx.x + warp, gridDim.x, lane,
                                  blockIdx.x == 0 && warp == 0);
    if (lane == 0) s_part[warp] = at;
  }
  __syncthreads();
  begin = s_part[0];
  end = s_part[1];
  return !(same_item(begin, end) && begin.unit == end.unit);
}

// ---------------------------------------------------------------------------
// Partial results.  Slot 2 c: the item that began in an earlier block and
// goes on in (or ends with) block c; slot 2 c + 1: the item that begins in
// block c and goes on.  A slot holds R rows of {O[D] unnormalised, max (base
// 2), sum, -, -} and a header {used, the item ends here, first key on a bad
// page, rows} {first token row, first query head, group, the first token's
// limit_of_token}.
// ---------------------------------------------------------------------------

template <int D>
constexpr int kPartStride = D + 4;  // floats of a row

template <int D, int R>
__device__ __forceinline__ float* part_row(const PagedArgs& p, int slot,
                                           int row) {
  return p.part + (static_cast<size_t>(slot) * R + row) * kPartStride<D>;
}

__device__ __forceinline__ void clear_headers(const PagedArgs& p) {
  if (threadIdx.x < 2)
    p.head[2 * (2 * blockIdx.x + threadIdx.x)] = make_int4(0, 0, 0, 0);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  return pack_half2(lo, hi);
}

// The two 16-bit values of a packed pair, exactly.
template <bool BF16>
__device__ __forceinline__ float2 unpack_pair(uint32_t w) {
  if (BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Sum of the weights' sizes over the sum of what their rounding to 16 bits
// left: O of the rounded weights times it is a mean of V again.  Without it a
// row that one key dominates is off by that key's rounding (1.4 times the
// error of rounding the output alone).  Sizes, since INT8 scales may have
// either sign: every term is off by at most a half step, so the ratio is too.
__device__ __forceinline__ float round_off(float sum, float rounded) {
  return rounded != 0.0f ? sum / rounded : 1.0f;
}

// ln of 2^m l; -inf where nothing was summed.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l != 0.0f ? (m + log2f(l)) * 0.69314718055994530942f : -CUDART_INF_F;
}

constexpr float kNone = -__builtin_huge_valf();  // maximum of no keys
constexpr int kNoBadKey = 0x7fffffff;            // no key is on a bad page

// Running maximum m, sum l and output o of key ranges, added as
// m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m), o likewise.
template <int V>
struct Acc {
  float m, l, o[V];
  __device__ __forceinline__ void clear() {
    m = kNone;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
  }
  __device__ __forceinline__ void add(float mb, float lb, const float (&ob)[V]) {
    const float mn = fmaxf(m, mb);
    const float mz = mn == kNone ? 0.0f : mn;
    const float fa = ex2_approx(m - mz), fb = ex2_approx(mb - mz);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = o[i] * fa + ob[i] * fb;
    l = l * fa + lb * fb;
    m = mn;
  }
};

// Adds the partial results of the item that begins in block blockIdx.x and
// goes on in the next ones, in key order.  W warps share a row (each takes
// every W-th piece); a block of W * rows-per-block warps starts at row
// blockIdx.y * rows-per-block.  Bound by the latency of three dependent
// loads (headers, statistics and rows); rows of up to four pieces are in
// flight at once.
template <int D, bool BF16, int R, int W, int ROWS>
__global__ void __launch_bounds__(32 * W * ROWS)
    paged_merge_kernel(const __grid_constant__ PagedArgs p, int blocks) {
  constexpr int V = D / 32;  // channels of a lane
  __shared__ float s_acc[W > 1 ? W * ROWS : 1][D + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  const int r = blockIdx.y * ROWS + warp / W;
  const int wr = warp % W;
  pdl_wait();
  const int4 h = p.head[2 * (2 * c + 1)];
  if (!h.x || blockIdx.y * ROWS >= h.w) return;
  const int4 it = p.head[2 * (2 * c + 1) + 1];
  Acc<V> acc;
  acc.clear();
  int bad_key = h.z;
  bool done = false;
  auto load = [&](int slot, float& m, float& l, float (&o)[V]) {
    const float* x = part_row<D, R>(p, slot, r);
    m = x[D];
    l = x[D + 1];
    if (V == 4) {
      const float4 v = reinterpret_cast<const float4*>(x)[lane];
      o[0] = v.x, o[1] = v.y, o[V > 2 ? 2 : 0] = v.z, o[V > 3 ? 3 : 0] = v.w;
    } else {
      const float2 v = reinterpret_cast<const float2*>(x)[lane];
      o[0] = v.x, o[1] = v.y;
    }
  };
  const bool row = r < h.w;
  if (row && wr == 0) {
    float m, l, o[V];
    load(2 * c + 1, m, l, o);
    acc.add(m, l, o);
  }
  int k = 1;  // pieces seen
  for (int b0 = c + 1; b0 < blocks && !done; b0 += 32) {
    int4 n = make_int4(0, 0, 0, 0);
    if (b0 + lane < blocks) n = p.head[4 * (b0 + lane)];
    unsigned used = __ballot_sync(0xffffffffu, n.x != 0);
    const unsigned ends = __ballot_sync(0xffffffffu, n.x != 0 && n.y != 0);
    if (ends) {
      used &= 0xffffffffu >> (32 - __ffs(ends));
      done = true;
    }
    bad_key = min(bad_key, __reduce_min_sync(0xffffffffu, (used >> lane) & 1
                                                              ? n.z : kNoBadKey));
    while (used) {
      float m[4], l[4], o[4][V];
      int got = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // this warp's next piece
        int bit = -1;
        while (used) {
          const int t = __ffs(used) - 1;
          used &= used - 1;
          if (k++ % W == wr) {
            bit = t;
            break;
          }
        }
        if (bit >= 0 && row) {
          load(2 * (b0 + bit), m[j], l[j], o[j]);
          got = j + 1;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < got) acc.add(m[j], l[j], o[j]);
    }
  }
  if (W > 1) {
    float* s = s_acc[warp];
#pragma unroll
    for (int i = 0; i < V; ++i) s[lane * V + i] = acc.o[i];
    if (lane == 0) {
      s[D] = acc.m;
      s[D + 1] = acc.l;
    }
    __syncthreads();
    if (wr != 0) return;
    for (int w = 1; w < W; ++w) {
      const float* t = s_acc[warp + w];
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = t[lane * V + i];
      acc.add(t[D], t[D + 1], o);
    }
  }
  if (!done || !row) return;
  // a row that sees a key of a bad page keeps its outputs
  if (it.w + (p.causal ? r / it.z : 0) > bad_key) return;
  const int tok = it.x + r / it.z;
  const int hq = it.y + r % it.z;
  const float il = 1.0f / acc.l;
  uint32_t out[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i)
    out[i] = acc.l == 0.0f
                 ? 0u
                 : pack_pair<BF16>(acc.o[2 * i] * il, acc.o[2 * i + 1] * il);
  uint16_t* dst = p.out + (static_cast<int64_t>(tok) * p.hq + hq) * D;
  if (V == 4)
    reinterpret_cast<uint2*>(dst)[lane] = make_uint2(out[0], out[V / 2 - 1]);
  else
    reinterpret_cast<uint32_t*>(dst)[lane] = out[0];
  if (p.lse && lane == 0)
    p.lse[static_cast<int64_t>(hq) * p.total_tokens + tok] = lse_of(acc.m, acc.l);
}

// Launches the merge behind `blocks` blocks of an attention kernel on the
// same stream (it may be scheduled while that kernel drains).
template <int D, bool BF16, int R, int W, int ROWS>
cudaError_t launch_merge(const PagedArgs& a, int blocks, int rows,
                         cudaStream_t stream) {
  return launch_behind(paged_merge_kernel<D, BF16, R, W, ROWS>,
                       dim3(blocks, (rows + ROWS - 1) / ROWS), dim3(32 * W * ROWS),
                       0, stream, a, blocks);
}

// Workspace: headers first, then the partial rows.
inline void carve_workspace(PagedArgs& a, void* workspace, int blocks) {
  a.head = static_cast<int4*>(workspace);
  a.part = reinterpret_cast<float*>(a.head + 4 * blocks);
}

constexpr size_t workspace_of(int blocks, int rows, int head_dim) {
  return static_cast<size_t>(2 * blocks) *
         (static_cast<size_t>(rows) * (head_dim + 4) * sizeof(float) +
          2 * sizeof(int4));
}

}  // namespace tilemix
