// Rotary positions of Q and K, and the append of new K / V rows to the pages
// of the cache (rotated on the way, 16-bit or INT8).
//
// Mathematics.  Pair i of a token at position p turns by a = p f_i: (x_a,
// x_b) -> (x_a c - x_b s, x_b c + x_a s).  The angle is formed in double, p
// f_i / 2 pi is reduced to [-1/2, 1/2] turns there, and only the remainder
// becomes fp32, so the rotation of position 10^6 is as exact as that of 10.
// INT8 rows take absmax times fl(1 / 127) over their d channels (of the row as
// rounded to 16 bits, so that append(x) after a rotary call and the fused
// append agree bit for bit) and the quantiser's code definition for that scale
// (quant_code.cuh; |x / scale| stays below 127.0001).
//
// What bounds it: memory traffic (INT8: instructions).  One block takes a few
// tokens: its threads first make the tokens' cosines and sines (shared by all
// heads) in shared memory, then every thread walks units of two 16-byte
// vectors, which hold eight whole pairs in either layout, over the heads of
// its token.  Rotating 32768 tokens of 24 + 8 heads, d 128: 92-97 us, 5.5-5.8
// TB/s; the same with appending 16 prompts of 28 + 2 x 4 heads 244 us, 5.9
// TB/s; 32768 tokens of 2 x 32 heads to INT8 pages 165 us, 4.9 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "paged.h"
#include "ptx.cuh"
#include "quant_code.cuh"

namespace tilemix {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // of a block
constexpr double kInvTwoPi = 0.15915494309189533577;
constexpr float kInv127 = 1.0f / 127.0f;

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      half2_bits_to_float2(w[i], f[2 * i], f[2 * i + 1]);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rotates the eight pairs of a unit.  HALF: a holds the pairs' first
// channels, b their second ones; INTERLEAVED: a is pairs 0..3, b pairs 4..7.
// One product rounds before the fused multiply-add, as written.
__device__ __forceinline__ void turn1(float& x, float& y, float2 t) {
  const float nx = __fmaf_rn(x, t.x, -__fmul_rn(y, t.y));
  const float ny = __fmaf_rn(y, t.x, __fmul_rn(x, t.y));
  x = nx;
  y = ny;
}

__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8],
                                     const float2* cs, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn1(a[2 * i], a[2 * i + 1], cs[i]);
      turn1(b[2 * i], b[2 * i + 1], cs[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn1(a[i], b[i], cs[i]);
  }
}

// The last sequence whose start is <= t (a warp looks at 32 starts a step);
// always in [0, batch).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch,
                                             int t, int lane) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const unsigned below =
        __ballot_sync(0xffffffffu, i < hi && cu[i] <= t);
    // starts do not decrease in a valid call, so the set bits are the low
    // ones; a decreasing cu_seqlens only changes which sequence is checked
    const int n = max(__popc(below) - 1, 0);
    lo = lo + n * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

// What an append refuses a sequence for.
__device__ __forceinline__ bool bad_sequence(const RopeArgs& p, int start,
                                             int end, int len) {
  return start < 0 || end < start || end > p.total_tokens || len < end - start ||
         len > (static_cast<long long>(p.max_pages) << p.page_shift);
}

// Where a token's rows go (append): page id and slot, or page < 0.
struct Place {
  int page, slot, pos;
  int64_t at, scale_at;  // INT8: head 0's row and scale
};

template <bool BF16, int MODE>  // 0 rotary, 1 append 16-bit, 2 append INT8
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const __grid_constant__ RopeArgs p, int tokens_per_block) {
  extern __shared__ float2 cs_all[];  // [tokens_per_block][rot_dim / 2]
  __shared__ Place place[kMaxTokens];
  pdl_wait();
  const int t0 = blockIdx.x * tokens_per_block;
  const int nt = min(tokens_per_block, p.total_tokens - t0);
  const int half = p.rot_dim >> 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (MODE != 0) {
    // Block 0 looks every sequence over, those without new tokens included (by
    // its last warps, which have no token to place in a small call).
    if (blockIdx.x == 0 && p.status)
      for (int b = static_cast<int>(threadIdx.x) - kThreads / 2; b < p.batch;
           b += kThreads / 2) {
        if (b < 0) break;
        const int start = p.cu_seqlens[b], end = p.cu_seqlens[b + 1];
        if (bad_sequence(p, start, end, p.kv_lens[b]))
          report_status(p.status, kStatusBadSeqlens);
      }
    // one warp per token finds its sequence and checks its place
    for (int tt = warp; tt < nt; tt += kThreads / 32) {
      const int t = t0 + tt;
      Place pl{-1, 0, 0, 0, 0};
      if (t < p.cu_seqlens[p.batch]) {
        const int b = find_sequence(p.cu_seqlens, p.batch, t, lane);
        const int start = p.cu_seqlens[b], end = p.cu_seqlens[b + 1];
        const int len = p.kv_lens[b];
        const long long pos = static_cast<long long>(len) - (end - start) + (t - start);
        if (t < start || t >= end || bad_sequence(p, start, end, len)) {
          // (before the first sequence: padding)
          if (lane == 0 && !(b == 0 && t < start))
            report_status(p.status, kStatusBadSeqlens);
        } else {
          const int page =
              p.page_table[b * p.table_stride + (pos >> p.page_shift)];
          if (page < 0 || page >= p.num_pages) {
            if (lane == 0) report_status(p.status, kStatusBadPages);
          } else {
            const int slot = static_cast<int>(pos & ((1 << p.page_shift) - 1));
            pl = Place{page, slot, static_cast<int>(pos),
                       page * p.page_stride + slot * p.token_stride,
                       (static_cast<int64_t>(page) * p.hk << p.page_shift) + slot};
          }
        }
      }
      if (lane == 0) place[tt] = pl;
    }
    __syncthreads();
  }
  if (p.freqs) {
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int tt = i / half, j = i - tt * half;
      int pos;
      if (MODE != 0) {
        if (place[tt].page < 0) continue;
        pos = p.positions ? p.positions[t0 + tt] : place[tt].pos;
      } else {
        pos = p.positions[t0 + tt];
      }
      const double turns = static_cast<double>(pos) * p.freqs[j] * kInvTwoPi;
      const float r = static_cast<float>(turns - rint(turns));
      float s, c;
      sincospif(2.0f * r, &s, &c);
      cs_all[i] = make_float2(c * p.attn_factor, s * p.attn_factor * p.sign);
    }
  }
  __syncthreads();

  // Units of a head: rot_dim / 16 rotated ones, then pass-through pairs of
  // vectors.  A head's units sit on neighbouring threads.
  const int units = p.head_dim >> 4;
  const int rot_units = p.freqs ? p.rot_dim >> 4 : 0;
  const int slots = kThreads / units;  // heads in flight
  const int u = threadIdx.x % units;
  const int slot0 = threadIdx.x / units;
  const int heads = p.hq + p.hk + p.hv;
  const bool rotated = u < rot_units;
  // first and second vector of the unit (in vectors of 8 channels)
  int v0, v1;
  if (rotated && !p.interleaved) {
    v0 = u;
    v1 = u + rot_units;
  } else {
    v0 = 2 * u;
    v1 = 2 * u + 1;
  }
  if constexpr (MODE != 2) {
    // Tokens outside, heads inside: a block's reads are neighbours (heads
    // outside took 1.2 times as long).
    for (int tt = 0; tt < nt; ++tt) {
      if (MODE != 0 && place[tt].page < 0) continue;
      const int64_t t = t0 + tt;
      const float2* cs = cs_all + tt * half + 8 * u;
      for (int h0 = 0; h0 < heads; h0 += slots) {
        const int h = h0 + slot0;
        const bool live = slot0 < slots && h < heads;
        const bool is_q = h < p.hq, is_v = h >= p.hq + p.hk;
        const int hl = is_q ? h : is_v ? h - p.hq - p.hk : h - p.hq;
        const RowTensor in = is_q ? p.q : is_v ? p.v : p.k;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (live) {
          const uint4* src =
              reinterpret_cast<const uint4*>(in.p + t * in.st + hl * in.sh);
          a = src[v0];
          b = src[v1];
        }
        if (rotated && !is_v) {
          float fa[8], fb[8];
          unpack8<BF16>(a, fa);
          unpack8<BF16>(b, fb);
          turn(fa, fb, cs, p.interleaved != 0);
          a = pack8<BF16>(fa);
          b = pack8<BF16>(fb);
        }
        if (MODE == 0 || is_q) {
          if (live) {
            const RowTensor out = is_q ? p.q_out : p.k_out;
            uint4* dst = reinterpret_cast<uint4*>(out.p + t * out.st + hl * out.sh);
            dst[v0] = a;
            dst[v1] = b;
          }
          continue;
        }
        const int64_t at = place[tt].page * p.page_stride +
                           place[tt].slot * p.token_stride + hl * p.head_stride;
        if (live) {
          uint4* dst = reinterpret_cast<uint4*>(
              static_cast<uint16_t*>(is_v ? p.v_pages : p.k_pages) + at);
          dst[v0] = a;
          dst[v1] = b;
        }
      }
    }
  } else {
    // INT8 rows are bound by instructions, not by HBM: a thread keeps its head
    // over the block's tokens, so that addresses cost an addition a token, and
    // the next token's loads are in flight meanwhile (tokens outside: 208 us
    // where this takes 174).  Every lane runs the same rounds, since rows
    // reduce over lanes.
    for (int h0 = 0; h0 < heads; h0 += slots) {
      const int h = h0 + slot0;
      const bool mine = slot0 < slots && h < heads;
      const bool is_q = h < p.hq, is_v = h >= p.hq + p.hk;
      const int hl = is_q ? h : is_v ? h - p.hq - p.hk : h - p.hq;
      const RowTensor in = is_q ? p.q : is_v ? p.v : p.k;
      const uint16_t* src = in.p + static_cast<int64_t>(t0) * in.st + hl * in.sh;
      const int64_t head_at = hl * p.head_stride;
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      auto fetch = [&](int tt) {
        if (mine && tt < nt && place[tt].page >= 0) {
          const uint4* x = reinterpret_cast<const uint4*>(src + tt * in.st);
          a = x[v0];
          b = x[v1];
        }
      };
      fetch(0);
      for (int tt = 0; tt < nt; ++tt) {
        const bool live = mine && place[tt].page >= 0;
        uint4 xa = a, xb = b;
        fetch(tt + 1);
        float fa[8], fb[8];
        unpack8<BF16>(xa, fa);
        unpack8<BF16>(xb, fb);
        if (rotated && !is_v) {
          turn(fa, fb, cs_all + tt * half + 8 * u, p.interleaved != 0);
          xa = pack8<BF16>(fa);
          xb = pack8<BF16>(fb);
          unpack8<BF16>(xa, fa);
          unpack8<BF16>(xb, fb);
        }
        if (is_q && live) {
          uint4* y = reinterpret_cast<uint4*>(p.q_out.p + static_cast<int64_t>(t0 + tt) * p.q_out.st +
                                              hl * p.q_out.sh);
          y[v0] = xa;
          y[v1] = xb;
        }
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmax3_nan(m, fabsf(fa[i]), fabsf(fb[i]));
        // units is 4 or 8 (head_dim 64 or 128): a head's lanes are an aligned
        // group of that many
        for (int o = units >> 1; o > 0; o >>= 1)
          m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (live && !is_q) {
          // (m - m: 0, but NaN where the row has NaN or infinity, so that what
          // reads it is NaN)
          const float sc = __fmaf_rn(m, kInv127, __fsub_rn(m, m));
          const float rcp = m != 0.0f ? __frcp_rn(sc) : 0.0f;
          uint32_t ca[8], cb[8];
          quant_codes8(fa, sc, rcp, ca);
          quant_codes8(fb, sc, rcp, cb);
          const uint2 ya = make_uint2(pack_low_bytes4(ca[0], ca[1], ca[2], ca[3]),
                                      pack_low_bytes4(ca[4], ca[5], ca[6], ca[7]));
          const uint2 yb = make_uint2(pack_low_bytes4(cb[0], cb[1], cb[2], cb[3]),
                                      pack_low_bytes4(cb[4], cb[5], cb[6], cb[7]));
          int8_t* row = static_cast<int8_t*>(is_v ? p.v_pages : p.k_pages) +
                        place[tt].at + head_at;
          if (v1 == v0 + 1) {
            *reinterpret_cast<uint4*>(row + v0 * 8) =
                make_uint4(ya.x, ya.y, yb.x, yb.y);
          } else {
            *reinterpret_cast<uint2*>(row + v0 * 8) = ya;
            *reinterpret_cast<uint2*>(row + v1 * 8) = yb;
          }
          if (u == 0)
            (is_v ? p.v_scale
                  : p.k_scale)[place[tt].scale_at +
                             (static_cast<int64_t>(hl) << p.page_shift)] = sc;
        }
      }
    }
  }
}

template <bool BF16, int MODE>
cudaError_t launch_one(const RopeArgs& a, cudaStream_t stream) {
  // few tokens: a block each, so that all SMs work; many: their places and
  // angles are shared work
  constexpr int kMany = MODE == 2 ? kMaxTokens : 4;
  const int tpb = a.total_tokens >= 1024 ? kMany : 1;
  const int grid = (a.total_tokens + tpb - 1) / tpb;
  const size_t smem = a.freqs ? tpb * (a.rot_dim / 2) * sizeof(float2) : 0;
  return launch_behind(rope_kernel<BF16, MODE>, dim3(grid), dim3(kThreads), smem,
                       stream, a, tpb);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool bf16, int mode,
                        cudaStream_t stream) {
  if (mode == 0)
    return bf16 ? launch_one<true, 0>(a, stream) : launch_one<false, 0>(a, stream);
  if (mode == 1)
    return bf16 ? launch_one<true, 1>(a, stream) : launch_one<false, 1>(a, stream);
  return bf16 ? launch_one<true, 2>(a, stream) : launch_one<false, 2>(a, stream);
}

}  // namespace tilemix
