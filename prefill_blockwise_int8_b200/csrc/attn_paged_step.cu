// Attention of few new tokens over a paged KV cache: calls of at most 16 packed
// rows a sequence (INT8: 32), as decoded tokens are.  It would serve any call,
// at the cost of reading the cache once per 16 rows.
//
// Mathematics.  The query heads of one KV head and the new tokens pack into
// rows (row = token * group + head), so a KV head's keys are read once for
// all of them.  Per row: running maximum m (base-2 logits), sum l and
// unnormalised output O, merged over key ranges by
//   m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m), O likewise.
// O is rescaled lazily: m only moves when a key exceeds it by more than 2^8,
// so P <= 2^8 fits fp16.  l adds P before it is rounded for the product, so
// lse keeps fp32 accuracy.
// INT8 pages: K codes convert exactly to the query's 16-bit type and their
// scale multiplies the fp32 score.  V codes convert exactly to fp16; their
// scale joins P, which is then P sv 2^-E with 2^E the (lazily raised) power
// of two above the sizes of the scales seen, so that small scales do not fall
// into fp16 subnormals and large ones do not overflow.
//
// Work split.  All keys of all (sequence, KV head, 16-row tile) items, in
// units of four groups, form one line; block c takes the c-th equal part of it.
// An item that one block holds whole is written out; the others leave partial
// results that the merge kernel adds in key order.  No block waits for
// another, and the split follows from the lengths alone.
//
// What bounds it: HBM.  Each warp owns every fourth group of 16 or 32 keys of
// a block's part and runs alone (private m, l, O and a private ring of TMA
// slots, no block barrier in the loop), so a block keeps 4 rings of loads in
// flight.  The products are small (two m16n8k16 per key for d = 128, a fifth
// of the tensor rate at full HBM speed), hence warp-level mma fragments that
// never leave registers.  64 single tokens over 1K..32K keys, 32/8 heads, d
// 128: 705 us, 6.3 TB/s.  INT8 keys are bound by instructions instead (code
// conversion and its latencies): 8 tokens over 8K..16K, 32/32 heads, 176 us,
// 4.6 TB/s.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "paged_common.cuh"
#include "ptx.cuh"

namespace tilemix {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;    // packed rows of an item (mma M)
constexpr int kGridMax = 148 * 3;

// Blocks of an SM.  16-bit pages of 128 channels are bound by HBM with two
// (215 registers a thread); the others by the latency of their own
// instructions, which a third block hides.
template <int D, bool INT8>
constexpr int kBlocksPerSm = D == 64 || INT8 ? 3 : 2;

template <int D, bool INT8>
struct Cfg {
  static constexpr int kElem = INT8 ? 1 : 2;
  // Keys of a ring slot: as many as leave two slots of a warp.  With 32 the
  // maxima, votes and copies of a slot cost half as much per key.
  static constexpr int kGroup = paged_step_group(D, INT8);
  static constexpr int kUnit = kWarps * kGroup;  // keys of a unit of work
  static constexpr int kTile = kGroup * D * kElem;  // K or V bytes of a slot
  static constexpr int kScale = INT8 ? 2 * kGroup * 4 : 0;
  static constexpr int kSlot = 2 * kTile;
  // 24 KB of ring per warp (16 with three blocks), at most 8 slots
  static constexpr int kBytes = kBlocksPerSm<D, INT8> == 3 ? 16384 : 24576;
  static constexpr int kSlots = kBytes / kSlot > 8 ? 8 : kBytes / kSlot;
  static constexpr int kRing = kSlots * kSlot;
  static constexpr int kRingAll = kWarps * kRing;
  static constexpr int kScaleOff = kRingAll;
  static constexpr int kScaleAll = kWarps * kSlots * kScale;
  static constexpr int kBarOff = kScaleOff + kScaleAll;
  static constexpr int kSmem = kBarOff + kWarps * kSlots * 8 + 1024;
  // 16 rows of O, and m, l, merged through the warp's own ring
  static constexpr int kMergeStride = D + 4;
  static_assert(kRows * kMergeStride * 4 <= kRing, "merge area");
};

__device__ __forceinline__ void ldm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr));
}

__device__ __forceinline__ void ldm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr));
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4],
                                         uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, bool BF16, bool INT8>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<D, INT8>)
    step_kernel(const __grid_constant__ PagedArgs p) {
  using C = Cfg<D, INT8>;
  constexpr int G = C::kGroup;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, q4 = lane & 3;  // fragment row, quad column
  uint8_t* ring = smem + warp * C::kRing;
  const uint32_t ring_a = smem_u32(ring);
  uint8_t* scales = smem + C::kScaleOff + warp * C::kSlots * C::kScale;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff) + warp * C::kSlots;
  __shared__ int s_bad;  // the item's first key on a bad page; -1: a wait ran out
  if (lane == 0) {
    for (int s = 0; s < C::kSlots; ++s)
      mbar_init(&bars[s], s == 0 && p.test_expire_wait ? 2 : 1);
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  if (threadIdx.x == 0) s_bad = kNoBadKey;
  pdl_wait();
  clear_headers(p);
  pdl_launch();
  const Line<kRows, C::kUnit> line(p);
  Cursor cur, end;
  if (!find_part(p, line, warp, lane, cur, end) || cur.b >= p.batch) return;
  SeqGeom g = seq_geom(p, cur.b, false);
  uint32_t issued = 0, consumed = 0;  // ring slots, over all items
  bool dead = false;                  // a wait ran out

  while (cur.b < p.batch) {
    const bool at_end = same_item(cur, end);
    const int units = line.units(p, g, cur.qt);
    const int ua = cur.unit;
    const int ub = at_end ? end.unit : units;
    if (ua >= ub) {
      if (at_end) break;
      line.next(p, g, cur);
      continue;
    }
    const int nrows = line.rows(p, g, cur.qt);
    const int tok0 = line.first_token(cur.qt);
    const int head0 = cur.kvh * p.group + line.first_head(cur.qt);
    const int keys = line.keys(p, g, cur.qt);         // the tile's limit
    const int keys_min = keys_of_token(p, g, tok0);   // its first row's
    // rows of this thread: g8 and g8 + 8
    int lim[2];
    const uint16_t* qrow[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g8 + 8 * i;
      const int tok = tok0 + r / p.group;
      lim[i] = r < nrows ? keys_of_token(p, g, tok) : 0;
      qrow[i] = r < nrows ? p.q + static_cast<int64_t>(g.start + tok) * p.q_st +
                                static_cast<int64_t>(head0 + r % p.group) * p.q_sh
                          : nullptr;
    }

    // this warp's groups of units [ua, ub): i-th at key k0 + i units
    const int k0 = ua * C::kUnit + warp * G;
    const int kend = min(keys, ub * C::kUnit);
    const int nst = dead || k0 >= kend ? 0 : (kend - k0 + C::kUnit - 1) / C::kUnit;
    const int32_t* trow = p.page_table + cur.b * p.table_stride;
    // A group comes in pieces of whole pages (one, or two of 16 keys); lane l
    // holds the page of piece pid_base + l and issues piece l of a group.
    const int box_shift = min(p.page_shift, G == 32 ? 5 : 4);
    const int ppg_shift = (G == 32 ? 5 : 4) - box_shift;
    int pid = 0, pid_base = -32;
    // keys whose V counts: the rows that see a bad page are not written, so
    // from its first key on V may be anything finite, as behind the end
    int vlen = g.len;
    auto fetch_pids = [&](int base) {
      pid_base = base;
      const int i = base + lane;
      const long long key = k0 + static_cast<long long>(i >> ppg_shift) * C::kUnit +
                            ((i & ((1 << ppg_shift) - 1)) << box_shift);
      int bad = kNoBadKey;
      pid = 0;
      if (i >> ppg_shift < nst && key < g.len) {
        pid = trow[key >> p.page_shift];
        if (pid < 0 || pid >= p.num_pages) {
          bad = static_cast<int>(key);
          atomicMin(&s_bad, bad);
          report_status(p.status, kStatusBadPages);
          pid = 0;
        }
      }
      vlen = min(vlen, __reduce_min_sync(0xffffffffu, bad));
    };
    auto issue = [&](int i) {
      const int first = i << ppg_shift;
      if (first - pid_base >= 32) fetch_pids(first);
      const int id = __shfl_sync(0xffffffffu, pid, (first - pid_base + lane) & 31);
      const uint32_t s = issued % C::kSlots;
      const int key = k0 + i * C::kUnit + (lane << box_shift);
      const int live = min(G, g.len - (k0 + i * C::kUnit));
      const int pieces = (live + (1 << box_shift) - 1) >> box_shift;
      if (lane == 0)
        mbar_arrive_expect_tx(&bars[s], (pieces << box_shift) *
                                            (2 * D * C::kElem + (INT8 ? 8 : 0)));
      if (G == 32) __syncwarp();
      if (lane < pieces) {
        const int slot = key & ((1 << p.page_shift) - 1);
        uint8_t* dst = ring + s * C::kSlot;
        if (INT8) {
          dst += (lane << box_shift) * D;
          tma_load_4d(dst, &p.tm_k, &bars[s], 0, slot, cur.kvh, id);
          tma_load_4d(dst + C::kTile, &p.tm_v, &bars[s], 0, slot, cur.kvh, id);
          const int64_t at =
              ((static_cast<int64_t>(id) * p.hkv + cur.kvh) << p.page_shift) + slot;
          uint8_t* sd = scales + s * C::kScale + (4 * lane << box_shift);
          bulk_load(sd, p.k_scale + at, 4 << box_shift, &bars[s]);
          bulk_load(sd + G * 4, p.v_scale + at, 4 << box_shift, &bars[s]);
        } else {
          dst += (lane << box_shift) * 128;
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(dst + c * G * 128, &p.tm_k, &bars[s], c * 64, slot, cur.kvh,
                        id);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(dst + C::kTile + c * G * 128, &p.tm_v, &bars[s], c * 64, slot,
                        cur.kvh, id);
        }
      }
      ++issued;
    };
    if (nst > 0) fetch_pids(0);
    int next = 0;
    for (; next < C::kSlots && next < nst; ++next) issue(next);

    // Q fragments of the whole tile.  INT8: the contraction runs over the
    // channels in the order 64 j + 16 q + 4 s + e (quad q, k-step 4 j + s),
    // so that a thread's codes of four k-steps are 16 consecutive bytes.
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const int c0 = INT8 ? 64 * (s >> 2) + 16 * q4 + 4 * (s & 3) : 16 * s + 2 * q4;
      const int c1 = INT8 ? c0 + 2 : c0 + 8;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qf[s][i] = qrow[i] ? *reinterpret_cast<const uint32_t*>(qrow[i] + c0) : 0u;
        qf[s][2 + i] =
            qrow[i] ? *reinterpret_cast<const uint32_t*>(qrow[i] + c1) : 0u;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F};  // running max (base 2)
    float l[2] = {0.0f, 0.0f};                    // this thread's sums
    // sums of the weights as O has them: rounded, and (INT8: times the size
    // of their scales) before that
    float lr[2] = {0.0f, 0.0f}, lw[2] = {0.0f, 0.0f};
    float inv = 0.0f;  // INT8: 2^-E of the V scales (0: none seen)

    for (int i = 0; i < nst; ++i) {
      const uint32_t s = consumed % C::kSlots;
      const bool got = mbar_wait(&bars[s], (consumed / C::kSlots) & 1, nullptr);
      if (!__all_sync(0xffffffffu, got)) {
        report_status(p.status, kStatusTimeout);
        dead = true;
        break;
      }
      ++consumed;
      const uint32_t ka = ring_a + s * C::kSlot;
      const uint32_t va = ka + C::kTile;
      const int key0 = k0 + i * C::kUnit;
      // column fragment j holds keys 8 j .. 8 j + 7: this thread's key0 + 8 j
      // + ca and + cb (INT8 rows are taken in the order 0, 4, 1, 5, 2, 6, 3,
      // 7, which spreads a quarter warp's 16-byte reads over all banks)
      constexpr int F = G / 8;
      const int ca = INT8 ? q4 : 2 * q4, cb = INT8 ? q4 + 4 : 2 * q4 + 1;
      float sc[F][4];
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[j][e] = 0.0f;
      if (INT8) {
        const int kr = (g8 >> 1) | ((g8 & 1) << 2);
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint32_t off = (8 * j + kr) * D + 64 * c + 16 * q4;
            const uint4 w = lds128(ka + swz(off, D == 128 ? 7u : 3u));
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              uint32_t b0, b1;
              if (BF16) i8x4_to_bf2x2(ws[t], b0, b1);
              else i8x4_to_h2x2(ws[t], b0, b1);
              mma16816<BF16>(sc[j], qf[4 * c + t], b0, b1);
            }
          }
      } else {
        // lanes 0-7 keys 0-7 low channels, 8-15 the same keys' high
        // channels, 16-31 keys 8-15
        const int kr = (lane & 7) + ((lane >> 4) << 3);
        const int hi = (lane >> 3) & 1;
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
#pragma unroll
          for (int j = 0; j < F; j += 2) {
            const uint32_t off =
                (t >> 2) * G * 128 + (8 * j + kr) * 128 + (t & 3) * 32 + hi * 16;
            uint32_t b[4];
            ldm_x4(ka + swz(off, 7u), b);
            mma16816<BF16>(sc[j], qf[t], b[0], b[1]);
            mma16816<BF16>(sc[j + 1], qf[t], b[2], b[3]);
          }
      }
      // scores in base-2 logits; masked ones -inf (by position, whatever the
      // slot held)
      const uint32_t sa = smem_u32(scales + s * C::kScale);
      float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
      float svm = 0.0f;
      const bool masked = key0 + G > keys_min;
#pragma unroll
      for (int j = 0; j < F; ++j) {
        float ka_ = p.scale_log2, kb_ = p.scale_log2;
        if (INT8) {
          ka_ *= __uint_as_float(lds32(sa + (8 * j + ca) * 4));
          kb_ *= __uint_as_float(lds32(sa + (8 * j + cb) * 4));
        }
        sc[j][0] *= ka_, sc[j][2] *= ka_;
        sc[j][1] *= kb_, sc[j][3] *= kb_;
        if (masked) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + 8 * j + ((e & 1) ? cb : ca) >= lim[e >> 1])
              sc[j][e] = -CUDART_INF_F;
        }
        mx[0] = fmaxf(mx[0], fmaxf(sc[j][0], sc[j][1]));
        mx[1] = fmaxf(mx[1], fmaxf(sc[j][2], sc[j][3]));
      }
      // A quad's maxima only matter when one passes the reference by more
      // than 2^8; the lanes vote on their own first.
      bool grow = mx[0] > m[0] + kRescaleThreshold || mx[1] > m[1] + kRescaleThreshold;
      if (INT8) {
        // the largest live V scale (slots past the end may hold anything)
        const float v =
            lane < G ? __uint_as_float(lds32(sa + G * 4 + 4 * (lane & (G - 1)))) : 0.0f;
        svm = key0 + lane < vlen ? fabsf(v) : 0.0f;
        grow |= inv == 0.0f ? svm > 0.0f : svm * inv > 32.0f;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        }
        float f = 1.0f;
        if (INT8) {
#pragma unroll
          for (int x = 16; x > 0; x >>= 1)
            svm = fmaxf(svm, __shfl_xor_sync(0xffffffffu, svm, x));
          if (svm > 0.0f && (inv == 0.0f || svm * inv > 32.0f)) {
            const int e = min(max(ilogbf(svm) + 1, -126), 126);
            const float ninv = ldexpf(1.0f, -e);
            f = inv == 0.0f ? 0.0f : ninv / inv;
            inv = ninv;
          }
        }
        float al[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          al[r] = 1.0f;
          if (mx[r] > m[r] + kRescaleThreshold) {
            al[r] = ex2_approx(m[r] - mx[r]);
            m[r] = mx[r];
          }
          l[r] *= al[r];
          al[r] *= f;
          lr[r] *= al[r];
          lw[r] *= al[r];
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][0] *= al[0];
          o[j][1] *= al[0];
          o[j][2] *= al[1];
          o[j][3] *= al[1];
        }
      }
      // P; a row that has seen no key keeps m = -inf and P = 0
      const float mu[2] = {m[0] == -CUDART_INF_F ? 0.0f : m[0],
                           m[1] == -CUDART_INF_F ? 0.0f : m[1]};
      const bool tail = key0 + G > vlen;
#pragma unroll
      for (int h = 0; h < G / 16; ++h) {
        uint32_t pf[4];
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          const int j = 2 * h + jj;
          float va_ = 1.0f, vb_ = 1.0f;
          if (INT8) {
            va_ = __uint_as_float(lds32(sa + G * 4 + (8 * j + ca) * 4)) * inv;
            vb_ = __uint_as_float(lds32(sa + G * 4 + (8 * j + cb) * 4)) * inv;
            if (tail) {  // P = 0 times the scale of a slot past the end is 0
              if (key0 + 8 * j + ca >= vlen) va_ = 0.0f;
              if (key0 + 8 * j + cb >= vlen) vb_ = 0.0f;
            }
          }
          float e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            e4[e] = ex2_approx(sc[j][e] - mu[e >> 1]);
            l[e >> 1] += e4[e];
            if (INT8) e4[e] *= (e & 1) ? vb_ : va_;
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            pf[2 * jj + r] = pack_pair<BF16 && !INT8>(e4[2 * r], e4[2 * r + 1]);
            const float2 x = unpack_pair<BF16 && !INT8>(pf[2 * jj + r]);
            // (sizes: weights of both signs would cancel in the ratio)
            lr[r] += fabsf(x.x) + fabsf(x.y);
            if (INT8) lw[r] += fabsf(e4[2 * r]) + fabsf(e4[2 * r + 1]);
          }
        }
        if (INT8) {
          // any int8 code is finite: P = 0 is enough behind the end.
          // ldmatrix rows in the order of the score columns: row 2q -> q, ...
          const int r8 = lane & 7;
          const int kr = 16 * h + ((r8 >> 1) | ((r8 & 1) << 2)) + ((lane >> 3) & 1) * 8;
          const int hi = lane >> 4;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t b[4];
            ldm_x4_t(va + swz(kr * D + c * 32 + hi * 16, D == 128 ? 7u : 3u), b);
            // b[0], b[1]: keys 0-7, 8-15 of 16 channels; b[2], b[3]: the next
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t y0 = b[2 * x] ^ 0x80808080u;
              const uint32_t y1 = b[2 * x + 1] ^ 0x80808080u;
              const __half2 bias = __float2half2_rn(1152.0f);
              uint32_t xe = __byte_perm(y0, 0x64646464u, 0x4240);
              uint32_t xo = __byte_perm(y0, 0x64646464u, 0x4341);
              uint32_t ye = __byte_perm(y1, 0x64646464u, 0x4240);
              uint32_t yo = __byte_perm(y1, 0x64646464u, 0x4341);
              auto sub = [&](uint32_t& z) {
                const __half2 t = __hsub2(*reinterpret_cast<__half2*>(&z), bias);
                z = *reinterpret_cast<const uint32_t*>(&t);
              };
              sub(xe);
              sub(xo);
              sub(ye);
              sub(yo);
              // even and odd channels of the 16 as two n-tiles
              mma16816<false>(o[4 * c + 2 * x], pf, xe, ye);
              mma16816<false>(o[4 * c + 2 * x + 1], pf, xo, yo);
            }
          }
        } else {
          // V rows past the sequence's end may hold NaN: cleared in registers
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          if (tail) {
            const int live = vlen - key0 - 16 * h;  // keys 2 q4, + 1, + 8, + 9
            auto keep = [&](int k) {
              return (k < live ? 0x0000ffffu : 0u) | (k + 1 < live ? 0xffff0000u : 0u);
            };
            keep0 = keep(2 * q4);
            keep1 = keep(2 * q4 + 8);
          }
          const int kr = 16 * h + (lane & 7) + ((lane >> 3) & 1) * 8;
          const int hi = lane >> 4;
#pragma unroll
          for (int t = 0; t < D / 16; ++t) {
            const uint32_t off = (t >> 2) * G * 128 + kr * 128 + (t & 3) * 32 + hi * 16;
            uint32_t b[4];
            ldm_x4_t(va + swz(off, 7u), b);
            if (tail) {
              b[0] &= keep0;
              b[1] &= keep1;
              b[2] &= keep0;
              b[3] &= keep1;
            }
            mma16816<BF16>(o[2 * t], pf, b[0], b[1]);
            mma16816<BF16>(o[2 * t + 1], pf, b[2], b[3]);
          }
        }
      }
      __syncwarp();
      if (next < nst) {
        issue(next);
        ++next;
      }
    }
    if (dead) {  // let the copies in flight land (bounded), read nothing
      for (; consumed < issued; ++consumed)
        mbar_wait(&bars[consumed % C::kSlots], (consumed / C::kSlots) & 1, nullptr);
    }
    // ---- the four warps' results merge through their own rings ----
    float* mine = reinterpret_cast<float*>(ring);
    float back[2];  // O of the exact weights, INT8: back to the scale of V
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      auto quad = [](float x) {
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        return x + __shfl_xor_sync(0xffffffffu, x, 2);
      };
      l[r] = quad(l[r]);
      back[r] = round_off(INT8 ? quad(lw[r]) : l[r], quad(lr[r]));
      if (INT8) back[r] = inv > 0.0f ? back[r] / inv : 0.0f;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float* row = mine + (g8 + 8 * r) * C::kMergeStride;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        if (INT8) {
          // tiles 2 j', 2 j' + 1: channels 16 j' + 4 q4 + {0, 2} and {1, 3}
          const int c = 16 * (j >> 1) + 4 * q4 + (j & 1);
          row[c] = o[j][2 * r] * back[r];
          row[c + 2] = o[j][2 * r + 1] * back[r];
        } else {
          *reinterpret_cast<float2*>(row + 8 * j + 2 * q4) =
              make_float2(o[j][2 * r] * back[r], o[j][2 * r + 1] * back[r]);
        }
      }
      if (q4 == 0) {
        row[D] = m[r];
        row[D + 1] = l[r];
      }
    }
    if (dead) atomicMin(&s_bad, -1);
    __syncthreads();
    const int bad = s_bad;
    const bool whole = ua == 0 && ub == units;
    const int slot = 2 * blockIdx.x + (ua == 0 ? 1 : 0);
    // thread: row threadIdx / 8, channels 4 (threadIdx % 8) + 32 k
    {
      const int r = threadIdx.x >> 3, c8 = threadIdx.x & 7;
      float mw[kWarps], mt = -CUDART_INF_F;
      const float* rows[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        rows[w] = reinterpret_cast<const float*>(smem + w * C::kRing) +
                  r * C::kMergeStride;
        mw[w] = rows[w][D];
        mt = fmaxf(mt, mw[w]);
      }
      float f[kWarps], lt = 0.0f;
      const float mz = mt == -CUDART_INF_F ? 0.0f : mt;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        f[w] = ex2_approx(mw[w] - mz);
        lt += f[w] * rows[w][D + 1];
      }
      // (a partial result is judged by the merge, which knows all pieces)
      if (r < nrows &&
          !(whole && keys_of_token(p, g, tok0 + r / p.group) > bad)) {
        const int tok = g.start + tok0 + r / p.group;
        const int h = head0 + r % p.group;
        const float il = 1.0f / lt;
        uint16_t* dst = p.out + (static_cast<int64_t>(tok) * p.hq + h) * D;
        float* prow = part_row<D, kRows>(p, slot, r);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const int c = 4 * c8 + 32 * k;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(rows[w] + c);
            a.x += f[w] * v.x;
            a.y += f[w] * v.y;
            a.z += f[w] * v.z;
            a.w += f[w] * v.w;
          }
          if (whole) {
            *reinterpret_cast<uint2*>(dst + c) =
                lt == 0.0f ? make_uint2(0u, 0u)
                           : make_uint2(pack_pair<BF16>(a.x * il, a.y * il),
                                        pack_pair<BF16>(a.z * il, a.w * il));
          } else {
            *reinterpret_cast<float4*>(prow + c) = a;
          }
        }
        if (c8 == 0) {
          if (whole) {
            if (p.lse)
              p.lse[static_cast<int64_t>(h) * p.total_tokens + tok] = lse_of(mt, lt);
          } else {
            prow[D] = mt;
            prow[D + 1] = lt;
          }
        }
      }
    }
    if (!whole && threadIdx.x == 0) {
      p.head[2 * slot] = make_int4(1, ub == units ? 1 : 0, bad, nrows);
      p.head[2 * slot + 1] = make_int4(g.start + tok0, head0, p.group,
                                       limit_of_token(p, g, tok0));
    }
    // the rings take TMA writes again: order the generic accesses before
    fence_proxy_async_smem();
    __syncthreads();
    if (threadIdx.x == 0) s_bad = kNoBadKey;
    __syncthreads();

    if (at_end) break;
    line.next(p, g, cur);
  }
}

template <int D, bool BF16, bool INT8>
cudaError_t launch_one(PagedArgs a, cudaStream_t stream) {
  using C = Cfg<D, INT8>;
  auto kern = step_kernel<D, BF16, INT8>;
  cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  constexpr int grid = 148 * kBlocksPerSm<D, INT8>;
  e = launch_behind(kern, dim3(grid), dim3(kThreads), C::kSmem, stream, a);
  if (e != cudaSuccess) return e;
  const int rows = static_cast<int>(
      min(static_cast<long long>(kRows),
          static_cast<long long>(a.max_q_len) * a.group));
  return launch_merge<D, BF16, kRows, 4, 1>(a, grid, rows, stream);
}

template <int D>
cudaError_t launch_d(const PagedArgs& a, const PagedShape& s,
                     cudaStream_t stream) {
  if (s.int8)
    return s.bf16 ? launch_one<D, true, true>(a, stream)
                  : launch_one<D, false, true>(a, stream);
  return s.bf16 ? launch_one<D, true, false>(a, stream)
                : launch_one<D, false, false>(a, stream);
}

}  // namespace

size_t paged_step_workspace_bytes(int head_dim) {
  return workspace_of(kGridMax, kRows, head_dim);
}

cudaError_t launch_paged_step(const PagedArgs& args, const PagedShape& s,
                              void* workspace, cudaStream_t stream) {
  PagedArgs a = args;
  carve_workspace(a, workspace, kGridMax);
  return s.head_dim == 128 ? launch_d<128>(a, s, stream)
                           : launch_d<64>(a, s, stream);
}

}  // namespace tilemix
