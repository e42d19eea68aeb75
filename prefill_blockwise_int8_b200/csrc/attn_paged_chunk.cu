// Attention of many new tokens over a paged KV cache (a prompt's chunk,
// verified drafts, a decoder over an encoder's states).
//
// Mathematics.  As in the step kernel: the query heads of one KV head and
// the new tokens pack into rows; per row a running maximum m (base-2 logits,
// moved lazily, see kLag), sum l and unnormalised output O.  INT8 pages: K
// codes convert exactly to the query's type and their scale multiplies the
// fp32 score; V codes convert exactly to fp16 and their scale joins P as P sv
// 2^-E, 2^E a power of two near the scales seen (raised, with O rescaled, when
// a scale passes 16 times it), so that products stay inside fp16's range.  The
// sign of a V scale goes to its codes, so weights are never negative.
//
// B200 design.  One CTA per SM takes an equal part of the line of all items
// (256 packed rows of a sequence and KV head, times its keys in units of
// 128); an item cut between CTAs leaves partial results for the merge
// kernel.  Inside a CTA:
//   warps 0-3, 4-7  softmax of the two 128-row query tiles, one thread per
//               row (= TMEM lane) with a step's 64 scores in registers: no
//               exchange between threads.  They load Q (any group size and
//               stride), write P over the scores they have read, rescale O
//               when a maximum moves, and finish O / l;
//   warp 8      TMA producer: pages through {64 channels, page} boxes into
//               one ring of K and V tiles (INT8: raw tiles and scales);
//   warps 9, 10 issue tcgen05.mma of one query tile each: S_t = Q_t K^T of
//               64 keys a step, two steps ahead of the softmax, and O_t +=
//               P_t V with P_t in TMEM; they clear the rows of the last V
//               tile behind the sequence's end;
//   warps 12-15 (INT8) convert raw tiles to 16-bit ones.
// TMEM per query tile: two S buffers of 64 columns, O in 128; P over the
// first 32 columns of its S.
//
// What bounds it: the softmax of a step, 1740 cycles (INT8 2580) of which the
// exponentials are 1020 with both tiles at them, where the MMAs take 1280
// (N = 64 products of shared memory run at 3/4 of the full rate; with 128-key
// steps they take 1024, but P V and Q K^T then stand in the softmax's way and
// a step is slower).  2048 tokens over 32768 keys, 32/8 heads, d 128, bf16:
// 1.08-1.12 ms back to back (by the clock), 950-990 TFLOP/s; eight ragged
// chunks over INT8 keys, 24/8 heads: 0.578 ms, 482 TFLOP/s.
#include <cuda.h>

#include "attn_common.cuh"
#include "paged_common.cuh"

namespace tilemix {
namespace {

constexpr int kM = 128;       // rows of a query tile = TMEM lanes
constexpr int kRows = 2 * kM; // packed rows of an item
constexpr int kN = 128;       // keys of a unit and of a K or V tile
constexpr int kStep = 64;     // keys of a softmax step
constexpr int kGridMax = 148;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpConv = 12;
constexpr int kScRing = 4;    // tiles whose INT8 scales are kept

template <int D, bool BF16, bool INT8>
struct Cfg {
  static constexpr int kThreads = INT8 ? 512 : 384;
  // Registers after the split: softmax warps (256 threads) and the others;
  // 256 a + (kThreads - 256) b = the launch's total (512 * 128, 384 * 168).
  static constexpr int kRegsSoftmax = INT8 ? 184 : 208;
  static constexpr int kRegsOther = INT8 ? 72 : 88;
  static_assert(256 * kRegsSoftmax + (kThreads - 256) * kRegsOther ==
                kThreads * (INT8 ? 128 : 168), "register split");
  // How far (base 2) a row's maximum may pass the reference of its
  // exponentials before O is rescaled.  A rescale stalls the query tile for
  // some 1000 cycles, and with a lag of 8 every fourth step of scores with a
  // spread of 7 had one in some row; P <= 2^15 fits fp16 (INT8: 2^11 times
  // scales of up to 2^4), and nothing is lost below, where the reference is
  // never above the maximum.  In bf16 O, 2^24 max |V| keys, stays far inside
  // fp32.
  static constexpr float kLag = INT8 ? 11.0f : BF16 ? 24.0f : 15.0f;
  static constexpr float kScaleLag = 16.0f;
  // Of eight pairs of exponentials, how many run on the FMA pipe instead of
  // the exponential unit: 2048 tokens over 32768 keys back to back 1114 us
  // with none, 1098 with 1, 1096 with 2; INT8, whose scales fill the FMA pipe,
  // 530 with none, 545 with 2 (single cold passes).
  static constexpr int kPolyOf8 = INT8 ? 0 : 2;
  static constexpr int kQTile = kM * D * 2;
  static constexpr int kTile = kN * D * 2;
  static constexpr int kSlots = INT8 ? 3 : D == 128 ? 5 : 8;
  static constexpr int kRaw = kN * D;
  static constexpr int kRawSlots = INT8 ? 3 : 0;
  static constexpr int kRingOff = 2 * kQTile;
  static constexpr int kRawOff = kRingOff + kSlots * kTile;
  static constexpr int kRawScOff = kRawOff + kRawSlots * kRaw;  // [raw][2][128]
  static constexpr int kRawLiveOff = kRawScOff + kRawSlots * kN * 8;  // [raw] ints
  static constexpr int kKscOff = kRawLiveOff + (INT8 ? 16 : 0);
  static constexpr int kVscOff = kKscOff + (INT8 ? kScRing * kN * 4 : 0);
  static constexpr int kExpOff = kVscOff + (INT8 ? kScRing * kN * 4 : 0);
  static constexpr int kBadOff = kExpOff + 4 * kScRing;
  static constexpr int kBarOff = kBadOff + 8;
  // barriers
  static constexpr int kBarQ = 0;                    // [tile]
  static constexpr int kBarS = 2;                    // [tile][buffer]
  static constexpr int kBarP = 6;                    // [tile][buffer]
  static constexpr int kBarO = 10;                   // [tile][step parity]
  static constexpr int kBarFull = 14;                // [slot]
  static constexpr int kBarEmpty = kBarFull + kSlots;
  static constexpr int kBarRawFull = kBarEmpty + kSlots;
  static constexpr int kBarRawEmpty = kBarRawFull + kRawSlots;
  static constexpr int kBarSc = kBarRawEmpty + kRawSlots;  // [kScRing]
  static constexpr int kBarDrain = kBarSc + (INT8 ? kScRing : 0);
  static constexpr int kNumBars = kBarDrain + 2;
  static constexpr int kSmem = kBarOff + 8 * kNumBars + 16 + 1024;
  static_assert(kSmem + 64 <= 232448, "shared memory");
  static_assert(kBarOff % 8 == 0, "barrier alignment");
};

// What the warps of a CTA know of a segment (an item's units [ua, ub)).
struct Segment {
  SeqGeom g;
  int kvh, ua, ub, units;
  int nrows, tok0, head0;
  int keys;   // of the item's last row
  int steps;  // of kStep keys (the last tile may have one only)
};

// Calls f(segment) for this CTA's part of the line, in order, until f
// returns false.  Every warp walks it by itself.
template <class F>
__device__ __forceinline__ void for_segments(const PagedArgs& p,
                                             const Line<kRows, kN>& line,
                                             Cursor cur, const Cursor& end,
                                             F&& f) {
  if (cur.b >= p.batch) return;
  Segment s;
  s.g = seq_geom(p, cur.b, false);
  while (cur.b < p.batch) {
    const bool at_end = same_item(cur, end);
    s.units = line.units(p, s.g, cur.qt);
    s.ua = cur.unit;
    s.ub = at_end ? end.unit : s.units;
    if (s.ua < s.ub) {
      s.kvh = cur.kvh;
      s.nrows = line.rows(p, s.g, cur.qt);
      s.tok0 = line.first_token(cur.qt);
      s.head0 = cur.kvh * p.group + line.first_head(cur.qt);
      s.keys = line.keys(p, s.g, cur.qt);
      s.steps = min(2 * s.ub, max(1, (s.keys + kStep - 1) / kStep)) - 2 * s.ua;
      if (!f(s, cur.b)) return;
    }
    if (at_end) return;
    line.next(p, s.g, cur);
  }
}

// The first of sequence b's keys [lo, hi) that lies on a page out of range,
// kNoBadKey when none does; by a converged warp.
__device__ __forceinline__ int first_bad_key(const PagedArgs& p, int b, int lo,
                                          int hi, int lane) {
  const int32_t* trow = p.page_table + b * p.table_stride;
#pragma unroll 1
  for (int i = lo >> p.page_shift; lo < hi && i <= (hi - 1) >> p.page_shift; i += 32) {
    bool bad = false;
    if (i + lane <= (hi - 1) >> p.page_shift) {
      const int id = trow[i + lane];
      bad = id < 0 || id >= p.num_pages;
    }
    const unsigned any = __ballot_sync(0xffffffffu, bad);
    if (any) return max(lo, (i + __ffs(any) - 1) << p.page_shift);
  }
  return kNoBadKey;
}

// One key row of codes (D bytes at row r of `src`, swizzled) -> 16-bit row r
// of a K or V tile (D/64 chunks of [128][128 B], 128-byte swizzle).  FLIP:
// the signs of all of them are changed where `flip` is the pair's sign bits.
template <int D, bool BF16, bool FLIP = false>
__device__ __forceinline__ void convert_codes(const uint8_t* src, uint8_t* dst,
                                              int r, uint32_t flip = 0) {
  constexpr uint32_t sm = D == 128 ? 7u : 3u;
#pragma unroll
  for (int u = 0; u < D / 16; ++u) {
    const uint4 in = *reinterpret_cast<const uint4*>(src + swz(r * D + u * 16, sm));
    const uint32_t w[4] = {in.x, in.y, in.z, in.w};
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF16) i8x4_to_bf2x2(w[i], h[2 * i], h[2 * i + 1]);
      else i8x4_to_h2x2(w[i], h[2 * i], h[2 * i + 1]);
      if (FLIP) h[2 * i] ^= flip, h[2 * i + 1] ^= flip;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t o = (u >> 2) * (kN * 128) + r * 128 + ((2 * u + e) & 7) * 16;
      *reinterpret_cast<uint4*>(dst + swz(o, 7)) =
          make_uint4(h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3]);
    }
  }
}

template <int D, bool BF16, bool INT8>
__global__ void __launch_bounds__(Cfg<D, BF16, INT8>::kThreads, 1)
    chunk_kernel(const __grid_constant__ PagedArgs p) {
  using C = Cfg<D, BF16, INT8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const Line<kRows, kN> line(p);
  uint8_t* ring = smem + C::kRingOff;
  float* ksc = reinterpret_cast<float*>(smem + C::kKscOff);
  float* vsc = reinterpret_cast<float*>(smem + C::kVscOff);
  volatile float* vexp = reinterpret_cast<volatile float*>(smem + C::kExpOff);
  // set once the producer has met a bad page, and never cleared: whoever
  // finds it set looks at the pages of its own keys (first_bad_key)
  volatile int* bad_seen = reinterpret_cast<volatile int*>(smem + C::kBadOff);
  // INT8: keys of a raw tile before its end and its first bad page: the V
  // behind them counts for no row that is written
  volatile int* raw_live = reinterpret_cast<volatile int*>(smem + C::kRawLiveOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (warp == kWarpProducer && lane == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars[C::kBarQ + t], 4);  // one arrival per softmax warp
      mbar_init(&bars[C::kBarS + 2 * t], 1);
      mbar_init(&bars[C::kBarS + 2 * t + 1], 1);
      mbar_init(&bars[C::kBarP + 2 * t], 4);
      mbar_init(&bars[C::kBarP + 2 * t + 1], 4);
      mbar_init(&bars[C::kBarO + 2 * t], 1);
      mbar_init(&bars[C::kBarO + 2 * t + 1], 1);
    }
    // the timeout path's test: one arrival more than ever comes for the first V
    const int held = p.test_expire_wait ? 1 : 0;
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&bars[C::kBarFull + s], INT8 ? 4 : s == 1 ? 1 + held : 1);
      mbar_init(&bars[C::kBarEmpty + s], 2);  // both MMA warps
    }
    if (INT8) {
      for (int s = 0; s < C::kRawSlots; ++s) {
        mbar_init(&bars[C::kBarRawFull + s], s == 1 ? 1 + held : 1);
        mbar_init(&bars[C::kBarRawEmpty + s], 4);
      }
      for (int s = 0; s < kScRing; ++s) {
        mbar_init(&bars[C::kBarSc + s], 4);
      }
    }
    mbar_init(&bars[C::kBarDrain], 1);
    mbar_init(&bars[C::kBarDrain + 1], 1);
    *abort_flag = 0;
    *bad_seen = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  if (warp == kWarpMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();
  clear_headers(p);
  pdl_launch();
  tc_fence_before();
  Cursor begin, end;
  const bool any = find_part(p, line, warp, lane, begin, end);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (!any) {
    if (warp == kWarpMma) tmem_dealloc(tmem, 512);
    return;
  }

  auto fail = [&]() {
    *abort_flag = 1;
    report_status(p.status, kStatusTimeout);
  };
  // warp-wide wait; false once some wait ran out anywhere in the CTA
  auto wait = [&](int bar, uint32_t parity) -> bool {
    parity &= 1u;
    if (__all_sync(0xffffffffu, mbar_try_wait(&bars[bar], parity))) return true;
    const bool got = mbar_wait(&bars[bar], parity, abort_flag);
    return __all_sync(0xffffffffu, got);
  };

  if (warp >= 8) {
    regs_dec<C::kRegsOther>();
    if (warp == kWarpProducer) {
      // =================== TMA producer ===================
      // A tile's K and V come in pieces of min(page, 128) keys; lane l
      // issues piece l / chunks, channel chunk l % chunks.
      constexpr int kChunks = INT8 ? 1 : D / 64;
      constexpr int kStages = INT8 ? C::kRawSlots : C::kSlots;
      constexpr int kFull = INT8 ? C::kBarRawFull : C::kBarFull;
      constexpr int kEmpty = INT8 ? C::kBarRawEmpty : C::kBarEmpty;
      const int bt_shift = min(p.page_shift, 7);
      const int bt = 1 << bt_shift;  // keys of a piece
      const int piece = lane / kChunks, chunk = lane % kChunks;
      uint32_t idx = 0;  // tiles loaded
      bool ok = true;
      for_segments(p, line, begin, end, [&](const Segment& s, int b) {
        const int32_t* trow = p.page_table + b * p.table_stride;
        auto loads = [&](int n) {  // this lane has a piece of tile n
          return piece * bt < kN && n * kN + piece * bt < s.g.len;
        };
        auto page_of = [&](int n) {
          return loads(n) ? trow[(n * kN + piece * bt) >> p.page_shift] : 0;
        };
        int id_next = page_of(s.ua);
        for (int n = s.ua; n < s.ub && ok; ++n) {
          int id = id_next;
          if (n + 1 < s.ub) id_next = page_of(n + 1);
          const bool load = loads(n);
          // Rows that see no key of a bad page are computed, so V has to be
          // finite there: it reads as zeros (the box lies outside the map), or
          // for INT8 as another page whose V scales the converters clear.
          const bool bad = load && (id < 0 || id >= p.num_pages);
          if (bad) {
            report_status(p.status, kStatusBadPages);
            *bad_seen = 1;
            id = INT8 ? 0 : p.num_pages;
          }
          const int live = min(kN, s.g.len - n * kN);
          const unsigned bad_lanes = __ballot_sync(0xffffffffu, bad);
          const uint32_t pieces = live > 0 ? (live + bt - 1) >> bt_shift : 0;
          const uint32_t bytes = pieces * bt * (INT8 ? D : D * 2);
          const int slot_key = (n * kN + piece * bt) & ((1 << p.page_shift) - 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t st = idx % kStages;
            if (idx >= kStages && !wait(kEmpty + st, idx / kStages - 1)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              if (INT8 && kv == 0)
                raw_live[st] = bad_lanes ? (__ffs(bad_lanes) - 1) * bt : live;
              mbar_arrive_expect_tx(
                  &bars[kFull + st], bytes + (INT8 && kv == 0 ? pieces * bt * 8 : 0));
            }
            __syncwarp();
            if (load) {
              const CUtensorMap* tm = kv ? &p.tm_v : &p.tm_k;
              uint64_t* bar = &bars[kFull + st];
              if (INT8) {
                tma_load_4d(smem + C::kRawOff + st * C::kRaw + piece * bt * D, tm,
                            bar, 0, slot_key, s.kvh, id);
                if (kv == 0) {  // the scales of K and V come with K
                  const int64_t at =
                      ((static_cast<int64_t>(id) * p.hkv + s.kvh) << p.page_shift) +
                      slot_key;
                  uint8_t* sc = smem + C::kRawScOff + (st * 2 * kN + piece * bt) * 4;
                  bulk_load(sc, p.k_scale + at, bt * 4, bar);
                  bulk_load(sc + kN * 4, p.v_scale + at, bt * 4, bar);
                }
              } else {
                tma_load_4d(ring + st * C::kTile + chunk * (kN * 128) +
                                piece * bt * 128,
                            tm, bar, chunk * 64, slot_key, s.kvh, id);
              }
            }
            ++idx;
          }
        }
        return ok;
      });
      if (!ok) fail();
      // Copies in flight land (bounded) before the CTA may exit, whoever
      // gave up: this warp may have issued its last one by then.
      const uint32_t first = idx > kStages ? idx - kStages : 0;
      for (uint32_t i = first; i < idx; ++i)
        mbar_wait(&bars[kFull + i % kStages], (i / kStages) & 1, nullptr);
    } else if (warp == kWarpMma || warp == kWarpMma + 1) {
      // =================== MMA issuers ===================
      // One warp per query tile: a wait between two products costs about 100
      // cycles of an idle tensor core (its queue holds little more than the
      // product it runs), unless the other tile's warp issues meanwhile.
      const int t = warp - kWarpMma;
      constexpr uint32_t kFmtQ = BF16 ? 1 : 0;
      constexpr uint32_t kFmtP = BF16 && !INT8 ? 1 : 0;
      constexpr uint32_t id_s = instr_desc(1, kFmtQ, kFmtQ, 0, 0, kStep, kM);
      constexpr uint32_t id_o = instr_desc(1, kFmtP, kFmtP, 0, 1, D, kM);
      const uint64_t dq = desc_k_f16(smem_u32(smem + t * C::kQTile), kM * 128, 0);
      const uint64_t dk = desc_k_f16(smem_u32(ring), kN * 128, 0);
      const uint64_t dv = desc_v(smem_u32(ring), kN * 128, 0);
      // Everything that picks a slot, a phase or a descriptor is made warp-
      // uniform, so the issue path runs on the uniform datapath: with
      // per-thread values an MMA took 90 cycles to issue, above the 64 it
      // takes to run.
      const uint32_t tb = uniform(tmem + t * 256);
      uint64_t* bar_s = &bars[C::kBarS + 2 * t];
      uint64_t* bar_o = &bars[C::kBarO + 2 * t];
      uint32_t base = 0;  // ring tiles of earlier segments
      uint32_t gs = 0;    // steps so far
      uint32_t nq = 0;
      bool ok = true;
      auto full = [&](uint32_t i) {
        return ok = wait(C::kBarFull + i % C::kSlots, i / C::kSlots);
      };
      // S of step i (half `half` of the K tile in ring tile r), by one lane
      auto issue_s = [&](uint32_t i, uint32_t r, uint32_t half) {
        const uint64_t k = dk + (r % C::kSlots) * (C::kTile >> 4) +
                           half * (kStep * 128 / 16);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t o = (ks >> 2) * (kM * 128 / 16) + k_step(ks);
          mma_f16_ss(tb + (i & 1) * kStep, dq + o, k + o, id_s, ks > 0 ? 1u : 0u);
        }
        mma_commit(bar_s + (i & 1));
      };
      auto free_slot = [&](uint32_t i) {
        mma_commit(&bars[C::kBarEmpty + i % C::kSlots]);
      };
      for_segments(p, line, begin, end, [&](const Segment& s, int) {
        const int ua = uniform(s.ua), len = uniform(s.g.len);
        const int steps = uniform(s.steps);
        const uint32_t tiles = uniform(s.ub) - ua;
        if (t * kM >= uniform(s.nrows)) {  // this query tile is empty
          for (uint32_t i = 0; i < 2 * tiles; ++i) {
            // (not before the slot is full: its phases stay in order)
            if (!full(base + i)) return false;
            if (elect_one()) free_slot(base + i);
            __syncwarp();
          }
          base += 2 * tiles;
          return true;
        }
        // two steps' scores are made ahead of the softmax
        if (!full(base)) return false;
        if (!(ok = wait(C::kBarQ + t, nq++))) return false;
        tc_fence_after();
        if (elect_one()) {
          issue_s(gs, base, 0);
          if (steps > 1) issue_s(gs + 1, base, 1);
          free_slot(base);
        }
        __syncwarp();
        for (int j = 0; j < steps; ++j, ++gs) {
          const uint32_t half = j & 1;
          const uint32_t ik = base + ((j + 2) & ~1);  // K tile of step j + 2
          const uint32_t iv = ik - 1;                 // V tile of step j
          const bool ahead = j + 2 < steps;
          // one vote for all that the step needs, usually there by now
          bool ready = mbar_try_wait(&bars[C::kBarP + 2 * t + (gs & 1)], (gs >> 1) & 1);
          if (half == 0) {
            ready &= mbar_try_wait(&bars[C::kBarFull + iv % C::kSlots],
                                   (iv / C::kSlots) & 1);
            if (ahead)
              ready &= mbar_try_wait(&bars[C::kBarFull + ik % C::kSlots],
                                     (ik / C::kSlots) & 1);
          }
          if (!__all_sync(0xffffffffu, ready)) {
            if (!(ok = wait(C::kBarP + 2 * t + (gs & 1), gs >> 1))) return false;
            if (half == 0 && (!full(iv) || (ahead && !full(ik)))) return false;
          }
          if (!INT8 && half == 0 && len - (ua + (j >> 1)) * kN < kN) {
            // rows behind the sequence's end may hold anything: P there is
            // 0, but 0 times NaN is not (both warps write the same zeros)
            const int r0 = max(len - (ua + (j >> 1)) * kN, 0);
            for (int c = 0; c < D / 64; ++c) {
              uint4* z = reinterpret_cast<uint4*>(
                  ring + (iv % C::kSlots) * C::kTile + c * (kN * 128) + r0 * 128);
              for (int i = lane; i < (kN - r0) * 8; i += 32)
                z[i] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          tc_fence_after();
          if (elect_one()) {
            // O += P V of step j; S of step j + 2 overwrites P of step j:
            // products of one thread run in the order they were issued
            const uint64_t v = dv + (iv % C::kSlots) * (C::kTile >> 4) +
                               half * (kStep * 128 / 16);
#pragma unroll
            for (int ks = 0; ks < kStep / 16; ++ks)
              mma_f16_ts(tb + 128, tb + (gs & 1) * kStep + ks * 8,
                         v + ks * (16 * 128 / 16), id_o, ks > 0 || j > 0 ? 1u : 0u);
            // (by step parity, as S and P: step gs is not waited for before
            // step gs - 2 has completed, so a wait cannot mistake the phase)
            mma_commit(bar_o + (gs & 1));
            if (ahead) issue_s(gs + 2, ik, half);
            if (half || j + 1 == steps) free_slot(iv);
            if (ahead && (half || j + 3 == steps)) free_slot(ik);
          }
          __syncwarp();
        }
        base += 2 * tiles;
        return true;
      });
      if (!ok) fail();
      // every MMA issued above has finished once this completes
      if (elect_one()) mma_commit(&bars[C::kBarDrain + t]);
      __syncwarp();
      mbar_wait(&bars[C::kBarDrain + t], 0, nullptr);
      __syncwarp();
    } else if (INT8 && warp >= kWarpConv) {
      // =================== INT8 converters (4 warps) ===================
      const int r = (warp - kWarpConv) * 32 + lane;  // key row of a tile
      uint32_t idx = 0, tile = 0;
      float inv = 0.0f;  // 2^-E; 0 while no scale has been seen
      bool ok = true;
      for_segments(p, line, begin, end, [&](const Segment& s, int) {
        inv = 0.0f;  // O begins anew with every segment
        for (int n = s.ua; n < s.ub; ++n, ++tile) {
          uint32_t flip = 0;  // sign bits of a pair, where this row's V scale is < 0
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++idx) {
            const uint32_t raw = idx % (INT8 ? C::kRawSlots : 1);
            const uint32_t st = idx % C::kSlots;
            const uint32_t sr = tile % kScRing;
            if (!wait(C::kBarRawFull + raw, idx / (INT8 ? C::kRawSlots : 1)) ||
                (idx >= C::kSlots && !wait(C::kBarEmpty + st, idx / C::kSlots - 1))) {
              ok = false;
              return false;
            }
            const float* sc =
                reinterpret_cast<const float*>(smem + C::kRawScOff) + raw * 2 * kN;
            uint8_t* dst = ring + st * C::kTile;
            const uint8_t* src = smem + C::kRawOff + raw * C::kRaw;
            if (kv == 0) {
              const int live = raw_live[raw];
              const float* sv = sc + kN;
              float top = 0.0f;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (4 * lane + j < live) top = fmaxf(top, fabsf(sv[4 * lane + j]));
#pragma unroll
              for (int o = 16; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              if (top > 0.0f && (inv == 0.0f || top * inv > C::kScaleLag)) {
                const int e = min(max(ilogbf(top) + 1, -126), 126);
                inv = ldexpf(1.0f, -e);
              }
              ksc[sr * kN + r] = r < live ? sc[r] * p.scale_log2 : 0.0f;
              // weights keep one sign (see round_off); V's codes take it
              vsc[sr * kN + r] = r < live ? fabsf(sv[r]) * inv : 0.0f;
              flip = sv[r] < 0.0f ? 0x80008000u : 0u;
              if (r == 0) vexp[sr] = inv;
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars[C::kBarSc + sr]);
              convert_codes<D, BF16>(src, dst, r);
            } else {
              // rows behind the end: any code is finite, and P is 0 there
              if (__any_sync(0xffffffffu, flip != 0))
                convert_codes<D, false, true>(src, dst, r, flip);
              else
                convert_codes<D, false>(src, dst, r);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&bars[C::kBarFull + st]);
              mbar_arrive(&bars[C::kBarRawEmpty + raw]);
            }
          }
        }
        return true;
      });
      if (!ok) fail();
    }
  } else {
    regs_inc<C::kRegsSoftmax>();
    // =================== softmax ===================
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;  // row of the tile
    const uint32_t ta =
        tmem + t * 256 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    uint8_t* sq = smem + t * C::kQTile;
    uint32_t gs = 0;    // steps of this query tile so far
    uint32_t tile = 0;  // key tiles of earlier segments
    bool ok = true;
    for_segments(p, line, begin, end, [&](const Segment& s, int b) {
      if (t * kM >= s.nrows) {
        tile += s.ub - s.ua;
        return true;
      }
      // ---- Q: D/8 threads a row, 16 bytes each ----
      {
        constexpr int kU = D / 8, kRowStep = kM / kU;
        const int u = r % kU;
        uint4 x[kU];
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const int row = t * kM + r / kU + k * kRowStep;
          x[k] = make_uint4(0, 0, 0, 0);
          if (row < s.nrows)
            x[k] = *reinterpret_cast<const uint4*>(
                p.q + static_cast<int64_t>(s.g.start + s.tok0 + row / p.group) * p.q_st +
                static_cast<int64_t>(s.head0 + row % p.group) * p.q_sh + u * 8);
        }
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const int row = r / kU + k * kRowStep;
          *reinterpret_cast<uint4*>(
              sq + swz((u >> 3) * (kM * 128) + row * 128 + (u & 7) * 16, 7)) = x[k];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[C::kBarQ + t]);
      }
      const int row = t * kM + r;
      const int lim = row < s.nrows
                          ? keys_of_token(p, s.g, s.tok0 + row / p.group)
                          : 0;
      // keys that every live row of the warp's tile sees
      const int lim_min = keys_of_token(p, s.g, s.tok0 + t * kM / p.group);
      float m_run = -CUDART_INF_F, l_run = 0.0f;
      // INT8: sums of the weights P sv 2^-E as O has them, rounded, and before
      float l_rnd = 0.0f, l_wgt = 0.0f;
      float inv = 0.0f;
      for (int j = 0; j < s.steps; ++j, ++gs) {
        const int key0 = s.ua * kN + j * kStep;
        const uint32_t kt = tile + (j >> 1);  // key tile, its scales' slot
        const uint32_t sc_at = (kt % kScRing) * kN + (j & 1) * kStep;
        const uint32_t sa = ta + (gs & 1) * kStep;
        if (!wait(C::kBarS + 2 * t + (gs & 1), gs >> 1)) return ok = false;
        tc_fence_after();
        uint32_t sv[kStep];
        tmem_ld32_at(sa, sv, 0);
        tmem_ld32_at(sa, sv, 32);
        // INT8: the key scales, all fetched while the scores arrive.  (Their
        // barrier is waited for behind S: a warp that had no part in earlier
        // segments could be laps ahead of it and mistake the phase.)
        uint4 ks[INT8 ? kStep / 4 : 1];
        if (INT8) {
          if (!(j & 1) && !wait(C::kBarSc + kt % kScRing, kt / kScRing))
            return ok = false;
          const uint32_t kc = smem_u32(ksc + sc_at);
#pragma unroll
          for (int i = 0; i < kStep / 4; ++i) ks[i] = lds128(kc + 16 * i);
        }
        tmem_ld_wait();
        if (INT8) {  // logits: the keys' scales differ
#pragma unroll
          for (int i = 0; i < kStep; i += 4) {
            const uint4 w = ks[INT8 ? i / 4 : 0];
            const float2 a = __fmul2_rn(
                make_float2(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])),
                make_float2(__uint_as_float(w.x), __uint_as_float(w.y)));
            const float2 b = __fmul2_rn(
                make_float2(__uint_as_float(sv[i + 2]), __uint_as_float(sv[i + 3])),
                make_float2(__uint_as_float(w.z), __uint_as_float(w.w)));
            sv[i] = __float_as_uint(a.x), sv[i + 1] = __float_as_uint(a.y);
            sv[i + 2] = __float_as_uint(b.x), sv[i + 3] = __float_as_uint(b.y);
          }
        }
        if (key0 + kStep > lim_min) {  // by position, whatever the slot held
          const int hl = lim - key0;
#pragma unroll
          for (int i = 0; i < kStep; ++i)
            if (i >= hl) sv[i] = 0xff800000u;  // -inf
        }
        // a NaN or +inf score makes the maximum NaN, and with it the row
        float mx;
        {
          float a[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            a[k] = fmax_nan(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1]));
#pragma unroll
          for (int i = 16; i < kStep; i += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              a[k] = fmax3_nan(a[k], __uint_as_float(sv[i + 2 * k]),
                               __uint_as_float(sv[i + 2 * k + 1]));
          mx = fmax3_nan(fmax3_nan(a[0], a[1], a[2]), fmax3_nan(a[3], a[4], a[5]),
                         fmax_nan(a[6], a[7]));
        }
        const float c = INT8 ? 1.0f : p.scale_log2;
        mx = mx == -CUDART_INF_F ? mx : mx * c;
        if (mx == CUDART_INF_F) mx = CUDART_NAN_F;
        bool need = !(mx <= m_run + C::kLag);
        float alpha = 1.0f;
        if (need) {
          alpha = ex2_approx(m_run - mx);
          m_run = mx;
          l_run *= alpha;
        }
        if (INT8) {
          const float ve = vexp[kt % kScRing];
          if (ve != inv) {
            alpha *= inv == 0.0f ? 0.0f : ve / inv;
            inv = ve;
            need = true;
          }
        }
        if (j > 0 && __any_sync(0xffffffffu, need)) {
          // the products of the step before have to be done
          if (!wait(C::kBarO + 2 * t + ((gs - 1) & 1), (gs - 1) >> 1))
            return ok = false;
          tc_fence_after();
          if (INT8) {
            l_rnd *= alpha;
            l_wgt *= alpha;
          }
#pragma unroll 1
          for (int oc = 0; oc < D; oc += 64) {
            uint32_t o[64];
            tmem_ld32_at(ta + 128 + oc, o, 0);
            tmem_ld32_at(ta + 128 + oc, o, 32);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 64; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
#pragma unroll
            for (int i = 0; i < 64; i += 16) tmem_st16(ta + 128 + oc + i, o + i);
          }
        }
        // INT8: P sv is never exact, not even of the key that dominates a
        // row, so its rounding is followed and divided out at the end (see
        // round_off); where no key has 1/32 of its row so far the roundings
        // average out.  (Ragged chunks 524 us without it, 576 with it, 596
        // with it in every step.  16-bit P of a row's maximum is exact unless
        // the reference lags, and following it took 1.05 times as long.)
        const bool heavy =
            INT8 && __any_sync(0xffffffffu,
                               !(ex2_approx(mx - m_run) < 0.03125f * l_run));
        const float mu = m_run == -CUDART_INF_F ? 0.0f : m_run;
        const float2 c2 = make_float2(c, c), nm = make_float2(-mu, -mu);
        float2 ps[2], pr[2], pw[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) ps[k] = pr[k] = pw[k] = make_float2(0.f, 0.f);
        const uint32_t vc = smem_u32(vsc + sc_at);
#pragma unroll
        for (int q = 0; q < kStep / 32; ++q) {
          uint32_t pk[16];
          uint4 vs[INT8 ? 8 : 1];
          if (INT8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) vs[i] = lds128(vc + 128 * q + 16 * i);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int k = 32 * q + 2 * i;
            const float2 sc =
                make_float2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1]));
            const float2 x = INT8 ? __fadd2_rn(sc, nm) : __ffma2_rn(sc, c2, nm);
            float2 e = (i & 7) < C::kPolyOf8
                           ? ex2_poly2(x)
                           : make_float2(ex2_approx(x.x), ex2_approx(x.y));
            ps[i & 1] = __fadd2_rn(ps[i & 1], e);
            if (INT8) {
              const uint4 v4 = vs[INT8 ? i / 2 : 0];
              e = __fmul2_rn(
                  e, (i & 1) ? make_float2(__uint_as_float(v4.z), __uint_as_float(v4.w))
                             : make_float2(__uint_as_float(v4.x), __uint_as_float(v4.y)));
            }
            pk[i] = pack_pair<BF16 && !INT8>(e.x, e.y);
            if (INT8) pw[i & 1] = __fadd2_rn(pw[i & 1], e);
          }
          if (INT8 && heavy) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              pr[i & 1] = __fadd2_rn(pr[i & 1], unpack_pair<BF16 && !INT8>(pk[i]));
          }
          tmem_st16(sa + 16 * q, pk);
        }
        auto total = [](const float2(&x)[2]) {
          const float2 y = __fadd2_rn(x[0], x[1]);
          return y.x + y.y;
        };
        l_run += total(ps);
        if (INT8) {
          const float wgt = total(pw);
          l_wgt += wgt;
          l_rnd += heavy ? total(pr) : wgt;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[C::kBarP + 2 * t + (gs & 1)]);
      }
      tile += s.ub - s.ua;
      // ---- O_t / l, or a partial result ----
      if (!wait(C::kBarO + 2 * t + ((gs - 1) & 1), (gs - 1) >> 1)) return ok = false;
      tc_fence_after();
      const bool whole = s.ua == 0 && s.ub == s.units;
      int bad_key = kNoBadKey;
      if (__any_sync(0xffffffffu, *bad_seen))
        bad_key = first_bad_key(p, b, s.ua * kN, min(s.ub * kN, s.g.len), lane);
      const int slot = 2 * blockIdx.x + (s.ua == 0 ? 1 : 0);
      // (a partial result is judged by the merge, which knows all pieces)
      const int new_tok = s.tok0 + row / p.group;
      const bool live = row < s.nrows &&
                        !(whole && keys_of_token(p, s.g, new_tok) > bad_key);
      const int tok = s.g.start + new_tok;
      const int h = s.head0 + row % p.group;
      float f = 1.0f;  // O of the exact weights, at the scale of V
      if (INT8) f = inv > 0.0f ? round_off(l_wgt, l_rnd) / inv : 0.0f;
      if (whole) f = l_run == 0.0f ? 0.0f : f / l_run;
      const bool none = whole && l_run == 0.0f;
      uint16_t* dst = p.out + (static_cast<int64_t>(tok) * p.hq + h) * D;
      float* prow = part_row<D, kRows>(p, slot, row);
#pragma unroll 1
      for (int oc = 0; oc < D; oc += 32) {
        uint32_t o[32];
        tmem_ld32(ta + 128 + oc, o);
        tmem_ld_wait();
        if (live) {
          if (whole) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = none ? 0u
                            : pack_pair<BF16>(__uint_as_float(o[8 * v + 2 * i]) * f,
                                              __uint_as_float(o[8 * v + 2 * i + 1]) * f);
              reinterpret_cast<uint4*>(dst + oc)[v] =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              reinterpret_cast<float4*>(prow + oc)[v] = make_float4(
                  __uint_as_float(o[4 * v]) * f, __uint_as_float(o[4 * v + 1]) * f,
                  __uint_as_float(o[4 * v + 2]) * f,
                  __uint_as_float(o[4 * v + 3]) * f);
          }
        }
      }
      if (live) {
        if (!whole) {
          prow[D] = m_run;
          prow[D + 1] = l_run;
        } else if (p.lse) {
          p.lse[static_cast<int64_t>(h) * p.total_tokens + tok] =
              lse_of(m_run, l_run);
        }
      }
      if (!whole && threadIdx.x == 0) {
        p.head[2 * slot] =
            make_int4(1, s.ub == s.units ? 1 : 0, bad_key, s.nrows);
        p.head[2 * slot + 1] = make_int4(s.g.start + s.tok0, s.head0, p.group,
                                         limit_of_token(p, s.g, s.tok0));
      }
      tc_fence_before();  // these reads come before the next segment's MMAs
      return true;
    });
    if (!ok) fail();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

template <int D, bool BF16, bool INT8>
cudaError_t launch_one(const PagedArgs& a, cudaStream_t stream) {
  using C = Cfg<D, BF16, INT8>;
  auto kern = chunk_kernel<D, BF16, INT8>;
  cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_behind(kern, dim3(kGridMax), dim3(C::kThreads), C::kSmem, stream, a);
  if (e != cudaSuccess) return e;
  const int rows = static_cast<int>(
      min(static_cast<long long>(kRows),
          static_cast<long long>(a.max_q_len) * a.group));
  return launch_merge<D, BF16, kRows, 1, 8>(a, kGridMax, rows, stream);
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

size_t paged_chunk_workspace_bytes(int head_dim) {
  return workspace_of(kGridMax, kRows, head_dim);
}

cudaError_t launch_paged_chunk(const PagedArgs& args, const PagedShape& s,
                               void* workspace, cudaStream_t stream) {
  PagedArgs a = args;
  carve_workspace(a, workspace, kGridMax);
  return s.head_dim == 128 ? launch_d<128>(a, s, stream)
                           : launch_d<64>(a, s, stream);
}

}  // namespace tilemix
