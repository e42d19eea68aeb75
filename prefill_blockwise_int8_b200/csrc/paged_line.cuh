// Problem geometry of the paged attention kernels and the split of all key
// work over the grid.  Nothing here but integers and warp votes, so the split
// is checked on the host too (tests/line_split.cpp emulates the warp).
#pragma once

#include "internal.h"
#include "paged.h"

namespace tilemix {

// One sequence as the kernels see it.
struct SeqGeom {
  int start, n, len;  // first token row, new tokens, keys
};

// Sequence b; n = 0 when it has no new tokens or fails a check (reported
// when `report`).
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

// Keys that new token i sees: those below this position, none when negative.
__device__ __forceinline__ int limit_of_token(const PagedArgs& p,
                                              const SeqGeom& g, int i) {
  return p.causal ? g.len - g.n + i + 1 : g.len;
}
__device__ __forceinline__ int keys_of_token(const PagedArgs& p,
                                             const SeqGeom& g, int i) {
  return max(0, limit_of_token(p, g, i));
}

// An item of work (a sequence, a KV head and a tile of at most R packed rows
// of them) and a unit of U keys in it.
struct Cursor {
  int b, kvh, qt, unit;
};

__device__ __forceinline__ bool same_item(const Cursor& a, const Cursor& b) {
  return a.qt == b.qt && a.kvh == b.kvh && a.b == b.b;
}

// The line of all items.  A tile packs whole tokens (tpt of them, each with
// the `group` query heads of the KV head; row = token * group + head) or,
// for a group above R, one token's heads in `hs` parts.  An item weighs its
// keys plus kItemKeys for what it costs to begin and end one; every block
// takes an equal part of the line, cut at units of U keys, so the split
// follows from the lengths alone.
template <int R, int U>
struct Line {
  static constexpr int kItemKeys = U / 2;
  int tpt, hs;

  __device__ __forceinline__ explicit Line(const PagedArgs& p)
      : tpt(max(1, R / p.group)), hs((p.group + R - 1) / R) {}

  __device__ __forceinline__ int blocks(const SeqGeom& g) const {
    return (g.n + tpt - 1) / tpt;
  }
  __device__ __forceinline__ int tiles(const SeqGeom& g) const {
    return blocks(g) * hs;
  }
  // keys of the tile's last row
  __device__ __forceinline__ int keys(const PagedArgs& p, const SeqGeom& g,
                                      int qt) const {
    return keys_of_token(p, g, min((qt / hs + 1) * tpt, g.n) - 1);
  }
  __device__ __forceinline__ int units(const PagedArgs& p, const SeqGeom& g,
                                       int qt) const {
    return max(1, (keys(p, g, qt) + U - 1) / U);
  }
  __device__ __forceinline__ int first_token(int qt) const {
    return qt / hs * tpt;
  }
  __device__ __forceinline__ int first_head(int qt) const {
    return qt % hs * R;
  }
  __device__ __forceinline__ int rows(const PagedArgs& p, const SeqGeom& g,
                                      int qt) const {
    return hs > 1 ? min(R, p.group - first_head(qt))
                  : min(tpt, g.n - first_token(qt)) * p.group;
  }
  // Weight of the first k token blocks of one KV head; never negative, and
  // never less for a larger k (`locate` searches for where a sum is passed).
  __device__ __forceinline__ long long prefix(const PagedArgs& p,
                                              const SeqGeom& g, int k) const {
    // a sequence without new tokens has no last block, whatever it has cached
    if (k == 0) return 0;
    const long long fixed = static_cast<long long>(k) * kItemKeys;
    if (!p.causal) return hs * (fixed + static_cast<long long>(k) * g.len);
    const int nb = blocks(g);
    const long long base = g.len - g.n;
    const long long full = k < nb ? k : k - 1;  // of tpt tokens; the last one's keys are all
    // block j (from 1) has base + j tpt keys, none while that is negative
    const long long none = base < 0 ? min(full, -base / tpt) : 0;
    const long long m = full - none;
    const long long sum =
        m * base + tpt * (m * (full + none + 1) / 2) + (k == nb ? g.len : 0);
    return hs * (fixed + sum);
  }

  // The item and unit at c / parts of the line, by all lanes of a warp;
  // {batch, 0, 0, 0} at its end.  `report`: this warp reports bad sequences.
  __device__ __forceinline__ Cursor locate(const PagedArgs& p, int c, int parts,
                                           int lane, bool report) const {
    // weights of one KV head of 32 sequences at a time
    auto per_head = [&](int b0, bool rep) -> long long {
      const int b = b0 + lane;
      if (b >= p.batch) return 0;
      const SeqGeom g = seq_geom(p, b, rep);
      return prefix(p, g, blocks(g));
    };
    const long long first = per_head(0, report);
    long long total = first;
    for (int b0 = 32; b0 < p.batch; b0 += 32) total += per_head(b0, report);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      total += __shfl_xor_sync(0xffffffffu, total, o);
    total *= p.hkv;
    // (tiles times keys: above 2^54 no call would end, so the product fits)
    long long w = total * c / parts;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const long long head = b0 == 0 ? first : per_head(b0, false);
      long long incl = head * p.hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, incl > w);
      if (past == 0) {
        w -= __shfl_sync(0xffffffffu, incl, 31);
        continue;
      }
      const int l = __ffs(past) - 1;
      const long long ph = __shfl_sync(0xffffffffu, head, l);
      long long rem = w - (__shfl_sync(0xffffffffu, incl, l) - ph * p.hkv);
      Cursor at;
      at.b = b0 + l;
      // the head: the last whose weights before it are at most rem
      at.kvh = last_below(0, p.hkv, lane, [&](int k) { return k * ph <= rem; });
      rem -= at.kvh * ph;
      const SeqGeom g = seq_geom(p, at.b, false);
      const int lo = last_below(0, blocks(g), lane,
                                [&](int k) { return prefix(p, g, k) <= rem; });
      rem -= prefix(p, g, lo);
      const int wi = kItemKeys + keys(p, g, lo * hs);
      const int part = hs > 1 ? static_cast<int>(rem / wi) : 0;
      at.qt = lo * hs + part;
      rem -= static_cast<long long>(part) * wi;
      at.unit = rem <= kItemKeys ? 0 : static_cast<int>(rem - kItemKeys) / U;
      return at;
    }
    return Cursor{p.batch, 0, 0, 0};
  }

  // The largest k in [lo, hi) with f(k), f true at lo and then false from
  // some k on; a warp tests 32 values at a time.
  template <class F>
  __device__ __forceinline__ static int last_below(int lo, int hi, int lane,
                                                   F&& f) {
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) >> 5;
      const long long k = lo + static_cast<long long>(lane) * step;
      const unsigned yes =
          __ballot_sync(0xffffffffu, k < hi && f(static_cast<int>(k)));
      lo += max(__popc(yes) - 1, 0) * step;
      hi = min(hi, lo + step);
    }
    return lo;
  }

  // The first unit of the next item ({batch, 0, 0, 0} after the last); `g`
  // follows.
  __device__ __forceinline__ void next(const PagedArgs& p, SeqGeom& g,
                                       Cursor& c) const {
    c.unit = 0;
    if (++c.qt < tiles(g)) return;
    c.qt = 0;
    if (++c.kvh < p.hkv) return;
    c.kvh = 0;
    while (++c.b < p.batch) {
      g = seq_geom(p, c.b, false);
      if (g.n != 0) return;
    }
  }
};

}  // namespace tilemix
