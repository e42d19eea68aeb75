// Host check of the paged attention kernels' split of key work (Line in
// paged_line.cuh, the source the kernels are built from).  A warp's 32 lanes
// run as fibers that meet at every vote and shuffle, so `locate` runs as on
// the device; the walk below is the kernels' own.  Every (sequence, KV head,
// tile, unit of keys) has to be taken by exactly one block.
//
//   line_split <seed> <cases>   random cases; prints the first fault, exits 1
//   line_split - ...            one case from the arguments (see main)
#include <ucontext.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

using std::max;
using std::min;

namespace warp {

constexpr int kLanes = 32;
ucontext_t scheduler, lanes[kLanes];
std::vector<char> stacks[kLanes];
long long posted[2][kLanes];
int count[kLanes];
bool finished[kLanes];
int lane;
std::function<void(int)> body;

void enter() {
  body(lane);
  finished[lane] = true;
  swapcontext(&lanes[lane], &scheduler);
}

// Posts this lane's value and returns everybody's, once all have posted.
const long long* meet(long long v) {
  const int at = count[lane]++ & 1;
  posted[at][lane] = v;
  swapcontext(&lanes[lane], &scheduler);
  return posted[at];
}

void run(std::function<void(int)> f) {
  body = std::move(f);
  for (int i = 0; i < kLanes; ++i) {
    if (stacks[i].empty()) stacks[i].resize(1 << 16);
    getcontext(&lanes[i]);
    lanes[i].uc_stack.ss_sp = stacks[i].data();
    lanes[i].uc_stack.ss_size = stacks[i].size();
    lanes[i].uc_link = &scheduler;
    makecontext(&lanes[i], enter, 0);
    finished[i] = false;
    count[i] = 0;
  }
  for (long rounds = 0;; ++rounds) {
    int done = 0;
    for (lane = 0; lane < kLanes; ++lane) {
      if (!finished[lane]) swapcontext(&scheduler, &lanes[lane]);
      done += finished[lane];
    }
    if (done == kLanes) return;
    if (done != 0 || rounds > 100000) {
      std::printf(done ? "lanes diverge at a vote\n" : "locate does not end\n");
      std::exit(1);
    }
  }
}

}  // namespace warp

template <class T>
T __shfl_xor_sync(unsigned, T v, int o) {
  return static_cast<T>(warp::meet(v)[warp::lane ^ o]);
}
template <class T>
T __shfl_up_sync(unsigned, T v, int o) {
  const long long* all = warp::meet(v);
  return static_cast<T>(all[warp::lane >= o ? warp::lane - o : warp::lane]);
}
template <class T>
T __shfl_sync(unsigned, T v, int l) {
  return static_cast<T>(warp::meet(v)[l & 31]);
}
inline unsigned __ballot_sync(unsigned, bool p) {
  const long long* all = warp::meet(p);
  unsigned m = 0;
  for (int i = 0; i < 32; ++i) m |= static_cast<unsigned>(all[i] != 0) << i;
  return m;
}
inline int __popc(unsigned m) { return __builtin_popcount(m); }
inline int __ffs(unsigned m) { return __builtin_ffs(static_cast<int>(m)); }
inline int atomicCAS(int* p, int was, int now) {
  const int old = *p;
  if (old == was) *p = now;
  return old;
}

#include "paged_line.cuh"

using namespace tilemix;

struct Case {
  std::vector<int> cu{0}, lens;
  PagedArgs p{};
  int status = 0;
  void finish() {
    p.batch = static_cast<int>(lens.size());
    p.total_tokens = cu.back();
    p.cu_seqlens = cu.data();
    p.kv_lens = lens.data();
    p.status = &status;
    p.hq = p.group * p.hkv;
    p.page_shift = 4;
    p.max_pages = 1 << 26;
  }
  void print() const {
    std::printf("hkv %d group %d causal %d max_q %d max_kv %d\nnew ", p.hkv,
                p.group, p.causal, p.max_q_len, p.max_kv_len);
    for (size_t b = 0; b < lens.size(); ++b) std::printf("%d,", cu[b + 1] - cu[b]);
    std::printf("\nlens ");
    for (int n : lens) std::printf("%d,", n);
    std::printf("\n");
  }
};

template <int R, int U>
bool check(const Case& c, int parts) {
  const PagedArgs& p = c.p;
  const Line<R, U> line(p);
  auto bad = [&](const char* what, const Cursor& at) {
    std::printf("Line<%d, %d> over %d blocks: %s at sequence %d head %d tile %d "
                "unit %d\n", R, U, parts, what, at.b, at.kvh, at.qt, at.unit);
    c.print();
    return false;
  };
  for (int b = 0; b < p.batch; ++b) {
    const SeqGeom g = seq_geom(p, b, false);
    for (int k = 0; k <= line.blocks(g); ++k) {
      const long long w = line.prefix(p, g, k);
      if (w < 0 || (k > 0 && w < line.prefix(p, g, k - 1)))
        return bad("weights decrease", Cursor{b, 0, k, 0});
    }
  }
  std::vector<Cursor> at(parts + 1);
  for (int i = 0; i <= parts; ++i) {
    Cursor lane_at[32];
    warp::run([&](int lane) {
      lane_at[lane] = line.locate(p, i, parts, lane, false);
    });
    at[i] = lane_at[0];
    for (const Cursor& x : lane_at)
      if (!same_item(x, at[i]) || x.unit != at[i].unit)
        return bad("lanes disagree", x);
    const Cursor& x = at[i];
    if (x.b == p.batch) continue;
    if (x.b < 0 || x.b > p.batch) return bad("outside", x);
    const SeqGeom g = seq_geom(p, x.b, false);
    if (g.n == 0 || x.kvh < 0 || x.kvh >= p.hkv || x.qt < 0 ||
        x.qt >= line.tiles(g) || x.unit < 0 || x.unit >= line.units(p, g, x.qt))
      return bad("outside", x);
  }
  // the kernels' walk of one part
  std::map<std::tuple<int, int, int>, std::vector<char>> taken;
  for (int i = 0; i < parts; ++i) {
    Cursor cur = at[i];
    const Cursor end = at[i + 1];
    if ((same_item(cur, end) && cur.unit == end.unit) || cur.b >= p.batch) continue;
    SeqGeom g = seq_geom(p, cur.b, false);
    while (cur.b < p.batch) {
      const bool at_end = same_item(cur, end);
      const int units = line.units(p, g, cur.qt);
      const int ub = at_end ? end.unit : units;
      auto& t = taken[{cur.b, cur.kvh, cur.qt}];
      t.resize(units);
      for (int u = cur.unit; u < ub; ++u) {
        if (t[u]) return bad("taken twice", cur);
        t[u] = 1;
      }
      if (at_end) break;
      line.next(p, g, cur);
    }
  }
  for (int b = 0; b < p.batch; ++b) {
    const SeqGeom g = seq_geom(p, b, false);
    for (int h = 0; h < p.hkv; ++h)
      for (int qt = 0; qt < line.tiles(g); ++qt) {
        const auto it = taken.find({b, h, qt});
        const int units = line.units(p, g, qt);
        for (int u = 0; u < units; ++u)
          if (it == taken.end() || !it->second[u])
            return bad("never taken", Cursor{b, h, qt, u});
      }
  }
  return true;
}

bool check_all(const Case& c) {
  return check<256, 128>(c, 148) && check<16, 64>(c, 296) &&
         check<16, 128>(c, 444) && check<16, 64>(c, 3);
}

std::vector<int> numbers(const char* s) {
  std::vector<int> v;
  for (char* e; *s; s = *e ? e + 1 : e) v.push_back(std::strtol(s, &e, 10));
  return v;
}

int main(int argc, char** argv) {
  if (argc == 8 && argv[1][0] == '-') {
    // - new,new,.. len,len,.. hkv group causal max_q_len
    Case c;
    for (int m : numbers(argv[2])) c.cu.push_back(c.cu.back() + m);
    c.lens = numbers(argv[3]);
    c.p.hkv = std::atoi(argv[4]);
    c.p.group = std::atoi(argv[5]);
    c.p.causal = std::atoi(argv[6]);
    c.p.max_q_len = std::atoi(argv[7]);
    c.p.max_kv_len = 1 << 30;
    c.finish();
    return check_all(c) ? 0 : 1;
  }
  std::mt19937 rng(std::atoi(argv[1]));
  auto pick = [&](int lo, int hi) {
    return std::uniform_int_distribution<int>(lo, hi)(rng);
  };
  for (int i = 0; i < std::atoi(argv[2]); ++i) {
    Case c;
    const int batch = pick(0, 9) ? pick(1, 6) : pick(30, 70);
    const int most = pick(0, 1) ? 1 : pick(0, 2) ? pick(1, 40) : pick(1, 700);
    const int longest = batch > 6 ? 300 : pick(1, 6000);
    const int idle = pick(0, 3);
    for (int b = 0; b < batch; ++b) {
      c.cu.push_back(c.cu.back() + (pick(0, 3) < idle ? 0 : pick(1, most)));
      c.lens.push_back(pick(0, 4) ? pick(0, longest) : pick(0, 20));
      // some that fail a check: they take no part
      if (!pick(0, 30)) c.lens.back() = pick(0, 1) ? -1 : longest + 1;
    }
    const int groups[] = {1, 2, 3, 4, 5, 7, 8, 16, 24, 40, 128};
    c.p.hkv = pick(1, 8);
    c.p.group = groups[pick(0, 10)];
    c.p.causal = pick(0, 3) != 0;
    c.p.max_q_len = most;
    c.p.max_kv_len = longest;
    c.finish();
    if (!check_all(c)) return 1;
  }
  return 0;
}
