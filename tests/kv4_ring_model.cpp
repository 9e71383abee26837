// A model on the host of one CTA of the attention over the 4-bit cache: the
// producer, the copies that land in any order, and the consumer warps, with
// the kernel's own order of tiles and choice of barriers (kv4_ring.cuh) or,
// to show that the model finds the fault, with one barrier a stage.
//
// Barriers are what mbarriers are: a phase completes, and a wait by parity
// passes unless the phase under way has that parity.  A run picks one of what
// can happen next at random until all is done; what it looks for: a warp that
// passes a wait without its block, a copy into a stage that is in use, tiles
// taken never or twice, and a state in which nothing can happen.
//
// Output: a line for each shape and rule, "nt p rule runs faults".
#include <cstdio>
#include <random>
#include <vector>

#include "kv4_ring.cuh"

using namespace fm;

template <int STAGES>
struct OneBarrier {
  static int stage(uint32_t blk) { return (int)(blk % STAGES); }
  static int full(uint32_t blk) { return (int)(blk % STAGES); }
  static uint32_t full_parity(uint32_t blk) { return blk / STAGES % 2; }
  static uint32_t empty_parity(uint32_t blk) { return (blk / STAGES + 1) % 2; }
};

// What a wait by `parity` says where `done` phases have completed.
static bool passes(uint32_t done, uint32_t parity) { return done % 2 != parity; }

struct Warp {
  size_t seg = 0;
  int x = -1;          // its tile, -1: the segment is to be begun
  bool using_it = false, at_barrier = false;
  uint32_t blk = 0;
};

template <class R, int STAGES, int WARPS, int MOST>
bool run(std::mt19937& rng, const std::vector<int>& segments, const std::vector<bool>& bytes, int slowness) {
  const uint32_t total = (uint32_t)bytes.size();
  std::vector<uint32_t> base(segments.size() + 1, 0);
  for (size_t i = 0; i < segments.size(); ++i) base[i + 1] = base[i] + (uint32_t)segments[i];
  std::vector<uint32_t> full_done(2 * STAGES, 0), empty_done(STAGES, 0);
  std::vector<int> empty_left(STAGES, kTiles), content(STAGES, -1);
  std::vector<bool> landed(total, false);
  std::vector<int> taken(total * kTiles, 0);
  std::vector<uint32_t> under_way;
  std::vector<Warp> warps(WARPS);
  uint32_t issued = 0;
  const auto land = [&](uint32_t b) {
    landed[b] = true;
    ++full_done[R::full(b)];
  };
  for (;;) {
    std::vector<int> can;  // -2: the producer, -1: a copy lands, w: warp w
    if (issued < total && passes(empty_done[R::stage(issued)], R::empty_parity(issued))) can.push_back(-2);
    if (!under_way.empty()) can.push_back(-1);
    bool all_over = true;
    for (int w = 0; w < WARPS; ++w) {
      Warp& v = warps[w];
      if (v.seg == segments.size()) continue;
      all_over = false;
      if (v.at_barrier) {
        bool all = true;
        for (const Warp& o : warps) all = all && (o.seg > v.seg || o.at_barrier);
        if (all) can.push_back(w);
      } else if (v.x < 0 || v.using_it) {
        can.push_back(w);
      } else if (passes(full_done[R::full(v.blk)], R::full_parity(v.blk))) {
        can.push_back(w);
      }
    }
    if (all_over && issued == total && under_way.empty()) break;
    if (can.empty()) return false;
    int what = can[rng() % can.size()];
    if (what == -1 && can.size() > 1 && rng() % slowness) continue;  // copies are slow
    if (what == -2) {
      const uint32_t b = issued++;
      const int s = R::stage(b);
      for (const Warp& o : warps)
        if (o.using_it && R::stage(o.blk) == s) return false;
      content[s] = (int)b;
      if (bytes[b]) under_way.push_back(b);
      else land(b);
    } else if (what == -1) {
      const size_t i = rng() % under_way.size();
      const uint32_t b = under_way[i];
      under_way.erase(under_way.begin() + (long)i);
      land(b);
    } else {
      Warp& v = warps[what];
      const auto go = [&](int x) {  // to tile x, or to the barrier at the segment's end
        const TileOrder<WARPS, MOST> order(segments[v.seg] * kTiles);
        v.x = x;
        if (x >= order.n_tiles) v.at_barrier = true;
        else v.blk = base[v.seg] + (uint32_t)(x / kTiles);
      };
      if (v.at_barrier) {
        const size_t seg = v.seg;
        for (Warp& o : warps)
          if (o.seg == seg) {
            o.at_barrier = false;
            o.x = -1;
            ++o.seg;
          }
      } else if (v.x < 0) {
        go(TileOrder<WARPS, MOST>(segments[v.seg] * kTiles).first(what));
      } else if (!v.using_it) {
        if (!landed[v.blk] || content[R::stage(v.blk)] != (int)v.blk) return false;
        v.using_it = true;
      } else {
        const TileOrder<WARPS, MOST> order(segments[v.seg] * kTiles);
        const int n = order.count(v.x), s = R::stage(v.blk);
        if (v.x % kTiles + n > kTiles) return false;  // tiles of one block
        for (int i = 0; i < n; ++i) ++taken[base[v.seg] * kTiles + (size_t)(v.x + i)];
        empty_left[s] -= n;
        if (empty_left[s] < 0) return false;
        if (empty_left[s] == 0) {
          empty_left[s] = kTiles;
          ++empty_done[s];
        }
        v.using_it = false;
        go(order.next(v.x, what));
      }
    }
  }
  for (int t : taken)
    if (t != 1) return false;
  return true;
}

template <class R, int NT, int P>
void shape(const char* rule, int runs) {
  constexpr int S = ring_stages(NT), W = ring_warps(NT, P), M = ring_most(NT, P);
  std::mt19937 rng(12345);
  int faults = 0;
  for (int i = 0; i < runs; ++i) {
    std::vector<int> segments;
    int total = 0;
    for (int n = 1 + (int)(rng() % 4); n > 0; --n) {
      segments.push_back(1 + (int)(rng() % (rng() % 2 ? 6 : 40)));
      total += segments.back();
    }
    std::vector<bool> bytes;  // runs of blocks whose pages are there, and of others
    bool on = rng() % 4 != 0;
    const bool gaps = rng() % 2 != 0;
    while ((int)bytes.size() < total) {
      for (int n = 1 + (int)(rng() % 6); n > 0 && (int)bytes.size() < total; --n) bytes.push_back(on || !gaps);
      on = !on;
    }
    const int slow[4] = {1, 4, 30, 300};
    faults += !run<R, S, W, M>(rng, segments, bytes, slow[rng() % 4]);
  }
  std::printf("%d %d %s %d %d\n", NT, P, rule, runs, faults);
}

int main() {
  const int runs = 1500;
  shape<Ring<ring_stages(1)>, 1, 1>("two", runs);
  shape<Ring<ring_stages(1)>, 1, 2>("two", runs);
  shape<Ring<ring_stages(2)>, 2, 1>("two", runs);
  shape<Ring<ring_stages(2)>, 2, 2>("two", runs);
  shape<OneBarrier<ring_stages(1)>, 1, 1>("one", runs);
  shape<OneBarrier<ring_stages(1)>, 1, 2>("one", runs);
  shape<OneBarrier<ring_stages(2)>, 2, 1>("one", runs);
  shape<OneBarrier<ring_stages(2)>, 2, 2>("one", runs);
  return 0;
}
