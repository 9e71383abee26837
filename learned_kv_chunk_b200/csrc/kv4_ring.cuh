// kv4_ring.cuh -- how the warps of a CTA of the attention over the 4-bit cache
// (kv4_attention.cu) share its ring of stages: which tiles of a segment a
// consumer warp takes, in which order, and which barrier says that a block has
// landed.  Plain C++, for the kernel and for a model of it on the host.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define FM_RING_FN __host__ __device__ __forceinline__
#else
#define FM_RING_FN inline
#endif

namespace fm {

constexpr int kTok = 32;     // tokens of a tile
constexpr int kBlock = 128;  // tokens of a stage, the unit in which work is shared out
constexpr int kTiles = kBlock / kTok;

// The shapes: nt tiles of 8 query rows, p pieces of a query.  Consumer warps,
// stages, and the tiles that a warp takes at a time.
constexpr int ring_warps(int nt, int p) { return nt == 1 && p == 1 ? 7 : 5; }
constexpr int ring_stages(int nt) { return nt == 1 ? 5 : 4; }
constexpr int ring_most(int nt, int p) { return nt == 1 && p == 1 ? 2 : 1; }

// A segment's tiles in turn: pairs (of one block) as long as there are two for
// each warp where MOST is 2, then single ones.
template <int WARPS, int MOST>
struct TileOrder {
  int n_tiles, n_double;
  FM_RING_FN explicit TileOrder(int n) : n_tiles(n), n_double(MOST == 2 ? n / (2 * WARPS) * (2 * WARPS) : 0) {}
  FM_RING_FN int first(int warp) const { return MOST == 2 && n_double ? 2 * warp : warp; }
  FM_RING_FN int count(int x) const { return MOST == 2 && x < n_double ? 2 : 1; }  // tiles taken from x on
  FM_RING_FN int next(int x, int warp) const {
    const int n = count(x), y = x + n * WARPS;
    return MOST == 2 && n == 2 && y >= n_double ? n_double + warp : y;
  }
};

// Block `blk` of a CTA (counted over all its segments) goes to stage blk % STAGES
// and completes a phase of one of the stage's TWO barriers, in turn.  A wait by
// parity also passes while the phase before is still open, so it is safe only
// if that phase (the barrier's use before this one) is known to be complete.  A
// warp skips blocks: with one barrier a stage it could pass on the block STAGES
// earlier that it never waited for, and read it as this one while it lands.
// With two, the barrier's use before is block blk - 2 STAGES.  Tiles in turn
// take a warp at most STAGES blocks on, so it has seen a block b >= blk - STAGES
// land (or the segment begins less than STAGES blocks earlier, and every block
// before that has landed).  Block b was copied after b - STAGES had been used,
// and blk - 2 STAGES is not later than that.
template <int STAGES>
struct Ring {
  static FM_RING_FN int stage(uint32_t blk) { return (int)(blk % STAGES); }
  static FM_RING_FN int full(uint32_t blk) { return (int)(2 * (blk % STAGES) + (blk / STAGES) % 2); }
  static FM_RING_FN uint32_t full_parity(uint32_t blk) { return blk / (2 * STAGES) % 2; }
  static FM_RING_FN uint32_t empty_parity(uint32_t blk) { return (blk / STAGES + 1) % 2; }  // of the producer's wait before it
};
template <int STAGES, int WARPS, int MOST>
constexpr bool ring_is_sound() {
  return (WARPS * MOST + kTiles - 1) / kTiles <= STAGES;
}

}  // namespace fm
