// kv4_attention.cu -- attention over the 4-bit paged cache (fm_kv4_attention).
//
// Mathematics.  The codes go to the matrix instructions as f16.  A code times its
// group's scale is exact there within 2^-14 .. 2^12 (other tiles: relative to its
// record's largest scale, to 2^-25 of that).  Queries are scaled to a largest
// element of 2^7 and rounded (two pieces for fp32), softmax weights to 2^-11 (two
// pieces: 2^-22): f16 halves what a weight moves through registers, and 16-bit
// outputs lose as much or more.  S^T = K q^T and O^T = V^T P^T by m16n8k16, tokens
// (then dimensions) in the 16 rows and query rows in the 8 columns, so 8 query
// heads of a kv head fill an instruction and no row of it is padding.
//   * A lane's 16 bytes of a key's codes are one scale group: the dimensions of a
//     step of 16 are permuted to fit, for queries and keys alike.  A value's codes
//     are paired by token in registers, so neither operand crosses lanes; the
//     weights do, by an 8 x 8 transposition (movmatrix).
//   * Softmax in log2 units with a running maximum per row that moves only when a
//     weight would exceed 2^6 times it: the test is one vote, the sums' rescaling
//     rare.  Weights are held times 2^8, so that f16 reaches 2^-33 of the largest.
//   * Work: (row, kv head, tile of query rows) units times blocks of 128 tokens,
//     shared evenly by one wave of CTAs whatever the rows' lengths; a unit that
//     several CTAs share is merged by a second kernel.
//   * A producer warp copies whole pages into a ring of stages (bulk copies; a
//     list's entries by 16-byte asynchronous copies) and looks a block's pages up
//     while the block before it waits.
//
// What bounds it.  The copies alone run at the memory's rate (8 rows of 131072
// tokens, 8 kv heads: 1.14 GB in 187 us, 6.1 TB/s).  With the arithmetic it is 237
// us, 4.8 TB/s, and no pipe is full: 58 % of the issue slots, the ALU at 52 %, the
// tensor pipe at 25 %.  Accumulators and dequantised operands live in the registers
// of the warps that use them, which leaves 16 warps an SM, and each waits on its
// own chain: 32 tokens of a kv head are 128 conversions, 128 products with the
// scales, 64 selections and shifts and 32 matrix instructions, about 590
// instructions with the rest.  A tile of the general form takes three and
// a half times as long (4 x 65536 tokens with a group of zeros in every other tile:
// 160 us, 71 without).  In short calls the start counts: a warp's first tile takes 9000 to
// 12000 cycles where later ones take 2000, with its data there or not, and a change
// of units 8000 (merge, queries).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "kv4.cuh"
#include "kv4_ring.cuh"

namespace fm {
namespace {

constexpr int kMaxTq = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
  Kv4View c;
  const void* q;
  int64_t q_stride;
  void* out;
  const int32_t* kv_len;
  const int32_t* kv_start;
  const int32_t* idx;
  const int32_t* count;
  const float* slopes;
  int Tq, n_q, max_len, max_sel, window;
  float coef, softcap, cap_log2;
  uint32_t page_magic;  // ceil(2^32 / (page_size / 16)), 0 for a page of 16
  int row_tiles;
  bool whole;           // a unit is one CTA's
  int run;              // tokens that lie together: the largest power of two in a page, at most a block; list: a block
  // the partial results of units that several CTAs share: two slots a CTA, its first segment's and its last's
  struct Share* share;  // [CTAs]
  float2* part_ml;      // [CTAs][2][rows of a tile]: the maximum (log2 units), the sum
  float* part_o;        // [CTAs][2][rows of a tile][128]
};

// What a CTA says of the unit in which its range begins, if it is the second
// of those that share it: where the parts are.
struct Share {
  int b, unit;       // row (-1: nothing to merge), kv head * row_tiles + row tile
  int parts, slot0;  // parts: those of the CTA before this one (at slot0), of this one and of the next ones
};

// A CTA has consumer warps and a producer warp, together a multiple of what fills
// the four schedulers' register files: 16 warps of 128 registers an SM where 8
// rows and one piece suffice, 12 of 168 for 16 rows or two pieces.  More query
// rows of a kv head make more units (tiles of 32 rows, at 255 registers and 8
// warps an SM, took 1.4 times as long as two of 16 on 32-row calls).  A stage
// holds a block of four tiles of 32 tokens (twice as many stages of two tiles took 251
// us where this takes 240, 8 x 131072 tokens); the consumers take a segment's tiles in
// turn (as they came free saved 2 %, but summed in another order each time).
template <int NT, int P>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kWarps = ring_warps(NT, P);  // consumers
  static constexpr int kThreads = 32 * (kWarps + 1);
};
constexpr int kCtas = 2;     // that an SM holds

constexpr float kNoMax = -3.402823466e38f;  // the maximum of a row that has seen nothing: no number is below it
constexpr float kLazy = 6.f;              // the maximum may be exceeded by 2^6 before the sums are rescaled
constexpr float kLift = 8.f;              // weights are held times 2^8: at most 2^14 in f16
// Where a value's scale passes 2^72 the outputs could leave fp32's range: from such a tile on a segment's sums are
// held 2^64 lower (and its tiles take the general form, as f16 would not hold such weights).
constexpr uint32_t kHugeScale = 127 + 72;
constexpr float kDrop = 64.f;
constexpr int kORow = 132;         // floats between rows of the warps' outputs in shared memory

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with a zero accumulator.
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The four code bytes of w as four f16 pairs (low nibble in the low half).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// The lowest code byte of w as a f16 pair.
__device__ __forceinline__ uint32_t e2m1x2_to_f16(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(h)
      : "r"(w));
  return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The 8x8 b16 matrix whose row g lies in lanes 4g .. 4g+3, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// cap * tanh(y) in log2 units = cap - 2 cap / (1 + e^2y), within 2^-22 cap: up to
// kFarCap 2^-16 of a logit, a thirty-second of what the f16 weights of 16-bit calls lose.  Above
// it small y go by the series of tanh (its next term is below 2^-26 y for |y| < 1/4); the
// test for that costs 3 % (32 rows of up to 8192 tokens with a cap: 53.2 us, 51.5 without).
// fp32 calls take tanhf, within two units of the result at every cap (32 rows in fp32: 62.5 us,
// 61.3 by the difference).
constexpr float kFarCap = 64.f;
__device__ __forceinline__ float capped(const AttnArgs& a, float y) {
  return a.cap_log2 - __fdividef(2.f * a.cap_log2, 1.f + ex2(y * (2.f * kLog2e)));
}
__device__ __forceinline__ float tanh_near(float y) {
  const float z = y * y;
  float p = fmaf(z, 62.f / 2835.f, -17.f / 315.f);
  p = fmaf(z, p, 2.f / 15.f);
  p = fmaf(z, p, -1.f / 3.f);
  return fmaf(y * z, p, y);
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Arrives on `bar` once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ int g_kv4_err;  // kDevErrTimeout once a wait of the attention's ran out

// The factors of a record's groups.  A tile whose scale bytes all lie in
// [113, 139] (2^-14 .. 2^12: what real keys and values have) is FAST: a group's
// factor is the f16 number of that exponent, (byte - 112) << 10, and its
// products with a code are exact.  Any other tile takes the general form: each
// record's factors are relative to its largest scale 2^r.  That multiplies the
// score (keys); for values it joins the exponent of the weight that goes to the
// product, and of that only: the running maximum and the sum of weights know no
// sizes.  A tile's products are relative to its largest weight times size, and
// join the outputs by one factor a row, so tokens of any size, zeros among them,
// keep their part in both sums.
__device__ __forceinline__ bool fast_scales(uint32_t a, uint32_t b) {
  // bytes + 116 in [224, 255] is [108, 139], + 15 in [128, 255] is [113, 240]; a
  // byte that carries into its neighbour fails the first test itself
  const uint32_t t = ((a + 0x74747474u) & (b + 0x74747474u)) | 0x1f1f1f1fu;
  const uint32_t s = ((a + 0x0f0f0f0fu) & (b + 0x0f0f0f0fu)) | 0x7f7f7f7fu;
  return (t & s) == 0xffffffffu;
}
// Two f16 factors from the bytes 0 and 2 of p (bytes 1 and 3 are 0).
__device__ __forceinline__ uint32_t fast_factor(uint32_t p) { return p * 1024u - 112u * 1024u * 65537u; }

__device__ __forceinline__ uint32_t byte_of(uint32_t w, int i) { return (w >> (8 * i)) & 255u; }
__device__ __forceinline__ bool has_nan(uint32_t w) {
  return byte_of(w, 0) == 255u || byte_of(w, 1) == 255u || byte_of(w, 2) == 255u || byte_of(w, 3) == 255u;
}
// The largest scale byte that is not NaN.
__device__ __forceinline__ uint32_t top_scale(uint32_t w) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r = max(r, byte_of(w, i) == 255u ? 0u : byte_of(w, i));
  return r;
}
// The factor of a score, held within fp32's numbers: a query and a key that give 0 have a score of 0, however
// large the scale, the query and the key's scales are (a NaN stays).
__device__ __forceinline__ float bounded(float x) {
  constexpr float kMost = 3.402823466e38f;
  return x > kMost ? kMost : x < -kMost ? -kMost : x;
}
// f16 bits of 2^(byte i - r), 0 below 2^-25.
__device__ __forceinline__ uint32_t group_factor(uint32_t w, int i, uint32_t r) {
  const __half h = __float2half_rn(__int_as_float(max(127 + (int)byte_of(w, i) - (int)r, 0) << 23));
  return __half_as_ushort(h);
}

// A block in shared memory: of the keys and of the values, runs of `run` tokens,
// each the codes of its tokens and then their scales, as a page's block has them
// (a page of at most 128 tokens, a power of two, is one run and one copy).
template <bool LIST>
struct alignas(16) Stage {
  uint8_t k[kBlock * kKvBytes], v[kBlock * kKvBytes];
  int pos[LIST ? kBlock : 1];  // the entries' positions, -1: none
  uint32_t there;              // no list: bit i, tokens 16i .. 16i + 15 are there
};

// x / 16 / (page_size / 16) for x < 2^30: the page of a position.
__device__ __forceinline__ int page_index(const AttnArgs& a, int pos) {
  const uint32_t x = (uint32_t)pos >> 4;
  return a.page_magic ? (int)__umulhi(x, a.page_magic) : (int)x;
}

// What a row holds: its length and first visible position, its tokens (list
// entries) [from, to), cut into blocks; one block even if it has none, for its
// output.  A unit costs its blocks and kUnitCost more (its queries, the merge of
// its warps' sums): work is shared out by that cost.
constexpr int kUnitCost = 4;
struct Range {
  int len, start, from, to, blocks, cost;
};
template <bool LIST>
__device__ __forceinline__ Range row_range(const AttnArgs& a, int b) {
  Range r;
  r.len = max(0, min(__ldg(a.kv_len + b), a.max_len));
  r.start = a.kv_start ? max(0, __ldg(a.kv_start + b)) : 0;
  if (LIST) {
    r.from = 0;
    r.to = max(0, min(__ldg(a.count + b), a.max_sel));
  } else {
    const int p = r.len - a.Tq;  // the first query's position
    r.from = (a.window > 0 ? max(r.start, p - a.window + 1) : r.start) & ~(kBlock - 1);
    r.to = r.len;
  }
  r.blocks = max(1, (r.to - r.from + kBlock - 1) / kBlock);
  r.cost = a.whole ? 1 : r.blocks + kUnitCost;
  return r;
}

// The place of query row r (token r / G, head r % G of the kv head) among [B, Tq, n_q].
__device__ __forceinline__ int64_t out_row(const AttnArgs& a, int b, int kh, int G, int r) {
  const int tq = r / G;
  return ((int64_t)b * a.Tq + tq) * a.n_q + kh * G + (r - tq * G);
}

__device__ __forceinline__ uint64_t div_small(uint64_t x, uint64_t y) {
  return ((x | y) >> 32) == 0 ? (uint32_t)x / (uint32_t)y : x / y;
}

__device__ __forceinline__ void arrive_many(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

template <int N>
__device__ __forceinline__ void named_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

// The walk over a CTA's blocks: segments of units (a row's kv head and tile of
// query rows), in the same order for the producer and the consumers.
template <bool LIST>
struct Walk {
  int64_t w, end, base;  // where it is and ends among all costs; the cost of the rows before b (for one unit)
  int b, units;
  Range rg;
  // the current segment: blocks [i0, i1) of a unit; i1 = i0 where only a unit's extra cost lies in the range
  int unit, i0, i1;
  int64_t next_w;
  __device__ __forceinline__ void segment(bool whole) {
    const int64_t x = w - base * units;
    unit = (int)div_small(x, rg.cost);
    if (whole) {
      next_w = w + 1;
      i0 = 0;
      i1 = rg.blocks;
      return;
    }
    const int x0 = (int)(x - (int64_t)unit * rg.cost), x1 = (int)min((int64_t)rg.cost, x0 + (end - w));
    next_w = w + (x1 - x0);
    i0 = min(x0, rg.blocks);
    i1 = min(x1, rg.blocks);
  }
  __device__ __forceinline__ bool more() const { return w < end; }
  __device__ __forceinline__ void next(const AttnArgs& a) {
    w = next_w;
    if (w >= end) return;
    if (w == (base + rg.cost) * units) {  // the next row
      base += rg.cost;
      rg = row_range<LIST>(a, ++b);
    }
    segment(a.whole);
  }
};

template <class T, int NT, int P, bool LIST>
__global__ void __launch_bounds__(Shape<NT, P>::kThreads, kCtas) kv4_attn_kernel(const AttnArgs a) {
  using S = Shape<NT, P>;
  constexpr int kRows = S::kRows, H = 2, kWarps = S::kWarps;  // H: 16-token halves of a tile
  constexpr bool kQReg = NT == 1;
  using St = Stage<LIST>;
  constexpr int kStages = ring_stages(NT), kMost = ring_most(NT, P);
  static_assert(ring_is_sound<kStages, kWarps, kMost>());
  using RingT = Ring<kStages>;
  extern __shared__ __align__(128) uint8_t smem[];
  St* ring = reinterpret_cast<St*>(smem);
  // the queries, when they are not kept in registers, then the merge's outputs of four warps
  uint2* sq = reinterpret_cast<uint2*>(ring + kStages);
  float* so = reinterpret_cast<float*>(sq + (kQReg ? 0 : NT * P * 8 * 32));
  __shared__ uint64_t full[2 * kStages], empty[kStages];
  __shared__ int64_t sums[kWarps + 1], found[2];
  __shared__ float2 sml[4][kRows];
  __shared__ float scoef[kRows];
  __shared__ int abort_flag;
  __shared__ int4 place[kTiles];  // of a tile in a stage: its halves' codes and scales
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.n_q / a.c.n_heads;

  // ---- this CTA's share of the work
  Walk<LIST> wk;
  wk.w = wk.end = 0;
  wk.units = a.c.n_heads * a.row_tiles;
  {
    if (threadIdx.x == 0) {
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&full[2 * i], LIST ? 64 : 1);
        mbar_init(&full[2 * i + 1], LIST ? 64 : 1);
        mbar_init(&empty[i], kTiles);
      }
      abort_flag = 0;
      for (int i = 0; i < kTiles; ++i) {
        const int t0 = kTok * i, t1 = t0 + 16, s0 = t0 / a.run, s1 = t1 / a.run;
        place[i] = make_int4(s0 * a.run * kKvBytes + (t0 - s0 * a.run) * kKvCodeBytes,
                             s0 * a.run * kKvBytes + a.run * kKvCodeBytes + (t0 - s0 * a.run) * kKvScaleBytes,
                             s1 * a.run * kKvBytes + (t1 - s1 * a.run) * kKvCodeBytes,
                             s1 * a.run * kKvBytes + a.run * kKvCodeBytes + (t1 - s1 * a.run) * kKvScaleBytes);
      }
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    int64_t total;
    bool mine_to_do = true;
    const auto take_share = [&] {  // of `total`
      const int64_t n_cta = min((int64_t)gridDim.x, total);
      mine_to_do = blockIdx.x < n_cta;
      if (!mine_to_do) return;
      wk.w = div_small(total * blockIdx.x, n_cta);
      wk.end = div_small(total * (blockIdx.x + 1), n_cta);
    };
    if (a.c.B <= 32) {  // every warp finds its place by itself, a lane a row
      const Range r = row_range<LIST>(a, min(lane, a.c.B - 1));
      int upto = lane < a.c.B ? r.cost : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += x;
      }
      total = (int64_t)__shfl_sync(0xffffffffu, upto, 31) * wk.units;
      take_share();
      wk.b = min(__popc(__ballot_sync(0xffffffffu, (int64_t)upto * wk.units <= wk.w)), a.c.B - 1);
      wk.base = __shfl_sync(0xffffffffu, upto - r.cost, wk.b);
      wk.rg = {__shfl_sync(0xffffffffu, r.len, wk.b),  __shfl_sync(0xffffffffu, r.start, wk.b),
               __shfl_sync(0xffffffffu, r.from, wk.b), __shfl_sync(0xffffffffu, r.to, wk.b),
               __shfl_sync(0xffffffffu, r.blocks, wk.b), __shfl_sync(0xffffffffu, r.cost, wk.b)};
    } else {  // rows in order, `per` a thread
      const int per = (a.c.B + S::kThreads - 1) / S::kThreads, first = threadIdx.x * per;
      int64_t mine = 0;
      for (int i = first; i < min(first + per, a.c.B); ++i) mine += row_range<LIST>(a, i).cost;
      int64_t upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += x;
      }
      if (lane == 31) sums[warp] = upto;
      __syncthreads();
      total = 0;
#pragma unroll
      for (int i = 0; i < kWarps + 1; ++i) {
        if (i < warp) upto += sums[i];
        total += sums[i];
      }
      total *= wk.units;
      take_share();
      int64_t before = upto - mine;
      if (mine_to_do && wk.w >= before * wk.units && wk.w < upto * wk.units) {
        int i = first;
        for (;; ++i) {
          const int cost = row_range<LIST>(a, i).cost;
          if (wk.w < (before + cost) * wk.units) break;
          before += cost;
        }
        found[0] = i;
        found[1] = before;
      }
      __syncthreads();
      if (mine_to_do) {
        wk.b = (int)found[0];
        wk.base = found[1];
        wk.rg = row_range<LIST>(a, wk.b);
      }
    }
    if (!mine_to_do) {
      if (threadIdx.x == 0 && !a.whole) a.share[blockIdx.x].b = -1;
      return;
    }
    wk.segment(a.whole);
    const int64_t n_cta = min((int64_t)gridDim.x, total);
    if (threadIdx.x == 32 && !a.whole) {
      // the CTAs c with total * c / n_cta <= x own block x: the last of them is ((x + 1) * n_cta - 1) / total
      Share sh = {-1, wk.unit, 0, 0};
      const int64_t w0 = wk.base * wk.units + (int64_t)wk.unit * wk.rg.cost, w1 = w0 + wk.rg.blocks;
      const int64_t prev = blockIdx.x ? (int64_t)div_small(total * (blockIdx.x - 1), n_cta) : 0;
      if (wk.i0 > 0 && wk.i0 < wk.rg.blocks && prev <= w0) {
        sh.b = wk.b;
        sh.parts = (int)div_small(w1 * n_cta - 1, total) - (int)blockIdx.x + 2;
        sh.slot0 = 2 * ((int)blockIdx.x - 1) + (w0 > prev ? 1 : 0);
      }
      a.share[blockIdx.x] = sh;
    }
    __syncthreads();  // the barriers are there
  }

  if (warp == kWarps) {
    // ---- the producer: a stage for every block, as soon as the consumers have left it
    const int scales_at = a.c.page_size * kKvCodeBytes;
    bool ok = true;
    uint32_t blk = 0;  // blocks so far
    for (; ok && wk.more(); wk.next(a)) {
      const int kh = wk.unit / a.row_tiles;
      const int32_t* table = a.c.table + wk.b * a.c.table_stride;
      const uint8_t* kp = a.c.k + kh * a.c.head_stride;
      const uint8_t* vp = a.c.v + kh * a.c.head_stride;
      // looked up a block ahead: list, the positions of entries lane + 32e; otherwise, a lane a run (`run` tokens of
      // a page lie together), its page
      constexpr int kPer = kBlock / 32;
      int ahead[LIST ? kPer : 1];
      const auto look = [&](int i) {
        const int n = wk.rg.from + i * kBlock;
        if constexpr (LIST) {
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            const int x = n + 32 * e + lane;
            ahead[e] = i < wk.i1 && x < wk.rg.to ? __ldg(a.idx + (int64_t)wk.b * a.max_sel + x) : -1;
          }
        } else {
          const int at = n + lane * a.run;
          ahead[0] = i < wk.i1 && lane * a.run < kBlock && at < wk.rg.to ? __ldg(table + page_index(a, at)) : -1;
        }
      };
      look(wk.i0);
      for (int i = wk.i0; i < wk.i1; ++i) {
        const int n = wk.rg.from + i * kBlock;
        const int stage = RingT::stage(blk);
        uint64_t* landed = &full[RingT::full(blk)];
        St& st = ring[stage];
        if constexpr (LIST) {
          int pos[kPer], page[kPer];
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            pos[e] = ahead[e] < 0 || ahead[e] >= wk.rg.len ? -1 : ahead[e];
            page[e] = pos[e] >= 0 ? __ldg(table + page_index(a, pos[e])) : -1;
          }
          look(i + 1);
          ok = mbar_wait_bounded(&empty[stage], RingT::empty_parity(blk), &abort_flag, &g_kv4_err);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            if (page[e] < 0 || page[e] >= a.c.n_pages) page[e] = pos[e] = -1;
            const int64_t from = max(page[e], 0) * a.c.page_stride;
            const int slot = pos[e] >= 0 ? pos[e] - page_index(a, pos[e]) * a.c.page_size : 0;
            const int64_t off = pos[e] >= 0 ? from + slot * kKvCodeBytes : -1;
            st.pos[32 * e + lane] = pos[e];
            if (pos[e] >= 0) {
              const int to = kBlock * kKvCodeBytes + (32 * e + lane) * kKvScaleBytes;
              cp_async4(st.k + to, kp + from + scales_at + slot * kKvScaleBytes);
              cp_async4(st.v + to, vp + from + scales_at + slot * kKvScaleBytes);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {  // four lanes an entry's 64 bytes
              const int x = 8 * r + (lane >> 2);
              const int64_t o = __shfl_sync(0xffffffffu, off, x);
              if (o >= 0) {
                cp_async16(st.k + (32 * e + x) * kKvCodeBytes + 16 * (lane & 3), kp + o + 16 * (lane & 3));
                cp_async16(st.v + (32 * e + x) * kKvCodeBytes + 16 * (lane & 3), vp + o + 16 * (lane & 3));
              }
            }
          }
          cp_async_arrive(landed);
          mbar_arrive(landed);
        } else {
          const int page = ahead[0];
          look(i + 1);
          const bool there = page >= 0 && page < a.c.n_pages;
          const uint32_t runs = __ballot_sync(0xffffffffu, there);
          const uint32_t chunks = __ballot_sync(0xffffffffu, lane * 16 < kBlock && ((runs >> (lane * 16 / a.run)) & 1u));
          ok = mbar_wait_bounded(&empty[stage], RingT::empty_parity(blk), &abort_flag, &g_kv4_err);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            st.there = chunks;
            mbar_arrive_expect_tx(landed, (uint32_t)__popc(runs) * a.run * kKvBytes * 2);
          }
          __syncwarp();
          if (there) {
            const int at = n + lane * a.run, slot = at - page_index(a, at) * a.c.page_size;
            const int64_t from = page * a.c.page_stride;
            uint8_t* ks = st.k + lane * a.run * kKvBytes;
            uint8_t* vs = st.v + lane * a.run * kKvBytes;
            if (a.run == a.c.page_size) {
              bulk_g2s(ks, kp + from, a.run * kKvBytes, landed);
              bulk_g2s(vs, vp + from, a.run * kKvBytes, landed);
            } else {
              const int codes = a.run * kKvCodeBytes, scales = a.run * kKvScaleBytes;
              bulk_g2s(ks, kp + from + slot * kKvCodeBytes, codes, landed);
              bulk_g2s(vs, vp + from + slot * kKvCodeBytes, codes, landed);
              bulk_g2s(ks + codes, kp + from + scales_at + slot * kKvScaleBytes, scales, landed);
              bulk_g2s(vs + codes, vp + from + scales_at + slot * kKvScaleBytes, scales, landed);
            }
          }
        }
        ++blk;
      }
      if (!ok) break;
    }
    // the last copies into every stage land before the CTA ends, whichever wait ran out
    for (uint32_t b = blk > kStages ? blk - kStages : 0; b < blk; ++b) mbar_drain(&full[RingT::full(b)], RingT::full_parity(b), &g_kv4_err);
    return;
  }

  // ---- the consumers
  const int g = lane >> 2, t = lane & 3;
  const int tk = (g >> 1) + 4 * (g & 1);  // the token of key row g (row g + 8: + 8)
  const int grp = g >> 1;                 // the scale group of dims 16g ..
  const bool bent = a.softcap > 0.f || a.slopes;
  uint32_t blocks_done = 0;               // of the segments before
  int slot = 0;                           // of the segment's partial result: 0 if the range begins with it
  bool ok = true;
  for (; wk.more(); wk.next(a)) {
    if (wk.i0 == wk.i1) {
      slot = 1;
      continue;
    }
    const Range& rg = wk.rg;
    const bool complete = wk.i0 == 0 && wk.i1 == rg.blocks;
    const int kh = wk.unit / a.row_tiles, r0 = (wk.unit - kh * a.row_tiles) * kRows;
    const int rows = min(kRows, a.Tq * G - r0), len = rg.len;
    const int p_first = len - a.Tq + r0 / G, p_last = len - a.Tq + (r0 + rows - 1) / G;
    const auto low_of = [&](int p) { return a.window > 0 ? max(rg.start, p - a.window + 1) : rg.start; };
    const int lo_first = low_of(p_first), lo_last = low_of(p_last);

    // the queries: row g of each tile, dims 32t .. 32t+31, as f16 pieces of q * 2^-e, |.| < 2^8.  One tile: every
    // warp keeps them; more: a warp a tile puts them into shared memory
    uint32_t qf[kQReg ? P : 1][8][2];
    float coef[NT][2];            // of columns 2t, 2t + 1: scale * 2^e (* log2 e without a cap)
    float slope[NT][2];
    int pq[NT][2];
    const auto row_at = [&](int r, int& tq) {  // query row r of the segment: its token, and its head
      tq = (r0 + r) / G;
      return kh * G + (r0 + r - tq * G);
    };
    if (kQReg || warp < NT) {
      const int nt = kQReg ? 0 : warp, r = nt * 8 + g;
      float v[32];
      if (r < rows) {
        int tq;
        const int head = row_at(r, tq);
        const T* q = static_cast<const T*>(a.q) + ((int64_t)wk.b * a.Tq + tq) * a.q_stride + head * kKvDim + 32 * t;
#pragma unroll
        for (int i = 0; i < 4; ++i) load8(q + 8 * i, *reinterpret_cast<float(*)[8]>(v + 8 * i));
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
      }
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) m = fmax_nan(m, fabsf(v[i]));
      m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = max(-110, min(120, (int)(__float_as_uint(m) >> 23) - 127 - 7));  // m * 2^-e in [2^7, 2^8)
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      // (one that is not finite makes its scores NaN, as scores of minus infinity alone would pass for masked ones;
      // a cap turns infinite scores into finite ones)
      const bool finite = m < INFINITY;
      const float c = finite || a.softcap > 0.f ? bounded(a.coef * __uint_as_float((uint32_t)(127 + e) << 23)) : nan_f32();
      if constexpr (kQReg) {
        coef[0][0] = __shfl_sync(0xffffffffu, c, 8 * t);
        coef[0][1] = __shfl_sync(0xffffffffu, c, 8 * t + 4);
      } else if (t == 0) {
        scoef[r] = c;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = v[4 * j + 2 * i] * down, y = v[4 * j + 2 * i + 1] * down;
          hi[i] = pack_f16(x, y);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi[i]));
          lo[i] = finite ? pack_f16(x - f.x, y - f.y) : 0u;
        }
        if constexpr (kQReg) {
          qf[0][j][0] = hi[0];
          qf[0][j][1] = hi[1];
          if constexpr (P == 2) {
            qf[P - 1][j][0] = lo[0];
            qf[P - 1][j][1] = lo[1];
          }
        } else {
          sq[((nt * P) * 8 + j) * 32 + lane] = make_uint2(hi[0], hi[1]);
          if constexpr (P == 2) sq[((nt * P + 1) * 8 + j) * 32 + lane] = make_uint2(lo[0], lo[1]);
        }
      }
    }
    if constexpr (!kQReg) named_barrier<32 * kWarps>();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = nt * 8 + 2 * t + i;
        int tq;
        const int head = row_at(min(r, rows - 1), tq);
        pq[nt][i] = len - a.Tq + tq;
        slope[nt][i] = a.slopes ? __ldg(a.slopes + head) * kLog2e : 0.f;
        if constexpr (!kQReg) coef[nt][i] = scoef[r];
      }

    // the running maximum is kLift - base; lim is -infinity until the row has seen something
    float o[NT][8][4], base[NT][2], lim[NT][2], l[NT][2];
    bool low = false;  // held kDrop lower
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
      base[nt][0] = base[nt][1] = 0.f;
      lim[nt][0] = lim[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    // One tile.  FAST: its scales are within f16's range (fast_scales).  WHOLE: every row sees all its tokens.
    const auto tile = [&](auto fast_c, auto whole_c, const St& st, int in_stage, const int4 pl, int j0, uint32_t there) {
      constexpr bool FAST = decltype(fast_c)::value, WHOLE = decltype(whole_c)::value;
      const int at = in_stage * kTok;
      const int codes[2] = {pl.x, pl.z}, scales[2] = {pl.y, pl.w};  // of its halves
      const auto k_scales = [&](int h, int k) {  // of the key of token k of half h
        return *reinterpret_cast<const uint32_t*>(st.k + scales[h] + k * kKvScaleBytes);
      };
      const auto v_scales = [&](int h, int k) {
        return *reinterpret_cast<const uint32_t*>(st.v + scales[h] + k * kKvScaleBytes);
      };
      if constexpr (!FAST) {
        const uint32_t r = top_scale(lane < 16 ? v_scales(0, lane) : v_scales(1, lane - 16));
        if (!low && __any_sync(0xffffffffu, r > kHugeScale)) {
          low = true;
          const float f = ex2(-kDrop);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              base[nt][i] -= kDrop;
              lim[nt][i] -= kDrop;
              l[nt][i] *= f;
#pragma unroll
              for (int d = 0; d < 8; ++d) {
                o[nt][d][i] *= f;
                o[nt][d][i + 2] *= f;
              }
            }
        }
      }
      const float lift = !FAST && low ? kLift - kDrop : kLift;
      // position of token k of the tile, -1 where none is
      const auto pos_at = [&](int k) { return LIST ? st.pos[at + k] : (there >> (k >> 4)) & 1u ? j0 + k : -1; };
      // ---- scores: S[token][row] = K q^T
      float s[H][NT][4];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        uint32_t f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w = k_scales(h, 8 * i + tk);
          if constexpr (FAST) f[i] = fast_factor(__byte_perm(w, 0, 0x4040 + 0x0101 * t));
          else f[i] = group_factor(w, t, top_scale(w)) * 0x10001u;
        }
        const uint4 k0 = *reinterpret_cast<const uint4*>(st.k + codes[h] + tk * kKvCodeBytes + 16 * t);
        const uint4 k1 = *reinterpret_cast<const uint4*>(st.k + codes[h] + (8 + tk) * kKvCodeBytes + 16 * t);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t x[4], y[4];
          e2m1x8_to_f16(w0[i], x);
          e2m1x8_to_f16(w1[i], y);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t A[4] = {hmul2(x[2 * k], f[0]), hmul2(y[2 * k], f[1]), hmul2(x[2 * k + 1], f[0]),
                                   hmul2(y[2 * k + 1], f[1])};
            const int j = 2 * i + k;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int p = 0; p < P; ++p) {
                const uint2 q2 = kQReg ? make_uint2(qf[kQReg ? p : 0][j][0], qf[kQReg ? p : 0][j][1])
                                       : sq[((nt * P + p) * 8 + j) * 32 + lane];
                if (j == 0 && p == 0) mma_f16_zero(s[h][nt], A, q2.x, q2.y);
                else mma_f16(s[h][nt], A, q2.x, q2.y);
              }
          }
        }
      }
      // ---- softmax weights in log2 units
      float k_top[H][2], v_exp[H][2];
      if constexpr (!FAST) {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = k_scales(h, 8 * i + tk), r = top_scale(w);
            k_top[h][i] = has_nan(w) ? nan_f32() : e8m0_value(r);
            v_exp[h][i] = (float)((int)top_scale(v_scales(h, 8 * i + tk)) - 127);
          }
      }
      uint32_t pf[H][NT][P][2];
      float grow[NT][2];  // general form: the factor of a row's products
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const auto k_coef = [&](int h, int c) {  // what a score is multiplied by
          return FAST ? coef[nt][c & 1] : bounded(coef[nt][c & 1] * k_top[h][c >> 1]);
        };
        // x: log2 of the weights, relative to the running maximum and times 2^kLift.  [half][c]: tokens tk, tk,
        // tk + 8, tk + 8; columns 2t, 2t + 1, 2t, 2t + 1
        float x[H][4];
        if (!bent) {
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              x[h][c] = fmaf(s[h][nt][c], k_coef(h, c), base[nt][c & 1]);
        } else {
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              x[h][c] = s[h][nt][c] * k_coef(h, c);
          if (a.softcap > 0.f) {  // coef holds scale / softcap
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float y = x[h][c];
                if constexpr (P == 2) {  // fp32
                  x[h][c] = a.cap_log2 * tanhf(y);
                } else {
                  x[h][c] = capped(a, y);
                  if (a.softcap > kFarCap && fabsf(y) < 0.25f) x[h][c] = a.cap_log2 * tanh_near(y);
                }
              }
          }
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (a.slopes)
                x[h][c] = fmaf(slope[nt][c & 1], (float)(pos_at(16 * h + 8 * (c >> 1) + tk) - pq[nt][c & 1]), x[h][c]);
              x[h][c] += base[nt][c & 1];
            }
        }
        if constexpr (!WHOLE) {
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int j = pos_at(16 * h + 8 * (c >> 1) + tk), p = pq[nt][c & 1];
              if (j > p || j < low_of(p)) x[h][c] = -INFINITY;
            }
        }
        // the maximum moves only where a weight would pass 2^(kLift + kLazy), or at what a row sees first
        float m[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) m[i] = fmaxf(fmaxf(x[0][i], x[0][i + 2]), fmaxf(x[1][i], x[1][i + 2]));
        if (__any_sync(0xffffffffu, m[0] > lim[nt][0] || m[1] > lim[nt][1])) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = m[i];
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            if (top > lim[nt][i]) {
              const float down = top - lift;
              const float f = lim[nt][i] == -INFINITY ? 0.f : ex2(-down);  // a row's first: there is nothing to rescale
              base[nt][i] -= down;
              lim[nt][i] = lift + kLazy;
#pragma unroll
              for (int h = 0; h < H; ++h) {
                x[h][i] -= down;
                x[h][i + 2] -= down;
              }
              l[nt][i] *= f;
#pragma unroll
              for (int d = 0; d < 8; ++d) {
                o[nt][d][i] *= f;
                o[nt][d][i + 2] *= f;
              }
            }
          }
        }
        if constexpr (!FAST) {  // the sum, then the weights times sizes, relative to their largest in the tile
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              l[nt][c & 1] += ex2(x[h][c]);
              x[h][c] += v_exp[h][c >> 1];
            }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(fmaxf(x[0][i], x[0][i + 2]), fmaxf(x[1][i], x[1][i + 2]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float up = fmaxf(top - kLift, -120.f);  // a row that sees nothing here: its weights are 0 all the same
            grow[nt][i] = ex2(up);
#pragma unroll
            for (int h = 0; h < H; ++h) {
              x[h][i] -= up;
              x[h][i + 2] -= up;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
          float w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            w[c] = ex2(x[h][c]);
            if constexpr (FAST) l[nt][c & 1] += w[c];
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t hi = pack_f16(w[2 * i], w[2 * i + 1]);
            pf[h][nt][0][i] = transpose8x8(hi);
            if constexpr (P == 2) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              pf[h][nt][1][i] = transpose8x8(pack_f16(w[2 * i] - f.x, w[2 * i + 1] - f.y));
            }
          }
        }
      }
      if constexpr (!FAST) {
        // a NaN scale makes its dimensions NaN for the rows that see the token, and for no other
        const uint32_t nans = __ballot_sync(0xffffffffu, has_nan(lane < 16 ? v_scales(0, lane) : v_scales(1, lane - 16)));
#pragma unroll 1
        for (int k = 0; k < kTok; ++k) {
          if (!((nans >> k) & 1u) || byte_of(k < 16 ? v_scales(0, k) : v_scales(1, k - 16), grp) != 255u) continue;
          const int j = pos_at(k);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (j <= pq[nt][i] && j >= low_of(pq[nt][i]))
#pragma unroll
                for (int d = 0; d < 8; ++d) o[nt][d][i] = o[nt][d][i + 2] = nan_f32();
        }
      }
      // ---- outputs: O[dim][row] += V^T P^T
      if constexpr (FAST) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          uint32_t f[2];  // factors of tokens (t, t + 4) and (t + 8, t + 12) for dims 16g ..
          uint2 vr[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) vr[i] = *reinterpret_cast<const uint2*>(st.v + codes[h] + (4 * i + t) * kKvCodeBytes + 8 * g);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t wa = v_scales(h, 8 * i + t), wb = v_scales(h, 8 * i + 4 + t);
            f[i] = fast_factor(__byte_perm(wa, wb, 0x4400 + 0x1111 * grp) & 0x00ff00ffu);
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // dims 16g .. +7, then +8 .. +15
            uint32_t ev[2][4], od[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t wa = half ? vr[2 * i].y : vr[2 * i].x, wb = half ? vr[2 * i + 1].y : vr[2 * i + 1].x;
              e2m1x8_to_f16((wa & 0x0f0f0f0fu) | ((wb << 4) & 0xf0f0f0f0u), ev[i]);
              e2m1x8_to_f16(((wa >> 4) & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u), od[i]);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const uint32_t A[4] = {hmul2(ev[0][m], f[0]), hmul2(od[0][m], f[0]), hmul2(ev[1][m], f[1]),
                                     hmul2(od[1][m], f[1])};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int p = 0; p < P; ++p) mma_f16(o[nt][4 * half + m], A, pf[h][nt][p][0], pf[h][nt][p][1]);
            }
          }
        }
      } else {
        uint32_t f[H][2];
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t wa = v_scales(h, 8 * i + t), wb = v_scales(h, 8 * i + 4 + t);
            const uint32_t fa = byte_of(wa, grp) == 255u ? 0u : group_factor(wa, grp, top_scale(wa));
            const uint32_t fb = byte_of(wb, grp) == 255u ? 0u : group_factor(wb, grp, top_scale(wb));
            f[h][i] = fa | (fb << 16);
          }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t ev[H][2], od[H][2];
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint8_t* at = st.v + codes[h] + (8 * i + t) * kKvCodeBytes + 8 * g + 4 * half;
              const uint32_t wa = *reinterpret_cast<const uint32_t*>(at);
              const uint32_t wb = *reinterpret_cast<const uint32_t*>(at + 4 * kKvCodeBytes);
              ev[h][i] = (wa & 0x0f0f0f0fu) | ((wb << 4) & 0xf0f0f0f0u);
              od[h][i] = ((wa >> 4) & 0x0f0f0f0fu) | (wb & 0xf0f0f0f0u);
            }
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            float acc[NT][4];
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const uint32_t A[4] = {hmul2(e2m1x2_to_f16(ev[h][0] >> (8 * m)), f[h][0]),
                                     hmul2(e2m1x2_to_f16(od[h][0] >> (8 * m)), f[h][0]),
                                     hmul2(e2m1x2_to_f16(ev[h][1] >> (8 * m)), f[h][1]),
                                     hmul2(e2m1x2_to_f16(od[h][1] >> (8 * m)), f[h][1])};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int p = 0; p < P; ++p) {
                  if (h == 0 && p == 0) mma_f16_zero(acc[nt], A, pf[h][nt][p][0], pf[h][nt][p][1]);
                  else mma_f16(acc[nt], A, pf[h][nt][p][0], pf[h][nt][p][1]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                o[nt][4 * half + m][c] = fmaf(acc[nt][c], grow[nt][c & 1], o[nt][4 * half + m][c]);
          }
        }
      }
    };
    // Tiles in turn; where the warps' registers allow, two at a time as long as there are two for each warp (one
    // at a time: 252 us where this takes 240, 8 x 131072 tokens).
    const TileOrder<kWarps, kMost> order((wk.i1 - wk.i0) * kTiles);
    for (int x = order.first(warp); x < order.n_tiles; x = order.next(x, warp)) {
      const int n = order.count(x);  // tiles from x on, of one block
      const uint32_t blk = blocks_done + (uint32_t)(x / kTiles);
      const int first = x % kTiles;
      St& st = ring[RingT::stage(blk)];
      const int j0 = rg.from + wk.i0 * kBlock + x * kTok;  // the first token (list: entry)
      // a wait that ran out ends the work, not the walk: the barriers below want every warp
      if (ok) ok = mbar_wait_bounded(&full[RingT::full(blk)], RingT::full_parity(blk), &abort_flag, &g_kv4_err);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        const uint32_t there = LIST ? 0u : st.there >> (first * H);
        uint32_t kw[kMost], vw[kMost];  // the scales of this lane's token in each tile
        int at[kMost];
        bool clear = !low;  // seen whole, and with fast scales
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          const int tile_i = i < n ? first + i : first;
          const int4 pl = place[tile_i];
          at[i] = (lane < 16 ? pl.y : pl.w) + (lane & 15) * kKvScaleBytes;
          kw[i] = *reinterpret_cast<const uint32_t*>(st.k + at[i]);
          vw[i] = *reinterpret_cast<const uint32_t*>(st.v + at[i]);
          clear = clear && fast_scales(kw[i], vw[i]);
          if constexpr (LIST) {
            const int j = st.pos[tile_i * kTok + lane];
            clear = clear && j >= lo_last && j <= p_first;
          }
        }
        if constexpr (!LIST) {
          const uint32_t all = n == 2 ? 15u : 3u;
          clear = clear && j0 >= lo_last && j0 + n * kTok - 1 <= p_first && (there & all) == all;
        }
        if (__all_sync(0xffffffffu, clear)) {
#pragma unroll 1
          for (int i = 0; i < n; ++i)
            tile(std::true_type{}, std::true_type{}, st, first + i, place[first + i], j0 + i * kTok, there >> (i * H));
        } else {
#pragma unroll 1
          for (int i = 0; i < n; ++i) {
            // what no row sees may hold anything: its scales are made harmless
            const int j = LIST ? st.pos[(first + i) * kTok + lane]
                               : (there >> (i * H + (lane >> 4))) & 1u ? j0 + i * kTok + lane : -1;
            const bool seen = j >= lo_first && j <= p_last;
            const int last = kMost - 1;
            if (!seen) {
              *reinterpret_cast<uint32_t*>(st.k + (i ? at[last] : at[0])) = 0x7f7f7f7fu;
              *reinterpret_cast<uint32_t*>(st.v + (i ? at[last] : at[0])) = 0x7f7f7f7fu;
            }
            const bool fast = !low && __all_sync(0xffffffffu, !seen || fast_scales(i ? kw[last] : kw[0], i ? vw[last] : vw[0]));
            const bool whole = __all_sync(0xffffffffu, j >= lo_last && j <= p_first);
            const bool any = __any_sync(0xffffffffu, seen);
            __syncwarp();
            if (any) {
              const int4 pl = place[first + i];
              if (!fast) tile(std::false_type{}, std::false_type{}, st, first + i, pl, j0 + i * kTok, there >> (i * H));
              else if (whole) tile(std::true_type{}, std::true_type{}, st, first + i, pl, j0 + i * kTok, there >> (i * H));
              else tile(std::true_type{}, std::false_type{}, st, first + i, pl, j0 + i * kTok, there >> (i * H));
            }
          }
          fence_proxy_async_smem();  // the stage's next copy comes after these
        }
        __syncwarp();
        if (lane == 0) arrive_many(&empty[RingT::stage(blk)], n);
      }
    }
    blocks_done += (uint32_t)(wk.i1 - wk.i0);

    // ---- the warps' sums merged in shared memory: those past the fourth add to the first ones, then all threads add
    // up the four
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], x);
    float M[NT][2];  // the maxima less kLift, which all sums have
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) M[nt][i] = lim[nt][i] == -INFINITY ? kNoMax : -base[nt][i];
    const auto put = [&](int to) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = nt * 8 + 2 * t + i;
          float* row = so + (to * kRows + r) * kORow;
#pragma unroll
          for (int d = 0; d < 8; ++d)  // dims 16g + 2d, + 1 at 16d + 2g, + 1
            *reinterpret_cast<float2*>(row + 16 * d + 2 * g) = make_float2(o[nt][d][i], o[nt][d][i + 2]);
          if (g == 0) sml[to][r] = make_float2(M[nt][i], l[nt][i]);
        }
    };
    if (warp >= 4) put(warp - 4);
    named_barrier<32 * kWarps>();
    if (warp < kWarps - 4) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = nt * 8 + 2 * t + i;
          const float* row = so + (warp * kRows + r) * kORow;
          const float2 ml = sml[warp][r];
          const float m = fmaxf(M[nt][i], ml.x), f0 = ex2(M[nt][i] - m), f1 = ex2(ml.x - m);
          M[nt][i] = m;
          l[nt][i] = l[nt][i] * f0 + ml.y * f1;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            const float2 x = *reinterpret_cast<const float2*>(row + 16 * d + 2 * g);
            o[nt][d][i] = o[nt][d][i] * f0 + x.x * f1;
            o[nt][d][i + 2] = o[nt][d][i + 2] * f0 + x.y * f1;
          }
        }
    }
    named_barrier<32 * kWarps>();
    if (warp < 4) put(warp);
    named_barrier<32 * kWarps>();
    for (int x = threadIdx.x; x < rows * kKvDim; x += 32 * kWarps) {
      const int r = x / kKvDim, d = x % kKvDim;
      const int at = r * kORow + ((d & 15) >> 1) * 16 + (d >> 4) * 2 + (d & 1);
      float m = kNoMax, num = 0.f, den = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, sml[i][r].x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 ml = sml[i][r];
        const float f = ex2(ml.x - m);
        den = fmaf(f, ml.y, den);
        num = fmaf(f, so[i * kRows * kORow + at], num);
      }
      if (complete) {
        store1(static_cast<T*>(a.out) + out_row(a, wk.b, kh, G, r0 + r) * kKvDim + d, den == 0.f ? 0.f : num / den);
      } else {
        const int64_t R = ((int64_t)blockIdx.x * 2 + slot) * kRows + r;
        a.part_o[R * kKvDim + d] = num;
        if (d == 0) a.part_ml[R] = make_float2(m, den);
      }
    }
    slot = 1;
    named_barrier<32 * kWarps>();  // the shared memory is used again
  }
}

// Merges the parts of the units that several CTAs share.  CTA c looks at what
// CTA c + 1 of the attention said of the unit in which its range begins; out =
// sum 2^(m_s - m) o_s / sum 2^(m_s - m) l_s, a lane four dimensions.  WIDE (few
// units, many parts): a CTA a row, the parts shared by its eight warps;
// otherwise a warp a row.
constexpr int kCombineThreads = 256, kCombineWarps = kCombineThreads / 32;
template <class T, bool WIDE>
__global__ void __launch_bounds__(kCombineThreads) kv4_combine_kernel(const AttnArgs a, int tile_rows) {
  __shared__ float4 so[WIDE ? kCombineThreads : 1];
  __shared__ float2 sml[kCombineWarps];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int4 raw = __ldcg(reinterpret_cast<const int4*>(a.share + blockIdx.x + 1));
  const Share sh = {raw.x, raw.y, raw.z, raw.w};
  if (sh.b < 0) return;
  const int G = a.n_q / a.c.n_heads, kh = sh.unit / a.row_tiles, r0 = (sh.unit - kh * a.row_tiles) * tile_rows;
  const int rows = min(tile_rows, a.Tq * G - r0);
  constexpr int kStep = WIDE ? kCombineWarps : 1, kUnroll = 8;
  for (int r = WIDE ? blockIdx.y : warp; r < rows; r += WIDE ? gridDim.y : kCombineWarps) {
    float m = kNoMax, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = WIDE ? warp : 0; i0 < sh.parts; i0 += kUnroll * kStep) {
      float2 ml[kUnroll];
      float4 o[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int i = i0 + k * kStep;
        ml[k] = make_float2(kNoMax, 0.f);
        o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < sh.parts) {
          const int64_t at = (int64_t)(i == 0 ? sh.slot0 : 2 * ((int)blockIdx.x + i)) * tile_rows + r;
          ml[k] = __ldcg(a.part_ml + at);
          o[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * kKvDim) + lane);
        }
      }
      float mn = m;
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) mn = fmaxf(mn, ml[k].x);
      const float f0 = ex2(m - mn);
      m = mn;
      den *= f0;
      num = make_float4(num.x * f0, num.y * f0, num.z * f0, num.w * f0);
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const float f = ex2(ml[k].x - m);
        den = fmaf(f, ml[k].y, den);
        num = make_float4(fmaf(f, o[k].x, num.x), fmaf(f, o[k].y, num.y), fmaf(f, o[k].z, num.z), fmaf(f, o[k].w, num.w));
      }
    }
    if constexpr (WIDE) {
      so[threadIdx.x] = num;
      if (lane == 0) sml[warp] = make_float2(m, den);
      __syncthreads();
      if (warp == 0) {
        m = kNoMax;
#pragma unroll
        for (int i = 0; i < kCombineWarps; ++i) m = fmaxf(m, sml[i].x);
        den = 0.f;
        num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kCombineWarps; ++i) {
          const float f = ex2(sml[i].x - m);
          const float4 v = so[32 * i + lane];
          den = fmaf(f, sml[i].y, den);
          num = make_float4(fmaf(f, v.x, num.x), fmaf(f, v.y, num.y), fmaf(f, v.z, num.z), fmaf(f, v.w, num.w));
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    T* out = static_cast<T*>(a.out) + out_row(a, sh.b, kh, G, r0 + r) * kKvDim + 4 * lane;
    const float inv = den == 0.f ? 0.f : 1.f / den;
    store1(out, num.x * inv);
    store1(out + 1, num.y * inv);
    store1(out + 2, num.z * inv);
    store1(out + 3, num.w * inv);
  }
}

// How a call is cut: units (a row's kv head and a tile of 8 * nt query rows)
// times blocks of tokens, shared evenly by as many CTAs as the GPU holds at once,
// however the rows' lengths differ.
struct AttnPlan {
  int nt, row_tiles, grid;
  bool whole;  // a unit is one CTA's: no parts to merge
  bool wide;   // few units: each is shared by many CTAs
};

constexpr int kSms = 148;
constexpr int kWholeBlocks = 4;

// For rows of up to `tokens` tokens (list entries) each.
AttnPlan plan_for(const fm_kv4_cache* c, const fm_kv4_attn_desc* d, int64_t tokens) {
  AttnPlan p;
  const int rows = d->Tq * (d->n_q_heads / c->n_kv_heads);
  p.nt = rows <= 8 ? 1 : 2;
  p.row_tiles = (rows + 8 * p.nt - 1) / (8 * p.nt);
  const int64_t units = (int64_t)c->B * c->n_kv_heads * p.row_tiles;
  // Up to 512 tokens a CTA does a whole unit, which saves the merge and its launch (one row of 500 tokens and 8 kv
  // heads: 12.1 us, shared out 12.4; of 1001 tokens: 14.5 and 12.4).
  const int64_t blocks = (tokens + kBlock - 1) / kBlock;
  p.whole = blocks <= kWholeBlocks;
  p.grid = (int)std::min<int64_t>(p.whole ? units : units * blocks, kSms * kCtas);
  p.wide = 8 * units <= p.grid;
  return p;
}

AttnPlan plan_of(const fm_kv4_cache* c, const fm_kv4_attn_desc* d) {
  int64_t tokens = d->idx ? d->max_sel : d->max_len;
  if (!d->idx && d->window > 0)  // a row reaches back window + Tq - 1 from the last token, from a multiple of 128
    tokens = std::min(tokens, (int64_t)d->window + d->Tq - 1 + kBlock - 1);
  return plan_for(c, d, tokens);
}

// Bytes of the workspace's parts.
struct AttnSpace {
  size_t share, ml, o;
  size_t total() const { return share + ml + o; }
};
AttnSpace space_of(const AttnPlan& p) {
  if (p.whole) return {16, 0, 0};
  const size_t rows = (size_t)p.grid * 2 * 8 * p.nt;
  return {((size_t)p.grid * sizeof(Share) + 15) / 16 * 16, rows * sizeof(float2), rows * kKvDim * sizeof(float)};
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

fm_status check_attn(const fm_kv4_cache* c, const fm_kv4_attn_desc* d) {
  if (fm_status s = check_kv4_cache(c)) return s;
  if (!d || !dtype_ok(d->dtype) || d->Tq < 1 || d->n_q_heads < 1 || d->n_q_heads > 1024 ||
      d->n_q_heads % c->n_kv_heads)
    return FM_ERR_INVALID_ARG;
  if (d->Tq > kMaxTq) return FM_ERR_UNSUPPORTED;
  if (d->max_len < 1 || d->max_len > (int64_t)c->max_pages * c->page_size) return FM_ERR_INVALID_ARG;
  if (d->idx && (!d->count || d->max_sel < 1 || d->max_sel > (1 << 30))) return FM_ERR_INVALID_ARG;
  // within 2^32, and a cap not below 2^-32: their quotient times a query's power of two is then a number for queries
  // up to 2^70, and held to the largest one beyond (bounded)
  constexpr float kMost = 4294967296.f;
  if (!(std::fabs(d->scale) <= kMost) || d->window < 0) return FM_ERR_INVALID_ARG;
  if (d->softcap != 0.f && !(d->softcap >= 1.f / kMost && d->softcap <= kMost)) return FM_ERR_INVALID_ARG;
  return FM_OK;
}

}  // namespace

// Set by the first call (captures included): until then there is no error to read, and fm_sync_status does not
// copy the word (40 us with the copy, 30 without).
static std::atomic<bool> g_kv4_called{false};

int take_kv4_error() {
  if (!g_kv4_called.load(std::memory_order_acquire)) return kDevErrNone;
  int h = kDevErrNone;
  if (cudaMemcpyFromSymbol(&h, g_kv4_err, sizeof(int)) != cudaSuccess) {
    cudaGetLastError();
    return kDevErrNone;
  }
  if (h != kDevErrNone) {
    const int zero = kDevErrNone;
    cudaMemcpyToSymbol(g_kv4_err, &zero, sizeof(int));
  }
  return h;
}

}  // namespace fm

using namespace fm;

extern "C" size_t fm_kv4_attention_workspace_bytes(const fm_kv4_cache* c, const fm_kv4_attn_desc* d) {
  if (check_attn(c, d) != FM_OK) return 0;
  // of the longest call with these sizes, whatever its window, with a list or without: space grows with the tokens
  return space_of(plan_for(c, d, std::max(d->max_len, d->max_sel))).total();
}

namespace {

template <class T, int NT, int P, bool LIST>
fm_status launch_attn(const AttnArgs& a, int grid, cudaStream_t stream) {
  using S = Shape<NT, P>;
  constexpr int kSmem = ring_stages(NT) * (int)sizeof(Stage<LIST>) + (NT == 1 ? 0 : NT * P * 8 * 32 * (int)sizeof(uint2)) +
                        4 * S::kRows * kORow * (int)sizeof(float);
  static_assert((kSmem + 2048) * kCtas <= 228 * 1024, "shared memory of an SM, with the static and the reserved parts");
  static PerDeviceOnce once;
  int dev = 0;
  cudaGetDevice(&dev);
  if (fm_status s = smem_limit_once(once, dev, kv4_attn_kernel<T, NT, P, LIST>, kSmem)) return s;
  kv4_attn_kernel<T, NT, P, LIST><<<grid, S::kThreads, kSmem, stream>>>(a);
  note_launch();
  return check_launch();
}

template <class T, bool LIST>
fm_status launch_attn_nt(const AttnArgs& a, int nt, int grid, cudaStream_t stream) {
  constexpr int P = sizeof(T) == 4 ? 2 : 1;
  if (nt == 1) return launch_attn<T, 1, P, LIST>(a, grid, stream);
  return launch_attn<T, 2, P, LIST>(a, grid, stream);
}

}  // namespace

extern "C" fm_status fm_kv4_attention(const fm_kv4_cache* c, const fm_kv4_attn_desc* d, void* ws, size_t ws_bytes,
                                      cudaStream_t stream) {
  if (fm_status s = check_attn(c, d)) return s;
  if (!d->q || !d->out || !d->kv_len || !ws) return FM_ERR_INVALID_ARG;
  if (d->q_stride < (int64_t)d->n_q_heads * kKvDim) return FM_ERR_INVALID_ARG;
  if (!aligned(d->q, 16) || !aligned(d->out, 16) || (d->q_stride * dtype_size(d->dtype)) % 16 || !aligned(ws, 16) ||
      !aligned(d->kv_len, 4) || !aligned(d->kv_start, 4) || !aligned(d->idx, 4) || !aligned(d->count, 4) ||
      !aligned(d->slopes, 4))
    return FM_ERR_ALIGNMENT;
  if (ws_bytes < fm_kv4_attention_workspace_bytes(c, d)) return FM_ERR_INVALID_ARG;
  if (!g_kv4_called.load(std::memory_order_relaxed)) g_kv4_called.store(true, std::memory_order_release);
  const AttnPlan p = plan_of(c, d);
  const AttnSpace sp = space_of(p);
  AttnArgs a = {};
  a.c = kv4_view(*c);
  a.q = d->q;
  a.q_stride = d->q_stride;
  a.out = d->out;
  a.kv_len = d->kv_len;
  a.kv_start = d->kv_start;
  a.idx = d->idx;
  a.count = d->count;
  a.slopes = d->slopes;
  a.Tq = d->Tq;
  a.n_q = d->n_q_heads;
  a.max_len = d->max_len;
  a.max_sel = d->max_sel;
  a.window = d->window < d->max_len ? d->window : 0;  // a window that no row outgrows is none
  a.softcap = d->softcap;
  a.cap_log2 = d->softcap * kLog2e;
  a.coef = d->softcap > 0.f ? d->scale / d->softcap : d->scale * kLog2e;
  const int q16 = c->page_size / 16;
  a.page_magic = q16 == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + q16 - 1) / q16);
  a.row_tiles = p.row_tiles;
  a.whole = p.whole;
  a.run = d->idx ? kBlock : std::min(c->page_size & -c->page_size, kBlock);
  uint8_t* at = static_cast<uint8_t*>(ws);
  a.share = reinterpret_cast<Share*>(at);
  a.part_ml = reinterpret_cast<float2*>(at + sp.share);
  a.part_o = reinterpret_cast<float*>(at + sp.share + sp.ml);
  return by_dtype(d->dtype, [&](auto* tag) -> fm_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    const fm_status s = d->idx ? launch_attn_nt<T, true>(a, p.nt, p.grid, stream)
                               : launch_attn_nt<T, false>(a, p.nt, p.grid, stream);
    if (s != FM_OK || p.whole || p.grid == 1) return s;
    const cudaError_t e =
        p.wide ? launch_overlapped(kv4_combine_kernel<T, true>, dim3(p.grid - 1, 8 * p.nt), dim3(kCombineThreads), 0,
                                   stream, a, 8 * p.nt)
               : launch_overlapped(kv4_combine_kernel<T, false>, dim3(p.grid - 1), dim3(kCombineThreads), 0, stream, a,
                                   8 * p.nt);
    if (e != cudaSuccess) return record_cuda_error(e);
    note_launch();
    return check_launch();
  });
}
