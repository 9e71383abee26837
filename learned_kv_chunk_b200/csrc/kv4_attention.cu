// kv4_attention.cu -- attention over the 4-bit paged cache (fm_kv4_attention).
#include <algorithm>
#include <cmath>

#include "kv4.cuh"

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
  int row_tiles, chunk, splits;
  float* part_o;        // [B * Tq * n_q, splits, 128]
  float2* part_ml;      // [B * Tq * n_q, splits]: the maximum (log2 units), the sum
};

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTok = 32;                  // tokens a warp takes at a time
constexpr int kBlockTok = kTok * kWarps;  // tokens a CTA takes at a time
constexpr float kNoMax = -1e30f;          // the running maximum of a row that has seen nothing
constexpr float kLazy = 6.f;              // the maximum may be exceeded by 2^6 before the sums are rescaled
constexpr float kLift = 8.f;              // weights are held times 2^8: at most 2^14 in f16
constexpr int kORow = 132;                // floats between rows of the warps' outputs in shared memory

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

__device__ __forceinline__ uint4 ldg128(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg64(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// What a warp keeps of the tokens it is at, written by one lane a token.
struct TokenInfo {
  float k_factor;   // 2^r of the key's largest scale r; the groups' factors are relative to it
  float v_exp;      // log2 of the value's
  float v_inv;      // 2^-v_exp
  int pos;          // position, -1 where there is none
  uint16_t kf[4];   // f16 factors of the key's groups, 2^(scale - r)
  uint16_t vf[4];   // and of the value's
};

__device__ __forceinline__ uint32_t max_byte(uint32_t w) {
  w = __vmaxu4(w, w >> 16);
  w = __vmaxu4(w, w >> 8);
  return w & 255u;
}

// f16 2^(byte - r) for r >= byte (0 below 2^-24).
__device__ __forceinline__ uint32_t group_factors(uint32_t w, int shift, uint32_t r) {
  const int e0 = 127 + (int)((w >> shift) & 255u) - (int)r, e1 = 127 + (int)((w >> (shift + 8)) & 255u) - (int)r;
  return pack_f16(__int_as_float(max(e0, 0) << 23), __int_as_float(max(e1, 0) << 23));
}

// Fills in a token's info; returns whether a scale of its value is NaN (the
// group's factor is then the f16 NaN 0x7fff, which no product may use).
__device__ __forceinline__ bool write_token(TokenInfo* ti, uint32_t kw, uint32_t vw, int pos) {
  if (pos < 0) kw = vw = 0u;
  const uint32_t kn = __vcmpeq4(kw, 0xffffffffu), vn = __vcmpeq4(vw, 0xffffffffu);  // NaN scales
  const uint32_t ks = kw & ~kn, vs = vw & ~vn;
  const uint32_t rk = max_byte(ks);
  uint32_t rv = max_byte(vs);
  rv = rv == 0u ? 127u : max(rv, 27u);  // a value of zeros has no size of its own; below 2^-100 none is kept
  TokenInfo t;
  t.k_factor = kn ? nan_f32() : __uint_as_float(rk ? rk << 23 : 0x00400000u);
  t.v_exp = (float)((int)rv - 127);
  t.v_inv = __uint_as_float(rv < 254u ? (254u - rv) << 23 : 0x00400000u);
  t.pos = pos;
  uint32_t f[4] = {group_factors(ks, 0, rk), group_factors(ks, 16, rk), group_factors(vs, 0, rv),
                   group_factors(vs, 16, rv)};
  if (vn) {
    f[2] |= __byte_perm(vn, 0, 0x1100) & 0x7fff7fffu;
    f[3] |= __byte_perm(vn, 0, 0x3322) & 0x7fff7fffu;
  }
  reinterpret_cast<uint4*>(ti)[0] = make_uint4(__float_as_uint(t.k_factor), __float_as_uint(t.v_exp),
                                               __float_as_uint(t.v_inv), (uint32_t)t.pos);
  reinterpret_cast<uint4*>(ti)[1] = make_uint4(f[0], f[1], f[2], f[3]);
  return vn != 0u;
}

// x / 16 / (page_size / 16) for x < 2^30: the page of a position.
__device__ __forceinline__ int page_index(const AttnArgs& a, int pos) {
  const uint32_t x = (uint32_t)pos >> 4;
  return a.page_magic ? (int)__umulhi(x, a.page_magic) : (int)x;
}

template <class T, int NT, int P, bool LIST>
__global__ void __launch_bounds__(kThreads) kv4_attn_kernel(const AttnArgs a) {
  constexpr int kRows = 8 * NT;
  constexpr bool kQReg = NT == 1;
  extern __shared__ __align__(16) uint8_t smem[];
  // [token infos of the warps][queries, when they are not kept in registers]; at the end the warps' outputs
  TokenInfo* info = reinterpret_cast<TokenInfo*>(smem) + (threadIdx.x >> 5) * kTok;
  uint2* sq = reinterpret_cast<uint2*>(smem + kWarps * kTok * sizeof(TokenInfo));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int b = blockIdx.z, split = blockIdx.x;
  const int kh = blockIdx.y / a.row_tiles, r0 = (blockIdx.y - kh * a.row_tiles) * kRows;
  const int G = a.n_q / a.c.n_heads, rows = min(kRows, a.Tq * G - r0);
  const int len = max(0, min(__ldg(a.kv_len + b), a.max_len));
  const int start = a.kv_start ? max(0, __ldg(a.kv_start + b)) : 0;
  const int p_first = len - a.Tq + r0 / G, p_last = len - a.Tq + (r0 + rows - 1) / G;
  const auto low_of = [&](int p) { return a.window > 0 ? max(start, p - a.window + 1) : start; };
  const int lo_first = low_of(p_first), lo_last = low_of(p_last);
  // this CTA's tokens (list entries): [n0, n1)
  int n0, n1;
  if (LIST) {
    n0 = split * a.chunk;
    n1 = min(n0 + a.chunk, max(0, min(__ldg(a.count + b), a.max_sel)));
    if (p_last < 0) n1 = 0;
  } else {
    n0 = (lo_first & ~(kTok - 1)) + split * a.chunk;
    n1 = min(n0 + a.chunk, p_last + 1);
  }
  const auto part_row = [&](int r) {  // the row's place among [B, Tq, n_q]
    const int tq = (r0 + r) / G;
    return ((int64_t)b * a.Tq + tq) * a.n_q + kh * G + (r0 + r - tq * G);
  };
  if (n0 >= n1) {  // nothing here
    if (a.splits > 1) {
      if ((int)threadIdx.x < rows)
        a.part_ml[part_row(threadIdx.x) * a.splits + split] = make_float2(-INFINITY, 0.f);
    } else {
      for (int i = threadIdx.x; i < rows * kKvDim; i += kThreads)
        store1(static_cast<T*>(a.out) + part_row(i / kKvDim) * kKvDim + i % kKvDim, 0.f);
    }
    return;
  }

  // the queries: row g of each tile, dims 32t .. 32t+31, as f16 pieces of q * 2^-e, |.| < 2^8
  uint32_t qf[kQReg ? P : 1][8][2];
  float coef[NT][2];            // of columns 2t, 2t + 1: scale * 2^e (* log2 e without a cap)
  float slope[NT][2];
  int pq[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + g;
    float v[32];
    if (r < rows) {
      const int tq = (r0 + r) / G;
      const T* q = static_cast<const T*>(a.q) + ((int64_t)b * a.Tq + tq) * a.q_stride +
                   (kh * G + (r0 + r - tq * G)) * kKvDim + 32 * t;
#pragma unroll
      for (int i = 0; i < 4; ++i) load8(q + 8 * i, *reinterpret_cast<float(*)[8]>(v + 8 * i));
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.f;
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(v[i]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int e = max(-110, min(120, (int)(__float_as_uint(m) >> 23) - 127 - 7));  // m * 2^-e in [2^7, 2^8)
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    const float c = a.coef * __uint_as_float((uint32_t)(127 + e) << 23);
    coef[nt][0] = __shfl_sync(0xffffffffu, c, 8 * t);
    coef[nt][1] = __shfl_sync(0xffffffffu, c, 8 * t + 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float x = v[4 * j + 2 * i] * down, y = v[4 * j + 2 * i + 1] * down;
        hi[i] = pack_f16(x, y);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi[i]));
        lo[i] = pack_f16(x - f.x, y - f.y);
      }
      if constexpr (kQReg) {
        qf[0][j][0] = hi[0];
        qf[0][j][1] = hi[1];
        if constexpr (P == 2) {
          qf[1][j][0] = lo[0];
          qf[1][j][1] = lo[1];
        }
      } else if (warp == 0) {
        sq[((nt * P) * 8 + j) * 32 + lane] = make_uint2(hi[0], hi[1]);
        if constexpr (P == 2) sq[((nt * P + 1) * 8 + j) * 32 + lane] = make_uint2(lo[0], lo[1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = min(nt * 8 + 2 * t + i, rows - 1), tq = (r0 + rr) / G;
      pq[nt][i] = len - a.Tq + tq;
      slope[nt][i] = a.slopes ? __ldg(a.slopes + kh * G + (r0 + rr - tq * G)) * kLog2e : 0.f;
    }
  }
  if constexpr (!kQReg) __syncthreads();

  float o[NT][8][4], M[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
    M[nt][0] = M[nt][1] = kNoMax;
    l[nt][0] = l[nt][1] = 0.f;
  }

  const int32_t* table = a.c.table + b * a.c.table_stride;
  const int64_t head_off = kh * a.c.head_stride;
  const int scales_at = a.c.page_size * kKvCodeBytes;
  const int tk = (g >> 1) + 4 * (g & 1);  // the token of key row g (row g + 8: + 8)

  // ---- addresses.  Contiguous: the pages of the two 16-token halves of the
  // next tile (-1: not there).  List: this lane's token.
  int page[2] = {-1, -1}, pos_next = -1;
  const auto find = [&](int n) {  // the pages (the token) of the tile at n
    if constexpr (LIST) {
      const int i = n + lane;
      pos_next = i < n1 ? __ldg(a.idx + (int64_t)b * a.max_sel + i) : -1;
      if (pos_next < 0 || pos_next >= len) pos_next = -1;
      page[0] = pos_next >= 0 ? __ldg(table + page_index(a, pos_next)) : -1;
      if (page[0] < 0 || page[0] >= a.c.n_pages) page[0] = pos_next = -1;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        page[h] = n + 16 * h < n1 ? __ldg(table + page_index(a, n + 16 * h)) : -1;
        if (page[h] >= a.c.n_pages) page[h] = -1;
      }
    }
  };
  uint4 kr[2][2];     // codes of tokens tk, tk + 8 of each half: dims 32t ..
  uint2 vr[2][4];     // codes of tokens t + 4i of each half: dims 16g ..
  uint32_t kw, vw;    // scales of token `lane`
  int pos_cur;        // its position
  int64_t row_off = 0;           // list: byte offset of this lane's token's codes (and its scales)
  const uint8_t* base[2] = {};   // contiguous: offset of each half's codes in the pools
  int64_t off[2] = {};
  const auto load_k = [&](int n) {
    if constexpr (LIST) {
      const int pg = pos_next >= 0 ? page_index(a, pos_next) : 0;
      const int slot = pos_next >= 0 ? pos_next - pg * a.c.page_size : 0;
      const int64_t blk = max(page[0], 0) * a.c.page_stride + head_off;
      row_off = blk + slot * kKvCodeBytes;
      kw = __ldg(reinterpret_cast<const uint32_t*>(a.c.k + blk + scales_at + slot * kKvScaleBytes));
      vw = __ldg(reinterpret_cast<const uint32_t*>(a.c.v + blk + scales_at + slot * kKvScaleBytes));
      pos_cur = pos_next;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          kr[h][i] = ldg128(a.c.k + __shfl_sync(0xffffffffu, row_off, 16 * h + 8 * i + tk) + 16 * t);
    } else {
      int slot[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int pg = page_index(a, n + 16 * h);
        slot[h] = page[h] >= 0 ? n + 16 * h - pg * a.c.page_size : 0;
        off[h] = max(page[h], 0) * a.c.page_stride + head_off;
      }
      const int mine = lane >> 4;
      const int64_t so = (mine ? off[1] : off[0]) + scales_at + ((mine ? slot[1] : slot[0]) + (lane & 15)) * kKvScaleBytes;
      kw = __ldg(reinterpret_cast<const uint32_t*>(a.c.k + so));
      vw = __ldg(reinterpret_cast<const uint32_t*>(a.c.v + so));
      pos_cur = (mine ? page[1] : page[0]) >= 0 ? n + lane : -1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        off[h] += slot[h] * kKvCodeBytes;
#pragma unroll
        for (int i = 0; i < 2; ++i) kr[h][i] = ldg128(a.c.k + off[h] + (8 * i + tk) * kKvCodeBytes + 16 * t);
      }
    }
  };
  const auto load_v = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (LIST) vr[h][i] = ldg64(a.c.v + __shfl_sync(0xffffffffu, row_off, 16 * h + 4 * i + t) + 8 * g);
        else vr[h][i] = ldg64(a.c.v + off[h] + (4 * i + t) * kKvCodeBytes + 8 * g);
      }
  };

  int n = n0 + warp * kTok;
  if (n < n1) {
    find(n);
    load_k(n);
    load_v();
    find(n + kBlockTok);
  }
  for (; n < n1; n += kBlockTok) {
    const bool v_nan = __any_sync(0xffffffffu, write_token(info + lane, kw, vw, pos_cur));
    // every row sees every token of the tile
    const bool whole = __all_sync(0xffffffffu, pos_cur >= lo_last && pos_cur <= p_first);
    __syncwarp();
    const bool more = n + kBlockTok < n1;
    // ---- scores: S[token][row] = K q^T
    float s[2][NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[h][nt][c] = 0.f;
      const uint32_t f0 = info[16 * h + tk].kf[t] * 0x10001u, f1 = info[16 * h + tk + 8].kf[t] * 0x10001u;
      const uint32_t w0[4] = {kr[h][0].x, kr[h][0].y, kr[h][0].z, kr[h][0].w};
      const uint32_t w1[4] = {kr[h][1].x, kr[h][1].y, kr[h][1].z, kr[h][1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x[4], y[4];
        e2m1x8_to_f16(w0[i], x);
        e2m1x8_to_f16(w1[i], y);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t A[4] = {hmul2(x[2 * k], f0), hmul2(y[2 * k], f1), hmul2(x[2 * k + 1], f0),
                                 hmul2(y[2 * k + 1], f1)};
          const int j = 2 * i + k;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int p = 0; p < P; ++p) {
              if constexpr (kQReg) {
                mma_f16(s[h][nt], A, qf[p][j][0], qf[p][j][1]);
              } else {
                const uint2 q2 = sq[((nt * P + p) * 8 + j) * 32 + lane];
                mma_f16(s[h][nt], A, q2.x, q2.y);
              }
            }
        }
      }
    }
    if (more) {
      // the next tile's keys; its values when this tile's are used up
      // (off / row_off move on, so this tile's values must be here already)
      load_k(n + kBlockTok);
    }
    // ---- softmax weights, in log2 units, times the value's size
    uint32_t pf[2][NT][P][2];
    {
      float4 ti[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) ti[h][i] = *reinterpret_cast<const float4*>(info + 16 * h + 8 * i + tk);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float u[2][4];  // [half][c]: rows tk, tk, tk + 8, tk + 8; columns 2t, 2t + 1, 2t, 2t + 1
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float4 w = ti[h][c >> 1];
            float x = s[h][nt][c] * (coef[nt][c & 1] * w.x);
            if (a.softcap > 0.f) {  // coef holds scale / softcap: cap * tanh(x) = cap - 2 cap / (1 + e^2x)
              const float e2 = ex2(x * (2.f * kLog2e));
              x = a.cap_log2 - __fdividef(2.f * a.cap_log2, 1.f + e2);
            }
            const int j = __float_as_int(w.w);
            if (a.slopes) x = fmaf(slope[nt][c & 1], (float)(j - pq[nt][c & 1]), x);
            u[h][c] = x + w.y;
          }
        if (!whole) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int j = __float_as_int(ti[h][c >> 1].w), p = pq[nt][c & 1];
              if (j > p || j < low_of(p)) u[h][c] = -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float m = fmaxf(fmaxf(u[0][i], u[0][i + 2]), fmaxf(u[1][i], u[1][i + 2]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          const bool up = m > M[nt][i] + kLazy;
          if (__any_sync(0xffffffffu, up)) {
            const float mn = up ? m : M[nt][i];
            const float f = ex2(M[nt][i] - mn);
            M[nt][i] = mn;
            l[nt][i] *= f;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              o[nt][d][i] *= f;
              o[nt][d][i + 2] *= f;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            w[c] = ex2(u[h][c] - (M[nt][c & 1] - kLift));
            l[nt][c & 1] = fmaf(w[c], ti[h][c >> 1].z, l[nt][c & 1]);
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
    }
    if (v_nan) {  // a NaN scale makes its dimensions NaN for the rows that see the token, and for no other
      for (int k = 0; k < kTok; ++k) {
        if (info[k].vf[g >> 1] != 0x7fffu) continue;
        const int j = info[k].pos;
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
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t f[2];  // factors of tokens (t, t + 4) and (t + 8, t + 12) for dims 16g ..
#pragma unroll
      for (int i = 0; i < 2; ++i)
        f[i] = info[16 * h + 8 * i + t].vf[g >> 1] | ((uint32_t)info[16 * h + 8 * i + 4 + t].vf[g >> 1] << 16);
      if (v_nan) {
#pragma unroll
        for (int i = 0; i < 2; ++i) f[i] &= ~__vcmpeq2(f[i], 0x7fff7fffu);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // dims 16g .. +7, then +8 .. +15
        uint32_t ev[2][4], od[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t wa = half ? vr[h][2 * i].y : vr[h][2 * i].x;
          const uint32_t wb = half ? vr[h][2 * i + 1].y : vr[h][2 * i + 1].x;
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
    __syncwarp();  // the infos are read
    if (more) {
      load_v();
      find(n + 2 * kBlockTok);
    }
  }

  // ---- the four warps' sums merged in shared memory
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], x);
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);                       // [warp][row][kORow]
  float2* sml = reinterpret_cast<float2*>(so + kWarps * kRows * kORow);  // [warp][row]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float* row = so + (warp * kRows + nt * 8 + 2 * t + i) * kORow;
#pragma unroll
      for (int d = 0; d < 8; ++d)  // dims 16g + 2d, + 1 at 16d + 2g, + 1
        *reinterpret_cast<float2*>(row + 16 * d + 2 * g) = make_float2(o[nt][d][i], o[nt][d][i + 2]);
      if (g == 0) sml[warp * kRows + nt * 8 + 2 * t + i] = make_float2(M[nt][i], l[nt][i]);
    }
  }
  __syncthreads();
  const int d = threadIdx.x;
  const int at = ((d & 15) >> 1) * 16 + (d >> 4) * 2 + (d & 1);
  for (int r = 0; r < rows; ++r) {
    float m = kNoMax, num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sml[w * kRows + r].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sml[w * kRows + r];
      const float f = ex2(ml.x - m);
      den = fmaf(f, ml.y, den);
      num = fmaf(f, so[(w * kRows + r) * kORow + at], num);
    }
    const int64_t R = part_row(r);
    if (a.splits > 1) {
      a.part_o[(R * a.splits + split) * kKvDim + d] = num;
      if (d == 0) a.part_ml[R * a.splits + split] = make_float2(den == 0.f ? -INFINITY : m, den);
    } else {
      store1(static_cast<T*>(a.out) + R * kKvDim + d, den == 0.f ? 0.f : num / den);
    }
  }
}

// out[row] = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s: one CTA a row, a
// dimension a thread.
template <class T>
__global__ void __launch_bounds__(kKvDim) kv4_combine_kernel(const float* __restrict__ part_o,
                                                             const float2* __restrict__ part_ml, int splits,
                                                             T* __restrict__ out) {
  grid_dependency_wait();
  const int64_t R = blockIdx.x;
  const int d = threadIdx.x;
  const float2* ml = part_ml + R * splits;
  float m = -INFINITY;
  for (int s = 0; s < splits; ++s) m = fmaxf(m, __ldg(ml + s).x);
  float num = 0.f, den = 0.f;
  if (m != -INFINITY)
    for (int s = 0; s < splits; ++s) {
      const float2 x = __ldg(ml + s);
      if (x.x == -INFINITY) continue;  // nothing there: no output was written
      const float f = ex2(x.x - m);
      den = fmaf(f, x.y, den);
      num = fmaf(f, __ldg(part_o + (R * splits + s) * kKvDim + d), num);
    }
  store1(out + R * kKvDim + d, den == 0.f ? 0.f : num / den);
}

// How a call is cut: row tiles of 8 * nt query rows, and splits of `chunk` tokens.
struct AttnPlan {
  int nt, row_tiles, chunk, splits;
};

constexpr int kSms = 148;

AttnPlan plan_of(const fm_kv4_cache* c, const fm_kv4_attn_desc* d) {
  AttnPlan p;
  const int rows = d->Tq * (d->n_q_heads / c->n_kv_heads);
  p.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  p.row_tiles = (rows + 8 * p.nt - 1) / (8 * p.nt);
  int64_t tokens = d->idx ? d->max_sel : d->max_len;
  if (!d->idx && d->window > 0)  // a row tile reaches back window + Tq - 1 from the last token, from a multiple of 32
    tokens = std::min(tokens, (int64_t)d->window + d->Tq - 1 + kTok - 1);
  const int64_t units = (int64_t)c->B * c->n_kv_heads * p.row_tiles;
  const int64_t want = (tokens * units + 12 * kSms - 1) / (12 * kSms);
  const int64_t chunk = std::max<int64_t>(kBlockTok, std::min<int64_t>((want + kBlockTok - 1) / kBlockTok * kBlockTok, 4096));
  p.chunk = (int)chunk;
  p.splits = (int)((tokens + chunk - 1) / chunk);
  return p;
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
  if (!std::isfinite(d->scale) || !std::isfinite(d->softcap) || d->softcap < 0.f || d->window < 0)
    return FM_ERR_INVALID_ARG;
  return FM_OK;
}

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" size_t fm_kv4_attention_workspace_bytes(const fm_kv4_cache* c, const fm_kv4_attn_desc* d) {
  if (check_attn(c, d) != FM_OK) return 0;
  const AttnPlan p = plan_of(c, d);
  if (p.splits == 1) return 16;
  return (size_t)c->B * d->Tq * d->n_q_heads * p.splits * (kKvDim + 2) * sizeof(float);
}

namespace {

template <class T, int NT, int P, bool LIST>
fm_status launch_attn(const AttnArgs& a, dim3 grid, cudaStream_t stream) {
  constexpr int kLoop = kWarps * kTok * (int)sizeof(TokenInfo) + (NT == 1 ? 0 : NT * P * 8 * 32 * (int)sizeof(uint2));
  constexpr int kEnd = kWarps * 8 * NT * (kORow * (int)sizeof(float) + (int)sizeof(float2));
  constexpr int kSmem = kLoop > kEnd ? kLoop : kEnd;
  static PerDeviceOnce once;
  int dev = 0;
  cudaGetDevice(&dev);
  if (fm_status s = smem_limit_once(once, dev, kv4_attn_kernel<T, NT, P, LIST>, kSmem)) return s;
  kv4_attn_kernel<T, NT, P, LIST><<<grid, kThreads, kSmem, stream>>>(a);
  note_launch();
  return check_launch();
}

template <class T, bool LIST>
fm_status launch_attn_nt(const AttnArgs& a, int nt, dim3 grid, cudaStream_t stream) {
  constexpr int P = sizeof(T) == 4 ? 2 : 1;
  if (nt == 1) return launch_attn<T, 1, P, LIST>(a, grid, stream);
  if (nt == 2) return launch_attn<T, 2, P, LIST>(a, grid, stream);
  return launch_attn<T, 4, P, LIST>(a, grid, stream);
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
  const AttnPlan p = plan_of(c, d);
  const int64_t rows = (int64_t)c->B * d->Tq * d->n_q_heads;
  if ((int64_t)c->n_kv_heads * p.row_tiles > 65535) return FM_ERR_UNSUPPORTED;
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
  a.window = d->window;
  a.softcap = d->softcap;
  a.cap_log2 = d->softcap * kLog2e;
  a.coef = d->softcap > 0.f ? d->scale / d->softcap : d->scale * kLog2e;
  const int q16 = c->page_size / 16;
  a.page_magic = q16 == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + q16 - 1) / q16);
  a.row_tiles = p.row_tiles;
  a.chunk = p.chunk;
  a.splits = p.splits;
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (p.splits > 1 ? rows * p.splits * kKvDim : 0));
  const dim3 grid(p.splits, c->n_kv_heads * p.row_tiles, c->B);
  return by_dtype(d->dtype, [&](auto* tag) -> fm_status {
    using T = std::remove_pointer_t<decltype(tag)>;
    const fm_status s = d->idx ? launch_attn_nt<T, true>(a, p.nt, grid, stream)
                               : launch_attn_nt<T, false>(a, p.nt, grid, stream);
    if (s != FM_OK || p.splits == 1) return s;
    const cudaError_t e = launch_overlapped(kv4_combine_kernel<T>, dim3((unsigned)rows), dim3(kKvDim), 0, stream,
                                            (const float*)a.part_o, (const float2*)a.part_ml, p.splits,
                                            static_cast<T*>(d->out));
    if (e != cudaSuccess) return record_cuda_error(e);
    note_launch();
    return check_launch();
  });
}
