// kv4_append.cu -- the producers of what the library's other calls read: keys
// and values appended to the 4-bit paged cache with the position rotation on
// the way (fm_kv4_append), and indexer keys as the 132-byte records that the
// scoring pass reads (fm_index_append).
//
// Mathematics.  A head of 128 dimensions belongs to 16 lanes, 8 consecutive
// dimensions each.  Rotation pairs (D - rd + j, D - rd/2 + j) lie rd/16 lanes
// apart, so a shuffle brings a lane its partners; its own cosines and sines stay
// in registers for all heads of the token.
//   * A rotated key value is x1 c - x2 s with c, s in fp32 and x of 8, 11 or 24
//     bits: each product is split into its fp32 rounding and the exact rest
//     (one fma), the two are added as a pair, and the pair is rounded once to
//     fp32 "to odd": truncated, the last bit set if anything was cut off.  A
//     number rounded to odd compares with any border of fewer bits as the
//     exact one does and rounds to any shorter type as the exact one does, so
//     codes and scales are those of the exact rotation.  Plain fp32 would move
//     one value in about ten million across a code's border, by a whole step of
//     the 4-bit type.
//   * Scale: the least power of two 2^e with max|x| <= 6 * 2^e (6 is the
//     largest e2m1 value), read from the exponent and mantissa bits of the
//     group's maximum; x * 2^-e is exact.
//
// What bounds them.  Small calls: the chain of loads (position, page, record) and
// the launch, 3.4 us for 64 tokens of 80 heads, 2.8 for 64 tokens of three indexer
// keys.  Prompts: the instructions of the rotation and the transform, issued in
// four of five cycles.  8192 tokens of 48 heads (210 MB read and written): 55 us,
// 3.8 TB/s, where a copy would take 32; 32768 tokens of three indexer keys
// (39 MB): 22 us, where a copy would take 6.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv4.cuh"

namespace fm {
namespace {

constexpr int kMaxTokens = 1 << 30;           // of a call: a CTA's token indices stay within 32 bits
constexpr int kAppThreads = 256;              // 16 heads of 16 lanes each
constexpr int kAppUnits = kAppThreads / 16;
constexpr int kAppWarps = kAppThreads / 32;

// cos and sin of the fp64 angle position * f, rounded to fp32 once, as query prep
// does.  The angle less the nearest multiple n of pi/2 (two fused steps with pi/2
// in two parts: exact to 2^-100 n), then the Taylor series of both functions to
// x^17 and x^16, whose next terms are below 2^-58 for |x| <= pi/4.  Beyond 2^40 the
// two parts of pi/2 would no longer do.
__device__ __forceinline__ float2 rope_cos_sin(int64_t position, double f) {
  const double x = (double)position * f;
  double s, c;
  if (fabs(x) < 1099511627776.0) {
    const double n = rint(x * 0.63661977236758134308);  // 2 / pi
    double r = fma(n, -1.57079632679489655800, x);
    r = fma(n, -6.12323399573676603587e-17, r);
    const double q = r * r;
    // 1 / 17!, -1 / 15!, ... and 1 / 16!, -1 / 14!, ...
    double a = 2.8114572543455206e-15, b = 4.7794773323873853e-14;
    a = fma(a, q, -7.6471637318198164e-13); b = fma(b, q, -1.1470745597729725e-11);
    a = fma(a, q, 1.6059043836821613e-10);  b = fma(b, q, 2.0876756987868099e-09);
    a = fma(a, q, -2.5052108385441720e-08); b = fma(b, q, -2.7557319223985888e-07);
    a = fma(a, q, 2.7557319223985893e-06);  b = fma(b, q, 2.4801587301587302e-05);
    a = fma(a, q, -1.9841269841269841e-04); b = fma(b, q, -1.3888888888888889e-03);
    a = fma(a, q, 8.3333333333333332e-03);  b = fma(b, q, 4.1666666666666664e-02);
    a = fma(a, q, -1.6666666666666666e-01); b = fma(b, q, -0.5);
    const double sn = fma(a * q, r, r), cn = fma(b, q, 1.0);
    const int k = (int)((long long)n & 3);
    s = (k & 1) ? cn : sn;
    c = (k & 1) ? sn : cn;
    if (k & 2) s = -s;
    if (k == 1 || k == 2) c = -c;
  } else {
    sincos(x, &s, &c);
  }
  return make_float2((float)c, (float)s);
}

// Two fp32 values at a time (packed arithmetic halves the instructions, which
// bound the appends).
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
constexpr uint64_t kMinusOnes = 0xbf800000bf800000ull;
// a - b: one rounding, of the difference.
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) { return f2_fma(b, kMinusOnes, a); }

// x c + o n as the rounded sum `hi` and what it leaves, `lo`: the products and
// their rests, added as a pair.
__device__ __forceinline__ void rot_pair(uint64_t x, uint64_t c, uint64_t o, uint64_t n, uint64_t& hi, uint64_t& lo) {
  const uint64_t p = f2_mul(x, c), q = f2_mul(o, n);
  const uint64_t pe = f2_fma(x, c, f2_mul(p, kMinusOnes)), qe = f2_fma(o, n, f2_mul(q, kMinusOnes));
  const uint64_t t = f2_add(p, q), z = f2_sub(t, p);
  const uint64_t te = f2_add(f2_sub(p, f2_sub(t, z)), f2_sub(q, z));
  const uint64_t rest = f2_add(te, f2_add(pe, qe));
  hi = f2_add(t, rest);
  lo = f2_sub(rest, f2_sub(hi, t));
}

// hi + lo rounded to odd: truncated, with the last bit set if anything was cut.
__device__ __forceinline__ float round_odd(float hi, float lo) {
  const int u = __float_as_int(hi);
  // of opposite signs: the exact value lies nearer to zero than hi
  const int odd = (u + ((u ^ __float_as_int(lo)) >> 31)) | 1;
  return fabsf(lo) > 0.f ? __int_as_float(odd) : hi;  // (an infinite or NaN hi has a NaN lo)
}

// x c + o n within 1.5 units of fp32's last place, whatever cancels: the second
// product's rounding is taken back.
__device__ __forceinline__ uint64_t rot_near(uint64_t x, uint64_t c, uint64_t o, uint64_t n) {
  const uint64_t q = f2_mul(o, n);
  return f2_add(f2_fma(x, c, q), f2_fma(o, n, f2_mul(q, kMinusOnes)));
}

// A token's cosines and sines in shared memory: 8 pairs in every 10, so that the
// lanes' 16-byte reads of 8 pairs each fall into different banks.
constexpr int cs_place(int j) { return j / 8 * 10 + j % 8; }
template <int RD>
constexpr int kCsSize = RD ? RD / 16 * 10 : 2;

// What lane l of 16 (dims 8l .. 8l+7) needs of them: a value becomes x c + other n,
// n the sine or its negative; in pairs of dims.
template <int RD>
struct Turn {
  uint64_t c[RD ? 4 : 1], n[RD ? 4 : 1];
  __device__ __forceinline__ void load(const float2* cs, int l) {
    if constexpr (RD != 0) {
      constexpr int kHalfLanes = RD / 16, kFirst = (kKvDim - RD) / 8;
      const bool in = l >= kFirst, second = l >= kFirst + kHalfLanes;
      const float4* p = reinterpret_cast<const float4*>(cs + (in ? 10 * (second ? l - kFirst - kHalfLanes : l - kFirst) : 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 w = p[i];
        c[i] = f2_pack(w.x, w.z);
        n[i] = second ? f2_pack(w.y, w.w) : f2_pack(-w.y, -w.w);
      }
    }
  }
};

// Rotates the lane's 8 values of a head.  How a value comes back: ODD rounded to
// odd (for codes: whatever rounds it again), FULL rounded to fp32, NEAR within
// 1.5 units of fp32.
enum RotMode { kRotOdd, kRotFull, kRotNear };
template <int RD, RotMode MODE>
__device__ __forceinline__ void rotate8(float (&x)[8], int l, const Turn<RD>& w) {
  if constexpr (RD != 0) {
    constexpr int kHalfLanes = RD / 16, kFirst = (kKvDim - RD) / 8;
    float other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(0xffffffffu, x[i], kHalfLanes);
    if (l < kFirst) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t a = f2_pack(x[2 * i], x[2 * i + 1]), b = f2_pack(other[2 * i], other[2 * i + 1]);
      if (MODE == kRotNear) {
        f2_unpack(rot_near(a, w.c[i], b, w.n[i]), x[2 * i], x[2 * i + 1]);
      } else {
        uint64_t hi, lo;
        rot_pair(a, w.c[i], b, w.n[i], hi, lo);
        f2_unpack(hi, x[2 * i], x[2 * i + 1]);
        if (MODE == kRotOdd) {
          float l0, l1;
          f2_unpack(lo, l0, l1);
          x[2 * i] = round_odd(x[2 * i], l0);
          x[2 * i + 1] = round_odd(x[2 * i + 1], l1);
        }
      }
    }
  }
}

// Quantises the lane's 8 values: the group's scale byte (4 lanes share one)
// and 8 codes.
__device__ __forceinline__ void quant8(const float (&x)[8], uint32_t& byte, uint32_t& codes) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmax_nan(m, fabsf(x[i]));
  m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (!(m < INFINITY)) {
    byte = 255u;
    codes = 0u;
    return;
  }
  // m = f * 2^(E - 127), 1 <= f < 2: 6 * 2^e = 1.5 * 2^(e + 2) >= m
  const uint32_t u = __float_as_uint(m);
  int e = (int)(u >> 23) - 127 - 2 + ((u & 0x7fffffu) > 0x400000u ? 1 : 0);
  e = max(-126, min(125, e));
  byte = m > 0.f ? (uint32_t)(e + 127) : 0u;
  const float r = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e: e in [-126, 125], a normal number
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(x[2 * i] * r, x[2 * i + 1] * r), __NV_E2M1, cudaRoundNearest)
         << (8 * i);
  // a zero keeps no sign
  const uint32_t nz = (w | (w >> 1) | (w >> 2)) & 0x11111111u;
  codes = w & (0x77777777u | (nz << 3));
}

// The values of 8 codes times a scale, as bf16 (exact), stored.
__device__ __forceinline__ void store_values(__nv_bfloat16* p, uint32_t codes, float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((codes >> (8 * i)) & 255u), __NV_E2M1);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

struct AppendArgs {
  Kv4View c;
  const void* x[3];          // q, k, v
  int64_t stride[3];
  const int32_t* seq;
  const int64_t* pos;
  const int64_t* positions;
  const double* inv_freq;
  int n_q, T, wpt;
  void* q_out;
  int64_t q_out_stride;
  __nv_bfloat16* hat[2];     // k, v
};

// `wpt` warps a token (8 / wpt tokens a CTA), or a CTA and a share of its heads
// where tokens are few: the token's cosines and sines once, then two heads a
// warp, of one kind, 16 lanes each.  The first heads' loads are under way while
// the angles are turned into cosines.
template <class T, int RD>
__global__ void __launch_bounds__(kAppThreads, sizeof(T) == 2 ? 4 : 3) kv4_append_kernel(const AppendArgs a) {
  __shared__ alignas(16) float2 cs[kAppWarps][kCsSize<RD>];
  const int warp = threadIdx.x >> 5, l = threadIdx.x & 15, second = (threadIdx.x >> 4) & 1;
  const int tpc = kAppWarps / a.wpt, local = warp / a.wpt, t = blockIdx.x * tpc + local;
  const bool in = t < a.T;
  const int n_kv = a.c.n_heads, kv2 = (n_kv + 1) / 2, q2 = (a.n_q + 1) / 2;
  const int items = 2 * kv2 + q2, step = gridDim.y * a.wpt;
  // an item is a pair of heads: kind 0 of keys, 1 of values, 2 of queries; a lane's eight dims of one of them
  const auto kind_of = [&](int it) { return it < kv2 ? 0 : it < 2 * kv2 ? 1 : 2; };
  const auto head_of = [&](int it, int kind) { return 2 * (it - kind * kv2) + second; };
  const T* src[3] = {static_cast<const T*>(a.x[1]) + t * a.stride[1] + 8 * l, static_cast<const T*>(a.x[2]) + t * a.stride[2] + 8 * l,
                     static_cast<const T*>(a.x[0]) + t * a.stride[0] + 8 * l};
  const auto load = [&](int it) {
    const int kind = kind_of(it), h = head_of(it, kind);
    Raw8<T> r = {};
    if (in && it < items && h < (kind == 2 ? a.n_q : n_kv))
      r = load_raw8((kind == 0 ? src[0] : kind == 1 ? src[1] : src[2]) + h * kKvDim);
    return r;
  };
  int item = blockIdx.y * a.wpt + warp - local * a.wpt;
  Raw8<T> ahead[2] = {load(item), load(item + step)};
  const int row = in ? __ldg(a.seq + t) : -1;
  const int64_t pos = in ? __ldg(a.pos + t) : -1;
  if (RD) {
    for (int i = threadIdx.x; i < tpc * (RD / 2); i += kAppThreads) {
      const int tt = blockIdx.x * tpc + i / (RD / 2), j = i % (RD / 2);
      if (tt < a.T)
        cs[i / (RD / 2)][cs_place(j)] = rope_cos_sin(__ldg((a.positions ? a.positions : a.pos) + tt), __ldg(a.inv_freq + j));
    }
  }
  int page = -1, slot = 0;
  if (row >= 0 && row < a.c.B && pos >= 0 && pos < (int64_t)a.c.max_pages * a.c.page_size) {
    const int pg = (int)pos / a.c.page_size;
    slot = (int)pos - pg * a.c.page_size;
    page = __ldg(a.c.table + row * a.c.table_stride + pg);
  }
  __syncthreads();
  if (page < 0 || page >= a.c.n_pages) return;  // padding
  Turn<RD> turn;
  turn.load(cs[local], l);
  for (; item < items; item += step) {
    float x[8];
    to_f32(ahead[0], x);
    ahead[0] = ahead[1];
    ahead[1] = load(item + 2 * step);
    const int kind = kind_of(item), h = head_of(item, kind);
    const bool on = h < (kind == 2 ? a.n_q : n_kv);
    if (kind == 2) {
      // fp32 rounds once; a 16-bit type from a value within 1.5 units of fp32
      rotate8<RD, sizeof(T) == 4 ? kRotFull : kRotNear>(x, l, turn);
      if (on) store8(static_cast<T*>(a.q_out) + t * a.q_out_stride + h * kKvDim + 8 * l, x);
      continue;
    }
    if (kind == 0) rotate8<RD, kRotOdd>(x, l, turn);
    uint32_t byte, codes;
    quant8(x, byte, codes);
    uint32_t b = byte << (8 * (l >> 2));  // the record's four scales, from lanes 0, 4, 8, 12
    b |= __shfl_xor_sync(0xffffffffu, b, 4);
    b |= __shfl_xor_sync(0xffffffffu, b, 8);
    if (!on) continue;
    uint8_t* blk = (kind == 0 ? a.c.k : a.c.v) + page * a.c.page_stride + h * a.c.head_stride;
    *reinterpret_cast<uint32_t*>(blk + slot * kKvCodeBytes + 4 * l) = codes;
    if (l == 0) *reinterpret_cast<uint32_t*>(blk + a.c.page_size * kKvCodeBytes + slot * kKvScaleBytes) = b;
    if (__nv_bfloat16* hat = kind == 0 ? a.hat[0] : a.hat[1])
      store_values(hat + ((int64_t)t * n_kv + h) * kKvDim + 8 * l, codes, e8m0_value(byte));
  }
}

struct IndexArgs {
  const void* k;
  int64_t stride;
  const int32_t* row;
  const int32_t* chunk;
  const int64_t* positions;
  const double* inv_freq;
  uint8_t* comp_k[kMaxLayers];
  int64_t row_stride;
  int T, L, B, N, hadamard, spread;
};

constexpr float kMinNormal = 1.17549435e-38f;  // 2^-126

// 16 lanes a key.  `spread` half-warps share a token's layers (all of them where
// tokens are few, otherwise one: a token's setup then serves all its layers).
template <class T, int RD>
__global__ void __launch_bounds__(kAppThreads) index_append_kernel(const IndexArgs a) {
  __shared__ alignas(16) float2 cs[kAppUnits][kCsSize<RD>];
  const int per = kAppUnits / a.spread;  // tokens a CTA
  const int w = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int tok = w / a.spread, t = blockIdx.x * per + tok;
  const bool in = tok < per && t < a.T;
  int layer = w - tok * a.spread;
  const T* src = static_cast<const T*>(a.k) + t * a.stride + 8 * l;
  Raw8<T> ahead = {};
  if (in) ahead = ldg_raw8(src + layer * kKvDim);
  const int row = in ? __ldg(a.row + t) : -1, chunk = in ? __ldg(a.chunk + t) : -1;
  const bool on = row >= 0 && row < a.B && chunk >= 0 && chunk < a.N;
  if (RD) {
    for (int i = threadIdx.x; i < per * (RD / 2); i += kAppThreads) {
      const int tt = blockIdx.x * per + i / (RD / 2), j = i % (RD / 2);
      if (tt < a.T) cs[i / (RD / 2)][cs_place(j)] = rope_cos_sin(__ldg(a.positions + tt), __ldg(a.inv_freq + j));
    }
    __syncthreads();
  }
  Turn<RD> turn;
  turn.load(cs[tok < per ? tok : 0], l);
  const int64_t at = on ? row * a.row_stride + (int64_t)chunk * kRecord : 0;
  // (a warp's two tokens go through the same number of layers)
  for (int i = 0; i < a.L; i += a.spread, layer += a.spread) {
    float x[8];
    to_f32(ahead, x);
    if (in && layer + a.spread < a.L) ahead = ldg_raw8(src + (layer + a.spread) * kKvDim);
    rotate8<RD, kRotNear>(x, l, turn);
    if (a.hadamard) {
#pragma unroll
      for (int s = 1; s < 8; s <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(i & s)) {
            const float p = x[i], q = x[i + s];
            x[i] = p + q;
            x[i + s] = p - q;
          }
#pragma unroll
      for (int s = 1; s < 16; s <<= 1) {
        const float sign = (l & s) ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)  // o + x, or o - x on the pair's second lane
          x[i] = fmaf(x[i], sign, __shfl_xor_sync(0xffffffffu, x[i], s));
      }
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmax_nan(m, fabsf(x[i]));
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
    if (!on || layer >= a.L) continue;
    // the transform's 128^-1/2 joins the scale
    float scale = m * (a.hadamard ? 0.08838834764831845f / 448.f : 1.f / 448.f);
    float inv = 448.f / m;
    if (scale < kMinNormal) scale = inv = 0.f;
    if (!(scale < INFINITY)) scale = nan_f32();
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
      c[i] = lo | (hi << 16);
    }
    // (chosen with constant indices: an index at run time would copy the array into local memory)
    uint8_t* keys = layer == 0 ? a.comp_k[0] : layer == 1 ? a.comp_k[1] : layer == 2 ? a.comp_k[2] : a.comp_k[3];
    uint32_t* rec = reinterpret_cast<uint32_t*>(keys + at);
    rec[2 * l] = c[0];
    rec[2 * l + 1] = c[1];
    if (l == 0) rec[32] = __float_as_uint(scale);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <class F>
fm_status by_rope_dim(int rd, F&& f) {
  if (rd == 0) return f(std::integral_constant<int, 0>{});
  if (rd == 64) return f(std::integral_constant<int, 64>{});
  return f(std::integral_constant<int, 128>{});
}

}  // namespace

fm_status check_kv4_cache(const fm_kv4_cache* c) {
  if (!c || !c->k_pages || !c->v_pages || !c->page_table) return FM_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->B < 1 || c->B > 65535 || c->max_pages < 1)
    return FM_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 1024 || c->page_size % 16) return FM_ERR_UNSUPPORTED;
  if ((int64_t)c->max_pages * c->page_size > ((int64_t)1 << 30)) return FM_ERR_INVALID_ARG;
  if (c->page_table_stride < c->max_pages) return FM_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || c->page_stride_bytes % 16 || c->head_stride_bytes % 16 ||
      (reinterpret_cast<uintptr_t>(c->page_table) & 3u))
    return FM_ERR_ALIGNMENT;
  const int64_t block = (int64_t)c->page_size * kKvBytes;
  const int64_t most = (int64_t)1 << 45;  // keeps every product below in range
  if (c->page_stride_bytes < block || c->head_stride_bytes < block || c->page_stride_bytes > most ||
      c->head_stride_bytes > most)
    return FM_ERR_INVALID_ARG;
  if (c->page_stride_bytes < c->n_kv_heads * c->head_stride_bytes &&
      c->head_stride_bytes / c->page_stride_bytes < c->n_pages)
    return FM_ERR_INVALID_ARG;
  return FM_OK;
}

}  // namespace fm

using namespace fm;

extern "C" fm_status fm_kv4_append(const fm_kv4_cache* c, const fm_kv4_append_desc* d, cudaStream_t stream) {
  if (fm_status s = check_kv4_cache(c)) return s;
  if (!d || !d->k || !d->v || !d->seq || !d->pos || d->T < 1 || d->T > kMaxTokens || !dtype_ok(d->dtype))
    return FM_ERR_INVALID_ARG;
  if (d->q && (!d->q_out || d->n_q_heads < 1 || d->n_q_heads > 1024)) return FM_ERR_INVALID_ARG;
  if (d->rope_dim != 0 && d->rope_dim != 64 && d->rope_dim != 128) return FM_ERR_UNSUPPORTED;
  if (d->rope_dim && !d->inv_freq) return FM_ERR_INVALID_ARG;
  const int es = dtype_size(d->dtype);
  const int64_t kv_width = (int64_t)c->n_kv_heads * kKvDim;
  if (d->k_stride < kv_width || d->v_stride < kv_width) return FM_ERR_INVALID_ARG;
  if (d->q && (d->q_stride < (int64_t)d->n_q_heads * kKvDim || d->q_out_stride < (int64_t)d->n_q_heads * kKvDim))
    return FM_ERR_INVALID_ARG;
  if (d->q == d->q_out && d->q && d->q_stride != d->q_out_stride) return FM_ERR_INVALID_ARG;
  if (!aligned16(d->k) || !aligned16(d->v) || (d->k_stride * es) % 16 || (d->v_stride * es) % 16 ||
      (d->q && (!aligned16(d->q) || !aligned16(d->q_out) || (d->q_stride * es) % 16 || (d->q_out_stride * es) % 16)) ||
      !aligned16(d->k_hat) || !aligned16(d->v_hat) || (reinterpret_cast<uintptr_t>(d->seq) & 3u) ||
      (reinterpret_cast<uintptr_t>(d->pos) & 7u) || (reinterpret_cast<uintptr_t>(d->positions) & 7u) ||
      (reinterpret_cast<uintptr_t>(d->inv_freq) & 7u))
    return FM_ERR_ALIGNMENT;
  // keys and values written to one place
  if (c->k_pages == c->v_pages || (d->k_hat && d->k_hat == d->v_hat)) return FM_ERR_INVALID_ARG;
  AppendArgs a = {};
  a.c = kv4_view(*c);
  a.x[0] = d->q; a.x[1] = d->k; a.x[2] = d->v;
  a.stride[0] = d->q_stride; a.stride[1] = d->k_stride; a.stride[2] = d->v_stride;
  a.seq = d->seq;
  a.pos = d->pos;
  a.positions = d->positions;
  a.inv_freq = d->inv_freq;
  a.n_q = d->q ? d->n_q_heads : 0;
  a.T = d->T;
  a.q_out = d->q_out;
  a.q_out_stride = d->q_out_stride;
  a.hat[0] = static_cast<__nv_bfloat16*>(d->k_hat);
  a.hat[1] = static_cast<__nv_bfloat16*>(d->v_hat);
  return by_dtype(d->dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    return by_rope_dim(d->rope_dim, [&](auto rd) {
      // Warps a token: as few as leave two CTAs an SM (a token's setup is then shared by more heads: 8192 tokens of
      // 48 heads take 68 us with eight warps each, 60 with four or two, 64 with one), eight where tokens are few, and then its
      // heads over as many CTAs as there are shares of 16, up to four CTAs an SM (64 tokens of 80 heads: 12.5 us in
      // one CTA a token, 4.3 in five).
      const int items = 2 * ((c->n_kv_heads + 1) / 2) + (a.n_q + 1) / 2;
      a.wpt = 2;
      while (a.wpt < kAppWarps && (int64_t)d->T * a.wpt < 2 * 148 * kAppWarps) a.wpt *= 2;
      const int y = a.wpt < kAppWarps ? 1 : std::max(1, std::min((items + kAppWarps - 1) / kAppWarps, 4 * 148 / d->T));
      const int tpc = kAppWarps / a.wpt;
      kv4_append_kernel<T, decltype(rd)::value><<<dim3((d->T + tpc - 1) / tpc, y), kAppThreads, 0, stream>>>(a);
      note_launch();
      return check_launch();
    });
  });
}

extern "C" fm_status fm_index_append(const void* k, int dtype, int64_t token_stride, int T, int L, const int32_t* row,
                                     const int32_t* chunk, const int64_t* positions, const double* inv_freq,
                                     int rope_dim, int hadamard, uint8_t* const* comp_k, int64_t row_stride_bytes,
                                     int B, int N, cudaStream_t stream) {
  if (!k || !row || !chunk || !comp_k || T < 1 || T > kMaxTokens || L < 1 || L > kMaxLayers || B < 1 || N < 1 || !dtype_ok(dtype))
    return FM_ERR_INVALID_ARG;
  if (rope_dim != 0 && rope_dim != 64 && rope_dim != 128) return FM_ERR_UNSUPPORTED;
  if (rope_dim && (!positions || !inv_freq)) return FM_ERR_INVALID_ARG;
  if (token_stride < (int64_t)L * kKvDim || row_stride_bytes < (int64_t)N * kRecord) return FM_ERR_INVALID_ARG;
  if (!aligned16(k) || (token_stride * dtype_size(dtype)) % 16 || row_stride_bytes % 4 ||
      (reinterpret_cast<uintptr_t>(row) & 3u) || (reinterpret_cast<uintptr_t>(chunk) & 3u) ||
      (reinterpret_cast<uintptr_t>(positions) & 7u) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u))
    return FM_ERR_ALIGNMENT;
  IndexArgs a = {};
  for (int l = 0; l < L; ++l) {
    if (!comp_k[l]) return FM_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(comp_k[l]) & 3u) return FM_ERR_ALIGNMENT;
    a.comp_k[l] = comp_k[l];
  }
  for (int l = 1; l < L; ++l)
    for (int m = 0; m < l; ++m)
      if (comp_k[l] == comp_k[m]) return FM_ERR_INVALID_ARG;  // two layers' records written to one place
  a.k = k;
  a.stride = token_stride;
  a.row = row;
  a.chunk = chunk;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.row_stride = row_stride_bytes;
  a.T = T; a.L = L; a.B = B; a.N = N;
  a.hadamard = hadamard != 0;
  // two CTAs an SM and more with a token a half-warp: 32768 tokens of three layers take 21 us (28 with a
  // half-warp a key); fewer tokens spread their layers
  a.spread = (int64_t)T >= 2 * 148 * kAppUnits ? 1 : L;
  const int per = kAppUnits / a.spread;
  const unsigned grid = (unsigned)(((int64_t)T + per - 1) / per);
  return by_dtype(dtype, [&](auto* tag) {
    using E = std::remove_pointer_t<decltype(tag)>;
    return by_rope_dim(rope_dim, [&](auto rd) {
      index_append_kernel<E, decltype(rd)::value><<<grid, kAppThreads, 0, stream>>>(a);
      note_launch();
      return check_launch();
    });
  });
}
