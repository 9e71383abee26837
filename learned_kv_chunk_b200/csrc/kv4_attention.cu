// kv4_attention.cu -- attention over the 4-bit paged cache (fm_kv4_attention).
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
  float scale, softcap;
};

// Codes and scales of position j of a row, or nullptr where its page is not there.
__device__ __forceinline__ const uint8_t* block_of(const Kv4View& c, const uint8_t* pool, int row, int head, int j,
                                                   int& slot) {
  const int pg = j / c.page_size;
  slot = j - pg * c.page_size;
  const int page = __ldg(c.table + row * c.table_stride + pg);
  return page < 0 || page >= c.n_pages ? nullptr : pool + page * c.page_stride + head * c.head_stride;
}

__device__ __forceinline__ float e2m1_f32(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float v = e ? __uint_as_float(((e + 126u) << 23) | (m << 22)) : 0.5f * (float)m;
  return (c & 8u) ? -v : v;
}

// One CTA a query head of a token: 128 positions at a time, a thread each for
// the scores, then a dimension each for the sum.
template <class T>
__global__ void __launch_bounds__(kKvDim) kv4_attn_simple_kernel(const AttnArgs a) {
  __shared__ float sq[kKvDim], sp[kKvDim], red[4];
  __shared__ const uint8_t* sv[kKvDim];  // the value block of a seen position, or nullptr
  __shared__ int sslot[kKvDim];
  const int t = blockIdx.x / a.n_q, h = blockIdx.x - t * a.n_q, b = blockIdx.y, d = threadIdx.x;
  const int kh = h / (a.n_q / a.c.n_heads);
  const int64_t qi = (int64_t)b * a.Tq + t;
  sq[d] = load1(static_cast<const T*>(a.q) + qi * a.q_stride + h * kKvDim + d);
  const int len = max(0, min(__ldg(a.kv_len + b), a.max_len));
  const int p = len - a.Tq + t;
  int lo = a.kv_start ? max(0, __ldg(a.kv_start + b)) : 0;
  if (a.window > 0) lo = max(lo, p - a.window + 1);
  const int n = a.idx ? max(0, min(__ldg(a.count + b), a.max_sel)) : p + 1;
  const float slope = a.slopes ? __ldg(a.slopes + h) : 0.f;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int i0 = a.idx ? 0 : (lo / kKvDim) * kKvDim; i0 < n; i0 += kKvDim) {
    const int i = i0 + d;
    int j = -1, slot = 0;
    if (i < n) j = a.idx ? __ldg(a.idx + (int64_t)b * a.max_sel + i) : i;
    const uint8_t* kb = nullptr;
    if (j >= lo && j <= p) kb = block_of(a.c, a.c.k, b, kh, j, slot);
    __syncthreads();
    float x = -INFINITY;
    if (kb) {
      float dot = 0.f;
      for (int g = 0; g < 4; ++g) {
        float part = 0.f;
        for (int c = 0; c < 16; ++c) {
          const uint32_t w = kb[slot * kKvCodeBytes + 16 * g + c];
          part = fmaf(e2m1_f32(w & 15u), sq[32 * g + 2 * c], part);
          part = fmaf(e2m1_f32(w >> 4), sq[32 * g + 2 * c + 1], part);
        }
        dot = fmaf(part, e8m0_value(kb[a.c.page_size * kKvCodeBytes + slot * kKvScaleBytes + g]), dot);
      }
      x = dot * a.scale;
      if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
      if (a.slopes) x = fmaf(slope, (float)(j - p), x);
    }
    sv[d] = kb ? a.c.v + (kb - a.c.k) : nullptr;
    sslot[d] = slot;
    float mx = x;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mx = fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    if ((d & 31) == 0) red[d >> 5] = mx;
    __syncthreads();
    const float mn = fmax_nan(m, fmax_nan(fmax_nan(red[0], red[1]), fmax_nan(red[2], red[3])));
    if (mn == -INFINITY) continue;
    const float f = exp2f((m - mn) * kLog2e);
    sp[d] = kb ? exp2f((x - mn) * kLog2e) : 0.f;
    m = mn;
    l *= f;
    o *= f;
    __syncthreads();
    for (int k = 0; k < kKvDim; ++k) {
      const uint8_t* vb = sv[k];
      if (!vb) continue;
      const uint32_t w = vb[sslot[k] * kKvCodeBytes + (d >> 1)];
      const float s = e8m0_value(vb[a.c.page_size * kKvCodeBytes + sslot[k] * kKvScaleBytes + (d >> 5)]);
      l += sp[k];
      o = fmaf(sp[k], e2m1_f32((d & 1) ? w >> 4 : w & 15u) * s, o);
    }
  }
  store1(static_cast<T*>(a.out) + (qi * a.n_q + h) * kKvDim + d, l == 0.f ? 0.f : o / l);
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
  return 16;
}

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
  a.scale = d->scale;
  a.softcap = d->softcap;
  return by_dtype(d->dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    kv4_attn_simple_kernel<T><<<dim3(d->Tq * d->n_q_heads, c->B), kKvDim, 0, stream>>>(a);
    note_launch();
    return check_launch();
  });
}
