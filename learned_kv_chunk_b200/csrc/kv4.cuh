// kv4.cuh -- what the kernels around the 4-bit paged cache share: the element
// types, the cache's addressing, and the formats' conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "fm_internal.cuh"

namespace fm {

constexpr int kKvDim = 128;        // head dimension
constexpr int kKvCodeBytes = 64;   // e2m1 codes of a record
constexpr int kKvScaleBytes = 4;   // e8m0 scales of a record, one for 32 dimensions
constexpr int kKvBytes = kKvCodeBytes + kKvScaleBytes;

inline int dtype_size(int dtype) { return dtype == FM_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == FM_F32 || dtype == FM_BF16 || dtype == FM_F16; }

// FM_OK when the cache's fields can be used as they are (kv4_append.cu).
fm_status check_kv4_cache(const fm_kv4_cache* c);

#if defined(__CUDACC__)

// The cache as the kernels take it.
struct Kv4View {
  uint8_t* k;
  uint8_t* v;
  int64_t page_stride, head_stride, table_stride;
  const int32_t* table;
  int n_pages, page_size, n_heads, B, max_pages;
};

inline Kv4View kv4_view(const fm_kv4_cache& c) {
  return {c.k_pages, c.v_pages, c.page_stride_bytes, c.head_stride_bytes, c.page_table_stride,
          c.page_table, c.n_pages, c.page_size, c.n_kv_heads, c.B, c.max_pages};
}

__device__ __forceinline__ float nan_f32() { return __int_as_float(0x7fffffff); }

// 2^(b - 127) for an e8m0 byte; NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return b == 255u ? nan_f32() : __uint_as_float(b ? b << 23 : 0x00400000u);
}

// Eight consecutive elements as they are (p 16-byte aligned), and as fp32.
template <class T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
// (an ordinary load: right for operands that the kernel also writes, such as queries rotated in place)
template <class T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
// The same through the read-only path: for what no thread of the kernel writes.
template <class T>
__device__ __forceinline__ Raw8<T> ldg_raw8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
__device__ __forceinline__ void to_f32(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.w[i].x);
    v[4 * i + 1] = __uint_as_float(r.w[i].y);
    v[4 * i + 2] = __uint_as_float(r.w[i].z);
    v[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
__device__ __forceinline__ void to_f32(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void to_f32(const Raw8<__half>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  to_f32(load_raw8(p), v);
}
template <class T>
__device__ __forceinline__ void ldg8(const T* p, float (&v)[8]) {
  to_f32(ldg_raw8(p), v);
}

// Eight fp32 values rounded to the type and stored (p 16-byte aligned).
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(__half* p, float v) { *p = __float2half_rn(v); }

// Calls f(pointer type tag) for the element type of `dtype`.
template <class F>
fm_status by_dtype(int dtype, F&& f) {
  if (dtype == FM_F32) return f(static_cast<float*>(nullptr));
  if (dtype == FM_BF16) return f(static_cast<__nv_bfloat16*>(nullptr));
  return f(static_cast<__half*>(nullptr));
}

#endif  // __CUDACC__

}  // namespace fm
