// add_rmsnorm.cu -- residual addition, RMSNorm and an e4m3 output with scales
// (fm_add_rmsnorm_fp8).
#include <cmath>

#include "kv4.cuh"

namespace fm {
namespace {

constexpr int kNormThreads = 256;
constexpr float kMinNormal = 1.17549435e-38f;  // 2^-126

struct NormArgs {
  const void* x;
  const void* residual;
  const void* gain;
  int64_t x_stride, r_stride;
  int H, group;
  float eps;
  void* sum_out;
  uint8_t* codes;
  float* scales;
};

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.f;
#pragma unroll
  for (int i = 0; i < kNormThreads / 32; ++i) r += red[i];
  return r;
}

// One CTA a row, three passes: the sum of squares, the groups' maxima, the codes.
template <class T>
__global__ void __launch_bounds__(kNormThreads) add_rmsnorm_simple_kernel(const NormArgs a) {
  __shared__ float red[kNormThreads / 32];
  const int64_t t = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
  const T* r = a.residual ? static_cast<const T*>(a.residual) + t * a.r_stride : nullptr;
  const T* gain = static_cast<const T*>(a.gain);
  const auto z_at = [&](int i) { return load1(x + i) + (r ? load1(r + i) : 0.f); };
  float ss = 0.f;
  for (int i = threadIdx.x; i < a.H; i += kNormThreads) {
    const float z = z_at(i);
    ss = fmaf(z, z, ss);
  }
  const float ms = block_sum(ss, red) / (float)a.H + a.eps;
  const float inv_rms = ms < INFINITY ? rsqrtf(ms) : nan_f32();
  const auto y_at = [&](int i) { return z_at(i) * inv_rms * (gain ? load1(gain + i) : 1.f); };
  const int lane = threadIdx.x & 31;
  float row_max = 0.f;
  if (a.group != kKvDim) {
    for (int i = threadIdx.x; i < a.H; i += kNormThreads) row_max = fmax_nan(row_max, fabsf(y_at(i)));
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) row_max = fmax_nan(row_max, __shfl_xor_sync(0xffffffffu, row_max, s));
    __syncthreads();
    if (lane == 0) red[threadIdx.x >> 5] = row_max;
    __syncthreads();
    for (int i = 0; i < kNormThreads / 32; ++i) row_max = fmax_nan(row_max, red[i]);
  }
  // a warp a group of 128: four elements a lane
  for (int g = threadIdx.x >> 5; g < a.H / kKvDim; g += kNormThreads / 32) {
    float y[4], z[4], m = row_max;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      z[k] = z_at(g * kKvDim + 4 * lane + k);
      y[k] = y_at(g * kKvDim + 4 * lane + k);
    }
    if (a.group == kKvDim) {
      m = fmax_nan(fmax_nan(fabsf(y[0]), fabsf(y[1])), fmax_nan(fabsf(y[2]), fabsf(y[3])));
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
    }
    float scale = m / 448.f;
    const float inv = scale >= kMinNormal ? 1.f / scale : 0.f;
    if (scale < kMinNormal) scale = 0.f;
    if (!(scale < INFINITY)) scale = nan_f32();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t at = t * a.H + g * kKvDim + 4 * lane + k;
      a.codes[at] = __nv_cvt_float_to_fp8(y[k] * inv, __NV_SATFINITE, __NV_E4M3);
      if (a.sum_out) store1(static_cast<T*>(a.sum_out) + at, z[k]);
    }
    if (lane == 0) {
      if (a.group == kKvDim) a.scales[t * (a.H / kKvDim) + g] = scale;
      else if (g == 0) a.scales[t] = scale;
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace fm

using namespace fm;

extern "C" fm_status fm_add_rmsnorm_fp8(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                        const void* gain, int dtype, int T, int H, float eps, int group, void* sum_out,
                                        uint8_t* codes, float* scales, cudaStream_t stream) {
  if (!x || !codes || !scales || !dtype_ok(dtype) || T < 1 || H < 1 || !(eps >= 0.f) || !std::isfinite(eps))
    return FM_ERR_INVALID_ARG;
  if (H % kKvDim || H > 65536 || (group != kKvDim && group != H)) return FM_ERR_UNSUPPORTED;
  if (x_stride < H || (residual && residual_stride < H)) return FM_ERR_INVALID_ARG;
  if (sum_out && ((sum_out == x && x_stride != H) || (sum_out == residual && residual_stride != H)))
    return FM_ERR_INVALID_ARG;
  const int es = dtype_size(dtype);
  if (!aligned16(x) || !aligned16(residual) || !aligned16(gain) || !aligned16(sum_out) || !aligned16(codes) ||
      (x_stride * es) % 16 || (residual && (residual_stride * es) % 16) || (reinterpret_cast<uintptr_t>(scales) & 3u))
    return FM_ERR_ALIGNMENT;
  NormArgs a = {x, residual, gain, x_stride, residual_stride, H, group, eps, sum_out, codes, scales};
  return by_dtype(dtype, [&](auto* tag) {
    using E = std::remove_pointer_t<decltype(tag)>;
    add_rmsnorm_simple_kernel<E><<<T, kNormThreads, 0, stream>>>(a);
    note_launch();
    return check_launch();
  });
}
