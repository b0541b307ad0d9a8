// layer_norm.cu -- layer norm over the last axis, forward and backward.
//
//   mean, rstd = 1 / sqrt(var + eps) per row;  xhat = (x - mean) rstd
//   y  = xhat w + b
//   dx = rstd (w dy - mean_j(w dy) - xhat mean_j(w dy xhat))
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// Statistics and sums are float32: the variance is the mean of squared
// differences from the mean (no cancellation), and dw, db are summed per CTA
// over its rows and then over the CTAs in a fixed order, so they are the same
// bit for bit from run to run.
#include "operators.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr int kLnThreads = 256;

template <typename W>
__device__ __forceinline__ float param(const void* p, int j, float none) {
  return p != nullptr ? to_f32(static_cast<const W*>(p)[j]) : none;
}

template <typename T, typename W>
__global__ void __launch_bounds__(kLnThreads) ln_forward_kernel(const LayerNormArgs a) {
  __shared__ float s_warp[kLnThreads / 32];
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const T* const x = static_cast<const T*>(a.x) + t * a.x_stride;
    T* const y = static_cast<T*>(a.y) + t * a.y_stride;
    float sum = 0.0f;
    for (int j = threadIdx.x; j < a.width; j += kLnThreads) sum += to_f32(x[j]);
    const float mean = block_sum<kLnThreads>(sum, s_warp) / a.width;
    float sq = 0.0f;
    for (int j = threadIdx.x; j < a.width; j += kLnThreads) {
      const float d = to_f32(x[j]) - mean;
      sq = fmaf(d, d, sq);
    }
    const float var = block_sum<kLnThreads>(sq, s_warp) / a.width;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    for (int j = threadIdx.x; j < a.width; j += kLnThreads)
      y[j] = from_f32<T>(fmaf((to_f32(x[j]) - mean) * rstd, param<W>(a.weight, j, 1.0f),
                              param<W>(a.bias, j, 0.0f)));
    if (threadIdx.x == 0) {
      a.mean[t] = mean;
      a.rstd[t] = rstd;
    }
  }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kLnThreads) ln_backward_kernel(const LayerNormArgs a) {
  __shared__ float s_warp[kLnThreads / 32];
  float* const pw = a.partial + static_cast<int64_t>(blockIdx.x) * a.width;
  float* const pb = pw + static_cast<int64_t>(a.parts) * a.width;
  bool first = true;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const T* const x = static_cast<const T*>(a.x) + t * a.x_stride;
    const T* const dy = static_cast<const T*>(a.dy) + t * a.dy_stride;
    T* const dx = static_cast<T*>(a.dx) + t * a.dx_stride;
    const float mean = a.mean[t], rstd = a.rstd[t];
    float s1 = 0.0f, s2 = 0.0f;
    for (int j = threadIdx.x; j < a.width; j += kLnThreads) {
      const float g = to_f32(dy[j]), h = (to_f32(x[j]) - mean) * rstd;
      const float wg = g * param<W>(a.weight, j, 1.0f);
      s1 += wg;
      s2 = fmaf(wg, h, s2);
      pw[j] = first ? g * h : fmaf(g, h, pw[j]);
      pb[j] = first ? g : pb[j] + g;
    }
    first = false;
    const float m1 = block_sum<kLnThreads>(s1, s_warp) / a.width;
    const float m2 = block_sum<kLnThreads>(s2, s_warp) / a.width;
    for (int j = threadIdx.x; j < a.width; j += kLnThreads) {
      const float h = (to_f32(x[j]) - mean) * rstd;
      const float wg = to_f32(dy[j]) * param<W>(a.weight, j, 1.0f);
      dx[j] = from_f32<T>(rstd * (wg - m1 - h * m2));
    }
  }
}

// dw, db: the CTAs' column sums in CTA order.
template <typename W>
__global__ void ln_reduce_kernel(const LayerNormArgs a) {
  const int j = blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= a.width) return;
  for (int which = 0; which < 2; ++which) {
    void* const out = which == 0 ? a.dweight : a.dbias;
    if (out == nullptr) continue;
    const float* p = a.partial + static_cast<int64_t>(which) * a.parts * a.width + j;
    float t = 0.0f;
    for (int i = 0; i < a.parts; ++i) t += p[static_cast<int64_t>(i) * a.width];
    static_cast<W*>(out)[j] = from_f32<W>(t);
  }
}

template <typename T, typename W>
cudaError_t forward(const LayerNormArgs& a, int sms, cudaStream_t s) {
  const int64_t most = 8LL * sms;
  ln_forward_kernel<T, W><<<static_cast<int>(a.rows < most ? a.rows : most), kLnThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, typename W>
cudaError_t backward(LayerNormArgs a, int sms, cudaStream_t s) {
  const int64_t most = static_cast<int64_t>(kNormPartsPerSm) * sms;
  a.parts = static_cast<int32_t>(a.rows < most ? a.rows : most);
  if (a.rows > 0) ln_backward_kernel<T, W><<<a.parts, kLnThreads, 0, s>>>(a);
  if (a.dweight != nullptr || a.dbias != nullptr)
    ln_reduce_kernel<W><<<(a.width + 127) / 128, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

#define ADAMW_LN_DISPATCH(fn)                                                     \
  if (dt == ADAMW_F32 && wdt == ADAMW_F32) return fn<float, float>(a, sms, s);    \
  if (dt == ADAMW_F16 && wdt == ADAMW_F32) return fn<__half, float>(a, sms, s);   \
  if (dt == ADAMW_F16 && wdt == ADAMW_F16) return fn<__half, __half>(a, sms, s);  \
  if (dt == ADAMW_BF16 && wdt == ADAMW_F32)                                       \
    return fn<__nv_bfloat16, float>(a, sms, s);                                   \
  if (dt == ADAMW_BF16 && wdt == ADAMW_BF16)                                      \
    return fn<__nv_bfloat16, __nv_bfloat16>(a, sms, s);                           \
  return cudaErrorInvalidValue;

cudaError_t launch_layer_norm_forward(adamw_dtype dt, adamw_dtype wdt, const LayerNormArgs& a,
                                      int sms, cudaStream_t s) {
  ADAMW_LN_DISPATCH(forward)
}
cudaError_t launch_layer_norm_backward(adamw_dtype dt, adamw_dtype wdt, const LayerNormArgs& a,
                                       int sms, cudaStream_t s) {
  ADAMW_LN_DISPATCH(backward)
}
#undef ADAMW_LN_DISPATCH

}  // namespace adamw
