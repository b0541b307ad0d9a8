// grad_norm.cu -- the global gradient norm over a plan's tensors, and clipping.
//
//   norm = sqrt(sum over every element of (g / scale)^2)
//   coef = min(1, max_norm / (norm + 1e-6));  clip_scale = scale / coef
//
// clip_scale is what the step kernels take as their loss scale (they multiply
// every grad by 1 / clip_scale), so a clipped step costs one more read of the
// grads and no write of them.  Every element is read once and squared in
// float32; 64 squares in four chains join a float64 sum, and the CTAs' sums are
// added in a fixed order by the last CTA to finish, so the norm is the same bit
// for bit from run to run.
#include "operators.h"
#include "rows.cuh"
#include "step_common.cuh"

namespace adamw {
namespace {

constexpr int kLoads = 8;                           // 16-byte loads in flight per thread
constexpr float kSumMax = 3.40282347e38f;           // the largest finite float32
// A float32 sum of squares below this may have lost squares to the subnormal
// range (each loses at most 2^-150, so above it the loss is under 2^-33).
constexpr float kSumMin = 7.70371977754894341e-34f;   // 2^-110

template <typename GT> constexpr int kPerLoad = 16 / sizeof(GT);

// The elements of one 16-byte word, widened exactly to float32.
template <typename GT>
__device__ __forceinline__ void widen(const uint4& w, float (&x)[kPerLoad<GT>]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(GT) == 4) {
      x[i] = __uint_as_float(v[i]);
    } else if constexpr (std::is_same<GT, __half>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
  }
}

// Sum of squares of the words base, base + kThreads, ... of a chunk: float32
// where that is safe, float64 squares where a partial sum left the range in
// which float32 holds them (a grad above 2^63 or a batch of grads all below
// 2^-58) or is not finite.  That rare path loads the words again, so that the
// common one keeps few registers live.
template <typename GT>
__device__ __noinline__ double sum_squares_wide(const uint4* q, int base, int words) {
  double d = 0.0;
  for (int u = 0; u < kLoads; ++u) {
    const int i = base + u * kThreads;
    if (i >= words) break;
    const uint4 w = __ldcs(q + i);
    float x[kPerLoad<GT>];
    widen<GT>(w, x);
    for (int e = 0; e < kPerLoad<GT>; ++e) d = fma((double)x[e], (double)x[e], d);
  }
  return d;
}
template <typename GT>
__device__ __forceinline__ double sum_squares(const uint4* q, int base, int words) {
  uint4 w[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int i = base + u * kThreads;
    w[u] = i < words ? __ldcs(q + i) : make_uint4(0u, 0u, 0u, 0u);
  }
  float2 s[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    float x[kPerLoad<GT>];
    widen<GT>(w[u], x);
#pragma unroll
    for (int i = 0; i < kPerLoad<GT>; i += 2) {
      const float2 p = make_float2(x[i], x[i + 1]);
      s[i / 2 & 1] = fma2(p, p, s[i / 2 & 1]);
    }
  }
  const float t = (s[0].x + s[1].x) + (s[0].y + s[1].y);
  if (t >= kSumMin && t <= kSumMax) return static_cast<double>(t);
  // zeros are common (rows of an embedding that no token used)
  uint32_t any = 0u;
#pragma unroll
  for (int u = 0; u < kLoads; ++u) any |= w[u].x | w[u].y | w[u].z | w[u].w;
  if ((any & (sizeof(GT) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) == 0u) return 0.0;
  return sum_squares_wide<GT>(q, base, words);
}

// The same for grads off the 16-byte grid, kRun elements at a time.
constexpr int kRun = 16;
template <typename GT>
__device__ __noinline__ double sum_squares_single_wide(const GT* g, int base, int len) {
  double d = 0.0;
  for (int u = 0; u < kRun && base + u * kThreads < len; ++u) {
    const double x = static_cast<double>(Grad<GT>::load1(g, base + u * kThreads));
    d = fma(x, x, d);
  }
  return d;
}
template <typename GT>
__device__ __forceinline__ double sum_squares_single(const GT* g, int base, int len) {
  float x[kRun], s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < kRun; ++u)
    x[u] = base + u * kThreads < len ? Grad<GT>::load1(g, base + u * kThreads) : 0.0f;
#pragma unroll
  for (int u = 0; u < kRun; ++u) s[u & 1] = fmaf(x[u], x[u], s[u & 1]);
  const float t = s[0] + s[1];
  bool zero = true;
#pragma unroll
  for (int u = 0; u < kRun; ++u) zero &= x[u] == 0.0f;
  if (zero) return 0.0;
  if (t >= kSumMin && t <= kSumMax) return static_cast<double>(t);
  return sum_squares_single_wide<GT>(g, base, len);
}

// sqrt(x) / d rounded to float32 from a float64 x >= 0, by a float32 root of the
// mantissa (float64 roots and divisions take most of a microsecond here).
__device__ __forceinline__ float root_over(double x, float d) {
  if (!(x > 0.0) || isinf(x)) return static_cast<float>(x) / d;
  int e;
  double m = frexp(x, &e);
  if (e & 1) {
    m *= 0.5;
    ++e;
  }
  return ldexpf(sqrtf(static_cast<float>(m)) / d, e / 2);
}

template <typename GT>
__global__ void __launch_bounds__(kThreads, kNormCtasPerSm) grad_norm_kernel(const NormArgs a) {
  constexpr int kPer = kPerLoad<GT>;
  double sum = 0.0;
  // the next chunk's place in memory is looked up while a chunk is summed
  const GT* next = nullptr;
  int next_len = 0;
  auto look = [&](int64_t c) {
    if (c >= a.n_chunks) return;
    const Chunk ch = a.chunks[c];
    next = static_cast<const GT*>(a.tensors[ch.tensor].g) + ch.start;
    next_len = ch.len;
  };
  look(blockIdx.x);
  for (int64_t c = blockIdx.x; c < a.n_chunks; c += gridDim.x) {
    const GT* const g = next;
    const int len = next_len;
    look(c + gridDim.x);
    if ((reinterpret_cast<uintptr_t>(g) & 15u) == 0u) {
      const uint4* const q = reinterpret_cast<const uint4*>(g);
      const int words = len / kPer;
      for (int base = threadIdx.x; base < words; base += kThreads * kLoads)
        sum += sum_squares<GT>(q, base, words);
      const int tail = words * kPer + threadIdx.x;
      if (tail < len) {
        const double x = static_cast<double>(Grad<GT>::load1(g, tail));
        sum = fma(x, x, sum);
      }
    } else {
      for (int base = threadIdx.x; base < len; base += kThreads * kRun)
        sum += sum_squares_single<GT>(g, base, len);
    }
  }

  __shared__ double s_warp[kThreads / 32];
  __shared__ bool s_last;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = sum;
  __syncthreads();
  uint32_t* const ticket = reinterpret_cast<uint32_t*>(a.partial + gridDim.x);
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) t += s_warp[i];
    a.partial[blockIdx.x] = t;
    __threadfence();
    s_last = atomicAdd(ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last || threadIdx.x >= 32) return;
  __threadfence();
  double total = 0.0;
  for (int i = threadIdx.x; i < gridDim.x; i += 32) total += __ldcg(a.partial + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if (threadIdx.x != 0) return;
  const float scale = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
  const float norm = root_over(total, fabsf(scale));
  *a.norm = norm;
  if (a.found_inf != nullptr) *a.found_inf = isfinite(norm) ? 0.0f : 1.0f;
  if (a.clip_scale != nullptr) {
    // at most max_norm keeps the scale itself, so an unclipped step is
    // bit-identical to one without the norm; a NaN norm gives a NaN scale, an
    // infinite one an infinite scale (grads of 0)
    const float over = (norm + 1e-6f) / a.max_norm;
    *a.clip_scale = isinf(a.max_norm) || over <= 1.0f ? scale : scale * over;
  }
  atomicExch(ticket, 0u);
}

template <typename GT>
__device__ __forceinline__ GT narrow(float x) {
  if constexpr (sizeof(GT) == 4) return x;
  else if constexpr (std::is_same<GT, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// g <- g * (1 / clip_scale) in place, rounded once to the grads' type.  The
// chunks are walked from the last to the first: the norm's pass ended there,
// so the end of the list is still in L2.
template <typename GT>
__global__ void __launch_bounds__(kThreads) clip_grads_kernel(const TensorDesc* tensors,
                                                              const Chunk* chunks,
                                                              int64_t n_chunks,
                                                              const float* clip_scale) {
  const float scale = *clip_scale;
  if (scale == 1.0f) return;                 // every grad stays as it is
  const float inv = __fdiv_rn(1.0f, scale);
  constexpr int kPer = kPerLoad<GT>;
  for (int64_t c = n_chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const Chunk ch = chunks[c];
    GT* const g = const_cast<GT*>(static_cast<const GT*>(tensors[ch.tensor].g)) + ch.start;
    int done = 0;
    if ((reinterpret_cast<uintptr_t>(g) & 15u) == 0u) {
      uint4* const q = reinterpret_cast<uint4*>(g);
      const int words = ch.len / kPer;
      done = words * kPer;
      for (int base = threadIdx.x; base < words; base += kThreads * 4) {
        uint4 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (base + u * kThreads < words) w[u] = q[base + u * kThreads];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (base + u * kThreads >= words) break;
          float x[kPer];
          widen<GT>(w[u], x);
          alignas(16) GT o[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) o[i] = narrow<GT>(__fmul_rn(x[i], inv));
          __stcs(q + base + u * kThreads, *reinterpret_cast<const uint4*>(o));
        }
      }
    }
    for (int i = done + threadIdx.x; i < ch.len; i += kThreads)
      g[i] = narrow<GT>(__fmul_rn(Grad<GT>::load1(g, i), inv));
  }
}

}  // namespace

cudaError_t launch_grad_norm(adamw_dtype gdt, const NormArgs& a, int grid, cudaStream_t s) {
  switch (gdt) {
    case ADAMW_F32: grad_norm_kernel<float><<<grid, kThreads, 0, s>>>(a); break;
    case ADAMW_F16: grad_norm_kernel<__half><<<grid, kThreads, 0, s>>>(a); break;
    case ADAMW_BF16: grad_norm_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_clip_grads(adamw_dtype gdt, const TensorDesc* tensors, const Chunk* chunks,
                              int64_t n_chunks, const float* clip_scale, int grid,
                              cudaStream_t s) {
  switch (gdt) {
    case ADAMW_F32:
      clip_grads_kernel<float><<<grid, kThreads, 0, s>>>(tensors, chunks, n_chunks, clip_scale);
      break;
    case ADAMW_F16:
      clip_grads_kernel<__half><<<grid, kThreads, 0, s>>>(tensors, chunks, n_chunks, clip_scale);
      break;
    case ADAMW_BF16:
      clip_grads_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(tensors, chunks, n_chunks,
                                                                 clip_scale);
      break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace adamw
