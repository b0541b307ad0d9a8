// rows.cuh -- device pieces shared by the row kernels (token_loss.cu,
// layer_norm.cu): element types and the fixed-order sum across a grid's CTAs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

namespace adamw {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Rounds once, to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// Two 16-bit elements in a 32-bit word, the first one low.
template <typename T>
__device__ __forceinline__ float2 unpack_pair(uint32_t v) {
  if constexpr (std::is_same<T, __half>::value)
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  else
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float2 x) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __float22half2_rn(x);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __float22bfloat162_rn(x);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Two float32 operations per instruction.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<const unsigned long long&>(x)),
        "l"(reinterpret_cast<const unsigned long long&>(y)),
        "l"(reinterpret_cast<const unsigned long long&>(z)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<const unsigned long long&>(x)),
        "l"(reinterpret_cast<const unsigned long long&>(y)));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<const unsigned long long&>(x)),
        "l"(reinterpret_cast<const unsigned long long&>(y)));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Sum over the CTA's threads, the same value in every thread.
template <int THREADS>
__device__ __forceinline__ float block_sum(float x, float* s_warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  if (THREADS == 32) return x;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = x;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) t += s_warp[i];
  return t;
}

// Kernels launched with early_start() may come up while the kernel before them
// on the stream still runs; they wait here before they touch memory.  Without
// it, wait_for_previous_kernel returns at once.
__device__ __forceinline__ void wait_for_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;");
}
inline unsigned early_start(cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  return 1;
}

// CTA `me` of `ctas` leaves four float64 sums (its thread 0's `mine`); the last
// one to arrive adds them in CTA order (the same bits whatever the order of
// arrival) and returns true with the totals in `out`, in its thread 0.  Called
// by every thread of those CTAs.
__device__ __forceinline__ bool last_cta_sums(const double (&mine)[4], double* partial,
                                              uint32_t* ticket, unsigned me, unsigned ctas,
                                              double (&out)[4]) {
  bool last = false;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) partial[4 * me + i] = mine[i];
    __threadfence();
    last = atomicAdd(ticket, 1u) == ctas - 1;
  }
  if (!__syncthreads_or(last)) return false;
  __threadfence();
  if (threadIdx.x < 32) {
    // lane 4 k + i: sum i of the CTAs k, k + 8, ... (float64 is slow here: as
    // few additions after one another as the layout allows)
    const unsigned i = threadIdx.x & 3u;
    double t = 0.0;
    for (unsigned c = threadIdx.x >> 2; c < ctas; c += 8) t += __ldcg(partial + 4 * c + i);
#pragma unroll
    for (int o = 16; o >= 4; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
#pragma unroll
    for (int m = 0; m < 4; ++m) out[m] = __shfl_sync(kFull, t, m);
    if (threadIdx.x == 0) atomicExch(ticket, 0u);
  }
  return threadIdx.x == 0;
}

}  // namespace
}  // namespace adamw
