// expert_rows.cu -- rows of tokens to their experts and back: dispatch (each row
// read once, written top_k times), combine (top_k rows joined in float32), and the
// combine's backward pass.
#include "block_ops.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr int kRowThreads = 256;

// A piece of a row: a 16-byte word, or one element where rows lie off the 16-byte grid.
template <typename T, bool VEC>
struct Piece {
  static constexpr int kN = VEC ? 16 / sizeof(T) : 1;
  typename std::conditional<VEC, uint4, T>::type v;
  __device__ __forceinline__ void zero() {
    if constexpr (VEC) v = make_uint4(0, 0, 0, 0);
    else v = from_f32<T>(0.0f);
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) v = __ldcs(reinterpret_cast<const uint4*>(p));
    else v = *p;
  }
  __device__ __forceinline__ void load_again(const T* p) {
    if constexpr (VEC) v = __ldg(reinterpret_cast<const uint4*>(p));
    else v = *p;
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC) __stcs(reinterpret_cast<uint4*>(p), v);
    else *p = v;
  }
  __device__ __forceinline__ void open(float (&f)[kN]) const {
    if constexpr (!VEC) {
      f[0] = to_f32(v);
    } else {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          f[i] = __uint_as_float(w[i]);
        } else {
          const float2 p = unpack_pair<T>(w[i]);
          f[2 * i] = p.x;
          f[2 * i + 1] = p.y;
        }
      }
    }
  }
  __device__ __forceinline__ void close(const float (&f)[kN]) {
    if constexpr (!VEC) {
      v = from_f32<T>(f[0]);
    } else {
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
        else w[i] = pack_pair<T>(make_float2(f[2 * i], f[2 * i + 1]));
      }
    }
  }
};

__device__ __forceinline__ bool has_row(int32_t slot, int64_t n_rows) {
  return slot >= 0 && slot < n_rows;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(const ExpertRowsArgs a) {
  using P = Piece<T, VEC>;
  const int64_t pieces = a.width / P::kN, n = a.tokens * pieces;
  const int64_t pace = static_cast<int64_t>(gridDim.x) * kRowThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; i < n; i += pace) {
    const int64_t t = i / pieces, c = (i - t * pieces) * P::kN;
    P p;
    p.load(static_cast<const T*>(a.x) + t * a.x_stride + c);
    for (int j = 0; j < a.top_k; ++j) {
      const int32_t slot = __ldg(a.slots + t * a.top_k + j);
      if (has_row(slot, a.n_rows)) p.store(static_cast<T*>(a.y) + slot * a.y_stride + c);
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const ExpertRowsArgs a) {
  using P = Piece<T, VEC>;
  const int64_t pieces = a.width / P::kN, n = a.tokens * pieces;
  const int64_t pace = static_cast<int64_t>(gridDim.x) * kRowThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; i < n; i += pace) {
    const int64_t t = i / pieces, c = (i - t * pieces) * P::kN;
    float sum[P::kN] = {};
    for (int j0 = 0; j0 < a.top_k; j0 += 4) {
      P p[4];
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = 0.0f;
        p[j].zero();
        if (j0 + j < a.top_k) {
          const int32_t slot = __ldg(a.slots + t * a.top_k + j0 + j);
          if (has_row(slot, a.n_rows)) {
            w[j] = a.weights != nullptr ? __ldg(a.weights + t * a.top_k + j0 + j) : 1.0f;
            p[j].load(static_cast<const T*>(a.ys) + slot * a.ys_stride + c);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[P::kN];
        p[j].open(f);
#pragma unroll
        for (int e = 0; e < P::kN; ++e) sum[e] = fmaf(w[j], f[e], sum[e]);
      }
    }
    P out;
    out.close(sum);
    out.store(static_cast<T*>(a.y) + t * a.y_stride + c);
  }
}

// A warp per assignment; the warps of one token follow one another and find its dy in L1.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowThreads) combine_backward_kernel(const ExpertRowsArgs a) {
  using P = Piece<T, VEC>;
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32);
  const int64_t n = a.tokens * a.top_k;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5); i < n;
       i += warps) {
    const int64_t t = i / a.top_k;
    const int32_t slot = __ldg(a.slots + i);
    float dot = 0.0f;
    if (has_row(slot, a.n_rows)) {
      const float w = __ldg(a.weights + i);
      const T* dy = static_cast<const T*>(a.x) + t * a.x_stride;
      const T* ys = static_cast<const T*>(a.ys) + slot * a.ys_stride;
      T* dys = static_cast<T*>(a.y) + slot * a.y_stride;
#pragma unroll 4
      for (int64_t c = lane * P::kN; c < a.width; c += 32 * P::kN) {
        P g, y;
        g.load_again(dy + c);
        y.load(ys + c);
        float gf[P::kN], yf[P::kN];
        g.open(gf);
        y.open(yf);
#pragma unroll
        for (int e = 0; e < P::kN; ++e) {
          dot = fmaf(gf[e], yf[e], dot);
          gf[e] *= w;
        }
        g.close(gf);
        g.store(dys + c);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
    if (lane == 0) a.dweights[i] = dot;
  }
}

template <typename T>
bool rows_on_grid(const void* p, int64_t stride) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * sizeof(T) % 16 == 0;
}
template <typename T>
bool vectors(const ExpertRowsArgs& a) {
  return a.width * sizeof(T) % 16 == 0 && rows_on_grid<T>(a.x, a.x_stride) &&
         rows_on_grid<T>(a.ys, a.ys_stride) && rows_on_grid<T>(a.y, a.y_stride);
}
unsigned ctas_for(int64_t work, int sms) {
  const int64_t ctas = (work + kRowThreads - 1) / kRowThreads, most = 64LL * sms;
  return static_cast<unsigned>(ctas < most ? ctas : most);
}

#define ADAMW_ROWS_LAUNCH(kernel, work)                                                       \
  if (vectors<T>(a)) kernel<T, true><<<ctas_for(work(16 / sizeof(T)), sms), kRowThreads, 0, s>>>(a); \
  else kernel<T, false><<<ctas_for(work(1), sms), kRowThreads, 0, s>>>(a);                    \
  return cudaGetLastError();

template <typename T>
cudaError_t dispatch(const ExpertRowsArgs& a, int sms, cudaStream_t s) {
  const auto work = [&](int64_t per) { return a.tokens * (a.width / per); };
  ADAMW_ROWS_LAUNCH(dispatch_kernel, work)
}
template <typename T>
cudaError_t combine(const ExpertRowsArgs& a, int sms, cudaStream_t s) {
  const auto work = [&](int64_t per) { return a.tokens * (a.width / per); };
  ADAMW_ROWS_LAUNCH(combine_kernel, work)
}
template <typename T>
cudaError_t combine_backward(const ExpertRowsArgs& a, int sms, cudaStream_t s) {
  const auto work = [&](int64_t) { return a.tokens * a.top_k * 32; };
  ADAMW_ROWS_LAUNCH(combine_backward_kernel, work)
}
#undef ADAMW_ROWS_LAUNCH

}  // namespace

#define ADAMW_ROWS_TYPE(fn)                              \
  if (dt == ADAMW_F32) return fn<float>(a, sms, s);      \
  if (dt == ADAMW_F16) return fn<__half>(a, sms, s);     \
  return fn<__nv_bfloat16>(a, sms, s);

cudaError_t launch_dispatch(adamw_dtype dt, const ExpertRowsArgs& a, int sms, cudaStream_t s) {
  ADAMW_ROWS_TYPE(dispatch)
}
cudaError_t launch_combine(adamw_dtype dt, const ExpertRowsArgs& a, int sms, cudaStream_t s) {
  ADAMW_ROWS_TYPE(combine)
}
cudaError_t launch_combine_backward(adamw_dtype dt, const ExpertRowsArgs& a, int sms,
                                    cudaStream_t s) {
  ADAMW_ROWS_TYPE(combine_backward)
}
#undef ADAMW_ROWS_TYPE

}  // namespace adamw
