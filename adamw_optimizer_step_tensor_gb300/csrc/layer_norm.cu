// layer_norm.cu -- layer norm over the last axis, forward and backward.
//
//   mean, rstd = 1 / sqrt(var + eps) per row;  xhat = (x - mean) rstd
//   y  = xhat w + b
//   dx = rstd (w dy - mean_j(w dy) - xhat mean_j(w dy xhat))
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// A group of G threads holds a row in registers, 16 elements a thread, and a
// resident grid walks the rows, the next row's loads under way while a row is
// worked on.  A thread has the same columns of every row: the weight stays in
// registers, and so do the column sums of the backward pass, which are added
// over a CTA's groups, then over the CTAs by a second kernel, always in the same
// order.  Statistics and sums are float32; the variance is the mean of squared
// differences from the mean (no cancellation).  What bounds both passes is
// DRAM: two (three) accesses per element.  Rows wider than 8192 take the plain
// loops at the end of this file.
#include "operators.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr int kEach = 16;              // elements per thread
constexpr int kMaxGroup = 512;
template <int G> constexpr int kCta = G < 128 ? 128 : G;
// Resident threads per SM, by the registers a thread needs: 80 in the forward
// pass, 128 in the backward pass.
constexpr int kForwardThreads = 768;
constexpr int kBackwardThreads = 512;

template <typename W>
__device__ __forceinline__ float param(const void* p, int j, float none) {
  return p != nullptr ? to_f32(static_cast<const W*>(p)[j]) : none;
}

// 16 elements of a row as loaded: 16-byte words where every row starts on the
// 16-byte grid, else single elements; thread tid has the columns
// (i G + tid) E .. + E - 1.
template <typename T, bool VEC, int G>
struct Piece {
  static constexpr int E = VEC ? 16 / sizeof(T) : 1;
  static constexpr int N = kEach / E;
  using Raw = typename std::conditional<VEC, uint4, T>::type;
  Raw raw[N];

  static __device__ __forceinline__ int column(int i, int tid) { return (i * G + tid) * E; }
  __device__ __forceinline__ void load(const T* row, int width, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (column(i, tid) < width)
        raw[i] = __ldcs(reinterpret_cast<const Raw*>(row + column(i, tid)));
  }
  // Element i * E + e; columns past the width hold garbage.
  __device__ __forceinline__ float at(int i, int e) const {
    if constexpr (!VEC) {
      return to_f32(raw[i]);
    } else {
      const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      if constexpr (sizeof(T) == 4) return __uint_as_float(v[e]);
      else if constexpr (std::is_same<T, __half>::value)
        return __half2float(__ushort_as_half(static_cast<unsigned short>(v[e / 2] >> (e % 2 * 16))));
      else return __uint_as_float(e % 2 ? v[e / 2] & 0xFFFF0000u : v[e / 2] << 16);
    }
  }
  // Stores f(i, e) at every column below the width, rounded once.
  template <typename F>
  static __device__ __forceinline__ void store(T* row, int width, int tid, F f) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (column(i, tid) < width) {
        alignas(16) T out[E];
#pragma unroll
        for (int e = 0; e < E; ++e) out[e] = from_f32<T>(f(i, e));
        __stcs(reinterpret_cast<Raw*>(row + column(i, tid)), *reinterpret_cast<const Raw*>(out));
      }
  }
};

// Sums over a group; every thread of it gets them.  Two places in turn, so that
// one barrier per sum is enough.
template <int G>
struct GroupSum {
  float2* part;          // this group's [2][G / 32]
  int group, turn = 0;
  __device__ __forceinline__ float2 operator()(float2 x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      x.x += __shfl_xor_sync(kFull, x.x, o);
      x.y += __shfl_xor_sync(kFull, x.y, o);
    }
    if (G > 32) {
      float2* const p = part + turn * (G / 32);
      turn ^= 1;
      if ((threadIdx.x & 31) == 0) p[threadIdx.x % G / 32] = x;
      if (kCta<G> == G) __syncthreads();
      else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(G) : "memory");
      x = p[0];
#pragma unroll
      for (int i = 1; i < G / 32; ++i) {
        x.x += p[i].x;
        x.y += p[i].y;
      }
    }
    return x;
  }
};

template <typename T, typename W, bool VEC, int G>
__global__ void __launch_bounds__(kCta<G>, kForwardThreads / kCta<G>)
ln_forward_kernel(const LayerNormArgs a) {
  using P = Piece<T, VEC, G>;
  constexpr int kGroups = kCta<G> / G;
  __shared__ float2 s_part[kGroups][2 * ((G + 31) / 32)];
  const int group = threadIdx.x / G, tid = threadIdx.x % G;
  GroupSum<G> group_sum{s_part[group], group};
  float w[kEach], b[kEach];
#pragma unroll
  for (int i = 0; i < P::N; ++i)
#pragma unroll
    for (int e = 0; e < P::E; ++e) {
      const int j = P::column(i, tid) + e;
      w[i * P::E + e] = j < a.width ? param<W>(a.weight, j, 1.0f) : 0.0f;
      b[i * P::E + e] = j < a.width ? param<W>(a.bias, j, 0.0f) : 0.0f;
    }
  const float inv_width = 1.0f / static_cast<float>(a.width);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  const T* const x = static_cast<const T*>(a.x);
  P next;
  if (t < a.rows) next.load(x + t * a.x_stride, a.width, tid);
  for (; t < a.rows; t += step) {
    const P p = next;
    if (t + step < a.rows) next.load(x + (t + step) * a.x_stride, a.width, tid);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < P::N; ++i)
      if (P::column(i, tid) < a.width) {
#pragma unroll
        for (int e = 0; e < P::E; ++e) sum += p.at(i, e);
      }
    const float mean = group_sum(make_float2(sum, 0.0f)).x * inv_width;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < P::N; ++i)
      if (P::column(i, tid) < a.width) {
#pragma unroll
        for (int e = 0; e < P::E; ++e) {
          const float d = p.at(i, e) - mean;
          sq = fmaf(d, d, sq);
        }
      }
    const float rstd = 1.0f / sqrtf(group_sum(make_float2(sq, 0.0f)).x * inv_width + a.eps);
    P::store(static_cast<T*>(a.y) + t * a.y_stride, a.width, tid, [&](int i, int e) {
      return fmaf((p.at(i, e) - mean) * rstd, w[i * P::E + e], b[i * P::E + e]);
    });
    if (tid == 0) {
      a.mean[t] = mean;
      a.rstd[t] = rstd;
    }
  }
}

template <typename T, typename W, bool VEC, int G>
__global__ void __launch_bounds__(kCta<G>, kBackwardThreads / kCta<G>)
ln_backward_kernel(const LayerNormArgs a) {
  using P = Piece<T, VEC, G>;
  constexpr int kGroups = kCta<G> / G;
  __shared__ float2 s_part[kGroups][2 * ((G + 31) / 32)];
  __shared__ float2 s_add[kGroups > 1 ? kEach * G : 1];
  let_next_kernel_start();
  const int group = threadIdx.x / G, tid = threadIdx.x % G;
  GroupSum<G> group_sum{s_part[group], group};
  float w[kEach], gw[kEach], gb[kEach];
#pragma unroll
  for (int i = 0; i < P::N; ++i)
#pragma unroll
    for (int e = 0; e < P::E; ++e) {
      const int j = P::column(i, tid) + e;
      w[i * P::E + e] = j < a.width ? param<W>(a.weight, j, 1.0f) : 0.0f;
      gw[i * P::E + e] = 0.0f;
      gb[i * P::E + e] = 0.0f;
    }
  const float inv_width = 1.0f / static_cast<float>(a.width);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  const T* const x = static_cast<const T*>(a.x);
  const T* const dy = static_cast<const T*>(a.dy);
  P next_x, next_g;
  float next_mean = 0.0f, next_rstd = 0.0f;
  auto fetch = [&](int64_t r) {
    if (r >= a.rows) return;
    next_x.load(x + r * a.x_stride, a.width, tid);
    next_g.load(dy + r * a.dy_stride, a.width, tid);
    next_mean = a.mean[r];
    next_rstd = a.rstd[r];
  };
  fetch(t);
  for (; t < a.rows; t += step) {
    const P px = next_x, pg = next_g;
    const float mean = next_mean, rstd = next_rstd;
    fetch(t + step);
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < P::N; ++i)
      if (P::column(i, tid) < a.width) {
#pragma unroll
        for (int e = 0; e < P::E; ++e) {
          const int k = i * P::E + e;
          const float g = pg.at(i, e), h = (px.at(i, e) - mean) * rstd, wg = g * w[k];
          s.x += wg;
          s.y = fmaf(wg, h, s.y);
          gw[k] = fmaf(g, h, gw[k]);
          gb[k] += g;
        }
      }
    s = group_sum(s);
    const float m1 = s.x * inv_width, m2 = s.y * inv_width;
    P::store(static_cast<T*>(a.dx) + t * a.dx_stride, a.width, tid, [&](int i, int e) {
      const float h = (px.at(i, e) - mean) * rstd;
      return rstd * (fmaf(pg.at(i, e), w[i * P::E + e], -m1) - h * m2);
    });
  }
  if (a.partial == nullptr) return;
  // the CTA's groups, in their order
  for (int g = 1; g < kGroups; ++g) {
    __syncthreads();
    if (group == g) {
#pragma unroll
      for (int k = 0; k < kEach; ++k) s_add[k * G + tid] = make_float2(gw[k], gb[k]);
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        gw[k] += s_add[k * G + tid].x;
        gb[k] += s_add[k * G + tid].y;
      }
    }
  }
  if (group != 0) return;
  float* const pw = a.partial + static_cast<int64_t>(blockIdx.x) * a.width;
  float* const pb = pw + static_cast<int64_t>(a.parts) * a.width;
#pragma unroll
  for (int i = 0; i < P::N; ++i)
#pragma unroll
    for (int e = 0; e < P::E; ++e) {
      const int j = P::column(i, tid) + e;
      if (j < a.width) {
        pw[j] = gw[i * P::E + e];
        pb[j] = gb[i * P::E + e];
      }
    }
}

// dw (blockIdx.y 0) and db (1): the CTAs' column sums, 32 columns per CTA, the
// parts split over 32 rows of threads and those joined in order.
constexpr int kTile = 32;
template <typename W>
__global__ void __launch_bounds__(kTile * kTile) ln_reduce_kernel(const LayerNormArgs a) {
  __shared__ float s_sum[kTile][kTile + 1];
  wait_for_previous_kernel();
  const int col = threadIdx.x % kTile, row = threadIdx.x / kTile;
  const int j = blockIdx.x * kTile + col;
  void* const out = blockIdx.y == 0 ? a.dweight : a.dbias;
  if (out == nullptr) return;
  const float* const p = a.partial + static_cast<int64_t>(blockIdx.y) * a.parts * a.width;
  float t = 0.0f;
  if (j < a.width) {
#pragma unroll 4
    for (int i = row; i < a.parts; i += kTile) t += __ldcg(p + static_cast<int64_t>(i) * a.width + j);
  }
  s_sum[row][col] = t;
  __syncthreads();
  // a warp per column: 32 sums in a fixed tree
  t = s_sum[col][row];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
  const int jt = blockIdx.x * kTile + row;
  if (col == 0 && jt < a.width) static_cast<W*>(out)[jt] = from_f32<W>(t);
}

// ---- rows wider than the registers of a group: two passes over the row

constexpr int kWideThreads = 512;

template <typename T, typename W>
__global__ void __launch_bounds__(kWideThreads) ln_forward_wide_kernel(const LayerNormArgs a) {
  __shared__ float s_warp[kWideThreads / 32];
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const T* const x = static_cast<const T*>(a.x) + t * a.x_stride;
    T* const y = static_cast<T*>(a.y) + t * a.y_stride;
    float sum = 0.0f;
    for (int j = threadIdx.x; j < a.width; j += kWideThreads) sum += to_f32(x[j]);
    const float mean = block_sum<kWideThreads>(sum, s_warp) / a.width;
    float sq = 0.0f;
    for (int j = threadIdx.x; j < a.width; j += kWideThreads) {
      const float d = to_f32(x[j]) - mean;
      sq = fmaf(d, d, sq);
    }
    const float rstd = 1.0f / sqrtf(block_sum<kWideThreads>(sq, s_warp) / a.width + a.eps);
    for (int j = threadIdx.x; j < a.width; j += kWideThreads)
      y[j] = from_f32<T>(fmaf((to_f32(x[j]) - mean) * rstd, param<W>(a.weight, j, 1.0f),
                              param<W>(a.bias, j, 0.0f)));
    if (threadIdx.x == 0) {
      a.mean[t] = mean;
      a.rstd[t] = rstd;
    }
  }
}

// The column sums live in the CTA's own row of partial sums.
template <typename T, typename W>
__global__ void __launch_bounds__(kWideThreads) ln_backward_wide_kernel(const LayerNormArgs a) {
  __shared__ float s_warp[kWideThreads / 32];
  let_next_kernel_start();
  float* const pw = a.partial + static_cast<int64_t>(blockIdx.x) * a.width;
  float* const pb = pw + static_cast<int64_t>(a.parts) * a.width;
  bool first = true;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const T* const x = static_cast<const T*>(a.x) + t * a.x_stride;
    const T* const dy = static_cast<const T*>(a.dy) + t * a.dy_stride;
    T* const dx = static_cast<T*>(a.dx) + t * a.dx_stride;
    const float mean = a.mean[t], rstd = a.rstd[t];
    float s1 = 0.0f, s2 = 0.0f;
    for (int j = threadIdx.x; j < a.width; j += kWideThreads) {
      const float g = to_f32(dy[j]), h = (to_f32(x[j]) - mean) * rstd;
      const float wg = g * param<W>(a.weight, j, 1.0f);
      s1 += wg;
      s2 = fmaf(wg, h, s2);
      pw[j] = first ? g * h : fmaf(g, h, pw[j]);
      pb[j] = first ? g : pb[j] + g;
    }
    first = false;
    const float m1 = block_sum<kWideThreads>(s1, s_warp) / a.width;
    const float m2 = block_sum<kWideThreads>(s2, s_warp) / a.width;
    for (int j = threadIdx.x; j < a.width; j += kWideThreads) {
      const float h = (to_f32(x[j]) - mean) * rstd;
      const float wg = to_f32(dy[j]) * param<W>(a.weight, j, 1.0f);
      dx[j] = from_f32<T>(rstd * (wg - m1 - h * m2));
    }
  }
}

// ---- launches

int64_t at_most(int64_t n, int64_t most) { return n < most ? n : most; }

template <typename T, typename W, bool VEC, int G>
void forward_group(const LayerNormArgs& a, int sms, cudaStream_t s) {
  constexpr int kGroups = kCta<G> / G;
  const int64_t ctas = at_most((a.rows + kGroups - 1) / kGroups,
                               static_cast<int64_t>(kForwardThreads / kCta<G>) * sms);
  ln_forward_kernel<T, W, VEC, G><<<static_cast<int>(ctas), kCta<G>, 0, s>>>(a);
}

template <typename T, typename W, bool VEC, int G>
int backward_group(LayerNormArgs a, int sms, cudaStream_t s) {
  constexpr int kGroups = kCta<G> / G;
  constexpr int kPerSm = kBackwardThreads / kCta<G>;
  static_assert(kPerSm <= kNormPartsPerSm, "partial sums of every CTA");
  a.parts = static_cast<int32_t>(
      at_most((a.rows + kGroups - 1) / kGroups, static_cast<int64_t>(kPerSm) * sms));
  if (a.dweight == nullptr && a.dbias == nullptr) a.partial = nullptr;
  ln_backward_kernel<T, W, VEC, G><<<a.parts, kCta<G>, 0, s>>>(a);
  return a.parts;
}

// The smallest group that holds the row at 16 elements a thread.
#define ADAMW_LN_GROUPS(fn, T, W, VEC)                                  \
  (a.width <= 32 * kEach    ? fn<T, W, VEC, 32>(a, sms, s)              \
   : a.width <= 64 * kEach  ? fn<T, W, VEC, 64>(a, sms, s)              \
   : a.width <= 128 * kEach ? fn<T, W, VEC, 128>(a, sms, s)             \
   : a.width <= 256 * kEach ? fn<T, W, VEC, 256>(a, sms, s)             \
                            : fn<T, W, VEC, 512>(a, sms, s))

bool on_grid(const void* p, int64_t stride_bytes) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0;
}

template <typename T, typename W>
cudaError_t forward(const LayerNormArgs& a, int sms, cudaStream_t s) {
  const int64_t z = sizeof(T);
  if (a.width > kMaxGroup * kEach)
    ln_forward_wide_kernel<T, W>
        <<<static_cast<int>(at_most(a.rows, 4LL * sms)), kWideThreads, 0, s>>>(a);
  else if (on_grid(a.x, a.x_stride * z) && on_grid(a.y, a.y_stride * z) && a.width * z % 16 == 0)
    ADAMW_LN_GROUPS(forward_group, T, W, true);
  else
    ADAMW_LN_GROUPS(forward_group, T, W, false);
  return cudaGetLastError();
}

template <typename T, typename W>
cudaError_t backward(LayerNormArgs a, int sms, cudaStream_t s) {
  const int64_t z = sizeof(T);
  if (a.rows == 0) {
    a.parts = 0;
  } else if (a.width > kMaxGroup * kEach) {
    a.parts = static_cast<int32_t>(at_most(a.rows, static_cast<int64_t>(kNormPartsPerSm) * sms));
    ln_backward_wide_kernel<T, W><<<a.parts, kWideThreads, 0, s>>>(a);
  } else if (on_grid(a.x, a.x_stride * z) && on_grid(a.dy, a.dy_stride * z) &&
             on_grid(a.dx, a.dx_stride * z) && a.width * z % 16 == 0) {
    a.parts = ADAMW_LN_GROUPS(backward_group, T, W, true);
  } else {
    a.parts = ADAMW_LN_GROUPS(backward_group, T, W, false);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (a.dweight == nullptr && a.dbias == nullptr)) return e;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>((a.width + kTile - 1) / kTile), 2);
  c.blockDim = dim3(kTile * kTile);
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = early_start(&attr);
  return cudaLaunchKernelEx(&c, ln_reduce_kernel<W>, a);
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
#undef ADAMW_LN_GROUPS

}  // namespace adamw
