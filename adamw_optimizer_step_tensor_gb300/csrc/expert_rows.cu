// expert_rows.cu -- rows of tokens to their experts and back: dispatch (each row
// read once, written top_k times), combine (top_k rows joined in float32), and the
// combine's backward pass.
//
// A warp takes a segment of a row, kEach pieces a lane, whose loads are all on their way
// before the first is used, or several rows of fewer pieces than lanes (32768 rows of
// 128 bf16: combine 17 -> 14 us); a piece is the widest of 16 bytes, 4 bytes and one element
// that every row starts on.  All bytes move once: DRAM bounds it (rows of 8192 x 4096 bf16, eight
// experts each: 446 us, 0.98 of the copy rate, over the four moves).
#include "block_ops.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr int kRowThreads = 256;

template <typename T, int BYTES>
struct Piece {
  static constexpr int kN = BYTES / static_cast<int>(sizeof(T));
  using Word = typename std::conditional<
      BYTES == 16, uint4, typename std::conditional<BYTES == 4, uint32_t, uint16_t>::type>::type;
  Word v;
  __device__ __forceinline__ void load(const T* p) { v = __ldcs(reinterpret_cast<const Word*>(p)); }
  __device__ __forceinline__ void load_again(const T* p) { v = __ldg(reinterpret_cast<const Word*>(p)); }
  __device__ __forceinline__ void store(T* p) const { __stcs(reinterpret_cast<Word*>(p), v); }
  __device__ __forceinline__ void open(float (&f)[kN]) const {
    if constexpr (kN == 1) {
      f[0] = to_f32(*reinterpret_cast<const T*>(&v));
    } else {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
      for (int i = 0; i < BYTES / 4; ++i) {
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
    if constexpr (kN == 1) {
      *reinterpret_cast<T*>(&v) = from_f32<T>(f[0]);
    } else {
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int i = 0; i < BYTES / 4; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
        else w[i] = pack_pair<T>(make_float2(f[2 * i], f[2 * i + 1]));
      }
    }
  }
};

__device__ __forceinline__ bool has_row(int32_t slot, int64_t n_rows) {
  return slot >= 0 && slot < n_rows;
}

// What a warp's lanes take: `lanes` of them (a power of two) a segment of `each` pieces of N a
// lane; with fewer than 32 a row is one segment, and the lanes' groups take rows next to one
// another.
//
// WHOLE: lanes is 32, as a constant (known only at run time it costs rows of 1601 fp32 65 us
// instead of 47), and the choice comes by shuffles.
template <int N, bool WHOLE>
struct Segments {
  int64_t unit, units, pace;
  int32_t per_row, narrow_step, each;
  int lane, lanes, sub;
  __device__ __forceinline__ int step() const { return WHOLE ? 32 * N : narrow_step; }
  __device__ __forceinline__ Segments(int64_t rows, int64_t width, int each_, int lanes_)
      : narrow_step(lanes_ * N), each(each_), lanes(WHOLE ? 32 : lanes_) {
    lane = threadIdx.x & (lanes - 1);
    sub = WHOLE ? 0 : (threadIdx.x & 31) / lanes;
    const int step = this->step(), at_once = WHOLE ? 1 : 32 / lanes;
    per_row = static_cast<int32_t>((width + step * each - 1) / (step * each));
    units = rows * per_row;
    unit = (static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + threadIdx.x / 32) * at_once + sub;
    pace = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32) * at_once;
  }
  __device__ __forceinline__ int64_t row() const {
    return units <= 0x7FFFFFFF ? static_cast<uint32_t>(unit) / static_cast<uint32_t>(per_row) : unit / per_row;
  }
  __device__ __forceinline__ int64_t column(int64_t row) const { return (unit - row * per_row) * (step() * each) + lane * N; }
};

constexpr int kDispatchEach = 4;
template <typename T, int BYTES, bool WHOLE>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(const ExpertRowsArgs a) {
  using P = Piece<T, BYTES>;
  Segments<P::kN, WHOLE> seg(a.tokens, a.width, kDispatchEach, a.lanes);
  for (; seg.unit < seg.units; seg.unit += seg.pace) {
    const int64_t t = seg.row(), c0 = seg.column(t);
    const T* x = static_cast<const T*>(a.x) + t * a.x_stride + c0;
    int32_t mine = -1;
    if (WHOLE && seg.lane < a.top_k) mine = __ldg(a.slots + t * a.top_k + seg.lane);
    P p[kDispatchEach];
#pragma unroll
    for (int i = 0; i < kDispatchEach; ++i)
      if (c0 + i * seg.step() < a.width) p[i].load(x + i * seg.step());
    for (int j = 0; j < a.top_k; ++j) {
      const int32_t slot = WHOLE ? __shfl_sync(kFull, mine, j) : __ldg(a.slots + t * a.top_k + j);
      if (!has_row(slot, a.n_rows)) continue;
      T* y = static_cast<T*>(a.y) + slot * a.y_stride + c0;
#pragma unroll
      for (int i = 0; i < kDispatchEach; ++i)
        if (c0 + i * seg.step() < a.width) p[i].store(y + i * seg.step());
    }
  }
}

template <int BYTES>
__host__ __device__ constexpr int combine_each() { return BYTES == 16 ? 2 : 4; }
template <typename T, int BYTES, bool WHOLE>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const ExpertRowsArgs a) {
  using P = Piece<T, BYTES>;
  constexpr int kEach = combine_each<BYTES>(), kRows = 4;
  Segments<P::kN, WHOLE> seg(a.tokens, a.width, kEach, a.lanes);
  for (; seg.unit < seg.units; seg.unit += seg.pace) {
    const int64_t t = seg.row(), c0 = seg.column(t);
    int32_t mine = -1;
    float weight = 1.0f;
    if (WHOLE && seg.lane < a.top_k) {
      mine = __ldg(a.slots + t * a.top_k + seg.lane);
      if (a.weights != nullptr) weight = __ldg(a.weights + t * a.top_k + seg.lane);
    }
    float sum[kEach][P::kN] = {};
    for (int j0 = 0; j0 < a.top_k; j0 += kRows) {
      P p[kRows][kEach];
      float w[kRows];
      int32_t slot[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        slot[j] = -1;
        w[j] = 1.0f;
        if (WHOLE) {
          slot[j] = __shfl_sync(kFull, mine, (j0 + j) & 31);
          w[j] = __shfl_sync(kFull, weight, (j0 + j) & 31);
          if (j0 + j >= a.top_k) slot[j] = -1;
        } else if (j0 + j < a.top_k) {
          slot[j] = __ldg(a.slots + t * a.top_k + j0 + j);
          if (a.weights != nullptr) w[j] = __ldg(a.weights + t * a.top_k + j0 + j);
        }
      }
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (has_row(slot[j], a.n_rows)) {
          const T* y = static_cast<const T*>(a.ys) + slot[j] * a.ys_stride + c0;
#pragma unroll
          for (int i = 0; i < kEach; ++i)
            if (c0 + i * seg.step() < a.width) p[j][i].load(y + i * seg.step());
        }
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (has_row(slot[j], a.n_rows)) {
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            float f[P::kN];
            p[j][i].open(f);
#pragma unroll
            for (int e = 0; e < P::kN; ++e) sum[i][e] = fmaf(w[j], f[e], sum[i][e]);
          }
        }
    }
    T* y = static_cast<T*>(a.y) + t * a.y_stride + c0;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (c0 + i * seg.step() < a.width) {
        P out;
        out.close(sum[i]);
        out.store(y + i * seg.step());
      }
  }
}

// The lanes of an assignment take its whole row; a token's assignments follow one another and
// find its dy in L1.
template <typename T, int BYTES, bool WHOLE>
__global__ void __launch_bounds__(kRowThreads) combine_backward_kernel(const ExpertRowsArgs a) {
  using P = Piece<T, BYTES>;
  constexpr int kEach = BYTES == 16 ? 4 : 8;
  const int lanes = WHOLE ? 32 : a.lanes, lane = threadIdx.x & (lanes - 1), step = lanes * P::kN;
  const int64_t pace = static_cast<int64_t>(gridDim.x) * (kRowThreads / lanes);
  const int64_t n = a.tokens * a.top_k;      // below 2^31
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kRowThreads / lanes) + threadIdx.x / lanes;
  const int64_t warp_first = first - (threadIdx.x & 31) / lanes;
  for (int64_t at = 0; warp_first + at < n; at += pace) {
    const int64_t i = first + at;
    const int64_t t = static_cast<uint32_t>(i) / static_cast<uint32_t>(a.top_k);
    const int32_t slot = i < n ? __ldg(a.slots + i) : -1;
    float dot = 0.0f;
    if (has_row(slot, a.n_rows)) {
      const float w = __ldg(a.weights + i);
      const T* dy = static_cast<const T*>(a.x) + t * a.x_stride;
      const T* ys = static_cast<const T*>(a.ys) + slot * a.ys_stride;
      T* dys = static_cast<T*>(a.y) + slot * a.y_stride;
      for (int64_t c = lane * P::kN; c < a.width; c += kEach * step) {
        P g[kEach], y[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u)
          if (c + u * step < a.width) {
            y[u].load(ys + c + u * step);
            g[u].load_again(dy + c + u * step);
          }
#pragma unroll
        for (int u = 0; u < kEach; ++u)
          if (c + u * step < a.width) {
            float gf[P::kN], yf[P::kN];
            g[u].open(gf);
            y[u].open(yf);
#pragma unroll
            for (int e = 0; e < P::kN; ++e) {
              dot = fmaf(gf[e], yf[e], dot);
              gf[e] *= w;
            }
            g[u].close(gf);
            g[u].store(dys + c + u * step);
          }
      }
    }
    for (int o = lanes / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
    if (lane == 0 && i < n) a.dweights[i] = dot;
  }
}

// The widest piece, in bytes, on whose grid every row starts and ends.
int piece_bytes(const ExpertRowsArgs& a, int size) {
  for (int bytes : {16, 4}) {
    const auto fits = [&](const void* p, int64_t stride) {
      return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * size % bytes == 0;
    };
    if (bytes >= size && a.width * size % bytes == 0 && fits(a.x, a.x_stride) && fits(a.ys, a.ys_stride) && fits(a.y, a.y_stride))
      return bytes;
  }
  return size;
}
// CTAs whose warps take `units` segments or rows, lanes of `lanes`: all at once, up to 32 for
// each SM.
unsigned ctas_for(int64_t units, int lanes, int sms) {
  const int64_t ctas = (units * lanes + kRowThreads - 1) / kRowThreads, most = 32LL * sms;
  return static_cast<unsigned>(ctas < most ? ctas : most);
}
int lanes_for(int64_t pieces) {
  int lanes = 1;
  while (lanes < 32 && lanes < pieces) lanes *= 2;
  return lanes;
}
int64_t segments(const ExpertRowsArgs& a, int64_t columns) { return a.tokens * ((a.width + columns - 1) / columns); }

template <typename T, int BYTES>
cudaError_t dispatch(const ExpertRowsArgs& a, int sms, cudaStream_t s) {
  const int64_t units = segments(a, a.lanes * kDispatchEach * Piece<T, BYTES>::kN);
  if (a.lanes == 32) dispatch_kernel<T, BYTES, true><<<ctas_for(units, a.lanes, sms), kRowThreads, 0, s>>>(a);
  else dispatch_kernel<T, BYTES, false><<<ctas_for(units, a.lanes, sms), kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int BYTES>
cudaError_t combine(const ExpertRowsArgs& a, int sms, cudaStream_t s) {
  const int64_t units = segments(a, a.lanes * combine_each<BYTES>() * Piece<T, BYTES>::kN);
  if (a.lanes == 32) combine_kernel<T, BYTES, true><<<ctas_for(units, a.lanes, sms), kRowThreads, 0, s>>>(a);
  else combine_kernel<T, BYTES, false><<<ctas_for(units, a.lanes, sms), kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int BYTES>
cudaError_t combine_backward(const ExpertRowsArgs& a, int sms, cudaStream_t s) {
  if (a.lanes == 32) combine_backward_kernel<T, BYTES, true><<<ctas_for(a.tokens * a.top_k, a.lanes, sms), kRowThreads, 0, s>>>(a);
  else combine_backward_kernel<T, BYTES, false><<<ctas_for(a.tokens * a.top_k, a.lanes, sms), kRowThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

#define ADAMW_ROWS_TYPE(fn)                                                                                  \
  const int size = dt == ADAMW_F32 ? 4 : 2, bytes = piece_bytes(a, size);                                    \
  a.lanes = lanes_for(a.width * size / bytes);                                                               \
  if (dt == ADAMW_F32) return bytes == 16 ? fn<float, 16>(a, sms, s) : fn<float, 4>(a, sms, s);              \
  if (dt == ADAMW_F16)                                                                                       \
    return bytes == 16 ? fn<__half, 16>(a, sms, s) : bytes == 4 ? fn<__half, 4>(a, sms, s) : fn<__half, 2>(a, sms, s); \
  return bytes == 16  ? fn<__nv_bfloat16, 16>(a, sms, s)                                                     \
         : bytes == 4 ? fn<__nv_bfloat16, 4>(a, sms, s)                                                      \
                      : fn<__nv_bfloat16, 2>(a, sms, s);

cudaError_t launch_dispatch(adamw_dtype dt, ExpertRowsArgs a, int sms, cudaStream_t s) {
  ADAMW_ROWS_TYPE(dispatch)
}
cudaError_t launch_combine(adamw_dtype dt, ExpertRowsArgs a, int sms, cudaStream_t s) {
  ADAMW_ROWS_TYPE(combine)
}
cudaError_t launch_combine_backward(adamw_dtype dt, ExpertRowsArgs a, int sms, cudaStream_t s) {
  ADAMW_ROWS_TYPE(combine_backward)
}
#undef ADAMW_ROWS_TYPE

}  // namespace adamw
