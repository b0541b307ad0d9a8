// dropout.cu -- dropout with a mask computed from a counter, and the add of the
// residual stream:  y = residual + (word >= threshold ? x scale : 0).
//
// The words are Philox4x32-10's: ten rounds of two 32 x 32 -> 64 bit products and
// two three-way exclusive ors give four words, for four elements.  The round keys
// are the same for every block and come as launch arguments.  Nothing of the mask
// goes through memory: the pass reads x (and the residual) and writes y, once.  With a residual
// DRAM bounds it (32768 x 4096 bf16: 118.7 us, the rate of a copy), without one the integer
// products of the generator nearly do (110 us, where a copy takes 79).
#include "block_ops.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr int kDropThreads = 256;
constexpr int kDropWords = 2;           // 16-byte words of each matrix on their way per thread

struct Words {
  uint32_t w[4];
};
// SHORT: fewer than 2^32 blocks.  Three of the forty products and exclusive ors are then the
// same for all of a thread's blocks.
template <bool SHORT>
__device__ __forceinline__ Words philox(uint64_t block, uint32_t step, const DropoutArgs& a) {
  uint32_t c0 = static_cast<uint32_t>(block), c1 = SHORT ? 0u : static_cast<uint32_t>(block >> 32);
  uint32_t c2 = step, c3 = a.site;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ a.key[2 * r];
    c1 = static_cast<uint32_t>(p1);
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ a.key[2 * r + 1];
    c3 = static_cast<uint32_t>(p0);
  }
  return {{c0, c1, c2, c3}};
}
__device__ __forceinline__ uint32_t step_of(const DropoutArgs& a) {
  return a.step != nullptr ? static_cast<uint32_t>(__ldg(a.step)) : 0u;
}
// A dropped x is not used: it may be NaN or infinite.  Two forms of the same value, the one
// without a selection where there is a residual to keep (32768 x 4096 bf16: 118 against 122 us;
// without a residual the other, 110 against 113).
template <bool RES>
__device__ __forceinline__ float drop(float x, float r, uint32_t word, const DropoutArgs& a) {
  const bool keep = word >= a.threshold && a.some;
  if constexpr (RES) {
    if (keep) r = fmaf(x, a.scale, r);
    return r;
  } else {
    return (keep ? x : 0.0f) * a.scale;
  }
}

// One 16-byte word of each matrix.
template <typename T, bool RES, bool SHORT>
__device__ __forceinline__ uint4 drop_word(uint4 x, uint4 r, uint64_t block, uint32_t step,
                                           const DropoutArgs& a) {
  uint32_t* xv = reinterpret_cast<uint32_t*>(&x);
  const uint32_t* rv = reinterpret_cast<const uint32_t*>(&r);
  if constexpr (std::is_same<T, float>::value) {
    const Words w = philox<SHORT>(block, step, a);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      xv[i] = __float_as_uint(drop<RES>(__uint_as_float(xv[i]), RES ? __uint_as_float(rv[i]) : 0.0f,
                                   w.w[i], a));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const Words w = philox<SHORT>(block + h, step, a);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 v = unpack_pair<T>(xv[2 * h + i]);
        const float2 q = RES ? unpack_pair<T>(rv[2 * h + i]) : make_float2(0.0f, 0.0f);
        xv[2 * h + i] = pack_pair<T>(make_float2(drop<RES>(v.x, q.x, w.w[2 * i], a),
                                                 drop<RES>(v.y, q.y, w.w[2 * i + 1], a)));
      }
    }
  }
  return x;
}

// Dense matrices on the 16-byte grid: one run of elements, by 16-byte words, then
// the last few.  a.width is the run's length.
template <typename T, bool RES, bool SHORT>
__global__ void __launch_bounds__(kDropThreads) dropout_dense_kernel(const DropoutArgs a) {
  constexpr int kPer = 16 / sizeof(T);
  const uint32_t step = step_of(a);
  const int64_t words = a.width / kPer;
  const uint4* x = static_cast<const uint4*>(a.x);
  const uint4* r = static_cast<const uint4*>(a.residual);
  uint4* y = static_cast<uint4*>(a.y);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kDropWords * kDropThreads) + threadIdx.x;
  uint4 xv[kDropWords], rv[kDropWords] = {};
#pragma unroll
  for (int u = 0; u < kDropWords; ++u) {
    const int64_t i = i0 + u * kDropThreads;
    if (i < words) {
      xv[u] = __ldcs(x + i);
      if (RES) rv[u] = __ldcs(r + i);
    }
  }
#pragma unroll
  for (int u = 0; u < kDropWords; ++u) {
    const int64_t i = i0 + u * kDropThreads;
    if (i < words)
      __stcs(y + i, drop_word<T, RES, SHORT>(xv[u], rv[u], static_cast<uint64_t>(i) * kPer / 4, step, a));
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x < a.width - words * kPer) {
    const int64_t i = words * kPer + threadIdx.x;
    const Words w = philox<SHORT>(static_cast<uint64_t>(i) / 4, step, a);
    const float q = RES ? to_f32(static_cast<const T*>(a.residual)[i]) : 0.0f;
    const uint32_t word = i % 4 == 0 ? w.w[0] : (i % 4 == 1 ? w.w[1] : (i % 4 == 2 ? w.w[2] : w.w[3]));
    static_cast<T*>(a.y)[i] = from_f32<T>(drop<RES>(to_f32(static_cast<const T*>(a.x)[i]), q, word, a));
  }
}

// Rows on the 16-byte grid, at strides: as the dense kernel, word by word of a row.  width is
// a multiple of a word's elements, so that words and blocks begin together.
template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads) dropout_rows_kernel(const DropoutArgs a) {
  constexpr int kPer = 16 / sizeof(T);
  const uint32_t step = step_of(a);
  const int64_t per_row = a.width / kPer, words = a.rows * per_row;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kDropWords * kDropThreads) + threadIdx.x;
  uint4 xv[kDropWords], rv[kDropWords] = {};
  int64_t row[kDropWords], col[kDropWords];
#pragma unroll
  for (int u = 0; u < kDropWords; ++u) {
    const int64_t i = i0 + u * kDropThreads;
    row[u] = words <= 0x7FFFFFFF ? static_cast<uint32_t>(i) / static_cast<uint32_t>(per_row) : i / per_row;
    col[u] = (i - row[u] * per_row) * kPer;
    if (i < words) {
      xv[u] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + row[u] * a.x_stride + col[u]));
      if (RES) rv[u] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(a.residual) + row[u] * a.r_stride + col[u]));
    }
  }
#pragma unroll
  for (int u = 0; u < kDropWords; ++u) {
    const int64_t i = i0 + u * kDropThreads;
    if (i < words)
      __stcs(reinterpret_cast<uint4*>(static_cast<T*>(a.y) + row[u] * a.y_stride + col[u]),
             drop_word<T, RES, false>(xv[u], rv[u], static_cast<uint64_t>(i) * kPer / 4, step, a));
  }
}

// Any strides and alignment: four elements of one block per thread, one at a time.
template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads) dropout_any_kernel(const DropoutArgs a) {
  const uint32_t step = step_of(a);
  const int64_t n = a.rows * a.width, blocks = (n + 3) / 4;
  const int64_t pace = static_cast<int64_t>(gridDim.x) * kDropThreads;
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * kDropThreads + threadIdx.x; b < blocks; b += pace) {
    const Words w = philox<false>(static_cast<uint64_t>(b), step, a);
    int64_t row = 0, col = 4 * b;
    if (a.rows > 1) {
      row = n <= 0x7FFFFFFF ? static_cast<uint32_t>(4 * b) / static_cast<uint32_t>(a.width) : 4 * b / a.width;
      col -= row * a.width;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * b + i < n) {
        const float q = RES ? to_f32(static_cast<const T*>(a.residual)[row * a.r_stride + col]) : 0.0f;
        const float v = to_f32(static_cast<const T*>(a.x)[row * a.x_stride + col]);
        static_cast<T*>(a.y)[row * a.y_stride + col] = from_f32<T>(drop<RES>(v, q, w.w[i], a));
        if (++col == a.width) {
          col = 0;
          ++row;
        }
      }
    }
  }
}

bool on_grid(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename T, bool RES>
cudaError_t drop_launch(DropoutArgs a, cudaStream_t s) {
  const bool dense = a.rows == 1 || (a.x_stride == a.width && a.y_stride == a.width &&
                                     (!RES || a.r_stride == a.width));
  const int64_t n = a.rows * a.width;
  if (dense && on_grid(a.x) && on_grid(a.y) && (!RES || on_grid(a.residual))) {
    const int64_t words = n / (16 / static_cast<int>(sizeof(T)));
    const int64_t ctas = (words + kDropWords * kDropThreads - 1) / (kDropWords * kDropThreads);
    if (ctas <= 0x7FFFFFFF) {
      a.width = n;
      const unsigned grid = static_cast<unsigned>(ctas > 0 ? ctas : 1);
      if (n <= (int64_t{1} << 34)) dropout_dense_kernel<T, RES, true><<<grid, kDropThreads, 0, s>>>(a);
      else dropout_dense_kernel<T, RES, false><<<grid, kDropThreads, 0, s>>>(a);
      return cudaGetLastError();
    }
  }
  constexpr int kPer = 16 / sizeof(T);
  if (on_grid(a.x) && on_grid(a.y) && (!RES || on_grid(a.residual)) && a.width % kPer == 0 && a.x_stride % kPer == 0 &&
      a.y_stride % kPer == 0 && (!RES || a.r_stride % kPer == 0)) {
    const int64_t words = n / kPer, ctas = (words + kDropWords * kDropThreads - 1) / (kDropWords * kDropThreads);
    if (ctas <= 0x7FFFFFFF) {
      dropout_rows_kernel<T, RES><<<static_cast<unsigned>(ctas), kDropThreads, 0, s>>>(a);
      return cudaGetLastError();
    }
  }
  if (dense) {                            // one run of elements off the grid
    a.width = n;
    a.rows = 1;
  }
  const int64_t ctas = ((n + 3) / 4 + kDropThreads - 1) / kDropThreads;
  dropout_any_kernel<T, RES><<<static_cast<unsigned>(ctas < 65536 ? ctas : 65536), kDropThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t drop_type(const DropoutArgs& a, cudaStream_t s) {
  return a.residual != nullptr ? drop_launch<T, true>(a, s) : drop_launch<T, false>(a, s);
}

}  // namespace

cudaError_t launch_dropout(adamw_dtype dt, const DropoutArgs& a, cudaStream_t s) {
  if (dt == ADAMW_F32) return drop_type<float>(a, s);
  if (dt == ADAMW_F16) return drop_type<__half>(a, s);
  return drop_type<__nv_bfloat16>(a, s);
}

}  // namespace adamw
