// group_norm.cu -- group norm with an activation over channels-last tensors, forward
// and backward with the gradients of its weight and bias.
//
// A sample [positions][channels] is cut into parts of whole positions and tiles of
// 256 pieces of channels (a piece: 16 bytes, or one element off the 16-byte grid).  A
// thread keeps one piece's channels over its rows, so weights and column sums stay in
// registers.  One launch takes the statistics of every (part, tile), the next joins
// those of its sample and writes the result; it goes through the items from the last to
// the first, whose elements the L2 still holds.
//
// Statistics: a thread sums x - K and its square, K the first of its own values, and
// starts anew every kRestart rows.  K is one of the values it is subtracted from, so
// with n of them the sum of squares is at most 2 n times the spread about their mean:
// the difference loses log2(2 n) bits at worst, whatever the mean.  From there on means
// and spreads are joined by counts: M2 = sum M2_i + n_i (mean_i - mean)^2.
#include "block_ops.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr int kGnThreads = 256;
constexpr int kGnWarps = kGnThreads / 32;
constexpr int kRestart = 64;
constexpr int kGnCtasPerSm = 4;
constexpr int kItemsPerSm = 8;          // items a call is cut into, if its samples are fewer
constexpr int kUnroll = 4;              // rows on their way per thread

// How a call is cut up.
struct GnCut {
  int32_t pieces;        // of a row
  int32_t tiles;         // of a row
  int32_t tile_channels; // of a whole tile
  int32_t at_once;       // rows a CTA takes at once
  int32_t parts;         // of a sample
  int64_t part_rows;
  int64_t items;         // samples x parts
  int32_t ctas;          // per tile
};

template <typename T, bool VEC>
constexpr int piece_size() { return VEC ? 16 / static_cast<int>(sizeof(T)) : 1; }

GnCut cut_for(int32_t channels, int64_t samples, int64_t positions, int per_piece, int sms) {
  GnCut c{};
  c.pieces = channels / per_piece;
  c.tiles = (c.pieces + kGnThreads - 1) / kGnThreads;
  const int wide = c.pieces < kGnThreads ? c.pieces : kGnThreads;
  c.tile_channels = wide * per_piece;
  c.at_once = kGnThreads / wide;
  int64_t parts = 1;
  if (samples > 0) {
    const int64_t aim = static_cast<int64_t>(kItemsPerSm) * sms, have = samples * c.tiles;
    parts = have < aim ? aim / have : 1;
    const int64_t most = (positions + c.at_once - 1) / c.at_once;
    if (parts > most) parts = most;
  }
  c.part_rows = (positions + parts - 1) / parts;
  c.parts = static_cast<int32_t>((positions + c.part_rows - 1) / c.part_rows);
  c.items = samples * c.parts;
  int64_t ctas = static_cast<int64_t>(kGnCtasPerSm) * sms / c.tiles;
  if (ctas > c.items) ctas = c.items;
  c.ctas = static_cast<int32_t>(ctas > 0 ? ctas : 1);
  return c;
}

template <typename T, bool VEC>
struct GnPiece {
  static constexpr int kN = piece_size<T, VEC>();
  typename std::conditional<VEC, uint4, T>::type v;
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) v = *reinterpret_cast<const uint4*>(p);
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

__device__ __forceinline__ float warp_total(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}
// For 16-bit elements the fast exponential: off by |z| 2^-24 and 2^-22, well below their rounding.
template <typename T>
__device__ __forceinline__ float sigmoid_of(float z) {
  return __fdividef(1.0f, 1.0f + (sizeof(T) == 4 ? expf(-z) : __expf(-z)));
}

// This thread's place in its tile.
template <int N>
struct GnPlace {
  int piece, row0;       // piece of the tile (-1: none), first row
  int c0, channels;      // the tile's first channel and its channels
  int g0, g1;            // its first and last group
  int per;
  __device__ __forceinline__ GnPlace(const GroupNormArgs& a, const GnCut& c) {
    const int tile = blockIdx.y, wide = c.tile_channels / N;
    c0 = tile * c.tile_channels;
    channels = min(c.tile_channels, a.channels - c0);
    per = a.channels / a.groups;
    g0 = c0 / per;
    g1 = (c0 + channels - 1) / per;
    piece = threadIdx.x % wide;
    row0 = threadIdx.x / wide;
    if (row0 >= c.at_once || piece * N >= channels) piece = -1;
  }
  __device__ __forceinline__ int channel(int i) const { return c0 + piece * N + i; }
};

struct GnItem {
  int64_t sample, first, end;
  int part;
  __device__ __forceinline__ GnItem(int64_t i, const GroupNormArgs& a, const GnCut& c) {
    sample = i / c.parts;
    part = static_cast<int>(i - sample * c.parts);
    first = part * c.part_rows;
    end = min(first + c.part_rows, a.positions);
  }
};

// Partial statistics of an item: group g of tile t at g + t (a tile that starts inside a
// group adds one, so the places are distinct).
__device__ __forceinline__ float2* item_stats(const GroupNormArgs& a, const GnCut& c, int64_t item) {
  return reinterpret_cast<float2*>(a.stats) + item * (a.groups + c.tiles);
}

// Rows of the thread row0 of an item.
__device__ __forceinline__ int64_t rows_of(const GnItem& it, int row0, int at_once) {
  const int64_t n = it.end - it.first - row0;
  return n > 0 ? (n + at_once - 1) / at_once : 0;
}

// ---------------------------------------------------------------- forward

template <typename T, bool VEC>
__global__ void __launch_bounds__(kGnThreads) gn_stats_kernel(const GroupNormArgs a, const GnCut c) {
  using P = GnPiece<T, VEC>;
  constexpr int N = P::kN;
  __shared__ float s_mean[kGnThreads * N], s_m2[kGnThreads * N];
  const GnPlace<N> at(a, c);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  for (int64_t item = blockIdx.x; item < c.items; item += gridDim.x) {
    const GnItem it(item, a, c);
    float mean[N] = {}, m2[N] = {};
    if (at.piece >= 0) {
      const T* x = static_cast<const T*>(a.x) + it.sample * a.x_sample + at.channel(0);
      float shift[N], sum[N], squares[N];
      int64_t done = 0, n = 0;
      const int64_t rows = rows_of(it, at.row0, c.at_once);
      for (int64_t i = 0; i < rows; i += kUnroll) {
        P p[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (i + u < rows) p[u].load(x + (it.first + at.row0 + (i + u) * c.at_once) * a.x_position);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (i + u >= rows) break;
          float f[N];
          p[u].open(f);
          if (n == 0) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
              shift[e] = f[e];
              sum[e] = squares[e] = 0.0f;
            }
          } else {
#pragma unroll
            for (int e = 0; e < N; ++e) {
              const float d = f[e] - shift[e];
              sum[e] += d;
              squares[e] = fmaf(d, d, squares[e]);
            }
          }
          if (++n == kRestart || i + u == rows - 1) {
            // joins this run's n values to the `done` before them
            const float fn = static_cast<float>(n), share = fn / static_cast<float>(done + n);
            const float inv = 1.0f / fn;
#pragma unroll
            for (int e = 0; e < N; ++e) {
              const float off = sum[e] * inv, here = shift[e] + off;
              const float spread = fmaxf(fmaf(-off, sum[e], squares[e]), 0.0f);
              const float d = here - mean[e];
              mean[e] = done == 0 ? here : fmaf(d, share, mean[e]);
              m2[e] += done == 0 ? spread : fmaf(d * d, static_cast<float>(done) * share, spread);
            }
            done += n;
            n = 0;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        s_mean[at.row0 * c.tile_channels + at.piece * N + e] = mean[e];
        s_m2[at.row0 * c.tile_channels + at.piece * N + e] = m2[e];
      }
    }
    __syncthreads();
    // per group, over its channels here and the CTA's rows of threads
    for (int g = at.g0 + warp; g <= at.g1; g += kGnWarps) {
      const int lo = max(g * at.per, at.c0) - at.c0;
      const int n_ch = min((g + 1) * at.per, at.c0 + at.channels) - at.c0 - lo;
      const int64_t len = it.end - it.first;
      const float inv = 1.0f / (static_cast<float>(len) * static_cast<float>(n_ch));
      float t = 0.0f;
      for (int r = 0; r < c.at_once; ++r) {
        const float n = static_cast<float>(rows_of(it, r, c.at_once));
        if (n == 0.0f) break;
        for (int k = lane; k < n_ch; k += 32) t = fmaf(n, s_mean[r * c.tile_channels + lo + k] - s_mean[lo], t);
      }
      const float m = s_mean[lo] + warp_total(t) * inv;
      float q = 0.0f;
      for (int r = 0; r < c.at_once; ++r) {
        const float n = static_cast<float>(rows_of(it, r, c.at_once));
        if (n == 0.0f) break;
        for (int k = lane; k < n_ch; k += 32) {
          const float d = s_mean[r * c.tile_channels + lo + k] - m;
          q += fmaf(n * d, d, s_m2[r * c.tile_channels + lo + k]);
        }
      }
      q = warp_total(q);
      if (lane == 0) item_stats(a, c, item)[g + blockIdx.y] = make_float2(m, q);
    }
    __syncthreads();
  }
  let_next_kernel_start();
}

// Group g's mean and spread over the sample, by a warp.
__device__ __forceinline__ float2 join_stats(const GroupNormArgs& a, const GnCut& c, int64_t sample, int g,
                                             int per) {
  const int lane = threadIdx.x & 31;
  const int t0 = g * per / c.tile_channels, t1 = ((g + 1) * per - 1) / c.tile_channels;
  const int n = c.parts * (t1 - t0 + 1);
  const float2* base = item_stats(a, c, sample * c.parts);
  const int64_t pitch = a.groups + c.tiles;
  const float all = static_cast<float>(a.positions) * static_cast<float>(per);
  const float first = __ldcg(base + g + t0).x;
  float t = 0.0f, q = 0.0f, m = 0.0f;
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    for (int i = lane; i < n; i += 32) {
      const int part = i / (t1 - t0 + 1), tile = t0 + i - part * (t1 - t0 + 1);
      const int64_t len = min(c.part_rows, a.positions - part * c.part_rows);
      const int ch = min((g + 1) * per, (tile + 1) * c.tile_channels) - max(g * per, tile * c.tile_channels);
      const float2 s = __ldcg(base + part * pitch + g + tile);
      const float w = static_cast<float>(len) * static_cast<float>(ch);
      if (pass == 0) {
        t = fmaf(w, s.x - first, t);
      } else {
        const float d = s.x - m;
        q += fmaf(w * d, d, s.y);
      }
    }
    if (pass == 0) m = first + warp_total(t) / all;
  }
  return make_float2(m, __frcp_rn(__fsqrt_rn(warp_total(q) / all + a.eps)));
}

template <typename W, int N>
__device__ __forceinline__ void load_weights(const GroupNormArgs& a, const GnPlace<N>& at, float (&w)[N],
                                             float (&b)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    w[e] = 1.0f;
    b[e] = 0.0f;
    if (at.piece >= 0) {
      if (a.weight != nullptr) w[e] = to_f32(static_cast<const W*>(a.weight)[at.channel(e)]);
      if (a.bias != nullptr) b[e] = to_f32(static_cast<const W*>(a.bias)[at.channel(e)]);
    }
  }
}

template <typename T, typename W, bool VEC, bool SILU>
__global__ void __launch_bounds__(kGnThreads) gn_apply_kernel(const GroupNormArgs a, const GnCut c) {
  using P = GnPiece<T, VEC>;
  constexpr int N = P::kN;
  __shared__ float2 s_stat[kGnThreads * N + 1];
  const GnPlace<N> at(a, c);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  float w[N], b[N];
  load_weights<W, N>(a, at, w, b);
  wait_for_previous_kernel();
  for (int64_t i = blockIdx.x; i < c.items; i += gridDim.x) {
    const int64_t item = c.items - 1 - i;
    const GnItem it(item, a, c);
    for (int g = at.g0 + warp; g <= at.g1; g += kGnWarps) {
      const float2 s = join_stats(a, c, it.sample, g, at.per);
      if (lane == 0) {
        s_stat[g - at.g0] = s;
        if (it.part == 0 && g * at.per >= at.c0) {
          a.mean[it.sample * a.groups + g] = s.x;
          a.rstd[it.sample * a.groups + g] = s.y;
        }
      }
    }
    __syncthreads();
    if (at.piece >= 0) {
      float mean[N], slope[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float2 s = s_stat[at.channel(e) / at.per - at.g0];
        mean[e] = s.x;
        slope[e] = s.y * w[e];
      }
      const T* x = static_cast<const T*>(a.x) + it.sample * a.x_sample + at.channel(0);
      T* y = static_cast<T*>(a.out) + it.sample * a.out_sample + at.channel(0);
      const int64_t rows = rows_of(it, at.row0, c.at_once);
      for (int64_t k = 0; k < rows; k += kUnroll) {
        P p[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (k + u < rows) p[u].load(x + (it.first + at.row0 + (k + u) * c.at_once) * a.x_position);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (k + u >= rows) break;
          float f[N];
          p[u].open(f);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float z = fmaf(f[e] - mean[e], slope[e], b[e]);
            f[e] = SILU ? z * sigmoid_of<T>(z) : z;
          }
          p[u].close(f);
          p[u].store(y + (it.first + at.row0 + (k + u) * c.at_once) * a.out_position);
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- backward

// dz of one element, and its xhat.
template <typename T, bool SILU>
__device__ __forceinline__ float slope_at(float dy, float xhat, float w, float b) {
  if (!SILU) return dy;
  const float z = fmaf(xhat, w, b);
  const float s = sigmoid_of<T>(z);
  return dy * (s * fmaf(z, 1.0f - s, 1.0f));
}

template <int N>
__device__ __forceinline__ void load_stats(const GroupNormArgs& a, const GnPlace<N>& at, int64_t sample,
                                           float (&mean)[N], float (&rstd)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int64_t g = sample * a.groups + at.channel(e) / at.per;
    mean[e] = __ldg(a.mean + g);
    rstd[e] = __ldg(a.rstd + g);
  }
}

// Per item and group the sums of w dz and w dz xhat; per CTA the columns' sums of dz xhat
// and dz.
template <typename T, typename W, bool VEC, bool SILU>
__global__ void __launch_bounds__(kGnThreads) gn_sums_kernel(const GroupNormArgs a, const GnCut c) {
  using P = GnPiece<T, VEC>;
  constexpr int N = P::kN;
  __shared__ float s_one[kGnThreads * N], s_two[kGnThreads * N];
  const GnPlace<N> at(a, c);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  float w[N], b[N], all_w[N] = {}, all_b[N] = {};
  load_weights<W, N>(a, at, w, b);
  for (int64_t item = blockIdx.x; item < c.items; item += gridDim.x) {
    const GnItem it(item, a, c);
    if (at.piece >= 0) {
      float mean[N], rstd[N], one[N] = {}, two[N] = {};
      load_stats<N>(a, at, it.sample, mean, rstd);
      const T* x = static_cast<const T*>(a.x) + it.sample * a.x_sample + at.channel(0);
      const T* dy = static_cast<const T*>(a.dy) + it.sample * a.dy_sample + at.channel(0);
      const int64_t rows = rows_of(it, at.row0, c.at_once);
      for (int64_t k = 0; k < rows; k += kUnroll) {
        P p[kUnroll], q[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (k + u < rows) {
            const int64_t l = it.first + at.row0 + (k + u) * c.at_once;
            p[u].load(x + l * a.x_position);
            q[u].load(dy + l * a.dy_position);
          }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (k + u >= rows) break;
          float f[N], g[N];
          p[u].open(f);
          q[u].open(g);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float xhat = (f[e] - mean[e]) * rstd[e];
            const float dz = slope_at<T, SILU>(g[e], xhat, w[e], b[e]);
            one[e] += dz;
            two[e] = fmaf(dz, xhat, two[e]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        all_b[e] += one[e];
        all_w[e] += two[e];
        s_one[at.row0 * c.tile_channels + at.piece * N + e] = one[e] * w[e];
        s_two[at.row0 * c.tile_channels + at.piece * N + e] = two[e] * w[e];
      }
    }
    __syncthreads();
    for (int g = at.g0 + warp; g <= at.g1; g += kGnWarps) {
      const int lo = max(g * at.per, at.c0) - at.c0;
      const int hi = min((g + 1) * at.per, at.c0 + at.channels) - at.c0;
      float one = 0.0f, two = 0.0f;
      for (int r = 0; r < c.at_once; ++r)
        for (int k = lo + lane; k < hi; k += 32) {
          one += s_one[r * c.tile_channels + k];
          two += s_two[r * c.tile_channels + k];
        }
      one = warp_total(one);
      two = warp_total(two);
      if (lane == 0) item_stats(a, c, item)[g + blockIdx.y] = make_float2(one, two);
    }
    __syncthreads();
  }
  let_next_kernel_start();
  if (a.dweight == nullptr && a.dbias == nullptr) return;
  if (at.piece >= 0) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      s_one[at.row0 * c.tile_channels + at.piece * N + e] = all_w[e];
      s_two[at.row0 * c.tile_channels + at.piece * N + e] = all_b[e];
    }
  }
  __syncthreads();
  float* out_w = a.columns + static_cast<int64_t>(blockIdx.x) * a.channels + at.c0;
  float* out_b = out_w + static_cast<int64_t>(gridDim.x) * a.channels;
  for (int k = threadIdx.x; k < at.channels; k += kGnThreads) {
    float one = 0.0f, two = 0.0f;
    for (int r = 0; r < c.at_once; ++r) {
      one += s_one[r * c.tile_channels + k];
      two += s_two[r * c.tile_channels + k];
    }
    out_w[k] = one;
    out_b[k] = two;
  }
}

template <typename T, typename W, bool VEC, bool SILU>
__global__ void __launch_bounds__(kGnThreads) gn_grad_kernel(const GroupNormArgs a, const GnCut c) {
  using P = GnPiece<T, VEC>;
  constexpr int N = P::kN;
  __shared__ float2 s_sum[kGnThreads * N + 1];
  const GnPlace<N> at(a, c);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  float w[N], b[N];
  load_weights<W, N>(a, at, w, b);
  wait_for_previous_kernel();
  const float inv = 1.0f / (static_cast<float>(a.positions) * static_cast<float>(at.per));
  for (int64_t i = blockIdx.x; i < c.items; i += gridDim.x) {
    const int64_t item = c.items - 1 - i;
    const GnItem it(item, a, c);
    for (int g = at.g0 + warp; g <= at.g1; g += kGnWarps) {
      const int t0 = g * at.per / c.tile_channels, t1 = ((g + 1) * at.per - 1) / c.tile_channels;
      const int n = c.parts * (t1 - t0 + 1);
      const float2* base = item_stats(a, c, it.sample * c.parts);
      float one = 0.0f, two = 0.0f;
      for (int k = lane; k < n; k += 32) {
        const int part = k / (t1 - t0 + 1), tile = t0 + k - part * (t1 - t0 + 1);
        const float2 s = __ldcg(base + static_cast<int64_t>(part) * (a.groups + c.tiles) + g + tile);
        one += s.x;
        two += s.y;
      }
      one = warp_total(one) * inv;
      two = warp_total(two) * inv;
      if (lane == 0) s_sum[g - at.g0] = make_float2(one, two);
    }
    __syncthreads();
    if (at.piece >= 0) {
      float mean[N], rstd[N];
      load_stats<N>(a, at, it.sample, mean, rstd);
      const T* x = static_cast<const T*>(a.x) + it.sample * a.x_sample + at.channel(0);
      const T* dy = static_cast<const T*>(a.dy) + it.sample * a.dy_sample + at.channel(0);
      T* dx = static_cast<T*>(a.out) + it.sample * a.out_sample + at.channel(0);
      const int64_t rows = rows_of(it, at.row0, c.at_once);
      for (int64_t k = 0; k < rows; k += 2) {
        P p[2], q[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (k + u < rows) {
            const int64_t l = it.first + at.row0 + (k + u) * c.at_once;
            p[u].load(x + l * a.x_position);
            q[u].load(dy + l * a.dy_position);
          }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (k + u >= rows) break;
          float f[N], g[N];
          p[u].open(f);
          q[u].open(g);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float2 s = s_sum[at.channel(e) / at.per - at.g0];
            const float xhat = (f[e] - mean[e]) * rstd[e];
            const float dz = slope_at<T, SILU>(g[e], xhat, w[e], b[e]);
            f[e] = rstd[e] * (fmaf(dz, w[e], -s.x) - xhat * s.y);
          }
          p[u].close(f);
          p[u].store(dx + (it.first + at.row0 + (k + u) * c.at_once) * a.out_position);
        }
      }
    }
    __syncthreads();
  }
}

// Sums the CTAs' column sums, in their order: blockIdx.y 0 the weight's, 1 the bias's.
template <typename W>
__global__ void __launch_bounds__(1024) gn_columns_kernel(const GroupNormArgs a, const int rows) {
  __shared__ float s_sum[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x % 32, r0 = threadIdx.x / 32;
  W* out = static_cast<W*>(blockIdx.y == 0 ? a.dweight : a.dbias);
  wait_for_previous_kernel();
  float t = 0.0f;
  if (col < a.channels)
    for (int r = r0; r < rows; r += 32)
      t += __ldcg(a.columns + (static_cast<int64_t>(blockIdx.y) * rows + r) * a.channels + col);
  s_sum[r0][threadIdx.x % 32] = t;
  __syncthreads();
  t = warp_total(s_sum[threadIdx.x % 32][threadIdx.x / 32]);
  const int mine = blockIdx.x * 32 + threadIdx.x / 32;
  if (threadIdx.x % 32 == 0 && out != nullptr && mine < a.channels) out[mine] = from_f32<W>(t);
}

// ---------------------------------------------------------------- launches

bool gn_on_grid(const void* p, int64_t sample, int64_t position, int64_t samples, int64_t positions, int size) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (samples < 2 || sample * size % 16 == 0) &&
                          (positions < 2 || position * size % 16 == 0));
}

template <typename K>
cudaError_t after(K kernel, dim3 grid, int threads, cudaStream_t s, const GroupNormArgs& a, const GnCut& c) {
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t l{};
  l.gridDim = grid;
  l.blockDim = dim3(threads);
  l.stream = s;
  l.attrs = &attr;
  l.numAttrs = early_start(&attr);
  return cudaLaunchKernelEx(&l, kernel, a, c);
}

template <typename T, typename W, bool VEC>
cudaError_t gn_forward(const GroupNormArgs& a, int sms, cudaStream_t s) {
  const GnCut c = cut_for(a.channels, a.samples, a.positions, piece_size<T, VEC>(), sms);
  const dim3 grid(c.ctas, c.tiles);
  gn_stats_kernel<T, VEC><<<grid, kGnThreads, 0, s>>>(a, c);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return a.silu ? after(gn_apply_kernel<T, W, VEC, true>, grid, kGnThreads, s, a, c)
                : after(gn_apply_kernel<T, W, VEC, false>, grid, kGnThreads, s, a, c);
}

template <typename T, typename W, bool VEC>
cudaError_t gn_backward(const GroupNormArgs& a, int sms, cudaStream_t s) {
  const GnCut c = cut_for(a.channels, a.samples, a.positions, piece_size<T, VEC>(), sms);
  const dim3 grid(c.ctas, c.tiles);
  cudaError_t e = cudaSuccess;
  if (a.samples > 0) {
    if (a.silu) gn_sums_kernel<T, W, VEC, true><<<grid, kGnThreads, 0, s>>>(a, c);
    else gn_sums_kernel<T, W, VEC, false><<<grid, kGnThreads, 0, s>>>(a, c);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (a.dweight != nullptr || a.dbias != nullptr) {
    const dim3 columns(static_cast<unsigned>((a.channels + 31) / 32), 2);
    gn_columns_kernel<W><<<columns, 1024, 0, s>>>(a, a.samples > 0 ? c.ctas : 0);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (a.samples == 0) return e;
  if (a.silu) gn_grad_kernel<T, W, VEC, true><<<grid, kGnThreads, 0, s>>>(a, c);
  else gn_grad_kernel<T, W, VEC, false><<<grid, kGnThreads, 0, s>>>(a, c);
  return cudaGetLastError();
}

template <typename T>
bool gn_vectors(const GroupNormArgs& a) {
  const int size = sizeof(T);
  return static_cast<int64_t>(a.channels) * size % 16 == 0 &&
         gn_on_grid(a.x, a.x_sample, a.x_position, a.samples, a.positions, size) &&
         gn_on_grid(a.dy, a.dy_sample, a.dy_position, a.samples, a.positions, size) &&
         gn_on_grid(a.out, a.out_sample, a.out_position, a.samples, a.positions, size);
}
template <typename T, typename W>
cudaError_t gn_forward_type(const GroupNormArgs& a, int sms, cudaStream_t s) {
  return gn_vectors<T>(a) ? gn_forward<T, W, true>(a, sms, s) : gn_forward<T, W, false>(a, sms, s);
}
template <typename T, typename W>
cudaError_t gn_backward_type(const GroupNormArgs& a, int sms, cudaStream_t s) {
  return gn_vectors<T>(a) ? gn_backward<T, W, true>(a, sms, s) : gn_backward<T, W, false>(a, sms, s);
}

}  // namespace

GroupNormSpace group_norm_space(int32_t channels, int32_t groups, int64_t max_samples, int sms) {
  GroupNormSpace n{};
  for (int per : {1, 4, 8}) {
    if (channels % per != 0) continue;
    const GnCut c = cut_for(channels, 0, 1, per, sms);
    const int64_t items = max_samples + static_cast<int64_t>(kItemsPerSm) * sms;
    const int64_t stats = items * (groups + c.tiles) * 2;
    int64_t ctas = static_cast<int64_t>(kGnCtasPerSm) * sms / c.tiles;
    if (ctas < 1) ctas = 1;
    const int64_t columns = 2 * ctas * channels;
    if (stats > n.stats) n.stats = stats;
    if (columns > n.columns) n.columns = columns;
  }
  return n;
}

cudaError_t prepare_group_norm() { return cudaSuccess; }

#define ADAMW_GN_DISPATCH(fn)                                                     \
  if (dt == ADAMW_F32 && wdt == ADAMW_F32) return fn<float, float>(a, sms, s);    \
  if (dt == ADAMW_F16 && wdt == ADAMW_F32) return fn<__half, float>(a, sms, s);   \
  if (dt == ADAMW_F16 && wdt == ADAMW_F16) return fn<__half, __half>(a, sms, s);  \
  if (dt == ADAMW_BF16 && wdt == ADAMW_F32)                                       \
    return fn<__nv_bfloat16, float>(a, sms, s);                                   \
  if (dt == ADAMW_BF16 && wdt == ADAMW_BF16)                                      \
    return fn<__nv_bfloat16, __nv_bfloat16>(a, sms, s);                           \
  return cudaErrorInvalidValue;

cudaError_t launch_group_norm_forward(adamw_dtype dt, adamw_dtype wdt, GroupNormArgs a, int sms,
                                      cudaStream_t s) {
  ADAMW_GN_DISPATCH(gn_forward_type)
}
cudaError_t launch_group_norm_backward(adamw_dtype dt, adamw_dtype wdt, GroupNormArgs a, int sms,
                                       cudaStream_t s) {
  ADAMW_GN_DISPATCH(gn_backward_type)
}
#undef ADAMW_GN_DISPATCH

}  // namespace adamw
