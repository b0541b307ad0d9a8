// group_norm_backward.cu -- group norm's backward pass:
//     dz = dy act'(z),  A = mean(w dz),  B = mean(w dz xhat) over the group
//     dx = rstd (w dz - A - xhat B),  dweight = sum dz xhat,  dbias = sum dz
// A and B come from the same sums per channel as the columns' (A = sum_c w_c sum dz), so a
// thread keeps sums of its channels alone.  Column sums go from threads to CTAs to a
// table [CTAs][channels], whose rows the last kernel adds in their order.
#include "group_norm_cluster.cuh"

namespace adamw {
namespace {

constexpr int kFlush = 64;              // samples whose column sums a thread adds up before they join the rest

// The CTA's column sums from its threads': s holds [2 kPairs][kGnThreads] pairs, of the weight
// and the bias in turn.  Rows of threads are added up by halves.  Called by all threads.
template <int N>
__device__ __forceinline__ void gn_columns_out(const GroupNormArgs& a, const GnCut& c, const GnPlace<N>& at, float2* s) {
  constexpr int kPairs = gn_pairs<N>();
  if (a.dweight == nullptr && a.dbias == nullptr) return;
  int half = 1;
  while (2 * half < c.at_once) half *= 2;
  if (c.at_once > 1)
    for (; half > 0; half /= 2) {
      __syncthreads();
      if (at.there && at.row0 < half && at.row0 + half < c.at_once) {
        float2* mine = s + threadIdx.x;
#pragma unroll
        for (int j = 0; j < 2 * kPairs; ++j) mine[j * kGnThreads] = add2(mine[j * kGnThreads], mine[j * kGnThreads + half * c.wide]);
      }
    }
  if (!at.there || at.row0 != 0) return;
  float* out = a.columns + static_cast<int64_t>(blockIdx.x) * a.channels + at.channel();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 w = s[(2 * (i / 2)) * kGnThreads + threadIdx.x], b = s[(2 * (i / 2) + 1) * kGnThreads + threadIdx.x];
    out[i] = i % 2 == 0 ? w.x : w.y;
    out[static_cast<int64_t>(gridDim.x) * a.channels + i] = i % 2 == 0 ? b.x : b.y;
  }
}

template <typename T, int N, bool SILU, int K>
__global__ void __launch_bounds__(kGnThreads, K == 1 ? 3 : 2) gn_backward_small_kernel(const GroupNormArgs a, const GnCut c) {
  using P = GnPiece<T, N>;
  constexpr int kPairs = gn_pairs<N>();
  __shared__ float2 s_sum[kGnThreads], s_group[kGnThreads];
  __shared__ float2 s_column[2 * kPairs][kGnThreads];     // sums of all but the last few samples
  const GnPlace<N> at(c);
  const int team = at.row0 / c.team_rows, row0 = at.row0 - team * c.team_rows;
  const bool mine = at.there && team < c.teams;
  float2 w[kPairs], b[kPairs], col_w[kPairs] = {}, col_b[kPairs] = {};
  gn_weights<T, N>(a.weight, a.weight_f32, 1.0f, at, w);
  gn_weights<T, N>(a.bias, a.weight_f32, 0.0f, at, b);
#pragma unroll
  for (int j = 0; j < 2 * kPairs; ++j) s_column[j][threadIdx.x] = both(0.0f);
  const float inv = 1.0f / (static_cast<float>(a.positions) * static_cast<float>(c.per));
  const int rows = static_cast<int>(a.positions);
  const int64_t pace = static_cast<int64_t>(gridDim.x) * c.teams;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * c.teams + team;
  // of a lone piece the next sample's is on its way, with its statistics
  const bool one_row = mine && row0 < rows;
  const T* x = static_cast<const T*>(a.x) + first * a.x_sample + row0 * a.x_position + at.channel();
  const T* dy = static_cast<const T*>(a.dy) + first * a.dy_sample + row0 * a.dy_position + at.channel();
  const float *mean = a.mean + first * a.groups + at.group, *rstds = a.rstd + first * a.groups + at.group;
  T* dx = static_cast<T*>(a.out) + first * a.out_sample + row0 * a.out_position + at.channel();
  P next_x, next_dy;
  float next_mean = 0.0f, next_rstd = 0.0f;
  if (K == 1 && one_row && first < a.samples) {
    next_x.load_last(x);
    next_dy.load_last(dy);
    next_mean = __ldg(mean);
    next_rstd = __ldg(rstds);
  }
  int since = 0;
  for (int64_t sample = first; sample - team < a.samples; sample += pace) {
    const bool live = mine && sample < a.samples;
    P p[K], q[K];
    float start, rstd;
    if constexpr (K == 1) {
      p[0] = next_x;
      q[0] = next_dy;
      rstd = next_rstd;
      start = -next_mean * rstd;
      if (one_row && sample + pace < a.samples) {
        next_x.load_last(x + pace * a.x_sample);
        next_dy.load_last(dy + pace * a.dy_sample);
        next_mean = __ldg(mean + pace * a.groups);
        next_rstd = __ldg(rstds + pace * a.groups);
      }
    } else {
      rstd = start = 0.0f;
      if (live) {
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (row0 + k * c.team_rows < rows) {
            p[k].load_last(x + k * c.team_rows * a.x_position);
            q[k].load_last(dy + k * c.team_rows * a.dy_position);
          }
        rstd = __ldg(rstds);
        start = -__ldg(mean) * rstd;
      }
    }
    float2 one = both(0.0f), two = both(0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (live && row0 + k * c.team_rows < rows) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 xhat = fma_of<N>(p[k].pair(i), both(rstd), both(start));
          const float2 dz = through<T, N, SILU>(q[k].pair(i), fma_of<N>(xhat, w[i], b[i]));
          col_b[i] = add_of<N>(col_b[i], dz);
          col_w[i] = fma_of<N>(dz, xhat, col_w[i]);
          const float2 g = mul2(dz, w[i]);
          one = add_of<N>(one, g);
          two = fma_of<N>(g, xhat, two);
        }
      }
    const float2 means = mul2(gn_team_sums(N == 1 ? make_float2(one.x, two.x) : make_float2(one.x + one.y, two.x + two.y), c, s_sum, s_group),
                              both(-inv));
    if (++since == kFlush) {
      since = 0;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        s_column[2 * i][threadIdx.x] = add_of<N>(s_column[2 * i][threadIdx.x], col_w[i]);
        s_column[2 * i + 1][threadIdx.x] = add_of<N>(s_column[2 * i + 1][threadIdx.x], col_b[i]);
        col_w[i] = col_b[i] = both(0.0f);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (live && row0 + k * c.team_rows < rows) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 xhat = fma_of<N>(p[k].pair(i), both(rstd), both(start));
          const float2 dz = through<T, N, SILU>(q[k].pair(i), fma_of<N>(xhat, w[i], b[i]));
          p[k].set(i, mul_of<N>(both(rstd), fma_of<N>(xhat, both(means.y), fma_of<N>(dz, w[i], both(means.x)))));
        }
        p[k].store(dx + k * c.team_rows * a.out_position);
      }
    x += pace * a.x_sample;
    dy += pace * a.dy_sample;
    dx += pace * a.out_sample;
    mean += pace * a.groups;
    rstds += pace * a.groups;
  }
  let_next_kernel_start();
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    s_column[2 * i][threadIdx.x] = add_of<N>(s_column[2 * i][threadIdx.x], col_w[i]);
    s_column[2 * i + 1][threadIdx.x] = add_of<N>(s_column[2 * i + 1][threadIdx.x], col_b[i]);
  }
  gn_columns_out<N>(a, c, at, &s_column[0][0]);
}

// As the forward pass's kernel for samples of one position and groups of neighbouring lanes.
constexpr int kLaneSamples = 2;
template <typename T, int N, bool SILU>
__global__ void __launch_bounds__(kGnThreads, 3) gn_backward_lanes_kernel(const GroupNormArgs a, const GnCut c) {
  using P = GnPiece<T, N>;
  constexpr int kPairs = gn_pairs<N>(), U = kLaneSamples;
  __shared__ float2 s_column[2 * kPairs][kGnThreads];     // sums of all but the last few samples
  const GnPlace<N> at(c);
  float2 w[kPairs], b[kPairs], col_w[kPairs] = {}, col_b[kPairs] = {};
  gn_weights<T, N>(a.weight, a.weight_f32, 1.0f, at, w);
  gn_weights<T, N>(a.bias, a.weight_f32, 0.0f, at, b);
#pragma unroll
  for (int j = 0; j < 2 * kPairs; ++j) s_column[j][threadIdx.x] = both(0.0f);
  const float inv = 1.0f / static_cast<float>(c.per);
  const int64_t pace = static_cast<int64_t>(gridDim.x) * c.teams;
  const T *x0 = static_cast<const T*>(a.x) + at.channel(), *dy0 = static_cast<const T*>(a.dy) + at.channel();
  int since = 0;
  for (int64_t n0 = static_cast<int64_t>(blockIdx.x) * c.teams; n0 < a.samples; n0 += U * pace) {
    P p[U], q[U];
    float rstd[U], start[U];
    float2 t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t sample = n0 + u * pace + at.row0;
      p[u].v = {};
      q[u].v = {};
      rstd[u] = start[u] = 0.0f;
      if (at.there && sample < a.samples) {
        p[u].load_last(x0 + sample * a.x_sample);
        q[u].load_last(dy0 + sample * a.dy_sample);
        rstd[u] = __ldg(a.rstd + sample * a.groups + at.group);
        start[u] = __ldg(a.mean + sample * a.groups + at.group);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = at.there && n0 + u * pace + at.row0 < a.samples;
      start[u] *= -rstd[u];
      float2 one = both(0.0f), two = both(0.0f);
      if (live) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 xhat = fma_of<N>(p[u].pair(i), both(rstd[u]), both(start[u]));
          const float2 dz = through<T, N, SILU>(q[u].pair(i), fma_of<N>(xhat, w[i], b[i]));
          col_b[i] = add_of<N>(col_b[i], dz);
          col_w[i] = fma_of<N>(dz, xhat, col_w[i]);
          const float2 g = mul2(dz, w[i]);
          one = add_of<N>(one, g);
          two = fma_of<N>(g, xhat, two);
        }
      }
      t[u] = N == 1 ? make_float2(one.x, two.x) : make_float2(one.x + one.y, two.x + two.y);
    }
    for (int o = 1; o < c.group_pieces; o *= 2)
#pragma unroll
      for (int u = 0; u < U; ++u)
        t[u] = add2(t[u], make_float2(__shfl_xor_sync(kFull, t[u].x, o), __shfl_xor_sync(kFull, t[u].y, o)));
    if (++since == kFlush / U) {
      since = 0;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        s_column[2 * i][threadIdx.x] = add_of<N>(s_column[2 * i][threadIdx.x], col_w[i]);
        s_column[2 * i + 1][threadIdx.x] = add_of<N>(s_column[2 * i + 1][threadIdx.x], col_b[i]);
        col_w[i] = col_b[i] = both(0.0f);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t sample = n0 + u * pace + at.row0;
      if (!at.there || sample >= a.samples) continue;
      const float2 means = mul2(t[u], both(-inv));
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 xhat = fma_of<N>(p[u].pair(i), both(rstd[u]), both(start[u]));
        const float2 dz = through<T, N, SILU>(q[u].pair(i), fma_of<N>(xhat, w[i], b[i]));
        p[u].set(i, mul_of<N>(both(rstd[u]), fma_of<N>(xhat, both(means.y), fma_of<N>(dz, w[i], both(means.x)))));
      }
      p[u].store(static_cast<T*>(a.out) + sample * a.out_sample + at.channel());
    }
  }
  let_next_kernel_start();
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    s_column[2 * i][threadIdx.x] = add_of<N>(s_column[2 * i][threadIdx.x], col_w[i]);
    s_column[2 * i + 1][threadIdx.x] = add_of<N>(s_column[2 * i + 1][threadIdx.x], col_b[i]);
  }
  gn_columns_out<N>(a, c, at, &s_column[0][0]);
}

__device__ __forceinline__ float2 gn_from(float2 t, int lanes) {
  return make_float2(__shfl_xor_sync(kFull, t.x, lanes), __shfl_xor_sync(kFull, t.y, lanes));
}
// The two means of groups first .. first + groups - 1 of a sample from its parts' sums, by a warp.
__device__ __noinline__ void gn_join_sums(const GroupNormArgs& a, const GnCut& c, const float2* stats, int64_t sample, int first,
                                             int groups) {
  const GnLanes l(groups);
  const int pitch = gn_pitch(a, c);
  const float inv = 1.0f / (static_cast<float>(a.positions) * static_cast<float>(c.per));
  for (int g0 = 0; g0 < groups; g0 += l.wide) {
    const int g = first + g0 + l.slot;
    float2 t = both(0.0f);
    if (g < first + groups) {
      for (int tile = g * c.group_pieces / c.wide; tile <= ((g + 1) * c.group_pieces - 1) / c.wide; ++tile) {
        const float2* p = stats + g + (c.aligned ? 0 : tile);
        for (int part = l.at; part < c.parts; part += 8 * l.share) {
          float2 v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            v[u] = both(0.0f);
            if (part + u * l.share < c.parts) v[u] = __ldcg(p + static_cast<int64_t>(part + u * l.share) * pitch);
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) t = add2(t, v[u]);
        }
      }
    }
    for (int o = l.wide; o < 32; o *= 2) t = add2(t, gn_from(t, o));
    if (l.at == 0 && g < first + groups)
      __stcg(reinterpret_cast<float2*>(a.joined) + sample * a.groups + g, mul2(t, both(inv)));
  }
}

template <typename T, int N, bool SILU>
__global__ void __launch_bounds__(kGnThreads, 3) gn_backward_cluster_kernel(const GroupNormArgs a, const GnCut c) {
  using P = GnPiece<T, N>;
  constexpr int kPairs = gn_pairs<N>(), kUnroll = N <= 2 ? 4 : 2;
  extern __shared__ uint4 s_tile[];
  __shared__ float2 s_sum[kGnThreads], s_group[kGnTileGroups], s_slots[2][kGnClusterMax][kGnTileGroups];
  gn_started(c.cluster);
  const GnPlace<N> at(c);
  const int rank = c.cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = rank * c.part_rows;
  const int rows = max(0, min(c.part_rows, static_cast<int>(a.positions) - first));
  const int tile_bytes = at.tile_pieces * P::kBytes;
  float2 w[kPairs], b[kPairs], all_w[kPairs] = {}, all_b[kPairs] = {};
  gn_weights<T, N>(a.weight, a.weight_f32, 1.0f, at, w);
  gn_weights<T, N>(a.bias, a.weight_f32, 0.0f, at, b);
  const float inv = 1.0f / (static_cast<float>(a.positions) * static_cast<float>(c.per));
  const int group = at.there ? at.group - at.first_group : 0;
  const int size = sizeof(T), other = c.part_rows * c.wide * P::kBytes;      // from x to dy
  const char* tile = reinterpret_cast<const char*>(s_tile) + (threadIdx.x % c.wide) * P::kBytes;
  const int row_bytes = c.at_once * tile_bytes;
  int turn = 0;
  bool all_started = false;
  for (int64_t sample = blockIdx.x / c.cluster; sample < a.samples; sample += gridDim.x / c.cluster) {
    __syncthreads();                    // the sample before is done with
    char* to = reinterpret_cast<char*>(s_tile);
    gn_fetch<P::kBytes>(to, reinterpret_cast<const char*>(static_cast<const T*>(a.x) + sample * a.x_sample + first * a.x_position) + at.tile0 * P::kBytes,
             rows, tile_bytes, a.x_position * size, c.unit);
    gn_fetch<P::kBytes>(to + other,
             reinterpret_cast<const char*>(static_cast<const T*>(a.dy) + sample * a.dy_sample + first * a.dy_position) + at.tile0 * P::kBytes,
             rows, tile_bytes, a.dy_position * size, c.unit);
    float rstd = 0.0f, start = 0.0f;
    if (at.there) {
      rstd = __ldg(a.rstd + sample * a.groups + at.group);
      start = -__ldg(a.mean + sample * a.groups + at.group) * rstd;
    }
    gn_fetched();
    gn_all_started(c.cluster, &all_started);
    float2 col_w[kPairs] = {}, col_b[kPairs] = {};
    if (at.there) {
      const char* p = tile + at.row0 * tile_bytes;
#pragma unroll kUnroll
      for (int l = at.row0; l < rows; l += c.at_once, p += row_bytes) {
        const P v = *reinterpret_cast<const P*>(p), g = *reinterpret_cast<const P*>(p + other);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const float2 xhat = fma_of<N>(v.pair(j), both(rstd), both(start));
          const float2 dz = through<T, N, SILU>(g.pair(j), fma_of<N>(xhat, w[j], b[j]));
          col_b[j] = add_of<N>(col_b[j], dz);
          col_w[j] = fma_of<N>(dz, xhat, col_w[j]);
        }
      }
    }
    float2 one = both(0.0f), two = both(0.0f);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      one = fma_of<N>(w[j], col_b[j], one);
      two = fma_of<N>(w[j], col_w[j], two);
      all_w[j] = add_of<N>(all_w[j], col_w[j]);
      all_b[j] = add_of<N>(all_b[j], col_b[j]);
    }
    gn_block_sums<N>(c, at, N == 1 ? make_float2(one.x, two.x) : make_float2(one.x + one.y, two.x + two.y), s_sum, s_group);
    // two sets of slots: a CTA may be a sample ahead of one that still reads
    gn_exchange(c.cluster, rank, at.groups, s_group, s_slots[turn]);
    float2 means = both(0.0f);
    for (int r = 0; r < c.cluster; ++r) means = add2(means, s_slots[turn][r][group]);
    turn ^= 1;
    means = mul2(means, both(-inv * rstd));
    if (!at.there) continue;
    T* dx = static_cast<T*>(a.out) + sample * a.out_sample + (first + at.row0) * a.out_position + at.channel();
    const int64_t pace = c.at_once * a.out_position;
    const char* p = tile + at.row0 * tile_bytes;
#pragma unroll kUnroll
    for (int l = at.row0; l < rows; l += c.at_once, p += row_bytes, dx += pace) {
      P v = *reinterpret_cast<const P*>(p);
      const P g = *reinterpret_cast<const P*>(p + other);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const float2 xhat = fma_of<N>(v.pair(j), both(rstd), both(start));
        const float2 dz = through<T, N, SILU>(g.pair(j), fma_of<N>(xhat, w[j], b[j]));
        v.set(j, fma_of<N>(xhat, both(means.y), fma_of<N>(mul_of<N>(dz, w[j]), both(rstd), both(means.x))));
      }
      v.store(dx);
    }
  }
  let_next_kernel_start();
  __syncthreads();                        // the last sample is done with
  float2* s_column = reinterpret_cast<float2*>(s_tile) + threadIdx.x;
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    s_column[2 * j * kGnThreads] = all_w[j];
    s_column[(2 * j + 1) * kGnThreads] = all_b[j];
  }
  gn_columns_out<N>(a, c, at, reinterpret_cast<float2*>(s_tile));
}

constexpr int kBackwardDepth = 10;      // steps on their way, at most 72 KB a CTA

// The items of the eight warps.  s_column: this thread's column sums, [2 kPairs][kGnThreads].
template <typename T, int N, bool SILU>
__device__ __forceinline__ void gn_backward_items(const GroupNormArgs& a, const GnCut& c, const GnPlace<N>& at, const GnPart& part,
                                                  const uint32_t* words, void* s_ring, float2 (*s_stat)[kGnThreads], float2* s_column) {
  using Ring = GnRing<T, N, 2, kBackwardDepth>;
  using P = GnPiece<T, N>;
  constexpr int kPairs = gn_pairs<N>();
  Ring ring(s_ring, a, c, part, at);
  float2 w[kPairs], b[kPairs];
  gn_weights<T, N>(a.weight, a.weight_f32, 1.0f, at, w);
  gn_weights<T, N>(a.bias, a.weight_f32, 0.0f, at, b);
#pragma unroll
  for (int j = 0; j < 2 * kPairs; ++j) s_column[j * kGnThreads] = both(0.0f);
  uint64_t limit = a.wait_ns;
  for (uint32_t n = 0; n < part.turns; ++n) {
    const GnTurn turn(n);
    const int64_t sample = part.sample(turn.batch, c);
    if (sample >= a.samples) continue;
    float rstd = 0.0f, start = 0.0f;
    if (at.there) {
      rstd = __ldg(a.rstd + sample * a.groups + at.group);
      start = -__ldg(a.mean + sample * a.groups + at.group) * rstd;
    }
    if (!turn.result) {
      float2 col_w[kPairs] = {}, col_b[kPairs] = {};
      for (int k = 0; k < part.steps; ++k) {
        P p[2];
        ring.get(p);                       // a dy of 0 where there is no row
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const float2 xhat = fma_of<N>(p[0].pair(j), both(rstd), both(start));
          const float2 dz = through<T, N, SILU>(p[1].pair(j), fma_of<N>(xhat, w[j], b[j]));
          col_b[j] = add_of<N>(col_b[j], dz);
          col_w[j] = fma_of<N>(dz, xhat, col_w[j]);
        }
      }
      float2 one = both(0.0f), two = both(0.0f);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        one = fma_of<N>(w[j], col_b[j], one);
        two = fma_of<N>(w[j], col_w[j], two);
        s_column[2 * j * kGnThreads] = add_of<N>(s_column[2 * j * kGnThreads], col_w[j]);
        s_column[(2 * j + 1) * kGnThreads] = add_of<N>(s_column[(2 * j + 1) * kGnThreads], col_b[j]);
      }
      float2 t = N == 1 ? make_float2(one.x, two.x) : make_float2(one.x + one.y, two.x + two.y);
      if (c.by_lanes)
        for (int o = 1; o < c.group_pieces; o *= 2) t = add2(t, gn_from(t, o));
      float2* s = s_stat[turn.batch % 2];
      if (turn.batch >= 2) gn_wait_freed(turn.batch % 2);
      if (!c.by_lanes) s[threadIdx.x] = t;
      else if (at.there && at.piece % c.group_pieces == 0) s[at.row0 * at.groups + at.group - at.first_group] = t;
      gn_filled(turn.batch % 2);
      continue;
    }
    const bool open = gn_wait_open(a, words, turn.batch, &limit);
    float2 means = both(0.0f);
    if (at.there) means = mul2(__ldcg(reinterpret_cast<const float2*>(a.joined) + sample * a.groups + at.group), both(-rstd));
    T* dx = static_cast<T*>(a.out) + sample * a.out_sample + static_cast<int64_t>(part.first + at.row0) * a.out_position + at.channel();
    const int64_t out_pace = c.at_once * a.out_position;
    const int rows = open ? ring.rows : 0;
    float2 slope[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) slope[j] = mul_of<N>(w[j], both(rstd));
    for (int k = 0; k < part.steps; ++k) {
      P p[2];
      ring.get(p);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const float2 xhat = fma_of<N>(p[0].pair(j), both(rstd), both(start));
        const float2 dz = through<T, N, SILU>(p[1].pair(j), fma_of<N>(xhat, w[j], b[j]));
        p[0].set(j, fma_of<N>(xhat, both(means.y), fma_of<N>(dz, slope[j], both(means.x))));
      }
      if (k < rows) p[0].store(dx);
      dx += out_pace;
    }
  }
}

template <typename T, int N, bool SILU>
__global__ void __launch_bounds__(kGnFusedThreads, kGnCtasPerSm) gn_backward_fused_kernel(const GroupNormArgs a, const GnCut c) {
  using Ring = GnRing<T, N, 2, kBackwardDepth>;
  constexpr int kPairs = gn_pairs<N>();
  extern __shared__ uint4 s_ring[];
  __shared__ float2 s_stat[2][kGnThreads];     // as in the forward pass
  float2* s_column = reinterpret_cast<float2*>(reinterpret_cast<char*>(s_ring) + Ring::kBytes) + threadIdx.x % kGnThreads;
  const GnPlace<N> at(c);
  const GnPart part(a, c);
  uint32_t* words = gn_words(a, c, part);
  const int tile_groups = at.groups;
  if (threadIdx.x >= kGnThreads) {
    const GnLanes lanes(tile_groups);
    const int place = part.part * gn_pitch(a, c) + at.first_group + (c.aligned ? 0 : blockIdx.y);
    for (uint32_t batch = 0; part.sample(batch, c) < a.samples; ++batch) {
      const int64_t sample = part.sample(batch, c);
      float2* stats = gn_stats(a, c, batch, part);
      const float2* s = s_stat[batch % 2];
      gn_wait_filled(batch % 2);
      for (int g0 = 0; g0 < tile_groups; g0 += lanes.wide) {
        const int g = g0 + lanes.slot;
        float2 u = both(0.0f);
        if (g < tile_groups) {
          if (c.by_lanes) {
            for (int r = lanes.at; r < c.at_once; r += lanes.share) u = add2(u, s[r * tile_groups + g]);
          } else {
            const int lo = max((at.first_group + g) * c.group_pieces, at.tile0) - at.tile0;
            const int q = min((at.first_group + g + 1) * c.group_pieces, at.tile0 + at.tile_pieces) - at.tile0 - lo;
            for (int e = lanes.at; e < q * c.at_once; e += lanes.share) u = add2(u, s[e / q * c.wide + lo + e % q]);
          }
        }
        for (int o = lanes.wide; o < 32; o *= 2) u = add2(u, gn_from(u, o));
        if (lanes.at == 0 && g < tile_groups) __stcg(stats + place + g, u);
      }
      if (part.sample(batch + 2, c) < a.samples) gn_freed(batch % 2);
      if (gn_arrive(c, words, batch)) {
        if (c.aligned) gn_join_sums(a, c, stats, sample, at.first_group, tile_groups);
        else gn_join_sums(a, c, stats, sample, 0, a.groups);
        gn_open(words, batch);
      }
    }
  } else {
    gn_backward_items<T, N, SILU>(a, c, at, part, words, s_ring, s_stat, s_column);
  }
  gn_columns_out<N>(a, c, at, reinterpret_cast<float2*>(reinterpret_cast<char*>(s_ring) + Ring::kBytes));
  gn_leave(a, c);
}

template <typename T, int N>
constexpr int gn_backward_smem() {
  return GnRing<T, N, 2, kBackwardDepth>::kBytes + 2 * gn_pairs<N>() * kGnThreads * static_cast<int>(sizeof(float2));
}

// Sums the CTAs' column sums, in their order: blockIdx.y 0 the weight's, 1 the bias's.
template <typename W>
__global__ void __launch_bounds__(1024) gn_columns_kernel(const GroupNormArgs a, const int rows) {
  __shared__ float s_sum[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x % 32, r0 = threadIdx.x / 32;
  W* out = static_cast<W*>(blockIdx.y == 0 ? a.dweight : a.dbias);
  wait_for_previous_kernel();
  float t = 0.0f;
  if (col < a.channels) {
#pragma unroll 4
    for (int r = r0; r < rows; r += 32)
      t += __ldcg(a.columns + (static_cast<int64_t>(blockIdx.y) * rows + r) * a.channels + col);
  }
  s_sum[r0][threadIdx.x % 32] = t;
  __syncthreads();
  t = warp_total(s_sum[threadIdx.x % 32][threadIdx.x / 32]);
  const int mine = blockIdx.x * 32 + threadIdx.x / 32;
  if (threadIdx.x % 32 == 0 && out != nullptr && mine < a.channels) out[mine] = from_f32<W>(t);
}

template <typename W>
cudaError_t gn_columns(const GroupNormArgs& a, int rows, cudaStream_t s) {
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t l{};
  l.gridDim = dim3(static_cast<unsigned>((a.channels + 31) / 32), 2);
  l.blockDim = dim3(1024);
  l.stream = s;
  l.attrs = &attr;
  l.numAttrs = early_start(&attr);
  return cudaLaunchKernelEx(&l, gn_columns_kernel<W>, a, rows);
}

template <typename T, int N, bool SILU>
cudaError_t gn_backward(const GroupNormArgs& a, int sms, cudaStream_t s) {
  const GnCut c = gn_cut(a, N, sms);
  const dim3 grid(c.ctas, c.tiles);
  if (a.samples > 0) {
    const GnKind kind = gn_kind(a, c);
    const cudaError_t e =
        kind == kGnCluster ? gn_cluster_launch(gn_backward_cluster_kernel<T, N, SILU>, gn_cluster_bytes(a, c, N), s, a, c)
        : kind == kGnFused ? gn_launch(gn_backward_fused_kernel<T, N, SILU>, grid, kGnFusedThreads, gn_backward_smem<T, N>(), s, a, c)
        : kind == kGnLanes ? gn_launch(gn_backward_lanes_kernel<T, N, SILU>, grid, kGnThreads, 0, s, a, c)
        : kind == kGnRow   ? gn_launch(gn_backward_small_kernel<T, N, SILU, 1>, grid, kGnThreads, 0, s, a, c)
                           : gn_launch(gn_backward_small_kernel<T, N, SILU, kSmallBackward>, grid, kGnThreads, 0, s, a, c);
    if (e != cudaSuccess) return e;
  }
  if (a.dweight == nullptr && a.dbias == nullptr) return cudaSuccess;
  const int rows = a.samples > 0 ? c.ctas : 0;
  return a.weight_f32 ? gn_columns<float>(a, rows, s) : gn_columns<T>(a, rows, s);
}
template <typename T>
cudaError_t gn_backward_type(const GroupNormArgs& a, int sms, cudaStream_t s) {
  constexpr int kWide = 16 / sizeof(T);
  const int n = gn_piece(a, sizeof(T));
  if (n == kWide) return a.silu ? gn_backward<T, kWide, true>(a, sms, s) : gn_backward<T, kWide, false>(a, sms, s);
  if constexpr (sizeof(T) == 2)
    if (n == 2) return a.silu ? gn_backward<T, 2, true>(a, sms, s) : gn_backward<T, 2, false>(a, sms, s);
  return a.silu ? gn_backward<T, 1, true>(a, sms, s) : gn_backward<T, 1, false>(a, sms, s);
}

template <typename T, int N, bool SILU>
cudaError_t gn_prepare_one() {
  const cudaError_t e = cudaFuncSetAttribute(gn_backward_fused_kernel<T, N, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             gn_backward_smem<T, N>());
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(gn_backward_cluster_kernel<T, N, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGnClusterBytes);
}
template <typename T, int N>
cudaError_t gn_prepare_backward() {
  const cudaError_t e = gn_prepare_one<T, N, true>();
  return e == cudaSuccess ? gn_prepare_one<T, N, false>() : e;
}

}  // namespace

cudaError_t prepare_group_norm_backward() {
  cudaError_t e = cudaSuccess;
  if (e == cudaSuccess) e = gn_prepare_backward<float, 4>();
  if (e == cudaSuccess) e = gn_prepare_backward<float, 1>();
  if (e == cudaSuccess) e = gn_prepare_backward<__half, 8>();
  if (e == cudaSuccess) e = gn_prepare_backward<__half, 2>();
  if (e == cudaSuccess) e = gn_prepare_backward<__half, 1>();
  if (e == cudaSuccess) e = gn_prepare_backward<__nv_bfloat16, 8>();
  if (e == cudaSuccess) e = gn_prepare_backward<__nv_bfloat16, 2>();
  if (e == cudaSuccess) e = gn_prepare_backward<__nv_bfloat16, 1>();
  return e;
}

cudaError_t launch_group_norm_backward(adamw_dtype dt, const GroupNormArgs& a, int sms, cudaStream_t s) {
  if (dt == ADAMW_F32) return gn_backward_type<float>(a, sms, s);
  if (dt == ADAMW_F16) return gn_backward_type<__half>(a, sms, s);
  return gn_backward_type<__nv_bfloat16>(a, sms, s);
}

}  // namespace adamw
