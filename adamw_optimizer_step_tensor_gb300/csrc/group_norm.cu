// group_norm.cu -- group norm with an activation over channels-last tensors: the forward pass
// (group_norm_cut.cpp: how calls are cut up).
//
// Statistics of the fused kernel: a thread sums x - K and its square, K the first of its
// own values, and starts anew after kRun values.  K is one of the n values it is subtracted
// from, so the sum of squares is at most 2 n times the spread about their mean: the
// difference loses log2(2 n) bits at worst, whatever the mean.  From there on spreads are
// joined by counts: M2 = sum M2_i + n_i (mean_i - mean)^2.  The mean itself comes from the
// sum of the values as they are, a thread's runs added with their rounding errors: a mean
// near 0 of large values keeps its bits, which the K would take.  The small kernel has the
// values in registers and sums about their mean.
#include "group_norm_cluster.cuh"

namespace adamw {
namespace {

constexpr int kRun = 64;                // values of a run of sums

template <typename T, int N, bool SILU, int K>
__global__ void __launch_bounds__(kGnThreads, K == 1 ? kSmallCtasPerSm : 2) gn_forward_small_kernel(const GroupNormArgs a, const GnCut c) {
  using P = GnPiece<T, N>;
  constexpr int kPairs = gn_pairs<N>();
  __shared__ float2 s_sum[kGnThreads], s_group[kGnThreads];
  const GnPlace<N> at(c);
  const int team = at.row0 / c.team_rows, row0 = at.row0 - team * c.team_rows;
  const bool mine = at.there && team < c.teams;
  float2 w[kPairs], b[kPairs];
  gn_weights<T, N>(a.weight, a.weight_f32, 1.0f, at, w);
  gn_weights<T, N>(a.bias, a.weight_f32, 0.0f, at, b);
  const float inv = 1.0f / (static_cast<float>(a.positions) * static_cast<float>(c.per));
  const int rows = static_cast<int>(a.positions);
  const int64_t pace = static_cast<int64_t>(gridDim.x) * c.teams;
  const T* x0 = static_cast<const T*>(a.x) + at.channel();
  P next;                                 // of a lone piece the next sample's is on its way
  if (K == 1 && mine && static_cast<int64_t>(blockIdx.x) * c.teams + team < a.samples && row0 < rows)
    next.load_last(x0 + (static_cast<int64_t>(blockIdx.x) * c.teams + team) * a.x_sample + row0 * a.x_position);
  for (int64_t n0 = static_cast<int64_t>(blockIdx.x) * c.teams; n0 < a.samples; n0 += pace) {
    const int64_t sample = n0 + team;
    const bool live = mine && sample < a.samples;
    const T* x = x0 + sample * a.x_sample;
    P p[K];
    float2 sum = both(0.0f);
    if constexpr (K == 1) {
      p[0] = next;
      if (mine && sample + pace < a.samples && row0 < rows)
        next.load_last(x + pace * a.x_sample + row0 * a.x_position);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int l = row0 + k * c.team_rows;
        if (live && l < rows) p[k].load_last(x + l * a.x_position);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (live && row0 + k * c.team_rows < rows) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) sum = add_of<N>(sum, p[k].pair(i));
      }
    const float mean = gn_team_sums(make_float2(sum.x + sum.y, 0.0f), c, s_sum, s_group).x * inv;
    float2 square = both(0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (live && row0 + k * c.team_rows < rows) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          float2 d = add_of<N>(p[k].pair(i), both(-mean));
          square = fma_of<N>(d, d, square);
        }
      }
    const float spread = gn_team_sums(make_float2(square.x + square.y, 0.0f), c, s_sum, s_group).x;
    const float rstd = __frcp_rn(__fsqrt_rn(fmaf(spread, inv, a.eps)));
    if (!live) continue;
    if (row0 == 0 && at.piece % c.group_pieces == 0) {
      a.mean[sample * a.groups + at.group] = mean;
      a.rstd[sample * a.groups + at.group] = rstd;
    }
    T* y = static_cast<T*>(a.out) + sample * a.out_sample + at.channel();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int l = row0 + k * c.team_rows;
      if (l < rows) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 xhat = mul_of<N>(add_of<N>(p[k].pair(i), both(-mean)), both(rstd));
          p[k].set(i, activate<T, N, SILU>(fma_of<N>(xhat, w[i], b[i])));
        }
        p[k].store(y + l * a.out_position);
      }
    }
  }
}

// Samples of one position whose groups are a power of two of neighbouring lanes (heads): no
// thread waits for another warp, and each has the pieces of kLaneSamples samples on their way.
// 4096 x 4096 bf16 in 64 groups: 23 us sample by sample.
constexpr int kLaneSamples = 4;
template <typename T, int N, bool SILU>
__global__ void __launch_bounds__(kGnThreads, kSmallCtasPerSm) gn_forward_lanes_kernel(const GroupNormArgs a, const GnCut c) {
  using P = GnPiece<T, N>;
  constexpr int kPairs = gn_pairs<N>(), U = kLaneSamples;
  const GnPlace<N> at(c);
  float2 w[kPairs], b[kPairs];
  gn_weights<T, N>(a.weight, a.weight_f32, 1.0f, at, w);
  gn_weights<T, N>(a.bias, a.weight_f32, 0.0f, at, b);
  const float inv = 1.0f / static_cast<float>(c.per);
  const int64_t pace = static_cast<int64_t>(gridDim.x) * c.teams;
  const T* x0 = static_cast<const T*>(a.x) + at.channel();
  for (int64_t n0 = static_cast<int64_t>(blockIdx.x) * c.teams; n0 < a.samples; n0 += U * pace) {
    P p[U];
    float sum[U], square[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t sample = n0 + u * pace + at.row0;
      if (at.there && sample < a.samples) p[u].load_last(x0 + sample * a.x_sample);
      else p[u].v = {};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 t = p[u].pair(0);
#pragma unroll
      for (int i = 1; i < kPairs; ++i) t = add_of<N>(t, p[u].pair(i));
      sum[u] = t.x + t.y;
    }
    for (int o = 1; o < c.group_pieces; o *= 2)
#pragma unroll
      for (int u = 0; u < U; ++u) sum[u] += __shfl_xor_sync(kFull, sum[u], o);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      sum[u] *= inv;                        // the mean
      float2 t = both(0.0f);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        float2 d = add_of<N>(p[u].pair(i), both(-sum[u]));
        t = fma_of<N>(d, d, t);
      }
      square[u] = t.x + t.y;
    }
    for (int o = 1; o < c.group_pieces; o *= 2)
#pragma unroll
      for (int u = 0; u < U; ++u) square[u] += __shfl_xor_sync(kFull, square[u], o);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t sample = n0 + u * pace + at.row0;
      if (!at.there || sample >= a.samples) continue;
      const float mean = sum[u], rstd = __frcp_rn(__fsqrt_rn(fmaf(square[u], inv, a.eps)));
      if (at.piece % c.group_pieces == 0) {
        a.mean[sample * a.groups + at.group] = mean;
        a.rstd[sample * a.groups + at.group] = rstd;
      }
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        p[u].set(i, activate<T, N, SILU>(fma_of<N>(mul_of<N>(add_of<N>(p[u].pair(i), both(-mean)), both(rstd)), w[i], b[i])));
      p[u].store(static_cast<T*>(a.out) + sample * a.out_sample + at.channel());
    }
  }
}

// A spread that roundings made negative is 0.  One that is no number stays so (fmaxf would make it 0):
// a value that is infinite or no number has no spread about any mean.
__device__ __forceinline__ float gn_spread(float x) { return x < 0.0f ? 0.0f : x; }
// Joins (count, mean, spread) u to t.
__device__ __forceinline__ float3 gn_merge_means(float3 t, float3 u) {
  const float all = t.x + u.x, share = __fdividef(u.x, all), d = u.y - t.y;
  if (t.x == 0.0f) return u;
  return make_float3(all, fmaf(d, share, t.y), t.z + fmaf(d * d, t.x * share, u.z));
}
// Joins (count, sum, spread) u to t.
__device__ __forceinline__ float3 gn_merge(float3 t, float3 u) {
  if (t.x == 0.0f) return u;
  if (u.x == 0.0f) return t;
  const float all = t.x + u.x, d = __fdividef(u.y, u.x) - __fdividef(t.y, t.x);
  return make_float3(all, t.y + u.y, t.z + fmaf(d * d, __fdividef(t.x * u.x, all), u.z));
}
// hi + lo += x, without the rounding error of hi.
__device__ __forceinline__ void add_exactly(float x, float* hi, float* lo) {
  const float s = *hi + x, of_x = s - *hi;
  *lo += (*hi - (s - of_x)) + (x - of_x);
  *hi = s;
}
__device__ __forceinline__ float3 gn_from(float3 t, int lanes) {
  return make_float3(__shfl_xor_sync(kFull, t.x, lanes), __shfl_xor_sync(kFull, t.y, lanes), __shfl_xor_sync(kFull, t.z, lanes));
}

// Means and reciprocal deviations of groups first .. first + groups - 1 of a sample from its
// parts' statistics, by a warp.
__device__ __noinline__ void gn_join(const GroupNormArgs& a, const GnCut& c, const float2* stats, int64_t sample, int first,
                                        int groups, int piece) {
  const GnLanes l(groups);
  const int pitch = gn_pitch(a, c);
  const float all = static_cast<float>(a.positions) * static_cast<float>(c.per), inv = 1.0f / all;
  for (int g0 = 0; g0 < groups; g0 += l.wide) {
    const int g = first + g0 + l.slot, p0 = g * c.group_pieces, p1 = p0 + c.group_pieces;
    float3 t = make_float3(0.0f, 0.0f, 0.0f);
    if (g < first + groups) {
      for (int tile = p0 / c.wide; tile <= (p1 - 1) / c.wide; ++tile) {
        const float ch = static_cast<float>((min(p1, (tile + 1) * c.wide) - max(p0, tile * c.wide)) * piece);
        const float2* p = stats + g + (c.aligned ? 0 : tile);
        for (int part = l.at; part < c.parts; part += 8 * l.share) {
          float2 v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (part + u * l.share < c.parts) v[u] = __ldcg(p + static_cast<int64_t>(part + u * l.share) * pitch);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int q = part + u * l.share;
            if (q < c.parts)
              t = gn_merge(t, make_float3(static_cast<float>(min(c.part_rows, static_cast<int>(a.positions) - q * c.part_rows)) * ch,
                                          v[u].x, v[u].y));
          }
        }
      }
    }
    for (int o = l.wide; o < 32; o *= 2) t = gn_merge(t, gn_from(t, o));
    if (l.at == 0 && g < first + groups) {
      a.mean[sample * a.groups + g] = __fdiv_rn(t.y, all);
      a.rstd[sample * a.groups + g] = __frcp_rn(__fsqrt_rn(fmaf(t.z, inv, a.eps)));
    }
  }
}

template <typename T, int N, bool SILU>
__global__ void __launch_bounds__(kGnThreads, 3) gn_forward_cluster_kernel(const GroupNormArgs a, const GnCut c) {
  using P = GnPiece<T, N>;
  constexpr int kPairs = gn_pairs<N>(), kUnroll = N <= 2 ? 8 : 4, kUnrollOut = N <= 2 ? 4 : 2;
  extern __shared__ uint4 s_tile[];
  __shared__ float2 s_sum[kGnThreads], s_group[kGnTileGroups], s_slots[2][kGnClusterMax][kGnTileGroups];
  __shared__ float s_here[kGnTileGroups];
  gn_started(c.cluster);
  const GnPlace<N> at(c);
  const int rank = c.cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = rank * c.part_rows;
  const int rows = max(0, min(c.part_rows, static_cast<int>(a.positions) - first));
  const int tile_bytes = at.tile_pieces * P::kBytes;
  float2 w[kPairs], b[kPairs];
  gn_weights<T, N>(a.weight, a.weight_f32, 1.0f, at, w);
  gn_weights<T, N>(a.bias, a.weight_f32, 0.0f, at, b);
  const float mine = rows > 0 ? __fdividef(1.0f, static_cast<float>(rows) * static_cast<float>(c.per)) : 0.0f;
  const float all = static_cast<float>(a.positions) * static_cast<float>(c.per), inv = 1.0f / all;
  const int group = at.there ? at.group - at.first_group : 0;
  const char* tile = reinterpret_cast<const char*>(s_tile) + (threadIdx.x % c.wide) * P::kBytes;
  const int row_bytes = c.at_once * tile_bytes;
  int turn = 0;
  bool all_started = false;
  for (int64_t sample = blockIdx.x / c.cluster; sample < a.samples; sample += gridDim.x / c.cluster) {
    __syncthreads();                    // the sample before is done with
    gn_fetch<P::kBytes>(reinterpret_cast<char*>(s_tile),
             reinterpret_cast<const char*>(static_cast<const T*>(a.x) + sample * a.x_sample + first * a.x_position) + at.tile0 * P::kBytes,
             rows, tile_bytes, a.x_position * static_cast<int64_t>(sizeof(T)), c.unit);
    gn_fetched();
    gn_all_started(c.cluster, &all_started);
    float2 t = both(0.0f);
    if (at.there) {
      const char* p = tile + at.row0 * tile_bytes;
#pragma unroll kUnroll
      for (int l = at.row0; l < rows; l += c.at_once, p += row_bytes) {
        const P v = *reinterpret_cast<const P*>(p);
        float2 of_row = v.pair(0);
#pragma unroll
        for (int j = 1; j < kPairs; ++j) of_row = add_of<N>(of_row, v.pair(j));
        t = add_of<N>(t, of_row);
      }
    }
    gn_block_sums<N>(c, at, make_float2(t.x + t.y, 0.0f), s_sum, s_group);
    // about this CTA's mean, whose rounding the differences' own sum takes back; the mean comes
    // from the values' sum (the differences of 16-bit values are all rounded the same way)
    const float here = s_group[group].x * mine;
    if (threadIdx.x < at.groups) s_here[threadIdx.x] = s_group[threadIdx.x].x;
    float2 off = both(0.0f);
    t = both(0.0f);
    if (at.there) {
      const char* p = tile + at.row0 * tile_bytes;
#pragma unroll kUnroll
      for (int l = at.row0; l < rows; l += c.at_once, p += row_bytes) {
        const P v = *reinterpret_cast<const P*>(p);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          float2 d = add_of<N>(v.pair(j), both(-here));
          off = add_of<N>(off, d);
          t = fma_of<N>(d, d, t);
        }
      }
    }
    __syncthreads();                    // s_group has been read
    gn_block_sums<N>(c, at, make_float2(off.x + off.y, t.x + t.y), s_sum, s_group);
    if (threadIdx.x < at.groups) {
      const float2 v = s_group[threadIdx.x];
      const float d = v.x * mine;
      s_group[threadIdx.x] = make_float2(s_here[threadIdx.x], gn_spread(fmaf(-d, v.x, v.y)));
    }
    __syncthreads();
    // two sets of slots: a CTA may be a sample ahead of one that still reads
    gn_exchange(c.cluster, rank, at.groups, s_group, s_slots[turn]);
    float3 u = make_float3(0.0f, 0.0f, 0.0f);
    for (int r = 0; r < c.cluster; ++r) {
      const int n = max(0, min(c.part_rows, static_cast<int>(a.positions) - r * c.part_rows));
      const float2 v = s_slots[turn][r][group];
      u = gn_merge(u, make_float3(static_cast<float>(n) * static_cast<float>(c.per), v.x, v.y));
    }
    turn ^= 1;
    const float mean = __fdiv_rn(u.y, all), rstd = __frcp_rn(__fsqrt_rn(fmaf(u.z, inv, a.eps)));
    if (!at.there) continue;
    if (rank == 0 && at.row0 == 0 && at.piece % c.group_pieces == 0) {
      a.mean[sample * a.groups + at.group] = mean;
      a.rstd[sample * a.groups + at.group] = rstd;
    }
    T* y = static_cast<T*>(a.out) + sample * a.out_sample + (first + at.row0) * a.out_position + at.channel();
    const int64_t pace = c.at_once * a.out_position;
    const char* p = tile + at.row0 * tile_bytes;
#pragma unroll kUnrollOut
    for (int l = at.row0; l < rows; l += c.at_once, p += row_bytes, y += pace) {
      P v = *reinterpret_cast<const P*>(p);
#pragma unroll
      for (int j = 0; j < kPairs; ++j)
        v.set(j, activate<T, N, SILU>(fma_of<N>(mul_of<N>(add_of<N>(v.pair(j), both(-mean)), both(rstd)), w[j], b[j])));
      v.store(y);
    }
  }
}

constexpr int kForwardDepth = 16;       // steps on their way, at most 60 KB a CTA

template <typename T, int N, bool SILU>
__global__ void __launch_bounds__(kGnFusedThreads, kGnCtasPerSm) gn_forward_fused_kernel(const GroupNormArgs a, const GnCut c) {
  using Ring = GnRing<T, N, 1, kForwardDepth>;
  using P = GnPiece<T, N>;
  constexpr int kPairs = gn_pairs<N>();
  extern __shared__ uint4 s_ring[];
  // sums and spreads of the threads (or, by lanes, of rows of threads and groups)
  __shared__ float2 s_stat[2][kGnThreads];
  const GnPlace<N> at(c);
  const GnPart part(a, c);
  uint32_t* words = gn_words(a, c, part);
  const int tile_groups = at.groups;
  if (threadIdx.x >= kGnThreads) {
    const GnLanes lanes(tile_groups);
    const int least = part.rows / c.at_once, more = part.rows - least * c.at_once;   // rows of a thread; those that have one more
    const int place = part.part * gn_pitch(a, c) + at.first_group + (c.aligned ? 0 : blockIdx.y);
    for (uint32_t batch = 0; part.sample(batch, c) < a.samples; ++batch) {
      const int64_t sample = part.sample(batch, c);
      float2* stats = gn_stats(a, c, batch, part);
      const float2* s = s_stat[batch % 2];
      gn_wait_filled(batch % 2);
      for (int g0 = 0; g0 < tile_groups; g0 += lanes.wide) {
        const int g = g0 + lanes.slot;
        float3 u = make_float3(0.0f, 0.0f, 0.0f);
        if (g < tile_groups) {
          if (c.by_lanes) {
            for (int r = lanes.at; r < c.at_once; r += lanes.share) {
              const float2 v = s[r * tile_groups + g];
              u = gn_merge(u, make_float3(static_cast<float>((least + (r < more)) * c.per), v.x, v.y));
            }
          } else {
            const int lo = max((at.first_group + g) * c.group_pieces, at.tile0) - at.tile0;
            const int q = min((at.first_group + g + 1) * c.group_pieces, at.tile0 + at.tile_pieces) - at.tile0 - lo;
            for (int e = lanes.at; e < q * c.at_once; e += lanes.share) {
              const int r = e / q;
              const float2 v = s[r * c.wide + lo + e - r * q];
              u = gn_merge(u, make_float3(static_cast<float>((least + (r < more)) * N), v.x, v.y));
            }
          }
        }
        for (int o = lanes.wide; o < 32; o *= 2) u = gn_merge(u, gn_from(u, o));
        if (lanes.at == 0 && g < tile_groups) __stcg(stats + place + g, make_float2(u.y, u.z));
      }
      if (part.sample(batch + 2, c) < a.samples) gn_freed(batch % 2);
      if (gn_arrive(c, words, batch)) {
        if (c.aligned) gn_join(a, c, stats, sample, at.first_group, tile_groups, N);
        else gn_join(a, c, stats, sample, 0, a.groups, N);
        gn_open(words, batch);
      }
    }
    gn_leave(a, c);
    return;
  }
  Ring ring(s_ring, a, c, part, at);
  float2 w[kPairs], b[kPairs];
  gn_weights<T, N>(a.weight, a.weight_f32, 1.0f, at, w);
  gn_weights<T, N>(a.bias, a.weight_f32, 0.0f, at, b);
  uint64_t limit = a.wait_ns;
  for (uint32_t n = 0; n < part.turns; ++n) {
    const GnTurn turn(n);
    const int64_t sample = part.sample(turn.batch, c);
    if (sample >= a.samples) continue;
    if (!turn.result) {
      float3 t = make_float3(0.0f, 0.0f, 0.0f);
      float shift = 0.0f, whole = 0.0f, rest = 0.0f;
      float2 raw = both(0.0f), sum = both(0.0f), square = both(0.0f);
      int run = 0;
      for (int k = 0; k < part.steps; ++k) {
        P p[1];
        ring.get(p);
        if (k >= ring.rows) continue;
        if (run == 0) shift = p[0].pair(0).x;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
          const float2 d = add_of<N>(p[0].pair(j), both(-shift));
          raw = add_of<N>(raw, p[0].pair(j));
          sum = add_of<N>(sum, d);
          square = fma_of<N>(d, d, square);
        }
        if (++run == kRun / N || k == ring.rows - 1) {
          const float count = static_cast<float>(run * N), total = sum.x + sum.y, off = __fdividef(total, count);
          t = gn_merge_means(t, make_float3(count, shift + off, gn_spread(fmaf(-off, total, square.x + square.y))));
          add_exactly(raw.x + raw.y, &whole, &rest);
          run = 0;
          raw = sum = square = both(0.0f);
        }
      }
      t.y = fabsf(whole) < INFINITY ? whole + rest : whole;      // the rest of an infinite sum is no number
      if (c.by_lanes)
        for (int o = 1; o < c.group_pieces; o *= 2) t = gn_merge(t, gn_from(t, o));
      float2* s = s_stat[turn.batch % 2];
      if (turn.batch >= 2) gn_wait_freed(turn.batch % 2);
      if (!c.by_lanes) s[threadIdx.x] = make_float2(t.y, t.z);
      else if (at.there && at.piece % c.group_pieces == 0) s[at.row0 * tile_groups + at.group - at.first_group] = make_float2(t.y, t.z);
      gn_filled(turn.batch % 2);
      continue;
    }
    const bool open = gn_wait_open(a, words, turn.batch, &limit);
    float mean = 0.0f, rstd = 0.0f;
    if (at.there) {
      mean = __ldcg(a.mean + sample * a.groups + at.group);
      rstd = __ldcg(a.rstd + sample * a.groups + at.group);
    }
    T* y = static_cast<T*>(a.out) + sample * a.out_sample + static_cast<int64_t>(part.first + at.row0) * a.out_position + at.channel();
    const int64_t out_pace = c.at_once * a.out_position;
    float2 slope[kPairs], start[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      slope[j] = mul_of<N>(w[j], both(rstd));
      start[j] = fma_of<N>(slope[j], both(-mean), b[j]);
    }
    const int rows = open ? ring.rows : 0;
    for (int k = 0; k < part.steps; ++k) {
      P p[1];
      ring.get(p);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) p[0].set(j, activate<T, N, SILU>(fma_of<N>(p[0].pair(j), slope[j], start[j])));
      if (k < rows) p[0].store(y);
      y += out_pace;
    }
  }
  gn_leave(a, c);
}

template <typename T, int N, bool SILU>
cudaError_t gn_forward(const GroupNormArgs& a, int sms, cudaStream_t s) {
  const GnCut c = gn_cut(a, N, sms);
  const dim3 grid(c.ctas, c.tiles);
  switch (gn_kind(a, c)) {
    case kGnCluster: return gn_cluster_launch(gn_forward_cluster_kernel<T, N, SILU>, gn_cluster_bytes(a, c, N), s, a, c);
    case kGnFused:
      return gn_launch(gn_forward_fused_kernel<T, N, SILU>, grid, kGnFusedThreads, GnRing<T, N, 1, kForwardDepth>::kBytes, s, a, c);
    case kGnLanes: return gn_launch(gn_forward_lanes_kernel<T, N, SILU>, grid, kGnThreads, 0, s, a, c);
    case kGnRow: return gn_launch(gn_forward_small_kernel<T, N, SILU, 1>, grid, kGnThreads, 0, s, a, c);
    default: return gn_launch(gn_forward_small_kernel<T, N, SILU, kSmallForward>, grid, kGnThreads, 0, s, a, c);
  }
}
template <typename T>
cudaError_t gn_forward_type(const GroupNormArgs& a, int sms, cudaStream_t s) {
  constexpr int kWide = 16 / sizeof(T);
  const int n = gn_piece(a, sizeof(T));
  if (n == kWide) return a.silu ? gn_forward<T, kWide, true>(a, sms, s) : gn_forward<T, kWide, false>(a, sms, s);
  if constexpr (sizeof(T) == 2)
    if (n == 2) return a.silu ? gn_forward<T, 2, true>(a, sms, s) : gn_forward<T, 2, false>(a, sms, s);
  return a.silu ? gn_forward<T, 1, true>(a, sms, s) : gn_forward<T, 1, false>(a, sms, s);
}

}  // namespace

template <typename T, int N, bool SILU>
cudaError_t gn_prepare_one() {
  const cudaError_t e = cudaFuncSetAttribute(gn_forward_fused_kernel<T, N, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             GnRing<T, N, 1, kForwardDepth>::kBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(gn_forward_cluster_kernel<T, N, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGnClusterBytes);
}
template <typename T, int N>
cudaError_t gn_prepare_forward() {
  const cudaError_t e = gn_prepare_one<T, N, true>();
  return e == cudaSuccess ? gn_prepare_one<T, N, false>() : e;
}
cudaError_t prepare_group_norm() {
  cudaError_t e = prepare_group_norm_backward();
  if (e == cudaSuccess) e = gn_prepare_forward<float, 4>();
  if (e == cudaSuccess) e = gn_prepare_forward<float, 1>();
  if (e == cudaSuccess) e = gn_prepare_forward<__half, 8>();
  if (e == cudaSuccess) e = gn_prepare_forward<__half, 2>();
  if (e == cudaSuccess) e = gn_prepare_forward<__half, 1>();
  if (e == cudaSuccess) e = gn_prepare_forward<__nv_bfloat16, 8>();
  if (e == cudaSuccess) e = gn_prepare_forward<__nv_bfloat16, 2>();
  if (e == cudaSuccess) e = gn_prepare_forward<__nv_bfloat16, 1>();
  return e;
}

cudaError_t launch_group_norm_forward(adamw_dtype dt, const GroupNormArgs& a, int sms, cudaStream_t s) {
  if (dt == ADAMW_F32) return gn_forward_type<float>(a, sms, s);
  if (dt == ADAMW_F16) return gn_forward_type<__half>(a, sms, s);
  return gn_forward_type<__nv_bfloat16>(a, sms, s);
}

}  // namespace adamw
