// group_norm_cluster.cuh -- group norm of samples that fit the shared memory of a cluster of
// CTAs: what its two passes share.
//
// A cluster of 1 to 8 CTAs takes one tile of whole groups of one sample at a time, each CTA
// its share of the positions.  The elements are copied to shared memory once, by whatever
// pieces lie on their grid in memory; statistics and results are computed there by pieces of
// one group.  Sums go from threads to the CTA and from there to every CTA of the cluster,
// one exchange per sample; before the first one all CTAs meet, since a CTA that has not started
// yet has no shared memory to write to.  Several CTAs share an SM, so that one copies while others compute.
#pragma once

#include "cluster.cuh"
#include "group_norm.cuh"

namespace adamw {
namespace {

// Starts the copies of this CTA's rows of a tile: `rows` rows of tile_bytes bytes, dense in
// shared memory.  from: the first row's first byte.  Asynchronous copies are of 4 bytes at least;
// single 16-bit elements that lie on no such grid (BYTES, of a piece, and unit are 2) come by loads,
// kAhead of them on their way (112 x 3589 x 58 bf16 in 2 groups: forward 125 us one by one, 69 with
// 16; backward 633 and 189; with 32 the registers do not suffice).
template <int BYTES>
__device__ __forceinline__ void gn_fetch(char* to, const char* from, int rows, int tile_bytes, int64_t row_bytes, int unit) {
  const int per_row = tile_bytes / unit;
  int row = threadIdx.x / per_row, col = threadIdx.x - row * per_row;
  const int row_step = kGnThreads / per_row, col_step = kGnThreads - row_step * per_row;
  const auto next = [&] {
    row += row_step;
    col += col_step;
    if (col >= per_row) {
      col -= per_row;
      ++row;
    }
  };
  if constexpr (BYTES == 2) {
    constexpr int kAhead = 16;
    while (unit == 2 && row < rows) {
      uint16_t v[kAhead];
      int at[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        at[u] = row < rows ? row * tile_bytes + col * 2 : -1;
        if (row < rows) v[u] = __ldg(reinterpret_cast<const uint16_t*>(from + row * row_bytes + col * 2));
        next();
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (at[u] >= 0) *reinterpret_cast<uint16_t*>(to + at[u]) = v[u];
    }
  }
  while (row < rows) {
    const char* src = from + row * row_bytes + col * unit;
    char* dst = to + row * tile_bytes + col * unit;
    if (unit == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    next();
  }
}
__device__ __forceinline__ void gn_fetched() {
  asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
  __syncthreads();
}

// Sums of pairs over the CTA's threads of each of the tile's groups, in s_group; called by
// all threads, with a barrier before it since s was last read.
template <int N>
__device__ __forceinline__ void gn_block_sums(const GnCut& c, const GnPlace<N>& at, float2 v, float2* s, float2* s_group) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  if (c.by_lanes) {
    for (int o = 1; o < c.group_pieces; o *= 2) {
      v.x += __shfl_xor_sync(kFull, v.x, o);
      v.y += __shfl_xor_sync(kFull, v.y, o);
    }
    if (at.there && at.piece % c.group_pieces == 0) s[at.row0 * at.groups + at.group - at.first_group] = v;
  } else {
    s[threadIdx.x] = v;
  }
  __syncthreads();
  const int q = c.by_lanes ? 1 : c.group_pieces, pitch = c.by_lanes ? at.groups : c.wide, n = q * c.at_once;
  if (n >= 8 || at.groups < 32) {
    for (int g = warp; g < at.groups; g += kGnWarps) {
      float2 t = both(0.0f);
      for (int e = lane; e < n; e += 32) {
        const int r = e / q;
        t = add2(t, s[r * pitch + g * q + e - r * q]);
      }
      t = make_float2(warp_total(t.x), warp_total(t.y));
      if (lane == 0) s_group[g] = t;
    }
  } else {
    for (int g = threadIdx.x; g < at.groups; g += kGnThreads) {
      float2 t = both(0.0f);
      for (int e = 0; e < n; ++e) t = add2(t, s[e / q * pitch + g * q + e % q]);
      s_group[g] = t;
    }
  }
  __syncthreads();
}

// Says that this CTA has started, and waits until all of the cluster have: the one on entry,
// the other once, before the first exchange, when the first sample's copies have hidden it.
__device__ __forceinline__ void gn_started(int size) {
  if (size > 1) cluster_arrive_all();
}
__device__ __forceinline__ void gn_all_started(int size, bool* known) {
  if (size > 1 && !*known) cluster_wait_all();
  *known = true;
}
// Hands this CTA's pairs per group to every CTA of the cluster: slots[rank][group].
__device__ __forceinline__ void gn_exchange(int size, int rank, int groups, const float2* mine, float2 (*slots)[kGnTileGroups]) {
  for (int i = threadIdx.x; i < groups * size; i += kGnThreads) {
    const int g = i / size, r = i - g * size;
    const float2 v = mine[g];
    if (size == 1) slots[0][g] = v;
    else cluster_store2(cluster_map(&slots[rank][g], r), v.x, v.y);
  }
  if (size == 1) __syncthreads();
  else cluster_sync();
}

}  // namespace

template <typename K>
cudaError_t gn_cluster_launch(K kernel, int smem, cudaStream_t s, const GroupNormArgs& a, const GnCut& c) {
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t l{};
  l.gridDim = dim3(c.ctas, c.tiles);
  l.blockDim = dim3(kGnThreads);
  l.dynamicSmemBytes = smem;
  l.stream = s;
  l.attrs = &attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = c.cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  l.numAttrs = c.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&l, kernel, a, c);
}

}  // namespace adamw
