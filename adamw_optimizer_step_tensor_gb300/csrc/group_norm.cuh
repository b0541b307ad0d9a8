// group_norm.cuh -- what group norm's forward and backward passes share: how a call is
// cut up, pieces of channels, the activation, and the order of work of the fused passes.
//
// A thread keeps one piece of channels (16 bytes, 4 bytes or one element: the widest
// that lies on its grid in every tensor and inside one group), so its group's statistics
// are two numbers, and its weights and column sums stay in registers.  A row's pieces
// are cut into tiles of at most 256; a CTA of 256 threads has one tile.
//
// Samples whose tile fits into the registers of a CTA or a part of it (`team`) are read
// once: statistics and result from the registers (the small kernels).  This takes tiles
// of whole groups.
//
// Larger samples are read twice by one launch (the fused kernels).  A sample is cut into
// parts; an item is the statistics of one part or the result of one.  CTAs take items in
// one order: the statistics of a batch of samples, then the results of the batch before
// it, whose elements the L2 still holds.  Tiles are narrow here (256 bytes of whole groups,
// if that suits), so that a tile of a sample has few parts: the warp that leaves the last
// statistics of one joins them, in the order of parts, and opens it for its results.  What
// that takes (about 5 us) has to pass while other items run, or every CTA waits for it.
// Only one warp of a CTA does it: the others go on to the next item.  An item waits only
// for items before it in that order, and all CTAs are resident (a cooperative launch), so
// every wait ends; each is bounded all the same.
#pragma once

#include "async_copy.cuh"
#include "block_ops.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr int kGnThreads = 256;
constexpr int kGnWarps = kGnThreads / 32;

// How a call is cut up.
struct GnCut {
  int32_t pieces, wide, tiles;   // of a row; of a tile; tiles of a row
  int32_t at_once;               // rows a CTA takes at once
  int32_t per;                   // channels of a group
  int32_t group_pieces;          // pieces of a group
  int32_t by_lanes;              // a group's pieces are a power of two of neighbouring lanes
  // small kernels
  int32_t team_rows;             // rows of threads per sample
  int32_t teams;                 // samples a CTA takes at once
  // fused kernels
  int32_t aligned;               // tiles are of whole groups: each of a sample's is open by itself
  int32_t parts;                 // of a sample
  int32_t batch;                 // samples of a batch
  int32_t part_rows;
  int32_t ctas;                  // per tile
};

template <typename T, int N>
struct GnPiece {
  static constexpr int kBytes = N * static_cast<int>(sizeof(T));
  using Word = typename std::conditional<
      kBytes == 16, uint4,
      typename std::conditional<kBytes == 4, uint32_t, uint16_t>::type>::type;
  Word v;
  __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const Word*>(p); }
  // for the last time
  __device__ __forceinline__ void load_last(const T* p) { v = __ldcs(reinterpret_cast<const Word*>(p)); }
  __device__ __forceinline__ void store(T* p) const { __stcs(reinterpret_cast<Word*>(p), v); }
  __device__ __forceinline__ uint32_t word(int i) const {
    if constexpr (kBytes == 16) return reinterpret_cast<const uint32_t*>(&v)[i];
    else return v;
  }
  // Elements 2 i and 2 i + 1 (0 behind a lone one).
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (sizeof(T) == 4) {
      if constexpr (N == 1) return make_float2(__uint_as_float(v), 0.0f);
      else return make_float2(__uint_as_float(word(2 * i)), __uint_as_float(word(2 * i + 1)));
    } else if constexpr (N == 1) {
      return make_float2(to_f32(*reinterpret_cast<const T*>(&v)), 0.0f);
    } else {
      return unpack_pair<T>(word(i));
    }
  }
  __device__ __forceinline__ void set(int i, float2 f) {
    if constexpr (N == 1) {
      *reinterpret_cast<T*>(&v) = from_f32<T>(f.x);
    } else if constexpr (sizeof(T) == 4) {
      reinterpret_cast<uint32_t*>(&v)[2 * i] = __float_as_uint(f.x);
      reinterpret_cast<uint32_t*>(&v)[2 * i + 1] = __float_as_uint(f.y);
    } else {
      reinterpret_cast<uint32_t*>(&v)[i] = pack_pair<T>(f);
    }
  }
};
template <int N>
__host__ __device__ constexpr int gn_pairs() { return (N + 1) / 2; }

__device__ __forceinline__ float warp_total(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

// sigmoid(z).  For 16-bit elements two share one reciprocal, 1 / (d d'), since the special
// function unit would bound the pass: three operations there instead of four.  Below
// -43 the sigmoid counts as that of -43 (2^-62), which keeps d d' in range.
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  if constexpr (sizeof(T) == 4) {
    return make_float2(__fdividef(1.0f, 1.0f + expf(-z.x)), __fdividef(1.0f, 1.0f + expf(-z.y)));
  } else {
    const float2 t = mul2(make_float2(fmaxf(z.x, -43.0f), fmaxf(z.y, -43.0f)), both(-1.4426950408889634f));
    float2 e;
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    const float2 d = add2(e, both(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d.x * d.y));
    return mul2(both(r), make_float2(d.y, d.x));
  }
}
// The activation's value at z, and dy times its slope there.
template <typename T, bool SILU>
__device__ __forceinline__ float2 activate(float2 z) {
  if constexpr (!SILU) return z;
  return mul2(z, sigmoid2<T>(z));
}
template <typename T, bool SILU>
__device__ __forceinline__ float2 through(float2 dy, float2 z) {
  if constexpr (!SILU) return dy;
  const float2 s = sigmoid2<T>(z);
  const float2 zs = mul2(z, s);                       // s (1 + z (1 - s)) = s + z s - s z s
  return mul2(dy, fma2(mul2(s, both(-1.0f)), zs, add2(s, zs)));
}

// This thread's place.
template <int N>
struct GnPlace {
  int piece;             // of the row
  int row0;              // its row of threads
  int group;
  bool there;
  int tile0, tile_pieces;
  int first_group, groups;   // that the tile touches
  __device__ __forceinline__ GnPlace(const GnCut& c) {
    tile0 = blockIdx.y * c.wide;
    tile_pieces = min(c.wide, c.pieces - tile0);
    row0 = threadIdx.x / c.wide;
    const int p = threadIdx.x - row0 * c.wide;
    piece = tile0 + p;
    there = row0 < c.at_once && p < tile_pieces;
    group = piece / c.group_pieces;
    first_group = tile0 / c.group_pieces;
    groups = (tile0 + tile_pieces - 1) / c.group_pieces - first_group + 1;
  }
  __device__ __forceinline__ int channel() const { return piece * N; }
};

// The weights (`one`: of the weight) of this thread's channels.
template <typename T, int N>
__device__ __forceinline__ void gn_weights(const void* p, bool f32, float one, const GnPlace<N>& at,
                                           float2 (&w)[gn_pairs<N>()]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float v = one;
    if (p != nullptr && at.there)
      v = f32 ? static_cast<const float*>(p)[at.channel() + i] : to_f32(static_cast<const T*>(p)[at.channel() + i]);
    if (i % 2 == 0) w[i / 2].x = v;
    else w[i / 2].y = v;
  }
  if constexpr (N == 1) w[0].y = 0.0f;
}

// ---------------------------------------------------------------- fused kernels

struct GnItem {
  bool result;           // the result of a part, else its statistics
  int64_t sample;
  int part, first, rows; // rows: of the part
};
// Units of batch x parts items: the statistics of batch 0, then in turn those of batch
// j and the results of batch j - 1.
__device__ __forceinline__ int64_t gn_items(const GroupNormArgs& a, const GnCut& c) {
  const int64_t batches = (a.samples + c.batch - 1) / c.batch;
  return (2 * batches + 1) * c.batch * c.parts;
}
__device__ __forceinline__ bool gn_item(uint32_t unit, uint32_t rest, const GroupNormArgs& a, const GnCut& c, GnItem* it) {
  it->result = unit > 0 && unit % 2 == 0;
  const uint32_t batch = it->result ? unit / 2 - 1 : (unit + 1) / 2;
  const uint32_t within = rest / static_cast<uint32_t>(c.parts);
  it->sample = static_cast<int64_t>(batch) * c.batch + within;
  it->part = static_cast<int>(rest - within * c.parts);
  it->first = it->part * c.part_rows;
  it->rows = min(c.part_rows, static_cast<int>(a.positions) - it->first);
  return it->sample < a.samples;
}
// Rows of a part that row0's threads have.
__device__ __forceinline__ int gn_rows(int rows, int row0, int at_once) {
  return rows > row0 ? (rows - row0 + at_once - 1) / at_once : 0;
}

// Partial statistics of a part: group g, or where tiles may begin inside a group g + t for
// tile t (each such tile adds one, so the places are distinct).
__device__ __forceinline__ int gn_pitch(const GroupNormArgs& a, const GnCut& c) { return a.groups + (c.aligned ? 0 : c.tiles); }
__device__ __forceinline__ float2* gn_stats(const GroupNormArgs& a, const GnCut& c, int64_t sample, int part) {
  return reinterpret_cast<float2*>(a.stats) + (sample * c.parts + part) * gn_pitch(a, c);
}

// Lanes of a warp that joins entries of several groups: `wide` groups side by side, and
// `share` lanes for each.
struct GnLanes {
  int wide, share, slot, at;
  __device__ __forceinline__ explicit GnLanes(int groups) {
    const int lane = threadIdx.x & 31;
    wide = 1;
    while (wide < groups && wide < 32) wide *= 2;
    share = 32 / wide;
    slot = lane % wide;
    at = lane / wide;
  }
};

// Words of a sample, or of a tile of one: items that left their statistics, and whether it
// is open.  All are 0 between calls: the last CTA to leave the kernel clears them.
__device__ __forceinline__ uint32_t* gn_words(const GroupNormArgs& a, const GnCut& c, int64_t sample) {
  return a.words + 2 * (c.aligned ? sample * c.tiles + blockIdx.y : sample);
}

// Called by a warp that has written an item's statistics: true if they are the sample's last.
__device__ __forceinline__ bool gn_arrive(const GroupNormArgs& a, const GnCut& c, int64_t sample) {
  __syncwarp();
  bool last = false;
  if ((threadIdx.x & 31) == 0) {
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(gn_words(a, c, sample)) : "memory");
    last = before == static_cast<uint32_t>(c.parts) * (c.aligned ? 1 : c.tiles) - 1;
  }
  return __shfl_sync(kFull, static_cast<int>(last), 0) != 0;
}
__device__ __forceinline__ void gn_open(const GroupNormArgs& a, const GnCut& c, int64_t sample) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(gn_words(a, c, sample) + 1), "r"(1u) : "memory");
  }
}
// A warp waits until the sample is open: false when the wait gave up.  One that gave up
// does not wait again.
__device__ __forceinline__ bool gn_wait_open(const GroupNormArgs& a, const GnCut& c, int64_t sample, uint64_t* limit_ns) {
  bool open = true;
  if ((threadIdx.x & 31) == 0) {
    const uint32_t* word = gn_words(a, c, sample) + 1;
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
    if (v == 0) {
      const uint64_t t0 = global_ns();
      while (true) {
        if (global_ns() - t0 >= *limit_ns) {
          atomicOr(a.fault, 1u);
          open = false;
          break;
        }
        __nanosleep(50);
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
        if (v != 0) break;
      }
    }
  }
  open = __shfl_sync(kFull, static_cast<int>(open), 0) != 0;
  if (!open) *limit_ns = 0;
  return open;
}
// Every CTA leaves by here; the last one clears the samples' words.
__device__ __forceinline__ void gn_leave(const GroupNormArgs& a, const GnCut& c) {
  __syncthreads();
  bool last = false;
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y - 1;
  }
  if (!__syncthreads_or(last)) return;
  const int64_t words = 2 * a.samples * (c.aligned ? c.tiles : 1);
  for (int64_t i = threadIdx.x; i < words; i += kGnThreads) a.words[i] = 0;
  if (threadIdx.x == 0) *a.ticket = 0;
}

// ---------------------------------------------------------------- small kernels

// The sum over each group's threads of one sample (one team), the same in all of them.
// s: kGnThreads floats; used by all threads of the CTA at the same time.
__device__ __forceinline__ float gn_team_sum(float x, const GnCut& c, float* s, float* s_group) {
  if (c.by_lanes && c.team_rows == 1) {
    for (int o = 1; o < c.group_pieces; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
  }
  const int row = threadIdx.x / c.wide, p = threadIdx.x - row * c.wide;
  const int tile_groups = c.wide / c.group_pieces;
  __syncthreads();
  s[threadIdx.x] = x;
  __syncthreads();
  const int all = c.teams * tile_groups, entries = c.team_rows * c.group_pieces;
  if (entries <= 16 || all >= kGnThreads / 2) {
    for (int g = threadIdx.x; g < all; g += kGnThreads) {
      const int team = g / tile_groups, q = g - team * tile_groups;
      float t = 0.0f;
      for (int r = 0; r < c.team_rows; ++r)
        for (int k = 0; k < c.group_pieces; ++k)
          t += s[(team * c.team_rows + r) * c.wide + q * c.group_pieces + k];
      s_group[g] = t;
    }
  } else {
    const int lane = threadIdx.x & 31;
    for (int g = threadIdx.x / 32; g < all; g += kGnWarps) {
      const int team = g / tile_groups, q = g - team * tile_groups;
      float t = 0.0f;
      for (int r = 0; r < c.team_rows; ++r)
        for (int k = lane; k < c.group_pieces; k += 32)
          t += s[(team * c.team_rows + r) * c.wide + q * c.group_pieces + k];
      t = warp_total(t);
      if (lane == 0) s_group[g] = t;
    }
  }
  __syncthreads();
  const int team = row / c.team_rows;
  return team < c.teams ? s_group[team * tile_groups + p / c.group_pieces] : 0.0f;
}

}  // namespace

// Cuts a call up (group_norm.cu).  `most`: pieces per thread of the small kernels; 0 rows
// of threads (team_rows) where the fused ones take it.
GnCut gn_cut(const GroupNormArgs& a, int piece, int most, int sms);
// The widest piece of the call, in elements of `size` bytes.
int gn_piece(const GroupNormArgs& a, int size);
constexpr int kGnCtasPerSm = 2;

template <typename K>
cudaError_t gn_launch(K kernel, dim3 grid, bool cooperative, cudaStream_t s, const GroupNormArgs& a, const GnCut& c) {
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t l{};
  l.gridDim = grid;
  l.blockDim = dim3(kGnThreads);
  l.stream = s;
  l.attrs = &attr;
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  l.numAttrs = cooperative ? 1 : 0;
  return cudaLaunchKernelEx(&l, kernel, a, c);
}

}  // namespace adamw
