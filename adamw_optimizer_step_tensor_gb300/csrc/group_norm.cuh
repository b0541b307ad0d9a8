// group_norm.cuh -- what group norm's forward and backward passes share: pieces of channels,
// the activation, and the order of work of the fused passes.
//
// A thread keeps one piece of channels (16 bytes, 4 bytes or one element: the widest
// that lies on its grid in every tensor and inside one group), so its group's statistics
// are two numbers, and its weights and column sums stay in registers.  A row's pieces
// are cut into tiles of at most 256; a CTA of 256 threads has one tile.
//
// Samples whose tile fits into the registers of a CTA or a part of it (`team`) are read
// once: statistics and result from the registers (the small kernels).  This takes tiles
// of whole groups, and so does the next larger size: samples whose tile fits into the
// shared memory of a cluster (group_norm_cluster.cuh).
//
// Still larger samples are read twice by one launch (the fused kernels), the second time out of
// the L2.  A sample is cut into parts; an item is the statistics of one part or the result
// of one.  A batch of samples has one part for each CTA of a tile, and a CTA takes the same
// part of every batch: the statistics of batch 0, then in turn those of batch j and the
// result of batch j - 1.  The warp that leaves the last statistics of a sample (of a tile of
// it, if tiles are of whole groups) joins them, in the order of parts, and opens it for its
// results; about 5 us that pass while other items run.  An item waits only for items before
// it in that order, and all CTAs are resident (a cooperative launch), so every wait ends;
// each is bounded all the same.
//
// Elements come in by asynchronous copies, each thread's into its own places of a ring in
// shared memory, which run ahead across items: no barrier, no registers, and the copies
// do not pause where an item ends or waits.  A ninth warp takes the threads' statistics
// over, adds them up and does all that concerns other CTAs; the eight go on at once.
//
// 16 x 4096 x 1024 bf16 in 32 groups: forward 66 us, backward 111 (a read and a write of each tensor
// take 40 and 59): instructions bound it, and the part of the second read that the L2 has lost.
#pragma once

#include "async_copy.cuh"
#include "block_ops.h"
#include "group_norm_cut.h"
#include "rows.cuh"

namespace adamw {

namespace {

constexpr int kGnWarps = kGnThreads / 32;
constexpr int kGnFusedThreads = kGnThreads + 32;

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

// Arithmetic on pairs of elements.  A lone element (N = 1) is the first of its pair; the other
// half is 0 and takes no instructions (112 x 3589 x 58 bf16 in 2 groups, whose pieces are single
// elements: forward 125 us with both halves, 118 without).
template <int N>
__device__ __forceinline__ float2 fma_of(float2 x, float2 y, float2 z) {
  if constexpr (N == 1) return make_float2(fmaf(x.x, y.x, z.x), 0.0f);
  else return fma2(x, y, z);
}
template <int N>
__device__ __forceinline__ float2 add_of(float2 x, float2 y) {
  if constexpr (N == 1) return make_float2(x.x + y.x, 0.0f);
  else return add2(x, y);
}
template <int N>
__device__ __forceinline__ float2 mul_of(float2 x, float2 y) {
  if constexpr (N == 1) return make_float2(x.x * y.x, 0.0f);
  else return mul2(x, y);
}

// sigmoid(z).  For 16-bit elements by the approximate exponential and reciprocal: off by
// |z| 2^-24 and a few 2^-23, well below the elements' rounding.  (One reciprocal for two
// elements, 1 / (d d'), took more instructions than it saved: the special function unit
// is not what bounds the pass.)
template <typename T>
__device__ __forceinline__ float sigmoid_of(float z) {
  if constexpr (sizeof(T) == 4) return __fdividef(1.0f, 1.0f + expf(-z));
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(e + 1.0f));
  return s;
}
template <typename T, int N>
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  if constexpr (N == 1) return make_float2(sigmoid_of<T>(z.x), 0.0f);
  if constexpr (sizeof(T) == 4) return make_float2(sigmoid_of<T>(z.x), sigmoid_of<T>(z.y));
  const float2 t = mul2(z, both(-1.4426950408889634f));
  float2 e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  const float2 d = add2(e, both(1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(d.y));
  return s;
}
// The activation's value at z, and dy times its slope there.
template <typename T, int N, bool SILU>
__device__ __forceinline__ float2 activate(float2 z) {
  if constexpr (!SILU) return z;
  return mul_of<N>(z, sigmoid2<T, N>(z));
}
template <typename T, int N, bool SILU>
__device__ __forceinline__ float2 through(float2 dy, float2 z) {
  if constexpr (!SILU) return dy;
  const float2 s = sigmoid2<T, N>(z);
  const float2 u = fma_of<N>(s, both(-1.0f), both(1.0f));   // 1 - s
  return mul_of<N>(mul_of<N>(dy, s), fma_of<N>(z, u, both(1.0f)));
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

// What a CTA does: item n of batches 0, 1, ... is the statistics of batch 0, then in turn
// those of batch j (n = 2 j - 1) and the results of batch j (n = 2 j + 2).
struct GnTurn {
  bool result;
  uint32_t batch;
  __device__ __forceinline__ explicit GnTurn(uint32_t n)
      : result(n > 0 && n % 2 == 0), batch(n == 0 ? 0 : (n % 2 == 0 ? n / 2 - 1 : (n + 1) / 2)) {}
};
// This CTA's part of its sample of each batch.
struct GnPart {
  uint32_t turns;        // items, the missing ones of the last batch among them
  int64_t sample0;       // its sample of batch 0
  int part, first, rows; // rows: of the part
  int steps;             // rows of a thread, at most
  __device__ __forceinline__ GnPart(const GroupNormArgs& a, const GnCut& c) {
    turns = 2 * static_cast<uint32_t>((a.samples + c.batch - 1) / c.batch) + 1;
    sample0 = blockIdx.x / c.parts;
    part = blockIdx.x % c.parts;
    first = part * c.part_rows;
    rows = min(c.part_rows, static_cast<int>(a.positions) - first);
    steps = (rows + c.at_once - 1) / c.at_once;
  }
  __device__ __forceinline__ int64_t sample(uint32_t batch, const GnCut& c) const {
    return sample0 + static_cast<int64_t>(batch) * c.batch;
  }
};
// Rows of a part that row0's threads have.
__device__ __forceinline__ int gn_rows(int rows, int row0, int at_once) {
  return rows > row0 ? (rows - row0 + at_once - 1) / at_once : 0;
}

// The two buffers in which the eight warps leave their statistics: filled (the eight arrive,
// the ninth waits) and free again (the ninth arrives, the eight wait, from the third on).
__device__ __forceinline__ void gn_filled(uint32_t buffer) {
  asm volatile("bar.arrive %0, %1;" ::"r"(1 + buffer), "n"(kGnFusedThreads) : "memory");
}
__device__ __forceinline__ void gn_wait_filled(uint32_t buffer) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + buffer), "n"(kGnFusedThreads) : "memory");
}
__device__ __forceinline__ void gn_freed(uint32_t buffer) {
  asm volatile("bar.arrive %0, %1;" ::"r"(3 + buffer), "n"(kGnFusedThreads) : "memory");
}
__device__ __forceinline__ void gn_wait_freed(uint32_t buffer) {
  asm volatile("bar.sync %0, %1;" ::"r"(3 + buffer), "n"(kGnFusedThreads) : "memory");
}

// Copies of a thread's pieces of `TENSORS` tensors, `DEPTH` - 1 steps ahead of its work: the
// place that is filled is the one whose piece was worked on a step ago.  A thread without a
// row for a step gets zeros, without a read.
template <typename T, int N, int TENSORS, int DEPTH>
struct GnRing {
  using P = GnPiece<T, N>;
  static constexpr int kTensor = kGnThreads * P::kBytes;      // bytes of one tensor's places
  static constexpr int kBytes = DEPTH * TENSORS * kTensor;
  const GroupNormArgs& a;
  const GnCut& c;
  const GnPart& part;
  uint32_t base, fill, take = 0;
  const char *x0, *dy0;  // of this thread's first row in sample 0 of the tensor
  const char *x, *dy;
  int64_t pace, dy_pace; // bytes
  uint32_t n = 0;
  int step = 0, steps;   // of the item whose copies run
  int rows;              // of this thread

  __device__ __forceinline__ GnRing(void* smem, const GroupNormArgs& a_, const GnCut& c_, const GnPart& part_,
                                    const GnPlace<N>& at)
      : a(a_), c(c_), part(part_), base(smem_u32(smem) + threadIdx.x * P::kBytes) {
    constexpr int kSize = sizeof(T);
    rows = at.there ? gn_rows(part.rows, at.row0, c.at_once) : 0;
    steps = part.steps;
    const int64_t row = part.first + at.row0;
    x0 = static_cast<const char*>(a.x) + (row * a.x_position + at.channel()) * kSize;
    pace = c.at_once * a.x_position * kSize;
    if (TENSORS == 2) {
      dy0 = static_cast<const char*>(a.dy) + (row * a.dy_position + at.channel()) * kSize;
      dy_pace = c.at_once * a.dy_position * kSize;
    }
    enter();
    fill = 0;
#pragma unroll 1
    for (int d = 0; d < DEPTH - 1; ++d) {
      put();
      fill += TENSORS * kTensor;
    }
  }
  // To the first item from n on that there is; behind the last one nothing is copied.
  __device__ __forceinline__ void enter() {
    step = 0;
    for (; n < part.turns; ++n) {
      const int64_t sample = part.sample(GnTurn(n).batch, c);
      if (sample < a.samples) {
        x = x0 + sample * a.x_sample * static_cast<int64_t>(sizeof(T));
        if (TENSORS == 2) dy = dy0 + sample * a.dy_sample * static_cast<int64_t>(sizeof(T));
        return;
      }
    }
    steps = 0x7FFFFFFF;
    step = 0x40000000;     // no thread has as many rows, and the end is far
  }
  __device__ __forceinline__ static void copy(uint32_t to, const char* from, bool there) {
    if constexpr (P::kBytes == 2) {                          // too few bytes for an asynchronous copy
      const uint16_t v = there ? *reinterpret_cast<const uint16_t*>(from) : uint16_t{0};
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(v) : "memory");
    } else if constexpr (P::kBytes == 4) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
    } else {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
    }
  }
  __device__ __forceinline__ void put() {
    const bool there = step < rows;
    copy(base + fill, x, there);
    x += pace;
    if (TENSORS == 2) {
      copy(base + fill + kTensor, dy, there);
      dy += dy_pace;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++step == steps) {
      ++n;
      enter();
    }
  }
  __device__ __forceinline__ static P at(uint32_t place) {
    P p;
    if constexpr (P::kBytes == 16)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(p.v.x), "=r"(p.v.y), "=r"(p.v.z), "=r"(p.v.w) : "r"(place) : "memory");
    else if constexpr (P::kBytes == 4)
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(p.v) : "r"(place) : "memory");
    else
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(p.v) : "r"(place) : "memory");
    return p;
  }
  // The next step's pieces; then the copies go one step further.
  __device__ __forceinline__ void get(P (&p)[TENSORS]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
#pragma unroll
    for (int t = 0; t < TENSORS; ++t) p[t] = at(base + take + t * kTensor);
    put();
    fill = take;
    take = take == kBytes - TENSORS * kTensor ? 0 : take + TENSORS * kTensor;
  }
};

// Partial statistics of a part: group g, or where tiles may begin inside a group g + t for
// tile t (each such tile adds one, so the places are distinct).
__device__ __forceinline__ int gn_pitch(const GroupNormArgs& a, const GnCut& c) { return a.groups + (c.aligned ? 0 : c.tiles); }
__device__ __forceinline__ float2* gn_stats(const GroupNormArgs& a, const GnCut& c, uint32_t batch, const GnPart& part) {
  return reinterpret_cast<float2*>(a.stats) +
         (static_cast<int64_t>(batch % kGnKept) * c.batch + part.sample0) * c.parts * gn_pitch(a, c);
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

// Words of the CTAs that share a sample (or a tile of one) of each batch: the number that
// left their statistics, for each of the batches kept, and the batches that are open.  They
// only grow; the last CTA to leave the kernel clears them.
__device__ __forceinline__ uint32_t* gn_words(const GroupNormArgs& a, const GnCut& c, const GnPart& part) {
  return a.words + kGnWords * (c.aligned ? part.sample0 * c.tiles + blockIdx.y : part.sample0);
}

// Called by a warp that has written an item's statistics: true if they are the sample's last.
__device__ __forceinline__ bool gn_arrive(const GnCut& c, uint32_t* words, uint32_t batch) {
  __syncwarp();
  bool last = false;
  if ((threadIdx.x & 31) == 0) {
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(words + batch % kGnKept) : "memory");
    const uint32_t all = static_cast<uint32_t>(c.parts) * (c.aligned ? 1 : c.tiles);
    last = before + 1 == all * (batch / kGnKept + 1);
  }
  last = __shfl_sync(kFull, static_cast<int>(last), 0) != 0;
  __syncwarp();          // what the first lane has acquired the others may read: a shuffle orders no memory
  return last;
}
__device__ __forceinline__ void gn_open(uint32_t* words, uint32_t batch) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0)
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(words + kGnKept), "r"(batch + 1) : "memory");
}
// A warp waits until its sample of the batch is open: false when the wait gave up.  One that
// gave up does not wait again.
__device__ __forceinline__ bool gn_wait_open(const GroupNormArgs& a, const uint32_t* words, uint32_t batch, uint64_t* limit_ns) {
  bool open = true;
  if ((threadIdx.x & 31) == 0) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(words + kGnKept) : "memory");
    if (v <= batch) {
      const uint64_t t0 = global_ns();
      while (true) {
        if (global_ns() - t0 >= *limit_ns) {
          atomicOr(a.fault, 1u);
          open = false;
          break;
        }
        __nanosleep(50);
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(words + kGnKept) : "memory");
        if (v > batch) break;
      }
    }
  }
  open = __shfl_sync(kFull, static_cast<int>(open), 0) != 0;
  __syncwarp();          // as in gn_arrive
  if (!open) *limit_ns = 0;
  return open;
}
// Every CTA leaves by here; the last one clears the words.
__device__ __forceinline__ void gn_leave(const GroupNormArgs& a, const GnCut& c) {
  __syncthreads();
  bool last = false;
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y - 1;
    __threadfence();
  }
  if (!__syncthreads_or(last)) return;
  for (int i = threadIdx.x; i < kGnWords * c.batch * (c.aligned ? c.tiles : 1); i += blockDim.x) a.words[i] = 0;
  if (threadIdx.x == 0) *a.ticket = 0;
}

// ---------------------------------------------------------------- small kernels

// The sums of two numbers over each group's threads of one sample (one team), the same in all
// of them.  s, s_group: kGnThreads pairs; used by all threads of the CTA at the same time.
__device__ __forceinline__ float2 gn_team_sums(float2 x, const GnCut& c, float2* s, float2* s_group) {
  if (c.by_lanes && c.team_rows == 1) {
    for (int o = 1; o < c.group_pieces; o <<= 1)
      x = add2(x, make_float2(__shfl_xor_sync(kFull, x.x, o), __shfl_xor_sync(kFull, x.y, o)));
    return x;
  }
  const int row = threadIdx.x / c.wide, p = threadIdx.x - row * c.wide;
  const int tile_groups = c.wide / c.group_pieces;
  __syncthreads();
  s[threadIdx.x] = x;
  __syncthreads();
  const int all = c.teams * tile_groups, q = c.group_pieces, entries = c.team_rows * q;
  // entry e of a group: piece e % q of row e / q.  A thread adds up a few entries, a warp many.
  if (entries <= 8 || all >= kGnThreads / 2) {
    for (int g = threadIdx.x; g < all; g += kGnThreads) {
      const int team = g / tile_groups, first = team * c.team_rows * c.wide + (g - team * tile_groups) * q;
      float2 t = both(0.0f);
      for (int r = 0; r < c.team_rows; ++r)
        for (int k = 0; k < q; ++k) t = add2(t, s[first + r * c.wide + k]);
      s_group[g] = t;
    }
  } else {
    const int lane = threadIdx.x & 31;
    for (int g = threadIdx.x / 32; g < all; g += kGnWarps) {
      const int team = g / tile_groups, first = team * c.team_rows * c.wide + (g - team * tile_groups) * q;
      float2 t = both(0.0f);
      for (int e = lane; e < entries; e += 32) {
        const int r = e / q;
        t = add2(t, s[first + r * (c.wide - q) + e]);
      }
      t = make_float2(warp_total(t.x), warp_total(t.y));
      if (lane == 0) s_group[g] = t;
    }
  }
  __syncthreads();
  const int team = row / c.team_rows;
  return team < c.teams ? s_group[team * tile_groups + p / q] : both(0.0f);
}

}  // namespace

template <typename K>
cudaError_t gn_launch(K kernel, dim3 grid, int threads, int smem, cudaStream_t s, const GroupNormArgs& a, const GnCut& c) {
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t l{};
  l.gridDim = grid;
  l.blockDim = dim3(threads);
  l.dynamicSmemBytes = smem;
  l.stream = s;
  l.attrs = &attr;
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  l.numAttrs = threads == kGnFusedThreads ? 1 : 0;
  return cudaLaunchKernelEx(&l, kernel, a, c);
}

}  // namespace adamw
