// router.cu -- routing of tokens to experts: scores, groups, the top_k choice and its
// weights, every assignment's place when all are ordered by expert, the gradient of
// the logits, and the balance step of the bias.
//
// One warp per token; lane l holds the logits of experts l V .. l V + V - 1.  The choice
// is top_k rounds of two warp-wide reductions: the largest key as an ordered integer,
// then the lowest expert that has it.  Where no bias takes part the order of the scores
// is that of the logits, and no score is computed for it.
//
// With a bias the keys are score + bias in float32, which are off by a few units of
// their last bits.  A choice in which any two keys that matter lie closer than that
// (about one token in a thousand) is made again from 64-bit scores, so that the experts
// are those of the definition and not of a rounding.
#include "block_ops.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr int kRouteWarps = 16;
constexpr int kRouteThreads = 32 * kRouteWarps;
constexpr int kBackWarps = 8;

// Floats as integers of the same order; 0 is below all of them and means "not there".
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);          // -0 and 0 are one value
  return (b & 0x80000000u) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) != 0 ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + expf(-z)); }

// Lane l's V logits, -inf behind the last expert.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int experts, bool vec, float (&z)[V]) {
  const int lane = threadIdx.x & 31;
  constexpr int kBytes = V * static_cast<int>(sizeof(T));
  if constexpr (kBytes >= 4) {
    if (vec) {                          // 32 V experts, rows on the grid of a lane's bytes
      constexpr int kWords = kBytes / 4;
      uint32_t w[kWords];
      const T* p = row + lane * V;
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p) + i);
          w[4 * i] = q.x;
          w[4 * i + 1] = q.y;
          w[4 * i + 2] = q.z;
          w[4 * i + 3] = q.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __ldcs(reinterpret_cast<const uint32_t*>(p) + i);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (sizeof(T) == 4) {
          z[i] = __uint_as_float(w[i]);
        } else {
          const float2 f = unpack_pair<T>(w[i / 2]);
          z[i] = i % 2 == 0 ? f.x : f.y;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    z[i] = e < experts ? to_f32(row[e]) : -INFINITY;
  }
}

// The weight of lane j's chosen logit z before `scale`; `row_top` and `row_sum` are the
// softmax's largest logit and sum over the whole row (used without renormalisation).
__device__ __forceinline__ float weight_of(float z, bool chosen, const adamw_router& r,
                                           float row_top, float row_sum) {
  if (r.renormalise) {
    // Only ratios count, so small scores are taken relative to the largest chosen one:
    // below a logit of -30 the sigmoid is e^z to the last bit.
    const float top = warp_max(chosen ? z : -INFINITY);
    const bool ratio = r.score == ADAMW_SCORE_SOFTMAX || top < -30.0f;
    const float s = chosen ? (ratio ? expf(z - top) : sigmoid(z)) : 0.0f;
    const float total = warp_sum(s);
    return chosen ? __fdiv_rn(s, total) : 0.0f;
  }
  if (!chosen) return 0.0f;
  return r.score == ADAMW_SCORE_SOFTMAX ? __fdiv_rn(expf(z - row_top), row_sum) : sigmoid(z);
}

// ---------------------------------------------------------------- the choice

// Best of lane-held keys: the largest, and the lowest expert that has it.  Returns
// false when none is there.  `at` is what each lane's best key stands for.
__device__ __forceinline__ bool warp_best(uint32_t key, uint32_t at, uint32_t* best_key,
                                          uint32_t* best_at) {
  *best_key = __reduce_max_sync(kFull, key);
  *best_at = __reduce_min_sync(kFull, key == *best_key ? at : 0xFFFFFFFFu);
  return *best_key != 0;
}
__device__ __forceinline__ bool warp_best(uint64_t key, uint32_t at, uint64_t* best_key,
                                          uint32_t* best_at) {
  const uint32_t hi = __reduce_max_sync(kFull, static_cast<uint32_t>(key >> 32));
  const uint32_t lo = __reduce_max_sync(
      kFull, static_cast<uint32_t>(key >> 32) == hi ? static_cast<uint32_t>(key) : 0u);
  *best_key = static_cast<uint64_t>(hi) << 32 | lo;
  *best_at = __reduce_min_sync(kFull, key == *best_key ? at : 0xFFFFFFFFu);
  return *best_key != 0;
}
__device__ __forceinline__ uint64_t ordered64(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return (b >> 63) != 0 ? ~b : b | 0x8000000000000000ull;
}

// The 64-bit choice, over the warp's own array of keys (in shared memory; -inf: not
// there).  Lane j gets the j-th expert, -1 without one.
__device__ __noinline__ int choose_exactly(const float* z, const float* bias, double* key,
                                           const adamw_router& r) {
  const int lane = threadIdx.x & 31, per = r.experts / r.groups;
  double top = -INFINITY, total = 0.0;
  if (r.score == ADAMW_SCORE_SOFTMAX) {
    for (int e = lane; e < r.experts; e += 32) top = fmax(top, static_cast<double>(z[e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, o));
    for (int e = lane; e < r.experts; e += 32) total += exp(static_cast<double>(z[e]) - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
  }
  for (int e = lane; e < r.experts; e += 32) {
    const double v = z[e];
    const float b = bias != nullptr ? bias[e] : 0.0f;
    const double s = r.score == ADAMW_SCORE_SOFTMAX ? exp(v - top) / total : 1.0 / (1.0 + exp(-v));
    key[e] = z[e] > -INFINITY && b > -INFINITY ? s + static_cast<double>(b) : -INFINITY;
  }
  __syncwarp();
  if (r.groups > 1) {
    double of = -INFINITY;
    if (lane < r.groups) {
      double one = -INFINITY, two = -INFINITY;
      for (int i = 0; i < per; ++i) {
        const double v = key[lane * per + i];
        if (v > one) {
          two = one;
          one = v;
        } else if (v > two) {
          two = v;
        }
      }
      of = r.group_score == ADAMW_GROUP_TOP2 && two > -INFINITY ? one + two : one;
    }
    uint64_t mine = of > -INFINITY ? ordered64(of) : 0;
    uint32_t kept = 0;
    for (int g = 0; g < r.top_groups; ++g) {
      uint64_t k;
      uint32_t at;
      if (!warp_best(mine, lane, &k, &at)) break;
      kept |= 1u << at;
      if (lane == static_cast<int>(at)) mine = 0;
    }
    for (int e = lane; e < r.experts; e += 32)
      if ((kept >> (e / per) & 1u) == 0) key[e] = -INFINITY;
    __syncwarp();
  }
  if (bias == nullptr) {                // in the groups the order is that of the logits
    for (int e = lane; e < r.experts; e += 32)
      if (key[e] > -INFINITY) key[e] = z[e];
    __syncwarp();
  }
  int id = -1;
  for (int j = 0; j < r.top_k; ++j) {
    uint64_t best = 0;
    uint32_t at = 0xFFFFFFFFu;
    for (int e = lane; e < r.experts; e += 32) {
      const uint64_t k = key[e] > -INFINITY ? ordered64(key[e]) : 0;
      if (k > best) {
        best = k;
        at = e;
      }
    }
    uint64_t k;
    uint32_t win;
    if (!warp_best(best, at, &k, &win)) break;
    if (lane == j) id = static_cast<int>(win);
    if (lane == static_cast<int>(win % 32)) key[win] = -INFINITY;
    __syncwarp();
  }
  return id;
}

// How far a float32 key may be off: a score's relative error (sigmoid: the exponential's,
// the quotient's and the sum's few units; softmax: the exponent's rounding too, |z - top|
// 2^-24, up to where the exponential is 0) and the sum's.  |score| <= |key| + |bias|.
__device__ __forceinline__ float key_error(float key, float bias, float relative) {
  return fmaf(relative, fabsf(key) + 2.0f * fabsf(bias), 1e-36f);
}

// Chooses from the lanes' logits.  bias: null, or shared memory.  Lane j gets the j-th
// expert (-1: none).  `z_row` and `exact` are shared memory of this warp alone.
template <int V>
__device__ __forceinline__ int choose(const float (&z)[V], const float* bias, bool bad, float top,
                                      float total, float* z_row, double* exact,
                                      const adamw_router& r) {
  const int lane = threadIdx.x & 31;
  const int per = r.experts / r.groups;
  const bool by_logit = bias == nullptr || bad;
  const bool by_group = r.groups > 1 && r.top_groups < r.groups;
  const bool two = by_group && r.group_score == ADAMW_GROUP_TOP2 && !bad;
  const float relative = r.score == ADAMW_SCORE_SOFTMAX ? 0x1p-17f : 0x1p-20f;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float k = z[i];
    bool there = z[i] > -INFINITY;
    if (bias != nullptr) {
      const int e = lane * V + i;
      const float b = e < r.experts ? bias[e] : 0.0f;
      there = there && b > -INFINITY;
      if (!bad) {
        const float s = r.score == ADAMW_SCORE_SOFTMAX ? __fdividef(expf(z[i] - top), total)
                                                       : sigmoid(z[i]);
        k = s + b;
      }
    }
    key[i] = there ? ordered(k) : 0u;
  }
  bool sure = true;
  if (by_group) {
    // lane g scores group g
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (e < r.experts) {
        float k = key[i] != 0 ? unordered(key[i]) : -INFINITY;
        if (two && by_logit && key[i] != 0)
          k = r.score == ADAMW_SCORE_SOFTMAX ? __fdividef(expf(k - top), total) : sigmoid(k);
        z_row[e] = k;
      }
    }
    __syncwarp();
    float one = -INFINITY, next = -INFINITY, off = 0.0f;
    if (lane < r.groups) {
      for (int i = 0; i < per; ++i) {
        const float v = z_row[lane * per + i];
        next = fmaxf(next, fminf(one, v));
        one = fmaxf(one, v);
      }
      if (!bad && (two || !by_logit)) {
        float b = 0.0f;                 // the group's largest bias bounds every key's error
        if (!by_logit)
          for (int i = 0; i < per; ++i) {
            const float v = fabsf(bias[lane * per + i]);
            b = v < INFINITY ? fmaxf(b, v) : b;
          }
        off = key_error(one, b, relative) + (two && next > -INFINITY ? key_error(next, b, relative) : 0.0f);
      }
    }
    const float of = two && next > -INFINITY ? one + next : one;
    uint32_t mine = of > -INFINITY ? ordered(of) : 0u;
    uint32_t kept = 0;
    float least = INFINITY;             // of a kept group's score, at its lowest
    for (int g = 0; g < r.top_groups; ++g) {
      uint32_t k, at;
      if (!warp_best(mine, lane, &k, &at)) break;
      kept |= 1u << at;
      if (lane == static_cast<int>(at)) {
        mine = 0;
        least = of - off;
      }
    }
    const float most = warp_max(mine != 0 ? of + off : -INFINITY);
    const float low = -warp_max(-least);
    // without errors equal scores went to the lowest group already
    sure = (!two && by_logit) || most < low || most == -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (e < r.experts && (kept >> (e / per) & 1u) == 0) key[i] = 0;
    }
  }
  int id = -1;
  uint32_t id_key = 0;
  for (int j = 0; j < r.top_k; ++j) {
    uint32_t best = 0, at = 0xFFFFFFFFu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] >= best && key[i] != 0) {
        best = key[i];
        at = lane * V + i;
      }
    uint32_t k, win;
    if (!warp_best(best, at, &k, &win)) break;
    if (lane == j) {
      id = static_cast<int>(win);
      id_key = k;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (static_cast<int>(win) == lane * V + i) key[i] = 0;
  }
  if (!by_logit) {
    // each chosen key, at its lowest, above all that come after it, at their highest
    float high = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] != 0) {
        const float k = unordered(key[i]);
        high = fmaxf(high, k + key_error(k, bias[lane * V + i], relative));
      }
    high = warp_max(high);
    const float k = id >= 0 ? unordered(id_key) : -INFINITY;
    const float off = id >= 0 ? key_error(k, bias[id], relative) : 0.0f;
    float after = id >= 0 ? k + off : high;
    if (lane == 31 || lane >= r.top_k) after = fmaxf(after, high);
    // the largest of the lanes after this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float v = __shfl_down_sync(kFull, after, o);
      if (lane + o < 32) after = fmaxf(after, v);
    }
    after = __shfl_down_sync(kFull, after, 1);
    if (lane == 31) after = high;
    sure = sure && (id < 0 || k - off > after || after == -INFINITY);
  }
  if (!__all_sync(kFull, sure)) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      if (e < r.experts) z_row[e] = z[i];
    }
    __syncwarp();
    id = choose_exactly(z_row, by_logit ? nullptr : bias, exact, r);
    __syncwarp();
  }
  return id;
}

// ---------------------------------------------------------------- places

// Places of one chunk's assignments, by all threads of a CTA.  `before` and `all`: for
// each expert the assignments of the chunks before this one, and of all chunks (shared
// memory, [experts]); `of_warp`: shared memory [warps][experts].
__device__ __forceinline__ void place_chunk(const RouteArgs& a, int first, int tokens, int* before,
                                            const int* all, int* of_warp, int* s_scan, bool write_starts) {
  const int experts = a.router.experts;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  // exclusive sum over the experts of all chunks' counts
  __syncthreads();
  int carry = 0;
  for (int e0 = 0; e0 < experts; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    const int n = e < experts ? all[e] : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s_scan[warp] = sum;
    __syncthreads();
    int ahead = carry;
    for (int w = 0; w < warp; ++w) ahead += s_scan[w];
    int whole = carry;
    for (int w = 0; w < warps; ++w) whole += s_scan[w];
    if (e < experts) {
      const int start = ahead + sum - n;
      before[e] += start;
      if (write_starts) a.starts[e] = start;
    }
    carry = whole;
    __syncthreads();
  }
  if (write_starts && threadIdx.x == 0) a.starts[experts] = carry;
  // each warp's run of assignments: counts, then places in order
  for (int i = threadIdx.x; i < warps * experts; i += blockDim.x) of_warp[i] = 0;
  __syncthreads();
  const int n = tokens * a.router.top_k;
  const int run = (n + warps - 1) / warps;
  const int lo = min(n, warp * run), hi = min(n, lo + run);
  const int64_t base = static_cast<int64_t>(first) * a.router.top_k;
  for (int i = lo + lane; i < hi; i += 32) {
    const int id = __ldcg(a.ids + base + i);
    if (id >= 0) atomicAdd(&of_warp[warp * experts + id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += blockDim.x) {
    int sum = before[e];
    for (int w = 0; w < warps; ++w) {
      const int c = of_warp[w * experts + e];
      of_warp[w * experts + e] = sum;
      sum += c;
    }
  }
  __syncthreads();
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const int id = i < hi ? __ldcg(a.ids + base + i) : -1;
    const uint32_t same = __match_any_sync(kFull, id);
    int slot = -1;
    if (id >= 0) slot = of_warp[warp * experts + id] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (id >= 0 && (same >> lane) == 1u) of_warp[warp * experts + id] += __popc(same);
    __syncwarp();
    if (i < hi) a.slots[base + i] = slot;
  }
}

// Warps that a CTA's places take: their counts fill at most 64 KB.
__host__ __device__ __forceinline__ int place_warps(int experts) {
  const int w = 16384 / experts;
  return w < 1 ? 1 : (w > kRouteWarps ? kRouteWarps : w);
}

// ---------------------------------------------------------------- kernels

// Shared memory of the routing kernel: the bias, this chunk's counts, and per warp a row
// of logits and one of 64-bit keys; the places use the rows' part again.
__host__ __device__ __forceinline__ int even(int n) { return (n + 1) & ~1; }
__host__ __device__ __forceinline__ size_t route_smem(int experts) {
  return sizeof(float) * (3 * even(experts)) + static_cast<size_t>(kRouteWarps) * even(experts) * 12;
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteArgs a, const bool vec) {
  extern __shared__ double s_all[];
  const int experts = a.router.experts, even_experts = even(experts);
  double* s_exact = s_all;                                        // [warps][even]
  float* s_rows = reinterpret_cast<float*>(s_exact + kRouteWarps * even_experts);
  float* s_bias = s_rows + kRouteWarps * even_experts;
  int* s_counts = reinterpret_cast<int*>(s_bias + even_experts);
  int* s_before = s_counts + even_experts;
  __shared__ int s_scan[32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int first = blockIdx.x * a.per_chunk;
  const int tokens = min(a.tokens - first, a.per_chunk);
  bool any = false;
  for (int e = threadIdx.x; e < experts; e += kRouteThreads) {
    s_counts[e] = 0;
    if (a.bias != nullptr) {
      const float b = __ldg(a.bias + e);
      s_bias[e] = b > -INFINITY ? b : -INFINITY;                  // NaN: not there
      any = any || !(b == 0.0f);
    }
  }
  // a bias of zeros changes nothing
  const float* bias = __syncthreads_or(any) ? s_bias : nullptr;
  const bool softmax = a.router.score == ADAMW_SCORE_SOFTMAX;
  // the row's largest logit and sum: for softmax keys and weights
  const bool sums = softmax && (bias != nullptr || !a.router.renormalise ||
                                (a.router.groups > 1 && a.router.group_score == ADAMW_GROUP_TOP2));
  for (int t = warp; t < tokens; t += kRouteWarps) {
    const T* row = static_cast<const T*>(a.logits) + (static_cast<int64_t>(first) + t) * a.stride;
    float z[V];
    load_row<T, V>(row, experts, vec, z);
    bool nan = false, inf = false;
    float top = -INFINITY, total = 1.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      nan = nan || z[i] != z[i];
      inf = inf || z[i] == INFINITY;
      z[i] = z[i] == z[i] ? z[i] : -INFINITY;
      top = fmaxf(top, z[i]);
    }
    const bool bad = __any_sync(kFull, nan || (softmax && inf));
    if (sums) {
      top = warp_max(top);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += z[i] > -INFINITY ? expf(z[i] - top) : 0.0f;
      total = warp_sum(sum);
    }
    const int id = choose<V>(z, bias, bad, top, total, s_rows + warp * even_experts,
                             s_exact + warp * even_experts, a.router);
    const float zj = id >= 0 ? to_f32(row[id]) : 0.0f;
    float w = a.router.scale * weight_of(zj, id >= 0, a.router, top, total);
    if (bad) w = __int_as_float(0x7FFFFFFF);
    if (lane < a.router.top_k) {
      const int64_t at = (static_cast<int64_t>(first) + t) * a.router.top_k + lane;
      a.ids[at] = id;
      a.weights[at] = w;
      if (id >= 0) atomicAdd(&s_counts[id], 1);
    }
  }
  if (a.slots == nullptr && a.starts == nullptr) return;
  __syncthreads();
  if (gridDim.x == 1) {
    for (int e = threadIdx.x; e < experts; e += kRouteThreads) s_before[e] = 0;
    place_chunk(a, first, tokens, s_before, s_counts, reinterpret_cast<int*>(s_all), s_scan, true);
  } else {
    for (int e = threadIdx.x; e < experts; e += kRouteThreads)
      a.counts[static_cast<int64_t>(blockIdx.x) * experts + e] = s_counts[e];
    let_next_kernel_start();
  }
}

// Every chunk's places from the table of counts.
__global__ void __launch_bounds__(kRouteThreads) place_kernel(const RouteArgs a) {
  extern __shared__ int s_place[];
  __shared__ int s_scan[32];
  const int experts = a.router.experts;
  int* before = s_place;
  int* all = before + experts;
  int* of_warp = all + experts;
  for (int e = threadIdx.x; e < 2 * experts; e += blockDim.x) before[e] = 0;
  wait_for_previous_kernel();
  __syncthreads();
  // thread = an expert and every `step`-th chunk; sums of whole numbers in any order
  const int wide = min(experts, static_cast<int>(blockDim.x));
  const int step = blockDim.x / wide;
  const int c0 = threadIdx.x / wide;
  if (c0 < step) {
    for (int e = threadIdx.x % wide; e < experts; e += wide) {
      int mine = 0, whole = 0;
#pragma unroll 8
      for (int c = c0; c < a.chunks; c += step) {
        const int n = __ldcg(a.counts + static_cast<int64_t>(c) * experts + e);
        whole += n;
        mine += c < static_cast<int>(blockIdx.x) ? n : 0;
      }
      atomicAdd(&before[e], mine);
      atomicAdd(&all[e], whole);
    }
  }
  const int first = blockIdx.x * a.per_chunk;
  place_chunk(a, first, min(a.tokens - first, a.per_chunk), before, all, of_warp, s_scan,
              blockIdx.x == 0);
}

template <typename T, int V>
__global__ void __launch_bounds__(32 * kBackWarps) route_backward_kernel(const RouteArgs a, const bool vec,
                                                                         const bool vec_out) {
  extern __shared__ float s_grad[];
  const adamw_router& r = a.router;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  float* mine = s_grad + warp * (32 * V);
  const bool softmax = r.score == ADAMW_SCORE_SOFTMAX;
  const bool dense = softmax && !r.renormalise;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kBackWarps + warp; t < a.tokens;
       t += static_cast<int64_t>(gridDim.x) * kBackWarps) {
    const T* row = static_cast<const T*>(a.logits) + t * a.stride;
    int id = -1;
    float zj = 0.0f, dw = 0.0f;
    if (lane < r.top_k) {
      id = __ldg(a.ids + t * r.top_k + lane);
      if (id < 0 || id >= r.experts) id = -1;
      if (id >= 0) {
        dw = r.scale * __ldg(a.dweights + t * r.top_k + lane);
        zj = to_f32(row[id]);
      }
    }
    float z[V], top = 0.0f, total = 1.0f;
    if (dense) {
      load_row<T, V>(row, r.experts, vec, z);
      top = -INFINITY;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        nan = nan || z[i] != z[i];
        top = fmaxf(top, z[i]);
      }
      top = warp_max(top);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += z[i] > -INFINITY ? expf(z[i] - top) : 0.0f;
      total = warp_sum(sum);
      if (__any_sync(kFull, nan)) total = __int_as_float(0x7FFFFFFF);
    }
    const float w = weight_of(zj, id >= 0, r, top, total);
    const float mean = warp_sum(id >= 0 ? dw * w : 0.0f);
    float d = 0.0f;                               // this lane's chosen logit's gradient
    if (dense) d = w * dw;
    else if (r.renormalise) d = w * (dw - mean) * (softmax ? 1.0f : sigmoid(-zj));
    else d = dw * w * sigmoid(-zj);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i) mine[i * 32 + lane] = 0.0f;
    __syncwarp();
    if (id >= 0) mine[id] = d;
    __syncwarp();
    T* out = static_cast<T*>(a.dlogits) + t * a.dstride;
    float g[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      g[i] = mine[lane * V + i];
      if (dense) g[i] -= z[i] > -INFINITY ? __fdiv_rn(expf(z[i] - top), total) * mean : 0.0f;
    }
    if (V * sizeof(T) >= 4 && vec_out) {
      constexpr int kWords = V * sizeof(T) >= 4 ? V * static_cast<int>(sizeof(T)) / 4 : 1;
      uint32_t word[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (sizeof(T) == 4) word[i] = __float_as_uint(g[i]);
        else word[i] = pack_pair<T>(make_float2(g[2 * i % V], g[(2 * i + 1) % V]));
      }
      uint32_t* p = reinterpret_cast<uint32_t*>(out + lane * V);
      if constexpr (kWords >= 4) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i)
          __stcs(reinterpret_cast<uint4*>(p) + i,
                 make_uint4(word[4 * i], word[4 * i + 1], word[4 * i + 2], word[4 * i + 3]));
      } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i) p[i] = word[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane * V + i < r.experts) out[lane * V + i] = from_f32<T>(g[i]);
    }
  }
}

__global__ void balance_kernel(const int32_t* starts, int32_t experts, float rate, float* bias) {
  const int64_t all = static_cast<int64_t>(starts[experts]) - starts[0];
  for (int e = threadIdx.x; e < experts; e += blockDim.x) {
    const int64_t over = (static_cast<int64_t>(starts[e + 1]) - starts[e]) * experts - all;
    if (over != 0) bias[e] += over > 0 ? -rate : rate;
  }
}

// ---------------------------------------------------------------- launches

template <typename T>
bool lanes_on_grid(const void* p, int64_t stride, int experts, int v) {
  const size_t bytes = v * sizeof(T), grid = bytes < 16 ? bytes : 16;
  return experts == 32 * v && bytes >= 4 && reinterpret_cast<uintptr_t>(p) % grid == 0 &&
         stride * sizeof(T) % grid == 0;
}

template <typename T, int V>
cudaError_t route_width(const RouteArgs& a, cudaStream_t s) {
  const bool vec = lanes_on_grid<T>(a.logits, a.stride, a.router.experts, V);
  route_kernel<T, V><<<a.chunks, kRouteThreads, route_smem(a.router.experts), s>>>(a, vec);
  return cudaGetLastError();
}
template <typename T, int V>
cudaError_t back_width(const RouteArgs& a, int sms, cudaStream_t s) {
  const bool vec = lanes_on_grid<T>(a.logits, a.stride, a.router.experts, V);
  const bool vec_out = lanes_on_grid<T>(a.dlogits, a.dstride, a.router.experts, V);
  const int64_t ctas = (a.tokens + kBackWarps - 1) / kBackWarps, most = 8LL * sms;
  route_backward_kernel<T, V><<<static_cast<unsigned>(ctas < most ? ctas : most), 32 * kBackWarps,
                                kBackWarps * 32 * V * sizeof(float), s>>>(a, vec, vec_out);
  return cudaGetLastError();
}

#define ADAMW_ROUTE_WIDTH(experts, CALL)  \
  ((experts) <= 32    ? CALL(1)           \
   : (experts) <= 64  ? CALL(2)           \
   : (experts) <= 128 ? CALL(4)           \
   : (experts) <= 256 ? CALL(8)           \
   : (experts) <= 512 ? CALL(16)          \
                      : CALL(32))

template <typename T>
cudaError_t route_type(const RouteArgs& a, cudaStream_t s) {
#define ADAMW_ROUTE_CALL(V) route_width<T, V>(a, s)
  return ADAMW_ROUTE_WIDTH(a.router.experts, ADAMW_ROUTE_CALL);
#undef ADAMW_ROUTE_CALL
}
template <typename T>
cudaError_t back_type(const RouteArgs& a, int sms, cudaStream_t s) {
#define ADAMW_ROUTE_CALL(V) back_width<T, V>(a, sms, s)
  return ADAMW_ROUTE_WIDTH(a.router.experts, ADAMW_ROUTE_CALL);
#undef ADAMW_ROUTE_CALL
}
template <typename T, int V>
cudaError_t prepare_width() {
  // what the most experts of this width take: one plan's must not shrink another's
  return cudaFuncSetAttribute(route_kernel<T, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(route_smem(32 * V)));
}
template <typename T>
cudaError_t prepare_type(int experts) {
#define ADAMW_ROUTE_CALL(V) prepare_width<T, V>()
  return ADAMW_ROUTE_WIDTH(experts, ADAMW_ROUTE_CALL);
#undef ADAMW_ROUTE_CALL
}
size_t place_smem(int experts) {
  return sizeof(int) * experts * (2 + place_warps(experts));
}

}  // namespace

int router_chunks(int sms) { return sms; }

cudaError_t prepare_router(const adamw_router& r) {
  cudaError_t e = prepare_type<float>(r.experts);
  if (e == cudaSuccess) e = prepare_type<__half>(r.experts);
  if (e == cudaSuccess) e = prepare_type<__nv_bfloat16>(r.experts);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(place_smem(kMaxExperts)));
  return e;
}

cudaError_t launch_route(adamw_dtype dt, RouteArgs a, int sms, cudaStream_t s) {
  // one CTA for what its warps take in two turns, else a share of every SM's
  const int64_t most = router_chunks(sms);
  int64_t chunks = a.tokens <= 2 * kRouteWarps ? 1 : (a.tokens + kRouteWarps - 1) / kRouteWarps;
  if (chunks > most) chunks = most;
  a.per_chunk = static_cast<int32_t>((a.tokens + chunks - 1) / chunks);
  a.chunks = a.per_chunk > 0 ? (a.tokens + a.per_chunk - 1) / a.per_chunk : 1;
  cudaError_t e = dt == ADAMW_F32   ? route_type<float>(a, s)
                  : dt == ADAMW_F16 ? route_type<__half>(a, s)
                                    : route_type<__nv_bfloat16>(a, s);
  if (e != cudaSuccess || a.chunks == 1 || a.starts == nullptr) return e;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(a.chunks));
  c.blockDim = dim3(32 * place_warps(a.router.experts));
  c.dynamicSmemBytes = place_smem(a.router.experts);
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = early_start(&attr);
  return cudaLaunchKernelEx(&c, place_kernel, a);
}

cudaError_t launch_route_backward(adamw_dtype dt, const RouteArgs& a, int sms, cudaStream_t s) {
  if (dt == ADAMW_F32) return back_type<float>(a, sms, s);
  if (dt == ADAMW_F16) return back_type<__half>(a, sms, s);
  return back_type<__nv_bfloat16>(a, sms, s);
}

cudaError_t launch_route_balance(const int32_t* starts, int32_t experts, float rate, float* bias,
                                 cudaStream_t s) {
  balance_kernel<<<1, experts < 256 ? 256 : 1024, 0, s>>>(starts, experts, rate, bias);
  return cudaGetLastError();
}

}  // namespace adamw
