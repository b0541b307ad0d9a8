// router.cu -- routing of tokens to experts: scores, groups, the top_k choice and its
// weights, every assignment's place when all are ordered by expert, the gradient of
// the logits, and the balance step of the bias.
//
// The choice is top_k rounds of a maximum over integers, each a key and the expert's number
// counted down, so that one maximum names the expert and of equal keys the lowest wins.  A
// lane keeps its two best and looks for a third only when both are gone.  Where no bias takes
// part the order of the scores is that of the logits, and no score is computed for it.
//
// Up to 256 experts, and up to 512 without groups, a token has a team of 8, 16 or 32 lanes and a
// warp several tokens (route_teams_kernel; groups of whole lanes): 5 and 2.5 times fewer
// instructions a token than with a warp for each (128 and 256 experts), and it is instructions
// that bound it.  Where 32 lanes of 16 experts do not hold the groups, or the experts, a warp
// takes a token (route_kernel).  65536 x 128 bf16, 8 chosen: 24 us for the choice, 8 for the places,
// 10 for the gradient (27 where the whole softmax has one: it reads a row twice).  65536 x 1024: 106
// us and 37.  All variants of the team kernel spill at the 72 registers that 28 warps leave, 44 to 332
// bytes a thread, most with 16 experts a lane in teams of 8 and 16.
//
// Keys are off by a few units of the scores' last bits and by the bits that the number takes
// (none that 16-bit logits have).  A choice in which two keys that matter lie closer than that
// (about one token in a thousand) is made again from 64-bit scores, so that the experts are those
// of the definition and not of a rounding: of the few experts that can matter, a lane each, or of
// all of them.
#include "block_ops.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr int kBackWarps = 8;
constexpr int kPlaceThreads = 1024;

// Experts of a lane where a warp takes a token, and the warps of its CTA.
constexpr int kWarpExperts = 32;
constexpr int kRouteWarps = 16;

// Floats as integers of the same order.  Up to kNone they stand for -inf, "not there"; 0
// is a key that has been taken.
constexpr uint32_t kNone = 0x007FFFFFu;
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);          // -0 and 0 are one value
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) != 0 ? o & 0x7FFFFFFFu : ~o);
}
// e^x and 1 / (1 + e^-x) for keys, whose errors the choice allows for: x log2 e is rounded
// once, then the hardware's 2^x and reciprocal.
__device__ __forceinline__ float key_exp(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 1.4426950408889634f));
  return e;
}
__device__ __forceinline__ float key_sigmoid(float x) {
  float s;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + key_exp(-x)));
  return s;
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

// The weight of a lane's chosen logit z before `scale`, among the WIDE neighbouring lanes of
// its token (0: `wide` of them); `row_top` and `row_sum` are the softmax's largest logit and
// sum over the whole row (used without renormalisation).
template <int WIDE>
__device__ __forceinline__ float weight_of(float z, bool chosen, const adamw_router& r,
                                           float row_top, float row_sum, int wide = WIDE) {
  if (WIDE > 0) wide = WIDE;
  if (r.renormalise) {
    // Only ratios count, so small scores are taken relative to the largest chosen one:
    // below a logit of -30 the sigmoid is e^z to the last bit.
    float top = chosen ? z : -INFINITY;
#pragma unroll
    for (int o = wide / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    const bool ratio = r.score == ADAMW_SCORE_SOFTMAX || top < -30.0f;
    const float s = chosen ? (ratio ? expf(z - top) : sigmoid(z)) : 0.0f;
    float total = s;
#pragma unroll
    for (int o = wide / 2; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
    return chosen ? __fdividef(s, total) : 0.0f;
  }
  if (!chosen) return 0.0f;
  return r.score == ADAMW_SCORE_SOFTMAX ? __fdividef(expf(z - row_top), row_sum) : sigmoid(z);
}
// Lanes of a token: the smallest power of two that holds its choice.
__host__ __device__ __forceinline__ int choice_lanes(int top_k) {
  int w = 1;
  while (w < top_k) w *= 2;
  return w;
}

// ---------------------------------------------------------------- the choice

__device__ __forceinline__ uint64_t ordered64(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return (b >> 63) != 0 ? ~b : b | 0x8000000000000000ull;
}
// The largest of the lanes' keys, and the lowest `at` of the lanes that have it; false when
// no key is there.
__device__ __forceinline__ bool warp_best(uint64_t key, uint32_t at, uint32_t* best_at) {
  const uint32_t hi = __reduce_max_sync(kFull, static_cast<uint32_t>(key >> 32));
  const uint32_t lo = __reduce_max_sync(
      kFull, static_cast<uint32_t>(key >> 32) == hi ? static_cast<uint32_t>(key) : 0u);
  const uint64_t best = static_cast<uint64_t>(hi) << 32 | lo;
  *best_at = __reduce_min_sync(kFull, key == best ? at : 0xFFFFFFFFu);
  return best != 0;
}

// The 64-bit choice from a token's logits, over the warp's own array of keys (in shared
// memory; -inf: not there).  by_logit: whatever the bias, the order is that of the logits, and
// `bad` that of groups too.  Lane j gets the j-th expert, -1 without one.
template <typename T>
__device__ __noinline__ int choose_exactly(const T* row, const float* bias, bool by_logit, bool bad, double* key,
                                           const adamw_router& r) {
  const int lane = threadIdx.x & 31, per = r.experts / r.groups;
  const bool by_group = r.groups > 1 && r.top_groups < r.groups;
  const bool scores = !bad && (!by_logit || (by_group && r.group_score == ADAMW_GROUP_TOP2));
  double top = -INFINITY, total = 1.0;
  if (scores && r.score == ADAMW_SCORE_SOFTMAX) {
    for (int e = lane; e < r.experts; e += 32) top = fmax(top, static_cast<double>(to_f32(row[e])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(kFull, top, o));
    total = 0.0;
    for (int e = lane; e < r.experts; e += 32) total += exp(static_cast<double>(to_f32(row[e])) - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
  }
  for (int e = lane; e < r.experts; e += 32) {
    const float z = to_f32(row[e]);
    const float b = bias != nullptr ? bias[e] : 0.0f;
    double s = z;
    if (scores) {
      s = r.score == ADAMW_SCORE_SOFTMAX ? exp(z - top) / total : 1.0 / (1.0 + exp(-s));
      if (!by_logit) s += static_cast<double>(b);
    }
    key[e] = z > -INFINITY && b > -INFINITY ? s : -INFINITY;       // a NaN is not there
  }
  __syncwarp();
  if (by_group) {
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
      of = r.group_score == ADAMW_GROUP_TOP2 && !bad && two > -INFINITY ? one + two : one;
    }
    uint64_t mine = of > -INFINITY ? ordered64(of) : 0;
    uint32_t kept = 0;
    for (int g = 0; g < r.top_groups; ++g) {
      uint32_t at;
      if (!warp_best(mine, lane, &at)) break;
      kept |= 1u << at;
      if (lane == static_cast<int>(at)) mine = 0;
    }
    for (int e = lane; e < r.experts; e += 32)
      if ((kept >> (e / per) & 1u) == 0) key[e] = -INFINITY;
    __syncwarp();
  }
  if (by_logit) {
    for (int e = lane; e < r.experts; e += 32)
      if (key[e] > -INFINITY) key[e] = to_f32(row[e]);
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
    uint32_t win;
    if (!warp_best(best, at, &win)) break;
    if (lane == j) id = static_cast<int>(win);
    if (lane == static_cast<int>(win % 32)) key[win] = -INFINITY;
    __syncwarp();
  }
  return id;
}

// Chooses from the lanes' logits (NaN as -inf).  bias: null, or shared memory with its largest
// magnitude.  Lane j gets the j-th expert (-1: none).  `own`: shared memory of this warp.
template <typename T>
__device__ __forceinline__ int choose(const T* row, float (&k)[kWarpExperts], const float* bias, float bias_max, bool bad, float top,
                                      float total, double* own, const RouteArgs& a) {
  constexpr int V = kWarpExperts;
  constexpr uint32_t kPlace = V - 1;
  const adamw_router& r = a.router;
  const int lane = threadIdx.x & 31, per = a.per_group;
  const bool softmax = r.score == ADAMW_SCORE_SOFTMAX;
  const bool by_logit = bias == nullptr || bad;
  const bool by_group = r.groups > 1 && r.top_groups < r.groups;
  const bool two = by_group && r.group_score == ADAMW_GROUP_TOP2 && !bad;
  // A score is off by at most this part of the row's largest (of 1 for the sigmoid): 2^-21 for
  // the exponential and the reciprocal (the argument's rounding counts |d| e^-d < 1), the sum's
  // V + 8 roundings, and the V units of the key's last bit that the place takes.
  const float inv = __fdividef(1.0f, total);
  const float off = (0x1p-20f + V * 0x1.8p-23f) * ((softmax ? inv : 1.0f) + 3.0f * bias_max) + 1e-36f;
  if (bias != nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 32 * i + lane;
      const float b = bias[min(e, r.experts - 1)];
      const float s = bad ? k[i] : (softmax ? key_exp(k[i] - top) * inv : key_sigmoid(k[i])) + b;
      k[i] = k[i] > -INFINITY && b > -INFINITY ? s : -INFINITY;
    }
  }
  bool sure = by_logit || bias_max < INFINITY;
  uint32_t kept = 0xFFFFFFFFu;
  if (by_group) {
    float2 tops = make_float2(-INFINITY, -INFINITY);
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = k[i];
      if (two && by_logit) v[i] = k[i] > -INFINITY ? (softmax ? key_exp(k[i] - top) * inv : key_sigmoid(k[i])) : -INFINITY;
    }
    float* lines = reinterpret_cast<float*>(own);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (32 * i + lane < r.experts) lines[32 * i + lane] = v[i];
    __syncwarp();
    const int share = 32 / choice_lanes(r.groups);         // lanes of a group
    const int group = lane / share;                        // that this lane scores
    if (group < r.groups)
      for (int i = lane - group * share; i < per; i += share) {
        const float x = lines[group * per + i];
        tops.y = fmaxf(tops.y, fminf(tops.x, x));
        tops.x = fmaxf(tops.x, x);
      }
    for (int o = 1; o < share; o *= 2) {
      const float x = __shfl_xor_sync(kFull, tops.x, o), y = __shfl_xor_sync(kFull, tops.y, o);
      tops.y = fmaxf(fminf(tops.x, x), fmaxf(tops.y, y));
      tops.x = fmaxf(tops.x, x);
    }
    __syncwarp();
    const float of = two && tops.y > -INFINITY ? tops.x + tops.y : tops.x;
    uint32_t mine = group < r.groups ? ordered(of) : 0u, least = 0;
    kept = 0;
    for (int g = 0; g < r.top_groups; ++g) {
      const uint32_t best = __reduce_max_sync(kFull, mine);
      if (best <= kNone) break;
      const int at = __shfl_sync(kFull, group, __ffs(__ballot_sync(kFull, mine == best)) - 1);
      kept |= 1u << at;
      least = best;
      if (group == at) mine = 0;
    }
    const uint32_t most = __reduce_max_sync(kFull, mine);
    // without scores equal groups went to the lowest already
    sure = sure && ((!two && by_logit) || most <= kNone || unordered(least) - unordered(most) > 4.0f * off);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((kept >> ((32 * i + lane) * a.group_factor >> 20) & 1u) == 0) k[i] = -INFINITY;
  }
  uint32_t key[V], best = 0, second = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = (ordered(k[i]) & ~kPlace) | (kPlace - i);
    second = max(second, min(best, key[i]));
    best = max(best, key[i]);
  }
  uint32_t mine = 0;
  int lane_of = 0;
  for (int j = 0; j < r.top_k; ++j) {
    const uint32_t most = __reduce_max_sync(kFull, best);
    if (most <= kNone) break;
    const int who = __ffs(__ballot_sync(kFull, best == most)) - 1;
    if (lane == j) {
      mine = most;
      lane_of = who;
    }
    if (lane == who) {
      best = second;
      second = 0;
    }
    if (__any_sync(kFull, best == 0)) {
      if (best == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) best = max(best, key[i] < most ? key[i] : 0u);
        if (best == 0) best = 1;           // none left
      }
    }
  }
  int id = mine > kNone ? 32 * static_cast<int>(kPlace - (mine & kPlace)) + lane_of : -1;
  // each chosen key is far enough above the one that comes after it
  if (!by_logit || sizeof(T) == 4) {
    const uint32_t rest = __reduce_max_sync(kFull, best);
    uint32_t after = __shfl_down_sync(kFull, mine, 1);
    if (lane == 31 || after == 0) after = rest;
    if (id >= 0 && after > kNone)
      sure = sure && (by_logit ? ((mine ^ after) & ~kPlace) != 0
                               : unordered(mine & ~kPlace) - unordered(after & ~kPlace) > 2.0f * off);
  }
  if (!__all_sync(kFull, sure)) {
    id = choose_exactly(row, bias, by_logit, bad, own, r);
    __syncwarp();
  }
  return id;
}

// ---------------------------------------------------------------- places

// Places of one chunk's assignments, by all threads of a CTA.  `before` and `all`: for
// each expert the assignments of the chunks before this one, and of all chunks (shared
// memory, [experts]); `of_warp`: shared memory [warps][experts].
__device__ __forceinline__ void place_chunk(const RouteArgs& a, int first, int tokens, int* before,
                                            const int* all, int* of_warp, int warps, int* s_scan, bool write_starts) {
  const int experts = a.router.experts;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  // the warps' runs of assignments are counted while the first warp adds up the experts
  const int n = tokens * a.router.top_k;
  const int run = (n + warps - 1) / warps;
  const int lo = warp < warps ? min(n, warp * run) : n, hi = min(n, lo + run);
  const int64_t base = static_cast<int64_t>(first) * a.router.top_k;
  constexpr int kIds = 4;                  // of a lane on their way at once
  int* mine = of_warp + warp * experts;
  const auto load = [&](int i0, int (&id)[kIds]) {
#pragma unroll
    for (int u = 0; u < kIds; ++u) {
      const int i = i0 + 32 * u + lane;
      id[u] = i < hi ? __ldcg(a.ids + base + i) : -1;
    }
  };
  const auto count = [&](const int (&id)[kIds]) {
#pragma unroll
    for (int u = 0; u < kIds; ++u)
      if (id[u] >= 0) atomicAdd(&mine[id[u]], 1);
  };
  int id[kIds];
  load(lo, id);
  for (int i = threadIdx.x; i < warps * experts; i += blockDim.x) of_warp[i] = 0;
  __syncthreads();
  count(id);
  for (int i0 = lo + 32 * kIds; i0 < hi; i0 += 32 * kIds) {
    int more[kIds];
    load(i0, more);
    count(more);
  }
  // exclusive sum of all chunks' counts over the experts, 1024 of them at most
  const int e = threadIdx.x;
  int sum = 0;
  for (int e0 = 0, carry = 0; e0 < experts; e0 += blockDim.x) {
    const int x = e0 + e;
    const int c = x < experts ? all[x] : 0;
    sum = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s_scan[warp] = sum;
    __syncthreads();
    int w = lane < static_cast<int>(blockDim.x / 32) ? s_scan[lane] : 0;
    int whole = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, whole, o);
      if (lane >= o) whole += v;
    }
    const int ahead = carry + __shfl_sync(kFull, whole - w, warp) + sum - c;
    if (x < experts) {
      before[x] += ahead;
      if (write_starts) a.starts[x] = ahead;
    }
    carry += __shfl_sync(kFull, whole, 31);
    if (write_starts && x + 1 == experts) a.starts[experts] = ahead + c;
    __syncthreads();
  }
  for (int x = threadIdx.x; x < experts; x += blockDim.x) {
    int at = before[x];
    for (int w = 0; w < warps; ++w) {
      const int c = of_warp[w * experts + x];
      of_warp[w * experts + x] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int i0 = lo; i0 < hi; i0 += 32 * kIds) {
    if (i0 > lo) load(i0, id);
#pragma unroll
    for (int u = 0; u < kIds; ++u) {
      const int i = i0 + 32 * u + lane;
      if (i0 + 32 * u >= hi) break;
      const uint32_t same = __match_any_sync(kFull, id[u]);
      int slot = -1;
      if (id[u] >= 0) slot = mine[id[u]] + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (id[u] >= 0 && (same >> lane) == 1u) mine[id[u]] += __popc(same);
      __syncwarp();
      if (i < hi) a.slots[base + i] = slot;
    }
  }
}

// Warps among which a chunk's assignments are dealt out: their counts fill at most 64 KB.
__host__ __device__ __forceinline__ int place_warps(int experts, int most) {
  const int w = 16384 / experts;
  return w < most ? w : most;
}

// ---------------------------------------------------------------- kernels

__host__ __device__ __forceinline__ int even(int n) { return (n + 1) & ~1; }
// Shared memory of the routing kernel: per warp a row of 64-bit keys (the places of a lone
// chunk use them again), the bias, this chunk's counts and its places' starts.
size_t route_smem(int experts) {
  return static_cast<size_t>(kRouteWarps) * even(experts) * sizeof(double) + sizeof(float) * 3 * even(experts);
}

// Lane l's V logits, -inf behind the last expert.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int experts, T (&z)[V]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 32 * i + lane;
    z[i] = e < experts ? __ldcs(row + e) : from_f32<T>(-INFINITY);
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kRouteWarps, 1) route_kernel(const RouteArgs a) {
  constexpr int V = kWarpExperts, kWarps = kRouteWarps, kThreads = 32 * kWarps;
  extern __shared__ double s_all[];
  const int experts = a.router.experts, even_experts = even(experts);
  float* s_bias = reinterpret_cast<float*>(s_all + kWarps * even_experts);
  int* s_counts = reinterpret_cast<int*>(s_bias + even_experts);
  int* s_before = s_counts + even_experts;
  __shared__ int s_scan[32];
  __shared__ uint32_t s_bias_max;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int first = blockIdx.x * a.per_chunk;
  const int tokens = min(a.tokens - first, a.per_chunk);
  const T* rows = static_cast<const T*>(a.logits) + static_cast<int64_t>(first) * a.stride;
  T next[V];
  if (warp < tokens) load_row<T, V>(rows + warp * a.stride, experts, next);
  if (threadIdx.x == 0) s_bias_max = 0;
  __syncthreads();
  bool any = false;
  for (int e = threadIdx.x; e < experts; e += kThreads) {
    s_counts[e] = 0;
    if (a.bias != nullptr) {
      const float b = __ldg(a.bias + e);
      s_bias[e] = b > -INFINITY ? b : -INFINITY;                  // NaN: not there
      any = any || !(b == 0.0f);
      if (b > -INFINITY) atomicMax(&s_bias_max, __float_as_uint(fabsf(b)));
    }
  }
  // a bias of zeros changes nothing
  const float* bias = __syncthreads_or(any) ? s_bias : nullptr;
  const float bias_max = __uint_as_float(s_bias_max);
  const bool softmax = a.router.score == ADAMW_SCORE_SOFTMAX;
  // the row's largest logit and sum: for softmax keys and weights
  const bool sums = softmax && (bias != nullptr || !a.router.renormalise ||
                                (a.router.groups > 1 && a.router.group_score == ADAMW_GROUP_TOP2));
  const int wide = choice_lanes(a.router.top_k);
  for (int t = warp; t < tokens; t += kWarps) {
    const T* row = rows + t * a.stride;
    float z[V];
    bool nan = false;
    float top = -INFINITY, total = 1.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float f = to_f32(next[i]);
      nan = nan || f != f;
      z[i] = fmaxf(f, -INFINITY);                                 // a NaN is not there
      top = fmaxf(top, z[i]);
    }
    if (t + kWarps < tokens) load_row<T, V>(row + kWarps * a.stride, experts, next);
    const bool bad = __any_sync(kFull, nan || (softmax && top == INFINITY));
    if (sums) {
      top = warp_max(top);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += z[i] > -INFINITY ? key_exp(z[i] - top) : 0.0f;
      total = warp_sum(sum);
    }
    const int id = choose<T>(row, z, bias, bias_max, bad, top, total, s_all + warp * even_experts, a);
    const float zj = id >= 0 ? to_f32(row[id]) : 0.0f;
    float w = a.router.scale * weight_of<0>(zj, id >= 0, a.router, top, total, wide);
    if (bad) w = __int_as_float(0x7FFFFFFF);
    if (lane < a.router.top_k) {
      const int64_t at = (static_cast<int64_t>(first) + t) * a.router.top_k + lane;
      a.ids[at] = id;
      a.weights[at] = w;
      if (id >= 0) atomicAdd(&s_counts[id], 1);
    }
  }
  if (a.starts == nullptr) return;
  __syncthreads();
  if (gridDim.x == 1) {
    for (int e = threadIdx.x; e < experts; e += kThreads) s_before[e] = 0;
    place_chunk(a, first, tokens, s_before, s_counts, reinterpret_cast<int*>(s_all), place_warps(experts, kWarps), s_scan, true);
  } else {
    for (int e = threadIdx.x; e < experts; e += kThreads)
      a.counts[static_cast<int64_t>(blockIdx.x) * a.pitch + e] = s_counts[e];
    let_next_kernel_start();
  }
}

// ---------------------------------------------------------------- teams

// Warps of a CTA, at most: 8192 x 256 float32 in 8 groups 26 us, with 24 (80 registers a thread
// for 72) 28.5.  A CTA of fewer tokens than they hold has fewer.
constexpr int kTeamWarps = 28;
constexpr uint32_t kNumber = 511;        // experts are numbered in a key's lowest bits
constexpr float kFirstUnit = 16400.0f;   // of the scores' scale: its keys lie above kNone

template <int LANES>
__device__ __forceinline__ uint32_t team_max(uint32_t x) {
  if constexpr (LANES == 32) return __reduce_max_sync(kFull, x);
#pragma unroll
  for (int o = LANES / 2; o > 0; o /= 2) x = max(x, __shfl_xor_sync(kFull, x, o));
  return x;
}
template <int LANES>
__device__ __forceinline__ float team_max(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o /= 2) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
  return x;
}
template <int LANES>
__device__ __forceinline__ float team_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o /= 2) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

// V logits of a lane from expert e0 on; -inf from `end` on.
template <typename T, int V>
struct TeamRow {
  static constexpr int kBytes = V * static_cast<int>(sizeof(T));
  uint32_t word[kBytes / 4];
  __device__ __forceinline__ void load(const T* row, int e0, int end, bool vec) {
    if (vec) {                            // whole rows, on the grid of a lane's bytes (16 at most)
      const T* p = row + e0;
      if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
          const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p) + i);
          word[4 * i] = q.x;
          word[4 * i + 1] = q.y;
          word[4 * i + 2] = q.z;
          word[4 * i + 3] = q.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i) word[i] = __ldcs(reinterpret_cast<const uint32_t*>(p) + i);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const T z = e0 + i < end ? __ldcs(row + e0 + i) : from_f32<T>(-INFINITY);
      if constexpr (sizeof(T) == 4) {
        word[i] = __float_as_uint(z);
      } else {
        const uint32_t h = *reinterpret_cast<const uint16_t*>(&z);
        word[i / 2] = i % 2 == 0 ? h : word[i / 2] | h << 16;
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(word[i]);
    const float2 f = unpack_pair<T>(word[i / 2]);
    return i % 2 == 0 ? f.x : f.y;
  }
};

// A token's key in 64 bits, of an expert's logit and bias: by the logit alone, or the softmax's
// (of the row's largest logit and sum) or the sigmoid's score.  Out of line: few tokens need it.
__device__ __noinline__ double exact_key(float z, float b, bool by_logit, bool softmax, double top, double total) {
  if (by_logit) return z;
  const double e = exp(softmax ? z - top : -static_cast<double>(z));
  return (softmax ? e / total : 1.0 / (1.0 + e)) + static_cast<double>(b);
}
// A team's sum of exponentials in 64 bits.  Called by all lanes of a warp together.
template <typename T, int LANES>
__device__ __noinline__ double exact_sum(const T* row, int e0, int end, int many, float top) {
  double t = 0.0;
  for (int i = 0; i < many && e0 + i < end; ++i) {
    const float z = to_f32(row[e0 + i]);
    t += z > -INFINITY ? exp(static_cast<double>(z) - top) : 0.0;
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o /= 2) t += __shfl_xor_sync(kFull, t, o);
  return t;
}

size_t team_smem(int experts, int warps) {
  return static_cast<size_t>(warps) * even(experts) * sizeof(double) + sizeof(float) * (3 * even(experts) + 32);
}

template <typename T, int LANES, int V>
__global__ void __launch_bounds__(32 * kTeamWarps, 1) route_teams_kernel(const RouteArgs a, const bool vec) {
  constexpr int kTokens = 32 / LANES;
  const int warps = blockDim.x / 32;
  extern __shared__ double s_all[];
  const adamw_router& r = a.router;
  const int experts = r.experts, even_experts = even(experts);
  float* s_bias = reinterpret_cast<float*>(s_all + warps * even_experts);     // V at a time may pass the last one
  int* s_counts = reinterpret_cast<int*>(s_bias + even_experts + 32);
  int* s_before = s_counts + even_experts;
  __shared__ int s_scan[32];
  __shared__ uint32_t s_bias_max;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, sub = lane / LANES, l = lane % LANES;
  const int first = blockIdx.x * a.per_chunk;
  const int tokens = min(a.tokens - first, a.per_chunk);
  const T* rows = static_cast<const T*>(a.logits) + static_cast<int64_t>(first) * a.stride;
  // A group has lanes of its own, a power of two of them (without groups all are one).
  const bool by_group = r.groups > 1 && r.top_groups < r.groups;
  const int per = by_group ? a.per_group : experts, group_lanes = by_group ? a.group_lanes : LANES, group = by_group ? l / group_lanes : 0;
  const int e0 = min(group * per + (l - group * group_lanes) * V, experts), end = min((group + 1) * per, experts);
  TeamRow<T, V> next;
  const int start = warp * kTokens + sub;
  if (start < tokens) next.load(rows + static_cast<int64_t>(start) * a.stride, e0, end, vec);
  if (threadIdx.x == 0) s_bias_max = 0;
  __syncthreads();
  bool any = false;
  for (int e = threadIdx.x; e < experts; e += 32 * warps) {
    s_counts[e] = 0;
    if (a.bias != nullptr) {
      const float b = __ldg(a.bias + e);
      s_bias[e] = b > -INFINITY ? b : -INFINITY;                  // NaN: not there
      any = any || !(b == 0.0f);
      if (b > -INFINITY) atomicMax(&s_bias_max, __float_as_uint(fabsf(b)));
    }
  }
  // a bias of zeros changes nothing
  const float* bias = __syncthreads_or(any) ? s_bias : nullptr;
  const float bias_max = __uint_as_float(s_bias_max);
  const bool softmax = r.score == ADAMW_SCORE_SOFTMAX;
  const bool two = by_group && r.group_score == ADAMW_GROUP_TOP2;
  const bool scored = bias != nullptr || two;           // keys are scores, not logits
  const bool sums = softmax && (scored || !r.renormalise);
  for (int t0 = warp * kTokens; t0 < tokens; t0 += warps * kTokens) {
    const int t = t0 + sub;
    const bool live = t < tokens;
    const T* row = rows + static_cast<int64_t>(live ? t : t0) * a.stride;
    float z[V];
    bool nan = false;
    float top = -INFINITY, total = 1.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float f = live ? next.at(i) : -INFINITY;
      nan = nan || f != f;
      z[i] = fmaxf(f, -INFINITY);                                 // a NaN is not there
      top = fmaxf(top, z[i]);
    }
    if (t + warps * kTokens < tokens) next.load(row + static_cast<int64_t>(warps * kTokens) * a.stride, e0, end, vec);
    constexpr uint32_t kTeam = kFull >> (32 - LANES);
    const bool bad = (__ballot_sync(kFull, nan || (softmax && top == INFINITY)) >> (sub * LANES) & kTeam) != 0;
    if (sums) {
      top = team_max<LANES>(top);
      float sum[V];
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = z[i] > -INFINITY ? key_exp(z[i] - top) : 0.0f;
#pragma unroll
      for (int half = V / 2; half > 0; half /= 2)
#pragma unroll
        for (int i = 0; i < half; ++i) sum[i] += sum[i + half];
      total = team_sum<LANES>(sum[0]);
    }
    // Scores become whole units of a scale from the lowest possible key to the highest, a
    // float's 23 bits by adding 2^23: off by a unit, and by their own errors, in 2^-24 of the
    // row's largest score.  Sigmoid: the exponential's 2 units and its argument's rounding, each
    // times s (1 - s), the sum's 1, the reciprocal's 2 and the bias's 1, below 6.  Softmax: the
    // exponential's 4, its argument's 2 roundings times |d| e^-d, the sum's 9 (of pairs, in a lane
    // and across the team) and the quotient's 5, the bias's 1, below 24.
    const float inv = __fdividef(1.0f, total), most_score = softmax ? inv : 1.0f;
    const float units = __fdividef(8388608.0f - 17000.0f, most_score + 2.0f * bias_max);
    const float off = (softmax ? 0x1.8p-20f : 0x1.8p-22f) * (most_score + bias_max) * units + 1.5f;
    uint32_t key[V], best = 0, second = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t number = kNumber - e0 - i;
      if (scored && !bad) {
        const float b = bias != nullptr ? bias[e0 + i] : 0.0f;
        const float s = (softmax ? key_exp(z[i] - top) * inv : key_sigmoid(z[i])) + b;
        const uint32_t unit = __float_as_uint(fmaf(s + bias_max, units, 8388608.0f + kFirstUnit));
        key[i] = z[i] > -INFINITY && b > -INFINITY ? unit << 9 | number : 0u;
      } else {
        const bool there = z[i] > -INFINITY && (bias == nullptr || bias[e0 + i] > -INFINITY);
        key[i] = there ? (ordered(z[i]) & ~kNumber) | number : 0u;
      }
      second = max(second, min(best, key[i]));
      best = max(best, key[i]);
    }
    bool sure = bias_max < INFINITY || !live;     // no scale holds an infinite bias
    double total64 = 0.0;                         // once it is needed
    // The warp's one answer to whether it has been computed.  Its value is none: of a padded row it
    // is 0, and the lanes that went to compute it again would leave the others at their shuffles.
    bool have_total = false;
    best = max(best, 1u);                         // 1: none left
    if (by_group) {
      uint32_t one = best, other = second;
      for (int o = 1; o < group_lanes; o *= 2) {
        const uint32_t x = __shfl_xor_sync(kFull, one, o), y = __shfl_xor_sync(kFull, other, o);
        other = max(min(one, x), max(other, y));
        one = max(one, x);
      }
      const bool summed = two && !bad;
      uint32_t mine = one >> 9;
      if (summed && one > kNone)
        // of one key alone: as if the other were 0, which lies bias_max above the scale's start
        mine += other > kNone ? other >> 9 : static_cast<uint32_t>(fmaf(bias_max, units, kFirstUnit));
      mine = one > kNone ? mine << 5 | (31 - group) : 0u;
      uint32_t least = 0;
      bool kept = false;
      for (int g = 0; g < r.top_groups; ++g) {
        const uint32_t most = team_max<LANES>(mine);
        if (most != 0) least = most;
        if (mine == most) {
          kept = true;
          mine = 0;
        }
      }
      const uint32_t most = team_max<LANES>(mine);
      const bool exact = !scored || bad;
      if (most != 0)
        sure = sure && (exact ? sizeof(T) == 2 || least >> 5 != most >> 5
                              : static_cast<float>((least >> 5) - (most >> 5)) > 2.0f * off * (summed ? 2.0f : 1.0f));
      if (__any_sync(kFull, !sure)) {
        if (softmax && scored) {
          total64 = exact_sum<T, LANES>(row, e0, end, V, top);
          have_total = true;
        }
        // again from the 64-bit keys of each lane's two best, if its third is far enough below
        uint32_t third = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) third = max(third, key[i] < second ? key[i] : 0u);
        const bool far = second <= kNone || third <= kNone || (exact ? second >> 9 != third >> 9 : static_cast<float>((second >> 9) - (third >> 9)) > 2.0f * off);
        double x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t k = i == 0 ? best : second;
          const int e = static_cast<int>(kNumber - (k & kNumber));
          x[i] = k > kNone ? exact_key(to_f32(row[e]), bias != nullptr ? bias[e] : 0.0f, exact, softmax, top, total64) : -INFINITY;
        }
        double one64 = fmax(x[0], x[1]), other64 = fmin(x[0], x[1]);
        for (int o = 1; o < group_lanes; o *= 2) {
          const double u = __shfl_xor_sync(kFull, one64, o), v = __shfl_xor_sync(kFull, other64, o);
          other64 = fmax(fmin(one64, u), fmax(other64, v));
          one64 = fmax(one64, u);
        }
        const double of = summed && other64 > -INFINITY ? one64 + other64 : one64;
        int before = 0;                    // groups that come before this lane's
        for (int g = 0; g < r.groups; ++g) {
          const double v = __shfl_sync(kFull, of, g * group_lanes, LANES);
          before += v > of || (v == of && g < group);
        }
        const bool all_far = (__ballot_sync(kFull, far) >> (sub * LANES) & kTeam) == kTeam;
        if (!sure && all_far && bias_max < INFINITY) {
          kept = before < r.top_groups && of > -INFINITY;
          sure = true;
        }
      }
      if (!kept) {
        best = 1;
        second = 0;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = kept ? key[i] : 0u;
    }
    const bool sure_of_groups = sure;
    uint32_t mine = 0;
    for (int j = 0; j < r.top_k; ++j) {
      const uint32_t most = team_max<LANES>(best);
      if (l == j) mine = most;
      if (best == most) {
        best = second;
        second = 0;
      }
      if (V > 2 && __any_sync(kFull, best == 0)) {
        if (best == 0) {
#pragma unroll
          for (int i = 0; i < V; ++i) best = max(best, key[i] < most ? key[i] : 0u);
          if (best == 0) best = 1;          // none left
        }
      }
    }
    int id = mine > kNone ? static_cast<int>(kNumber - (mine & kNumber)) : -1;
    // each chosen key is far enough above the one that comes after it
    const uint32_t rest = team_max<LANES>(best);
    uint32_t after = __shfl_down_sync(kFull, mine, 1, LANES);
    if (l == LANES - 1 || l + 1 >= r.top_k) after = rest;
    if (id >= 0 && after > kNone) {
      if (scored && !bad) sure = sure && static_cast<float>((mine >> 9) - (after >> 9)) > 2.0f * off;
      else if (sizeof(T) == 4) sure = sure && mine >> 9 != after >> 9;
    }
    sure = (__ballot_sync(kFull, sure) >> (sub * LANES) & kTeam) == kTeam;      // one answer for the team
    if (__any_sync(kFull, !sure && live)) {
      if (softmax && bias != nullptr && !have_total) total64 = exact_sum<T, LANES>(row, e0, end, V, top);
      // Again from 64-bit keys: as many best as the team has lanes, each in its lane, if the one
      // after them is far enough below the last chosen.
      const bool by_logit = bias == nullptr || bad, grouped = sure_of_groups;
      uint32_t mine64 = l < r.top_k ? mine : 0u;
      for (int j = r.top_k; j < LANES; ++j) {
        const uint32_t most = team_max<LANES>(best);
        if (l == j) mine64 = most;
        if (best == most) {
          best = 1;
#pragma unroll
          for (int i = 0; i < V; ++i) best = max(best, key[i] < most ? key[i] : 0u);
        }
      }
      const uint32_t last = __shfl_sync(kFull, mine, r.top_k - 1, LANES), then = team_max<LANES>(best);
      const bool far = then <= kNone || (scored && !bad ? static_cast<float>((last >> 9) - (then >> 9)) > 2.0f * off : last >> 9 != then >> 9);
      const int e = mine64 > kNone ? static_cast<int>(kNumber - (mine64 & kNumber)) : -1;
      const double x = e >= 0 ? exact_key(to_f32(row[e]), bias != nullptr ? bias[e] : 0.0f, by_logit, softmax, top, total64) : -INFINITY;
      int before = 0, now = -1;
      for (int j = 0; j < LANES; ++j) {
        const double v = __shfl_sync(kFull, x, j, LANES);
        const int other = __shfl_sync(kFull, e, j, LANES);
        before += other >= 0 && (v > x || (v == x && other < e));
      }
      for (int j = 0; j < LANES; ++j) {
        const int place = __shfl_sync(kFull, before, j, LANES), other = __shfl_sync(kFull, e, j, LANES);
        if (other >= 0 && place == l) now = other;
      }
      if (!sure && grouped && far && bias_max < INFINITY) {
        id = l < r.top_k ? now : -1;
        sure = true;
      }
    }
    uint32_t again = __ballot_sync(kFull, !sure && live);
    while (again != 0) {
      const int u = (__ffs(again) - 1) / LANES;
      const bool bad_u = __shfl_sync(kFull, static_cast<int>(bad), u * LANES) != 0;
      const int chosen = choose_exactly(rows + static_cast<int64_t>(t0 + u) * a.stride, bias, bias == nullptr || bad_u, bad_u,
                                        s_all + warp * even_experts, r);
      __syncwarp();
      const int got = __shfl_sync(kFull, chosen, l);
      if (sub == u) id = l < r.top_k ? got : -1;
      again &= ~(kTeam << (u * LANES));
    }
    const float zj = id >= 0 ? to_f32(row[id]) : 0.0f;
    float w = r.scale * weight_of<LANES>(zj, id >= 0, r, top, total);
    if (bad) w = __int_as_float(0x7FFFFFFF);
    if (live && l < r.top_k) {
      const int64_t at = (static_cast<int64_t>(first) + t) * r.top_k + l;
      a.ids[at] = id;
      a.weights[at] = w;
      if (id >= 0) atomicAdd(&s_counts[id], 1);
    }
  }
  if (a.starts == nullptr) return;
  __syncthreads();
  if (gridDim.x == 1) {
    for (int e = threadIdx.x; e < experts; e += 32 * warps) s_before[e] = 0;
    place_chunk(a, first, tokens, s_before, s_counts, reinterpret_cast<int*>(s_all), place_warps(experts, warps), s_scan, true);
  } else {
    for (int e = threadIdx.x; e < experts; e += 32 * warps)
      a.counts[static_cast<int64_t>(blockIdx.x) * a.pitch + e] = s_counts[e];
    let_next_kernel_start();
  }
}

// Every chunk's places from the table of counts, rows of `pitch` (a multiple of four).
__global__ void __launch_bounds__(kPlaceThreads) place_kernel(const RouteArgs a) {
  extern __shared__ int s_place[];
  __shared__ int s_scan[32];
  const int experts = a.router.experts;
  int* before = s_place;
  int* all = before + a.pitch;
  int* of_warp = all + a.pitch;
  for (int e = threadIdx.x; e < 2 * a.pitch; e += kPlaceThreads) before[e] = 0;
  wait_for_previous_kernel();
  __syncthreads();
  // thread = four experts and every `step`-th chunk; sums of whole numbers in any order
  const int quads = a.pitch / 4, step = kPlaceThreads / quads;
  const int q = threadIdx.x % quads, c0 = threadIdx.x / quads;
  if (c0 < step) {
    int4 mine = make_int4(0, 0, 0, 0), whole = mine;
    const int4* table = reinterpret_cast<const int4*>(a.counts) + q;
    for (int c = c0; c < a.chunks; c += 8 * step) {
      int4 n[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        n[u] = make_int4(0, 0, 0, 0);
        if (c + u * step < a.chunks) n[u] = __ldcg(table + static_cast<int64_t>(c + u * step) * quads);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool ahead = c + u * step < static_cast<int>(blockIdx.x);
        whole = make_int4(whole.x + n[u].x, whole.y + n[u].y, whole.z + n[u].z, whole.w + n[u].w);
        if (ahead) mine = make_int4(mine.x + n[u].x, mine.y + n[u].y, mine.z + n[u].z, mine.w + n[u].w);
      }
    }
    atomicAdd(&before[4 * q], mine.x);
    atomicAdd(&before[4 * q + 1], mine.y);
    atomicAdd(&before[4 * q + 2], mine.z);
    atomicAdd(&before[4 * q + 3], mine.w);
    atomicAdd(&all[4 * q], whole.x);
    atomicAdd(&all[4 * q + 1], whole.y);
    atomicAdd(&all[4 * q + 2], whole.z);
    atomicAdd(&all[4 * q + 3], whole.w);
  }
  const int first = blockIdx.x * a.per_chunk;
  place_chunk(a, first, min(a.tokens - first, a.per_chunk), before, all, of_warp, place_warps(experts, 32), s_scan,
              blockIdx.x == 0);
}

// The gradient: a warp takes as many tokens at once as fill its lanes, `wide` each.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kBackWarps) route_backward_kernel(const RouteArgs a, const bool vec) {
  extern __shared__ float s_grad[];
  const adamw_router& r = a.router;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int wide = a.wide, at_once = 32 / wide, sub = lane / wide, j = lane % wide;
  float* mine = s_grad + warp * (32 * V);
  const bool softmax = r.score == ADAMW_SCORE_SOFTMAX;
  const bool dense = softmax && !r.renormalise;
  const int64_t pace = static_cast<int64_t>(gridDim.x) * kBackWarps * at_once;
  for (int i = lane; i < 32 * V; i += 32) mine[i] = 0.0f;
  __syncwarp();
  int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kBackWarps + warp) * at_once;
  int next_id = -1;
  float next_dw = 0.0f;
  const auto fetch = [&](int64_t t) {
    next_id = -1;
    if (j < r.top_k && t < a.tokens) {
      next_id = __ldg(a.ids + t * r.top_k + j);
      next_dw = __ldg(a.dweights + t * r.top_k + j);
    }
  };
  fetch(t0 + sub);
  for (; t0 < a.tokens; t0 += pace) {
    const int64_t t = t0 + sub;
    const T* rows = static_cast<const T*>(a.logits);
    const int id = next_id >= 0 && next_id < r.experts ? next_id : -1;
    const float dw = id >= 0 ? r.scale * next_dw : 0.0f;
    const float zj = id >= 0 ? to_f32(rows[t * a.stride + id]) : 0.0f;
    fetch(t + pace);
    const int many = static_cast<int>(min(static_cast<int64_t>(at_once), a.tokens - t0));
    float top = 0.0f, total = 1.0f;
    if (dense) {
      for (int u = 0; u < many; ++u) {
        T z[V];
        load_row<T, V>(rows + (t0 + u) * a.stride, r.experts, z);
        float m = -INFINITY, sum = 0.0f;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float f = to_f32(z[i]);
          nan = nan || f != f;
          m = fmaxf(m, f);
        }
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float f = to_f32(z[i]);
          sum += f > -INFINITY ? expf(f - m) : 0.0f;
        }
        sum = __any_sync(kFull, nan) ? __int_as_float(0x7FFFFFFF) : warp_sum(sum);
        if (sub == u) {
          top = m;
          total = sum;
        }
      }
    }
    const float w = weight_of<0>(zj, id >= 0, r, top, total, wide);
    float mean = dw * w;
    for (int o = wide / 2; o > 0; o >>= 1) mean += __shfl_xor_sync(kFull, mean, o);
    float d = 0.0f;                               // this lane's chosen logit's gradient
    if (dense) d = w * dw;
    else if (r.renormalise) d = w * (dw - mean) * (softmax ? 1.0f : sigmoid(-zj));
    else d = dw * w * sigmoid(-zj);
    for (int u = 0; u < many; ++u) {
      const bool here = sub == u && id >= 0;
      if (here) mine[id] = d;
      __syncwarp();
      T* out = static_cast<T*>(a.dlogits) + (t0 + u) * a.dstride;
      if (dense) {
        const float m = __shfl_sync(kFull, mean, u * wide), row_top = __shfl_sync(kFull, top, u * wide),
                    row_sum = __shfl_sync(kFull, total, u * wide);
        T z[V];
        load_row<T, V>(rows + (t0 + u) * a.stride, r.experts, z);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float f = to_f32(z[i]);
          const float g = mine[32 * i + lane] - (f > -INFINITY || f != f ? __fdiv_rn(expf(f - row_top), row_sum) * m : 0.0f);
          if (32 * i + lane < r.experts) out[32 * i + lane] = from_f32<T>(g);
        }
      } else if (vec) {                           // rows on the 16-byte grid
        constexpr int kPer = 16 / sizeof(T);
        for (int e = lane * kPer; e < r.experts; e += 32 * kPer) {
          uint4 q;
          uint32_t* word = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) word[i] = __float_as_uint(mine[e + i]);
            else word[i] = pack_pair<T>(make_float2(mine[e + 2 * i], mine[e + 2 * i + 1]));
          }
          __stcs(reinterpret_cast<uint4*>(out + e), q);
        }
      } else {
        for (int e = lane; e < r.experts; e += 32) out[e] = from_f32<T>(mine[e]);
      }
      __syncwarp();
      if (here) mine[id] = 0.0f;
      __syncwarp();
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

template <typename T, int LANES, int V>
cudaError_t route_teams(const RouteArgs& a, cudaStream_t s) {
  constexpr int kGrid = V * sizeof(T) < 16 ? V * sizeof(T) : 16;
  const bool vec = a.router.experts == LANES * V && (a.router.groups == 1 || a.per_group % V == 0) && reinterpret_cast<uintptr_t>(a.logits) % kGrid == 0 &&
                   a.stride * sizeof(T) % kGrid == 0;
  const int need = (a.per_chunk + 32 / LANES - 1) / (32 / LANES), warps = need < 4 ? 4 : need < kTeamWarps ? need : kTeamWarps;
  route_teams_kernel<T, LANES, V><<<a.chunks, 32 * warps, team_smem(a.router.experts, warps), s>>>(a, vec);
  return cudaGetLastError();
}
// Lanes of a token's team, experts of a lane and lanes of a group: the fewest lanes that hold
// them.  0 lanes where none do and a warp takes the token.
struct Team {
  int lanes, experts, group_lanes;
};
Team team_for(const adamw_router& r) {
  const bool by_group = r.groups > 1 && r.top_groups < r.groups;
  const int groups = by_group ? r.groups : 1, per = r.experts / groups;
  for (int lanes = 8; lanes <= 32; lanes *= 2)
    for (int v = 4; v <= 16; v *= 2) {
      const int of_group = by_group ? choice_lanes((per + v - 1) / v) : (per + v - 1) / v;
      if (r.top_k <= lanes && groups * of_group <= lanes) return Team{lanes, v, of_group};
    }
  return Team{0, 0, 0};
}

#define ADAMW_ROUTE_TEAM(t, CALL)                                                             \
  ((t).lanes == 8    ? ((t).experts == 4 ? CALL(8, 4) : (t).experts == 8 ? CALL(8, 8) : CALL(8, 16))     \
   : (t).lanes == 16 ? ((t).experts == 4 ? CALL(16, 4) : (t).experts == 8 ? CALL(16, 8) : CALL(16, 16))  \
                     : ((t).experts == 4 ? CALL(32, 4) : (t).experts == 8 ? CALL(32, 8) : CALL(32, 16)))

template <typename T, int V>
cudaError_t back_width(RouteArgs a, int sms, cudaStream_t s) {
  // the lanes of a choice, or more where that leaves an SM fewer than 16 warps
  a.wide = choice_lanes(a.router.top_k);
  while (a.wide < 32 && static_cast<int64_t>(a.tokens) * a.wide < 32LL * 16 * sms) a.wide *= 2;
  const bool vec = reinterpret_cast<uintptr_t>(a.dlogits) % 16 == 0 && a.dstride * sizeof(T) % 16 == 0 &&
                   a.router.experts * sizeof(T) % 16 == 0;
  const int64_t per_cta = kBackWarps * (32 / a.wide);
  const int64_t ctas = (a.tokens + per_cta - 1) / per_cta, most = 8LL * sms;
  route_backward_kernel<T, V><<<static_cast<unsigned>(ctas < most ? ctas : most), 32 * kBackWarps,
                                kBackWarps * 32 * V * sizeof(float), s>>>(a, vec);
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
cudaError_t route_type(const RouteArgs& a, Team team, cudaStream_t s) {
#define ADAMW_ROUTE_CALL(LANES, V) route_teams<T, LANES, V>(a, s)
  if (team.lanes > 0) return ADAMW_ROUTE_TEAM(team, ADAMW_ROUTE_CALL);
#undef ADAMW_ROUTE_CALL
  route_kernel<T><<<a.chunks, 32 * kRouteWarps, route_smem(a.router.experts), s>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t back_type(const RouteArgs& a, int sms, cudaStream_t s) {
#define ADAMW_ROUTE_CALL(V) back_width<T, V>(a, sms, s)
  return ADAMW_ROUTE_WIDTH(a.router.experts, ADAMW_ROUTE_CALL);
#undef ADAMW_ROUTE_CALL
}
template <typename T, int LANES, int V>
cudaError_t prepare_team() {
  return cudaFuncSetAttribute(route_teams_kernel<T, LANES, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(team_smem(LANES * V, kTeamWarps)));
}
// What the most experts of a kernel take: one plan's must not shrink another's.
template <typename T>
cudaError_t prepare_type(Team team) {
#define ADAMW_ROUTE_CALL(LANES, V) prepare_team<T, LANES, V>()
  if (team.lanes > 0) return ADAMW_ROUTE_TEAM(team, ADAMW_ROUTE_CALL);
#undef ADAMW_ROUTE_CALL
  return cudaFuncSetAttribute(route_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(route_smem(32 * kWarpExperts)));
}
size_t place_smem(int experts) {
  return sizeof(int) * (2 * router_pitch(experts) + experts * place_warps(experts, 32));
}

}  // namespace

int router_chunks(int sms) { return sms; }
int router_pitch(int experts) { return (experts + 3) & ~3; }

cudaError_t prepare_router(const adamw_router& r) {
  const Team team = team_for(r);
  cudaError_t e = prepare_type<float>(team);
  if (e == cudaSuccess) e = prepare_type<__half>(team);
  if (e == cudaSuccess) e = prepare_type<__nv_bfloat16>(team);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 80 << 10);
  return e;
}

cudaError_t launch_route(adamw_dtype dt, RouteArgs a, int sms, cudaStream_t s) {
  // one CTA for what it takes in two turns, up to 64 tokens, which spares the second kernel;
  // else a share of every SM's, a third of a turn at least
  const Team team = team_for(a.router);
  const int turn = team.lanes > 0 ? kTeamWarps * (32 / team.lanes) : kRouteWarps;
  const int64_t most = router_chunks(sms), tokens = a.tokens;        // near 2^31 a sum leaves 32 bits
  int64_t chunks = tokens <= 2 * turn && tokens <= 64 ? 1 : (tokens + turn / 3 - 1) / (turn / 3);
  if (chunks > most) chunks = most;
  a.per_chunk = static_cast<int32_t>((tokens + chunks - 1) / chunks);
  a.chunks = a.per_chunk > 0 ? static_cast<int32_t>((tokens + a.per_chunk - 1) / a.per_chunk) : 1;
  a.pitch = router_pitch(a.router.experts);
  a.per_group = a.router.experts / a.router.groups;
  a.group_factor = ((1 << 20) + a.per_group - 1) / a.per_group;
  a.group_lanes = team.group_lanes;
  cudaError_t e = dt == ADAMW_F32   ? route_type<float>(a, team, s)
                  : dt == ADAMW_F16 ? route_type<__half>(a, team, s)
                                    : route_type<__nv_bfloat16>(a, team, s);
  if (e != cudaSuccess || a.chunks == 1 || a.starts == nullptr) return e;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(a.chunks));
  c.blockDim = dim3(kPlaceThreads);
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
