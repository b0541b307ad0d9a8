// token_loss_small.cu -- the token losses' row kernel for small vocabularies: a
// group of 32 to 512 threads holds a row's logits in registers (at most 8
// words of 16 bytes each), sums, and writes the gradient from them.  Rows are
// dealt out to the groups of a resident grid in turn.
//
// A row of 64 KB or less keeps an SM's share of DRAM busy for 3 us or less, much
// of which the ring kernel's hand-over from role to role costs by itself (8000
// bf16 rows of 16,384: 145 us there, 84 here); here many independent groups per
// SM overlap one another's waits.  Fetching the next row ahead into shared memory
// was slower (95 us): issue, not load latency, is what the groups share.
#include "token_rows.cuh"

namespace adamw {
namespace {

constexpr int kWordsEach = 8;
// Resident threads per SM: 64 registers each where a row fills a CTA, 80 where
// several rows share one.
template <int G> constexpr int kThreadsPerSm = G >= 256 ? 1024 : 768;

template <int G> constexpr int kCta = G < 128 ? 128 : G;

// A barrier among the G threads of a group.
template <int G>
__device__ __forceinline__ void group_sync(int group) {
  if (G == 32) __syncwarp();
  else if (kCta<G> == G) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(G) : "memory");
}

// The rows' order.  Gradients of known rows run from the last row to the first: the
// pass before ended there, so the end of the logits is still in L2.
__device__ __forceinline__ int64_t row_of(const LossArgs& a, Pass pass, int64_t i) {
  return pass == kPassGrad ? a.rows - 1 - i : i;
}

// This thread's entries of the gradient; each word is read by the thread that
// writes it, as the gradient may take the logits' place.
template <typename T>
__device__ __forceinline__ void far_gradient(const LossArgs& a, int64_t t, int64_t y, const RowSum& r,
                                             float coef, int tid, int threads) {
  const T* const z = static_cast<const T*>(a.logits) + t * a.stride;
  T* const dz = static_cast<T*>(a.dlogits) + t * a.dstride;
  const RowShare<T> share(z, a.vocab, 0, 1);
  const bool same_grid =
      (reinterpret_cast<uintptr_t>(dz) - reinterpret_cast<uintptr_t>(z)) % 16 == 0;
  const float f = coef / r.s;
  for (int m = tid; m < share.words; m += threads) {
    const int64_t first = share.first + static_cast<int64_t>(m) * kPerWord<T>;
    const uint4 w = reinterpret_cast<const uint4*>(share.base)[m];
    const uint4 d = far_grad_word<T>(a, w, r.c, f, coef, static_cast<int>(y - first));
    if (same_grid) {
      *reinterpret_cast<uint4*>(dz + first) = d;
    } else {
      const T* const el = reinterpret_cast<const T*>(&d);
      for (int x = 0; x < kPerWord<T>; ++x) dz[first + x] = el[x];
    }
  }
  const int e = tid < 16 ? ragged_element(share, a.vocab, tid) : -1;
  if (e >= 0) {
    const float d = f * far_power(half_below(to_f32(z[e]), r.c), a.k, a.k_lo);
    dz[e] = from_f32<T>(e == y ? d + coef : d);
  }
}
// What far rows add to the policy loss.
struct PolicySums {
  double policy, kl, clipped;
};

// The far rows of a group (see token_math.cuh), after its others: they are rare,
// and with their code among the rows' the kernel spilled (8000 bf16 rows of 20,001
// took 162 us instead of 146).  Where sums were taken a far row's log-probability
// is kFarMark until now; they are read again from memory, each word by the thread
// that writes its gradient, which may take the logits' place.
constexpr uint32_t kFarMark = 0x7FA5F0F0u;     // a NaN that no instruction gives
template <typename T, int G>
__device__ __noinline__ PolicySums far_rows(const LossArgs& a, Pass pass, float2* s_part) {
  constexpr int kGroups = kCta<G> / G;
  const int group = threadIdx.x / G, tid = threadIdx.x % G;
  const int lane = tid & 31, warp = tid >> 5;
  float2* const part = s_part + group * (G / 32);
  const float out_scale = a.inv_temp * (a.grad_scale != nullptr ? *a.grad_scale : 1.0f);
  PolicySums acc{0.0, 0.0, 0.0};
  group_sync<G>(group);                        // the marks are there
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kGroups + group; i < a.rows;
       i += static_cast<int64_t>(gridDim.x) * kGroups) {
    const int64_t t = row_of(a, pass, i);
    const int64_t y = label_of(a, t);
    if (y < 0 || y >= a.vocab) continue;
    const T* const z = static_cast<const T*>(a.logits) + t * a.stride;
    RowSum r;
    float slope = 0.0f;
    if (sums(pass)) {
      const bool marked = __float_as_uint(a.logps[t]) == kFarMark;
      group_sync<G>(group);                    // every thread has read the mark
      if (!marked) continue;
      r.c = lanes_max(far_max<T>(z, a.vocab, 0, 1, tid, G));
      if (G > 32) {
        if (lane == 0) part[warp].x = r.c;
        group_sync<G>(group);
        r.c = lanes_max(lane < G / 32 ? part[lane].x : -INFINITY);
      }
      r.s = lanes_sum(far_sum<T>(z, a.vocab, 0, 1, tid, G, r.c, a.k, a.k_lo));
      if (G > 32) {
        if (lane == 0) part[warp].y = r.s;
        group_sync<G>(group);
        r.s = lanes_sum(lane < G / 32 ? part[lane].y : 0.0f);
      }
      r.s = -r.s;
      const RowLog l = far_row_log(a, r, to_f32(z[y]));
      if (policy_pass(pass)) {
        const PolicyRow in{a.weights != nullptr ? a.weights[t] : 1.0f, a.advantages[t],
                           a.old_logps != nullptr ? a.old_logps[t] : 0.0f,
                           a.ref_logps != nullptr ? a.ref_logps[t] : 0.0f};
        const PolicyTerm p = policy_term(a, in, l.logp);
        slope = p.slope;
        acc.policy += p.policy;
        acc.kl += p.kl;
        acc.clipped += p.clipped;
      }
      group_sync<G>(group);                    // zy has been read
      if (tid == 0) {
        a.logps[t] = l.logp;
        if (a.lse != nullptr) a.lse[t] = l.lse;
        if (pass == kPassPrefer) a.row_stat[t] = make_float2(r.c, r.s);
      }
    } else {
      slope = a.row_coef[t];
      r = RowSum{a.row_stat[t].x, a.row_stat[t].y};
      if (slope == 0.0f || !r.far()) continue;
    }
    if (!writes_gradient(pass)) continue;
    far_gradient<T>(a, t, y, r, slope * out_scale, tid, G);
  }
  return acc;
}

template <typename T, int G>
__global__ void __launch_bounds__(kCta<G>, kThreadsPerSm<G> / kCta<G>) small_vocab_kernel(const __grid_constant__ LossArgs a, const Pass pass,
                                                              const bool same_grid) {
  constexpr int kGroups = kCta<G> / G;
  let_next_kernel_start();
  wait_for_previous_kernel();
  __shared__ float2 s_part[2][kCta<G> / 32];
  const int group = threadIdx.x / G, tid = threadIdx.x % G;
  const int lane = tid & 31, warp = tid >> 5;
  const float out_scale = a.inv_temp * (a.grad_scale != nullptr ? *a.grad_scale : 1.0f);
  const bool with_sums = sums(pass), with_grad = writes_gradient(pass);
  const float* const weights = pass == kPassGrad ? a.row_coef : a.weights;
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  int turn = 0;
  bool any_far = false;
  int64_t i = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  int64_t next_y = -1;
  float next_w = 0.0f;
  auto look = [&](int64_t at) {
    if (at < a.rows) {
      next_y = label_of(a, row_of(a, pass, at));
      next_w = weights != nullptr ? weights[row_of(a, pass, at)] : 1.0f;
    }
  };
  look(i);
  for (; i < a.rows; i += step) {
    const int64_t t = row_of(a, pass, i);
    const int64_t y = next_y;
    const float w = next_w;
    look(i + step);
    const bool live = y >= 0 && y < a.vocab && w != 0.0f;
    T* const dz = static_cast<T*>(a.dlogits) + t * a.dstride;
    if (pass == kPassPrefer && tid == 0) a.row_coef[t] = 0.0f;
    if (!live) {
      if (with_sums && tid == 0) {
        a.logps[t] = 0.0f;
        if (a.lse != nullptr) a.lse[t] = 0.0f;
      }
      if (with_grad) {
        const RowShare<T> out(dz, a.vocab, 0, 1);
        uint4* const q = reinterpret_cast<uint4*>(const_cast<unsigned char*>(out.base));
        for (int m = tid; m < out.words; m += G) q[m] = make_uint4(0, 0, 0, 0);
        const int e = tid < 16 ? ragged_element(out, a.vocab, tid) : -1;
        if (e >= 0) dz[e] = from_f32<T>(0.0f);
      }
      continue;
    }
    const T* const z = static_cast<const T*>(a.logits) + t * a.stride;
    const RowShare<T> share(z, a.vocab, 0, 1);
    const uint4* const q = reinterpret_cast<const uint4*>(share.base);
    uint4 v[kWordsEach];
#pragma unroll
    for (int m = 0; m < kWordsEach; ++m)
      v[m] = tid + m * G < share.words ? __ldcs(q + tid + m * G) : lowest_word<T>();
    const int e = tid < 16 ? ragged_element(share, a.vocab, tid) : -1;
    const float edge = e >= 0 ? to_f32(z[e]) : 0.0f;
    RowSum r{-kFar, 0.0f};
    float slope;
    if (with_sums) {
      const float zy = to_f32(z[y]);
      PolicyRow in{w, 0.0f, 0.0f, 0.0f};
      if (policy_pass(pass)) {
        in.adv = a.advantages[t];
        if (a.old_logps != nullptr) in.old = a.old_logps[t];
        if (a.ref_logps != nullptr) in.ref = a.ref_logps[t];
      }
#pragma unroll
      for (int m = 0; m < kWordsEach; m += 2)
        if (tid + m * G < share.words) {
          const uint4 two[2] = {v[m], v[m + 1]};
          add_words<T, 2>(a, two, r);
        }
      if (e >= 0) {
        r.raise(edge * a.k);
        r.s += exp2_fast(arg(a, edge, r.c));
      }
      r.join_lanes();
      if (G == 32) group_sync<G>(group);   // dlogits may be the logits: zy has been read
      if (G > 32) {
        // two places in turn, so that one barrier per row is enough
        float2* const part = s_part[turn] + group * (G / 32);
        turn ^= 1;
        if (lane == 0) part[warp] = make_float2(r.c, r.s);
        group_sync<G>(group);
        r = RowSum{-kFar, 0.0f};
        if (lane < G / 32) r = RowSum{part[lane].x, part[lane].y};
        r.join_lanes();
      }
      if (!r.ordinary()) {                 // the same in every thread of the group
        if (tid == 0) a.logps[t] = __uint_as_float(kFarMark);
        any_far = true;
        continue;
      }
      const RowLog l = row_log(a, r, zy);
      slope = 0.0f;
      if (policy_pass(pass)) {
        const PolicyTerm p = policy_term(a, in, l.logp);
        slope = p.slope;
        if (tid == 0) {
          acc[1] += p.policy;
          acc[2] += p.kl;
          acc[3] += p.clipped;
        }
      }
      if (tid == 0) {
        a.logps[t] = l.logp;
        if (a.lse != nullptr) a.lse[t] = l.lse;
        if (pass == kPassPrefer) a.row_stat[t] = make_float2(r.c, r.s);
      }
    } else {
      const float2 st = a.row_stat[t];
      r.c = st.x;
      r.s = st.y;
      slope = w;
    }
    if (!with_grad) continue;
    const float coef = slope * out_scale;
    if (r.far()) {
      any_far = true;
      continue;
    }
    const float f = grad_factor<T>(a, r, coef);
    const int at = static_cast<int>(y - share.first) - tid * kPerWord<T>;
#pragma unroll
    for (int m = 0; m < kWordsEach; ++m)
      if (tid + m * G < share.words) {
        const uint4 d = grad_word<T>(a, v[m], r.c, f, coef, at - m * G * kPerWord<T>);
        T* const out = dz + share.first + (tid + m * G) * kPerWord<T>;
        if (same_grid) {
          __stcs(reinterpret_cast<uint4*>(out), d);
        } else {
          const T* const el = reinterpret_cast<const T*>(&d);
#pragma unroll
          for (int x = 0; x < kPerWord<T>; ++x) out[x] = el[x];
        }
      }
    if (e >= 0) {
      float d = exp2_fast(grad_arg<T>(a, edge, r.c)) * f;
      if (e == y) d += coef;
      dz[e] = from_f32<T>(d);
    }
  }
  if (any_far) {
    const PolicySums far = far_rows<T, G>(a, pass, s_part[0]);
    acc[1] += far.policy;
    acc[2] += far.kl;
    acc[3] += far.clipped;
  }
  if (!policy_pass(pass)) return;
  // the groups' sums in their order, then the CTAs'
  __shared__ double s_acc[kGroups][4];
  double mine[4] = {acc[0], acc[1], acc[2], acc[3]}, out[4];
  if (kGroups > 1) {
    if (tid == 0)
      for (int m = 0; m < 4; ++m) s_acc[group][m] = acc[m];
    __syncthreads();
    if (threadIdx.x == 0)
      for (int g = 1; g < kGroups; ++g)
        for (int m = 0; m < 4; ++m) mine[m] += s_acc[g][m];
  }
  if (last_cta_sums(mine, a.partial, a.ticket, blockIdx.x, gridDim.x, out))
    write_policy_stats(a, out);
}

template <typename T, int G>
cudaError_t resident(int* ctas) {
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
      ctas, small_vocab_kernel<T, G>, kCta<G>, 0);
  return e == cudaSuccess && *ctas < 1 ? cudaErrorInvalidConfiguration : e;
}

template <typename T, int G>
cudaError_t launch_group(Pass pass, const LossArgs& a, bool same_grid, int64_t resident,
                         cudaStream_t s) {
  int64_t ctas = (a.rows + kCta<G> / G - 1) / (kCta<G> / G);
  if (ctas > resident) ctas = resident;
  if (ctas > kLossMaxCtas) ctas = kLossMaxCtas;
  if (ctas < 1) ctas = 1;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>(ctas));
  c.blockDim = dim3(kCta<G>);
  c.stream = s;
  c.attrs = &attr;
  // the second pass may come up while the one before drains
  c.numAttrs = pass == kPassGrad ? early_start(&attr) : 0;
  return cudaLaunchKernelEx(&c, small_vocab_kernel<T, G>, a, pass, same_grid);
}

}  // namespace

template <typename T>
cudaError_t prepare_small_vocab(int sms, int (&ctas)[kSmallGroups]) {
  cudaError_t e = resident<T, 32>(&ctas[0]);
  if (e == cudaSuccess) e = resident<T, 64>(&ctas[1]);
  if (e == cudaSuccess) e = resident<T, 128>(&ctas[2]);
  if (e == cudaSuccess) e = resident<T, 256>(&ctas[3]);
  if (e == cudaSuccess) e = resident<T, 512>(&ctas[4]);
  for (int& c : ctas) c *= sms;
  return e;
}

// The smallest group that holds the row: more rows at once per SM.
template <typename T>
cudaError_t launch_small_vocab(Pass pass, const LossArgs& a, bool same_grid, const int (&ctas)[kSmallGroups],
                               cudaStream_t s) {
  const int64_t words = static_cast<int64_t>(a.vocab) * sizeof(T) / 16;
  if (words <= 32 * kWordsEach) return launch_group<T, 32>(pass, a, same_grid, ctas[0], s);
  if (words <= 64 * kWordsEach) return launch_group<T, 64>(pass, a, same_grid, ctas[1], s);
  if (words <= 128 * kWordsEach) return launch_group<T, 128>(pass, a, same_grid, ctas[2], s);
  if (words <= 256 * kWordsEach) return launch_group<T, 256>(pass, a, same_grid, ctas[3], s);
  return launch_group<T, 512>(pass, a, same_grid, ctas[4], s);
}

#define ADAMW_SMALL_VOCAB(T)                                                                 \
  template cudaError_t prepare_small_vocab<T>(int, int (&)[kSmallGroups]);                              \
  template cudaError_t launch_small_vocab<T>(Pass, const LossArgs&, bool, const int (&)[kSmallGroups], \
                                             cudaStream_t)
ADAMW_SMALL_VOCAB(float);
ADAMW_SMALL_VOCAB(__half);
ADAMW_SMALL_VOCAB(__nv_bfloat16);
#undef ADAMW_SMALL_VOCAB

}  // namespace adamw
