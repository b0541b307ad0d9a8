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

template <typename T, int G>
__global__ void __launch_bounds__(kCta<G>, kThreadsPerSm<G> / kCta<G>) small_vocab_kernel(const LossArgs a, const Pass pass,
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
  int64_t i = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  // gradients of known rows run from the last row to the first: the pass
  // before ended there, so the end of the logits is still in L2
  auto row_of = [&](int64_t at) { return pass == kPassGrad ? a.rows - 1 - at : at; };
  int64_t next_y = -1;
  float next_w = 0.0f;
  auto look = [&](int64_t at) {
    if (at < a.rows) {
      next_y = label_of(a, row_of(at));
      next_w = weights != nullptr ? weights[row_of(at)] : 1.0f;
    }
  };
  look(i);
  for (; i < a.rows; i += step) {
    const int64_t t = row_of(i);
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
    RowSum r{kLowest, 0.0f};
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
        r = RowSum{kLowest, 0.0f};
        if (lane < G / 32) r = RowSum{part[lane].x, part[lane].y};
        r.join_lanes();
      }
      const Log2Sum l = log2_sum(r);
      const float logp = logp_of(a, zy, l);
      slope = 0.0f;
      if (policy_pass(pass)) {
        const PolicyTerm p = policy_term(a, in, logp);
        slope = p.slope;
        if (tid == 0) {
          acc[1] += p.policy;
          acc[2] += p.kl;
          acc[3] += p.clipped;
        }
      }
      if (tid == 0) {
        a.logps[t] = logp;
        if (a.lse != nullptr) a.lse[t] = lse_of(l);
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
