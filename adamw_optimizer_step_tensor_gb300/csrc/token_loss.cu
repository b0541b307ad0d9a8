// token_loss.cu -- losses on the log-probability of one token per row of
// logits, and their gradients.
//
// With z = logits / T, y the row's token, w its weight:
//   logp   = z_y - log sum_j exp z_j
//   dlogits_j = (d loss / d logp) * (1{j = y} - softmax(z)_j) / T
// Everything runs in base 2: with k = log2(e) / T, a_j = z_j k - c for a running
// reference c (the largest z k seen), S = sum_j 2^a_j, and
// logp = (z_y k - c - log2 S) * ln 2.  An fma rounds relative to the small
// difference, so large logits lose nothing, and the softmax is 2^a_j / S.
// Errors with the same sign for every token would add up over the tokens of a
// sequence, whose log ratios nearly cancel, so three of them are kept out: k is
// two float32 (k + k_lo); c is an integer (the ceiling of the largest z k), so
// moving a sum to another reference multiplies it by an exact power of two; and
// log2 S takes back the mean error of the hardware's 2^x.
#include <cmath>

#include "operators.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr int kRowThreads = 256;
constexpr double kLn2 = 0.69314718055994530942;
constexpr float kLowest = -3.40282347e38f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float arg(const LossArgs& a, float z, float c) {
  return fmaf(z, a.k_lo, fmaf(z, a.k, -c));
}
// The same for a gradient entry: 16-bit gradients do not see k_lo.
template <typename T>
__device__ __forceinline__ float grad_arg(const LossArgs& a, float z, float c) {
  return std::is_same<T, float>::value ? arg(a, z, c) : fmaf(z, a.k, -c);
}

// ex2.approx is exact at integers and elsewhere low by 4.9e-8 on average,
// whatever the fraction (measured on GB300 over 4 M arguments in [-17, 0); the
// spread around that is 3e-8): in log2 S that is 7.1e-8.
constexpr double kExp2Bias = 7.1e-8;

// log2 of S in float64: the exponent is exact, the mantissa's logarithm good to
// an ulp of a value below 1.
__device__ __forceinline__ double log2_wide(float s) {
  if (!(s > 0.0f && s <= 3.40282347e38f)) return static_cast<double>(log2f(s));
  int e;
  const float f = frexpf(s, &e);
  return static_cast<double>(e) + static_cast<double>(log2f(f)) + kExp2Bias;
}

// Reference c and S = sum 2^(z k - c).
struct RowSum {
  float c, s;
  __device__ __forceinline__ void join(float c2, float s2) {
    const float hi = fmaxf(c, c2);
    s = s * exp2_fast(c - hi) + s2 * exp2_fast(c2 - hi);
    c = hi;
  }
};

__device__ __forceinline__ int64_t label_of(const LossArgs& a, int64_t t) {
  return a.labels64 ? static_cast<const int64_t*>(a.labels)[t]
                    : static_cast<const int32_t*>(a.labels)[t];
}

// What one row adds to the policy loss, and d loss / d logp.
struct PolicyTerm {
  float policy, kl, clipped, slope;
};
__device__ __forceinline__ PolicyTerm policy_term(const LossArgs& a, int64_t t, float logp) {
  const float w = a.weights[t], adv = a.advantages[t];
  const float ratio = a.old_logps != nullptr ? expf(logp - a.old_logps[t]) : 1.0f;
  const float bound = fminf(fmaxf(ratio, a.clip_lo), a.clip_hi);
  const bool cut = bound * adv < ratio * adv;
  PolicyTerm r;
  r.policy = -w * ((cut ? bound : ratio) * adv);
  r.clipped = cut ? w : 0.0f;
  r.slope = cut ? 0.0f : -adv * ratio;
  r.kl = 0.0f;
  if (a.ref_logps != nullptr) {
    const float x = a.ref_logps[t] - logp;
    const float e = expm1f(x);
    r.kl = w * (e - x);
    r.slope = fmaf(-a.kl_coef, e, r.slope);
  }
  r.slope *= w;
  return r;
}

template <typename T, LossKind KIND>
__global__ void __launch_bounds__(kRowThreads) row_loss_kernel(const LossArgs a) {
  __shared__ float s_c[kRowThreads / 32], s_s[kRowThreads / 32];
  const int tid = threadIdx.x;
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  const float out_scale = a.inv_temp * (a.grad_scale != nullptr ? *a.grad_scale : 1.0f);
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const T* const z = static_cast<const T*>(a.logits) + t * a.stride;
    T* const dz = a.dlogits != nullptr ? static_cast<T*>(a.dlogits) + t * a.dstride : nullptr;
    const int64_t y = label_of(a, t);
    const bool live = y >= 0 && y < a.vocab && (a.weights == nullptr || a.weights[t] != 0.0f);
    if (KIND == kLossPrefer && tid == 0) a.row_coef[t] = 0.0f;
    if (!live) {
      if (tid == 0) {
        a.logps[t] = 0.0f;
        if (a.lse != nullptr) a.lse[t] = 0.0f;
      }
      if (KIND == kLossPolicy && dz != nullptr)
        for (int j = tid; j < a.vocab; j += kRowThreads) dz[j] = from_f32<T>(0.0f);
      continue;
    }
    RowSum r{kLowest, 0.0f};
    for (int j = tid; j < a.vocab; j += kRowThreads) {
      const float x = to_f32(z[j]);
      if (x * a.k > r.c) {
        const float c = ceilf(x * a.k);
        r.s *= exp2_fast(r.c - c);
        r.c = c;
      }
      r.s += exp2_fast(arg(a, x, r.c));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      r.join(__shfl_xor_sync(kFull, r.c, o), __shfl_xor_sync(kFull, r.s, o));
    const float zy = to_f32(z[y]);
    __syncthreads();
    if ((tid & 31) == 0) {
      s_c[tid >> 5] = r.c;
      s_s[tid >> 5] = r.s;
    }
    __syncthreads();
    r = RowSum{s_c[0], s_s[0]};
#pragma unroll
    for (int i = 1; i < kRowThreads / 32; ++i) r.join(s_c[i], s_s[i]);
    const double lse2 = static_cast<double>(r.c) + log2_wide(r.s);
    const float logp = static_cast<float>((static_cast<double>(zy) * a.k64 - lse2) * kLn2);
    if (tid == 0) {
      a.logps[t] = logp;
      if (a.lse != nullptr) a.lse[t] = static_cast<float>(lse2 * kLn2);
      if (KIND == kLossPrefer) a.row_stat[t] = make_float2(r.c, r.s);
    }
    if (KIND == kLossPolicy) {
      const PolicyTerm p = policy_term(a, t, logp);
      if (tid == 0) {
        acc[1] += p.policy;
        acc[2] += p.kl;
        acc[3] += p.clipped;
      }
      if (dz != nullptr) {
        const float coef = p.slope * out_scale;
        const float f = -coef / r.s;
        __syncthreads();   // dlogits may be the logits: everyone has read z[y]
        for (int j = tid; j < a.vocab; j += kRowThreads) {
          float d = exp2_fast(grad_arg<T>(a, to_f32(z[j]), r.c)) * f;
          if (j == y) d += coef;
          dz[j] = from_f32<T>(d);
        }
      }
    }
  }
  if (KIND == kLossPolicy) {
    double out[4];
    if (last_cta_sums(acc, a.partial, a.ticket, out)) {
      a.stats[0] = static_cast<float>(out[1] + static_cast<double>(a.kl_coef) * out[2]);
      a.stats[1] = static_cast<float>(out[1]);
      a.stats[2] = static_cast<float>(out[2]);
      a.stats[3] = static_cast<float>(out[3]);
    }
  }
}

// Sum over [lo, hi) of w (logp - ref), in every thread; rows without weight or
// token add nothing.
__device__ __forceinline__ bool pref_live(const LossArgs& a, int64_t t, float& w) {
  const int64_t y = label_of(a, t);
  w = a.weights != nullptr ? a.weights[t] : 1.0f;
  return w != 0.0f && y >= 0 && y < a.vocab;
}
__device__ double sequence_sum(const LossArgs& a, int64_t lo, int64_t hi, double* s_warp) {
  double x = 0.0;
  for (int64_t t = lo + threadIdx.x; t < hi; t += kRowThreads) {
    float w;
    if (pref_live(a, t, w))
      x += static_cast<double>(w) * (static_cast<double>(a.logps[t]) - a.ref_logps[t]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0;
  for (int i = 0; i < kRowThreads / 32; ++i) x += s_warp[i];
  return x;
}

// -log sigmoid(d)
__device__ __forceinline__ double minus_log_sigmoid(double d) {
  return log1p(exp(-fabs(d))) + fmax(-d, 0.0);
}

// One CTA per pair: both sequences' rewards, the pair's loss, and
// d loss / d logp of their rows.
__global__ void __launch_bounds__(kRowThreads) pair_kernel(const LossArgs a) {
  __shared__ double s_warp[kRowThreads / 32];
  const int p = blockIdx.x;
  int64_t lo[2], hi[2];
  double sum[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int s = p + side * a.pairs;
    lo[side] = min(max(static_cast<int64_t>(a.starts[s]), (int64_t)0), a.rows);
    hi[side] = min(max(static_cast<int64_t>(a.starts[s + 1]), lo[side]), a.rows);
    sum[side] = sequence_sum(a, lo[side], hi[side], s_warp);
  }
  const double beta = a.beta, e = a.smoothing;
  const double chosen = beta * sum[0], rejected = beta * sum[1], d = chosen - rejected;
  // d loss / d d = e - sigmoid(-d), over the pairs' mean
  const double sig = d >= 0.0 ? exp(-d) / (1.0 + exp(-d)) : 1.0 / (1.0 + exp(d));
  const float slope = static_cast<float>((e - sig) * beta / a.pairs);
  if (threadIdx.x == 0) {
    a.rewards[p] = static_cast<float>(chosen);
    a.rewards[p + a.pairs] = static_cast<float>(rejected);
  }
#pragma unroll
  for (int side = 0; side < 2; ++side)
    for (int64_t t = lo[side] + threadIdx.x; t < hi[side]; t += kRowThreads) {
      float w;
      if (pref_live(a, t, w)) a.row_coef[t] = w * (side == 0 ? slope : -slope);
    }
  const double mine[4] = {(1.0 - e) * minus_log_sigmoid(d) + e * minus_log_sigmoid(-d),
                          d > 0.0 ? 1.0 : 0.0, chosen, rejected};
  double out[4];
  if (last_cta_sums(mine, a.partial, a.ticket, out))
    for (int i = 0; i < 4; ++i) a.stats[i] = static_cast<float>(out[i] / a.pairs);
}

// dlogits of rows whose reference, sum and d loss / d logp are known.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) row_grad_kernel(const LossArgs a) {
  const int tid = threadIdx.x;
  const float out_scale = a.inv_temp * (a.grad_scale != nullptr ? *a.grad_scale : 1.0f);
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const T* const z = static_cast<const T*>(a.logits) + t * a.stride;
    T* const dz = static_cast<T*>(a.dlogits) + t * a.dstride;
    const float coef = a.row_coef[t] * out_scale;
    if (a.row_coef[t] == 0.0f) {
      for (int j = tid; j < a.vocab; j += kRowThreads) dz[j] = from_f32<T>(0.0f);
      continue;
    }
    const int64_t y = label_of(a, t);
    const float2 st = a.row_stat[t];
    const float f = -coef / st.y;
    for (int j = tid; j < a.vocab; j += kRowThreads) {
      float d = exp2_fast(grad_arg<T>(a, to_f32(z[j]), st.x)) * f;
      if (j == y) d += coef;
      dz[j] = from_f32<T>(d);
    }
  }
}

int row_grid(int64_t rows, int sms) {
  const int64_t most = 8LL * sms < kLossMaxCtas ? 8LL * sms : kLossMaxCtas;
  return static_cast<int>(rows < 1 ? 1 : (rows < most ? rows : most));
}

template <typename T>
cudaError_t launch_typed(LossKind kind, const LossArgs& a, int sms, cudaStream_t s) {
  const int grid = row_grid(a.rows, sms);
  switch (kind) {
    case kLossLogps: row_loss_kernel<T, kLossLogps><<<grid, kRowThreads, 0, s>>>(a); break;
    case kLossPolicy: row_loss_kernel<T, kLossPolicy><<<grid, kRowThreads, 0, s>>>(a); break;
    case kLossPrefer:
      row_loss_kernel<T, kLossPrefer><<<grid, kRowThreads, 0, s>>>(a);
      pair_kernel<<<a.pairs, kRowThreads, 0, s>>>(a);
      if (a.dlogits != nullptr && a.rows > 0)
        row_grad_kernel<T><<<grid, kRowThreads, 0, s>>>(a);
      break;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_loss(adamw_dtype dt, LossKind kind, const LossArgs& a, int sms,
                              cudaStream_t s) {
  switch (dt) {
    case ADAMW_F32: return launch_typed<float>(kind, a, sms, s);
    case ADAMW_F16: return launch_typed<__half>(kind, a, sms, s);
    case ADAMW_BF16: return launch_typed<__nv_bfloat16>(kind, a, sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace adamw
