// token_math.cuh -- arithmetic shared by the token-loss kernels.
//
// With z = logits / T, y the row's token, w its weight:
//   logp   = z_y - log sum_j exp z_j
//   dlogits_j = (d loss / d logp) * (1{j = y} - softmax(z)_j) / T
// Everything runs in base 2: with k = log2(e) / T, a_j = z_j k - c for a running
// reference c (the largest z k seen), S = sum_j 2^a_j, and
// logp = (z_y k - c - log2 S) * ln 2.  An fma rounds relative to the small
// difference, so large logits lose nothing, and the softmax is 2^a_j / S.
// Errors with the same sign for every token would add up over the tokens of a
// sequence, whose log ratios nearly cancel, so four of them are kept out: k is
// two float32 (k + k_lo); c is an integer (the ceiling of the largest z k), so
// moving a sum to another reference multiplies it by an exact power of two;
// log2 S takes back the mean error of the hardware's 2^x; and exponentials are
// summed in runs of 8 or 16 before they join a long sum, which would round the
// small ones away.
// That needs z k with its fraction, and no infinity: it holds for |z k| up to
// 2^23.  A running reference starts at -2^23, so a thread that has seen masked
// entries alone (-1e10, the type's lowest value) leaves a sum of 0 there.  A row
// whose largest z k lies beyond either end is summed anew around its largest
// logit m instead, with a_j = (z_j - m) k, which no size of the logits spoils.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "operators.h"
#include "rows.cuh"

namespace adamw {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kFar = 8388608.0f;             // 2^23
constexpr float kFaint = 8.67361738e-19f;      // 2^-60

// ex2.approx is exact at integers and elsewhere low by 4.9e-8 on average,
// whatever the fraction (measured on GB300 over 4 M arguments in [-17, 0); the
// spread around that is 3e-8): in log2 S that is 7.1e-8.
constexpr float kExp2Bias = 7.1e-8f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float arg(const LossArgs& a, float z, float c) {
  return fmaf(z, a.k_lo, fmaf(z, a.k, -c));
}
// The same for a gradient entry.  16-bit gradients leave out the k_lo of an entry's
// distance to c (under 2^-17 of it); the k_lo of c itself is in grad_factor.
template <typename T>
__device__ __forceinline__ float grad_arg(const LossArgs& a, float z, float c) {
  return std::is_same<T, float>::value ? arg(a, z, c) : fmaf(z, a.k, -c);
}

// Integer reference c and S = sum 2^(z k - c); of a far row c is its largest logit
// and s = -sum 2^((z - c) k), NaN with a NaN or +inf logit, -0 with nothing but -inf.
struct RowSum {
  float c, s;
  // Whether c and s are good as they are: not where the reference left the range in
  // which z k - c is, or nothing of weight came above -kFar (terms lost to underflow
  // weigh under 2^-36 of a sum that is not faint), or where s is NaN.
  __device__ __forceinline__ bool ordinary() const {
    return s >= kFaint && s <= 3.40282347e38f && c <= kFar;
  }
  __device__ __forceinline__ bool undefined() const { return isnan(s) && c <= kFar; }
  __device__ __forceinline__ bool far() const { return s < 0.0f; }
  __device__ __forceinline__ void raise(float zk) {
    if (zk > c) {
      const float hi = ceilf(zk);
      s *= exp2_fast(c - hi);
      c = hi;
    }
  }
  // Over the warp, the same in every lane: the largest reference by an integer
  // reduction (floats in integer order), then the sums at that reference.
  __device__ __forceinline__ void join_lanes() {
    const int bits = __float_as_int(c);
    const int top = __reduce_max_sync(kFull, bits ^ ((bits >> 31) & 0x7FFFFFFF));
    const float hi = __int_as_float(top ^ ((top >> 31) & 0x7FFFFFFF));
    s *= exp2_fast(c - hi);
    c = hi;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
  }
};

// c + log2 S of an ordinary sum as an integer plus a small rest, so that a
// difference to z_y k rounds relative to the difference.
struct Log2Sum {
  float whole, rest;
};
__device__ __forceinline__ Log2Sum log2_sum(const RowSum& r) {
  const uint32_t b = __float_as_uint(r.s);
  const float f = __uint_as_float((b & 0x007FFFFFu) | 0x3F800000u);     // [1, 2)
  const float e = static_cast<float>(static_cast<int>(b >> 23) - 127);
  return {r.c + e, log2f(f) + kExp2Bias};
}
__device__ __forceinline__ float logp_of(const LossArgs& a, float zy, const Log2Sum& l) {
  return (fmaf(zy, a.k, -l.whole) + fmaf(zy, a.k_lo, -l.rest)) * kLn2;
}
__device__ __forceinline__ float lse_of(const Log2Sum& l) { return (l.whole + l.rest) * kLn2; }

// What 2^a_j is multiplied by in the gradient's entries.
template <typename T>
__device__ __forceinline__ float grad_factor(const LossArgs& a, const RowSum& r, float coef) {
  const float f = -coef / fabsf(r.s);
  return std::is_same<T, float>::value || r.far() ? f : f * exp2_fast(r.c * a.k_part);
}

// (z - m) / 2 for the largest logit m of a far row: half of it, as the difference
// itself may pass float32.
__device__ __forceinline__ float half_below(float z, float m) { return fmaf(z, 0.5f, -0.5f * m); }
// 2^((z - m) k) of it.
__device__ __forceinline__ float far_power(float half, float k, float k_lo) {
  return exp2_fast(fmaf(half, 2.0f * k_lo, half * (2.0f * k)));
}

// A row's log-probability of a token with logit zy, and log sum exp.
struct RowLog {
  float logp, lse;
};
__device__ __forceinline__ RowLog row_log(const LossArgs& a, const RowSum& r, float zy) {
  const Log2Sum l = log2_sum(r);
  const float lse = lse_of(l);
  // a token far below its row has a log-probability that is its logit but for rounding
  return {fabsf(zy * a.k) < kFar ? logp_of(a, zy, l) : fmaf(zy, a.inv_temp, -lse), lse};
}
// The same of a far row, and of one with a NaN or without a finite logit.
__device__ __forceinline__ RowLog far_row_log(const LossArgs& a, const RowSum& r, float zy) {
  if (!r.far()) return {NAN, r.c == -INFINITY && r.s == 0.0f ? -INFINITY : NAN};
  const float log_s = lse_of(log2_sum(RowSum{0.0f, -r.s}));
  return {fmaf(half_below(zy, r.c), 2.0f * a.inv_temp, -log_s), fmaf(r.c, a.inv_temp, log_s)};
}

__device__ __forceinline__ int64_t label_of(const LossArgs& a, int64_t t) {
  return a.labels64 ? static_cast<const int64_t*>(a.labels)[t]
                    : static_cast<const int32_t*>(a.labels)[t];
}

// Inputs of one row's policy term.
struct PolicyRow {
  float w, adv, old, ref;
};
// What one row adds to the policy loss, and d loss / d logp.
struct PolicyTerm {
  float policy, kl, clipped, slope;
};
__device__ __forceinline__ PolicyTerm policy_term(const LossArgs& a, const PolicyRow& in,
                                                  float logp) {
  const float ratio = a.old_logps != nullptr ? expf(logp - in.old) : 1.0f;
  const float bound = fminf(fmaxf(ratio, a.clip_lo), a.clip_hi);
  // an advantage of 0 takes a ratio past float32 to 0
  auto gain = [&](float r) { return in.adv != 0.0f || isnan(r) ? r * in.adv : 0.0f; };
  const float full = gain(ratio), held = gain(bound);
  const bool cut = held < full;
  PolicyTerm r;
  r.policy = -in.w * (cut ? held : full);
  r.clipped = cut ? in.w : 0.0f;
  r.slope = cut ? 0.0f : -full;
  r.kl = 0.0f;
  if (a.ref_logps != nullptr) {
    // e^x - x - 1 is inf where e^x is, and a term without a coefficient adds
    // nothing, inf or not
    const float x = in.ref - logp;
    const float e = expm1f(x);
    r.kl = in.w * (isinf(e) ? e : e - x);
    if (a.kl_coef > 0.0f) r.slope = fmaf(-a.kl_coef, e, r.slope);
  }
  r.slope *= in.w;
  return r;
}

// stats from the rows' sums { -, policy, KL, clipped weight }.
__device__ __forceinline__ void write_policy_stats(const LossArgs& a, const double (&sum)[4]) {
  const double kl = a.kl_coef > 0.0f ? static_cast<double>(a.kl_coef) * sum[2] : 0.0;
  a.stats[0] = static_cast<float>(sum[1] + kl);
  a.stats[1] = static_cast<float>(sum[1]);
  a.stats[2] = static_cast<float>(sum[2]);
  a.stats[3] = static_cast<float>(sum[3]);
}

// ---- 16-byte words of a row: 8 or 4 elements, in pairs
template <typename T> constexpr int kPerWord = 16 / sizeof(T);

template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float2 (&x)[kPerWord<T> / 2]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  if constexpr (sizeof(T) == 4) {
    x[0] = make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
    x[1] = make_float2(__uint_as_float(v[2]), __uint_as_float(v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = unpack_pair<T>(v[i]);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float2 (&x)[kPerWord<T> / 2]) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
  } else {
    return make_uint4(pack_pair<T>(x[0]), pack_pair<T>(x[1]), pack_pair<T>(x[2]),
                      pack_pair<T>(x[3]));
  }
}

// A word of -inf: it adds nothing to a sum.
template <typename T>
__device__ __forceinline__ uint4 lowest_word() {
  constexpr uint32_t v = sizeof(T) == 4 ? 0xFF800000u
                                        : (std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u);
  return make_uint4(v, v, v, v);
}

// The largest element of N words, NaN ignored (16-bit types two at a time).
template <typename T, int N>
__device__ __forceinline__ float words_max(const uint4 (&w)[N]) {
  if constexpr (sizeof(T) == 4) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(w[i].x), __uint_as_float(w[i].y)),
                         fmaxf(__uint_as_float(w[i].z), __uint_as_float(w[i].w))));
    return m;
  } else {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    T2 m = reinterpret_cast<const T2*>(&w[0])[0];
#pragma unroll
    for (int i = 1; i < 4 * N; ++i) m = __hmax2(m, reinterpret_cast<const T2*>(&w[i / 4])[i % 4]);
    return fmaxf(to_f32(m.x), to_f32(m.y));
  }
}

// Adds the exponentials of N words to the row's sum.
template <typename T, int N>
__device__ __forceinline__ void add_words(const LossArgs& a, const uint4 (&w)[N], RowSum& r) {
  r.raise(words_max<T, N>(w) * a.k);
  const float2 k = both(a.k), k_lo = both(a.k_lo), c = both(-r.c);
  float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float2 x[kPerWord<T> / 2];
    unpack<T>(w[i], x);
#pragma unroll
    for (int j = 0; j < kPerWord<T> / 2; ++j) {
      const float2 e = fma2(x[j], k_lo, fma2(x[j], k, c));
      t = add2(t, make_float2(exp2_fast(e.x), exp2_fast(e.y)));
    }
  }
  r.s += t.x + t.y;
}

// The gradient of a word's logits: 2^a_j * f, plus coef at the token's place
// (`at`, outside [0, elements) when the token is elsewhere).
template <typename T>
__device__ __forceinline__ uint4 grad_word(const LossArgs& a, const uint4& w, float c, float f,
                                           float coef, int at) {
  float2 x[kPerWord<T> / 2];
  unpack<T>(w, x);
#pragma unroll
  for (int j = 0; j < kPerWord<T> / 2; ++j) {
    float2 e = fma2(x[j], both(a.k), both(-c));
    if (std::is_same<T, float>::value) e = fma2(x[j], both(a.k_lo), e);
    x[j] = mul2(make_float2(exp2_fast(e.x), exp2_fast(e.y)), both(f));
  }
  if (static_cast<unsigned>(at) < kPerWord<T>) {
#pragma unroll
    for (int j = 0; j < kPerWord<T> / 2; ++j) {
      if (2 * j == at) x[j].x += coef;
      if (2 * j + 1 == at) x[j].y += coef;
    }
  }
  return pack<T>(x);
}

// The same of a far row: f 2^((z - c) k).
template <typename T>
__device__ __forceinline__ uint4 far_grad_word(const LossArgs& a, const uint4& w, float c, float f,
                                               float coef, int at) {
  float2 x[kPerWord<T> / 2];
  unpack<T>(w, x);
#pragma unroll
  for (int j = 0; j < kPerWord<T> / 2; ++j) {
    x[j].x = f * far_power(half_below(x[j].x, c), a.k, a.k_lo) + (2 * j == at ? coef : 0.0f);
    x[j].y = f * far_power(half_below(x[j].y, c), a.k, a.k_lo) + (2 * j + 1 == at ? coef : 0.0f);
  }
  return pack<T>(x);
}

}  // namespace
}  // namespace adamw
