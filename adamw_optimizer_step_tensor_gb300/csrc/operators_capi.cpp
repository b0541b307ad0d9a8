// operators_capi.cpp -- the extern "C" entry points of the operators around
// the step: gradient norm and clip, token losses, layer norm.  Argument
// validation, the plans' workspaces, and launches.
#include <cmath>
#include <limits>
#include <memory>
#include <new>

#include "plan_calls.h"

using namespace adamw;

struct adamw_loss_plan {
  int device = -1;
  LossLimits limits{};
  int64_t max_rows = 0;
  int32_t max_pairs = 0;
  float2* d_stat = nullptr;
  float* d_coef = nullptr;
  double* d_partial = nullptr;   // kLossMaxCtas x 4 sums, then the ticket and the fault word
};

struct adamw_layer_norm_plan {
  int device = -1;
  int sms = 0;
  int32_t width = 0;
  float eps = 0.0f;
  uint64_t wait_ns = kNormWaitNs;
  float* d_partial = nullptr;
  uint32_t* d_fault = nullptr;
};

namespace {

void free_loss_plan(adamw_loss_plan* p) {
  if (!p) return;
  cudaFree(p->d_stat);
  cudaFree(p->d_coef);
  cudaFree(p->d_partial);
  delete p;
}

void free_layer_norm_plan(adamw_layer_norm_plan* p) {
  if (!p) return;
  cudaFree(p->d_partial);
  cudaFree(p->d_fault);
  delete p;
}

constexpr int64_t kMaxPlanRows = int64_t{1} << 40;

// Checks what every token loss shares and fills those launch arguments.
adamw_status loss_args(const adamw_loss_plan* plan, const adamw_logits* z, float* logps,
                       LossArgs* a) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  if (!z) return fail(ADAMW_EINVAL, "the logits record is NULL");
  if (!float_dtype(z->dtype)) return fail(ADAMW_EDTYPE, "unknown logits dtype %d", z->dtype);
  if (z->label_bytes != 4 && z->label_bytes != 8)
    return fail(ADAMW_EDTYPE, "labels must be 4- or 8-byte integers, not %d", z->label_bytes);
  if (z->rows < 0) return fail(ADAMW_EINVAL, "rows < 0");
  if (z->rows > plan->max_rows)
    return fail(ADAMW_EINVAL, "%lld rows, but the plan was made for %lld", (long long)z->rows,
                (long long)plan->max_rows);
  if (z->vocab < 1) return fail(ADAMW_EINVAL, "vocab < 1");
  if (z->vocab > (1 << 30)) return fail(ADAMW_EUNSUPPORTED, "vocab is more than 2^30");
  if (z->row_stride < z->vocab) return fail(ADAMW_EINVAL, "row_stride is less than vocab");
  if (!(z->temperature > 0.0f) || !std::isfinite(z->temperature))
    return fail(ADAMW_EINVAL, "temperature must be finite and > 0");
  *a = LossArgs{};
  if (z->rows > 0) {
    if (!z->logits || !z->labels || !logps)
      return fail(ADAMW_EINVAL, "logits, labels and logps must be set");
    if (!aligned(z->logits, dtype_bytes(z->dtype)) || !aligned(z->labels, z->label_bytes) ||
        !aligned(logps, 4))
      return fail(ADAMW_EALIGN, "a pointer is not aligned to its element size");
  }
  a->logits = z->logits;
  a->stride = z->row_stride;
  a->labels = z->labels;
  a->labels64 = z->label_bytes == 8;
  a->vocab = z->vocab;
  a->rows = z->rows;
  const double inv = 1.0 / static_cast<double>(z->temperature);
  a->inv_temp = static_cast<float>(inv);
  // k rounded down and k_lo > 0, so that -inf k + (-inf) k_lo stays -inf
  const double k = 1.4426950408889634074 * inv;
  a->k = static_cast<float>(k);
  if (a->k > k) a->k = std::nextafterf(a->k, 0.0f);
  a->k_lo = std::fmax(static_cast<float>(k - a->k), 1e-30f);
  a->k_part = a->k_lo / a->k;
  a->logps = logps;
  a->row_stat = plan->d_stat;
  a->row_coef = plan->d_coef;
  a->partial = plan->d_partial;
  a->ticket = reinterpret_cast<uint32_t*>(plan->d_partial + 4 * kLossMaxCtas);
  a->fault = a->ticket + 1;
  return ADAMW_OK;
}

adamw_status gradient_args(const adamw_logits* z, void* dlogits, int64_t stride,
                           const float* grad_scale_dev, LossArgs* a) {
  if (dlogits) {
    if (stride < z->vocab) return fail(ADAMW_EINVAL, "dlogits_stride is less than vocab");
    if (!aligned(dlogits, dtype_bytes(z->dtype)))
      return fail(ADAMW_EALIGN, "dlogits is not aligned to its element size");
    if (dlogits == z->logits && stride != z->row_stride)
      return fail(ADAMW_EINVAL, "dlogits in place of the logits needs the logits' row stride");
  }
  if (!aligned(grad_scale_dev, 4))
    return fail(ADAMW_EALIGN, "grad_scale_dev is not 4-byte aligned");
  a->dlogits = dlogits;
  a->dstride = stride;
  a->grad_scale = grad_scale_dev;
  return ADAMW_OK;
}

adamw_status layer_norm_args(const adamw_layer_norm_plan* plan, int dtype, int weight_dtype,
                             int64_t rows, const void* x, int64_t x_stride, const void* weight,
                             LayerNormArgs* a) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  if (!float_dtype(dtype) || !float_dtype(weight_dtype))
    return fail(ADAMW_EDTYPE, "unknown dtype %d / %d", dtype, weight_dtype);
  if (weight_dtype != ADAMW_F32 && weight_dtype != dtype)
    return fail(ADAMW_EUNSUPPORTED, "the weight is float32 or of the rows' own dtype");
  if (rows < 0) return fail(ADAMW_EINVAL, "rows < 0");
  if (x_stride < plan->width) return fail(ADAMW_EINVAL, "a row stride is less than the width");
  if (rows > 0 && !x) return fail(ADAMW_EINVAL, "x is NULL");
  if (!aligned(x, dtype_bytes(dtype)) || !aligned(weight, dtype_bytes(weight_dtype)))
    return fail(ADAMW_EALIGN, "a pointer is not aligned to its element size");
  *a = LayerNormArgs{};
  a->x = x;
  a->x_stride = x_stride;
  a->weight = weight;
  a->rows = rows;
  a->width = plan->width;
  a->eps = plan->eps;
  a->partial = plan->d_partial;
  a->wait_ns = plan->wait_ns;
  a->fault = plan->d_fault;
  return ADAMW_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- gradient norm

adamw_status adamw_grad_norm(adamw_plan* plan, float max_norm, const float* grad_scale_dev,
                             float* norm_dev, float* clip_scale_dev, float* found_inf_dev,
                             void* stream) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  if (!norm_dev) return fail(ADAMW_EINVAL, "norm_dev is NULL");
  if (!(max_norm > 0.0f)) return fail(ADAMW_EINVAL, "max_norm must be > 0 (INFINITY: no clipping)");
  if (!aligned(grad_scale_dev, 4) || !aligned(norm_dev, 4) || !aligned(clip_scale_dev, 4) ||
      !aligned(found_inf_dev, 4))
    return fail(ADAMW_EALIGN, "a scalar pointer is not 4-byte aligned");
  adamw_status st = check_current_device(plan->device, "plan");
  if (st != ADAMW_OK) return st;
  const NormArgs a{plan->d_tensors, plan->d_chunks, plan->n_chunks, plan->d_norm, grad_scale_dev,
                   max_norm, norm_dev, clip_scale_dev, found_inf_dev};
  cudaError_t e = launch_grad_norm(plan->gdt, a, plan->grid_norm, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch gradient norm");
}

adamw_status adamw_clip_grads(adamw_plan* plan, const float* clip_scale_dev, void* stream) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  if (!clip_scale_dev) return fail(ADAMW_EINVAL, "clip_scale_dev is NULL");
  if (!aligned(clip_scale_dev, 4))
    return fail(ADAMW_EALIGN, "clip_scale_dev is not 4-byte aligned");
  adamw_status st = check_current_device(plan->device, "plan");
  if (st != ADAMW_OK || plan->n_chunks == 0) return st;
  cudaError_t e = launch_clip_grads(plan->gdt, plan->d_tensors, plan->d_chunks, plan->n_chunks,
                                    clip_scale_dev, plan->grid_check,
                                    static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch gradient clip");
}

// ---------------------------------------------------------------- token losses

adamw_status adamw_loss_plan_create(int64_t max_rows, int32_t max_pairs, adamw_loss_plan** out) {
  if (!out) return fail(ADAMW_EINVAL, "out is NULL");
  *out = nullptr;
  if (max_rows < 0 || max_pairs < 0) return fail(ADAMW_EINVAL, "max_rows and max_pairs must be >= 0");
  if (max_rows > kMaxPlanRows)         // 16 TB of statistics; the byte counts wrap at 2^62
    return fail(ADAMW_EUNSUPPORTED, "more than 2^40 rows");
  if (max_pairs > kLossMaxCtas)
    return fail(ADAMW_EUNSUPPORTED, "more than %d pairs", kLossMaxCtas);
  int device = -1, sms = 0;
  adamw_status st = here(&device, &sms);
  if (st != ADAMW_OK) return st;
  std::unique_ptr<adamw_loss_plan, void (*)(adamw_loss_plan*)> p(new (std::nothrow) adamw_loss_plan,
                                                                 free_loss_plan);
  if (!p) return fail(ADAMW_ENOMEM, "out of host memory");
  p->device = device;
  p->max_rows = max_rows;
  p->max_pairs = max_pairs;
  const size_t sums = (4 * kLossMaxCtas + 1) * sizeof(double);
  cudaError_t e = prepare_token_loss(sms, &p->limits);
  if (e != cudaSuccess) return failed(e, "prepare the token loss kernels");
  e = cudaMalloc(&p->d_partial, sums);
  if (e == cudaSuccess && max_rows > 0) {
    e = cudaMalloc(&p->d_stat, static_cast<size_t>(max_rows) * sizeof(float2));
    if (e == cudaSuccess) e = cudaMalloc(&p->d_coef, static_cast<size_t>(max_rows) * sizeof(float));
  }
  if (e != cudaSuccess) return failed(e, "cudaMalloc(loss plan)", ADAMW_ENOMEM);
  if ((e = cudaMemset(p->d_partial, 0, sums)) != cudaSuccess ||
      (e = cudaStreamSynchronize(cudaStreamLegacy)) != cudaSuccess)
    return failed(e, "clear the loss plan");
  *out = p.release();
  return ADAMW_OK;
}

adamw_status adamw_loss_plan_status(const adamw_loss_plan* plan, uint32_t* fault_bits) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  return read_fault(plan->device, reinterpret_cast<uint32_t*>(plan->d_partial + 4 * kLossMaxCtas) + 1,
                    fault_bits);
}

adamw_status adamw_loss_plan_destroy(adamw_loss_plan* plan) { return destroy(plan, free_loss_plan); }

adamw_status adamw_token_logps(adamw_loss_plan* plan, const adamw_logits* z, float* logps,
                               float* lse, void* stream) {
  LossArgs a;
  adamw_status st = loss_args(plan, z, logps, &a);
  if (st != ADAMW_OK) return st;
  if (!aligned(lse, 4)) return fail(ADAMW_EALIGN, "lse is not 4-byte aligned");
  a.lse = lse;
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK || z->rows == 0) return st;
  cudaError_t e = launch_token_loss(static_cast<adamw_dtype>(z->dtype), kLossLogps, a,
                                    plan->limits, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch token log-probabilities");
}

adamw_status adamw_policy_loss(adamw_loss_plan* plan, const adamw_logits* z, const adamw_policy* p,
                               float* stats, float* logps, void* dlogits, int64_t dlogits_stride,
                               void* stream) {
  LossArgs a;
  adamw_status st = loss_args(plan, z, logps, &a);
  if (st != ADAMW_OK) return st;
  if (!p || !stats) return fail(ADAMW_EINVAL, "the policy record and stats must be set");
  if (z->rows > 0 && (!p->weights || !p->advantages))
    return fail(ADAMW_EINVAL, "weights and advantages must be set");
  if (!(p->clip_low >= 0.0f && p->clip_low <= 1.0f) || !(p->clip_high >= 0.0f))
    return fail(ADAMW_EINVAL, "clip_low must lie in [0, 1] and clip_high be >= 0");
  if (!(p->kl_coef >= 0.0f) || !std::isfinite(p->kl_coef))
    return fail(ADAMW_EINVAL, "kl_coef must be finite and >= 0");
  if (p->kl_coef > 0.0f && z->rows > 0 && !p->ref_logps)
    return fail(ADAMW_EINVAL, "a KL term needs ref_logps");
  if (!aligned(p->weights, 4) || !aligned(p->advantages, 4) || !aligned(p->old_logps, 4) ||
      !aligned(p->ref_logps, 4) || !aligned(stats, 4))
    return fail(ADAMW_EALIGN, "a pointer is not 4-byte aligned");
  if ((st = gradient_args(z, dlogits, dlogits_stride, p->grad_scale_dev, &a)) != ADAMW_OK) return st;
  a.weights = p->weights;
  a.advantages = p->advantages;
  a.old_logps = p->old_logps;
  a.ref_logps = p->ref_logps;
  a.clip_lo = 1.0f - p->clip_low;
  a.clip_hi = 1.0f + p->clip_high;
  a.kl_coef = p->kl_coef;
  a.stats = stats;
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK) return st;
  cudaError_t e = launch_token_loss(static_cast<adamw_dtype>(z->dtype), kLossPolicy, a,
                                    plan->limits, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch policy loss");
}

adamw_status adamw_preference_loss(adamw_loss_plan* plan, const adamw_logits* z,
                                   const adamw_preference* p, float* stats, float* rewards,
                                   float* logps, void* dlogits, int64_t dlogits_stride,
                                   void* stream) {
  LossArgs a;
  adamw_status st = loss_args(plan, z, logps, &a);
  if (st != ADAMW_OK) return st;
  if (!p || !stats || !rewards || !p->seq_starts)
    return fail(ADAMW_EINVAL, "the preference record, stats, rewards and seq_starts must be set");
  if (z->rows > 0 && !p->ref_logps) return fail(ADAMW_EINVAL, "ref_logps must be set");
  if (p->n_pairs < 1) return fail(ADAMW_EINVAL, "n_pairs < 1");
  if (p->n_pairs > plan->max_pairs)
    return fail(ADAMW_EINVAL, "%d pairs, but the plan was made for %d", p->n_pairs,
                plan->max_pairs);
  if (!(p->beta > 0.0f) || !std::isfinite(p->beta))
    return fail(ADAMW_EINVAL, "beta must be finite and > 0");
  if (!(p->label_smoothing >= 0.0f && p->label_smoothing < 0.5f))
    return fail(ADAMW_EINVAL, "label_smoothing must lie in [0, 0.5)");
  if (!aligned(p->weights, 4) || !aligned(p->ref_logps, 4) || !aligned(p->seq_starts, 4) ||
      !aligned(stats, 4) || !aligned(rewards, 4))
    return fail(ADAMW_EALIGN, "a pointer is not 4-byte aligned");
  if ((st = gradient_args(z, dlogits, dlogits_stride, p->grad_scale_dev, &a)) != ADAMW_OK) return st;
  a.weights = p->weights;
  a.ref_logps = p->ref_logps;
  a.starts = p->seq_starts;
  a.pairs = p->n_pairs;
  a.beta = p->beta;
  a.smoothing = p->label_smoothing;
  a.stats = stats;
  a.rewards = rewards;
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK) return st;
  cudaError_t e = launch_token_loss(static_cast<adamw_dtype>(z->dtype), kLossPrefer, a,
                                    plan->limits, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch preference loss");
}

// ---------------------------------------------------------------- layer norm

adamw_status adamw_layer_norm_plan_create(int32_t width, float eps, adamw_layer_norm_plan** out) {
  if (!out) return fail(ADAMW_EINVAL, "out is NULL");
  *out = nullptr;
  if (width < 1) return fail(ADAMW_EINVAL, "width < 1");
  if (width > (1 << 30)) return fail(ADAMW_EUNSUPPORTED, "width is more than 2^30");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(ADAMW_EINVAL, "eps must be finite and >= 0");
  int device = -1, sms = 0;
  adamw_status st = here(&device, &sms);
  if (st != ADAMW_OK) return st;
  std::unique_ptr<adamw_layer_norm_plan, void (*)(adamw_layer_norm_plan*)> p(
      new (std::nothrow) adamw_layer_norm_plan, free_layer_norm_plan);
  if (!p) return fail(ADAMW_ENOMEM, "out of host memory");
  p->device = device;
  p->sms = sms;
  p->width = width;
  p->eps = eps;
  const size_t n = 2 * static_cast<size_t>(norm_parts(width, sms)) * width * sizeof(float);
  cudaError_t e = prepare_layer_norm(width);
  if (e != cudaSuccess) return failed(e, "prepare the layer norm kernels");
  e = cudaMalloc(&p->d_partial, n);
  if (e == cudaSuccess) e = cudaMalloc(&p->d_fault, sizeof(uint32_t));
  if (e != cudaSuccess) return failed(e, "cudaMalloc(layer norm plan)", ADAMW_ENOMEM);
  if ((e = cudaMemset(p->d_fault, 0, sizeof(uint32_t))) != cudaSuccess ||
      (e = cudaStreamSynchronize(cudaStreamLegacy)) != cudaSuccess)
    return failed(e, "clear the layer norm plan");
  *out = p.release();
  return ADAMW_OK;
}

adamw_status adamw_layer_norm_plan_status(const adamw_layer_norm_plan* plan, uint32_t* fault_bits) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  return read_fault(plan->device, plan->d_fault, fault_bits);
}

adamw_status adamw_layer_norm_plan_set_wait_limit(adamw_layer_norm_plan* plan, int32_t limit_us) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  if (limit_us < 0) return fail(ADAMW_EINVAL, "limit_us < 0");
  plan->wait_ns = static_cast<uint64_t>(limit_us) * 1000u;
  return ADAMW_OK;
}

adamw_status adamw_layer_norm_plan_destroy(adamw_layer_norm_plan* plan) {
  return destroy(plan, free_layer_norm_plan);
}

adamw_status adamw_layer_norm_forward(adamw_layer_norm_plan* plan, adamw_dtype dtype,
                                      adamw_dtype weight_dtype, int64_t rows, const void* x,
                                      int64_t x_stride, const void* weight, const void* bias,
                                      void* y, int64_t y_stride, float* mean, float* rstd,
                                      void* stream) {
  LayerNormArgs a;
  adamw_status st = layer_norm_args(plan, dtype, weight_dtype, rows, x, x_stride, weight, &a);
  if (st != ADAMW_OK) return st;
  if (rows > 0 && (!y || !mean || !rstd)) return fail(ADAMW_EINVAL, "y, mean and rstd must be set");
  if (y_stride < plan->width) return fail(ADAMW_EINVAL, "a row stride is less than the width");
  if (rows > 1 && y == x && y_stride != x_stride)
    return fail(ADAMW_EINVAL, "y in place of x needs x's row stride");
  if (!aligned(bias, dtype_bytes(weight_dtype)) || !aligned(y, dtype_bytes(dtype)) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return fail(ADAMW_EALIGN, "a pointer is not aligned to its element size");
  a.bias = bias;
  a.y = y;
  a.y_stride = y_stride;
  a.mean = mean;
  a.rstd = rstd;
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK || rows == 0) return st;
  cudaError_t e = launch_layer_norm_forward(dtype, weight_dtype, a, plan->sms,
                                            static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch layer norm");
}

adamw_status adamw_layer_norm_backward(adamw_layer_norm_plan* plan, adamw_dtype dtype,
                                       adamw_dtype weight_dtype, int64_t rows, const void* dy,
                                       int64_t dy_stride, const void* x, int64_t x_stride,
                                       const void* weight, const float* mean, const float* rstd,
                                       void* dx, int64_t dx_stride, void* dweight, void* dbias,
                                       void* stream) {
  LayerNormArgs a;
  adamw_status st = layer_norm_args(plan, dtype, weight_dtype, rows, x, x_stride, weight, &a);
  if (st != ADAMW_OK) return st;
  if (rows > 0 && (!dy || !mean || !rstd || !dx))
    return fail(ADAMW_EINVAL, "dy, mean, rstd and dx must be set");
  if (dy_stride < plan->width || dx_stride < plan->width)
    return fail(ADAMW_EINVAL, "a row stride is less than the width");
  if (rows > 1 && ((dx == dy && dx_stride != dy_stride) || (dx == x && dx_stride != x_stride)))
    return fail(ADAMW_EINVAL, "dx in place of another matrix needs its row stride");
  if (!aligned(dy, dtype_bytes(dtype)) || !aligned(dx, dtype_bytes(dtype)) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(dweight, dtype_bytes(weight_dtype)) ||
      !aligned(dbias, dtype_bytes(weight_dtype)))
    return fail(ADAMW_EALIGN, "a pointer is not aligned to its element size");
  a.dy = dy;
  a.dy_stride = dy_stride;
  a.dx = dx;
  a.dx_stride = dx_stride;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dweight = dweight;
  a.dbias = dbias;
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK) return st;
  cudaError_t e = launch_layer_norm_backward(dtype, weight_dtype, a, plan->sms,
                                             static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch layer norm backward");
}

}  // extern "C"
