// block_capi.cpp -- the extern "C" entry points of a block's operators between
// its matrix products: dropout, routing, experts' rows, group norm.  Argument
// validation, the plans' workspaces, and launches.
#include <atomic>
#include <cmath>
#include <memory>
#include <new>

#include "block_ops.h"
#include "operators.h"
#include "plan_calls.h"

using namespace adamw;

struct adamw_router_plan {
  int device = -1;
  int sms = 0;
  adamw_router router{};
  int64_t max_tokens = 0;
  int32_t* d_counts = nullptr;
};

struct adamw_group_norm_plan {
  int device = -1;
  int sms = 0;
  int32_t channels = 0, groups = 0;
  int64_t max_samples = 0;
  float eps = 0.0f;
  adamw_activation activation = ADAMW_ACT_NONE;
  uint64_t wait_ns = kNormWaitNs;
  float* d_space = nullptr;      // column sums, statistics, joined ones
  int64_t stats_at = 0, joined_at = 0;
  uint32_t* d_words = nullptr;   // the kernels' words, then the ticket and the fault word
  int64_t n_words = 0;
};

namespace {

// The group norm's kernels ask for their shared memory once on a device.
cudaError_t prepare_group_norm_once(int device) {
  constexpr int kDevices = 64;
  static std::atomic<bool> done[kDevices];
  if (device < kDevices && done[device].load()) return cudaSuccess;
  const cudaError_t e = prepare_group_norm();
  if (e == cudaSuccess && device < kDevices) done[device].store(true);
  return e;
}

void free_router_plan(adamw_router_plan* p) {
  if (!p) return;
  cudaFree(p->d_counts);
  delete p;
}

void free_group_norm_plan(adamw_group_norm_plan* p) {
  if (!p) return;
  cudaFree(p->d_space);
  cudaFree(p->d_words);
  delete p;
}

// Offsets are counted in 64 bits: rows x stride elements of 4 bytes must stay below 2^62.
constexpr int64_t kMaxElements = int64_t{1} << 60;

// A matrix of rows: its pointer, alignment and stride.
adamw_status matrix(const char* name, const void* p, int64_t rows, int64_t width, int64_t stride,
                    int dtype) {
  if (stride < width) return fail(ADAMW_EINVAL, "%s: the row stride is less than the width", name);
  if (rows > 0 && stride > kMaxElements / rows)
    return fail(ADAMW_EUNSUPPORTED, "%s: more than 2^60 elements", name);
  if (rows > 0 && !p) return fail(ADAMW_EINVAL, "%s must be set", name);
  if (!aligned(p, dtype_bytes(dtype)))
    return fail(ADAMW_EALIGN, "%s is not aligned to its element size", name);
  return ADAMW_OK;
}

adamw_status words(const char* name, const void* p, bool needed) {
  if (needed && !p) return fail(ADAMW_EINVAL, "%s must be set", name);
  if (!aligned(p, 4)) return fail(ADAMW_EALIGN, "%s is not 4-byte aligned", name);
  return ADAMW_OK;
}

// What every call on a router plan shares.
adamw_status router_call(const adamw_router_plan* plan, int dtype, int64_t tokens) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  if (!float_dtype(dtype)) return fail(ADAMW_EDTYPE, "unknown dtype %d", dtype);
  if (tokens < 0) return fail(ADAMW_EINVAL, "tokens < 0");
  if (tokens > plan->max_tokens)
    return fail(ADAMW_EINVAL, "%lld tokens, but the plan was made for %lld", (long long)tokens,
                (long long)plan->max_tokens);
  return ADAMW_OK;
}

RouteArgs route_args(const adamw_router_plan* plan, int64_t tokens, const void* logits,
                     int64_t stride) {
  RouteArgs a{};
  a.router = plan->router;
  a.logits = logits;
  a.stride = stride;
  a.tokens = static_cast<int32_t>(tokens);
  a.counts = plan->d_counts;
  return a;
}

// What the three moves of experts' rows share; `moved` is the matrix of n_rows rows.
adamw_status rows_call(const adamw_router_plan* plan, int dtype, int64_t tokens, int64_t width,
                       const int32_t* slots, int64_t n_rows) {
  adamw_status st = router_call(plan, dtype, tokens);
  if (st != ADAMW_OK) return st;
  if (width < 1) return fail(ADAMW_EINVAL, "width < 1");
  if (width > (1 << 30)) return fail(ADAMW_EUNSUPPORTED, "width is more than 2^30");
  if (n_rows < 0) return fail(ADAMW_EINVAL, "the number of rows is < 0");
  return words("slots", slots, tokens > 0);
}

adamw_status group_norm_args(const adamw_group_norm_plan* plan, int dtype, int weight_dtype,
                             int64_t samples, int64_t positions, const void* weight,
                             const void* bias, GroupNormArgs* a) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  if (!float_dtype(dtype) || !float_dtype(weight_dtype))
    return fail(ADAMW_EDTYPE, "unknown dtype %d / %d", dtype, weight_dtype);
  if (weight_dtype != ADAMW_F32 && weight_dtype != dtype)
    return fail(ADAMW_EUNSUPPORTED, "the weight is float32 or of the elements' own dtype");
  if (samples < 0) return fail(ADAMW_EINVAL, "samples < 0");
  if (samples > plan->max_samples)
    return fail(ADAMW_EINVAL, "%lld samples, but the plan was made for %lld", (long long)samples,
                (long long)plan->max_samples);
  if (positions < 1) return fail(ADAMW_EINVAL, "positions < 1: a group of no elements has no mean");
  if (positions > INT32_MAX) return fail(ADAMW_EUNSUPPORTED, "more than 2^31 - 1 positions");
  if (!aligned(weight, dtype_bytes(weight_dtype)) || !aligned(bias, dtype_bytes(weight_dtype)))
    return fail(ADAMW_EALIGN, "a pointer is not aligned to its element size");
  *a = GroupNormArgs{};
  a->weight = weight;
  a->bias = bias;
  a->samples = samples;
  a->positions = positions;
  a->channels = plan->channels;
  a->groups = plan->groups;
  a->eps = plan->eps;
  a->size = static_cast<int32_t>(dtype_bytes(dtype));
  a->weight_f32 = weight_dtype == ADAMW_F32;
  a->silu = plan->activation == ADAMW_ACT_SILU;
  a->columns = plan->d_space;
  a->stats = plan->d_space + plan->stats_at;
  a->joined = plan->d_space + plan->joined_at;
  a->words = plan->d_words;
  a->ticket = plan->d_words + plan->n_words;
  a->fault = a->ticket + 1;
  a->wait_ns = plan->wait_ns;
  return ADAMW_OK;
}

// A channels-last tensor of the call; its strides are taken over for lone samples and positions too.
adamw_status channels_last(const char* name, const adamw_channels_last* t, const GroupNormArgs& a,
                           int dtype, bool written) {
  if (!t) return fail(ADAMW_EINVAL, "%s must be set", name);
  adamw_status st = matrix(name, t->data, a.samples > 0 ? a.positions : 0, a.channels,
                           t->position_stride, dtype);
  if (st != ADAMW_OK) return st;
  const int64_t span = (a.positions - 1) * t->position_stride + a.channels;
  if (t->sample_stride < 0) return fail(ADAMW_EINVAL, "%s: the sample stride is < 0", name);
  if (a.samples > 1) {
    if (t->sample_stride > kMaxElements / a.samples)
      return fail(ADAMW_EUNSUPPORTED, "%s: more than 2^60 elements", name);
    if (written && t->sample_stride < span && a.positions > 1 &&
        t->position_stride < a.samples * t->sample_stride)
      return fail(ADAMW_EINVAL, "%s has overlapping samples", name);
    if (written && t->sample_stride < a.channels)
      return fail(ADAMW_EINVAL, "%s has overlapping samples", name);
  }
  return ADAMW_OK;
}

bool same_strides(const adamw_channels_last* a, const adamw_channels_last* b, int64_t samples,
                  int64_t positions) {
  return (samples < 2 || a->sample_stride == b->sample_stride) &&
         (positions < 2 || a->position_stride == b->position_stride);
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- dropout

adamw_status adamw_dropout(adamw_dtype dtype, int64_t rows, int64_t width, const void* x,
                           int64_t x_stride, const void* residual, int64_t residual_stride, void* y,
                           int64_t y_stride, float p, uint64_t seed, const int32_t* step_dev,
                           uint32_t site, void* stream) {
  if (!float_dtype(dtype)) return fail(ADAMW_EDTYPE, "unknown dtype %d", static_cast<int>(dtype));
  if (rows < 0 || width < 0) return fail(ADAMW_EINVAL, "rows and width must be >= 0");
  if (!(p >= 0.0f && p <= 1.0f)) return fail(ADAMW_EINVAL, "p must lie in [0, 1]");
  const int64_t n = width == 0 ? 0 : rows;
  adamw_status st = matrix("x", x, n, width, x_stride, dtype);
  if (st == ADAMW_OK && residual) st = matrix("residual", residual, n, width, residual_stride, dtype);
  if (st == ADAMW_OK) st = matrix("y", y, n, width, y_stride, dtype);
  if (st == ADAMW_OK) st = words("step_dev", step_dev, false);
  if (st != ADAMW_OK) return st;
  if (n > 1 && ((y == x && y_stride != x_stride) ||
                (y == residual && y_stride != residual_stride)))
    return fail(ADAMW_EINVAL, "y in place of another matrix needs its row stride");
  if (n == 0) return ADAMW_OK;
  DropoutArgs a{};
  a.x = x;
  a.residual = residual;
  a.y = y;
  a.rows = rows;
  a.width = width;
  a.x_stride = x_stride;
  a.r_stride = residual_stride;
  a.y_stride = y_stride;
  // p 2^32 to the nearest whole number: exact from p = 2^-8 up.  It is 2^32 only for p = 1
  // (the next smaller float32 is 1 - 2^-24), where nothing is kept and no scale is needed.
  const double words_dropped = std::nearbyint(static_cast<double>(p) * 4294967296.0);
  a.some = p < 1.0f;
  a.threshold = a.some ? static_cast<uint32_t>(words_dropped) : 0u;
  a.scale = a.some ? static_cast<float>(1.0 / (1.0 - static_cast<double>(p))) : 0.0f;
  a.site = site;
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
  for (int r = 0; r < 10; ++r) {
    a.key[2 * r] = k0;
    a.key[2 * r + 1] = k1;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  a.step = step_dev;
  cudaError_t e = launch_dropout(dtype, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch dropout");
}

// ---------------------------------------------------------------- routing

adamw_status adamw_router_plan_create(const adamw_router* r, int64_t max_tokens,
                                      adamw_router_plan** out) {
  if (!out) return fail(ADAMW_EINVAL, "out is NULL");
  *out = nullptr;
  if (!r) return fail(ADAMW_EINVAL, "the router record is NULL");
  if (r->score != ADAMW_SCORE_SOFTMAX && r->score != ADAMW_SCORE_SIGMOID)
    return fail(ADAMW_EDTYPE, "unknown score %d", r->score);
  if (r->group_score != ADAMW_GROUP_MAX && r->group_score != ADAMW_GROUP_TOP2)
    return fail(ADAMW_EDTYPE, "unknown group score %d", r->group_score);
  if (r->experts < 1 || r->top_k < 1 || r->groups < 1 || r->top_groups < 1 || max_tokens < 0)
    return fail(ADAMW_EINVAL, "experts, top_k, groups and top_groups must be >= 1, max_tokens >= 0");
  if (r->experts > kMaxExperts) return fail(ADAMW_EUNSUPPORTED, "more than %d experts", kMaxExperts);
  if (r->top_k > kMaxTopK) return fail(ADAMW_EUNSUPPORTED, "top_k is more than %d", kMaxTopK);
  if (r->groups > kMaxGroups) return fail(ADAMW_EUNSUPPORTED, "more than %d groups", kMaxGroups);
  if (r->experts % r->groups != 0) return fail(ADAMW_EINVAL, "groups must divide experts");
  if (r->top_groups > r->groups) return fail(ADAMW_EINVAL, "top_groups is more than groups");
  if (r->top_k > r->top_groups * (r->experts / r->groups))
    return fail(ADAMW_EINVAL, "top_k is more than the experts of top_groups groups");
  if (!(r->scale > 0.0f) || !std::isfinite(r->scale))
    return fail(ADAMW_EINVAL, "scale must be finite and > 0");
  if (max_tokens > INT32_MAX / r->top_k)
    return fail(ADAMW_EUNSUPPORTED, "max_tokens * top_k is 2^31 or more");
  int device = -1, sms = 0;
  adamw_status st = here(&device, &sms);
  if (st != ADAMW_OK) return st;
  std::unique_ptr<adamw_router_plan, void (*)(adamw_router_plan*)> p(
      new (std::nothrow) adamw_router_plan, free_router_plan);
  if (!p) return fail(ADAMW_ENOMEM, "out of host memory");
  p->device = device;
  p->sms = sms;
  p->router = *r;
  p->max_tokens = max_tokens;
  cudaError_t e = prepare_router(*r);
  if (e != cudaSuccess) return failed(e, "prepare the routing kernels");
  e = cudaMalloc(&p->d_counts,
                 static_cast<size_t>(router_chunks(sms)) * router_pitch(r->experts) * sizeof(int32_t));
  if (e != cudaSuccess) return failed(e, "cudaMalloc(router plan)", ADAMW_ENOMEM);
  *out = p.release();
  return ADAMW_OK;
}

adamw_status adamw_router_plan_destroy(adamw_router_plan* plan) {
  return destroy(plan, free_router_plan);
}

adamw_status adamw_route(adamw_router_plan* plan, adamw_dtype dtype, int64_t tokens,
                         const void* logits, int64_t row_stride, const float* bias, float* weights,
                         int32_t* ids, int32_t* slots, int32_t* starts, void* stream) {
  adamw_status st = router_call(plan, dtype, tokens);
  if (st != ADAMW_OK) return st;
  if ((st = matrix("logits", logits, tokens, plan->router.experts, row_stride, dtype)) != ADAMW_OK ||
      (st = words("bias", bias, false)) != ADAMW_OK ||
      (st = words("weights", weights, tokens > 0)) != ADAMW_OK ||
      (st = words("ids", ids, tokens > 0)) != ADAMW_OK ||
      (st = words("slots", slots, starts && tokens > 0)) != ADAMW_OK ||
      (st = words("starts", starts, slots != nullptr)) != ADAMW_OK)
    return st;
  RouteArgs a = route_args(plan, tokens, logits, row_stride);
  a.bias = bias;
  a.weights = weights;
  a.ids = ids;
  a.slots = slots;
  a.starts = starts;
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK) return st;
  if (tokens == 0 && !starts) return ADAMW_OK;
  cudaError_t e = launch_route(dtype, a, plan->sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch routing");
}

adamw_status adamw_route_backward(adamw_router_plan* plan, adamw_dtype dtype, int64_t tokens,
                                  const void* logits, int64_t row_stride, const int32_t* ids,
                                  const float* dweights, void* dlogits, int64_t dlogits_stride,
                                  void* stream) {
  adamw_status st = router_call(plan, dtype, tokens);
  if (st != ADAMW_OK) return st;
  const int32_t experts = plan->router.experts;
  if ((st = matrix("logits", logits, tokens, experts, row_stride, dtype)) != ADAMW_OK ||
      (st = matrix("dlogits", dlogits, tokens, experts, dlogits_stride, dtype)) != ADAMW_OK ||
      (st = words("ids", ids, tokens > 0)) != ADAMW_OK ||
      (st = words("dweights", dweights, tokens > 0)) != ADAMW_OK)
    return st;
  if (tokens > 1 && dlogits == logits && dlogits_stride != row_stride)
    return fail(ADAMW_EINVAL, "dlogits in place of the logits needs the logits' row stride");
  RouteArgs a = route_args(plan, tokens, logits, row_stride);
  a.ids = const_cast<int32_t*>(ids);
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.dstride = dlogits_stride;
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK || tokens == 0) return st;
  cudaError_t e = launch_route_backward(dtype, a, plan->sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch routing backward");
}

adamw_status adamw_route_balance(adamw_router_plan* plan, const int32_t* starts, float rate,
                                 float* bias, void* stream) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  adamw_status st = words("starts", starts, true);
  if (st != ADAMW_OK || (st = words("bias", bias, true)) != ADAMW_OK) return st;
  if (!(rate >= 0.0f) || !std::isfinite(rate))
    return fail(ADAMW_EINVAL, "rate must be finite and >= 0");
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK) return st;
  cudaError_t e = launch_route_balance(starts, plan->router.experts, rate, bias,
                                       static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch the balance step");
}

// ---------------------------------------------------------------- experts' rows

adamw_status adamw_route_dispatch(adamw_router_plan* plan, adamw_dtype dtype, int64_t tokens,
                                  int64_t width, const void* x, int64_t x_stride,
                                  const int32_t* slots, void* xs, int64_t xs_rows,
                                  int64_t xs_stride, void* stream) {
  adamw_status st = rows_call(plan, dtype, tokens, width, slots, xs_rows);
  if (st != ADAMW_OK ||
      (st = matrix("x", x, tokens, width, x_stride, dtype)) != ADAMW_OK ||
      (st = matrix("xs", xs, tokens > 0 ? xs_rows : 0, width, xs_stride, dtype)) != ADAMW_OK)
    return st;
  if (xs == x && tokens > 0 && xs_rows > 0) return fail(ADAMW_EINVAL, "xs may not be x");
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK || tokens == 0 || xs_rows == 0)
    return st;
  ExpertRowsArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.y = xs;
  a.y_stride = xs_stride;
  a.slots = slots;
  a.tokens = tokens;
  a.width = width;
  a.n_rows = xs_rows;
  a.top_k = plan->router.top_k;
  cudaError_t e = launch_dispatch(dtype, a, plan->sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch dispatch");
}

adamw_status adamw_route_combine(adamw_router_plan* plan, adamw_dtype dtype, int64_t tokens,
                                 int64_t width, const void* ys, int64_t ys_rows,
                                 int64_t ys_stride, const int32_t* slots, const float* weights,
                                 void* y, int64_t y_stride, void* stream) {
  adamw_status st = rows_call(plan, dtype, tokens, width, slots, ys_rows);
  if (st != ADAMW_OK ||
      (st = matrix("ys", ys, tokens > 0 ? ys_rows : 0, width, ys_stride, dtype)) != ADAMW_OK ||
      (st = matrix("y", y, tokens, width, y_stride, dtype)) != ADAMW_OK ||
      (st = words("weights", weights, false)) != ADAMW_OK)
    return st;
  if (y == ys && tokens > 0) return fail(ADAMW_EINVAL, "y may not be ys");
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK || tokens == 0) return st;
  ExpertRowsArgs a{};
  a.ys = ys;
  a.ys_stride = ys_stride;
  a.y = y;
  a.y_stride = y_stride;
  a.slots = slots;
  a.weights = weights;
  a.tokens = tokens;
  a.width = width;
  a.n_rows = ys_rows;
  a.top_k = plan->router.top_k;
  cudaError_t e = launch_combine(dtype, a, plan->sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch combine");
}

adamw_status adamw_route_combine_backward(adamw_router_plan* plan, adamw_dtype dtype,
                                          int64_t tokens, int64_t width, const void* dy,
                                          int64_t dy_stride, const void* ys, int64_t ys_rows,
                                          int64_t ys_stride, const int32_t* slots,
                                          const float* weights, void* dys, int64_t dys_stride,
                                          float* dweights, void* stream) {
  adamw_status st = rows_call(plan, dtype, tokens, width, slots, ys_rows);
  const int64_t n_rows = tokens > 0 ? ys_rows : 0;
  if (st != ADAMW_OK ||
      (st = matrix("dy", dy, tokens, width, dy_stride, dtype)) != ADAMW_OK ||
      (st = matrix("ys", ys, n_rows, width, ys_stride, dtype)) != ADAMW_OK ||
      (st = matrix("dys", dys, n_rows, width, dys_stride, dtype)) != ADAMW_OK ||
      (st = words("weights", weights, tokens > 0)) != ADAMW_OK ||
      (st = words("dweights", dweights, tokens > 0)) != ADAMW_OK)
    return st;
  if (n_rows > 1 && dys == ys && dys_stride != ys_stride)
    return fail(ADAMW_EINVAL, "dys in place of ys needs its row stride");
  if (n_rows > 0 && dys == dy) return fail(ADAMW_EINVAL, "dys may not be dy");
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK || tokens == 0) return st;
  ExpertRowsArgs a{};
  a.x = dy;
  a.x_stride = dy_stride;
  a.ys = ys;
  a.ys_stride = ys_stride;
  a.y = dys;
  a.y_stride = dys_stride;
  a.slots = slots;
  a.weights = weights;
  a.dweights = dweights;
  a.tokens = tokens;
  a.width = width;
  a.n_rows = ys_rows;
  a.top_k = plan->router.top_k;
  cudaError_t e = launch_combine_backward(dtype, a, plan->sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch combine backward");
}

// ---------------------------------------------------------------- group norm

adamw_status adamw_group_norm_plan_create(int32_t channels, int32_t groups, int64_t max_samples,
                                          float eps, adamw_activation activation,
                                          adamw_group_norm_plan** out) {
  if (!out) return fail(ADAMW_EINVAL, "out is NULL");
  *out = nullptr;
  if (channels < 1 || groups < 1 || max_samples < 0)
    return fail(ADAMW_EINVAL, "channels and groups must be >= 1, max_samples >= 0");
  if (channels > kMaxChannels) return fail(ADAMW_EUNSUPPORTED, "more than %d channels", kMaxChannels);
  if (channels % groups != 0) return fail(ADAMW_EINVAL, "groups must divide channels");
  if (max_samples > (int64_t{1} << 40) / groups)
    return fail(ADAMW_EUNSUPPORTED, "more than 2^40 groups in all");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(ADAMW_EINVAL, "eps must be finite and >= 0");
  if (activation != ADAMW_ACT_NONE && activation != ADAMW_ACT_SILU)
    return fail(ADAMW_EDTYPE, "unknown activation %d", static_cast<int>(activation));
  int device = -1, sms = 0;
  adamw_status st = here(&device, &sms);
  if (st != ADAMW_OK) return st;
  std::unique_ptr<adamw_group_norm_plan, void (*)(adamw_group_norm_plan*)> p(
      new (std::nothrow) adamw_group_norm_plan, free_group_norm_plan);
  if (!p) return fail(ADAMW_ENOMEM, "out of host memory");
  p->device = device;
  p->sms = sms;
  p->channels = channels;
  p->groups = groups;
  p->max_samples = max_samples;
  p->eps = eps;
  p->activation = activation;
  const GroupNormSpace n = group_norm_space(channels, groups, max_samples, sms);
  p->stats_at = (n.columns + 3) & ~int64_t{3};
  p->joined_at = p->stats_at + ((n.stats + 3) & ~int64_t{3});
  p->n_words = n.words;
  cudaError_t e = prepare_group_norm_once(device);
  if (e != cudaSuccess) return failed(e, "prepare the group norm kernels");
  e = cudaMalloc(&p->d_space, (p->joined_at + n.joined) * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc(&p->d_words, (n.words + 2) * sizeof(uint32_t));
  if (e != cudaSuccess) return failed(e, "cudaMalloc(group norm plan)", ADAMW_ENOMEM);
  if ((e = cudaMemset(p->d_words, 0, (n.words + 2) * sizeof(uint32_t))) != cudaSuccess ||
      (e = cudaStreamSynchronize(cudaStreamLegacy)) != cudaSuccess)
    return failed(e, "clear the group norm plan");
  *out = p.release();
  return ADAMW_OK;
}

adamw_status adamw_group_norm_plan_status(adamw_group_norm_plan* plan, uint32_t* fault_bits) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  uint32_t* d_fault = plan->d_words + plan->n_words + 1;
  const adamw_status st = read_fault(plan->device, d_fault, fault_bits);
  if (st != ADAMW_ETIMEOUT) return st;
  cudaError_t e = cudaMemset(d_fault, 0, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
  return e == cudaSuccess ? st : failed(e, "clear the fault word");
}

adamw_status adamw_group_norm_plan_set_wait_limit(adamw_group_norm_plan* plan, int32_t limit_us) {
  if (!plan) return fail(ADAMW_EINVAL, "plan is NULL");
  if (limit_us < 0) return fail(ADAMW_EINVAL, "limit_us < 0");
  plan->wait_ns = static_cast<uint64_t>(limit_us) * 1000u;
  return ADAMW_OK;
}

adamw_status adamw_group_norm_plan_destroy(adamw_group_norm_plan* plan) {
  return destroy(plan, free_group_norm_plan);
}

adamw_status adamw_group_norm_forward(adamw_group_norm_plan* plan, adamw_dtype dtype,
                                      adamw_dtype weight_dtype, int64_t samples, int64_t positions,
                                      const adamw_channels_last* x, const void* weight,
                                      const void* bias, const adamw_channels_last* y, float* mean,
                                      float* rstd, void* stream) {
  GroupNormArgs a;
  adamw_status st = group_norm_args(plan, dtype, weight_dtype, samples, positions, weight, bias, &a);
  if (st != ADAMW_OK || (st = channels_last("x", x, a, dtype, false)) != ADAMW_OK ||
      (st = channels_last("y", y, a, dtype, true)) != ADAMW_OK ||
      (st = words("mean", mean, samples > 0)) != ADAMW_OK ||
      (st = words("rstd", rstd, samples > 0)) != ADAMW_OK)
    return st;
  if (y->data == x->data && !same_strides(x, y, samples, positions))
    return fail(ADAMW_EINVAL, "y in place of x needs x's strides");
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK || samples == 0) return st;
  a.x = x->data;
  a.x_sample = x->sample_stride;
  a.x_position = x->position_stride;
  a.out = const_cast<void*>(y->data);
  a.out_sample = y->sample_stride;
  a.out_position = y->position_stride;
  a.mean = mean;
  a.rstd = rstd;
  cudaError_t e = launch_group_norm_forward(dtype, a, plan->sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch group norm");
}

adamw_status adamw_group_norm_backward(adamw_group_norm_plan* plan, adamw_dtype dtype,
                                       adamw_dtype weight_dtype, int64_t samples,
                                       int64_t positions, const adamw_channels_last* dy,
                                       const adamw_channels_last* x, const void* weight,
                                       const void* bias, const float* mean, const float* rstd,
                                       const adamw_channels_last* dx, void* dweight, void* dbias,
                                       void* stream) {
  GroupNormArgs a;
  adamw_status st = group_norm_args(plan, dtype, weight_dtype, samples, positions, weight, bias, &a);
  if (st != ADAMW_OK || (st = channels_last("dy", dy, a, dtype, false)) != ADAMW_OK ||
      (st = channels_last("x", x, a, dtype, false)) != ADAMW_OK ||
      (st = channels_last("dx", dx, a, dtype, true)) != ADAMW_OK ||
      (st = words("mean", mean, samples > 0)) != ADAMW_OK ||
      (st = words("rstd", rstd, samples > 0)) != ADAMW_OK)
    return st;
  if (!aligned(dweight, dtype_bytes(weight_dtype)) || !aligned(dbias, dtype_bytes(weight_dtype)))
    return fail(ADAMW_EALIGN, "a pointer is not aligned to its element size");
  if ((dx->data == dy->data && !same_strides(dx, dy, samples, positions)) ||
      (dx->data == x->data && !same_strides(dx, x, samples, positions)))
    return fail(ADAMW_EINVAL, "dx in place of another tensor needs its strides");
  if ((st = check_current_device(plan->device, "plan")) != ADAMW_OK) return st;
  a.x = x->data;
  a.x_sample = x->sample_stride;
  a.x_position = x->position_stride;
  a.dy = dy->data;
  a.dy_sample = dy->sample_stride;
  a.dy_position = dy->position_stride;
  a.out = const_cast<void*>(dx->data);
  a.out_sample = dx->sample_stride;
  a.out_position = dx->position_stride;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dweight = dweight;
  a.dbias = dbias;
  cudaError_t e = launch_group_norm_backward(dtype, a, plan->sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ADAMW_OK : failed(e, "launch group norm backward");
}

}  // extern "C"
