// operators.h -- launch arguments of the operators around the step: the global
// gradient norm and clip, the token losses, and layer norm.
#pragma once

#include <cstdint>

#include "internal.h"

namespace adamw {

// ---- global gradient norm (grad_norm.cu)
constexpr int kNormCtasPerSm = 4;

struct NormArgs {
  const TensorDesc* tensors;
  const Chunk* chunks;
  int64_t n_chunks;
  double* partial;             // [grid + 1]; the last word holds the ticket, 0 between launches
  const float* grad_scale;     // may be null
  float max_norm;              // +inf: no clipping
  float* norm;
  float* clip_scale;           // may be null
  float* found_inf;            // may be null
};
cudaError_t launch_grad_norm(adamw_dtype gdt, const NormArgs& a, int grid, cudaStream_t s);
cudaError_t launch_clip_grads(adamw_dtype gdt, const TensorDesc* tensors, const Chunk* chunks,
                              int64_t n_chunks, const float* clip_scale, int grid,
                              cudaStream_t s);

// ---- token losses (token_loss.cu)
enum LossKind { kLossLogps = 0, kLossPolicy = 1, kLossPrefer = 2 };

struct LossArgs {
  const void* logits;
  int64_t stride;              // elements between rows of logits
  void* dlogits;               // null: forward only
  int64_t dstride;
  const void* labels;
  int32_t labels64;            // int64 labels, else int32
  int32_t vocab;
  int64_t rows;
  const float* weights;        // null: every row counts
  const float* advantages;     // policy
  const float* old_logps;      // policy; null: the row's own (ratio 1)
  const float* ref_logps;      // policy: null without the KL term; preference: required
  const float* grad_scale;     // may be null
  float k, k_lo;               // log2(e) / temperature = k + k_lo, k_lo > 0
  float k_part;                // k_lo / k
  float inv_temp;
  float clip_lo, clip_hi;      // 1 - low, 1 + high
  float kl_coef;
  float beta, smoothing;       // preference
  const int32_t* starts;       // preference: [2 * pairs + 1]
  int32_t pairs;
  float* logps;
  float* lse;                  // may be null
  float* stats;                // [4]
  float* rewards;              // preference: [2 * pairs]
  // plan-owned
  float2* row_stat;            // per row (reference c, sum of 2^(z k - c))
  float* row_coef;             // per row d loss / d logp
  double* partial;             // [4 per CTA]
  uint32_t* ticket;            // 0 between launches
  uint32_t* fault;             // nonzero: a bounded wait gave up (bit per site)
};
constexpr int kLossMaxCtas = 4096;   // partial sums the plan holds
constexpr int kSmallGroups = 5;      // group sizes of the small-vocabulary kernel
struct LossLimits {
  int sms;
  int clusters[4];             // clusters of 1, 2, 4, 8 CTAs resident at once
  int small_ctas[3][kSmallGroups];        // per adamw_dtype: resident CTAs of the small-vocabulary kernels
};
cudaError_t prepare_token_loss(int sms, LossLimits* lim);
cudaError_t launch_token_loss(adamw_dtype dt, LossKind kind, const LossArgs& a,
                              const LossLimits& lim, cudaStream_t s);

// ---- layer norm (layer_norm.cu)
struct LayerNormArgs {
  const void* x;
  const void* dy;              // backward
  const void* weight;          // null: 1
  const void* bias;            // null: 0
  void* y;                     // forward
  void* dx;                    // backward
  float* mean;
  float* rstd;
  void* dweight;               // may be null
  void* dbias;                 // may be null
  int64_t rows, x_stride, dy_stride, y_stride, dx_stride;
  int32_t width;
  float eps;
  float* partial;              // plan-owned: [2][parts][width]
  int32_t parts;
  int32_t add;                 // add to the partial sums that are there
  int32_t stages;              // rows on their way per group
  int32_t period;              // rows this far apart lie alike on the 16-byte grid
  uint64_t wait_ns;            // limit of a wait
  uint32_t* fault;             // nonzero: a bounded wait gave up
};
constexpr uint64_t kNormWaitNs = 2000000000ull;   // 2 s, unless the plan has another
cudaError_t prepare_layer_norm(int32_t width);
cudaError_t launch_layer_norm_forward(adamw_dtype dt, adamw_dtype wdt, const LayerNormArgs& a,
                                      int sms, cudaStream_t s);
cudaError_t launch_layer_norm_backward(adamw_dtype dt, adamw_dtype wdt, const LayerNormArgs& a,
                                       int sms, cudaStream_t s);
// Rows of column sums the backward pass keeps per plan, at most kNormPartsPerSm per SM.
constexpr int kNormPartsPerSm = 4;
int64_t norm_parts(int32_t width, int sms);

}  // namespace adamw
