// block_ops.h -- launch arguments of a block's operators between its matrix
// products: dropout, routing to experts and the experts' rows, group norm.
#pragma once

#include <cstdint>

#include "internal.h"

namespace adamw {

// ---- dropout (dropout.cu)
struct DropoutArgs {
  const void* x;
  const void* residual;        // may be null
  void* y;
  int64_t rows, width, x_stride, r_stride, y_stride;
  uint32_t threshold;          // words below it are dropped
  uint32_t some;               // 0: everything is dropped (p = 1)
  float scale;                 // 1 / (1 - p)
  uint32_t site;
  uint32_t key[20];            // the ten rounds' keys, low word first
  const int32_t* step;         // may be null
};
cudaError_t launch_dropout(adamw_dtype dt, const DropoutArgs& a, cudaStream_t s);

// ---- routing (router.cu)
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kMaxGroups = 32;

struct RouteArgs {
  adamw_router router;
  const void* logits;
  int64_t stride;
  int32_t tokens;
  const float* bias;           // may be null
  float* weights;
  int32_t* ids;
  int32_t* slots;              // null: no places
  int32_t* starts;             // null: no places
  const float* dweights;       // backward
  int32_t wide;                // backward: lanes of a token
  void* dlogits;               // backward
  int64_t dstride;
  int32_t* counts;             // plan-owned: [chunks][pitch]
  int32_t pitch;               // experts, up to a multiple of four
  int32_t per_group;           // experts of a group
  int32_t group_lanes;         // lanes of a group in a team
  int32_t group_factor;        // e * factor >> 20 is the group of e < 1024
  int32_t chunks;              // CTAs that share the tokens, in their order
  int32_t per_chunk;           // tokens of a chunk
};
// Chunks of a plan at most: its table of counts has as many rows.
int router_chunks(int sms);
int router_pitch(int experts);
cudaError_t prepare_router(const adamw_router& router);
cudaError_t launch_route(adamw_dtype dt, RouteArgs a, int sms, cudaStream_t s);
cudaError_t launch_route_backward(adamw_dtype dt, const RouteArgs& a, int sms, cudaStream_t s);
cudaError_t launch_route_balance(const int32_t* starts, int32_t experts, float rate, float* bias,
                                 cudaStream_t s);

// ---- experts' rows (expert_rows.cu)
struct ExpertRowsArgs {
  const void* x;               // dispatch: x; combine backward: dy.  [tokens][width]
  int64_t x_stride;
  const void* ys;              // combine, combine backward.  [n_rows][width]
  int64_t ys_stride;
  void* y;                     // combine: y [tokens]; dispatch: xs, combine backward: dys [n_rows]
  int64_t y_stride;
  const int32_t* slots;
  const float* weights;        // may be null (combine)
  float* dweights;
  int64_t tokens, width, n_rows;
  int32_t top_k;
  int32_t lanes;               // of a row, a power of two
};
cudaError_t launch_dispatch(adamw_dtype dt, ExpertRowsArgs a, int sms, cudaStream_t s);
cudaError_t launch_combine(adamw_dtype dt, ExpertRowsArgs a, int sms, cudaStream_t s);
cudaError_t launch_combine_backward(adamw_dtype dt, ExpertRowsArgs a, int sms, cudaStream_t s);

// ---- group norm (group_norm.cu, group_norm_backward.cu)
struct GroupNormArgs {
  const void* x;
  const void* dy;              // backward
  const void* weight;          // null: 1
  const void* bias;            // null: 0
  void* out;                   // y or dx
  int64_t x_sample, x_position, dy_sample, dy_position, out_sample, out_position;
  float* mean;
  float* rstd;
  void* dweight;               // may be null
  void* dbias;                 // may be null
  int64_t samples, positions;
  int32_t channels, groups;
  int32_t size;                // bytes of an element
  int32_t weight_f32;          // weights are float32, else of the elements' type
  int32_t silu;
  float eps;
  // plan-owned
  float* stats;                // statistics of parts of samples
  float* joined;               // backward: two means per sample and group
  float* columns;              // column sums [2][CTAs][channels]
  uint32_t* words;             // of the CTAs that share samples, 0 between calls
  uint32_t* ticket;            // CTAs that have left the kernel, 0 between calls
  uint32_t* fault;             // nonzero: a bounded wait gave up
  uint64_t wait_ns;            // limit of a wait
};
constexpr int kMaxChannels = 1 << 16;
struct GroupNormSpace {
  int64_t stats, joined, columns, words;   // 4-byte words of each
};
GroupNormSpace group_norm_space(int32_t channels, int32_t groups, int64_t max_samples, int sms);
cudaError_t prepare_group_norm();
cudaError_t prepare_group_norm_backward();
cudaError_t launch_group_norm_forward(adamw_dtype dt, const GroupNormArgs& a, int sms, cudaStream_t s);
cudaError_t launch_group_norm_backward(adamw_dtype dt, const GroupNormArgs& a, int sms, cudaStream_t s);

}  // namespace adamw
