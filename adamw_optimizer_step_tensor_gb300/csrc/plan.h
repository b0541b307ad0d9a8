// plan.h -- the plan behind the opaque adamw_plan handle and the error helpers
// of the entry points.  Host code only.
#pragma once

#include "internal.h"
#include "operators.h"

using namespace adamw;

struct adamw_plan {
  int device = -1;
  adamw_mode mode = ADAMW_MODE_FP32;
  adamw_dtype gdt = ADAMW_F32;
  int32_t n_tensors = 0;
  int64_t total_numel = 0;
  int64_t n_chunks = 0;
  int grid = 1;
  int block_threads = kThreads;   // threads per CTA of the step kernel
  int grid_check = 1;
  TensorDesc* d_tensors = nullptr;
  Chunk* d_chunks = nullptr;
  StepScratch* d_scratch = nullptr;
  QTables* d_qt = nullptr;
  int refine = 1;              // Q8: thresholds per bucket lookup of the current maps
  bool bulk = false;           // launch the bulk-staged step kernel
  // fused check + step (adamw_step_amp): its own chunk table, sized for its own
  // co-resident grid (fp32 and bf16+remainder plans only)
  Chunk* d_chunks_fused = nullptr;
  int64_t n_chunks_fused = 0;
  int grid_fused = 0;
  bool has_slow = false;       // every tensor carries an AdEMAMix slow EMA
  bool has_v = true;           // every tensor carries exp_avg_sq (false: Lion-only plan)
  int grid_sqrt_div = 1;       // grid of the RMSprop / Adagrad kernels (2 CTAs per SM)
  // Adam-mini plans (adamw_mini_plan_create): blocks sharing one v
  bool mini = false;
  int64_t n_blocks = 0, n_red = 0;
  int grid_red = 1;
  // plans small enough to sit in shared memory whole (small_kernels.cu): the
  // tensor table as kernel parameters, one piece of one tensor per CTA
  bool small = false;
  bool small_fused = false;    // adamw_step_amp takes the fused small path too
  SmallArgs small_args{};
  int small_grid = 0;
  int small_smem = 0;
  int small_smem_fused = 0;
  MiniBlock* d_blocks = nullptr;
  int32_t* d_chunk_blk = nullptr;
  int64_t* d_red_chunks = nullptr;
  double* d_partial = nullptr;
  uint32_t* d_arrived = nullptr;
  float* d_blk_r = nullptr;
  // gradient norm (grad_norm.cu): grid_norm partial sums and a ticket
  double* d_norm = nullptr;
  int grid_norm = 1;
};

namespace adamw {

// Records the calling thread's error message (adamw_last_error) and returns st.
adamw_status fail(adamw_status st, const char* fmt, ...);
adamw_status cuda_fail(cudaError_t e, const char* what);
// EINVAL unless `device`, on which `what` was created, is the current one.
adamw_status check_current_device(int device, const char* what);

inline bool aligned(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

}  // namespace adamw
