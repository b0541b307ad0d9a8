// plan_calls.h -- what the entry points of the operators share: errors of the CUDA
// runtime, the current device, fault words and the end of a plan.  Host code only.
#pragma once

#include "plan.h"

namespace adamw {

inline bool float_dtype(int d) { return d == ADAMW_F32 || d == ADAMW_F16 || d == ADAMW_BF16; }
inline size_t dtype_bytes(int d) { return d == ADAMW_F32 ? 4 : 2; }

// A CUDA call's failure.  The runtime keeps it for the thread until it is read: left
// there, the next launch would report it as its own.
inline adamw_status failed(cudaError_t e, const char* what, adamw_status st = ADAMW_ECUDA) {
  cudaGetLastError();
  if (st == ADAMW_ECUDA) return cuda_fail(e, what);
  return fail(st, "%s: %s", what, cudaGetErrorString(e));
}

// The current device and its SM count.
inline adamw_status here(int* device, int* sms) {
  cudaError_t e = cudaGetDevice(device);
  if (e != cudaSuccess) return failed(e, "cudaGetDevice");
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *device);
  if (e != cudaSuccess) return failed(e, "cudaDeviceGetAttribute");
  return ADAMW_OK;
}

// Frees a plan's device memory with its device current, after all work on it.
template <typename PLAN>
adamw_status destroy(PLAN* plan, void (*release)(PLAN*)) {
  if (!plan) return ADAMW_OK;
  int prev = -1;
  cudaGetDevice(&prev);
  cudaSetDevice(plan->device);
  cudaDeviceSynchronize();
  release(plan);
  if (prev >= 0) cudaSetDevice(prev);
  return ADAMW_OK;
}

// Reads a plan's fault word after all work on the device.
inline adamw_status read_fault(int device, const uint32_t* d_fault, uint32_t* fault_bits) {
  adamw_status st = check_current_device(device, "plan");
  if (st != ADAMW_OK) return st;
  cudaError_t e = cudaDeviceSynchronize();
  uint32_t bits = 0;
  if (e == cudaSuccess) e = cudaMemcpy(&bits, d_fault, sizeof bits, cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return failed(e, "read fault word");
  if (fault_bits) *fault_bits = bits;
  if (bits != 0) return fail(ADAMW_ETIMEOUT, "a bounded wait gave up (fault bits 0x%x)", bits);
  return ADAMW_OK;
}

}  // namespace adamw
