// api_common.h -- what the files that implement the C ABI share: argument-check helpers, the
// per-device error word and the tensor-map encoder's entry point (both defined in api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "cpattn.h"

namespace cpattn {

// Address of the current device's error word (nullptr when it cannot be looked up).
int* device_error_word();

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode_fn();

// Raises a kernel's dynamic shared-memory limit, once per device (one static object per kernel).
class SmemOptIn {
 public:
  cudaError_t operator()(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? CPATTN_OK : CPATTN_ERR_CUDA; }

inline int elem_size(int dtype) { return dtype == CPATTN_BF16 ? 2 : (dtype == CPATTN_F32 ? 4 : 0); }

}  // namespace cpattn
