// Argument checks shared by the host sides of the operators around the layer.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

inline bool aligned(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline int status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }
constexpr int64_t kMaxStride = (1LL << 31) - 1;

// A row stride: 0 means contiguous.  False when it is not one.
inline bool stride(int64_t given, int64_t least, long *out) {
  *out = static_cast<long>(given == 0 ? least : given);
  return given == 0 || (given >= least && given <= kMaxStride);
}

}  // namespace moe
