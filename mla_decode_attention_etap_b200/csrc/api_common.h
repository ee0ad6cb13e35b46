// Host helpers shared by the translation units of the C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace mla {

// Records the error's text for mla_last_cuda_error (per thread) and returns MLA_ERR_CUDA.
int record_cuda_error(cudaError_t e, const char *what);

inline bool is_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace mla
