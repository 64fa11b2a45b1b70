// What the C entry points that touch the GPU share (api.cu, pages_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "tq_internal.h"

namespace tq {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline tq_status cuda_status(cudaError_t e, const char* where) {
    if (e == cudaSuccess) return TQ_OK;
    return fail(TQ_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

// No exception (an allocation that fails) leaves a C entry.
template <typename F>
tq_status guarded(const char* where, F f) noexcept {
    try {
        return f();
    } catch (...) {
        try {
            return fail(TQ_ERR_CUDA, std::string(where) + ": out of host memory");
        } catch (...) {
            return TQ_ERR_CUDA;
        }
    }
}

}  // namespace tq
