// Argument checks shared by the C ABI's entry points.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/kmeans_gb300.h"

namespace km {

constexpr int64_t kMaxIndex = 0x7fffffffLL;  // labels and member lists use 32-bit indices

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline int check_ws(const void *ws, size_t ws_bytes, size_t need) {
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return KMEANS_ERR_WORKSPACE;
    if (ws_bytes < need) return KMEANS_ERR_WORKSPACE;
    return KMEANS_OK;
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? KMEANS_OK : KMEANS_ERR_CUDA; }

}  // namespace km
