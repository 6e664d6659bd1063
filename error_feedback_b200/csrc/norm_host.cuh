// Host helpers of the layer norm calls.
#pragma once

#include <cuda_runtime.h>

#include "topk_ef.h"
#include "host.cuh"
#include "kernels_norm.cuh"

namespace tke {

constexpr int SMS = 148;

inline bool norm_sizes_ok(int64_t T, int64_t D) {
    return T >= 0 && T <= MAX_N && D >= 1 && D <= (int64_t)1 << 24;
}

inline bool pointer_ok(const void* p, int32_t type) { return p && aligned(p, type_size(type)); }

inline bool rows16(const void* p, int64_t ld, size_t size) {
    return aligned(p, 16) && (size_t)ld * size % 16 == 0;
}

// Blocks of a kernel that run at once.
template <typename K>
int resident(K kernel, int threads) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess || n < 1)
        n = 1;
    return n * SMS;
}

}  // namespace tke
