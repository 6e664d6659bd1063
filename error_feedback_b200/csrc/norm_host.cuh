// Host helpers of the layer norm calls.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

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

// Blocks of a kernel that run at once, with `smem` bytes each (which it is allowed to have).
template <typename K>
int resident(K kernel, int threads, size_t smem) {
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess)
        return 0;
    return n * SMS;
}

// The same, found once for each device; 0: the launch cannot work.
struct Resident {
    std::atomic<int> n[64];
    template <typename K>
    int get(K kernel, int threads, size_t smem) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return resident(kernel, threads, smem);
        int v = n[dev].load();
        if (!v) n[dev].store(v = resident(kernel, threads, smem));
        return v;
    }
};

}  // namespace tke
