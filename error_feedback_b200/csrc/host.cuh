// Host helpers shared by the translation units of the C ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "topk_ef.h"

namespace tke {

constexpr int64_t MAX_N = 2147483647LL;
constexpr size_t ALIGN = 256;

inline size_t align_up(size_t x, size_t a = ALIGN) { return (x + a - 1) / a * a; }

inline bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }

// Bytes of an element of type t (0: no such type).
inline size_t type_size(int32_t t) {
    return t == TOPK_EF_F32 ? 4 : t == TOPK_EF_BF16 || t == TOPK_EF_F16 ? 2 : 0;
}

// Calls f with a value of the C++ type of element type t.
template <typename F>
cudaError_t with_type(int32_t t, F f) {
    switch (t) {
        case TOPK_EF_F32: return f(float{});
        case TOPK_EF_BF16: return f(__nv_bfloat16{});
        default: return f(__half{});
    }
}

// Records the error for topk_ef_last_cuda_error; returns TOPK_EF_ERR_CUDA.
int cuda_fail(cudaError_t e);

// What topk_ef_set_test_flags has set.
int test_flags();

// Bracket a kernel launch for the tracing calls.
void trace_before(cudaStream_t st, const char* name);
void trace_after(cudaStream_t st);

// Launch with programmatic stream serialisation: the kernel may be scheduled
// while the previous kernel on the stream is still running, and waits for it
// (griddepcontrol.wait) before touching anything that kernel produces.
template <typename Kern, typename Arg>
cudaError_t launch_pdl(Kern kernel, dim3 grid, int block, cudaStream_t st, const Arg& arg,
                       size_t smem = 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, arg);
}

// As launch_pdl, with clusters of `cluster` blocks.
template <typename Kern, typename Arg>
cudaError_t launch_clusters(Kern kernel, unsigned grid, unsigned cluster, int block, size_t smem,
                            cudaStream_t st, const Arg& arg) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {cluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, arg);
}

}  // namespace tke
