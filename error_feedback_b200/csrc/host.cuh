// Host helpers shared by the translation units of the C ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>
#include <utility>

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

// What an argument takes of the memory: `rows` of `width` bytes, `ld` bytes apart (ld >= width
// where there are several), from lo to before hi.
struct Region {
    uint64_t lo, hi, rows, ld, width;
    Region(const void* p, int64_t n, uint64_t apart, uint64_t bytes)
        : lo(0), hi(0), rows((uint64_t)n), ld(apart), width(bytes) {
        if (!p || n <= 0 || !bytes) return;
        lo = (uint64_t)(uintptr_t)p;
        hi = lo + (rows - 1) * ld + width;
    }
};
inline Region vector_of(const void* p, int64_t n, size_t size) { return {p, 1, 0, (uint64_t)n * size}; }
inline Region rows_of(const void* p, int64_t T, int64_t ld, int64_t n, size_t size) {
    return {p, T, (uint64_t)ld * size, (uint64_t)n * size};
}

// Whether two arguments whose ranges overlap share a byte.  (Columns of one buffer do not.)
inline bool rows_meet(Region a, Region b) {
    if (a.rows > b.rows) std::swap(a, b);
    if (a.rows > 1 && a.ld == b.ld) {
        // the later one's first row lies in the other's as all of its rows do
        if (a.lo < b.lo) std::swap(a, b);
        const uint64_t k = (a.lo - b.lo) / b.ld, at = (a.lo - b.lo) % b.ld;
        return at < b.width || (k + 1 < b.rows && at + a.width > b.ld);
    }
    for (uint64_t i = 0, lo = a.lo; i < a.rows; ++i, lo += a.ld) {
        // the first of the other's rows that ends after lo
        uint64_t j = 0;
        if (lo >= b.lo + b.width) j = b.rows == 1 ? 1 : (lo - b.lo - b.width) / b.ld + 1;
        if (j < b.rows && b.lo + j * b.ld < lo + a.width) return true;
    }
    return false;
}
inline bool meet(const Region& a, const Region& b) { return a.lo < b.hi && b.lo < a.hi && rows_meet(a, b); }

// Whether any of one list shares a byte with any of the other, or two of one list.
inline bool any_meet(std::initializer_list<Region> a, std::initializer_list<Region> b) {
    for (const Region& x : a)
        for (const Region& y : b)
            if (meet(x, y)) return true;
    return false;
}
inline bool any_meet(std::initializer_list<Region> a) {
    for (auto x = a.begin(); x != a.end(); ++x)
        for (auto y = x + 1; y != a.end(); ++y)
            if (meet(*x, *y)) return true;
    return false;
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
