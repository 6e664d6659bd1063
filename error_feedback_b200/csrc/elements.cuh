// Element types of the embedding and Muon kernels: conversions, 16-byte
// accesses of eight elements, and the waits of chained launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace tke {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// One rounding to nearest even: what an fp32 result becomes in the output type.
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// Eight consecutive elements; p is 16-byte aligned.  (Plain loads: a chained
// kernel starts before the one that writes its input ends, which the
// read-only cache does not allow for.)
template <typename T>
struct Vec8 {
    uint4 q[sizeof(T) / 2];
};
// 32 bytes of one lane in one access where they are aligned to it: two of 16 at
// a stride of 32 would touch every sector twice (a fill of 2 GB: 4.2 against
// 6.4 TB/s).
__device__ __forceinline__ void load32b(const void* p, uint4* q) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(q[0].x), "=r"(q[0].y), "=r"(q[0].z), "=r"(q[0].w), "=r"(q[1].x),
                   "=r"(q[1].y), "=r"(q[1].z), "=r"(q[1].w)
                 : "l"(p));
}
__device__ __forceinline__ void store32b(void* p, const uint4* q) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(q[0].x),
                 "r"(q[0].y), "r"(q[0].z), "r"(q[0].w), "r"(q[1].x), "r"(q[1].y), "r"(q[1].z),
                 "r"(q[1].w)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T* p) {
    Vec8<T> v;
    const uint4* s = reinterpret_cast<const uint4*>(p);
    if (sizeof(T) == 4 && (uintptr_t)p % 32 == 0) {
        load32b(p, v.q);
    } else {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v.q[i] = s[i];
    }
    return v;
}
template <typename T>
__device__ __forceinline__ float elem8(const Vec8<T>& v, int j) {
    return to_f32(reinterpret_cast<const T*>(&v)[j]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x) {
    Vec8<T> v;
#pragma unroll
    for (int j = 0; j < 8; ++j) reinterpret_cast<T*>(&v)[j] = from_f32<T>(x[j]);
    uint4* d = reinterpret_cast<uint4*>(p);
    if (sizeof(T) == 4 && (uintptr_t)p % 32 == 0) {
        store32b(p, v.q);
    } else {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) d[i] = v.q[i];
    }
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;"); }

}  // namespace tke
