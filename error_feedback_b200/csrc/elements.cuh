// Element types of the calls beside compress and merge: conversions, 16-byte accesses of
// eight elements, arithmetic on pairs, and the waits of chained launches.
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

// The larger value; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Two values a register pair, two values an instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 parts(f32x2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Two 16-bit elements as such a pair ...
__device__ __forceinline__ f32x2 widen(__nv_bfloat162 w) {
    const uint32_t b = *reinterpret_cast<const uint32_t*>(&w);
    return pair(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u));
}
__device__ __forceinline__ f32x2 widen(__half2 w) {
    const float2 v = __half22float2(w);
    return pair(v.x, v.y);
}
// ... and packs them again.
__device__ __forceinline__ uint32_t narrow(f32x2 a, __nv_bfloat16) {
    const float2 v = parts(a);
    const __nv_bfloat162 w = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&w);
}
__device__ __forceinline__ uint32_t narrow(f32x2 a, __half) {
    const float2 v = parts(a);
    const __half2 w = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&w);
}

template <typename T> struct Twin;
template <> struct Twin<__nv_bfloat16> { typedef __nv_bfloat162 type; static constexpr bool bf16 = true; };
template <> struct Twin<__half> { typedef __half2 type; static constexpr bool bf16 = false; };

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;"); }

}  // namespace tke
