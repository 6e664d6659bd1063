// Layer norm over the rows of a matrix.
//
//   mean = 1/D sum x,  rstd = (1/D sum (x - mean)^2 + eps)^(-1/2),  y = (x - mean) rstd w + b
//
// All sums are fp32, of the row less its first element c: at most sqrt(D) deviations
// from the mean, so an offset common to a row costs no bits.  The variance
// is a sum of squares of differences, never a difference of sums: each warp sums the
// squares of the differences from its own elements' mean, and the warps' (count,
// sum, squares) are joined by sum n (mean_w - mean)^2.
//
// A row is held in registers by 8 to 512 threads between the statistics and the result, 8 to
// 64 elements each (32 of fp32): the fewer threads, the less joining, and what is in flight
// is the warps' rows.  (16 elements a thread with the next row loaded ahead took 33
// instructions an element, most of them for joining, and 108 us for 16,384 x 4,096 bf16.)
// Rows past NM_MAX_D columns are read again instead.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "elements.cuh"
#include "topk_ef.h"

namespace tke {

constexpr int NM_MAX_D = 16384;

struct NormParams {
    const void* x;
    const void* w;                 // or null
    const void* b;                 // or null
    void* y;
    float* mean;                   // or null
    float* rstd;                   // or null
    int64_t T, D, ldx, ldy;
    int32_t w_type, b_type;
    float eps, inv_d;
};

__device__ __forceinline__ float load_as(const void* p, int32_t type, int64_t i) {
    if (type == TOPK_EF_F32) return static_cast<const float*>(p)[i];
    if (type == TOPK_EF_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
    return to_f32(static_cast<const __half*>(p)[i]);
}

// The thread's elements of a row of G threads: groups of 8 columns (VEC; 16-byte aligned), or
// columns G apart (rows that start anywhere).  Element e of thread t:
template <int G, bool VEC>
__device__ __forceinline__ int norm_col(int t, int e) {
    return VEC ? ((e / 8) * G + t) * 8 + e % 8 : e * G + t;
}

template <typename T, int N, bool VEC>
struct RowRegs {
    Vec8<T> v[N];                  // 8 N elements
    __device__ __forceinline__ float get(int e) const {
        return to_f32(reinterpret_cast<const T*>(v)[e]);
    }
    // elements 2 i and 2 i + 1
    __device__ __forceinline__ f32x2 two(int i) const {
        if constexpr (sizeof(T) == 4) {
            return reinterpret_cast<const f32x2*>(v)[i];
        } else {
            return widen(reinterpret_cast<const typename Twin<T>::type*>(v)[i]);
        }
    }
    __device__ __forceinline__ void put_two(int i, f32x2 a) {
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<f32x2*>(v)[i] = a;
        } else {
            reinterpret_cast<uint32_t*>(v)[i] = narrow(a, T{});
        }
    }
};

// Loads the thread's elements; those past the row's end are zero.
template <typename T, int G, int N, bool VEC>
__device__ __forceinline__ void load_row(const T* row, int t, int D, RowRegs<T, N, VEC>& r) {
    if (VEC) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (j * G + t) * 8;
            if (c < D) {
                r.v[j] = load8(row + c);
            } else {
#pragma unroll
                for (int k = 0; k < (int)(sizeof(T) / 2); ++k) r.v[j].q[k] = make_uint4(0, 0, 0, 0);
            }
        }
    } else {
        T* e = reinterpret_cast<T*>(r.v);
#pragma unroll
        for (int j = 0; j < 8 * N; ++j) {
            const int c = j * G + t;
            e[j] = c < D ? row[c] : from_f32<T>(0.0f);
        }
    }
}

template <typename T, int G, int N, bool VEC>
__device__ __forceinline__ void store_row(T* row, int t, int D, const RowRegs<T, N, VEC>& r) {
    if (VEC) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (j * G + t) * 8;
            if (c >= D) continue;
            if (sizeof(T) == 4 && (uintptr_t)(row + c) % 32 == 0) {
                store32b(row + c, r.v[j].q);
            } else {
#pragma unroll
                for (int k = 0; k < (int)(sizeof(T) / 2); ++k)
                    reinterpret_cast<uint4*>(row + c)[k] = r.v[j].q[k];
            }
        }
    } else {
        const T* e = reinterpret_cast<const T*>(r.v);
#pragma unroll
        for (int j = 0; j < 8 * N; ++j) {
            const int c = j * G + t;
            if (c < D) row[c] = e[j];
        }
    }
}

// Eight consecutive weights from c on (c and p 16-byte aligned steps), as pairs.
__device__ __forceinline__ void load8_as(const void* p, int32_t type, int c, f32x2* o) {
    if (type == TOPK_EF_F32) {
        RowRegs<float, 1, true> r;
        r.v[0] = load8(static_cast<const float*>(p) + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = r.two(i);
    } else if (type == TOPK_EF_BF16) {
        RowRegs<__nv_bfloat16, 1, true> r;
        r.v[0] = load8(static_cast<const __nv_bfloat16*>(p) + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = r.two(i);
    } else {
        RowRegs<__half, 1, true> r;
        r.v[0] = load8(static_cast<const __half*>(p) + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = r.two(i);
    }
}

// Elements that the lanes of one warp (VEC: or part of it) hold of a row; t0: the row's
// thread that the lanes start at.
template <int G, int N, bool VEC>
__device__ __forceinline__ int warp_count(int t0, int D) {
    constexpr int L = G < 32 ? G : 32;
    int n = 0;
    if (VEC) {
#pragma unroll
        for (int j = 0; j < N; ++j) n += min(max(D - (j * G + t0) * 8, 0), L * 8);
    } else {
#pragma unroll
        for (int j = 0; j < 8 * N; ++j) n += min(max(D - (j * G + t0), 0), L);
    }
    return n;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ f32x2 both(float x) { return pair(x, x); }

template <int G>
constexpr int NORM_BLOCK = G <= 32 ? 128 : G;
// Blocks of an SM: registers for 128 bytes of a row in each thread.
template <typename TX, int G, int N, bool VEC>
constexpr int NORM_RESIDENT =
    (N * (int)sizeof(TX) >= 16 || (!VEC && N >= 4) ? 640 : 1024) / NORM_BLOCK<G>;

// G threads a row, 8 N elements a thread; a block of G threads, or of four warps that
// each hold one row or several.  Bound by the bytes of x and y.
template <typename TX, typename TY, int G, int N, bool VEC>
__global__ void __launch_bounds__(NORM_BLOCK<G>, NORM_RESIDENT<TX, G, N, VEC>) norm_kernel(const NormParams p) {
    constexpr int E = 8 * N, ROWS = NORM_BLOCK<G> / G, L = G < 32 ? G : 32, W = G / 32;
    __shared__ float2 s_part[2][W > 1 ? W : 1];
    pdl_launch();
    const int t = (int)(threadIdx.x % G), D = (int)p.D;
    const TX* x = static_cast<const TX*>(p.x);
    TY* y = static_cast<TY*>(p.y);
    pdl_wait();
    // elements of this warp's lanes, and of the warp that a lane joins for
    const float n = (float)warp_count<G, N, VEC>(t - t % L, D);
    const float inv_n = n > 0.0f ? 1.0f / n : 0.0f;
    const int lane = (int)lane_id();
    const float k = W > 1 && lane < W ? (float)warp_count<G, N, VEC>(lane * 32, D) : 0.0f;
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int flip = 0;
    // (the lanes of a warp go on together: a warp's last rows may not exist)
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < p.T; r0 += step) {
        const int64_t r = r0 + (G <= 32 ? threadIdx.x / G : 0);
        const bool here = r < p.T;
        const TX* row = x + (here ? r : 0) * p.ldx;
        RowRegs<TX, N, VEC> v;
        load_row<TX, G, N, VEC>(row, t, D, v);
        const float c = to_f32(row[0]);
        const auto in = [&](int e) { return norm_col<G, VEC>(t, VEC ? e / 8 * 8 : e) < D; };
        f32x2 sum2 = 0;
        float sum = 0.0f;
        if (VEC) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (in(8 * j)) {
#pragma unroll
                    for (int i = 4 * j; i < 4 * j + 4; ++i) sum2 = add2(sum2, add2(v.two(i), both(-c)));
                }
            const float2 s = parts(sum2);
            sum = s.x + s.y;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) sum += in(e) ? v.get(e) - c : 0.0f;
        }
        // the mean of the warp's elements, less c, and the squares of the distances from it
        float m = lanes_sum<L>(sum) * inv_n;
        f32x2 sq2 = 0;
        float sq = 0.0f;
        if (VEC) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (in(8 * j)) {
#pragma unroll
                    for (int i = 4 * j; i < 4 * j + 4; ++i) {
                        const f32x2 d = add2(add2(v.two(i), both(-c)), both(-m));
                        sq2 = fma2(d, d, sq2);
                    }
                }
            const float2 s = parts(sq2);
            sq = s.x + s.y;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float d = in(e) ? (v.get(e) - c) - m : 0.0f;
                sq = fmaf(d, d, sq);
            }
        }
        sq = lanes_sum<L>(sq);
        if (W > 1) {
            if (lane == 0) s_part[flip][t / 32] = make_float2(m, sq);
            __syncthreads();
            const float2 o = lane < W ? s_part[flip][lane] : make_float2(0.0f, 0.0f);
            flip ^= 1;
            m = warp_sum(k * o.x) * p.inv_d;
            const float d = o.x - m;
            sq = warp_sum(fmaf(k * d, d, o.y));
        }
        const float rstd = rsqrtf(fmaf(sq, p.inv_d, p.eps));
        if (here) {
            RowRegs<TY, N, VEC> o;
            if (VEC) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (!in(8 * j)) continue;
                    f32x2 w[4], b[4];
                    const int col = norm_col<G, VEC>(t, 8 * j);
                    if (p.w) load8_as(p.w, p.w_type, col, w);
                    if (p.b) load8_as(p.b, p.b_type, col, b);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x2 d = add2(add2(v.two(4 * j + i), both(-c)), both(-m));
                        const f32x2 xh = mul2(d, both(rstd));
                        o.put_two(4 * j + i, p.w ? fma2(xh, w[i], p.b ? b[i] : 0ull)
                                                 : p.b ? add2(xh, b[i]) : xh);
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int col = norm_col<G, VEC>(t, e);
                    const float w = p.w && col < D ? load_as(p.w, p.w_type, col) : 1.0f;
                    const float b = p.b && col < D ? load_as(p.b, p.b_type, col) : 0.0f;
                    reinterpret_cast<TY*>(o.v)[e] =
                        from_f32<TY>(fmaf(((v.get(e) - c) - m) * rstd, w, b));
                }
            }
            store_row<TY, G, N, VEC>(y + r * p.ldy, t, D, o);
            if (t == 0) {
                if (p.mean) p.mean[r] = c + m;
                if (p.rstd) p.rstd[r] = rstd;
            }
        }
    }
}

// Rows of any length: one block a row, three passes over it.
constexpr int NL_THREADS = 512;

template <typename TX, typename TY>
__global__ void __launch_bounds__(NL_THREADS) norm_long_kernel(const NormParams p) {
    __shared__ float s_red[33];
    pdl_launch();
    pdl_wait();
    for (int64_t r = blockIdx.x; r < p.T; r += gridDim.x) {
        const TX* x = static_cast<const TX*>(p.x) + r * p.ldx;
        TY* y = static_cast<TY*>(p.y) + r * p.ldy;
        const float first = to_f32(x[0]);
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < p.D; c += NL_THREADS) s += to_f32(x[c]) - first;
        const float mean = block_sum(s, s_red) / (float)p.D;       // (less `first`; the syncs in
        float sq = 0.0f;                                           // block_sum: y may be x)
        for (int64_t c = threadIdx.x; c < p.D; c += NL_THREADS) {
            const float d = (to_f32(x[c]) - first) - mean;
            sq = fmaf(d, d, sq);
        }
        const float rstd = rsqrtf(fmaf(block_sum(sq, s_red), p.inv_d, p.eps));
        for (int64_t c = threadIdx.x; c < p.D; c += NL_THREADS) {
            const float w = p.w ? load_as(p.w, p.w_type, c) : 1.0f;
            const float b = p.b ? load_as(p.b, p.b_type, c) : 0.0f;
            y[c] = from_f32<TY>(fmaf(((to_f32(x[c]) - first) - mean) * rstd, w, b));
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = first + mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

}  // namespace tke
