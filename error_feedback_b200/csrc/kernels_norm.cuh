// Layer norm over the rows of a matrix, and its gradient.
//
//   mean = 1/D sum x,  rstd = (1/D sum (x - mean)^2 + eps)^(-1/2)
//   y    = (x - mean) rstd w + b
//   with xh = (x - mean) rstd and g = dy w:
//   dx   = rstd (g - 1/D sum g - xh 1/D sum (g xh)),  dw = sum_t dy xh,  db = sum_t dy
//
// All sums are fp32, of the row less its first element c: at most sqrt(D) deviations
// from the mean, so an offset common to a row costs no bits.  The variance
// is a sum of squares of differences, never a difference of sums: each warp sums the
// squares of the differences from its own elements' mean, and the warps' (count,
// sum, squares) are joined by sum n (mean_w - mean)^2.
//
// Rows of up to NM_MAX_D (forward) and NM_MAX_GRAD_D (gradient) columns are read
// once and held in registers between the statistics and the result; longer
// ones are read again.  A block keeps to its columns over all of its rows, so w, b and
// the gradient's column sums stay in registers too.  Column sums leave one fp32 row per
// block, added in block order by a second kernel: no floating-point atomics.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "elements.cuh"
#include "topk_ef.h"

namespace tke {

constexpr int NM_MAX_D = 16384;
constexpr int NM_MAX_GRAD_D = 8192;

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

// The thread's elements of one row: groups of 8 columns (VEC; 16-byte aligned), or
// columns G apart (rows that start anywhere).  Element e of thread t:
template <int G, bool VEC>
__device__ __forceinline__ int64_t norm_col(int t, int e) {
    return VEC ? ((int64_t)(e / 8) * G + t) * 8 + e % 8 : (int64_t)e * G + t;
}

template <typename T, int N, bool VEC>
struct RowRegs {
    Vec8<T> v[N];                  // 8 N elements
    __device__ __forceinline__ float get(int e) const {
        return to_f32(reinterpret_cast<const T*>(v)[e]);
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
__device__ __forceinline__ void store_row(T* row, int t, int D, const float* x) {
    if (VEC) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (j * G + t) * 8;
            if (c < D) store8(row + c, x + j * 8);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8 * N; ++j) {
            const int c = j * G + t;
            if (c < D) row[c] = from_f32<T>(x[j]);
        }
    }
}

// Elements of the warp that starts at thread t0 of its row's G threads, of D.
template <int G, int N, bool VEC>
__device__ __forceinline__ int warp_count(int t0, int D) {
    int n = 0;
    if (VEC) {
#pragma unroll
        for (int j = 0; j < N; ++j) n += min(max(D - (j * G + t0) * 8, 0), 256);
    } else {
#pragma unroll
        for (int j = 0; j < 8 * N; ++j) n += min(max(D - (j * G + t0), 0), 32);
    }
    return n;
}

// Mean and reciprocal deviation of what G threads hold of a row; n elements (columns
// in(e)) belong to the warp.  s: 3 G / 32 floats that the previous row's call has
// not used.
template <int G, int E, typename I>
__device__ __forceinline__ float2 row_statistics(const float* x, I in, int n, float D, float inv_d,
                                                 float eps, float* s) {
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) sum += in(e) ? x[e] : 0.0f;
    sum = warp_sum(sum);
    const float m = n > 0 ? sum / (float)n : 0.0f;
    float sq = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float d = in(e) ? x[e] - m : 0.0f;
        sq = fmaf(d, d, sq);
    }
    sq = warp_sum(sq);
    if (G == 32) return make_float2(m, rsqrtf(fmaf(sq, inv_d, eps)));
    constexpr int W = G / 32;
    const int w = (int)(threadIdx.x % G) / 32;
    if (lane_id() == 0) {
        s[w] = sum;
        s[W + w] = sq;
        s[2 * W + w] = (float)n;
    }
    __syncthreads();
    float tot = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) tot += s[i];
    const float mean = tot / D;
    float var = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float k = s[2 * W + i];
        const float d = k > 0.0f ? s[i] / k - mean : 0.0f;
        var += fmaf(k * d, d, s[W + i]);
    }
    return make_float2(mean, rsqrtf(fmaf(var, inv_d, eps)));
}

template <int G>
constexpr int NORM_BLOCK = G < 256 ? (G == 32 ? 256 : G) : G;

// G threads a row, 8 N elements a thread.
template <typename TX, typename TY, int G, int N, bool VEC>
__global__ void __launch_bounds__(NORM_BLOCK<G>) norm_kernel(const NormParams p) {
    constexpr int E = 8 * N, ROWS = NORM_BLOCK<G> / G;
    __shared__ float s_red[2][3 * G / 32];
    pdl_launch();
    const int t = (int)(threadIdx.x % G), D = (int)p.D;
    const TX* x = static_cast<const TX*>(p.x);
    TY* y = static_cast<TY*>(p.y);
    pdl_wait();
    float w[E], b[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int64_t c = norm_col<G, VEC>(t, e);
        w[e] = p.w && c < D ? load_as(p.w, p.w_type, c) : 1.0f;
        b[e] = p.b && c < D ? load_as(p.b, p.b_type, c) : 0.0f;
    }
    const int n = warp_count<G, N, VEC>(t & ~31, D);
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / G;
    int flip = 0;
    RowRegs<TX, N, VEC> next;
    float next_c = 0.0f;
    if (r < p.T) {
        load_row<TX, G, N, VEC>(x + r * p.ldx, t, D, next);
        next_c = to_f32(x[r * p.ldx]);
    }
    for (; r < p.T; r += step) {
        const RowRegs<TX, N, VEC> v = next;
        if (r + step < p.T) load_row<TX, G, N, VEC>(x + (r + step) * p.ldx, t, D, next);
        const float c = next_c;
        if (r + step < p.T) next_c = to_f32(x[(r + step) * p.ldx]);
        auto in = [&](int e) { return norm_col<G, VEC>(t, e) < D; };
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = v.get(e) - c;
        const float2 m = row_statistics<G, E>(o, in, n, (float)D, p.inv_d, p.eps, s_red[flip]);
        flip ^= 1;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf((o[e] - m.x) * m.y, w[e], b[e]);
        store_row<TY, G, N, VEC>(y + r * p.ldy, t, D, o);
        if (t == 0) {
            if (p.mean) p.mean[r] = c + m.x;
            if (p.rstd) p.rstd[r] = m.y;
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

// ----------------------------------------------------------------- gradient

struct NormGradParams {
    const void* dy;
    const void* x;
    const float* mean;
    const float* rstd;
    const void* w;                 // or null
    void* dx;                      // x's type
    float* part;                   // [parts][2][D]: column sums of dy xh and of dy; or null
    int64_t T, D, ldy, ldx, lddx;
    int32_t w_type;
    float inv_d;
};

template <typename TX, typename TD, int G, int N, bool VEC>
__global__ void __launch_bounds__(NORM_BLOCK<G>) norm_grad_kernel(const NormGradParams p) {
    constexpr int E = 8 * N, BLOCK = NORM_BLOCK<G>, ROWS = BLOCK / G, W = G / 32;
    __shared__ float s_red[2][2 * W];
    __shared__ float s_col[ROWS > 1 ? G * E : 1];
    pdl_launch();
    const int t = (int)(threadIdx.x % G), D = (int)p.D;
    const TX* x = static_cast<const TX*>(p.x);
    const TD* dy = static_cast<const TD*>(p.dy);
    TX* dx = static_cast<TX*>(p.dx);
    pdl_wait();
    float w[E], dw[E], db[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int64_t c = norm_col<G, VEC>(t, e);
        w[e] = p.w && c < D ? load_as(p.w, p.w_type, c) : 1.0f;
        dw[e] = db[e] = 0.0f;
    }
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / G;
    int flip = 0;
    RowRegs<TX, N, VEC> nx;
    RowRegs<TD, N, VEC> nd;
    float nm = 0.0f, nr = 0.0f;
    auto fetch = [&](int64_t row) {
        load_row<TX, G, N, VEC>(x + row * p.ldx, t, D, nx);
        load_row<TD, G, N, VEC>(dy + row * p.ldy, t, D, nd);
        nm = p.mean[row];
        nr = p.rstd[row];
    };
    if (r < p.T) fetch(r);
    for (; r < p.T; r += step) {
        const RowRegs<TX, N, VEC> vx = nx;
        const RowRegs<TD, N, VEC> vd = nd;
        const float mean = nm, rstd = nr;
        if (r + step < p.T) fetch(r + step);
        // (dy is 0 past the end, so nothing there counts)
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float d = vd.get(e), xh = (vx.get(e) - mean) * rstd, g = d * w[e];
            s1 += g;
            s2 = fmaf(g, xh, s2);
            dw[e] = fmaf(d, xh, dw[e]);
            db[e] += d;
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (G > 32) {
            const int wi = t / 32;
            if (lane_id() == 0) {
                s_red[flip][wi] = s1;
                s_red[flip][W + wi] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                s1 += s_red[flip][i];
                s2 += s_red[flip][W + i];
            }
            flip ^= 1;
        }
        s1 *= p.inv_d;
        s2 *= p.inv_d;
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float xh = (vx.get(e) - mean) * rstd;
            o[e] = rstd * (fmaf(vd.get(e), w[e], -s1) - xh * s2);
        }
        store_row<TX, G, N, VEC>(dx + r * p.lddx, t, D, o);
    }
    if (!p.part) return;
    float* part = p.part + (int64_t)blockIdx.x * 2 * p.D;
#pragma unroll
    for (int k = 0; k < 2; ++k, part += p.D) {
        float* v = k ? db : dw;
        // the block's rows, in order
        for (int i = ROWS - 1; i > 0; --i) {
            if ((int)threadIdx.x / G == i) {
#pragma unroll
                for (int e = 0; e < E; ++e) s_col[e * G + t] = v[e];
            }
            __syncthreads();
            if ((int)threadIdx.x / G == i - 1) {
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] += s_col[e * G + t];
            }
            __syncthreads();
        }
        if ((int)threadIdx.x < G) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int64_t c = norm_col<G, VEC>(t, e);
                if (c < D) part[c] = v[e];
            }
        }
    }
}

// Rows of any length: dx by one block a row, two passes over it.
template <typename TX, typename TD>
__global__ void __launch_bounds__(NL_THREADS) norm_grad_long_kernel(const NormGradParams p) {
    __shared__ float s_red[33];
    pdl_launch();
    pdl_wait();
    for (int64_t r = blockIdx.x; r < p.T; r += gridDim.x) {
        const TX* x = static_cast<const TX*>(p.x) + r * p.ldx;
        const TD* dy = static_cast<const TD*>(p.dy) + r * p.ldy;
        TX* dx = static_cast<TX*>(p.dx) + r * p.lddx;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < p.D; c += NL_THREADS) {
            const float g = to_f32(dy[c]) * (p.w ? load_as(p.w, p.w_type, c) : 1.0f);
            s1 += g;
            s2 = fmaf(g, (to_f32(x[c]) - mean) * rstd, s2);
        }
        s1 = block_sum(s1, s_red) * p.inv_d;
        s2 = block_sum(s2, s_red) * p.inv_d;
        for (int64_t c = threadIdx.x; c < p.D; c += NL_THREADS) {
            const float w = p.w ? load_as(p.w, p.w_type, c) : 1.0f;
            const float xh = (to_f32(x[c]) - mean) * rstd;
            dx[c] = from_f32<TX>(rstd * (fmaf(to_f32(dy[c]), w, -s1) - xh * s2));
        }
    }
}

// ... and their column sums, 32 rows of blocks by NL_COLS columns.
constexpr int NL_COLS = 256, NL_PARTS = 32;

template <typename TX, typename TD>
__global__ void __launch_bounds__(NL_COLS) norm_cols_kernel(const NormGradParams p) {
    pdl_launch();
    pdl_wait();
    const int64_t c = (int64_t)blockIdx.x * NL_COLS + threadIdx.x;
    if (c >= p.D) return;
    const TX* x = static_cast<const TX*>(p.x) + c;
    const TD* dy = static_cast<const TD*>(p.dy) + c;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = blockIdx.y; r < p.T; r += gridDim.y) {
        const float d = to_f32(dy[r * p.ldy]);
        dw = fmaf(d, (to_f32(x[r * p.ldx]) - p.mean[r]) * p.rstd[r], dw);
        db += d;
    }
    float* part = p.part + (int64_t)blockIdx.y * 2 * p.D;
    part[c] = dw;
    part[p.D + c] = db;
}

// ------------------------------------------------- the blocks' column sums

struct NormSumParams {
    const float* part;             // [parts][2][D]
    Ctrl* ctrl;
    void* out[2];                  // dw, db (either or both)
    int64_t D;
    int32_t parts, type[2], accumulate;
};

// 32 columns a block; its 8 warps take every eighth part each, in order.
constexpr int NS_WARPS = 8;

__global__ void __launch_bounds__(32 * NS_WARPS) norm_sum_kernel(const NormSumParams p) {
    __shared__ float s[NS_WARPS][32];
    pdl_wait();
    const int k = (int)blockIdx.y, lane = (int)lane_id(), w = (int)warp_id();
    if (blockIdx.x == 0 && k == 0 && threadIdx.x == 0) {
        p.ctrl->path_small = 0;
        p.ctrl->status = 0;
    }
    if (!p.out[k]) return;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < p.D) {
        const float* q = p.part + k * p.D + c;
#pragma unroll 4
        for (int i = w; i < p.parts; i += NS_WARPS) v += q[(int64_t)i * 2 * p.D];
    }
    s[w][lane] = v;
    __syncthreads();
    if (w != 0 || c >= p.D) return;
#pragma unroll
    for (int i = 1; i < NS_WARPS; ++i) v += s[i][lane];
    switch (p.type[k]) {
        case TOPK_EF_F32: {
            float* o = static_cast<float*>(p.out[k]) + c;
            *o = p.accumulate ? *o + v : v;
            break;
        }
        case TOPK_EF_BF16: {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out[k]) + c;
            *o = from_f32<__nv_bfloat16>(p.accumulate ? to_f32(*o) + v : v);
            break;
        }
        default: {
            __half* o = static_cast<__half*>(p.out[k]) + c;
            *o = from_f32<__half>(p.accumulate ? to_f32(*o) + v : v);
        }
    }
}

}  // namespace tke
