// The gradient of layer norm.  With xh = (x - mean) rstd and g = dy w:
//
//   dx = rstd (g - 1/D sum g - xh 1/D sum (g xh)),  dw = sum_t dy xh,  db = sum_t dy
//
// A row is held in registers by 8 to 1,024 threads, 16 elements each (8 of fp32), which keep to
// their columns over all of a block's rows, so w and the column sums stay in registers.
// Column sums leave one fp32 row per block, added in a fixed order by a second kernel: no
// floating-point atomics.  Rows past NM_MAX_GRAD_D columns are read again instead.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "elements.cuh"
#include "kernels_norm.cuh"

namespace tke {

constexpr int NM_MAX_GRAD_D = 16384;

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

// Threads of a gradient's block: rows of fewer threads share one.
template <int G>
constexpr int GRAD_BLOCK = G < 256 ? 256 : G;

// Waits for the G threads of a row (G > 32: a barrier of its own for each row of the block).
template <int G>
__device__ __forceinline__ void row_sync() {
    if (G == GRAD_BLOCK<G>) {
        __syncthreads();
    } else {
        asm volatile("bar.sync %0, %1;" ::"r"((int)threadIdx.x / G + 1), "n"(G) : "memory");
    }
}

// G threads a row, 8 N elements a thread.  Bound by the bytes of x, dy and dx; 32 registers of
// column sums, and the next row's x and dy on their way, leave an SM 16 warps.
template <typename TX, typename TD, int G, int N, bool VEC>
__global__ void __launch_bounds__(GRAD_BLOCK<G>) norm_grad_kernel(const NormGradParams p) {
    constexpr int E = 8 * N, BLOCK = GRAD_BLOCK<G>, ROWS = BLOCK / G, L = G < 32 ? G : 32, W = G < 32 ? 1 : G / 32;
    // (1,024 threads have 64 registers each: no next row, w from memory)
    constexpr bool AHEAD = G < 1024;
    __shared__ float2 s_part[2][BLOCK / 32];
    __shared__ float s_col[ROWS > 1 ? G * E : 1];
    pdl_launch();
    const int t = (int)(threadIdx.x % G), D = (int)p.D;
    const TX* x = static_cast<const TX*>(p.x);
    const TD* dy = static_cast<const TD*>(p.dy);
    TX* dx = static_cast<TX*>(p.dx);
    pdl_wait();
    const auto weight = [&](int e) {
        const int c = norm_col<G, VEC>(t, e);
        return p.w && c < D ? load_as(p.w, p.w_type, c) : 1.0f;
    };
    f32x2 w[AHEAD ? E / 2 : 1], dw[E / 2], db[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        if (AHEAD) w[i] = pair(weight(2 * i), weight(2 * i + 1));
        dw[i] = db[i] = 0;
    }
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / G;
    int flip = 0;
    RowRegs<TX, N, VEC> nx;
    RowRegs<TD, N, VEC> nd;
    float nm = 0.0f, nr = 0.0f;
    const auto fetch = [&](int64_t row) {
        load_row<TX, G, N, VEC>(x + row * p.ldx, t, D, nx);
        load_row<TD, G, N, VEC>(dy + row * p.ldy, t, D, nd);
        nm = p.mean[row];
        nr = p.rstd[row];
    };
    // (the lanes of a warp go on together: a warp's last rows may not exist; they count as rows
    // of dy = 0)
    const int64_t first = r - (G < 32 ? lane_id() / G : 0);
    const int64_t rounds = first < p.T ? ceil_div64(p.T - first, step) : 0;
    if (AHEAD && r < p.T) fetch(r);
    for (int64_t i0 = 0; i0 < rounds; ++i0, r += step) {
        const bool here = r < p.T;
        if (!AHEAD) fetch(r);
        if (!here) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                nx.v[j] = Vec8<TX>{};
                nd.v[j] = Vec8<TD>{};
            }
        }
        const RowRegs<TX, N, VEC> vx = nx;
        const RowRegs<TD, N, VEC> vd = nd;
        const float mean = here ? nm : 0.0f, rstd = here ? nr : 0.0f;
        if (AHEAD && r + step < p.T) fetch(r + step);
        // (dy is 0 past the end, so nothing there counts)
        f32x2 s1 = 0, s2 = 0;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const f32x2 d = vd.two(i), xh = mul2(add2(vx.two(i), both(-mean)), both(rstd));
            const f32x2 g = mul2(d, AHEAD ? w[i] : pair(weight(2 * i), weight(2 * i + 1)));
            s1 = add2(s1, g);
            s2 = fma2(g, xh, s2);
            dw[i] = fma2(d, xh, dw[i]);
            db[i] = add2(db[i], d);
        }
        const float2 a = parts(s1), b = parts(s2);
        float g1 = lanes_sum<L>(a.x + a.y), g2 = lanes_sum<L>(b.x + b.y);
        if (W > 1) {
            const int warp = (int)warp_id(), lane = (int)lane_id();
            if (lane == 0) s_part[flip][warp] = make_float2(g1, g2);
            row_sync<G>();
            const float2 o = lane < W ? s_part[flip][warp / W * W + lane] : make_float2(0.0f, 0.0f);
            flip ^= 1;
            g1 = warp_sum(o.x);
            g2 = warp_sum(o.y);
        }
        g1 *= p.inv_d * rstd;
        g2 *= p.inv_d * rstd;
        if (here) {
            RowRegs<TX, N, VEC> o;
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const f32x2 xh = mul2(add2(vx.two(i), both(-mean)), both(rstd));
                const f32x2 g =
                    mul2(vd.two(i), AHEAD ? w[i] : pair(weight(2 * i), weight(2 * i + 1)));
                o.put_two(i, fma2(xh, both(-g2), fma2(g, both(rstd), both(-g1))));
            }
            store_row<TX, G, N, VEC>(dx + r * p.lddx, t, D, o);
        }
    }
    if (!p.part) return;
    float* part = p.part + (int64_t)blockIdx.x * 2 * p.D;
    const int mine = (int)threadIdx.x / G;
#pragma unroll
    for (int k = 0; k < 2; ++k, part += p.D) {
        f32x2* v = k ? db : dw;
        // the block's rows, in order
        for (int i = ROWS - 1; i > 0; --i) {
            __syncthreads();
            if (mine == i) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {
                    const float2 f = parts(v[e]);
                    s_col[2 * e * G + t] = f.x;
                    s_col[(2 * e + 1) * G + t] = f.y;
                }
            }
            __syncthreads();
            if (mine == i - 1) {
#pragma unroll
                for (int e = 0; e < E / 2; ++e)
                    v[e] = add2(v[e], pair(s_col[2 * e * G + t], s_col[(2 * e + 1) * G + t]));
            }
        }
        if (mine == 0) {
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                const float2 f = parts(v[e]);
                const int c0 = norm_col<G, VEC>(t, 2 * e), c1 = norm_col<G, VEC>(t, 2 * e + 1);
                if (c0 < D) part[c0] = f.x;
                if (c1 < D) part[c1] = f.y;
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

// 32 columns a block; its 16 warps take every 16th part each, in order.
constexpr int NS_WARPS = 16;

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
#pragma unroll 8
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
