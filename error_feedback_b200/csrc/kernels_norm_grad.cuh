// The gradient of layer norm.  With xh = (x - mean) rstd and g = dy w:
//
//   dx = rstd (g - 1/D sum g - xh 1/D sum (g xh)),  dw = sum_t dy xh,  db = sum_t dy
//
// A row is held in registers by 8 to 1,024 threads, 16 elements each, which keep to their columns
// over all of a block's rows, so w and the column sums stay in registers, with the rows that
// follow on their way into a ring of shared memory (kernels_norm.cuh).  Column sums leave one
// fp32 row per block, added in a fixed order by a second kernel: no floating-point atomics.
// 1,024 threads (rows past NG_COLS_D) have no registers for the sums: a kernel of its own reads
// x and dy for them first (2,048 x 16,384 bf16: 125 us with the sums in the same kernel, 80 so).
// Rows past NM_MAX_D columns are read again instead of held.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "elements.cuh"
#include "kernels_norm.cuh"

namespace tke {

constexpr int NG_COLS_D = 8192;

// Rows of the rings of x and dy: what 227 KB hold.
template <typename TX, typename TD, int G>
constexpr int NG_SLOTS = G < 1024 || sizeof(TX) + sizeof(TD) == 4 ? 3 : sizeof(TX) + sizeof(TD) == 6 ? 2 : 1;

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

// G threads a row.  Bound by the bytes of x, dy and dx: 32,768 x 4,096 bf16 in 142.5 to 147 us
// with the sum of the parts, 5.5 to 5.65 TB/s.  500 x 1,024 takes 6.8, the latency of two launches.
template <typename TX, typename TD, int G, int V>
__global__ void __launch_bounds__(NORM_BLOCK<G>, G <= 256 ? 2 : 1)
    norm_grad_kernel(const NormGradParams p) {
    constexpr int E = NR_ELEMS, ROWS = NORM_BLOCK<G> / G, L = G < 32 ? G : 32, W = G < 64 ? 1 : G / 32;
    constexpr int S = NG_SLOTS<TX, TD, G>, BX = NR_BYTES<TX, G, V>, BD = NR_BYTES<TD, G, V>;
    constexpr int BYTES = BX + BD;
    // (1,024 threads have 64 registers each: no column sums, and w from memory beside fp32 rows)
    constexpr bool HOLD = G < 1024, HOLD_W = HOLD || sizeof(TX) + sizeof(TD) == 4;
    constexpr int LEFT = S > 1 ? S - 2 : 0;            // groups of copies that need not have landed
    extern __shared__ __align__(16) char s_ring[];     // [row of the block][S][x, dy]
    __shared__ float2 s_part[2][NORM_BLOCK<G> / 32];
    pdl_launch();
    const int t = (int)(threadIdx.x % G), D = (int)p.D;
    const TX* x = static_cast<const TX*>(p.x);
    const TD* dy = static_cast<const TD*>(p.dy);
    TX* dx = static_cast<TX*>(p.dx);
    char* ring = s_ring + threadIdx.x / G * (S * BYTES);
    const uint32_t ring_at = smem_u32(ring);
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / G;
    // (the lanes of a warp go on together: a warp's last rows may not exist)
    const int64_t first = r - (G < 32 ? lane_id() / G : 0);
    const int64_t rounds = first < p.T ? ceil_div64(p.T - first, step) : 0;
    const auto copy = [&](int slot, int64_t row) {
        if (row < p.T) {
            copy_row<TX, G, V>(ring_at + slot * BYTES, x + row * p.ldx, t, D);
            copy_row<TD, G, V>(ring_at + slot * BYTES + BX, dy + row * p.ldy, t, D);
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) copy(i, r + i * step);
    // what is not copied of the next row: its statistics, and the first elements of rows that
    // start within a word
    float next_mean = 0.0f, next_rstd = 0.0f;
    TX next_x = from_f32<TX>(0.0f);
    TD next_d = from_f32<TD>(0.0f);
    const auto fetch = [&](int64_t row) {
        if (row >= p.T) return;
        next_mean = p.mean[row];
        next_rstd = p.rstd[row];
        if (V == 1 && sizeof(TX) == 2) next_x = x[row * p.ldx];
        if (V == 1 && sizeof(TD) == 2) next_d = dy[row * p.ldy];
    };
    fetch(r);
    const uint32_t mask = elems_mask<G, V>(t, D);
    f32x2 w[E / 2], dw[HOLD ? E / 2 : 1], db[HOLD ? E / 2 : 1];
    if (HOLD_W) row_weights<G, V>(p.w, p.w_type, t, D, 1.0f, w);
#pragma unroll
    for (int i = 0; HOLD && i < E / 2; ++i) dw[i] = db[i] = 0;
    copies_wait<LEFT>();
    row_sync<G>();
    int flip = 0, slot = 0, free_slot = S > 1 ? S - 1 : 0;
    for (int64_t i = 0; i < rounds; ++i, r += step) {
        copy(free_slot, r + (S - 1) * step);
        if (S == 1) {
            copies_wait<0>();
            row_sync<G>();
        }
        RowRegs<TX> vx;
        RowRegs<TD> vd;
        read_row<TX, G, V>(ring + slot * BYTES, x + r * p.ldx, t, mask, next_x, vx);
        read_row<TD, G, V>(ring + slot * BYTES + BX, dy + r * p.ldy, t, mask, next_d, vd);
        if (G < 32 && r >= p.T) {
            // (a row that does not exist leaves the sums as they are)
            vx = RowRegs<TX>{};
            vd = RowRegs<TD>{};
        }
        const float mean = r < p.T ? next_mean : 0.0f, rstd = r < p.T ? next_rstd : 0.0f;
        fetch(r + step);
        free_slot = slot;
        slot = slot + 1 == S ? 0 : slot + 1;
        // (dy is 0 past the end, so nothing there counts)
        f32x2 s1 = 0, s2 = 0;
        if (!HOLD_W) row_weights<G, V>(p.w, p.w_type, t, D, 1.0f, w);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            const f32x2 d = vd.two(e), xh = mul2(add2(vx.two(e), both(-mean)), both(rstd));
            const f32x2 g = mul2(d, w[e]);
            s1 = add2(s1, g);
            s2 = fma2(g, xh, s2);
            if constexpr (HOLD) {
                dw[e] = fma2(d, xh, dw[e]);
                db[e] = add2(db[e], d);
            }
        }
        const float2 a = parts(s1), b = parts(s2);
        copies_wait<LEFT>();                          // (the next row, before the barrier)
        const float2 tot = row_parts<G>(
            make_float2(lanes_sum<L>(a.x + a.y), lanes_sum<L>(b.x + b.y)), s_part, flip, [](float2 o, float2) {
                return make_float2(lanes_sum<W>(o.x), lanes_sum<W>(o.y));
            });
        const float g1 = tot.x * p.inv_d * rstd, g2 = tot.y * p.inv_d * rstd;
        if (r < p.T) {
            if (!HOLD_W) row_weights<G, V>(p.w, p.w_type, t, D, 1.0f, w);
            RowRegs<TX> o;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                const f32x2 xh = mul2(add2(vx.two(e), both(-mean)), both(rstd));
                const f32x2 g = mul2(vd.two(e), w[e]);
                o.put_two(e, fma2(xh, both(-g2), fma2(g, both(rstd), both(-g1))));
            }
            store_row<TX, G, V>(dx + r * p.lddx, t, D, o);
        }
    }
    if constexpr (HOLD) {
        if (!p.part) return;
        float* s_col = reinterpret_cast<float*>(s_ring);   // (all copies have landed and been read)
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
                    const int c0 = norm_col<G, V>(t, 2 * e), c1 = norm_col<G, V>(t, 2 * e + 1);
                    if (c0 < D) part[c0] = f.x;
                    if (c1 < D) part[c1] = f.y;
                }
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

// The column sums alone: a thread takes V columns, blocks in y take every NL_PARTS-th row, four
// of them on their way at once.
constexpr int NL_COLS = 128, NL_AHEAD = 4;
constexpr int64_t NL_PARTS = 64;

template <typename TX, typename TD, int V>
__global__ void __launch_bounds__(NL_COLS) norm_cols_kernel(const NormGradParams p) {
    pdl_launch();
    pdl_wait();
    const int64_t c = ((int64_t)blockIdx.x * NL_COLS + threadIdx.x) * V;
    if (c >= p.D) return;
    const TX* x = static_cast<const TX*>(p.x) + c;
    const TD* dy = static_cast<const TD*>(p.dy) + c;
    float dw[V] = {}, db[V] = {};
    for (int64_t r0 = blockIdx.y; r0 < p.T; r0 += (int64_t)NL_AHEAD * gridDim.y) {
        TX vx[NL_AHEAD][V];
        TD vd[NL_AHEAD][V];
        float mean[NL_AHEAD], rstd[NL_AHEAD];
#pragma unroll
        for (int i = 0; i < NL_AHEAD; ++i) {
            const int64_t r = r0 + (int64_t)i * gridDim.y;
            if (r >= p.T) continue;
            mean[i] = p.mean[r];
            rstd[i] = p.rstd[r];
            if constexpr (V > 1) {
#pragma unroll
                for (int k = 0; k < V * (int)sizeof(TX) / 8; ++k)
                    reinterpret_cast<uint2*>(vx[i])[k] = reinterpret_cast<const uint2*>(x + r * p.ldx)[k];
#pragma unroll
                for (int k = 0; k < V * (int)sizeof(TD) / 8; ++k)
                    reinterpret_cast<uint2*>(vd[i])[k] = reinterpret_cast<const uint2*>(dy + r * p.ldy)[k];
            } else {
                vx[i][0] = x[r * p.ldx];
                vd[i][0] = dy[r * p.ldy];
            }
        }
#pragma unroll
        for (int i = 0; i < NL_AHEAD; ++i) {
            if (r0 + (int64_t)i * gridDim.y >= p.T) continue;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float d = to_f32(vd[i][k]);
                dw[k] = fmaf(d, (to_f32(vx[i][k]) - mean[i]) * rstd[i], dw[k]);
                db[k] += d;
            }
        }
    }
    float* part = p.part + (int64_t)blockIdx.y * 2 * p.D + c;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        part[k] = dw[k];
        part[p.D + k] = db[k];
    }
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
