// Layer norm over the rows of a matrix.
//
//   mean = 1/D sum x,  rstd = (1/D sum (x - mean)^2 + eps)^(-1/2),  y = (x - mean) rstd w + b
//
// All sums are fp32, and an offset common to a row costs no bits: each warp sums the
// differences of its elements from their own (rounded) mean m_w, which makes good the
// rounding, and their squares, and the warps' parts are joined by their distances from the
// first one's, so the variance is a sum of squares of differences, never a difference of
// sums, and x - mean is (x - m_w) less a small rest.  The mean that is given out is the
// plain sum's, unless it is far more than the deviation: then m_0 and the rest are nearer.
//
// A row is held in registers by 8 to 1,024 threads, 16 elements each, between the statistics
// and the result; w and b stay in registers over all rows of a block.  The rows that follow
// are on their way into a ring of shared memory (NR_SLOTS rows, asynchronous copies), so
// what is in flight takes no registers.  (Loads into registers one row ahead: 108 us
// instead of 50.5 for 16,384 x 4,096 bf16; 64 elements a thread, w and b converted for every
// row, nothing ahead: 74.)  Rows past NM_MAX_D columns are read again instead.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "async.cuh"
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

constexpr int NR_ELEMS = 16;               // of a thread and row

// Columns of a group that a thread takes as a whole: 16 bytes of the wider type, so that a
// warp's accesses are consecutive.  (Two accesses of 16 bytes at a stride of 32 touch every
// sector twice: 102 us for 16,384 x 4,096 fp32 to bf16 instead of 68.)
template <typename TA, typename TB>
constexpr int NORM_GROUP = sizeof(TA) + sizeof(TB) == 4 ? 8 : 4;

// Column of element e of thread t of a row of G threads: groups of V columns, or V = 1 (rows
// that start anywhere).
template <int G, int V>
__device__ __forceinline__ int norm_col(int t, int e) {
    return ((e / V) * G + t) * V + e % V;
}

// Elements of a thread that every row has: rows take the fewest threads that hold them.
template <int G>
constexpr int NORM_FULL = G > 8 ? NR_ELEMS / 2 : 0;

template <typename T>
struct RowRegs {
    uint32_t q[NR_ELEMS * sizeof(T) / 4];
    // elements 2 i and 2 i + 1
    __device__ __forceinline__ f32x2 two(int i) const {
        if constexpr (sizeof(T) == 4) {
            return pair(__uint_as_float(q[2 * i]), __uint_as_float(q[2 * i + 1]));
        } else {
            return widen(reinterpret_cast<const typename Twin<T>::type*>(q)[i]);
        }
    }
    __device__ __forceinline__ void put_two(int i, f32x2 a) {
        if constexpr (sizeof(T) == 4) {
            const float2 f = parts(a);
            q[2 * i] = __float_as_uint(f.x);
            q[2 * i + 1] = __float_as_uint(f.y);
        } else {
            q[i] = narrow(a, T{});
        }
    }
};

// Stores the thread's elements of a row.
template <typename T, int G, int V>
__device__ __forceinline__ void store_row(T* row, int t, int D, const RowRegs<T>& r) {
    constexpr int WORDS = V * (int)sizeof(T) / 4;
    if (V > 1) {
#pragma unroll
        for (int j = 0; j < NR_ELEMS / V; ++j) {
            const int c = (j * G + t) * V;
            const uint32_t* q = r.q + j * WORDS;
            if (j * V >= NORM_FULL<G> && c >= D) continue;
            if (WORDS == 4) {
                *reinterpret_cast<uint4*>(row + c) = make_uint4(q[0], q[1], q[2], q[WORDS - 1]);
            } else {
                *reinterpret_cast<uint2*>(row + c) = make_uint2(q[0], q[1]);
            }
        }
    } else {
        const T* e = reinterpret_cast<const T*>(r.q);
#pragma unroll
        for (int j = 0; j < NR_ELEMS; ++j) {
            const int c = j * G + t;
            if (j < NORM_FULL<G> || c < D) row[c] = e[j];
        }
    }
}

// V consecutive weights from c on (p and c in steps of 16 bytes), as pairs; without p each is
// `none`.
template <typename T, int V>
__device__ __forceinline__ void load_group(const T* p, f32x2* o) {
    RowRegs<T> r;
    constexpr int WORDS = V * (int)sizeof(T) / 4;
#pragma unroll
    for (int k = 0; k < WORDS / 2; ++k) {
        const uint2 v = reinterpret_cast<const uint2*>(p)[k];
        r.q[2 * k] = v.x;
        r.q[2 * k + 1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) o[i] = r.two(i);
}
template <int V>
__device__ __forceinline__ void load_as(const void* p, int32_t type, int c, float none, f32x2* o) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) o[i] = pair(none, none);
    } else if (type == TOPK_EF_F32) {
        load_group<float, V>(static_cast<const float*>(p) + c, o);
    } else if (type == TOPK_EF_BF16) {
        load_group<__nv_bfloat16, V>(static_cast<const __nv_bfloat16*>(p) + c, o);
    } else {
        load_group<__half, V>(static_cast<const __half*>(p) + c, o);
    }
}
// The thread's weights of a row, as load_as.
template <int G, int V>
__device__ __forceinline__ void row_weights(const void* p, int32_t type, int t, int D, float none,
                                            f32x2* o) {
    if constexpr (V > 1) {
#pragma unroll
        for (int j = 0; j < NR_ELEMS / V; ++j) {
            const int c = norm_col<G, V>(t, j * V);
            load_as<V>(c < D ? p : nullptr, type, c, none, o + j * V / 2);
        }
    } else {
        const auto at = [&](int e) {
            const int c = norm_col<G, V>(t, e);
            return p && c < D ? load_as(p, type, c) : none;
        };
#pragma unroll
        for (int i = 0; i < NR_ELEMS / 2; ++i) o[i] = pair(at(2 * i), at(2 * i + 1));
    }
}

// Elements that the lanes of one warp (or part of it) hold of a row; t0: the row's thread that
// the lanes start at.
template <int G, int V>
__device__ __forceinline__ int warp_count(int t0, int D) {
    constexpr int L = G < 32 ? G : 32;
    int n = 0;
#pragma unroll
    for (int j = 0; j < NR_ELEMS / V; ++j) n += min(max(D - (j * G + t0) * V, 0), L * V);
    return n;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ f32x2 both(float x) { return pair(x, x); }

// Threads of a block: rows of fewer threads share one.
template <int G>
constexpr int NORM_BLOCK = G < 256 ? 256 : G;

// Waits for the G threads of a row (32 < G < 256: a barrier of its own for each row of the block).
template <int G>
__device__ __forceinline__ void row_sync() {
    if (G <= 32) {
        __syncwarp();
    } else if (G >= 256) {
        __syncthreads();
    } else {
        asm volatile("bar.sync %0, %1;" ::"r"((int)threadIdx.x / G + 1), "n"(G) : "memory");
    }
}

// ------------------------------------------------------ rows through a ring

// Rows of the ring: what 227 KB leave of an SM's three blocks (768 threads).
template <typename T, int G>
constexpr int NR_SLOTS = sizeof(T) == 2 ? 4 : G >= 1024 ? 2 : 3;

// Bytes of one row of G threads in it.  (Rows that start anywhere: in their 16-byte granules.)
template <typename T, int G, int V>
constexpr int NR_BYTES = G * NR_ELEMS * (int)sizeof(T) + (V > 1 ? 0 : 32);

__device__ __forceinline__ void copy_async16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async8(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
// `bytes` (2 or 4) of a word; zero after them.
__device__ __forceinline__ void copy_async4(uint32_t to, const void* from, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N groups of the thread's copies are on their way.
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Begins to copy a row of D elements.  Of a row that starts within a 4-byte word the first
// element is left out (read_row takes it from the caller).
template <typename T, int G, int V>
__device__ __forceinline__ void copy_row(uint32_t slot, const T* row, int t, int D) {
    if (V > 1) {
        constexpr int BYTES = V * (int)sizeof(T);
#pragma unroll
        for (int j = 0; j < NR_ELEMS / V; ++j) {
            const int c = (j * G + t) * V;
            if (j * V >= NORM_FULL<G> && c >= D) continue;
            const uint32_t to = slot + (uint32_t)(j * G + t) * BYTES;
            if (BYTES == 16) {
                copy_async16(to, row + c);
            } else {
                copy_async8(to, row + c);
            }
        }
    } else {
        const int lead = (int)((uintptr_t)row & 15), end = lead + D * (int)sizeof(T);
        const char* from = reinterpret_cast<const char*>(row) - lead;
#pragma unroll
        for (int i = 0; i < NR_ELEMS * (int)sizeof(T) / 16 + 1; ++i) {
            const int at = (i * G + t) * 16;
            if (at >= lead && at + 16 <= end) {
                copy_async16(slot + at, from + at);
            } else if (at < end) {
                // the row's ragged ends
                for (int w = at; w < at + 16; w += 4)
                    if (w >= lead && w < end) copy_async4(slot + w, from + w, min(4, end - w));
            }
        }
    }
}

// Bit e: element e of the thread is in the row.
template <int G, int V>
__device__ __forceinline__ uint32_t elems_mask(int t, int D) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < NR_ELEMS; ++e) m |= (uint32_t)(norm_col<G, V>(t, e) < D) << e;
    return m;
}

// The thread's elements of a copied row; zero where it has none.  `first`: the row's first.
template <typename T, int G, int V>
__device__ __forceinline__ void read_row(const char* slot, const T* row, int t, uint32_t mask, T first,
                                         RowRegs<T>& r) {
    if (V > 1) {
        constexpr int WORDS = V * (int)sizeof(T) / 4;
#pragma unroll
        for (int j = 0; j < NR_ELEMS / V; ++j) {
            const bool in = j * V < NORM_FULL<G> || (mask >> V * j & 1);
            uint32_t* q = r.q + j * WORDS;
            if (WORDS == 4) {
                const uint4 v = in ? reinterpret_cast<const uint4*>(slot)[j * G + t] : make_uint4(0, 0, 0, 0);
                q[0] = v.x;
                q[1] = v.y;
                q[2] = v.z;
                q[WORDS - 1] = v.w;
            } else {
                const uint2 v = in ? reinterpret_cast<const uint2*>(slot)[j * G + t] : make_uint2(0, 0);
                q[0] = v.x;
                q[1] = v.y;
            }
        }
    } else {
        const int lead = (int)((uintptr_t)row & 15);
        const T* at = reinterpret_cast<const T*>(slot + lead) + t;
        T* e = reinterpret_cast<T*>(r.q);
#pragma unroll
        for (int j = 0; j < NR_ELEMS; ++j) e[j] = j < NORM_FULL<G> || (mask >> j & 1) ? at[j * G] : from_f32<T>(0.0f);
        if (sizeof(T) == 2 && t == 0 && (lead & 2)) e[0] = first;
    }
}

// f(v of the row's warp lane % W, v of its first warp), where v is what each of a warp's lanes
// has found for its warp; s: two places a warp, `flip` the ones that the last call did not
// use.  (Rows of one warp: f(v, v).)  Also a barrier of the row.
template <int G, typename P, typename F>
__device__ __forceinline__ auto row_parts(P v, P (*s)[NORM_BLOCK<G> / 32], int& flip, F f) {
    constexpr int W = G < 64 ? 1 : G / 32;
    if constexpr (W == 1) {
        __syncwarp();
        return f(v, v);
    } else {
        const int warp = (int)warp_id(), lane = (int)lane_id();
        if (lane == 0) s[flip][warp] = v;
        row_sync<G>();
        const P o = s[flip][warp / W * W + lane % W], first = s[flip][warp / W * W];
        flip ^= 1;
        return f(o, first);
    }
}

// The pair of elements 2 e and 2 e + 1, 0 where the thread has none.
template <int G, int V>
__device__ __forceinline__ f32x2 masked(f32x2 a, uint32_t mask, int e) {
    if (2 * e < NORM_FULL<G>) return a;
    if (V > 1) return mask >> 2 * e & 1 ? a : 0;
    const float2 f = parts(a);
    return pair(mask >> 2 * e & 1 ? f.x : 0.0f, mask >> (2 * e + 1) & 1 ? f.y : 0.0f);
}

// G threads a row.  Bound by the bytes of x and y: 16,384 x 4,096 bf16 in 50.5 to 53.5 us, 5.0 to
// 5.3 TB/s; 30,011 x 1,001 fp32 to bf16, rows that start anywhere, in 44 to 47, 3.8 to 4.1 TB/s.
template <typename TX, typename TY, int G, int V>
__global__ void __launch_bounds__(NORM_BLOCK<G>, G <= 256 ? 3 : 1) norm_kernel(const NormParams p) {
    constexpr int E = NR_ELEMS, ROWS = NORM_BLOCK<G> / G, L = G < 32 ? G : 32, W = G < 64 ? 1 : G / 32;
    constexpr int S = NR_SLOTS<TX, G>, BYTES = NR_BYTES<TX, G, V>;
    extern __shared__ __align__(16) char s_ring[];     // [row of the block][S][BYTES]
    __shared__ float4 s_part[2][NORM_BLOCK<G> / 32];   // mean, rest, squares, sum of a warp's elements
    pdl_launch();
    const int t = (int)(threadIdx.x % G), D = (int)p.D, lane = (int)lane_id();
    const TX* x = static_cast<const TX*>(p.x);
    TY* y = static_cast<TY*>(p.y);
    char* ring = s_ring + threadIdx.x / G * (S * BYTES);
    const uint32_t ring_at = smem_u32(ring);
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / G;
    // (the lanes of a warp go on together: a warp's last rows may not exist)
    const int64_t first = r - (G < 32 ? lane / G : 0);
    const int64_t rounds = first < p.T ? ceil_div64(p.T - first, step) : 0;
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
        if (r + i * step < p.T) copy_row<TX, G, V>(ring_at + i * BYTES, x + (r + i * step) * p.ldx, t, D);
        copies_commit();
    }
    // (the first element of a 16-bit row that starts within a word is not copied)
    TX next_first = from_f32<TX>(0.0f);
    if (V == 1 && sizeof(TX) == 2 && r < p.T) next_first = x[r * p.ldx];
    // elements of this warp's lanes, and of the warp that a lane joins for
    const float n = (float)warp_count<G, V>(t - t % L, D), inv_n = n > 0.0f ? 1.0f / n : 0.0f;
    const float k = W > 1 ? (float)warp_count<G, V>(lane % W * 32, D) : (float)D;
    const uint32_t mask = elems_mask<G, V>(t, D);
    f32x2 w[E / 2], b[E / 2];
    row_weights<G, V>(p.w, p.w_type, t, D, 1.0f, w);
    row_weights<G, V>(p.b, p.b_type, t, D, 0.0f, b);
    copies_wait<S - 2>();
    row_sync<G>();
    int flip = 0, slot = 0, free_slot = S - 1;
    for (int64_t i = 0; i < rounds; ++i, r += step) {
        const TX* row = x + r * p.ldx;
        if (r + (S - 1) * step < p.T)
            copy_row<TX, G, V>(ring_at + free_slot * BYTES, row + (S - 1) * step * p.ldx, t, D);
        copies_commit();
        RowRegs<TX> v;
        read_row<TX, G, V>(ring + slot * BYTES, row, t, mask, next_first, v);
        if (V == 1 && sizeof(TX) == 2 && r + step < p.T) next_first = row[step * p.ldx];
        free_slot = slot;
        slot = slot + 1 == S ? 0 : slot + 1;
        f32x2 sum = 0;                                 // (0 past the row's end)
#pragma unroll
        for (int e = 0; e < E / 2; ++e) sum = add2(sum, v.two(e));
        const float2 s = parts(sum);
        const float total = lanes_sum<L>(s.x + s.y), m0 = total * inv_n;
        f32x2 d[E / 2], sq2 = 0, rest2 = 0;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            d[e] = masked<G, V>(add2(v.two(e), both(-m0)), mask, e);
            sq2 = fma2(d[e], d[e], sq2);
            rest2 = add2(rest2, d[e]);
        }
        const float2 q = parts(sq2), u = parts(rest2);
        const float rest = lanes_sum<L>(u.x + u.y) * inv_n, sq = lanes_sum<L>(q.x + q.y);
        copies_wait<S - 2>();                          // (the next row, before the barrier)
        // m_0 of the first warp, the row's mean less that, the squares about the mean, the sum
        const float4 tot = row_parts<G>(
            make_float4(m0, rest, sq, total), s_part, flip, [&](float4 o, float4 w0) {
                const float far = (o.x - w0.x) + o.y;
                const float m = lanes_sum<W>(k * far) * p.inv_d, off = far - m;
                const float about = fmaf(k * off, off, fmaf(-k * o.y, o.y, o.z));
                return make_float4(w0.x, m, lanes_sum<W>(about), lanes_sum<W>(o.w));
            });
        const float var = max_nan(tot.z, 0.0f) * p.inv_d, rstd = rsqrtf(var + p.eps);
        const f32x2 off = both((m0 - tot.x) - tot.y);
        if (r < p.T) {
            RowRegs<TY> o;
#pragma unroll
            for (int e = 0; e < E / 2; ++e)
                o.put_two(e, fma2(mul2(add2(d[e], off), both(rstd)), w[e], b[e]));
            store_row<TY, G, V>(y + r * p.ldy, t, D, o);
            if (t == 0) {
                const float mean = tot.x + tot.y;
                if (p.mean) p.mean[r] = mean * mean > 256.0f * var ? mean : tot.w * p.inv_d;
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
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < p.D; c += NL_THREADS) s += to_f32(x[c]);
        const float total = block_sum(s, s_red), m0 = total / (float)p.D;
        float sq = 0.0f, rest = 0.0f;
        for (int64_t c = threadIdx.x; c < p.D; c += NL_THREADS) {
            const float d = to_f32(x[c]) - m0;
            sq = fmaf(d, d, sq);
            rest += d;
        }
        rest = block_sum(rest, s_red) / (float)p.D;    // (the barriers in block_sum: y may be x)
        const float var = max_nan(fmaf(block_sum(sq, s_red), p.inv_d, -rest * rest), 0.0f);
        const float rstd = rsqrtf(var + p.eps), mean = m0 + rest;
        for (int64_t c = threadIdx.x; c < p.D; c += NL_THREADS) {
            const float w = p.w ? load_as(p.w, p.w_type, c) : 1.0f;
            const float b = p.b ? load_as(p.b, p.b_type, c) : 0.0f;
            y[c] = from_f32<TY>(fmaf(((to_f32(x[c]) - m0) - rest) * rstd, w, b));
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = mean * mean > 256.0f * var ? mean : m0;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

}  // namespace tke
