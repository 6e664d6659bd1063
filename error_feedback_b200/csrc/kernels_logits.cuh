// Losses over a vocabulary: log-probabilities of given tokens with entropy and the
// largest alternatives, their gradient, and distillation from a teacher's top logits.
//
// With c = scale log2(e), a row's softmax is held as  p_i = 2^(c z_i - m) / s,
// s = sum 2^(c z_i - m), u = sum 2^(c z_i - m) (c z_i - m), so that
//     log p_i = ln2 (c z_i - m - log2 s),   entropy = ln2 (log2 s - u / s),
//     log of the sum = ln2 m + ln s.
// m is the largest c z rounded up to a whole number: each thread raises its own when a
// group of values passes it, and a change of m scales s by an exact power of two.
// One ex2 a value and one packed fma two; the maxima take two values an instruction.
//
// Values below -2^17 / c are left out at first: if the row's m ends above -2^16, their p
// is 0.  If m ends past +-2^16, where c z - m would lose bits, or nothing is left, the
// row is read again and summed with the exact differences z - max (a row all of
// whose tokens are masked by -1e9 or by the type's lowest value is uniform).
// -inf (a forbidden token) has p = 0 and counts nowhere.  NaN and +inf make the row
// NaN.
//
// A row is worked on by a team: a warp or four (many rows, short ones above all: the chain of
// a row's steps overlaps with other rows' reads), a block of eight, or a cluster of blocks while
// there are few rows, each block an equal share of the row's 128-byte lines.  Rows start
// anywhere; whole lines are read as 32 bytes a thread.
#pragma once

#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "async.cuh"
#include "common.cuh"
#include "elements.cuh"
#include "topk_ef.h"

namespace tke {

constexpr int LG_SMALL = 128;              // lines of a row that one warp takes
constexpr int LG_LINE = 128;               // bytes of a line (a group of the top selection)
constexpr int LG_FLIGHT = 4;               // 32-byte chunks that a thread loads at once
constexpr float LG_START = -3.402823466e38f;     // m before any value
constexpr float LG_FAR = 65536.0f;         // most |m| whose differences are exact enough
constexpr float LN2 = 0.693147180559945309f, LOG2E = 1.44269504088896341f;
constexpr float LN2_HI = 0.693145751953125f;         // 16 bits: times a whole m exact
constexpr float LN2_LO = 1.42860682030941723e-6f;    // ln 2 - LN2_HI
constexpr int TL_MAX_TOP = 128;
constexpr int TL_MAX_LINES = 16384;        // of a row, for the top selection
constexpr int DL_MAX_K = 256;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
constexpr int CHUNK = 32 / (int)sizeof(T);         // elements of 32 bytes

// W warps: a whole block, or each warp of a block of 8.
template <int W>
struct Team {
    static constexpr int WARPS = W, THREADS = W * 32;
    static constexpr int BLOCK = W == 1 ? 256 : THREADS;
    static constexpr int TEAMS = BLOCK / THREADS;
    static __device__ __forceinline__ int thread() { return (int)(threadIdx.x % THREADS); }
    static __device__ __forceinline__ int team() { return (int)(threadIdx.x / THREADS); }
    static __device__ __forceinline__ void sync() {
        if (W == 1) {
            __syncwarp();
        } else {
            __syncthreads();
        }
    }
    // Exclusive prefix over the team; s: 33 words.
    static __device__ __forceinline__ uint32_t excl_scan(uint32_t v, uint32_t* s, uint32_t* total) {
        if (W > 1) return block_excl_scan(v, s, total);
        const uint32_t incl = warp_incl_scan(v);
        *total = __shfl_sync(0xFFFFFFFFu, incl, 31);
        return incl - v;
    }
};

// A row's elements by position in the 128-byte lines that they lie in: position
// `lead` holds the first.
template <typename T>
struct LineRow {
    const T* line;                 // 128-byte aligned; row = line + lead
    int32_t lead, end;             // first position and the one after the last
    __device__ __forceinline__ LineRow(const T* row, int64_t V) {
        const uintptr_t a = (uintptr_t)row;
        lead = (int32_t)(a % LG_LINE / sizeof(T));
        line = reinterpret_cast<const T*>(a - a % LG_LINE);
        end = lead + (int32_t)V;
    }
    __device__ __forceinline__ int32_t lines() const {
        return (end + LG_LINE / (int)sizeof(T) - 1) / (LG_LINE / (int)sizeof(T));
    }
};

template <typename T>
struct Chunk {
    uint4 q[2];
    __device__ __forceinline__ float get(int i) const {
        return to_f32(reinterpret_cast<const T*>(q)[i]);
    }
};

// Chunk j of the row; -inf where the row has no element.
template <typename T>
__device__ __forceinline__ void load_chunk(const LineRow<T>& r, int32_t j, Chunk<T>& c) {
    const int32_t p = j * CHUNK<T>;
    if (p >= r.lead && p + CHUNK<T> <= r.end) {
        load32b(r.line + p, c.q);
    } else {
        T* e = reinterpret_cast<T*>(c.q);
#pragma unroll
        for (int i = 0; i < CHUNK<T>; ++i)
            e[i] = p + i >= r.lead && p + i < r.end ? r.line[p + i] : from_f32<T>(-CUDART_INF_F);
    }
}
// (written once and first to leave L2, which holds what is read again: distillation of 2,048 x
// 131,072 bf16 237 us without, 228 with it)
__device__ __forceinline__ void store32b_first(void* p, const uint4* q) {
    asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(q[0].x),
                 "r"(q[0].y), "r"(q[0].z), "r"(q[0].w), "r"(q[1].x), "r"(q[1].y), "r"(q[1].z),
                 "r"(q[1].w)
                 : "memory");
}

// A chunk of the result at position pos of rows that lie like row (out = row - lead).
template <typename T, typename TO>
__device__ __forceinline__ void store_chunk(const LineRow<T>& row, TO* out, int32_t pos,
                                            const Chunk<TO>& o) {
    if (pos >= row.lead && pos + CHUNK<T> <= row.end) {
        store32b_first(out + pos, o.q);
    } else {
        const TO* x = reinterpret_cast<const TO*>(o.q);
#pragma unroll
        for (int i = 0; i < CHUNK<T>; ++i)
            if (pos + i >= row.lead && pos + i < row.end) out[pos + i] = x[i];
    }
}
template <typename T>
__device__ __forceinline__ void no_chunk(Chunk<T>& c) {
    T* e = reinterpret_cast<T*>(c.q);
#pragma unroll
    for (int i = 0; i < CHUNK<T>; ++i) e[i] = from_f32<T>(-CUDART_INF_F);
}

struct Soft {
    float m, s, u;
};

__device__ __forceinline__ f32x2 ex2_2(f32x2 a) {
    const float2 v = parts(a);
    return pair(ex2(v.x), ex2(v.y));
}

template <typename T>
__device__ __forceinline__ void put_pair(Chunk<T>& q, int i, f32x2 a) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<f32x2*>(q.q)[i] = a;
    } else {
        reinterpret_cast<uint32_t*>(q.q)[i] = narrow(a, T{});
    }
}
// The pairs of a chunk, not below `low` (NaN stays), and its largest value (of what was
// there; NaN if there is one).
template <typename T>
struct Pairs {
    typedef typename Twin<T>::type T2;
    static __device__ __forceinline__ float largest(const Chunk<T>& q) {
        const T2* w = reinterpret_cast<const T2*>(q.q);
        T2 m = __hmax2_nan(w[0], w[1]);
#pragma unroll
        for (int i = 2; i < 8; ++i) m = __hmax2_nan(m, w[i]);
        const float2 v = parts(widen(m));
        return max_nan(v.x, v.y);
    }
    // (bf16 holds `low` near enough: m is at most 2^16, so it is off by 256 / c at most;
    // fp16 may not reach it)
    template <bool CUT>
    static __device__ __forceinline__ f32x2 get(const Chunk<T>& q, int i, float low) {
        T2 w = reinterpret_cast<const T2*>(q.q)[i];
        if (CUT && T2_IS_BF16) {
            T2 l;
            l.x = l.y = from_f32<T>(low);
            w = __hmax2_nan(w, l);
        }
        const f32x2 v = widen(w);
        if (!CUT || T2_IS_BF16) return v;
        const float2 f = parts(v);
        return pair(max_nan(f.x, low), max_nan(f.y, low));
    }
    static constexpr bool T2_IS_BF16 = Twin<T>::bf16;
};
template <>
struct Pairs<float> {
    static __device__ __forceinline__ float largest(const Chunk<float>& q) {
        float m = q.get(0);
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max_nan(m, q.get(i));
        return m;
    }
    template <bool CUT>
    static __device__ __forceinline__ f32x2 get(const Chunk<float>& q, int i, float low) {
        const float a = q.get(2 * i), b = q.get(2 * i + 1);
        return CUT ? pair(max_nan(a, low), max_nan(b, low)) : pair(a, b);
    }
};

// What a thread has summed: s and u in two halves each, and the value below which
// 2^(c z - m) is 0 (fp32's smallest is 2^-126, and ex2 flushes; t must stay finite in u).
struct Running {
    float m, low;
    f32x2 s, u;
};
constexpr float LG_BELOW = 400.0f;

// Adds chunks; `top` gets the largest value of each (NaN if it holds one).
template <typename T, bool ENTROPY, int N>
__device__ __forceinline__ void add_chunks(const Chunk<T>* q, float* top, Running& a, float c,
                                           float inv_c) {
    float all = -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < N; ++k) all = max_nan(all, top[k] = Pairs<T>::largest(q[k]));
    const float reach = all * c;
    if (reach < -2.0f * LG_FAR) return;
    if (!(reach <= a.m)) {
        const float m = ceilf(reach), f = ex2(a.m - m);
        const f32x2 ff = pair(f, f);
        if (ENTROPY) a.u = mul2(fma2(pair(a.m - m, a.m - m), a.s, a.u), ff);
        a.s = mul2(a.s, ff);
        a.m = m;
        a.low = (m - LG_BELOW) * inv_c;
    }
    const f32x2 cc = pair(c, c), mm = pair(-a.m, -a.m);
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < CHUNK<T> / 2; ++i) {
            const f32x2 t = fma2(Pairs<T>::template get<ENTROPY>(q[k], i, a.low), cc, mm), e = ex2_2(t);
            a.s = add2(a.s, e);
            if (ENTROPY) a.u = fma2(e, t, a.u);
        }
}

// The lanes' statistics, joined in every lane.
__device__ __forceinline__ Soft warp_join(Soft a) {
    float m = a.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float f = ex2(a.m - m);
    a.u = fmaf(a.m - m, a.s, a.u) * f;
    a.s *= f;
    a.m = m;
    a.s = warp_sum(a.s);
    a.u = warp_sum(a.u);
    return a;
}

__device__ __forceinline__ uint32_t order_key(float x) {      // order of the values, NaN on top
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(x + 0.0f);             // (-0 is 0)
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// f(FLIGHT chunks, the number of the first, those of the others THREADS apart, end) for the
// chunks of lines [line0, line1); a chunk from `end` on holds nothing but -inf.  Every thread
// of a warp makes the same calls.  BACK: the last batch first, which L2 still holds.  Batches
// that lie in the row as a whole are loaded without a check of each chunk (with it and the
// check of the running maximum for each chunk: 7.3 instructions an element, without 5.7).
template <int W, int FLIGHT, bool BACK = false, typename T, typename F>
__device__ __forceinline__ void for_chunks(const LineRow<T>& row, int32_t line0, int32_t line1, F f) {
    constexpr int N = Team<W>::THREADS;
    const int32_t end = line1 * 4;
    const int32_t in0 = (row.lead + CHUNK<T> - 1) / CHUNK<T>, in1 = min(end, row.end / CHUNK<T>);
#pragma unroll 1
    for (int32_t i0 = line0 * 4; i0 < end; i0 += N * FLIGHT) {
        const int32_t j0 = BACK ? line0 * 4 + (end - 1 - i0) / (N * FLIGHT) * (N * FLIGHT) : i0;
        Chunk<T> q[FLIGHT];
        const int32_t j = j0 + Team<W>::thread();
        if (j0 >= in0 && j0 + N * FLIGHT <= in1) {
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) load32b(row.line + (j + k * N) * CHUNK<T>, q[k].q);
        } else {
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) {
                if (j + k * N < end) {
                    load_chunk(row, j + k * N, q[k]);
                } else {
                    no_chunk(q[k]);
                }
            }
        }
        f(q, j, end);
    }
}

// The statistics of all threads of a row, in each of them (s_soft: W + 1 entries).  Also a
// barrier of the team and cluster.
template <int W>
__device__ __forceinline__ Soft row_join(Soft a, int blocks, Soft* s_soft) {
    a = warp_join(a);
    if (W == 1) return a;
    if (lane_id() == 0) s_soft[warp_id()] = a;
    __syncthreads();
    const Soft none = {LG_START, 0.0f, 0.0f};
    a = warp_join(lane_id() < W ? s_soft[lane_id()] : none);
    if (blocks == 1) return a;
    if (threadIdx.x == 0) s_soft[W] = a;
    cluster_sync();
    a = none;
    if ((int)lane_id() < blocks) {
        const uint32_t at = in_block(smem_u32(&s_soft[W]), lane_id());
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(a.m) : "r"(at));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(a.s) : "r"(at + 4));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(a.u) : "r"(at + 8));
    }
    return warp_join(a);
}

// A row's softmax: p(z) = 2^(c z - m) / s, or 2^(c (z - m)) / s where m is far.
struct RowSoft {
    float m, s, u, log2s;
    bool far;
    __device__ __forceinline__ float shifted(float z, float c) const {
        return far ? c * (z - m) : fmaf(z, c, -m);
    }
    __device__ __forceinline__ float prob(float z, float c) const {        // (times s)
        return s == 0.0f ? 0.0f : ex2(shifted(z, c));
    }
    __device__ __forceinline__ float log_prob(float z, float c, float scale) const {
        if (z == -CUDART_INF_F && s == s) return z;
        if (far) return fmaf(z - m, scale, -logf(s));
        const float t = fmaf(z, c, -m);
        return t < -LG_FAR ? fmaf(z, scale, -log_sum(scale)) : LN2 * (t - log2s);     // (t may overflow)
    }
    __device__ __forceinline__ float log_sum(float scale) const {
        if (s == 0.0f) return -CUDART_INF_F;
        return far ? fmaf(m, scale, logf(s)) : fmaf(m, LN2_HI, fmaf(m, LN2_LO, logf(s)));
    }
    __device__ __forceinline__ float entropy() const {
        return s == 0.0f ? 0.0f : LN2 * (log2s - u / s);
    }
};

// The row again, with its largest value as the reference.  (Rare, and the same for all
// blocks of the cluster.)
template <int W, typename T>
__device__ __forceinline__ Soft far_row(const LineRow<T>& row, int32_t line0, int32_t line1, float c,
                                        int blocks, Soft* s_soft) {
    float top = -CUDART_INF_F;
    for_chunks<W, 1>(row, line0, line1, [&](const Chunk<T>* q, int32_t, int32_t) {
#pragma unroll
        for (int i = 0; i < CHUNK<T>; ++i) top = max_nan(top, q->get(i));
    });
    // (as a sum of one term, whose reference it is)
    if (blocks > 1) cluster_sync(); else Team<W>::sync();      // what s_soft held has been read
    top = max_nan(row_join<W>({top, 0.0f, 0.0f}, blocks, s_soft).m, LG_START);     // (finite: -inf - top is -inf)
    if (blocks > 1) cluster_sync(); else Team<W>::sync();
    Soft a = {0.0f, 0.0f, 0.0f};
    for_chunks<W, 1>(row, line0, line1, [&](const Chunk<T>* q, int32_t, int32_t) {
#pragma unroll
        for (int i = 0; i < CHUNK<T>; ++i) {
            const float t = c * (q->get(i) - top), e = ex2(t);
            a.s += e;
            a.u = fmaf(e, fmaxf(t, -1e4f), a.u);
        }
    });
    a = row_join<W>(a, blocks, s_soft);
    a.m = top;
    return a;
}

// A row's softmax from what its threads have summed.
template <int W, typename T>
__device__ __forceinline__ RowSoft join_softmax(const LineRow<T>& row, int32_t line0, int32_t line1,
                                                float c, int blocks, Soft* s_soft, const Running& run) {
    const float2 s = parts(run.s), u = parts(run.u);
    Soft a = {run.m, s.x + s.y, u.x + u.y};
    a = row_join<W>(a, blocks, s_soft);
    RowSoft r;
    r.far = a.s == 0.0f || !(fabsf(a.m) <= LG_FAR) || a.s != a.s;
    if (r.far) a = far_row<W>(row, line0, line1, c, blocks, s_soft);
    r.m = a.m;
    r.s = a.s;
    r.u = a.u;
    r.log2s = log2f(a.s);
    return r;
}

// 32-byte chunks of a group, whose largest value the top selection keeps: a warp's rows are
// short, and so are their groups (16,384 rows of 8,000 bf16, top 100: 758 us by lines, 157 so).
template <int W>
constexpr int GROUP = W == 1 ? 1 : 4;

// The thread's part of the sums of a row, of which a block takes lines [line0, line1); TOP:
// the largest value of each line in tops[line].
template <int W, typename T, bool ENTROPY, bool TOP>
__device__ __forceinline__ Running row_sums(const LineRow<T>& row, int32_t line0, int32_t line1,
                                            float c, float* tops) {
    constexpr int N = Team<W>::THREADS;
    Running run = {LG_START, LG_START, 0, 0};
    const float inv_c = 1.0f / c;
    for_chunks<W, LG_FLIGHT>(row, line0, line1, [&](const Chunk<T>* q, int32_t j, int32_t end) {
        float top[LG_FLIGHT];
        add_chunks<T, ENTROPY, LG_FLIGHT>(q, top, run, c, inv_c);
        if (TOP) {
#pragma unroll
            for (int k = 0; k < LG_FLIGHT; ++k) {
                if (GROUP<W> == 1) {
                    if (j + k * N < end) tops[j + k * N] = top[k];
                    continue;
                }
                float line = max_nan(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], 1));
                line = max_nan(line, __shfl_xor_sync(0xFFFFFFFFu, line, 2));
                if ((threadIdx.x & 3) == 0 && j + k * N < end) tops[(j + k * N) >> 2] = line;
            }
        }
    });
    return run;
}

// ------------------------------------------- log-probabilities of given tokens

struct LogprobParams {
    const void* z;
    const void* ids;               // or null
    float* logprob;                // or null, like each of these
    float* entropy;
    float* lse;
    int32_t* top_ids;              // [T][top]
    float* top_logprobs;
    Ctrl* ctrl;
    int64_t T, V, ldz, padding;
    int32_t id64, top, blocks;     // blocks of a row's cluster
    int32_t scan;                  // the first cluster checks the ids
    float c, scale;
};

__device__ __forceinline__ int64_t load_id(const void* ids, int32_t id64, int64_t i) {
    return id64 ? static_cast<const int64_t*>(ids)[i] : (int64_t)static_cast<const int32_t*>(ids)[i];
}

// One block: the status of a call whose ids are few.
__device__ __forceinline__ void scan_ids(const void* ids, int32_t id64, int64_t n, int64_t V,
                                         int64_t padding, bool negative_ok, Ctrl* ctrl) {
    int bad = 0;
    for (int64_t i = threadIdx.x; ids && i < n; i += blockDim.x) {
        const int64_t id = load_id(ids, id64, i);
        bad |= (id < 0 && !negative_ok && id != padding) || (id >= V && id != padding);
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        ctrl->path_small = 0;
        ctrl->status = bad ? ST_BAD_INPUT : 0u;
    }
}

// The groups that hold any of the row's elements.
template <int W, typename T>
__device__ __forceinline__ int first_group(const LineRow<T>& row) {
    return row.lead / (GROUP<W> * CHUNK<T>);
}
template <int W, typename T>
__device__ __forceinline__ int end_group(const LineRow<T>& row) {
    return (row.end + GROUP<W> * CHUNK<T> - 1) / (GROUP<W> * CHUNK<T>);
}

constexpr int TL_BINS = 512;               // 32 an octave of 1 + m - c z

template <int W>
struct TopShared {
    static constexpr int GROUPS = W == 1 ? 256 : 512;      // that are read again
    static constexpr int LIST = W == 1 ? 256 : 512;        // candidates that are ranked
    uint32_t hist[TL_BINS];
    uint32_t groups, n;                    // lengths of the lists
    uint32_t count[2 * W];
    uint32_t scan[33];
    uint16_t group[GROUPS];
    __align__(16) unsigned long long list[LIST];   // key, then the lower index first
};

// Sum of v over the team (every thread gets it); `flip`: not the last call's.
template <int W>
__device__ __forceinline__ uint32_t team_count(uint32_t v, uint32_t* s, int flip) {
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    if (W == 1) return v;
    if (lane_id() == 0) s[flip * W + warp_id()] = v;
    __syncthreads();
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) n += s[flip * W + i];
    return n;
}

// The largest key that at least `want` of the team's keys reach, bit by bit;
// `count(k)` counts the thread's keys >= k.  LOW: bits below it are equal in all keys.
template <int W, int LOW, typename F>
__device__ __forceinline__ uint32_t team_threshold(uint32_t want, uint32_t* s, F count) {
    uint32_t k = 0;
#pragma unroll 1
    for (int bit = 31; bit >= LOW; --bit) {
        const uint32_t up = k | (1u << bit);
        if (team_count<W>(count(up), s, bit & 1) >= want) k = up;
    }
    Team<W>::sync();
    return k;
}

// 1 + m - c z, at least 1: falls as z grows, and its bits count bins.
__device__ __forceinline__ float depth(float z, float c, float m) {
    return fmaxf(fmaf(-z, c, m), 0.0f) + 1.0f;
}
__device__ __forceinline__ uint32_t depth_bin(float d) {
    return min((__float_as_uint(d) - 0x3F800000u) >> 18, (uint32_t)TL_BINS - 1);
}

// The first bin up to which the histogram holds `want` (every warp finds it), and how many.
__device__ __forceinline__ uint32_t bin_of(const uint32_t* hist, uint32_t want, uint32_t& upto) {
    constexpr int EACH = TL_BINS / 32;
    const uint32_t lane = lane_id();
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) n += hist[lane * EACH + ((i + lane) & (EACH - 1))];
    const uint32_t incl = warp_incl_scan(n);
    const int src = __ffs(__ballot_sync(0xFFFFFFFFu, incl >= want)) - 1;
    const uint32_t run = __shfl_sync(0xFFFFFFFFu, incl - n, src);
    const uint32_t v = lane < EACH ? hist[src * EACH + lane] : 0u;
    const uint32_t in2 = run + warp_incl_scan(v);
    const int at = __ffs(__ballot_sync(0xFFFFFFFFu, in2 >= want)) - 1;
    upto = __shfl_sync(0xFFFFFFFFu, in2, at);
    return (uint32_t)(src * EACH + at);
}

// The lists by exact counts, where the bins hold too many: the K-th largest of the groups'
// largest values, t; the groups above it and the first of those at it; of their
// elements the ones above the K-th largest of them and the first of those at it.
template <int W, typename T>
__device__ __forceinline__ void list_exactly(const LineRow<T>& row, int K, const float* tops,
                                             TopShared<W>& S) {
    constexpr int N = Team<W>::THREADS;
    constexpr int LOW = sizeof(T) == 4 ? 0 : 13;       // bf16 keys end 16 bits up, fp16's 13
    // (keys whose low bits are set, a negative value's, compare as the value they stand for)
    constexpr uint32_t mask = ~((1u << LOW) - 1);
    const int tid = Team<W>::thread();
    const int g_first = first_group<W>(row), g_end = end_group<W>(row), groups = g_end - g_first;
    const int want = min(min(K, groups), TopShared<W>::GROUPS);
    const int per = (groups + N - 1) / N;
    // the thread's groups are neighbours, so that a scan over threads is one over groups
    const int g0 = min(g_end, g_first + tid * per), g1 = min(g_end, g0 + per);
    uint32_t t = 0;
    if (groups > K)
        t = team_threshold<W, LOW>((uint32_t)K, S.count, [&](uint32_t k) {
            uint32_t n = 0;
            for (int g = g_first + tid; g < g_end; g += N) n += order_key(tops[g]) >= k;
            return n;
        });
    uint32_t above = 0, equal = 0;
    for (int g = g0; g < g1; ++g) {
        const uint32_t k = order_key(tops[g]) & mask;
        above += k > t;
        equal += k == t;
    }
    uint32_t tot;
    const uint32_t before = Team<W>::excl_scan(above << 16 | equal, S.scan, &tot);
    {
        const uint32_t quota = (uint32_t)want - (tot >> 16);
        uint32_t a = before >> 16, e = before & 0xFFFF;
        for (int g = g0; g < g1; ++g) {
            const uint32_t k = order_key(tops[g]) & mask;
            if (k > t || (k == t && e < quota)) S.group[a + min(e, quota)] = (uint16_t)g;
            a += k > t;
            e += k == t;
        }
    }
    Team<W>::sync();
    // f(key, position) for their elements, in order: the thread's chunks are neighbours too
    const int chunks = want * GROUP<W>, each = (chunks + N - 1) / N;
    const auto elements = [&](auto f) {
#pragma unroll 1
        for (int j = tid * each; j < min(chunks, tid * each + each); ++j) {
            const int32_t chunk = S.group[j / GROUP<W>] * GROUP<W> + j % GROUP<W>;
            Chunk<T> q;
            load_chunk(row, chunk, q);
#pragma unroll
            for (int e = 0; e < CHUNK<T>; ++e) {
                const int32_t pos = chunk * CHUNK<T> + e;
                if (pos >= row.lead && pos < row.end) f(order_key(q.get(e)), pos);
            }
        }
    };
    uint32_t n = 0;
    elements([&](uint32_t, int32_t) { ++n; });
    n = team_count<W>(n, S.count, 0);
    Team<W>::sync();
    const uint32_t need = min((uint32_t)K, n);
    const uint32_t cut = team_threshold<W, LOW>(need, S.count, [&](uint32_t k) {
        uint32_t c = 0;
        elements([&](uint32_t key, int32_t) { c += key >= k; });
        return c;
    });
    above = equal = 0;
    elements([&](uint32_t key, int32_t) {
        above += (key & mask) > cut;
        equal += (key & mask) == cut;
    });
    const uint32_t b = Team<W>::excl_scan(above << 16 | equal, S.scan, &tot);
    const uint32_t quota = need - (tot >> 16);
    n = b & 0xFFFF;                                         // equal ones before the thread's
    uint32_t first = (b >> 16) + min(n, quota);
    elements([&](uint32_t key, int32_t pos) {
        const bool eq = (key & mask) == cut;
        if ((key & mask) > cut || (eq && n < quota))
            S.list[first++] = (unsigned long long)key << 32 | (uint32_t)(row.end - 1 - pos);
        n += eq;
    });
    if (tid == 0) S.n = need;
    Team<W>::sync();
}

// The top K of the row by (value descending, index ascending), one team.
//
// The K-th largest value is at least the K-th largest of the groups' largest ones.  A
// histogram of those by their distance from the row's largest gives a bin that holds it;
// the groups up to that bin are read again, and their elements up to it, hardly more than
// K, are ranked by comparing each with each.  (While groups are few, a histogram of all
// elements instead: near K groups have too many elements up to the least of them.)  (Exact counts over 16 or 32 bits of the
// lines' keys instead of bins: 380 us more for 4,096 rows of 131,072 bf16.)
template <int W, typename T>
__device__ __forceinline__ void select_top(const LogprobParams& p, const LineRow<T>& row, int64_t r,
                                           const float* tops, TopShared<W>& S, const RowSoft& soft) {
    constexpr int N = Team<W>::THREADS, LIST = TopShared<W>::LIST;
    const int tid = Team<W>::thread();
    const int g_first = first_group<W>(row), g_end = end_group<W>(row), groups = g_end - g_first;
    const int K = p.top;
    const float c = p.c, m = soft.m;
    bool exactly = soft.far;                   // (distances mean nothing)
    if (!exactly) {
        for (int i = tid; i < TL_BINS; i += N) S.hist[i] = 0;
        if (tid == 0) S.groups = S.n = 0;
        Team<W>::sync();
        const bool some = groups > (W == 1 ? 2 * K : K), binned = some || p.V > LIST;
        uint32_t bin = TL_BINS - 1;
        if (some) {
            for (int g = g_first + tid; g < g_end; g += N)
                atomicAdd(&S.hist[depth_bin(depth(tops[g], c, m))], 1u);
        } else if (binned) {
            for (int j = tid; j < row.lines() * 4; j += N) {
                Chunk<T> q;
                load_chunk(row, j, q);
#pragma unroll
                for (int e = 0; e < CHUNK<T>; ++e) {
                    const int32_t pos = j * CHUNK<T> + e;
                    if (pos >= row.lead && pos < row.end)
                        atomicAdd(&S.hist[depth_bin(depth(q.get(e), c, m))], 1u);
                }
            }
        }
        if (binned) {
            Team<W>::sync();
            uint32_t upto;
            bin = bin_of(S.hist, (uint32_t)min((int64_t)K, p.V), upto);
            exactly = upto > (uint32_t)(some ? TopShared<W>::GROUPS : LIST);
        }
        if (!exactly) {
            // (the last bin has no end)
            const float edge = bin == TL_BINS - 1 ? CUDART_INF_F
                                                  : __uint_as_float(0x3F800000u + ((bin + 1) << 18));
            const auto within = [&](float z) { return depth(z, c, m) < edge || bin == TL_BINS - 1; };
            if (some) {
                for (int g = g_first + tid; g < g_end; g += N)
                    if (within(tops[g])) S.group[atomicAdd(&S.groups, 1u)] = (uint16_t)g;
                Team<W>::sync();
            }
            const int chunks = some ? (int)S.groups * GROUP<W> : row.lines() * 4;
            for (int j = tid; j < chunks; j += N) {
                const int32_t chunk = some ? S.group[j / GROUP<W>] * GROUP<W> + j % GROUP<W> : j;
                const int32_t pos = chunk * CHUNK<T>;
                Chunk<T> q;
                load_chunk(row, chunk, q);
                // which are within, then places for all of them at once
                uint32_t in = 0;
#pragma unroll
                for (int e = 0; e < CHUNK<T>; ++e) in |= (uint32_t)within(q.get(e)) << e;
                if (pos < row.lead) in &= ~0u << min(row.lead - pos, 31);
                if (pos + CHUNK<T> > row.end) in &= (1u << max(row.end - pos, 0)) - 1;
                if (in == 0) continue;
                uint32_t at = atomicAdd(&S.n, (uint32_t)__popc(in));
#pragma unroll
                for (int e = 0; e < CHUNK<T>; ++e)
                    if (in >> e & 1) {
                        if (at < LIST)
                            S.list[at] = (unsigned long long)order_key(q.get(e)) << 32 |
                                         (uint32_t)(row.end - 1 - pos - e);
                        ++at;
                    }
            }
            Team<W>::sync();
            exactly = S.n > LIST;
            Team<W>::sync();
        }
    }
    if (exactly) list_exactly<W>(row, K, tops, S);
    const uint32_t n = S.n;
    for (uint32_t i = tid; i < n; i += N) {
        const unsigned long long mine = S.list[i];
        uint32_t rank = 0;
#pragma unroll 4
        for (uint32_t j = 0; j + 1 < n; j += 2) {
            const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(S.list + j);
            rank += (two.x > mine) + (two.y > mine);
        }
        if (n & 1) rank += S.list[n - 1] > mine;
        if (rank < (uint32_t)K) {
            const float z = key_value((uint32_t)(mine >> 32));
            const int32_t id = row.end - 1 - (int32_t)(uint32_t)mine - row.lead;
            if (p.top_ids) p.top_ids[r * K + rank] = id;
            if (p.top_logprobs) p.top_logprobs[r * K + rank] = soft.log_prob(z, p.c, p.scale);
        }
    }
    for (int i = (int)min((int64_t)K, p.V) + tid; i < K; i += N) {
        if (p.top_ids) p.top_ids[r * K + i] = -1;
        if (p.top_logprobs) p.top_logprobs[r * K + i] = -CUDART_INF_F;
    }
}

// Bound by the bytes of z without the top (4,096 x 131,072 bf16: 160 to 178 us, 6.0 to 6.7 TB/s),
// with it by the selection, during which a block reads nothing (top 64: 207 to 226 us, top 128:
// 250; short rows: 16,384 x 8,000, top 20, 86 us, top 100, 157, most of it the ranks).  One row
// of 131,072 fp32 with its top 20, 16 blocks: 9 us, the chain of its steps.
template <int W, bool TOP>
constexpr int LOGPROB_BLOCKS = (TOP ? 3 : 4) * 256 / Team<W>::BLOCK;       // of an SM

template <int W, typename T, bool ENTROPY, bool TOP>
__global__ void __launch_bounds__(Team<W>::BLOCK, LOGPROB_BLOCKS<W, TOP>)
    logprob_kernel(const LogprobParams p) {
    constexpr int N = Team<W>::THREADS, TEAMS = Team<W>::TEAMS;
    extern __shared__ __align__(16) float s_dyn[];     // TOP: the groups' largest values
    __shared__ Soft s_soft[W + 1];
    __shared__ TopShared<W> S[TEAMS];
    pdl_launch();
    pdl_wait();
    const int64_t block = (int64_t)(blockIdx.x / (unsigned)p.blocks) - p.scan;
    const int rank = (int)(blockIdx.x % (unsigned)p.blocks), tid = Team<W>::thread();
    if (block < 0) {
        if (rank == 0) scan_ids(p.ids, p.id64, p.T, p.V, p.padding, false, p.ctrl);
        return;
    }
    const int64_t r = block * TEAMS + Team<W>::team();
    if (r >= p.T) return;
    float* s_tops = s_dyn + Team<W>::team() * (LG_SMALL * 4);
    int64_t id = -1;
    bool skip = false, ok = false;
    if (p.ids) {
        id = load_id(p.ids, p.id64, r);
        skip = id == p.padding;
        ok = id >= 0 && id < p.V;
        if (!skip && !ok && !p.scan && rank == 0 && tid == 0) atomicOr(&p.ctrl->status, ST_BAD_INPUT);
    }
    if (skip) {
        if (rank != 0) return;
        if (tid == 0) {
            if (p.logprob) p.logprob[r] = 0.0f;
            if (p.entropy) p.entropy[r] = 0.0f;
            if (p.lse) p.lse[r] = 0.0f;
        }
        for (int i = tid; TOP && i < p.top; i += N) {
            if (p.top_ids) p.top_ids[r * p.top + i] = -1;
            if (p.top_logprobs) p.top_logprobs[r * p.top + i] = -CUDART_INF_F;
        }
        return;
    }
    const T* z = static_cast<const T*>(p.z) + r * p.ldz;
    float zt = 0.0f;
    if (ok && rank == 0 && tid == N - 32) zt = to_f32(z[id]);
    const LineRow<T> row(z, p.V);
    const int32_t lines = row.lines();
    const int32_t share = ((lines + p.blocks - 1) / p.blocks + 3) & ~3;
    const int32_t line0 = min(lines, rank * share), line1 = min(lines, line0 + share);
    const Running run = row_sums<W, T, ENTROPY, TOP>(row, line0, line1, p.c, s_tops);
    const RowSoft a = join_softmax<W>(row, line0, line1, p.c, p.blocks, s_soft, run);
    if (TOP && rank == 0) {
        // the other blocks' lines, several on their way at once
        if (W > 1 && p.blocks > 1) {
            constexpr int AHEAD = 4;
            for (int32_t l0 = share; l0 < lines; l0 += AHEAD * N * 4) {
                float4 k[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int32_t l = l0 + (i * N + tid) * 4;      // (of one block: shares of fours)
                    if (l < lines)
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(k[i].x), "=f"(k[i].y), "=f"(k[i].z), "=f"(k[i].w)
                                     : "r"(in_block(smem_u32(s_tops + l), (uint32_t)(l / share))));
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int32_t l = l0 + (i * N + tid) * 4;
                    if (l < lines) *reinterpret_cast<float4*>(s_tops + l) = k[i];
                }
            }
        }
        Team<W>::sync();
        select_top<W, T>(p, row, r, s_tops, S[Team<W>::team()], a);
    }
    // (by the last warp: the first ones rank)
    if (rank == 0 && tid == N - 32) {
        if (p.logprob) p.logprob[r] = ok ? a.log_prob(zt, p.c, p.scale) : 0.0f;
        if (ENTROPY && p.entropy) p.entropy[r] = a.entropy();
        if (p.lse) p.lse[r] = a.log_sum(p.scale);
    }
    if (W > 1 && p.blocks > 1) cluster_sync();     // no block leaves while its memory is read
}

// ------------------------------------- their gradient in the logits

struct LogprobGradParams {
    const void* z;
    const void* ids;               // or null
    const float* lse;
    const float* entropy;          // or null
    const float* g;                // or null: gradient of the log-probabilities
    const float* h;                // or null: of the entropies
    void* dz;
    Ctrl* ctrl;
    int64_t T, V, ldz, lddz, padding;
    int32_t id64, parts;           // warps of a row
    int32_t scan;                  // the first block checks the ids
    float c, scale;
};

constexpr int LD_THREADS = 128, LD_WARPS = LD_THREADS / 32;
constexpr int LD_LINES = 128;              // lines of a row that one warp takes
// Most |lse| whose p = exp(scale z - lse) is kept: an fp32 lse is off by 2^-24 of itself twice
// (its sum's, its rounding), so p by 2^-16 at most.
constexpr float LD_LSE = 128.0f;

// The gradient of a row whose lse is too far from 0 to hold log p (or is -inf where the row is
// not): a team sums the row again, and reads it a third time.  (One team a row, since others'
// results may lie where it reads.)  2,048 x 131,072 bf16, all rows far: 266 us, none: 165.
template <int W, typename T, typename TO, bool SAME, bool ENTROPY>
__device__ __forceinline__ void far_gradient(const T* z, TO* dz, int32_t V, int32_t id, float c, float g,
                                             float h, float H, Soft* s_soft) {
    constexpr int N = Team<W>::THREADS;
    const LineRow<T> row(z, V);
    const int32_t lines = row.lines();
    const Running run = row_sums<W, T, false, false>(row, 0, lines, c, nullptr);
    const RowSoft a = join_softmax<W>(row, 0, lines, c, 1, s_soft, run);
    const bool none = a.s == 0.0f;                     // (all -inf)
    // with p = 2^t / s: -p (g + h (log p + H)) = 2^t (k0 + k1 t), and g more at the token
    const float inv = none ? 0.0f : 1.0f / a.s;
    const float k1 = ENTROPY && !none ? -h * LN2 * inv : 0.0f;
    const float k0 = none ? 0.0f : (ENTROPY ? fmaf(-h, H - LN2 * a.log2s, -g) : -g) * inv;
    const auto values = [&](f32x2 v) {
        f32x2 t = a.far ? mul2(add2(v, pair(-a.m, -a.m)), pair(c, c))
                        : fma2(v, pair(c, c), pair(-a.m, -a.m));
        const f32x2 e = ex2_2(t);
        if (!ENTROPY) return mul2(e, pair(k0, k0));
        const float2 f = parts(t);                     // (times e, which is 0 there)
        t = pair(max_nan(f.x, -1e4f), max_nan(f.y, -1e4f));
        return mul2(e, fma2(t, pair(k1, k1), pair(k0, k0)));
    };
    if (none) g = 0.0f;
    if (SAME) {
        const int32_t token = id < 0 ? -1 : id + row.lead;
        for_chunks<W, 2>(row, 0, lines, [&](const Chunk<T>* q, int32_t j, int32_t end) {
#pragma unroll
            for (int k = 0; k < 2; ++k, j += N) {
                if (j >= end) continue;
                const int32_t pos = j * CHUNK<T>;
                Chunk<TO> o;
#pragma unroll
                for (int i = 0; i < CHUNK<T> / 2; ++i) {
                    f32x2 v = values(Pairs<T>::template get<false>(q[k], i, 0.0f));
                    if (token >> 1 == (pos >> 1) + i)
                        v = add2(v, pair(token & 1 ? 0.0f : g, token & 1 ? g : 0.0f));
                    put_pair(o, i, v);
                }
                store_chunk(row, dz - row.lead, pos, o);
            }
        });
    } else {
#pragma unroll 4
        for (int32_t i = Team<W>::thread(); i < V; i += N) {
            float v = parts(values(pair(to_f32(z[i]), 0.0f))).x;
            if (i == id) v += g;
            dz[i] = from_f32<TO>(v);
        }
    }
}

// What a warp knows of its row.
template <bool ENTROPY>
struct GradRow {
    int64_t r;
    int32_t part, id;              // id: -1 for none
    bool there, skip, bad;
    float lse, g, h, H;
    __device__ __forceinline__ GradRow(const LogprobGradParams& p, int64_t item) {
        r = item / p.parts;
        part = (int)(item - r * p.parts);
        id = -1;
        there = r < p.T;
        skip = !there;
        bad = false;
        lse = g = h = H = 0.0f;
        if (!there) return;
        if (p.ids) {
            const int64_t v = load_id(p.ids, p.id64, r);
            skip = v == p.padding;
            if (v >= 0 && v < p.V) {
                id = (int32_t)v;
            } else {
                bad = !skip;
            }
        }
        lse = p.lse[r];
        g = id >= 0 && p.g ? p.scale * p.g[r] : 0.0f;
        if (ENTROPY) {
            h = p.scale * p.h[r];
            H = p.entropy[r];
        }
        skip = skip || (g == 0.0f && h == 0.0f);
    }
    __device__ __forceinline__ bool far() const { return !skip && fabsf(lse) > LD_LSE; }
};

// The far rows that the warps of a block have the first part of, by the whole block; of a
// call whose rows are a warp each, the calling warp's.  (A call, so that it costs the other rows
// no registers.)
template <typename T, typename TO, bool SAME, bool ENTROPY>
__device__ __noinline__ void far_rows(const LogprobGradParams& p) {
    __shared__ Soft s_soft[LD_WARPS + 1];
    const int64_t first = ((int64_t)blockIdx.x - p.scan) * LD_WARPS;
    const auto gradient = [&](auto team, const GradRow<ENTROPY>& at) {
        far_gradient<decltype(team)::WARPS, T, TO, SAME, ENTROPY>(
            static_cast<const T*>(p.z) + at.r * p.ldz, static_cast<TO*>(p.dz) + at.r * p.lddz, (int32_t)p.V, at.id,
            p.c, at.g, at.h, at.H, s_soft);
    };
    if (p.parts == 1) {
        gradient(Team<1>{}, GradRow<ENTROPY>(p, first + warp_id()));
        return;
    }
    for (int i = 0; i < LD_WARPS; ++i) {
        const GradRow<ENTROPY> at(p, first + i);
        if (!at.far() || at.part != 0) continue;
        gradient(Team<LD_WARPS>{}, at);
        __syncthreads();
    }
}

// dz_i = scale (g (delta_i,id - p_i) - h p_i (log p_i + entropy)), a warp a part of a row.
// Bound by the bytes of z and dz: 2,048 x 131,072 bf16 with both gradients in 162 us, 6.5 TB/s.
// SAME: z's and dz's rows lie alike in their lines.
template <typename T, typename TO, bool SAME, bool ENTROPY>
__global__ void __launch_bounds__(LD_THREADS, SAME ? 7 : 16)
    logprob_grad_kernel(const __grid_constant__ LogprobGradParams p) {
    pdl_launch();
    pdl_wait();
    if (p.scan && blockIdx.x == 0) {
        scan_ids(p.ids, p.id64, p.T, p.V, p.padding, false, p.ctrl);
        return;
    }
    const int lane = (int)lane_id();
    const int64_t item = ((int64_t)blockIdx.x - p.scan) * LD_WARPS + warp_id();
    GradRow<ENTROPY> at(p, item);
    // (the row's values are loaded again after the call, so that none is kept over it)
    if (p.parts == 1 ? at.far() : __syncthreads_or(at.far() && at.part == 0) != 0) {
        far_rows<T, TO, SAME, ENTROPY>(p);
        at = GradRow<ENTROPY>(p, item);
    }
    if (at.bad && !p.scan && at.part == 0 && lane == 0) atomicOr(&p.ctrl->status, ST_BAD_INPUT);
    if (!at.there || at.far()) return;
    const int64_t r = at.r;
    const int part = at.part;
    const T* z = static_cast<const T*>(p.z) + r * p.ldz;
    TO* dz = static_cast<TO*>(p.dz) + r * p.lddz;
    const int32_t id = at.id;
    const bool skip = at.skip;
    const float lse = at.lse, g = at.g, h = at.h, H = at.H;
    // -p (g + h (log p + H)), and g more at the token
    const float k0 = fmaf(-h, H, -g);
    auto values = [&](f32x2 v) {
        f32x2 t = fma2(v, pair(p.scale, p.scale), pair(-lse, -lse));
        if (ENTROPY) {                                     // (times e, which is 0 there)
            const float2 f = parts(t);
            t = pair(max_nan(f.x, -1e4f), max_nan(f.y, -1e4f));
        }
        const f32x2 e = ex2_2(mul2(t, pair(LOG2E, LOG2E)));
        return mul2(e, ENTROPY ? fma2(t, pair(-h, -h), pair(k0, k0)) : pair(-g, -g));
    };
    const LineRow<T> row(z, p.V);
    const int32_t lines = row.lines();
    // (the row is too long for as many parts as there are blocks: more rounds)
    for (int32_t line0 = part * LD_LINES; line0 < lines; line0 += p.parts * LD_LINES) {
        const int32_t line1 = min(lines, line0 + LD_LINES);
        if (SAME) {
            TO* out = dz - row.lead;
            const int32_t token = id < 0 ? -1 : id + row.lead;
            if (skip) {
                const Chunk<TO> zero = {};
                for (int32_t j = line0 * 4 + lane; j < line1 * 4; j += 32)
                    store_chunk(row, out, j * CHUNK<T>, zero);
                continue;
            }
            for_chunks<1, LG_FLIGHT>(row, line0, line1, [&](const Chunk<T>* q, int32_t j, int32_t end) {
#pragma unroll
                for (int k = 0; k < LG_FLIGHT; ++k, j += 32) {
                    if (j >= end) continue;
                    const int32_t pos = j * CHUNK<T>;
                    Chunk<TO> o;
#pragma unroll
                    for (int i = 0; i < CHUNK<T> / 2; ++i) {
                        f32x2 v = values(Pairs<T>::template get<false>(q[k], i, 0.0f));
                        if (token >> 1 == (pos >> 1) + i)
                            v = add2(v, pair(token & 1 ? 0.0f : g, token & 1 ? g : 0.0f));
                        put_pair(o, i, v);
                    }
                    store_chunk(row, out, pos, o);
                }
            });
        } else {
            constexpr int32_t per = LG_LINE / (int)sizeof(T);
            const int32_t i1 = min(line1 * per, row.end) - row.lead;
            for (int32_t i = max(line0 * per - row.lead, 0) + lane; i < i1; i += 32) {
                float v = 0.0f;
                if (!skip) {
                    v = parts(values(pair(to_f32(z[i]), 0.0f))).x;
                    if (i == id) v += g;
                }
                dz[i] = from_f32<TO>(v);
            }
        }
    }
}

// ------------------------------------ distillation from a teacher's top logits

struct DistillParams {
    const void* z;
    const void* ids;               // [T][K]
    const void* teacher;           // [T][K]
    const float* weight;           // or null
    float* loss;                   // or null
    void* dz;                      // or null
    Ctrl* ctrl;
    int64_t T, V, ldz, lddz;
    int32_t id64, teacher_type, K, blocks;
    int32_t scan;                  // the first cluster checks the ids
    float c, scale;
};

__device__ __forceinline__ float teacher_at(const DistillParams& p, int64_t i) {
    if (p.teacher_type == TOPK_EF_F32) return static_cast<const float*>(p.teacher)[i];
    if (p.teacher_type == TOPK_EF_BF16)
        return to_f32(static_cast<const __nv_bfloat16*>(p.teacher)[i]);
    return to_f32(static_cast<const __half*>(p.teacher)[i]);
}

// f times the probabilities of a chunk.
template <typename T, typename TO>
__device__ __forceinline__ Chunk<TO> grad_chunk(const Chunk<T>& v, const RowSoft& a, float c, float f) {
    Chunk<TO> o;
    if (!a.far) {
        const f32x2 cc = pair(c, c), mm = pair(-a.m, -a.m), ff = pair(f, f);
#pragma unroll
        for (int e = 0; e < CHUNK<T> / 2; ++e)
            put_pair(o, e, mul2(ex2_2(fma2(Pairs<T>::template get<false>(v, e, 0.0f), cc, mm)), ff));
    } else {
        TO* x = reinterpret_cast<TO*>(o.q);
#pragma unroll
        for (int e = 0; e < CHUNK<T>; ++e) x[e] = from_f32<TO>(f * a.prob(v.get(e), c));
    }
    return o;
}

// The teacher's entries, and what each warp has found of its own: their largest logit, the sum
// of their powers over it, and its part of the loss.
template <int W>
struct TeacherShared {
    float t[DL_MAX_K];
    __align__(16) int32_t id[DL_MAX_K];
    float2 soft[W];
    float gap[W];
};

// Largest logit and sum of powers over it, of two sets.
__device__ __forceinline__ float2 join_powers(float2 a, float2 b, float c) {
    const float m = max_nan(a.x, b.x);
    if (m == -CUDART_INF_F) return make_float2(m, 0.0f);
    return make_float2(m, fmaf(a.y, ex2((a.x - m) * c), b.y * ex2((b.x - m) * c)));
}

// loss = weight sum_k q_k (log q_k - log p_{id_k}),  q = softmax(scale teacher);
// dz = weight scale (p - q).  SAME: z's and dz's rows lie alike in their lines.
//
// Bound by the bytes of z and dz, and for short rows by the chain of a row's steps: so
// thread k keeps the teacher's k-th entry in registers, its softmax and the loss ride on the
// barriers that the row's sums and the gradient need anyway (a barrier for each step: 70 us
// instead of 65 for 4,096 rows of 8,192 bf16 by eight warps each; by four 43, by one, which is what
// it takes, 46, as rows of 16 KB go: 16,384 of them 153 and 122).  For the
// gradient the row is read again, out of L2: 228 to 234 us for 2,048 x 131,072 bf16 (4.5 to 4.6
// TB/s of z and dz), 115 for 4,096 x 32,768.  (Kept in shared memory instead, with the next row
// copied behind it, by blocks of 8, 16 or 32 warps: 255 to 290, and 148.  Fewer blocks fit, and
// they all read or all write at the same time.)
template <int W, typename T, typename TO, bool SAME>
__global__ void __launch_bounds__(Team<W>::BLOCK, 3 * 256 / Team<W>::BLOCK) distill_kernel(const DistillParams p) {
    constexpr int N = Team<W>::THREADS, TEAMS = Team<W>::TEAMS;
    constexpr int OWN = DL_MAX_K / N;                  // entries of a thread
    __shared__ Soft s_soft[W + 1];
    __shared__ TeacherShared<W> s_teacher[TEAMS];
    pdl_launch();
    pdl_wait();
    const int64_t block = (int64_t)(blockIdx.x / (unsigned)p.blocks) - p.scan;
    const int rank = (int)(blockIdx.x % (unsigned)p.blocks), tid = Team<W>::thread();
    if (block < 0) {
        if (rank == 0) scan_ids(p.ids, p.id64, p.T * p.K, p.V, -1, true, p.ctrl);
        return;
    }
    const int64_t r = block * TEAMS + Team<W>::team();
    if (r >= p.T) return;
    TeacherShared<W>& S = s_teacher[Team<W>::team()];
    const T* z = static_cast<const T*>(p.z) + r * p.ldz;
    TO* dz = static_cast<TO*>(p.dz) + r * p.lddz;
    const float weight = p.weight ? p.weight[r] : 1.0f;
    int32_t id[OWN];
    float t[OWN], zk[OWN];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int k = i * N + tid;
        int64_t v = -1;
        t[i] = -CUDART_INF_F;
        if (k < p.K) {
            v = load_id(p.ids, p.id64, r * p.K + k);
            t[i] = teacher_at(p, r * p.K + k);
        }
        bad |= v >= p.V;
        id[i] = v < 0 || v >= p.V ? -1 : (int32_t)v;
    }
    const LineRow<T> row(z, p.V);
    const int32_t lines = row.lines(), share = (lines + p.blocks - 1) / p.blocks;
    const int32_t line0 = min(lines, rank * share), line1 = min(lines, line0 + share);
    if (bad && !p.scan && rank == 0) atomicOr(&p.ctrl->status, ST_BAD_INPUT);
    RowSoft a = {};
    float2 teacher = make_float2(-CUDART_INF_F, 1.0f);
    float inv = 0.0f;
    if (weight != 0.0f) {                          // (the same in all blocks of the cluster)
        const Running run = row_sums<W, T, false, false>(row, line0, line1, p.c, nullptr);
        // the warp's part of the teacher's softmax, joined after the row's barrier
        float2 own = make_float2(-CUDART_INF_F, 0.0f);
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            if (i * N >= p.K) break;
            if (id[i] < 0) t[i] = -CUDART_INF_F;
            own.x = max_nan(own.x, t[i]);
            if (i * N + tid < p.K) {
                S.t[i * N + tid] = t[i];
                S.id[i * N + tid] = id[i];
            }
            zk[i] = id[i] >= 0 ? to_f32(z[id[i]]) : 0.0f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) own.x = max_nan(own.x, __shfl_xor_sync(0xFFFFFFFFu, own.x, o));
        if (own.x != -CUDART_INF_F) {
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                if (i * N >= p.K) break;
                own.y += ex2((t[i] - own.x) * p.c);
            }
            own.y = warp_sum(own.y);
        }
        if (W > 1 && lane_id() == 0) S.soft[warp_id()] = own;
        a = join_softmax<W>(row, line0, line1, p.c, p.blocks, s_soft, run);
        inv = a.s == 0.0f ? 0.0f : 1.0f / a.s;
        if (W == 1) {
            __syncwarp();
            teacher = own;
        } else {
            teacher = S.soft[0];
#pragma unroll
            for (int i = 1; i < W; ++i) teacher = join_powers(teacher, S.soft[i], p.c);
        }
    }
    const bool none = teacher.x == -CUDART_INF_F;      // no entry counts
    const float w = weight * p.scale, f = w * inv;
    // the loss, and the gradient at the thread's tokens: the first entry of a token takes all of
    // its q
    float gap = 0.0f, at[OWN];
    bool first[OWN];
    if (!none) {
        const float log_sum = logf(teacher.y), inv_sum = 1.0f / teacher.y;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int k = i * N + tid;
            first[i] = false;
            if (i * N >= p.K) continue;
            const float q = ex2((t[i] - teacher.x) * p.c) * inv_sum;
            if (rank == 0 && id[i] >= 0 && q != 0.0f)
                gap += q * (fmaf(t[i] - teacher.x, p.scale, -log_sum) - a.log_prob(zk[i], p.c, p.scale));
            const int32_t line = id[i] >= 0 ? (id[i] + row.lead) / (LG_LINE / (int)sizeof(T)) : -1;
            first[i] = p.dz && line >= line0 && line < line1;
            if (!first[i]) continue;
            // (entries of the same token are rare; a branch for each equal pair would be taken
            // by one lane at a time)
            int same = 0, before = 0;
#pragma unroll 4
            for (int j = 0; j < p.K; j += 4) {
                const int4 v = *reinterpret_cast<const int4*>(S.id + j);
                const int e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    const int is = e[l] == id[i] && j + l < p.K;
                    same += is;
                    before += is & (j + l < k);
                }
            }
            first[i] = before == 0;
            float all = q;
            if (same > 1 && first[i]) {
                all = 0.0f;
                for (int j = k; j < p.K; ++j)
                    if (S.id[j] == id[i]) all = fmaf(ex2((S.t[j] - teacher.x) * p.c), inv_sum, all);
            }
            at[i] = w * fmaf(a.prob(zk[i], p.c), inv, -all);
        }
        gap = warp_sum(gap);
        if (W > 1 && lane_id() == 0) S.gap[warp_id()] = gap;
    }
    if (p.dz) {
        if (!SAME) {
            constexpr int32_t per = LG_LINE / (int)sizeof(T);
            const int32_t i1 = min(line1 * per, row.end) - row.lead;
            for (int32_t i = max(line0 * per - row.lead, 0) + tid; i < i1; i += N)
                dz[i] = from_f32<TO>(none ? 0.0f : f * a.prob(to_f32(z[i]), p.c));
        } else if (none) {
            const Chunk<TO> zero = {};
            for (int32_t j = line0 * 4 + tid; j < line1 * 4; j += N)
                store_chunk(row, dz - row.lead, j * CHUNK<T>, zero);
        } else {
            for_chunks<W, 2, true>(row, line0, line1, [&](const Chunk<T>* v, int32_t j, int32_t end) {
#pragma unroll
                for (int k = 0; k < 2; ++k, j += N)
                    if (j < end)
                        store_chunk(row, dz - row.lead, j * CHUNK<T>, grad_chunk<T, TO>(v[k], a, p.c, f));
            });
        }
    }
    Team<W>::sync();
    if (!none) {
#pragma unroll
        for (int i = 0; i < OWN; ++i)
            if (first[i]) dz[id[i]] = from_f32<TO>(at[i]);
    }
    if (rank == 0 && tid == 0 && p.loss) {
        if (W > 1 && !none) {
            gap = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) gap += S.gap[i];
        }
        p.loss[r] = none ? 0.0f : weight * gap;
    }
    if (W > 1 && weight != 0.0f && p.blocks > 1) cluster_sync();   // no block leaves while its memory is read
}

}  // namespace tke
