// Losses over a vocabulary: log-probabilities of given tokens with entropy and the
// largest alternatives, their gradient, and distillation from a teacher's top logits.
//
// With c = scale log2(e), a row's softmax is held as  p_i = 2^(c z_i - m) / s,
// s = sum 2^(c z_i - m), u = sum 2^(c z_i - m) (c z_i - m), so that
//     log p_i = ln2 (c z_i - m - log2 s),   entropy = ln2 (log2 s - u / s),
//     log of the sum = ln2 m + ln s.
// m is a whole number near the largest c z: each thread raises its own when a group of
// values passes it by 2^RAISE, and a change of m scales s by an exact power of two.
// One fma and one ex2 a value; the rest rides on 32-byte groups.
//
// Values below -2^17 / c are left out at first: if the row's m ends above -2^16, their p
// is 0.  If m ends past +-2^16, where c z - m would lose bits, or nothing is left, the
// row is read again and summed with the exact differences z - max (a row all of
// whose tokens are masked by -1e9 or by the type's lowest value is uniform).
// -inf (a forbidden token) has p = 0 and counts nowhere.  NaN and +inf make the row
// NaN.
//
// One thread-block cluster a row, each block an equal share of the row's 128-byte
// lines: rows start anywhere, and whole lines are read as 32 bytes a thread.
#pragma once

#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "async.cuh"
#include "common.cuh"
#include "elements.cuh"
#include "topk_ef.h"

namespace tke {

constexpr int LG_THREADS = 256, LG_WARPS = LG_THREADS / 32;
constexpr int LG_LINE = 128;               // bytes of a line (a group of the top selection)
constexpr int LG_FLIGHT = 4;               // 32-byte chunks that a thread loads at once
constexpr float LG_RAISE = 8.0f;
constexpr float LG_START = -3e38f;         // m before any value
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
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

template <typename T>
constexpr int CHUNK = 32 / (int)sizeof(T);         // elements of 32 bytes

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
template <typename T>
__device__ __forceinline__ void no_chunk(Chunk<T>& c) {
    T* e = reinterpret_cast<T*>(c.q);
#pragma unroll
    for (int i = 0; i < CHUNK<T>; ++i) e[i] = from_f32<T>(-CUDART_INF_F);
}

struct Soft {
    float m, s, u;
};

// Adds a chunk; returns its largest value (NaN if it holds one).
template <typename T, bool ENTROPY>
__device__ __forceinline__ float add_chunk(const Chunk<T>& q, Soft& a, float c) {
    float v[CHUNK<T>];
#pragma unroll
    for (int i = 0; i < CHUNK<T>; ++i) v[i] = q.get(i);
    float top = v[0];
#pragma unroll
    for (int i = 1; i < CHUNK<T>; ++i) top = max_nan(top, v[i]);
    const float reach = top * c;
    if (reach < -2.0f * LG_FAR) return top;
    if (!(reach <= a.m + LG_RAISE)) {
        const float m = ceilf(reach), f = ex2(a.m - m);
        if (ENTROPY) a.u = fmaf(a.m - m, a.s, a.u) * f;
        a.s *= f;
        a.m = m;
    }
    float s[2] = {0.0f, 0.0f}, u[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < CHUNK<T>; ++i) {
        const float t = fmaf(v[i], c, -a.m), e = ex2(t);
        s[i & 1] += e;
        if (ENTROPY) u[i & 1] = fmaf(e, fmaxf(t, -1e4f), u[i & 1]);      // (e is 0 there)
    }
    a.s += s[0] + s[1];
    if (ENTROPY) a.u += u[0] + u[1];
    return top;
}

__device__ __forceinline__ Soft join(const Soft& a, const Soft& b) {
    const float m = fmaxf(a.m, b.m), fa = ex2(a.m - m), fb = ex2(b.m - m);
    return {m, fmaf(a.s, fa, b.s * fb), fmaf(a.m - m, a.s, a.u) * fa + fmaf(b.m - m, b.s, b.u) * fb};
}

__device__ __forceinline__ Soft warp_join(Soft a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Soft b;
        b.m = __shfl_xor_sync(0xFFFFFFFFu, a.m, o);
        b.s = __shfl_xor_sync(0xFFFFFFFFu, a.s, o);
        b.u = __shfl_xor_sync(0xFFFFFFFFu, a.u, o);
        a = join(a, b);
    }
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

// f(chunk, its number, whether it belongs to the block) for the chunks of lines
// [line0, line1); every thread of a warp makes the same calls.
template <typename T, typename F>
__device__ __forceinline__ void for_chunks(const LineRow<T>& row, int32_t line0, int32_t line1, F f) {
    const int32_t end = line1 * 4;
    for (int32_t j0 = line0 * 4; j0 < end; j0 += LG_THREADS * LG_FLIGHT) {
        Chunk<T> q[LG_FLIGHT];
#pragma unroll
        for (int k = 0; k < LG_FLIGHT; ++k) {
            const int32_t j = j0 + k * LG_THREADS + (int32_t)threadIdx.x;
            if (j < end) {
                load_chunk(row, j, q[k]);
            } else {
                no_chunk(q[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < LG_FLIGHT; ++k) {
            const int32_t j = j0 + k * LG_THREADS + (int32_t)threadIdx.x;
            f(q[k], j, j < end);
        }
    }
}

// The statistics of all the cluster's blocks, in every block (s_soft: LG_WARPS + 1
// entries).  Also a barrier of the cluster.
__device__ __forceinline__ Soft row_join(Soft a, int blocks, Soft* s_soft) {
    a = warp_join(a);
    if (lane_id() == 0) s_soft[warp_id()] = a;
    __syncthreads();
    const Soft none = {LG_START, 0.0f, 0.0f};
    a = warp_join(lane_id() < LG_WARPS ? s_soft[lane_id()] : none);
    if (blocks == 1) return a;
    if (threadIdx.x == 0) s_soft[LG_WARPS] = a;
    cluster_sync();
    a = none;
    if ((int)lane_id() < blocks) {
        const uint32_t at = in_block(smem_u32(&s_soft[LG_WARPS]), lane_id());
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
template <typename T>
__device__ __forceinline__ Soft far_row(const LineRow<T>& row, int32_t line0, int32_t line1, float c,
                                     int blocks, Soft* s_soft) {
    float top = -CUDART_INF_F;
    for_chunks(row, line0, line1, [&](const Chunk<T>& q, int32_t, bool) {
#pragma unroll
        for (int i = 0; i < CHUNK<T>; ++i) top = max_nan(top, q.get(i));
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (blocks > 1) cluster_sync(); else __syncthreads();      // what s_soft held has been read
    if (lane_id() == 0) s_soft[warp_id()].m = top;
    __syncthreads();
    top = s_soft[0].m;
#pragma unroll
    for (int i = 1; i < LG_WARPS; ++i) top = max_nan(top, s_soft[i].m);
    if (blocks > 1) {
        if (threadIdx.x == 0) s_soft[LG_WARPS].m = top;
        cluster_sync();
        if ((int)lane_id() < blocks) {
            const uint32_t at = in_block(smem_u32(&s_soft[LG_WARPS]), lane_id());
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(top) : "r"(at));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        cluster_sync();
    } else {
        __syncthreads();
    }
    Soft a = {0.0f, 0.0f, 0.0f};
    if (top != -CUDART_INF_F)
        for_chunks(row, line0, line1, [&](const Chunk<T>& q, int32_t, bool) {
#pragma unroll
            for (int i = 0; i < CHUNK<T>; ++i) {
                const float t = c * (q.get(i) - top), e = ex2(t);
                a.s += e;
                a.u = fmaf(e, fmaxf(t, -1e4f), a.u);
            }
        });
    a = row_join(a, blocks, s_soft);
    a.m = top;
    return a;
}

// The softmax of a row, of which a block takes lines [line0, line1); TOP: the
// largest key of each of them in keys[line].
template <typename T, bool ENTROPY, bool TOP>
__device__ __forceinline__ RowSoft row_softmax(const LineRow<T>& row, int32_t line0, int32_t line1,
                                               float c, int blocks, Soft* s_soft, uint32_t* keys) {
    Soft a = {LG_START, 0.0f, 0.0f};
    for_chunks(row, line0, line1, [&](const Chunk<T>& q, int32_t j, bool mine) {
        float top = add_chunk<T, ENTROPY>(q, a, c);
        if (TOP) {
            top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            if ((threadIdx.x & 3) == 0 && mine) keys[j >> 2] = order_key(top);
        }
    });
    a = row_join(a, blocks, s_soft);
    RowSoft r;
    r.far = a.s == 0.0f || !(fabsf(a.m) <= LG_FAR) || a.s != a.s;
    if (r.far) a = far_row(row, line0, line1, c, blocks, s_soft);
    r.m = a.m;
    r.s = a.s;
    r.u = a.u;
    r.log2s = log2f(a.s);
    return r;
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
    int32_t scan;                  // the last cluster checks the ids
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

// Sum of v over the block (every thread gets it); s: 2 x LG_WARPS words, `flip` the
// half that the last call did not use.
__device__ __forceinline__ uint32_t block_count(uint32_t v, uint32_t* s, int flip) {
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    if (lane_id() == 0) s[flip * LG_WARPS + warp_id()] = v;
    __syncthreads();
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < LG_WARPS; ++i) n += s[flip * LG_WARPS + i];
    return n;
}

// The largest key that at least `want` of the block's keys reach, bit by bit;
// `count(k)` counts the thread's keys >= k.  LOW: bits below it are equal in all keys.
template <int LOW, typename F>
__device__ __forceinline__ uint32_t block_threshold(uint32_t want, uint32_t* s, F count) {
    uint32_t k = 0;
    for (int bit = 31; bit >= LOW; --bit) {
        const uint32_t up = k | (1u << bit);
        if (block_count(count(up), s, bit & 1) >= want) k = up;
    }
    __syncthreads();
    return k;
}

constexpr int TL_LIST = 512;               // candidates that are ranked by comparison

struct TopShared {
    uint32_t count[2 * LG_WARPS];
    uint32_t scan[33];
    uint32_t line[TL_MAX_TOP];
    unsigned long long list[TL_LIST];      // key, then the lower index first
};

// The top K of the row by (value descending, index ascending), one block.
//
// The K-th largest of the lines' largest values, t, is at most the K-th largest
// value; the lines above t and the first of those that equal it, K in all,
// hold every element above t and the first ones at t.  So K lines are read again, and
// what reaches t in them, hardly more than K values unless they are ordered, is
// ranked by comparing each with each.  The time does not depend on the order of the row.
template <typename T>
__device__ void select_top(const LogprobParams& p, const LineRow<T>& row, int64_t r,
                           const uint32_t* keys, TopShared& S, const RowSoft& soft) {
    constexpr int LOW = sizeof(T) == 4 ? 0 : 13;       // bf16 keys end 16 bits up, fp16's 13
    const int tid = (int)threadIdx.x;
    const int lines = row.lines(), K = p.top, want = min(K, lines);
    const int per = (lines + LG_THREADS - 1) / LG_THREADS;
    // the thread's lines are neighbours, so that a scan over threads is one over lines
    const int l0 = min(lines, tid * per), l1 = min(lines, l0 + per);
    uint32_t t = 0;
    if (lines > K)
        t = block_threshold<LOW>((uint32_t)K, S.count, [&](uint32_t k) {
            uint32_t n = 0;
            for (int l = l0; l < l1; ++l) n += keys[l] >= k;
            return n;
        });
    // (keys whose low bits are set, a negative value's, compare as the value they stand for)
    const uint32_t mask = LOW ? ~((1u << LOW) - 1) : 0xFFFFFFFFu;
    uint32_t above = 0, equal = 0, all_above;
    for (int l = l0; l < l1; ++l) {
        const uint32_t k = keys[l] & mask;
        above += k > t;
        equal += k == t;
    }
    uint32_t tot;
    const uint32_t before = block_excl_scan(above << 16 | equal, S.scan, &tot);
    all_above = tot >> 16;
    {
        const uint32_t quota = (uint32_t)want - all_above;
        uint32_t a = before >> 16, e = before & 0xFFFF;
        for (int l = l0; l < l1; ++l) {
            const uint32_t k = keys[l] & mask;
            if (k > t || (k == t && e < quota)) S.line[a + min(e, quota)] = (uint32_t)l;
            a += k > t;
            e += k == t;
        }
    }
    __syncthreads();
    // candidates, in order: the thread's chunks are neighbours of the lines' list
    constexpr int MOST = TL_MAX_TOP * 4 / LG_THREADS;
    const int chunks = want * 4, each = (chunks + LG_THREADS - 1) / LG_THREADS;
    Chunk<T> q[MOST];
    int32_t at[MOST] = {};
    uint32_t n = 0;
    auto key_of_pos = [&](int i, int e) -> uint32_t {      // 0: not an element
        const int32_t pos = at[i] + e;
        return pos >= row.lead && pos < row.end ? order_key(q[i].get(e)) : 0u;
    };
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        const int j = tid * each + i;
        at[i] = 0x40000000;                                 // past every row
        if (i < each && j < chunks) {
            const int32_t chunk = (int32_t)S.line[j >> 2] * 4 + (j & 3);
            at[i] = chunk * CHUNK<T>;
            load_chunk(row, chunk, q[i]);
        } else {
            no_chunk(q[i]);
        }
#pragma unroll
        for (int e = 0; e < CHUNK<T>; ++e) {
            const uint32_t k = key_of_pos(i, e);
            n += k != 0 && (k & mask) >= t;
        }
    }
    uint32_t first = block_excl_scan(n, S.scan, &tot), cut = t, quota = 0xFFFFFFFFu;
    const uint32_t need = min((uint32_t)K, tot);
    if (tot > TL_LIST) {
        // many at or above t: exactly those that belong to the top K
        cut = block_threshold<LOW>(need, S.count, [&](uint32_t k) {
            uint32_t c = 0;
#pragma unroll
            for (int i = 0; i < MOST; ++i)
#pragma unroll
                for (int e = 0; e < CHUNK<T>; ++e) c += key_of_pos(i, e) >= k;
            return c;
        });
        above = equal = 0;
#pragma unroll
        for (int i = 0; i < MOST; ++i)
#pragma unroll
            for (int e = 0; e < CHUNK<T>; ++e) {
                const uint32_t k = key_of_pos(i, e);
                above += k != 0 && (k & mask) > cut;
                equal += k != 0 && (k & mask) == cut;
            }
        const uint32_t b = block_excl_scan(above << 16 | equal, S.scan, &tot);
        quota = need - (tot >> 16);
        n = b & 0xFFFF;                                     // equal ones before the thread's
        first = (b >> 16) + min(n, quota);
        tot = need;
    } else {
        n = 0;
    }
#pragma unroll
    for (int i = 0; i < MOST; ++i)
#pragma unroll
        for (int e = 0; e < CHUNK<T>; ++e) {
            const uint32_t k = key_of_pos(i, e);
            const bool eq = k != 0 && (k & mask) == cut;
            if (k != 0 && ((k & mask) > cut || (eq && n < quota)))
                S.list[first++] = (unsigned long long)k << 32 | (uint32_t)(row.end - 1 - (at[i] + e));
            n += eq;
        }
    __syncthreads();
    for (uint32_t i = tid; i < tot; i += LG_THREADS) {
        const unsigned long long mine = S.list[i];
        uint32_t rank = 0;
        for (uint32_t j = 0; j < tot; ++j) rank += S.list[j] > mine;
        if (rank < (uint32_t)K) {
            const float z = key_value((uint32_t)(mine >> 32));
            const int32_t id = row.end - 1 - (int32_t)(uint32_t)mine - row.lead;
            if (p.top_ids) p.top_ids[r * K + rank] = id;
            if (p.top_logprobs) p.top_logprobs[r * K + rank] = soft.log_prob(z, p.c, p.scale);
        }
    }
    for (int i = (int)min((int64_t)K, p.V) + tid; i < K; i += LG_THREADS) {
        if (p.top_ids) p.top_ids[r * K + i] = -1;
        if (p.top_logprobs) p.top_logprobs[r * K + i] = -CUDART_INF_F;
    }
}

template <typename T, bool ENTROPY, bool TOP>
__global__ void __launch_bounds__(LG_THREADS) logprob_kernel(const LogprobParams p) {
    extern __shared__ uint32_t s_keys[];               // TOP: [blocks][lines]
    __shared__ Soft s_soft[LG_WARPS + 1];
    __shared__ TopShared S;
    pdl_launch();
    pdl_wait();
    const int64_t r = blockIdx.x / (unsigned)p.blocks;
    const int rank = (int)(blockIdx.x - r * p.blocks);
    if (r == p.T) {
        if (rank == 0) scan_ids(p.ids, p.id64, p.T, p.V, p.padding, false, p.ctrl);
        return;
    }
    const int tid = (int)threadIdx.x;
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
        for (int i = tid; TOP && i < p.top; i += LG_THREADS) {
            if (p.top_ids) p.top_ids[r * p.top + i] = -1;
            if (p.top_logprobs) p.top_logprobs[r * p.top + i] = -CUDART_INF_F;
        }
        return;
    }
    const T* z = static_cast<const T*>(p.z) + r * p.ldz;
    float zt = 0.0f;
    if (ok && rank == 0 && tid == 0) zt = to_f32(z[id]);
    const LineRow<T> row(z, p.V);
    const int32_t lines = row.lines();
    const int32_t share = (lines + p.blocks - 1) / p.blocks;
    const int32_t line0 = min(lines, rank * share), line1 = min(lines, line0 + share);
    const RowSoft a =
        row_softmax<T, ENTROPY, TOP>(row, line0, line1, p.c, p.blocks, s_soft, s_keys);
    if (rank == 0 && tid == 0) {
        if (p.logprob) p.logprob[r] = ok ? a.log_prob(zt, p.c, p.scale) : 0.0f;
        if (ENTROPY && p.entropy) p.entropy[r] = a.entropy();
        if (p.lse) p.lse[r] = a.log_sum(p.scale);
    }
    if (TOP && rank == 0) {
        // the other blocks' keys
        if (p.blocks > 1)
            for (int32_t l = line1 + tid; l < lines; l += LG_THREADS) {
                uint32_t k;
                asm volatile("ld.shared::cluster.u32 %0, [%1];"
                             : "=r"(k)
                             : "r"(in_block(smem_u32(s_keys + l), (uint32_t)(l / share))));
                s_keys[l] = k;
            }
        __syncthreads();
        select_top<T>(p, row, r, s_keys, S, a);
    }
    if (p.blocks > 1) cluster_sync();      // no block leaves while its memory is read
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
    int32_t id64, parts;           // blocks of a row
    int32_t scan;                  // the last block checks the ids
    float scale;
};

constexpr int LD_THREADS = 128;

// dz_i = scale (g (delta_i,id - p_i) - h p_i (log p_i + entropy)).  SAME: z's and dz's
// rows lie alike in their lines.
template <typename T, typename TO, bool SAME>
__global__ void __launch_bounds__(LD_THREADS) logprob_grad_kernel(const LogprobGradParams p) {
    pdl_launch();
    pdl_wait();
    const int64_t r = blockIdx.x / (unsigned)p.parts;
    const int part = (int)(blockIdx.x - r * p.parts);
    if (r == p.T) {
        scan_ids(p.ids, p.id64, p.T, p.V, p.padding, false, p.ctrl);
        return;
    }
    const T* z = static_cast<const T*>(p.z) + r * p.ldz;
    TO* dz = static_cast<TO*>(p.dz) + r * p.lddz;
    int64_t id = -1;
    bool skip = false, ok = false;
    if (p.ids) {
        id = load_id(p.ids, p.id64, r);
        skip = id == p.padding;
        ok = id >= 0 && id < p.V;
        if (!skip && !ok && !p.scan && part == 0 && threadIdx.x == 0)
            atomicOr(&p.ctrl->status, ST_BAD_INPUT);
    }
    const float lse = p.lse[r];
    const float g = ok && p.g ? p.scale * p.g[r] : 0.0f, h = p.h ? p.scale * p.h[r] : 0.0f;
    const float H = p.h ? p.entropy[r] : 0.0f;
    skip = skip || (g == 0.0f && h == 0.0f) || lse == -CUDART_INF_F;
    // -(p (g + h (log p + H))), and g at the token
    auto value = [&](float v, int32_t i) {
        const float t = max_nan(fmaf(v, p.scale, -lse), -1e4f), e = ex2(t * LOG2E);
        const float k = fmaf(h, t + H, g);
        return fmaf(-e, k, i == (int32_t)id ? g : 0.0f);
    };
    if (SAME) {
        const LineRow<T> row(z, p.V);
        TO* out = dz - row.lead;
        const int32_t end = row.lines() * 4;
        for (int32_t j0 = part * LD_THREADS * LG_FLIGHT; j0 < end;
             j0 += p.parts * LD_THREADS * LG_FLIGHT) {
            Chunk<T> q[LG_FLIGHT];
#pragma unroll
            for (int k = 0; k < LG_FLIGHT; ++k) {
                const int32_t j = j0 + k * LD_THREADS + (int32_t)threadIdx.x;
                if (!skip && j < end) load_chunk(row, j, q[k]);
            }
#pragma unroll
            for (int k = 0; k < LG_FLIGHT; ++k) {
                const int32_t j = j0 + k * LD_THREADS + (int32_t)threadIdx.x;
                if (j >= end) continue;
                const int32_t pos = j * CHUNK<T>;
                Chunk<TO> o;
                TO* x = reinterpret_cast<TO*>(o.q);
#pragma unroll
                for (int i = 0; i < CHUNK<T>; ++i)
                    x[i] = from_f32<TO>(skip ? 0.0f : value(q[k].get(i), pos + i - row.lead));
                if (pos >= row.lead && pos + CHUNK<T> <= row.end) {
                    store32b(out + pos, o.q);
                } else {
#pragma unroll
                    for (int i = 0; i < CHUNK<T>; ++i)
                        if (pos + i >= row.lead && pos + i < row.end) out[pos + i] = x[i];
                }
            }
        }
    } else {
        for (int32_t i = part * LD_THREADS + (int32_t)threadIdx.x; i < (int32_t)p.V;
             i += p.parts * LD_THREADS)
            dz[i] = from_f32<TO>(skip ? 0.0f : value(to_f32(z[i]), i));
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
    int32_t id64, teacher_type, K, blocks, scan;
    float c, scale;
};

__device__ __forceinline__ float block_max_nan(float v, float* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (lane_id() == 0) s[warp_id()] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int i = 1; i < LG_WARPS; ++i) v = max_nan(v, s[i]);
    __syncthreads();
    return v;
}

__device__ __forceinline__ float teacher_at(const DistillParams& p, int64_t i) {
    if (p.teacher_type == TOPK_EF_F32) return static_cast<const float*>(p.teacher)[i];
    if (p.teacher_type == TOPK_EF_BF16)
        return to_f32(static_cast<const __nv_bfloat16*>(p.teacher)[i]);
    return to_f32(static_cast<const __half*>(p.teacher)[i]);
}

// loss = weight sum_k q_k (log q_k - log p_{id_k}),  q = softmax(scale teacher);
// dz = weight scale (p - q).  Thread k keeps the teacher's k-th entry.
template <typename T, typename TO, bool SAME>
__global__ void __launch_bounds__(LG_THREADS) distill_kernel(const DistillParams p) {
    __shared__ Soft s_soft[LG_WARPS + 1];
    __shared__ float s_red[33];
    __shared__ int32_t s_id[DL_MAX_K];
    __shared__ float s_q[DL_MAX_K];
    pdl_launch();
    pdl_wait();
    const int64_t r = blockIdx.x / (unsigned)p.blocks;
    const int rank = (int)(blockIdx.x - r * p.blocks), tid = (int)threadIdx.x;
    if (r == p.T) {
        if (rank == 0) scan_ids(p.ids, p.id64, p.T * p.K, p.V, -1, true, p.ctrl);
        return;
    }
    const T* z = static_cast<const T*>(p.z) + r * p.ldz;
    int64_t id = -1;
    float tz = -CUDART_INF_F, zk = 0.0f;
    if (tid < p.K) {
        id = load_id(p.ids, p.id64, r * p.K + tid);
        if (id >= p.V) {
            if (!p.scan && rank == 0) atomicOr(&p.ctrl->status, ST_BAD_INPUT);
            id = -1;
        }
    }
    const float weight = p.weight ? p.weight[r] : 1.0f;
    bool skip = weight == 0.0f;
    if (!skip && id >= 0) {
        tz = teacher_at(p, r * p.K + tid);
        zk = to_f32(z[id]);
    }
    float big = -CUDART_INF_F;
    if (!skip) {
        big = block_max_nan(tz, s_red);
        skip = big == -CUDART_INF_F;               // no entry counts
    }
    const LineRow<T> row(z, p.V);
    const int32_t lines = row.lines(), share = (lines + p.blocks - 1) / p.blocks;
    const int32_t line0 = min(lines, rank * share), line1 = min(lines, line0 + share);
    RowSoft a = {};
    float q = 0.0f, inv = 0.0f;
    if (!skip) {                                   // (the same in all blocks of the cluster)
        const float tq = tz - big;
        q = ex2(tq * p.c);
        const float sum = block_sum(q, s_red);
        q /= sum;
        a = row_softmax<T, false, false>(row, line0, line1, p.c, p.blocks, s_soft, nullptr);
        if (rank == 0 && p.loss) {
            float part = 0.0f;
            if (q != 0.0f)
                part = q * (fmaf(tq, p.scale, -logf(sum)) - a.log_prob(zk, p.c, p.scale));
            part = block_sum(part, s_red);
            if (tid == 0) p.loss[r] = weight * part;
        }
        s_id[tid] = (int32_t)id;
        s_q[tid] = q;
        inv = a.s == 0.0f ? 0.0f : 1.0f / a.s;
        __syncthreads();
    } else if (rank == 0 && tid == 0 && p.loss) {
        p.loss[r] = 0.0f;
    }
    if (p.dz) {
        TO* dz = static_cast<TO*>(p.dz) + r * p.lddz;
        const float w = weight * p.scale, f = w * inv;
        auto prob = [&](float v) { return a.prob(v, p.c); };
        if (SAME) {
            TO* out = dz - row.lead;
            const int32_t end = line1 * 4;
            for (int32_t j0 = line0 * 4; j0 < end; j0 += LG_THREADS * LG_FLIGHT) {
                Chunk<T> v[LG_FLIGHT];
#pragma unroll
                for (int k = 0; k < LG_FLIGHT; ++k) {
                    const int32_t j = j0 + k * LG_THREADS + tid;
                    if (!skip && j < end) load_chunk(row, j, v[k]);
                }
#pragma unroll
                for (int k = 0; k < LG_FLIGHT; ++k) {
                    const int32_t j = j0 + k * LG_THREADS + tid;
                    if (j >= end) continue;
                    const int32_t pos = j * CHUNK<T>;
                    Chunk<TO> o;
                    TO* x = reinterpret_cast<TO*>(o.q);
#pragma unroll
                    for (int i = 0; i < CHUNK<T>; ++i)
                        x[i] = from_f32<TO>(skip ? 0.0f : f * prob(v[k].get(i)));
                    if (pos >= row.lead && pos + CHUNK<T> <= row.end) {
                        store32b(out + pos, o.q);
                    } else {
#pragma unroll
                        for (int i = 0; i < CHUNK<T>; ++i)
                            if (pos + i >= row.lead && pos + i < row.end) out[pos + i] = x[i];
                    }
                }
            }
        } else {
            const int32_t per = LG_LINE / (int)sizeof(T);
            const int32_t i1 = min(line1 * per, row.end) - row.lead;
            for (int32_t i = max(line0 * per - row.lead, 0) + tid; i < i1; i += LG_THREADS)
                dz[i] = from_f32<TO>(skip ? 0.0f : f * prob(to_f32(z[i])));
        }
        if (!skip) {
            // the teacher's tokens: the first entry of each takes all of its q
            __syncthreads();
            const int32_t line = id >= 0 ? ((int32_t)id + row.lead) / (LG_LINE / (int)sizeof(T)) : -1;
            if (line >= line0 && line < line1) {
                float all = 0.0f;
                bool first = true;
                for (int j = 0; j < p.K; ++j)
                    if (s_id[j] == (int32_t)id) {
                        all += s_q[j];
                        first = first && j >= tid;
                    }
                if (first) dz[id] = from_f32<TO>(w * (prob(zk) * inv - all));
            }
        }
    }
    if (!skip && p.blocks > 1) cluster_sync();     // no block leaves while its memory is read
}

}  // namespace tke
