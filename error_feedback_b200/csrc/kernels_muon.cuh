// Orthogonalisation of an update by Newton-Schulz products (the Muon
// optimiser's iteration):
//
//     X <- u / (||u||_F + eps);   steps times:  A = X X^T,  X <- a X + (b A + c A A) X
//
// (X^T X and products from the right when X is tall: A is always p x p with
// p the short side.)  Three products per step on the tensor cores, each with
// its elementwise part in the epilogue: gram (A), square (B = b A + c A A) and
// update (X' = a X + B X).  A and B are symmetric: only tiles that touch the
// lower triangle are computed, and the epilogue writes them to both sides.
//
// Numbers: X is held as a pair of fp16 values, hi + lo / MU_LO (22 bits), times a
// power of two that keeps typical entries near 1; A and B likewise times MU_SA.  A step
// multiplies small singular values by a (3.4 five times in a row), so a
// rounding of X itself would be amplified 485 times: the term a X is taken
// from hi + lo.  For bf16 outputs the products read hi alone (11 bits; bf16
// operands would leave an error six times a bf16 output's own rounding); for
// fp32 and fp16 outputs each product is hi hi + (hi lo + lo hi) / MU_LO.  All sums are fp32.
// lo is held times MU_LO because fp16's range ends 2^-24 below the typical entry:
// a row of 1e-5 of the others would keep 7 bits of its 22, and be 3e-4 off in the
// result, one of 1e-6 4e-3 (plain fp32: 2e-6; so held 2e-6, and 1e-4 at 1e-8).
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "elements.cuh"

namespace tke {

constexpr float MU_SA = 2048.0f;           // scale of A and B
constexpr int MU_LO_BITS = 11;             // what fp16 leaves of 2^15 at most is 2^3: no overflow
constexpr float MU_LO = 1 << MU_LO_BITS;   // scale of what fp16 leaves of X, A and B
constexpr float MU_REACH = 4.0f;           // |p(x)| the coefficients may reach (host check)
constexpr int MU_MAX_LIFT = 60;             // (see muon_scale_kernel)
// The tensor core truncates where it adds 16 products to an fp32 accumulator: a
// sum of squares of n such adds comes out low, by 5.4e-8 n of its value on
// average (measured for n = 2 .. 60: 4.9e-8 n to 7.0e-8 n, with a spread of 5e-8
// in all; 2^-24 = 6.0e-8).  With 22 bits accumulators are kept short, and
// what is left is multiplied back in the gram and the square, whose diagonals are
// sums of squares.  The update's terms have both signs: there the factor makes
// it worse.  A 128 x 24,576 matrix is 8.1e-6 off without, 3.5e-6 with it (plain
// fp32: 1.4e-6), one of 2,048 x 8,192 1.2e-5 and 7.5e-6 (5.2e-6).
constexpr float MU_LOW = 5.4e-8f;
constexpr uint64_t MU_WAIT_NS = 2000000000ull;

__device__ __forceinline__ float below_half(float x) {     // what fp16 leaves of x, as it is held
    return MU_LO * (x - __half2float(__float2half_rn(x)));
}
__device__ __forceinline__ float of_pair(float hi, float lo) { return fmaf(lo, 1.0f / MU_LO, hi); }

// ------------------------------------------------------- momentum and norm

constexpr int MN_THREADS = 256;
constexpr int MN_MAX_PARTS = 1184;         // partial sums of one matrix
template <typename TG>
constexpr int MN_FLIGHT = sizeof(TG) == 2 ? 4 : 2;     // groups of 8 elements that a thread loads at once

struct MuonPreParams {
    const void* grad;
    float* momentum;               // or null
    double* part;                  // [B][parts]: sums of squares
    __half* hi;                    // [B][rows][ldx]
    __half* lo;
    int32_t* lift;                 // [B]: X is held times 2^lift (scale kernel)
    Ctrl* ctrl;
    int64_t rows, cols, ldx, ld_g, stride_g, stride_x, parts;
    int64_t row_groups, groups;    // groups of 8 columns: of a row, of a matrix
    float mu;
    int32_t nesterov;
    double eps, S;
    int32_t flat;                  // grad, momentum and X are contiguous, in 16-byte steps
};

// u of up to 8 consecutive elements of one row; FIRST: the momentum is
// updated, else it has been.  Returns how many there are.
template <typename TG, bool FIRST>
__device__ __forceinline__ int muon_u8(const MuonPreParams& p, int64_t b, int64_t r, int64_t c,
                                       float* u) {
    const int n = (int)min((int64_t)8, p.cols - c);
    const TG* g = static_cast<const TG*>(p.grad) + b * p.stride_g + r * p.ld_g + c;
    const bool full = n == 8;
    if (full && (uintptr_t)g % 16 == 0) {
        const Vec8<TG> v = load8(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = elem8(v, j);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = j < n ? to_f32(g[j]) : 0.0f;
    }
    if (!p.momentum) return n;
    float* mp = p.momentum + (b * p.rows + r) * p.cols + c;
    const bool vec = full && (uintptr_t)mp % 16 == 0;
    float m[8];
    if (vec) {
        const Vec8<float> v = load8(mp);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = elem8(v, j);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = j < n ? mp[j] : 0.0f;
    }
    if (FIRST) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = fmaf(p.mu, m[j], u[j]);
        if (vec) {
            store8(mp, m);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) mp[j] = m[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = p.nesterov ? fmaf(p.mu, m[j], u[j]) : m[j];
    return n;
}

// m <- mu m + g, and the partial sums of u^2 (64 bits, fixed order).  Eight
// elements per thread at a time; bound by the bytes of g and m (4,096 x 4,096
// fp32: 28 us, 7 TB/s with what L2 holds).
template <typename TG>
__global__ void __launch_bounds__(MN_THREADS, 3) muon_norm_kernel(const MuonPreParams p) {
    __shared__ double s_red[33];
    pdl_launch();
    pdl_wait();
    const int64_t b = blockIdx.y;
    if (blockIdx.x == 0 && b == 0 && threadIdx.x == 0) {
        p.ctrl->path_small = 0;
        p.ctrl->status = 0;
    }
    // squares of 8 elements in fp32, their sums in 64 bits; in 64 bits throughout
    // where fp32 would not hold the squares (conversions of every element would set
    // the pace: 85 us for 25,088 x 4,096 bf16)
    double sum = 0.0;
    auto add8 = [&](const float* u) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(u[j], u[j], s);
        if (s > 1e-25f && s < 1e35f) {
            sum += (double)s;
        } else {
            for (int j = 0; j < 8; ++j) sum = fma((double)u[j], (double)u[j], sum);
        }
    };
    const int64_t step = (int64_t)gridDim.x * MN_THREADS;
    if (p.flat) {
        const TG* g = static_cast<const TG*>(p.grad) + b * p.stride_g;
        float* mom = p.momentum ? p.momentum + b * p.groups * 8 : nullptr;
        for (int64_t i = (int64_t)blockIdx.x * MN_THREADS + threadIdx.x; i < p.groups;
             i += MN_FLIGHT<TG> * step) {
            Vec8<TG> gv[MN_FLIGHT<TG>];
            Vec8<float> mv[MN_FLIGHT<TG>];
#pragma unroll
            for (int k = 0; k < MN_FLIGHT<TG>; ++k)
                if (i + k * step < p.groups) {
                    gv[k] = load8(g + (i + k * step) * 8);
                    if (mom) mv[k] = load8(mom + (i + k * step) * 8);
                }
#pragma unroll
            for (int k = 0; k < MN_FLIGHT<TG>; ++k) {
                if (i + k * step >= p.groups) continue;
                float m[8], u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    u[j] = elem8(gv[k], j);
                    if (mom) {
                        m[j] = fmaf(p.mu, elem8(mv[k], j), u[j]);
                        u[j] = p.nesterov ? fmaf(p.mu, m[j], u[j]) : m[j];
                    }
                }
                add8(u);
                if (mom) store8(mom + (i + k * step) * 8, m);
            }
        }
    } else {
        for (int64_t i = (int64_t)blockIdx.x * MN_THREADS + threadIdx.x; i < p.groups; i += step) {
            const int64_t r = i / p.row_groups;
            float u[8];
            muon_u8<TG, true>(p, b, r, (i - r * p.row_groups) * 8, u);
            add8(u);
        }
    }
    const double tot = block_sum(sum, s_red);
    if (threadIdx.x == 0) p.part[b * p.parts + blockIdx.x] = tot;
}

// X = u * S * 2^lift / (||u|| + eps) as a pair.  lift is 0 unless eps holds
// the norm of X below 1: then it brings the entries to where fp16 has all its
// bits, and the products take it back as fast as X can grow.
template <typename TG>
__global__ void __launch_bounds__(MN_THREADS, 3) muon_scale_kernel(const MuonPreParams p) {
    __shared__ double s_red[33];
    pdl_launch();
    pdl_wait();
    const int64_t b = blockIdx.y;
    double sq = 0.0;
    for (int64_t i = threadIdx.x; i < p.parts; i += MN_THREADS) sq += p.part[b * p.parts + i];
    sq = block_sum(sq, s_red);
    const double norm = sqrt(sq);
    int lift = 0;
    if (norm > 0.0 && norm < p.eps) lift = min(MU_MAX_LIFT, ilogb((norm + p.eps) / norm));
    if (blockIdx.x == 0 && threadIdx.x == 0) p.lift[b] = lift;
    const double f = scalbn(p.S, lift) / (norm + p.eps);
    const int64_t step = (int64_t)gridDim.x * MN_THREADS;
    // (the factor of a norm near fp32's ends would not be an fp32 value)
    const float f32 = (float)f;
    const bool plain = f > 1e-36 && f < 1e36;
    auto put = [&](int64_t o, float* u) {
        float l[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u[j] = plain ? u[j] * f32 : (float)((double)u[j] * f);
            l[j] = below_half(u[j]);
        }
        store8(p.hi + o, u);
        store8(p.lo + o, l);
    };
    if (p.flat) {
        const TG* g = static_cast<const TG*>(p.grad) + b * p.stride_g;
        const float* mom = p.momentum ? p.momentum + b * p.groups * 8 : nullptr;
        for (int64_t i = (int64_t)blockIdx.x * MN_THREADS + threadIdx.x; i < p.groups;
             i += MN_FLIGHT<TG> * step) {
            Vec8<TG> gv[MN_FLIGHT<TG>];
            Vec8<float> mv[MN_FLIGHT<TG>];
#pragma unroll
            for (int k = 0; k < MN_FLIGHT<TG>; ++k)
                if (i + k * step < p.groups) {
                    gv[k] = load8(g + (i + k * step) * 8);
                    if (mom) mv[k] = load8(mom + (i + k * step) * 8);
                }
#pragma unroll
            for (int k = 0; k < MN_FLIGHT<TG>; ++k) {
                if (i + k * step >= p.groups) continue;
                float u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    u[j] = elem8(gv[k], j);
                    if (mom) {
                        const float m = elem8(mv[k], j);
                        u[j] = p.nesterov ? fmaf(p.mu, m, u[j]) : m;
                    }
                }
                put(b * p.stride_x + (i + k * step) * 8, u);
            }
        }
    } else {
        for (int64_t i = (int64_t)blockIdx.x * MN_THREADS + threadIdx.x; i < p.groups; i += step) {
            const int64_t r = i / p.row_groups, c = (i - r * p.row_groups) * 8;
            float u[8];
            muon_u8<TG, false>(p, b, r, c, u);
            // (rows of X are padded to 64 columns)
            put(b * p.stride_x + r * p.ldx + c, u);
        }
    }
}

// ------------------------------------------------------- tensor-core products

// Two blocks (a cluster on two SMs) hold one 256 x 256 tile: each loads its 128
// rows of the left operand and its 128 columns of the right one, and one
// thread of the first issues products that both tensor cores run.
constexpr int GM_EPI_WARPS = 8;
constexpr int GM_THREADS = 128 + 32 * GM_EPI_WARPS;    // load, product, 2 idle, epilogue
constexpr int GM_TILE = 256, GM_ROWS = 128, GM_K = 64;
constexpr int GM_HAND = 2;                             // 22 bits: stages of one hand-over
constexpr int GM_BOX = 64 * 64 * 2;                    // bytes of one 64 x 64 fp16 box
constexpr int GM_OP = GM_ROWS * GM_K * 2;              // one operand of one block and stage
constexpr int GM_RING = 6 * 2 * GM_OP;                 // 196,608 bytes of stages
constexpr int GM_SMEM = GM_RING + 1024;                // + alignment

enum { MU_GRAM = 0, MU_SQUARE = 1, MU_UPDATE = 2, MU_LAST = 3 };

struct GemmParams {
    // hi, lo of both operands: 128 rows (columns) x 64 of K, and 64 of the right
    // one's.  K contiguous: {K, rows, 1, batch}, zeros outside.  The other way
    // round: {64, K, columns / 64, batch}: 64 K rows of one or two chunks of 64.
    CUtensorMap a[2], b[2], b_half[2];
    int32_t M, N, K, batch, tiles_m, tiles_n, tiles;   // tiles: of one matrix
    int32_t stages, width;         // clusters: stages of the ring, columns of an update's tile
    int32_t k_first, k_blocks;     // clusters: the 64s of K of this launch
    int32_t add;                   // clusters: the gram's sums are added to what dst holds
    int32_t whole;                 // pairs: tiles taken whole, the others in two halves of columns
    int32_t a_mn, b_mn;            // operand's M (N) dimension is the contiguous one
    int32_t n_fast;                // neighbouring tiles differ in N
    int32_t mode, out_type;
    float alpha, beta;             // value = alpha * sum + beta * src
    const int32_t* lift;           // [batch]
    int32_t drop, drop_next;       // what earlier steps have taken off lift, and this one
    const __half* src[2];          // elementwise operand (square: A, update: X)
    __half* dst[2];
    int64_t ld, stride;            // of src and dst
    void* out;                     // last update: the user's matrix
    int64_t ld_out, stride_out;
    int32_t out_align;             // its rows start on 16, 4 or 2-byte boundaries
    int32_t stall;                 // test hook: the products wait for what never comes
    Ctrl* ctrl;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits for a phase; gives up after MU_WAIT_NS, or once another warp has.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up,
                                          uint32_t* status) {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t it = 0; it < SPIN_LIMIT * 16u; ++it) {
        if (mbar_try(bar, parity)) return true;
        if (*gave_up) return false;
        if ((it & 63u) == 63u && global_ns() - t0 > MU_WAIT_NS) break;
    }
    *gave_up = 1;
    atomicOr(status, ST_TIMEOUT);
    return false;
}

// One box (128 or 64 rows or columns from `at`, 64 of K from `k`) into this
// block's shared memory, counted on its barrier.
__device__ __forceinline__ void tma_box1(uint32_t dst, const CUtensorMap* map, bool mn, int at, int k,
                                         int b, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(mn ? 0 : k), "r"(mn ? k : at), "r"(mn ? at >> 6 : 0), "r"(b), "r"(bar)
        : "memory");
}
// The same, counted on a barrier of either block of a pair.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, bool mn, int at, int k,
                                        int b, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(mn ? 0 : k), "r"(mn ? k : at), "r"(mn ? at >> 6 : 0), "r"(b), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t in_block(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle.  K-major: rows of 64 K
// values (128 bytes), 8-row groups 1,024 bytes apart.  M/N-major: boxes of 64
// M/N values x 64 K rows, 8,192 bytes apart, 8-row groups 1,024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn, int box = GM_BOX) {
    const uint64_t lead = mn ? (uint64_t)(box >> 4) : 1ull;
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (lead << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// D (+)= A B^T on one SM, and on a pair of SMs.
__device__ __forceinline__ void mma_f16_1(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// D = A B^T + D / MU_LO
__device__ __forceinline__ void mma_f16_lower(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p, %4;\n\t}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(idesc), "n"(MU_LO_BITS)
        : "memory");
}
__device__ __forceinline__ void mma_commit1(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}
// ... of both blocks, from the pair's first one.
__device__ __forceinline__ void mma_commit_here(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}
// Arrives on the barrier at this place in both blocks once the products so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// (the registers hold the values after tmem_wait)
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
    tmem_load32(addr, r);
    tmem_wait();
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

struct TileAt {
    int b, m, n;       // batch, this block's first row, the tile's first column
};

// The t-th size x width tile of this call.  Symmetric outputs (width = size):
// tiles (i, j) with i >= j, row by row.
__device__ __forceinline__ TileAt tile_at(const GemmParams& p, int t, int size, int width) {
    TileAt r;
    r.b = t / p.tiles;
    t -= r.b * p.tiles;
    int i, j;
    if (p.mode <= MU_SQUARE) {
        i = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
        while (i * (i + 1) / 2 > t) --i;
        while ((i + 1) * (i + 2) / 2 <= t) ++i;
        j = t - i * (i + 1) / 2;
    } else if (p.n_fast) {
        i = t / p.tiles_n;
        j = t - i * p.tiles_n;
    } else {
        j = t / p.tiles_m;
        i = t - j * p.tiles_m;
    }
    r.m = i * size;
    r.n = j * width;
    return r;
}

// The u-th piece of work of a pair kernel: a whole tile, or half the columns
// of one of the last tiles.
struct Piece {
    TileAt at;         // (m: this block's rows; n: the piece's first column)
    int width;         // columns
    bool diagonal;     // of a symmetric output
};
__device__ __forceinline__ Piece piece_at(const GemmParams& p, int u, int rank) {
    Piece r;
    const int h = u - p.whole;
    r.at = tile_at(p, h < 0 ? u : p.whole + (h >> 1), GM_TILE, GM_TILE);
    r.diagonal = r.at.m == r.at.n;
    r.width = h < 0 ? GM_TILE : GM_TILE / 2;
    r.at.m += rank * GM_ROWS;
    if (h >= 0) r.at.n += (h & 1) * (GM_TILE / 2);
    return r;
}

// Sixteen fp16 values, 32 bytes: one whole memory sector for each lane.
__device__ __forceinline__ void load_half16(const __half* p, float* v) {
    uint4 q[2];
    load32b(p, q);
    const __half2* h = reinterpret_cast<const __half2*>(q);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 f = __half22float2(h[j]);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 columns of one row (each lane its own) of the caller's matrix: 32 or 16
// bytes at a time where its rows start on 16-byte boundaries, pairs of 16-bit
// values where they start on 4-byte ones, else the warp turns its 32 x 32 values
// and writes row by row.  (Five steps of 5 x 818 x 363 fp32: 232 us turned, 237 by
// single values; of 5 x 4,532 x 1,172 to bf16: 978 us turned, 950 by pairs.)
template <typename TO>
__device__ __forceinline__ void store_out(const GemmParams& p, int64_t b, int64_t row, int64_t c0,
                                          float* v) {
    TO* out = static_cast<TO*>(p.out) + b * p.stride_out;
    if (p.out_align >= (sizeof(TO) == 2 ? 4 : 16) && c0 + 32 <= p.N) {
        if (row >= p.M) return;
        TO* dst = out + row * p.ld_out + c0;
        constexpr int E = 32 / (int)sizeof(TO);
#pragma unroll
        for (int j = 0; j < 32; j += E) {
            uint4 r[2];
#pragma unroll
            for (int e = 0; e < E; ++e) reinterpret_cast<TO*>(r)[e] = from_f32<TO>(v[j + e]);
            if ((uintptr_t)dst % 32 == 0) {
                store32b(dst + j, r);
            } else if (p.out_align == 16) {
                reinterpret_cast<uint4*>(dst + j)[0] = r[0];
                reinterpret_cast<uint4*>(dst + j)[1] = r[1];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    reinterpret_cast<uint32_t*>(dst + j)[e] = reinterpret_cast<const uint32_t*>(r)[e];
            }
        }
        return;
    }
    const int lane = (int)lane_id();
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (j & s) continue;
            const float got = __shfl_xor_sync(0xFFFFFFFFu, lane & s ? v[j] : v[j + s], s);
            if (lane & s) v[j] = got;
            else v[j + s] = got;
        }
    TO* dst = out + (row - lane) * p.ld_out + c0 + lane;
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (row - lane + j < p.M && c0 + lane < p.N) dst[j * p.ld_out] = from_f32<TO>(v[j]);
}

// 32 columns of one row of fp16 pairs (hi, and lo where wanted).
__device__ __forceinline__ void store_pair(const GemmParams& p, int64_t o, const float* v,
                                           bool want_lo) {
#pragma unroll
    for (int j = 0; j < 32; j += 16) {
        uint4 q[2];
        uint32_t* r = reinterpret_cast<uint32_t*>(q);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = pack2(v[j + 2 * e], v[j + 2 * e + 1]);
        store32b(p.dst[0] + o + j, q);
        if (want_lo) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[e] = pack2(below_half(v[j + 2 * e]), below_half(v[j + 2 * e + 1]));
            store32b(p.dst[1] + o + j, q);
        }
    }
}

// What a tile's values are multiplied by besides alpha and beta: X is held
// times 2^k, k = max(0, lift - drop), and the next X times 2^max(0, lift -
// drop_next).
template <int MODE>
__device__ __forceinline__ void lift_factors(const GemmParams& p, int b, float* sum, float* src) {
    *sum = *src = 1.0f;
    const int lift = p.lift[b];
    if (lift == 0) return;
    const int k = max(0, lift - p.drop), next = max(0, lift - p.drop_next);
    if (MODE == MU_GRAM) *sum = exp2f((float)(-2 * k));
    else if (MODE == MU_UPDATE) *sum = *src = exp2f((float)(next - k));
    else if (MODE == MU_LAST) *sum = *src = exp2f((float)-k);
}

// The elementwise operand of one row's 32 columns: hi, or both.
template <bool EXACT, int MODE>
__device__ __forceinline__ void load_src32(const GemmParams& p, int64_t o, bool live, float* x) {
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = 0.0f;
    if (MODE != MU_GRAM && live) {
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
            load_half16(p.src[0] + o + j, x + j);
            if (EXACT || MODE >= MU_UPDATE) {
                float l[16];
                load_half16(p.src[1] + o + j, l);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[j + e] = of_pair(x[j + e], l[e]);
            }
        }
    }
}

// One row's 32 columns of a finished tile; v: the sums, x: the elementwise
// operand.  (Rows of src and dst are padded to 64 columns: 32 at a time stay
// inside.)  mirror: the tile lies below the diagonal, and its image above is
// written too (a warp's 32 rows are 32 consecutive columns there).
template <bool EXACT, int MODE>
__device__ __forceinline__ void epilogue32(const GemmParams& p, const TileAt& at, float alpha,
                                           float beta, int64_t row, int64_t c0, bool mirror,
                                           float* v, const float* x) {
    if (c0 >= p.N || (MODE != MU_LAST && row >= p.M)) return;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = MODE == MU_GRAM ? alpha * v[j] : fmaf(alpha, v[j], beta * x[j]);
    if (MODE == MU_LAST) {
        if (p.out_type == 0) store_out<float>(p, at.b, row, c0, v);
        else if (p.out_type == 1) store_out<__nv_bfloat16>(p, at.b, row, c0, v);
        else store_out<__half>(p, at.b, row, c0, v);
        return;
    }
    store_pair(p, at.b * p.stride + row * p.ld + c0, v, EXACT || MODE == MU_UPDATE);
    if (MODE <= MU_SQUARE && mirror) {
        const int64_t o = at.b * p.stride + c0 * p.ld + row;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            p.dst[0][o + j * p.ld] = __float2half_rn(v[j]);
            if (EXACT) p.dst[1][o + j * p.ld] = __float2half_rn(below_half(v[j]));
        }
    }
}

// Persistent pairs: pair x takes tiles x, x + pairs, ...  In each block one
// thread loads boxes by TMA into a ring of stages; in the first one thread
// issues the products into one of two TMEM accumulators (2 x 256 columns)
// while eight warps of each block drain the other.
//
// Bound by the tensor cores at the clock that the power cap leaves (the pipe is
// active 59 to 62% of a launch, 64 to 69% with 22 bits), by the rounds that leave
// pairs idle and by the last round's epilogue: gram, square and update of
// 4,096 x 4,096 in 61, 61 and 111 us at 1.6 GHz (1.1 to 1.25 PFLOP/s,
// symmetric products by half; with 22 bits 167, 172 and 315), of 25,088 x 4,096 in
// 356, 76 and 674.  (Five steps and the two passes before them: 1.23 ms; 1.34 to 1.5
// in calls that follow one another, at the 1.3 to 1.4 GHz of the power cap.)
//
// With 22 bits (see MU_LOW) the accumulator is handed over after every 128 of K
// and added up in registers with rounding to nearest: first the small products (hi
// lo, lo hi) of both stages, which the first of the large ones divides by MU_LO.
// The lo parts of a stage are free, and loaded again, before its hi parts.  (A
// hand-over of every 64, which needs no two stages at once, keeps the epilogue's
// warps busier than the tensor cores: 4,096 x 4,096 3.87 ms by 128, 4.61 by 64.)
template <bool EXACT, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GM_THREADS, 1)
    muon_gemm_kernel(const __grid_constant__ GemmParams p) {
    constexpr int PARTS = EXACT ? 2 : 1;
    constexpr int STAGE = PARTS * 2 * GM_OP;           // one block's bytes of a stage
    constexpr int STAGES = GM_RING / STAGE;
    constexpr int HALF = GM_TILE / 2;                  // columns of one epilogue warp
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t s_full[STAGES], s_empty[STAGES], s_empty_lo[STAGES];
    __shared__ __align__(8) uint64_t s_done[2], s_free[2], s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_gave_up;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const int warp = (int)warp_id(), lane = (int)lane_id();
    const int rank = (int)cluster_rank();
    const int pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;
    if (threadIdx.x == 0) {
        s_gave_up = 0;
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&s_full[s]), 1);
            mbar_init(smem_u32(&s_empty[s]), 1);
            mbar_init(smem_u32(&s_empty_lo[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&s_done[s]), 1);
            mbar_init(smem_u32(&s_free[s]), 2 * GM_EPI_WARPS);
        }
        mbar_init(smem_u32(&s_drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane < PARTS) {
        prefetch_map(&p.a[lane]);
        prefetch_map(&p.b[lane]);
        prefetch_map(&p.b_half[lane]);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(&s_tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_tmem;
    uint32_t* status = &p.ctrl->status;
    const int total = 2 * p.tiles * p.batch - p.whole;     // pieces
    const int kblocks = (p.K + GM_K - 1) / GM_K;
    pdl_launch();
    pdl_wait();

    // With 22 bits: 384 threads start with 168 registers each; the 128
    // running sums of an epilogue thread need more: 72 + 216 + 216 = 3 x 168.
    const int group = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x / 128, 0);
    if (group == 0) {
        if (EXACT) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0 && lane == 0) {
            // ---- loads (of what earlier kernels wrote with ordinary stores)
            asm volatile("fence.proxy.async;" ::: "memory");
            int stage = 0;
            uint32_t phase = 0, issued = 0;
            bool ok = true;
            for (int t = pair; t < total && ok; t += pairs) {
                const Piece piece = piece_at(p, t, rank);
                const TileAt at = piece.at;
                const int n0 = at.n + rank * (piece.width / 2);
                const CUtensorMap* right = piece.width == GM_TILE ? p.b : p.b_half;
                const uint32_t bytes = 2 * PARTS * (GM_OP + piece.width / 2 * GM_K * 2);
                for (int kb = 0; kb < kblocks; ++kb) {
                    const uint32_t bar = in_block(smem_u32(&s_full[stage]), 0);
                    const uint32_t dst = base + stage * STAGE;
                    const int k = kb * GM_K;
                    // (lo before hi: the order in which they become free)
#pragma unroll
                    for (int q = PARTS - 1; q >= 0; --q) {
                        if (!(ok = mbar_wait(smem_u32(q ? &s_empty_lo[stage] : &s_empty[stage]),
                                             phase ^ 1, &s_gave_up, status)))
                            break;
                        if (q == PARTS - 1) {
                            if (rank == 0) mbar_expect(smem_u32(&s_full[stage]), bytes);
                            ++issued;
                        }
                        tma_box(dst + q * GM_OP, &p.a[q], p.a_mn, at.m, k, at.b, bar);
                        tma_box(dst + (PARTS + q) * GM_OP, right + q, p.b_mn, n0, k, at.b, bar);
                    }
                    if (!ok) break;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // no copy is in flight when the pair ends (its first block counts both blocks')
            if (rank == 0)
                for (uint32_t j = issued < STAGES ? issued : STAGES; j > 0; --j) {
                    const uint32_t n = issued - j;
                    volatile int never = 0;
                    mbar_wait(smem_u32(&s_full[n % STAGES]), (n / STAGES) & 1, &never, status);
                }
        } else if (warp == 1 && lane == 0 && rank == 0) {
            // ---- products
            const uint32_t shape = (1u << 4) | ((uint32_t)p.a_mn << 15) | ((uint32_t)p.b_mn << 16) |
                                   ((GM_TILE / 16) << 24);
            const uint32_t a_step = p.a_mn ? 2048 : 32, b_step = p.b_mn ? 2048 : 32;
            const int chunk = EXACT ? GM_HAND : kblocks;
            int stage = 0, slot = 0;
            uint32_t phase = 0, slot_phase = 0;
            bool ok = !p.stall || mbar_wait(smem_u32(&s_done[0]), 0, &s_gave_up, status);
            for (int t = pair; t < total && ok; t += pairs) {
                const uint32_t width = t < p.whole ? GM_TILE : GM_TILE / 2;
                const uint32_t idesc = shape | ((width / 8) << 17);
                for (int kb = 0; kb < kblocks && ok; kb += chunk) {
                    if (!(ok = mbar_wait(smem_u32(&s_free[slot]), slot_phase ^ 1, &s_gave_up, status)))
                        break;
                    const uint32_t d = tmem + slot * GM_TILE;
                    const int n = min(chunk, kblocks - kb);
                    if (EXACT) {
                        int s = stage;
                        uint32_t ph = phase;
                        for (int j = 0; j < n; ++j) {
                            if (!(ok = mbar_wait(smem_u32(&s_full[s]), ph, &s_gave_up, status))) break;
                            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                            const uint32_t a0 = base + s * STAGE, b0 = a0 + PARTS * GM_OP;
#pragma unroll
                            for (int k = 0; k < GM_K / 16; ++k) {
                                mma_f16(d, smem_desc(a0 + k * a_step, p.a_mn),
                                        smem_desc(b0 + GM_OP + k * b_step, p.b_mn), idesc,
                                        j > 0 || k > 0);
                                mma_f16(d, smem_desc(a0 + GM_OP + k * a_step, p.a_mn),
                                        smem_desc(b0 + k * b_step, p.b_mn), idesc, true);
                            }
                            mma_commit(smem_u32(&s_empty_lo[s]));
                            if (++s == STAGES) {
                                s = 0;
                                ph ^= 1;
                            }
                        }
                        if (!ok) break;
                    }
                    for (int j = 0; j < n; ++j) {
                        if (!EXACT) {
                            if (!(ok = mbar_wait(smem_u32(&s_full[stage]), phase, &s_gave_up, status)))
                                break;
                            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        }
                        const uint32_t a0 = base + stage * STAGE, b0 = a0 + PARTS * GM_OP;
#pragma unroll
                        for (int k = 0; k < GM_K / 16; ++k) {
                            const uint64_t ah = smem_desc(a0 + k * a_step, p.a_mn);
                            const uint64_t bh = smem_desc(b0 + k * b_step, p.b_mn);
                            if (EXACT && j == 0 && k == 0) mma_f16_lower(d, ah, bh, idesc);
                            else mma_f16(d, ah, bh, idesc, j > 0 || k > 0);
                        }
                        mma_commit(smem_u32(&s_empty[stage]));
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                    if (!ok) break;
                    mma_commit(smem_u32(&s_done[slot]));
                    if (++slot == 2) {
                        slot = 0;
                        slot_phase ^= 1;
                    }
                }
            }
        }
    } else {
        if (EXACT) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ---- epilogue: warp w reads TMEM lanes 32 (w mod 4) .., half of the columns
        const int quad = warp & 3;
        int slot = 0;
        uint32_t slot_phase = 0;
        bool ok = true;
        auto drained = [&]() {
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(in_block(smem_u32(&s_free[slot]), 0));
            if (++slot == 2) {
                slot = 0;
                slot_phase ^= 1;
            }
        };
        auto wait_done = [&]() {
            ok = mbar_wait(smem_u32(&s_done[slot]), slot_phase, &s_gave_up, status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            return ok;
        };
        for (int t = pair; t < total && ok; t += pairs) {
            const Piece piece = piece_at(p, t, rank);
            const TileAt at = piece.at;
            const int cols = piece.width / 2, col = warp < 8 ? 0 : cols;     // this warp's
            const uint32_t src = tmem + col + ((uint32_t)(quad * 32) << 16);
            const int64_t row = at.m + quad * 32 + lane;
            float fs, fx;
            lift_factors<MODE>(p, at.b, &fs, &fx);
            const float low = EXACT && MODE <= MU_SQUARE
                                  ? MU_LOW * (GM_K / 16) * (float)min(kblocks, GM_HAND)
                                  : 0.0f;
            const float alpha = p.alpha * fs * (1.0f + low), beta = p.beta * fx;
            const int64_t o = at.b * p.stride + row * p.ld + at.n + col;
            const bool mirror = !piece.diagonal;
            float x[32];
            if (EXACT) {
                float sum[HALF];
#pragma unroll
                for (int c = 0; c < HALF; ++c) sum[c] = 0.0f;
                for (int kb = 0; kb < kblocks; kb += GM_HAND) {
                    if (!wait_done()) break;
#pragma unroll
                    for (int c = 0; c < HALF; c += 64) {
                        if (c >= cols) break;
                        float v[64];
                        tmem_load32(src + slot * GM_TILE + c, reinterpret_cast<uint32_t*>(v));
                        tmem_load32(src + slot * GM_TILE + c + 32, reinterpret_cast<uint32_t*>(v + 32));
                        tmem_wait();
#pragma unroll
                        for (int j = 0; j < 64; ++j) sum[c + j] += v[j];
                    }
                    if (kb + GM_HAND < kblocks) drained();
                }
                if (!ok) break;
                // back to where the last sums came from, for the loop below
#pragma unroll
                for (int c = 0; c < HALF; c += 32)
                    if (c < cols) tmem_st32(src + slot * GM_TILE + c, reinterpret_cast<uint32_t*>(sum + c));
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                load_src32<EXACT, MODE>(p, o, row < p.M && at.n + col < p.N, x);
            } else {
                load_src32<EXACT, MODE>(p, o, row < p.M && at.n + col < p.N, x);
                if (!wait_done()) break;
            }
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
                float v[32], next[32];
                load_src32<EXACT, MODE>(p, o + c + 32, c + 32 < cols && row < p.M &&
                                        at.n + col + c + 32 < p.N, next);
                tmem_ld32(src + slot * GM_TILE + c, reinterpret_cast<uint32_t*>(v));
                epilogue32<EXACT, MODE>(p, at, alpha, beta, row, at.n + col + c, mirror, v, x);
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = next[j];
            }
            drained();
        }
    }
    __syncthreads();
    // when a wait gave up, products may still be running: let them end before
    // their accumulators are freed
    if (s_gave_up && threadIdx.x == 32 && rank == 0) {
        volatile int never = 0;
        mma_commit_here(smem_u32(&s_drain));
        mbar_wait(smem_u32(&s_drain), 0, &never, status);
    }
    __syncthreads();
    cluster_sync();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------- products of few tiles: K over a cluster

// Where there are fewer 256 x 256 tiles than pairs of SMs: one 128 x 128 tile per
// cluster of 1, 2, 4 or 8 blocks, each of which takes a part of K.  The blocks' sums
// meet in shared memory: block r adds up the r-th part of the rows over all
// blocks, in block order, and finishes them.  Bound by latency: of 8 to 10 us a
// launch 2.5 pass between the products before and the first of its own, 1 to 3 in
// products, 2 to 3 in the exchange (64 KB into each SM) and 1 to 3 in the epilogue.
constexpr int SP_THREADS = 256;
constexpr int SP_TILE = 128;
constexpr int SP_MIN_STAGES = 3, SP_MAX_STAGES = 6;    // 11 bits: 3 leave room for two
                                                       // blocks an SM, 6 cover the latency of one
constexpr int SP_LD = SP_TILE + 4;                     // row of sums, in floats
constexpr int SP_MAX_SUM = 48;     // 22 bits: 64s of K of one block and launch (64 truncated adds)
constexpr int SP_SUMS = SP_TILE * SP_LD * 4;           // bytes of the sums, then the turned tile
constexpr int sp_smem(bool exact, int stages) {
    const int ring = stages * (exact ? 4 : 2) * GM_OP;
    const int after = SP_SUMS + (exact ? 2 : 1) * SP_TILE * (SP_TILE + 8) * 2;
    return (ring > after ? ring : after) + 1024;
}

// Four columns of one row; v: the sums, h and l: the elementwise operand (of a gram:
// the sums of the K before); v becomes the value.  (The last update's values are
// stored by store_rows.)
template <bool EXACT, int MODE>
__device__ __forceinline__ void epilogue4(const GemmParams& p, const TileAt& at, float alpha,
                                          float beta, int64_t row, int64_t c0, uint2 h, uint2 l,
                                          float* v) {
    const __half* hh = reinterpret_cast<const __half*>(&h);
    const __half* ll = reinterpret_cast<const __half*>(&l);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = MODE == MU_GRAM && !EXACT
                   ? alpha * v[j]
                   : fmaf(alpha, v[j], (MODE == MU_GRAM ? 1.0f : beta) *
                                           of_pair(__half2float(hh[j]), __half2float(ll[j])));
    if (row >= p.M || c0 >= p.N) return;
    if (MODE == MU_LAST) return;
    const int64_t o = at.b * p.stride + row * p.ld + c0;
    *reinterpret_cast<uint2*>(p.dst[0] + o) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    if (EXACT || MODE == MU_UPDATE)
        *reinterpret_cast<uint2*>(p.dst[1] + o) =
            make_uint2(pack2(below_half(v[0]), below_half(v[1])),
                       pack2(below_half(v[2]), below_half(v[3])));
}

// `rows` rows of `width` values of the last update, from shared memory: columns
// lane by lane, since the caller's rows may start anywhere.
template <typename TO>
__device__ __forceinline__ void store_rows(const GemmParams& p, const TileAt& at, int first, int rows,
                                           int width, const float* sums) {
    TO* out = static_cast<TO*>(p.out) + at.b * p.stride_out;
    const int64_t last = min((int64_t)width, p.N - (int64_t)at.n);
    for (int r = first + (int)warp_id(); r < first + rows; r += SP_THREADS / 32) {
        if (at.m + r >= p.M) return;
        TO* dst = out + (at.m + r) * p.ld_out + at.n;
        const float* src = sums + r * SP_LD;
#pragma unroll
        for (int j = 0; j < SP_TILE / 32; ++j) {
            const int c = j * 32 + (int)lane_id();
            if (c < last) dst[c] = from_f32<TO>(src[c]);
        }
    }
}

// Adds up, in block order, the sums of this block's part of the rows over the
// S blocks of the cluster, into its own.  Each warp has 16 loads of 512
// contiguous bytes in flight: it is their latency that costs.
template <int S>
__device__ __forceinline__ void add_blocks(float* sums, int rank) {
    constexpr int R = SP_TILE / S / (SP_THREADS / 32);
    const int row = rank * (SP_TILE / S) + (int)warp_id();
    const uint32_t mine = smem_u32(sums) + (uint32_t)(row * SP_LD + (int)lane_id() * 4) * 4;
    float4 y[S][R];
#pragma unroll
    for (int q = 0; q < S; ++q) {
        const uint32_t from = in_block(mine, q);
#pragma unroll
        for (int r = 0; r < R; ++r)
            asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(y[q][r].x), "=f"(y[q][r].y), "=f"(y[q][r].z), "=f"(y[q][r].w)
                         : "r"(from + (uint32_t)(r * (SP_THREADS / 32) * SP_LD * 4)));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float4 x = y[0][r];
#pragma unroll
        for (int q = 1; q < S; ++q) {
            x.x += y[q][r].x;
            x.y += y[q][r].y;
            x.z += y[q][r].z;
            x.w += y[q][r].w;
        }
        *reinterpret_cast<float4*>(sums + (row + r * (SP_THREADS / 32)) * SP_LD + lane_id() * 4) = x;
    }
}

// 22 bits: the large products of successive 64 of K go to three
// accumulators in turn and the small ones to a fourth, which keeps the
// truncated sums short (see muon_gemm_kernel).
template <bool EXACT, int MODE>
__global__ void __launch_bounds__(SP_THREADS) muon_split_kernel(const __grid_constant__ GemmParams p) {
    constexpr int PARTS = EXACT ? 2 : 1;
    constexpr int STAGE = PARTS * 2 * GM_OP;
    constexpr int BIG = EXACT ? 3 : 1;                 // accumulators of large products
    constexpr uint32_t COLS = EXACT ? 512 : 128;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t s_full[SP_MAX_STAGES], s_empty[SP_MAX_STAGES], s_done;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_gave_up;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const int warp = (int)warp_id(), lane = (int)lane_id();
    const int rank = (int)cluster_rank(), stages = p.stages;
    uint32_t split;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    if (threadIdx.x == 0) {
        s_gave_up = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_u32(&s_full[s]), 1);
            mbar_init(smem_u32(&s_empty[s]), 1);
        }
        mbar_init(smem_u32(&s_done), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane < PARTS) {
        prefetch_map(&p.a[lane]);
        prefetch_map(&p.b[lane]);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&s_tmem)), "n"(COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_tmem;
    uint32_t* status = &p.ctrl->status;
    // (an update that leaves SMs idle takes 64 columns at a time)
    const int width = MODE <= MU_SQUARE ? SP_TILE : p.width;
    const TileAt at = tile_at(p, (int)(blockIdx.x / split), SP_TILE, width);
    const int before = (int)((int64_t)p.k_blocks * rank / split), kb0 = p.k_first + before;
    const int n = (int)((int64_t)p.k_blocks * (rank + 1) / split) - before;
    pdl_launch();
    pdl_wait();

    if (warp == 0 && lane == 0) {
        asm volatile("fence.proxy.async;" ::: "memory");
        const CUtensorMap* right = width == SP_TILE ? p.b : p.b_half;
        int i = 0, s = 0;
        uint32_t phase = 0;
        for (; i < n; ++i) {
            if (!mbar_wait(smem_u32(&s_empty[s]), phase ^ 1, &s_gave_up, status)) break;
            const uint32_t bar = smem_u32(&s_full[s]);
            mbar_expect(bar, PARTS * (GM_OP + width * GM_K * 2));
            const uint32_t dst = base + s * STAGE;
            const int k = (kb0 + i) * GM_K;
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                tma_box1(dst + q * GM_OP, &p.a[q], p.a_mn, at.m, k, at.b, bar);
                tma_box1(dst + (PARTS + q) * GM_OP, right + q, p.b_mn, at.n, k, at.b, bar);
            }
            if (++s == stages) {
                s = 0;
                phase ^= 1;
            }
        }
        // no copy is in flight when the stages are used for the sums
        for (int j = max(0, i - stages); j < i; ++j) {
            volatile int never = 0;
            mbar_wait(smem_u32(&s_full[j % stages]), (j / stages) & 1, &never, status);
        }
    } else if (warp == 1 && lane == 0) {
        const uint32_t idesc = (1u << 4) | ((uint32_t)p.a_mn << 15) | ((uint32_t)p.b_mn << 16) |
                               ((uint32_t)(width / 8) << 17) | ((SP_TILE / 16) << 24);
        const uint32_t a_step = p.a_mn ? 2048 : 32, b_step = p.b_mn ? 2048 : 32;
        int s = 0;
        uint32_t phase = 0;
        const bool stalled = p.stall && !mbar_wait(smem_u32(&s_done), 0, &s_gave_up, status);
        for (int i = 0; i < n && !stalled; ++i) {
            if (!mbar_wait(smem_u32(&s_full[s]), phase, &s_gave_up, status)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t a0 = base + s * STAGE, b0 = a0 + PARTS * GM_OP;
            const uint32_t d = tmem + (i % BIG) * SP_TILE, small = tmem + BIG * SP_TILE;
#pragma unroll
            for (int k = 0; k < GM_K / 16; ++k) {
                const uint64_t ah = smem_desc(a0 + k * a_step, p.a_mn);
                const uint64_t bh = smem_desc(b0 + k * b_step, p.b_mn);
                mma_f16_1(d, ah, bh, idesc, i >= BIG || k > 0);
                if (EXACT) {
                    mma_f16_1(small, ah, smem_desc(b0 + GM_OP + k * b_step, p.b_mn), idesc,
                              i > 0 || k > 0);
                    mma_f16_1(small, smem_desc(a0 + GM_OP + k * a_step, p.a_mn), bh, idesc, true);
                }
            }
            mma_commit1(smem_u32(&s_empty[s]));
            if (++s == stages) {
                s = 0;
                phase ^= 1;
            }
        }
        mma_commit1(smem_u32(&s_done));
    }
    __syncwarp();
    // all warps drain the accumulators: rows 32 (warp mod 4) .., half of the columns
    {
        volatile int never = 0;
        mbar_wait(smem_u32(&s_done), 0, &never, status);
    }
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const int quad = warp & 3;
    float fs, fx;
    lift_factors<MODE>(p, at.b, &fs, &fx);
    const float alpha = p.alpha * fs, beta = p.beta * fx;
    const float low = MODE > MU_SQUARE ? 0.0f : MU_LOW * (GM_K / 16) * (float)n / (float)min(n, BIG);
    float* sums = reinterpret_cast<float*>(raw + (base - smem_u32(raw)));
#pragma unroll 1
    for (int c = (warp >> 2) * 32; c < width; c += 64) {
        float v[32];
        const uint32_t src = tmem + c + ((uint32_t)(quad * 32) << 16);
        tmem_ld32(src, reinterpret_cast<uint32_t*>(v));
        if (EXACT) {
            for (int a = 1; a <= BIG; ++a) {
                if (a < BIG && a >= n) continue;
                float w[32];
                tmem_ld32(src + a * SP_TILE, reinterpret_cast<uint32_t*>(w));
                const float by = a < BIG ? 1.0f : 1.0f / MU_LO;
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = fmaf(by, w[j], v[j]);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = fmaf(low, v[j], v[j]);
        }
        float* to = sums + (quad * 32 + lane) * SP_LD + c;
#pragma unroll
        for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(to + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
    if (split > 1) cluster_sync();
    else __syncthreads();
    if (split == 2) add_blocks<2>(sums, rank);
    else if (split == 4) add_blocks<4>(sums, rank);
    else if (split == 8) add_blocks<8>(sums, rank);

    // This block's rows, one (two of 64 columns) per warp at a time; the mirror
    // image is turned in shared memory.
    constexpr int U = 4;
    const int rows = SP_TILE / (int)split, pitch = rows + 8;
    const int lanes = width / 4, col = lane % lanes * 4;       // lanes of a row, first column
    const int step = SP_THREADS / lanes;                       // rows at a time
    const int64_t c0 = at.n + col;
    const bool mirror = MODE <= MU_SQUARE && at.m != at.n;
    __half* turned = reinterpret_cast<__half*>(sums + SP_TILE * SP_LD);    // [hi, lo][128][pitch]
    for (int r0 = (int)threadIdx.x / lanes; r0 < rows; r0 += U * step) {
        float4 x[U];
        uint2 h[U], l[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * step;
            const int64_t row = at.m + rank * rows + r, o = at.b * p.stride + row * p.ld + c0;
            h[u] = l[u] = make_uint2(0, 0);
            if (MODE == MU_GRAM ? EXACT && p.add : true) {
                if (r >= rows || row >= p.M || c0 >= p.N) continue;
                const __half* const* src = MODE == MU_GRAM ? p.dst : p.src;
                h[u] = *reinterpret_cast<const uint2*>(src[0] + o);
                if (EXACT || MODE >= MU_UPDATE)
                    l[u] = *reinterpret_cast<const uint2*>(src[1] + o);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = min(r0 + u * step, rows - 1);
            x[u] = *reinterpret_cast<const float4*>(sums + (rank * rows + r) * SP_LD + col);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * step;
            if (r >= rows) continue;
            float* v = reinterpret_cast<float*>(&x[u]);
            epilogue4<EXACT, MODE>(p, at, alpha, beta, at.m + rank * rows + r, c0, h[u], l[u], v);
            if (MODE == MU_LAST)
                *reinterpret_cast<float4*>(sums + (rank * rows + r) * SP_LD + col) = x[u];
            if (mirror) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    turned[(col + j) * pitch + r] = __float2half_rn(v[j]);
                    if (EXACT)
                        turned[(SP_TILE + col + j) * pitch + r] = __float2half_rn(below_half(v[j]));
                }
            }
        }
    }
    if (MODE == MU_LAST) {
        __syncthreads();
        if (p.out_type == 0) store_rows<float>(p, at, rank * rows, rows, width, sums);
        else if (p.out_type == 1) store_rows<__nv_bfloat16>(p, at, rank * rows, rows, width, sums);
        else store_rows<__half>(p, at, rank * rows, rows, width, sums);
    }
    if (mirror) {
        __syncthreads();
        const int groups = rows / 8;
        const int64_t row0 = at.m + rank * rows;
        for (int g = (int)threadIdx.x; g < groups * SP_TILE; g += SP_THREADS) {
            const int c = g / groups, r = g % groups * 8;
            if (row0 + r >= p.M) continue;
            // (a row of dst is padded to 64 columns)
            const int64_t o = at.b * p.stride + (at.n + c) * p.ld + row0 + r;
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
                *reinterpret_cast<uint4*>(p.dst[q] + o) =
                    *reinterpret_cast<const uint4*>(turned + (q * SP_TILE + c) * pitch + r);
        }
    }
    if (split > 1) cluster_sync();     // no block leaves while its sums are read
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(COLS));
}

// ------------------------------------------------ small matrices: one kernel

// A matrix whose short side is at most 128 and whose long side at most 4,096: a
// cluster of up to 16 blocks does the whole call, each with up to 256 columns of X
// (the short side as rows), with X, A and B in shared memory, the sums in TMEM and
// the three products of 22 bits throughout (they cost nothing here: each product
// waits for the one before).  Only the gram needs the other blocks: each adds up
// its part of the rows over all of them, in block order, and hands them out.  X is
// held with the short side as rows: chunks of 64 columns, 128 rows of 128 swizzled
// bytes each, which the gram reads as K-major and the update as N-major operand.
// Bound by latency, and with a wide short side by the exchange
// (64 KB into each block, and out of it): five steps of 64 x 27 take 31 us against
// 107 in 17 launches, 64 x 600 54 against 123, two of 2,000 x 128 104 against 150.
// What lies outside the matrix is zero and stays zero.
constexpr int TN_THREADS = 256;
constexpr int TN_ROWS = 128, TN_COLS = 256;            // of one block
constexpr int TN_MAX_BLOCKS = 16;                      // of a matrix
constexpr int TN_CHUNK = TN_ROWS * 128;                // bytes of 64 columns
constexpr int TN_X = TN_COLS / 64 * TN_CHUNK, TN_A = TN_ROWS / 64 * TN_CHUNK;   // hi (or lo)
constexpr int TN_SMEM = 2 * TN_X + 2 * TN_A + 1024;
constexpr int TN_MAX_STEPS = 64;
// groups of 8 columns that a thread adds up, at most: two blocks share 128 rows of 16
constexpr int TN_GROUPS = TN_ROWS / 2 * (TN_ROWS / 8) / TN_THREADS;

struct TinyParams {
    MuonPreParams pre;             // (rows, cols: the caller's; groups unused)
    float coef[3 * TN_MAX_STEPS];
    int8_t drop[TN_MAX_STEPS + 1]; // (saturated)
    int32_t steps, out_type;
    int32_t stall;                 // test hook: as in GemmParams
    float scale;
    void* out;
    int64_t ld_out, stride_out;
};

// Byte offset of 16-byte unit u of row r of a chunk.
__device__ __forceinline__ uint32_t tn_unit(int r, int u) {
    return (uint32_t)(r * 128 + ((u ^ (r & 7)) << 4));
}

// ... and of an fp32 value in the place of X's entry (r, c).
__device__ __forceinline__ uint32_t tn_f32(int r, int c) {
    return (uint32_t)(c >> 6) * TN_CHUNK + tn_unit(r, (c & 63) >> 3) + (c & 3) * 4 + (c & 4 ? TN_X : 0);
}

template <typename TG>
__global__ void __launch_bounds__(TN_THREADS, 1) muon_tiny_kernel(const __grid_constant__ TinyParams p) {
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t s_done, s_drain;
    __shared__ double s_red[33], s_norm;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_gave_up;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* mem = raw + (base - smem_u32(raw));
    const uint32_t x_at = base, a_at = base + 2 * TN_X;
    const int tid = (int)threadIdx.x, warp = (int)warp_id(), lane = (int)lane_id();
    if (tid == 0) {
        s_gave_up = 0;
        mbar_init(smem_u32(&s_done), 1);
        mbar_init(smem_u32(&s_drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(&s_tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    for (int i = tid; i < (2 * TN_X + 2 * TN_A) / 16; i += TN_THREADS)
        reinterpret_cast<uint4*>(mem)[i] = make_uint4(0, 0, 0, 0);
    pdl_launch();
    pdl_wait();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_tmem;
    uint32_t* status = &p.pre.ctrl->status;
    // this block's columns of X: [q0, q0 + Q) of the long side
    uint32_t blocks;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(blocks));
    const int rank = (int)cluster_rank(), cl = (int)blocks;
    const int64_t b = blockIdx.x / blocks;
    const bool tall = p.pre.rows > p.pre.cols;
    const int P = (int)(tall ? p.pre.cols : p.pre.rows), all = (int)(tall ? p.pre.rows : p.pre.cols);
    const int share = (all + cl - 1) / cl;
    const int q0 = rank * share, Q = min(all - q0, share);
    const int n = tall ? P : Q, total = P * Q;             // this block's part: rows of n
    const int64_t first = tall ? (int64_t)q0 * p.pre.cols : q0;
    if (blockIdx.x == 0 && tid == 0) {
        p.pre.ctrl->path_small = 0;
        p.pre.ctrl->status = 0;
    }

    // ---- momentum, norm, X
    const TG* g = static_cast<const TG*>(p.pre.grad) + b * p.pre.stride_g +
                  (tall ? q0 * p.pre.ld_g : q0);
    float* mom =
        p.pre.momentum ? p.pre.momentum + b * p.pre.rows * p.pre.cols + first : nullptr;
    // (u waits in X's place as fp32: a 16-byte unit of hi and of lo are 8 values)
    double sum = 0.0;
#pragma unroll 8
    for (int i = tid; i < total; i += TN_THREADS) {
        const int r = i / n, c = i - r * n;
        float u = to_f32(g[r * p.pre.ld_g + c]);
        if (mom) {
            const int64_t o = (int64_t)r * p.pre.cols + c;
            const float v = fmaf(p.pre.mu, mom[o], u);
            mom[o] = v;
            u = p.pre.nesterov ? fmaf(p.pre.mu, v, u) : v;
        }
        sum = fma((double)u, (double)u, sum);
        *reinterpret_cast<float*>(mem + (tall ? tn_f32(c, r) : tn_f32(r, c))) = u;
    }
    sum = block_sum(sum, s_red);
    if (cl > 1) {
        if (tid == 0) s_norm = sum;
        cluster_sync();
        double part = 0.0;
        for (int q = 0; q < cl; ++q) {
            double x;
            asm volatile("ld.shared::cluster.f64 %0, [%1];"
                         : "=d"(x) : "r"(in_block(smem_u32(&s_norm), q)));
            part += x;
        }
        sum = part;
    }
    const double norm = sqrt(sum);
    int lift = 0;
    if (norm > 0.0 && norm < p.pre.eps) lift = min(MU_MAX_LIFT, ilogb((norm + p.pre.eps) / norm));
    const double f = scalbn(p.pre.S, lift) / (norm + p.pre.eps);
    for (int i = tid; i < P * ((Q + 7) / 8); i += TN_THREADS) {
        const int r = i / ((Q + 7) / 8), c = i - r * ((Q + 7) / 8);
        const uint32_t o = (uint32_t)(c >> 3) * TN_CHUNK + tn_unit(r, c & 7);
        float4* ph = reinterpret_cast<float4*>(mem + o);
        float4* pl = reinterpret_cast<float4*>(mem + TN_X + o);
        const float4 u0 = *ph, u1 = *pl;
        float y[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = (float)((double)y[e] * f);
        *reinterpret_cast<uint4*>(ph) =
            make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
        *reinterpret_cast<uint4*>(pl) =
            make_uint4(pack2(below_half(y[0]), below_half(y[1])), pack2(below_half(y[2]), below_half(y[3])),
                       pack2(below_half(y[4]), below_half(y[5])), pack2(below_half(y[6]), below_half(y[7])));
    }

    // ---- the products
    const float S = (float)p.pre.S;
    const int quad = warp & 3, half = warp >> 2, row = quad * 32 + lane;
    const uint32_t lane_at = tmem + ((uint32_t)(quad * 32) << 16);
    uint32_t parity = 0;
    bool ok = true;
    for (int i = 0; i < 3 * p.steps; ++i) {
        const int step = i / 3, mode = i - step * 3;   // gram, square, update
        const bool update = mode == MU_UPDATE, last = i == 3 * p.steps - 1;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncthreads();
        if (tid == 0 && ok && !p.stall) {
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const int N = ((update ? Q : P) + 15) / 16 * 16, K = mode == MU_GRAM ? Q : P;
            const uint32_t idesc = (1u << 4) | ((uint32_t)update << 16) | ((uint32_t)(N / 8) << 17) |
                                   ((TN_ROWS / 16) << 24);
            const uint32_t left = mode == MU_GRAM ? x_at : a_at, left_lo = mode == MU_GRAM ? TN_X : TN_A;
            const uint32_t right = mode == MU_SQUARE ? a_at : x_at;
            const uint32_t right_lo = mode == MU_SQUARE ? TN_A : TN_X;
            for (int k = 0; k * 16 < K; ++k) {
                const uint32_t along = (uint32_t)(k >> 2) * TN_CHUNK + (k & 3) * 32;
                const uint32_t la = left + along, ra = right + (update ? (uint32_t)k * 2048 : along);
                const uint64_t lh = smem_desc(la, false), ll = smem_desc(la + left_lo, false);
                const uint64_t rh = smem_desc(ra, update, TN_CHUNK);
                const uint64_t rl = smem_desc(ra + right_lo, update, TN_CHUNK);
                mma_f16_1(tmem, lh, rh, idesc, k > 0);
                mma_f16_1(tmem + 256, lh, rl, idesc, k > 0);
                mma_f16_1(tmem + 256, ll, rh, idesc, true);
            }
            mma_commit1(smem_u32(&s_done));
        }
        // (once a wait has given up there are no more products and the next waits give up
        // at once; the block goes on, since the others of its cluster wait for it and read
        // its memory)
        const bool done = mbar_wait(smem_u32(&s_done), parity, &s_gave_up, status);
        ok = __syncthreads_and(done) && ok;
        parity ^= 1;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");

        const float* coef = p.coef + 3 * step;
        float alpha, beta = 0.0f;
        const int k = max(0, lift - p.drop[step]), next = max(0, lift - p.drop[step + 1]);
        if (mode == MU_GRAM) {
            alpha = MU_SA / (S * S) * exp2f((float)(-2 * k));
        } else if (mode == MU_SQUARE) {
            alpha = coef[2] / MU_SA;
            beta = coef[1];
        } else {
            const float by = last ? p.scale / S * exp2f((float)-k) : exp2f((float)(next - k));
            alpha = by / MU_SA;
            beta = by * coef[0];
        }
        if (!update) alpha *= 1.0f + MU_LOW * (float)(((mode == MU_GRAM ? Q : P) + 15) / 16);
        const bool exchange = mode == MU_GRAM && cl > 1;
        const int chunks = ((update ? Q : P) + 63) / 64;
        uint8_t* buf = mem + (update ? 0 : 2 * TN_X);
        const uint32_t lo_at = update ? TN_X : TN_A;
        for (int ch = half; ch < chunks; ch += 2) {
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
                float v[32], w[32];
                tmem_load32(lane_at + ch * 64 + c, reinterpret_cast<uint32_t*>(v));
                tmem_load32(lane_at + 256 + ch * 64 + c, reinterpret_cast<uint32_t*>(w));
                tmem_wait();
                uint8_t* at = buf + ch * TN_CHUNK;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint4* ph = reinterpret_cast<uint4*>(at + tn_unit(row, c / 8 + u));
                    uint4* pl = reinterpret_cast<uint4*>(at + lo_at + tn_unit(row, c / 8 + u));
                    float y[8];
                    if (mode == MU_GRAM) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = alpha * of_pair(v[u * 8 + e], w[u * 8 + e]);
                    } else {
                        const uint4 h = *ph, l = *pl;
                        const __half* hh = reinterpret_cast<const __half*>(&h);
                        const __half* ll = reinterpret_cast<const __half*>(&l);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            y[e] = fmaf(alpha, of_pair(v[u * 8 + e], w[u * 8 + e]),
                                        beta * of_pair(__half2float(hh[e]), __half2float(ll[e])));
                    }
                    if (last || exchange) {
                        // fp32 in place: a 16-byte unit of hi and of lo are 8 values
                        *ph = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]),
                                         __float_as_uint(y[2]), __float_as_uint(y[3]));
                        *pl = make_uint4(__float_as_uint(y[4]), __float_as_uint(y[5]),
                                         __float_as_uint(y[6]), __float_as_uint(y[7]));
                    } else {
                        *ph = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]),
                                         pack2(y[6], y[7]));
                        *pl = make_uint4(pack2(below_half(y[0]), below_half(y[1])),
                                         pack2(below_half(y[2]), below_half(y[3])),
                                         pack2(below_half(y[4]), below_half(y[5])),
                                         pack2(below_half(y[6]), below_half(y[7])));
                    }
                }
            }
        }
        if (exchange) {
            cluster_sync();
            const int rows = (P + cl - 1) / cl, groups = (P + 7) / 8;
            const int r0 = rank * rows, mine = max(0, min(P - r0, rows)) * groups;
            uint4 h[TN_GROUPS], l[TN_GROUPS];
#pragma unroll
            for (int it = 0; it < TN_GROUPS; ++it) {
                const int g = it * TN_THREADS + tid;
                if (g >= mine) continue;
                const int r = r0 + g / groups, c = g % groups;
                const uint32_t at = a_at + (uint32_t)(c >> 3) * TN_CHUNK + tn_unit(r, c & 7);
                float y[8] = {};
#pragma unroll 4
                for (int q = 0; q < cl; ++q) {
                    const uint32_t from = in_block(at, q);
                    float x[8];
                    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(from));
                    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                                 : "r"(from + TN_A));
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] += x[e];
                }
                h[it] = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]),
                                   pack2(y[6], y[7]));
                l[it] = make_uint4(pack2(below_half(y[0]), below_half(y[1])),
                                   pack2(below_half(y[2]), below_half(y[3])),
                                   pack2(below_half(y[4]), below_half(y[5])),
                                   pack2(below_half(y[6]), below_half(y[7])));
            }
            cluster_sync();                                // every sum is read
#pragma unroll
            for (int it = 0; it < TN_GROUPS; ++it) {
                const int g = it * TN_THREADS + tid;
                if (g >= mine) continue;
                const int r = r0 + g / groups, c = g % groups;
                const uint32_t at = a_at + (uint32_t)(c >> 3) * TN_CHUNK + tn_unit(r, c & 7);
                for (int q = 0; q < cl; ++q) {
                    const uint32_t to = in_block(at, q);
                    asm volatile("st.shared::cluster.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to),
                                 "r"(h[it].x), "r"(h[it].y), "r"(h[it].z), "r"(h[it].w)
                                 : "memory");
                    asm volatile("st.shared::cluster.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to + TN_A),
                                 "r"(l[it].x), "r"(l[it].y), "r"(l[it].z), "r"(l[it].w)
                                 : "memory");
                }
            }
            cluster_sync();
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (ok) {
        for (int i = tid; i < total; i += TN_THREADS) {
            const int r = i / n, c = i - r * n;
            const float y = *reinterpret_cast<const float*>(mem + (tall ? tn_f32(c, r) : tn_f32(r, c)));
            const int64_t to = b * p.stride_out + (tall ? q0 + r : r) * p.ld_out + (tall ? c : q0 + c);
            if (p.out_type == 0) static_cast<float*>(p.out)[to] = y;
            else if (p.out_type == 1) static_cast<__nv_bfloat16*>(p.out)[to] = __float2bfloat16_rn(y);
            else static_cast<__half*>(p.out)[to] = __float2half_rn(y);
        }
    } else {
        // products may still be running: let them end before their accumulators are freed
        volatile int never = 0;
        if (tid == 0) {
            mma_commit1(smem_u32(&s_drain));
            mbar_wait(smem_u32(&s_drain), 0, &never, status);
        }
        __syncthreads();
    }
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

}  // namespace tke
