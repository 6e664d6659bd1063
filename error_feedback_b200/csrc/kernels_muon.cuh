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
// Numbers: X is held as a pair of fp16 values, hi + lo (22 bits), times a power of
// two that keeps typical entries near 1; A and B likewise times MU_SA.  A step
// multiplies small singular values by a (3.4 five times in a row), so a
// rounding of X itself would be amplified 485 times: the term a X is taken
// from hi + lo.  For 16-bit outputs the products read hi alone (11 bits; bf16
// operands would leave an error six times a bf16 output's own rounding); for
// fp32 outputs each product is hi hi + hi lo + lo hi.  All sums are fp32.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "elements.cuh"

namespace tke {

constexpr float MU_SA = 2048.0f;           // scale of A and B
constexpr float MU_REACH = 4.0f;           // |p(x)| the coefficients may reach (host check)
constexpr int MU_MAX_LIFT = 60;
constexpr uint64_t MU_WAIT_NS = 2000000000ull;

// ------------------------------------------------------- momentum and norm

constexpr int MN_THREADS = 256;
constexpr int MN_MAX_PARTS = 512;          // partial sums of one matrix

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
// elements per thread at a time; bound by the bytes of g and m.
template <typename TG>
__global__ void __launch_bounds__(MN_THREADS) muon_norm_kernel(const MuonPreParams p) {
    __shared__ double s_red[33];
    pdl_launch();
    pdl_wait();
    const int64_t b = blockIdx.y;
    if (blockIdx.x == 0 && b == 0 && threadIdx.x == 0) {
        p.ctrl->path_small = 0;
        p.ctrl->status = 0;
    }
    double sum = 0.0;
    for (int64_t i = (int64_t)blockIdx.x * MN_THREADS + threadIdx.x; i < p.groups;
         i += (int64_t)gridDim.x * MN_THREADS) {
        const int64_t r = i / p.row_groups;
        float u[8];
        muon_u8<TG, true>(p, b, r, (i - r * p.row_groups) * 8, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fma((double)u[j], (double)u[j], sum);
    }
    const double tot = block_sum(sum, s_red);
    if (threadIdx.x == 0) p.part[b * p.parts + blockIdx.x] = tot;
}

// X = u * S * 2^lift / (||u|| + eps) as hi + lo.  lift is 0 unless eps holds
// the norm of X below 1: then it brings the entries to where fp16 has all its
// bits, and the products take it back as fast as X can grow.
template <typename TG>
__global__ void __launch_bounds__(MN_THREADS) muon_scale_kernel(const MuonPreParams p) {
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
    for (int64_t i = (int64_t)blockIdx.x * MN_THREADS + threadIdx.x; i < p.groups;
         i += (int64_t)gridDim.x * MN_THREADS) {
        const int64_t r = i / p.row_groups, c = (i - r * p.row_groups) * 8;
        float u[8], l[8];
        muon_u8<TG, false>(p, b, r, c, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u[j] = (float)((double)u[j] * f);
            l[j] = u[j] - __half2float(__float2half_rn(u[j]));
        }
        // (rows of X are padded to 64 columns)
        store8(p.hi + b * p.stride_x + r * p.ldx + c, u);
        store8(p.lo + b * p.stride_x + r * p.ldx + c, l);
    }
}

// ------------------------------------------------------- tensor-core products

// Two blocks (a cluster on two SMs) hold one 256 x 256 tile: each loads its 128
// rows of the left operand and its 128 columns of the right one, and one
// thread of the first issues products that both tensor cores run.
constexpr int GM_EPI_WARPS = 8;
constexpr int GM_THREADS = 128 + 32 * GM_EPI_WARPS;    // load, product, 2 idle, epilogue
constexpr int GM_TILE = 256, GM_ROWS = 128, GM_K = 64;
constexpr int GM_BOX = 64 * 64 * 2;                    // bytes of one 64 x 64 fp16 box
constexpr int GM_OP = GM_ROWS * GM_K * 2;              // one operand of one block and stage
constexpr int GM_RING = 6 * 2 * GM_OP;                 // 196,608 bytes of stages
constexpr int GM_SMEM = GM_RING + 1024;                // + alignment

enum { MU_GRAM = 0, MU_SQUARE = 1, MU_UPDATE = 2, MU_LAST = 3 };

struct GemmParams {
    CUtensorMap a[2], b[2];        // hi, lo of both operands
    int32_t M, N, K, batch, tiles_m, tiles_n, tiles;   // tiles: of one matrix
    int32_t a_mn, b_mn;            // operand's M (N) dimension is the contiguous one
    int32_t n_fast;                // neighbouring tiles differ in N
    int32_t mode, out_type;
    float alpha, beta;             // value = alpha * sum + beta * (src_hi + src_lo)
    const int32_t* lift;           // [batch]
    int32_t drop, drop_next;       // what earlier steps have taken off lift, and this one
    const __half* src[2];          // elementwise operand (square: A, update: X)
    __half* dst[2];
    int64_t ld, stride;            // of src and dst
    void* out;                     // last update: the user's matrix
    int64_t ld_out, stride_out;
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
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
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

// One 64 x 64 box into this block's shared memory; the bytes are counted on a
// barrier of either block of the pair.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                        uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
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
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn) {
    const uint64_t lead = mn ? (uint64_t)(GM_BOX >> 4) : 1ull;
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (lead << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void mma_f16(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
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

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}

struct TileAt {
    int b, m, n;       // batch, this block's first row, the tile's first column
};

// The t-th tile of this call, rank: 0 or 1 in the pair.  Symmetric outputs:
// tiles (i, j) with i >= j, row by row.
__device__ __forceinline__ TileAt tile_at(const GemmParams& p, int t, int rank) {
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
    r.m = i * GM_TILE + rank * GM_ROWS;
    r.n = j * GM_TILE;
    return r;
}

// Sixteen fp16 values, 32 bytes: one whole memory sector for each lane.
__device__ __forceinline__ void load_half16(const __half* p, float* v) {
    uint32_t r[8];
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[j]));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
}
__device__ __forceinline__ void store32b(void* p, const uint32_t* r) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float below_half(float x) {     // what fp16 leaves of x
    return x - __half2float(__float2half_rn(x));
}

template <typename TO>
__device__ __forceinline__ void store_out(const GemmParams& p, int64_t b, int64_t row, int64_t c0,
                                          const float* v) {
    TO* dst = static_cast<TO*>(p.out) + b * p.stride_out + row * p.ld_out + c0;
    if (c0 + 32 <= p.N && (uintptr_t)dst % 32 == 0) {
        constexpr int E = 32 / (int)sizeof(TO);
#pragma unroll
        for (int j = 0; j < 32; j += E) {
            uint32_t r[8];
#pragma unroll
            for (int e = 0; e < E; ++e) reinterpret_cast<TO*>(r)[e] = from_f32<TO>(v[j + e]);
            store32b(dst + j, r);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (c0 + j < p.N) dst[j] = from_f32<TO>(v[j]);
    }
}

// 32 columns of one row of fp16 pairs (hi, and lo where wanted).
__device__ __forceinline__ void store_pair(const GemmParams& p, int64_t o, const float* v,
                                           bool want_lo) {
#pragma unroll
    for (int j = 0; j < 32; j += 16) {
        uint32_t r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = pack2(v[j + 2 * e], v[j + 2 * e + 1]);
        store32b(p.dst[0] + o + j, r);
        if (want_lo) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[e] = pack2(below_half(v[j + 2 * e]), below_half(v[j + 2 * e + 1]));
            store32b(p.dst[1] + o + j, r);
        }
    }
}

// What a tile's values are multiplied by besides alpha and beta: X is held
// times 2^k, k = max(0, lift - drop), and the next X times 2^max(0, lift -
// drop_next).
__device__ __forceinline__ void lift_factors(const GemmParams& p, int b, float* sum, float* src) {
    *sum = *src = 1.0f;
    const int lift = p.lift[b];
    if (lift == 0) return;
    const int k = max(0, lift - p.drop), next = max(0, lift - p.drop_next);
    if (p.mode == MU_GRAM) *sum = exp2f((float)(-2 * k));
    else if (p.mode == MU_UPDATE) *sum = *src = exp2f((float)(next - k));
    else if (p.mode == MU_LAST) *sum = *src = exp2f((float)-k);
}

// One row's 32 columns of a finished tile; v: the sums.
template <bool EXACT>
__device__ __forceinline__ void epilogue32(const GemmParams& p, const TileAt& at, float alpha,
                                           float beta, int64_t row, int64_t c0, float* v) {
    const bool live = row < p.M && c0 < p.N;
    const int64_t o = at.b * p.stride + row * p.ld + c0;
    // (rows of src and dst are padded to 64 columns: 32 at a time stay inside)
    if (p.mode == MU_GRAM) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= alpha;
    } else if (live) {
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
            float h[16], l[16];
            load_half16(p.src[0] + o + j, h);
            if (EXACT || p.mode >= MU_UPDATE) {
                load_half16(p.src[1] + o + j, l);
#pragma unroll
                for (int e = 0; e < 16; ++e) h[e] += l[e];
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) v[j + e] = fmaf(alpha, v[j + e], beta * h[e]);
        }
    }
    if (p.mode == MU_LAST) {
        if (!live) return;
        if (p.out_type == 0) store_out<float>(p, at.b, row, c0, v);
        else if (p.out_type == 1) store_out<__nv_bfloat16>(p, at.b, row, c0, v);
        else store_out<__half>(p, at.b, row, c0, v);
        return;
    }
    if (p.mode == MU_UPDATE) {
        if (live) store_pair(p, o, v, true);
        return;
    }
    // Symmetric: columns up to the row, and their mirror image (a warp's 32
    // rows are 32 consecutive columns there).  Each entry is written by one
    // thread only.
    const int64_t row0 = row - lane_id();
    if (c0 > row0 + 31) return;
    const bool below = c0 + 31 <= row0;
    if (live && below) store_pair(p, o, v, EXACT);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const int64_t c = c0 + j;
        if (live && c <= row) {
            const __half h = __float2half_rn(v[j]);
            const __half l = __float2half_rn(v[j] - __half2float(h));
            if (!below) {
                p.dst[0][o + j] = h;
                if (EXACT) p.dst[1][o + j] = l;
            }
            if (c < row) {
                const int64_t om = at.b * p.stride + c * p.ld + row;
                p.dst[0][om] = h;
                if (EXACT) p.dst[1][om] = l;
            }
        }
    }
}

// Persistent pairs: pair x takes tiles x, x + pairs, ...  In each block one
// thread loads boxes by TMA into a ring of stages; in the first one thread
// issues the products into one of two TMEM accumulators (2 x 256 columns)
// while eight warps of each block drain the other.
//
// The tensor core's own fp32 accumulation truncates: a sum of K / 16 products
// of one sign comes out up to K / 16 half-steps low.  With fp32 output the
// accumulator is therefore handed over after every 64 of K, the small
// products (hi lo, lo hi) before the large, and added up in registers with
// rounding to nearest.
template <bool EXACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GM_THREADS, 1)
    muon_gemm_kernel(const __grid_constant__ GemmParams p) {
    constexpr int PARTS = EXACT ? 2 : 1;
    constexpr int STAGE = PARTS * 2 * GM_OP;           // one block's bytes of a stage
    constexpr int STAGES = GM_RING / STAGE;
    constexpr int HALF = GM_TILE / 2;                  // columns of one epilogue warp
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t s_full[STAGES], s_empty[STAGES], s_done[2], s_free[2], s_drain;
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
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&s_done[s]), 1);
            mbar_init(smem_u32(&s_free[s]), 2 * GM_EPI_WARPS);
        }
        mbar_init(smem_u32(&s_drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
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
    const int total = p.tiles * p.batch, kblocks = (p.K + GM_K - 1) / GM_K;
    pdl_launch();
    pdl_wait();
    if (EXACT) {
        // 384 threads start with 168 registers each; the 128 running sums of
        // an epilogue thread need more: 72 + 216 + 216 = 3 x 168
        if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    }

    if (warp == 0 && lane == 0) {
        // ---- loads (of what earlier kernels wrote with ordinary stores)
        asm volatile("fence.proxy.async;" ::: "memory");
        int stage = 0;
        uint32_t phase = 0, issued = 0;
        bool ok = true;
        for (int t = pair; t < total && ok; t += pairs) {
            const TileAt at = tile_at(p, t, rank);
            const int n0 = at.n + rank * GM_ROWS;
            for (int kb = 0; kb < kblocks; ++kb) {
                if (!(ok = mbar_wait(smem_u32(&s_empty[stage]), phase ^ 1, &s_gave_up, status)))
                    break;
                const uint32_t bar = in_block(smem_u32(&s_full[stage]), 0);
                if (rank == 0) mbar_expect(smem_u32(&s_full[stage]), 2 * STAGE);
                uint32_t dst = base + stage * STAGE;
                const int k = kb * GM_K;
#pragma unroll
                for (int q = 0; q < PARTS; ++q) {
#pragma unroll
                    for (int i = 0; i < GM_ROWS / 64; ++i, dst += GM_BOX) {
                        if (p.a_mn) tma_box(dst, &p.a[q], at.m + i * 64, k, at.b, bar);
                        else tma_box(dst, &p.a[q], k, at.m + i * 64, at.b, bar);
                    }
                }
#pragma unroll
                for (int q = 0; q < PARTS; ++q) {
#pragma unroll
                    for (int i = 0; i < GM_ROWS / 64; ++i, dst += GM_BOX) {
                        if (p.b_mn) tma_box(dst, &p.b[q], n0 + i * 64, k, at.b, bar);
                        else tma_box(dst, &p.b[q], k, n0 + i * 64, at.b, bar);
                    }
                }
                ++issued;
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
        const uint32_t idesc = (1u << 4) | ((uint32_t)p.a_mn << 15) | ((uint32_t)p.b_mn << 16) |
                               ((GM_TILE / 8) << 17) | ((GM_TILE / 16) << 24);
        const uint32_t a_step = p.a_mn ? 2048 : 32, b_step = p.b_mn ? 2048 : 32;
        int stage = 0, slot = 0;
        uint32_t phase = 0, slot_phase = 0;
        bool ok = true;
        for (int t = pair; t < total && ok; t += pairs) {
            for (int kb = 0; kb < kblocks; ++kb) {
                const bool begin = EXACT || kb == 0, end = EXACT || kb == kblocks - 1;
                if (begin) {
                    if (!(ok = mbar_wait(smem_u32(&s_free[slot]), slot_phase ^ 1, &s_gave_up,
                                         status)))
                        break;
                }
                if (!(ok = mbar_wait(smem_u32(&s_full[stage]), phase, &s_gave_up, status))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t d = tmem + slot * GM_TILE;
                const uint32_t a0 = base + stage * STAGE, b0 = a0 + PARTS * GM_OP;
                if (EXACT) {
#pragma unroll
                    for (int k = 0; k < GM_K / 16; ++k) {
                        mma_f16(d, smem_desc(a0 + k * a_step, p.a_mn),
                                smem_desc(b0 + GM_OP + k * b_step, p.b_mn), idesc, k > 0);
                        mma_f16(d, smem_desc(a0 + GM_OP + k * a_step, p.a_mn),
                                smem_desc(b0 + k * b_step, p.b_mn), idesc, true);
                    }
                }
#pragma unroll
                for (int k = 0; k < GM_K / 16; ++k)
                    mma_f16(d, smem_desc(a0 + k * a_step, p.a_mn),
                            smem_desc(b0 + k * b_step, p.b_mn), idesc, EXACT || kb > 0 || k > 0);
                mma_commit(smem_u32(&s_empty[stage]));
                if (end) {
                    mma_commit(smem_u32(&s_done[slot]));
                    if (++slot == 2) {
                        slot = 0;
                        slot_phase ^= 1;
                    }
                }
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp >= 4) {
        // ---- epilogue: warp w reads TMEM lanes 32 (w mod 4) .., half of the columns
        const int quad = warp & 3, col = warp < 8 ? 0 : HALF;
        const uint32_t src = tmem + col + ((uint32_t)(quad * 32) << 16);
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
            const TileAt at = tile_at(p, t, rank);
            const int64_t row = at.m + quad * 32 + lane;
            float fs, fx;
            lift_factors(p, at.b, &fs, &fx);
            const float alpha = p.alpha * fs, beta = p.beta * fx;
            if (EXACT) {
                float sum[HALF];
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!wait_done()) break;
#pragma unroll
                    for (int c = 0; c < HALF; c += 32) {
                        float v[32];
                        tmem_ld32(src + slot * GM_TILE + c, reinterpret_cast<uint32_t*>(v));
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[c + j] = kb == 0 ? v[j] : sum[c + j] + v[j];
                    }
                    drained();
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < HALF; c += 32)
                    epilogue32<EXACT>(p, at, alpha, beta, row, at.n + col + c, sum + c);
            } else {
                if (!wait_done()) break;
                for (int c = 0; c < HALF; c += 32) {
                    float v[32];
                    tmem_ld32(src + slot * GM_TILE + c, reinterpret_cast<uint32_t*>(v));
                    epilogue32<EXACT>(p, at, alpha, beta, row, at.n + col + c, v);
                }
                drained();
            }
        }
    }
    __syncthreads();
    // when a wait gave up, products may still be running: let them end before
    // their accumulators are freed
    if (s_gave_up && threadIdx.x == 32 && rank == 0) {
        volatile int never = 0;
        mma_commit(smem_u32(&s_drain));
        mbar_wait(smem_u32(&s_drain), 0, &never, status);
    }
    __syncthreads();
    cluster_sync();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

}  // namespace tke
