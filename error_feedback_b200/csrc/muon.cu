// Host side of muon_update (include/topk_ef.h): argument checks, workspace
// layout, launch sequence.
//
//   a small matrix: muon_tiny_kernel alone; else
//   muon_norm_kernel -> muon_scale_kernel -> steps times: gram, square and update
//   (the last update writes the caller's matrix), each by muon_gemm_kernel (many
//   tiles) or muon_split_kernel (few; once for every part of a long K)
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "topk_ef.h"
#include "common.cuh"
#include "host.cuh"
#include "kernels_muon.cuh"

using namespace tke;

namespace {

constexpr int64_t MU_MAX_SIDE = (int64_t)1 << 20;
constexpr int32_t MU_MAX_BATCH = 65535;
constexpr int32_t MU_MAX_STEPS = 64;
// 256 x 256 tiles of a product from which pairs of SMs take them, rather than
// clusters 128 x 128 tiles with K divided.  Below, the pairs that are left idle
// cost more than the clusters' exchange.  Five steps, 11 bits, pairs from 6, 12 or
// 25 tiles on: 800 x 3,000 (gram of 10 tiles) 247, 202 or 202 us, 768 x 1,024
// (update of 12) 166, 154 or 157, 1,500 x 1,500 (gram of 21) 241, 241 or 270.  22
// bits, from 25, 37 or 70: 2,048 x 2,048 (gram of 36) 633, 585 or 638, 1,100 x 2,500
// (update of 50) 384, 384 or 412, 2,304 x 2,304 (gram of 45) 945, 946 or 1,147.
// LONG: of 22 bits, where K is too long for one launch of the clusters (see
// SP_MAX_SUM); from 11 or 20 tiles on: 1,280 x 8,000 (gram of 15) 1,126 or 850 us, from
// 20 or 22: 1,500 x 4,000 (gram of 21) 806 or 842.
constexpr int64_t MU_PAIR_TILES_11 = 12, MU_PAIR_TILES_22 = 37, MU_PAIR_TILES_LONG = 20;

struct MuLayout {
    int64_t p, ldx, ldp, stride_x, stride_p, groups, parts;
    size_t ctrl, part, lift, x[2][2], a[2], b[2], total;
};

MuLayout muon_layout(int32_t B, int64_t m, int64_t n, bool exact) {
    MuLayout L;
    L.p = std::min(m, n);
    L.ldx = ceil_div64(n, 64) * 64;
    L.ldp = ceil_div64(L.p, 64) * 64;
    L.stride_x = m * L.ldx;
    L.stride_p = L.p * L.ldp;
    L.groups = m * ceil_div64(n, 8);
    L.parts = std::max<int64_t>(
        1, std::min<int64_t>(MN_MAX_PARTS, ceil_div64(L.groups, 2 * MN_THREADS)));
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes);
        return at;
    };
    L.ctrl = take(sizeof(Ctrl));
    L.part = take((size_t)B * L.parts * sizeof(double));
    L.lift = take((size_t)B * sizeof(int32_t));
    for (int i = 0; i < 2; ++i)
        for (int h = 0; h < 2; ++h) L.x[i][h] = take((size_t)B * L.stride_x * 2);
    for (int h = 0; h < 2; ++h) {
        const bool used = h == 0 || exact;
        L.a[h] = take(used ? (size_t)B * L.stride_p * 2 : 0);
        L.b[h] = take(used ? (size_t)B * L.stride_p * 2 : 0);
    }
    L.total = o;
    return L;
}

// Three products for 22 bits, or one for 11, which only bf16 output has: 300 x 300
// comes out 1.64e-3 off before the output's rounding, which is 1.65e-3 for bf16 but
// 2.1e-4 for fp16.  Not where the short side fits one tile: there are too few terms
// for the roundings to average out (70 x 6,000 in bf16: 2.9e-3 off in all), and the
// products wait for one another more than for the tensor cores.
bool muon_exact(int64_t m, int64_t n, int32_t out_type) {
    return out_type != TOPK_EF_BF16 || std::min(m, n) <= SP_TILE;
}

bool muon_sizes_ok(int32_t B, int64_t m, int64_t n) {
    return B >= 0 && B <= MU_MAX_BATCH && m >= 0 && m <= MU_MAX_SIDE && n >= 0 && n <= MU_MAX_SIDE;
}

// Largest |x (a + b s + c s^2)| (s = x^2), |b s + c s^2| and |a + b s + c s^2|
// for 0 <= x <= reach.
void polynomial_reach(const float* k, double reach, double* most_p, double* most_q,
                      double* growth) {
    const double a = k[0], b = k[1], c = k[2];
    *most_p = *most_q = 0.0;
    *growth = std::fabs(a);
    auto at = [&](double s) {
        if (!(s >= 0.0 && s <= reach * reach)) return;
        *growth = std::max(*growth, std::fabs(a + s * (b + s * c)));
        *most_p = std::max(*most_p, std::fabs(std::sqrt(s) * (a + s * (b + s * c))));
        *most_q = std::max(*most_q, std::fabs(s * (b + s * c)));
    };
    at(reach * reach);
    // p' = a + 3 b s + 5 c s^2,  q' = b + 2 c s
    if (c != 0.0) {
        at(-b / (2.0 * c));
        const double d = 9.0 * b * b - 20.0 * a * c;
        if (d >= 0.0) {
            at((-3.0 * b + std::sqrt(d)) / (10.0 * c));
            at((-3.0 * b - std::sqrt(d)) / (10.0 * c));
        }
    } else if (b != 0.0) {
        at(-a / (3.0 * b));
    }
}

// The singular values start at 1 at most; X, A and B are held in fp16 under
// fixed scales, so the polynomials must not take them out of its range.
// drop[i]: bits that X can have grown by before step i.
bool coefficients_ok(const float* coef, int32_t steps, int32_t* drop) {
    double reach = 1.0;
    drop[0] = 0;
    for (int i = 0; i < steps; ++i) {
        const float* k = coef + 3 * i;
        if (!std::isfinite(k[0]) || !std::isfinite(k[1]) || !std::isfinite(k[2])) return false;
        double mp, mq, growth;
        polynomial_reach(k, reach, &mp, &mq, &growth);
        if (mp > MU_REACH || mq > MU_REACH * MU_REACH) return false;
        reach = mp;
        drop[i + 1] = drop[i] + (growth > 1.0 ? (int32_t)std::ceil(std::log2(growth)) : 0);
    }
    return true;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn(cudaError_t* e) {
    static std::atomic<void*> fn{nullptr};
    void* f = fn.load();
    if (!f) {
        cudaDriverEntryPointQueryResult q;
        *e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                              cudaEnableDefault, &q);
        if (*e != cudaSuccess) return nullptr;
        if (!f || q != cudaDriverEntryPointSuccess) {
            *e = cudaErrorNotSupported;
            return nullptr;
        }
        fn.store(f);
    }
    return reinterpret_cast<EncodeFn>(f);
}

// Boxes of an operand in [batch][rows][cols] fp16, 128-byte swizzle: `count`
// rows x 64 columns where the columns are K, else 64 rows x `count` columns
// (see GemmParams).
struct Operand {
    __half* base[2];
    int64_t rows, cols, ld, stride;
    bool mn;                       // the rows are K
};
bool encode(EncodeFn fn, CUtensorMap* map, const Operand& o, int part, int64_t batch, int count) {
    const bool mn = o.mn;
    const cuuint64_t dims[4] = {(cuuint64_t)(mn ? 64 : o.cols), (cuuint64_t)o.rows,
                                (cuuint64_t)(mn ? ceil_div64(o.cols, 64) : 1), (cuuint64_t)batch};
    const cuuint64_t strides[3] = {(cuuint64_t)o.ld * 2, 128, (cuuint64_t)o.stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(mn ? 64 : count), (cuuint32_t)(mn ? count / 64 : 1), 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, o.base[part], dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Calls f with the pair and split kernels of a precision and mode.
template <bool EXACT, typename F>
cudaError_t with_mode(int mode, F f) {
    switch (mode) {
        case MU_GRAM: return f(muon_gemm_kernel<EXACT, MU_GRAM>, muon_split_kernel<EXACT, MU_GRAM>);
        case MU_SQUARE:
            return f(muon_gemm_kernel<EXACT, MU_SQUARE>, muon_split_kernel<EXACT, MU_SQUARE>);
        case MU_UPDATE:
            return f(muon_gemm_kernel<EXACT, MU_UPDATE>, muon_split_kernel<EXACT, MU_UPDATE>);
        default: return f(muon_gemm_kernel<EXACT, MU_LAST>, muon_split_kernel<EXACT, MU_LAST>);
    }
}
template <typename F>
cudaError_t with_kernel(bool exact, int mode, F f) {
    return exact ? with_mode<true>(mode, f) : with_mode<false>(mode, f);
}

struct MuDevice {
    int pairs;                     // block pairs of muon_gemm_kernel that run at once
    int tiny[5];                   // clusters of 1, 2, .. 16 blocks of muon_tiny_kernel
    int clusters[4];               // clusters of 1, 2, 4, 8 blocks of muon_split_kernel, one block an SM
};

// Facts of the current device; its kernels' shared memory is set the first time.
cudaError_t muon_device(MuDevice* out) {
    static std::mutex mu;
    static MuDevice known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    if (known[dev].pairs > 0) {
        *out = known[dev];
        return cudaSuccess;
    }
    const int split_smem = sp_smem(false, SP_MAX_STAGES);
    for (int exact = 0; exact < 2; ++exact)
        for (int mode = MU_GRAM; mode <= MU_LAST; ++mode) {
            e = with_kernel(exact != 0, mode, [&](auto pair, auto split) {
                const cudaError_t r = cudaFuncSetAttribute(
                    pair, cudaFuncAttributeMaxDynamicSharedMemorySize, GM_SMEM);
                return r != cudaSuccess ? r
                                        : cudaFuncSetAttribute(
                                              split, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              exact ? sp_smem(true, SP_MIN_STAGES) : split_smem);
            });
            if (e != cudaSuccess) return e;
        }
    for (int32_t t = TOPK_EF_F32; t <= TOPK_EF_F16; ++t) {
        e = with_type(t, [&](auto type) {
            const cudaError_t r =
                cudaFuncSetAttribute(muon_tiny_kernel<decltype(type)>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, TN_SMEM);
            return r != cudaSuccess
                       ? r
                       : cudaFuncSetAttribute(muon_tiny_kernel<decltype(type)>,
                                              cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        });
        if (e != cudaSuccess) return e;
    }
    MuDevice d = {};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(GM_THREADS);
    cfg.dynamicSmemBytes = GM_SMEM;
    e = cudaOccupancyMaxActiveClusters(&d.pairs, muon_gemm_kernel<false, MU_UPDATE>, &cfg);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    cfg.blockDim = dim3(SP_THREADS);
    cfg.dynamicSmemBytes = split_smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    for (int i = 0; i < 4 && e == cudaSuccess; ++i) {
        cfg.gridDim = dim3(1u << i);
        attr[0].val.clusterDim = {1u << i, 1, 1};
        e = cudaOccupancyMaxActiveClusters(&d.clusters[i], muon_split_kernel<false, MU_UPDATE>, &cfg);
    }
    cfg.blockDim = dim3(TN_THREADS);
    cfg.dynamicSmemBytes = TN_SMEM;
    for (int i = 0; i < 5 && e == cudaSuccess; ++i) {
        cfg.gridDim = dim3(1u << i);
        attr[0].val.clusterDim = {1u << i, 1, 1};
        e = cudaOccupancyMaxActiveClusters(&d.tiny[i], muon_tiny_kernel<float>, &cfg);
    }
    if (e == cudaSuccess && d.pairs < 1) e = cudaErrorNotSupported;
    if (e == cudaSuccess) *out = known[dev] = d;
    return e;
}

}  // namespace

extern "C" {

size_t muon_workspace_bytes(int32_t B, int64_t rows, int64_t cols, int32_t out_type) {
    if (!muon_sizes_ok(B, rows, cols) || !type_size(out_type)) return 0;
    return muon_layout(B, rows, cols, muon_exact(rows, cols, out_type)).total;
}

int muon_update(const void* grad, int32_t grad_type, int64_t ld_grad, int64_t stride_grad,
                float* momentum, int32_t B, int64_t rows, int64_t cols, float mu, int32_t nesterov,
                float eps, const float* coef, int32_t steps, float scale, void* out,
                int32_t out_type, int64_t ld_out, int64_t stride_out, void* ws, size_t ws_bytes,
                void* stream) {
    const size_t need = muon_workspace_bytes(B, rows, cols, out_type);
    const size_t sg = type_size(grad_type), so = type_size(out_type);
    if (need == 0 || !ws || !aligned(ws, ALIGN) || !sg) return TOPK_EF_ERR_INVALID_ARG;
    if (steps < 1 || steps > MU_MAX_STEPS || !coef || !(eps >= 0.0f))
        return TOPK_EF_ERR_INVALID_ARG;
    int32_t drop[MU_MAX_STEPS + 1];
    if (!coefficients_ok(coef, steps, drop)) return TOPK_EF_ERR_INVALID_ARG;
    if (ld_grad < cols || ld_out < cols || (B > 1 && rows > 0 && cols > 0 &&
        (stride_grad < (rows - 1) * ld_grad + cols || stride_out < (rows - 1) * ld_out + cols)))
        return TOPK_EF_ERR_INVALID_ARG;
    const bool empty = B == 0 || rows == 0 || cols == 0;
    if (!empty && (!grad || !out || !aligned(grad, sg) || !aligned(out, so) ||
                   !aligned(momentum, 4)))
        return TOPK_EF_ERR_INVALID_ARG;
    // (a small matrix's block writes its output while others still read theirs)
    if (!empty && (momentum == grad || momentum == out ||
                   (out == grad && B > 1 && (out_type != grad_type || ld_out != ld_grad ||
                                             stride_out != stride_grad))))
        return TOPK_EF_ERR_INVALID_ARG;
    if (!empty && ceil_div64(rows, SP_TILE) * ceil_div64(cols, SP_TILE) * B > MAX_N / 8)
        return TOPK_EF_ERR_INVALID_ARG;
    if (ws_bytes < need) return TOPK_EF_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (empty) {
        e = cudaMemsetAsync(ws, 0, sizeof(Ctrl), st);
        return e == cudaSuccess ? TOPK_EF_OK : cuda_fail(e);
    }
    const bool exact = muon_exact(rows, cols, out_type), tall = rows > cols;
    const MuLayout L = muon_layout(B, rows, cols, exact);
    char* w = static_cast<char*>(ws);
    __half *x[2][2], *am[2], *bm[2];
    for (int h = 0; h < 2; ++h) {
        for (int i = 0; i < 2; ++i) x[i][h] = reinterpret_cast<__half*>(w + L.x[i][h]);
        am[h] = reinterpret_cast<__half*>(w + L.a[h]);
        bm[h] = reinterpret_cast<__half*>(w + L.b[h]);
    }
    // typical entries of X near 1, the largest below 2^15
    const double S = std::exp2(std::min(13.0, std::ceil(0.5 * std::log2((double)rows * cols))));

    MuDevice dev;
    if ((e = muon_device(&dev)) != cudaSuccess) return cuda_fail(e);
    const int32_t stall = (test_flags() & 4) != 0;
    MuonPreParams pp = {};
    pp.grad = grad;
    pp.momentum = momentum;
    pp.part = reinterpret_cast<double*>(w + L.part);
    pp.hi = x[0][0];
    pp.lo = x[0][1];
    pp.lift = reinterpret_cast<int32_t*>(w + L.lift);
    pp.ctrl = reinterpret_cast<Ctrl*>(w + L.ctrl);
    pp.rows = rows;
    pp.cols = cols;
    pp.ldx = L.ldx;
    pp.ld_g = ld_grad;
    pp.stride_g = stride_grad;
    pp.stride_x = L.stride_x;
    pp.parts = L.parts;
    pp.row_groups = ceil_div64(cols, 8);
    pp.groups = L.groups;
    pp.flat = ld_grad == cols && cols % 64 == 0 && aligned(grad, 16) &&
              stride_grad * (int64_t)sg % 16 == 0 && aligned(momentum, 16);
    pp.mu = mu;
    pp.nesterov = nesterov;
    pp.eps = eps;
    pp.S = S;
    // (clusters of 16 run only where so many SMs lie together)
    const int64_t longest = std::max(rows, cols);
    if (std::min(rows, cols) <= TN_ROWS &&
        longest <= (dev.tiny[4] > 0 ? TN_MAX_BLOCKS : TN_MAX_BLOCKS / 2) * TN_COLS) {
        // as few blocks as hold it, or more down to 64 columns each while all matrices
        // still run at once (64 x 600: 68 us with 4 blocks, 54 with 16; twenty of 100 x
        // 600 88 with 4, 220 with 16)
        int lg = 0;
        while ((TN_COLS << lg) < longest) ++lg;
        while (lg < 4 && (64 << lg) < longest && B <= dev.tiny[lg + 1]) ++lg;
        const unsigned blocks = 1u << lg;
        TinyParams tp = {};
        tp.pre = pp;
        std::copy(coef, coef + 3 * steps, tp.coef);
        for (int i = 0; i <= steps; ++i) tp.drop[i] = (int8_t)std::min(drop[i], 127);
        tp.steps = steps;
        tp.out_type = out_type;
        tp.stall = stall;
        tp.scale = scale;
        tp.out = out;
        tp.ld_out = ld_out;
        tp.stride_out = stride_out;
        trace_before(st, "muon_tiny_kernel");
        e = with_type(grad_type, [&](auto t) {
            return launch_clusters(muon_tiny_kernel<decltype(t)>, (unsigned)B * blocks, blocks,
                                   TN_THREADS, TN_SMEM, st, tp);
        });
        trace_after(st);
        return e == cudaSuccess ? TOPK_EF_OK : cuda_fail(e);
    }
    EncodeFn fn = encode_fn(&e);
    if (!fn) return cuda_fail(e);
    const int pairs = dev.pairs;
    const int32_t P = (int32_t)L.p, Q = (int32_t)std::max(rows, cols);
    // operand maps, made once for each use: gram, square and update of both X
    struct Maps {
        CUtensorMap a[2], b[2], b_half[2];
    };
    Maps maps[5];
    const int parts = exact ? 2 : 1;
    auto fill = [&](Maps& to, const Operand& a, const Operand& b) {
        bool ok = true;
        for (int h = 0; h < parts; ++h)
            ok = ok && encode(fn, &to.a[h], a, h, B, 128) && encode(fn, &to.b[h], b, h, B, 128) &&
                 encode(fn, &to.b_half[h], b, h, B, 64);
        return ok;
    };
    bool ok = true;
    for (int i = 0; i < 2; ++i) {
        Operand xo = {{x[i][0], x[i][1]}, rows, cols, L.ldx, L.stride_x, tall};
        const Operand bo = {{bm[0], bm[1]}, L.p, L.p, L.ldp, L.stride_p, false};
        ok = ok && fill(maps[i], xo, xo);
        xo.mn = !tall;
        ok = ok && (tall ? fill(maps[3 + i], xo, bo) : fill(maps[3 + i], bo, xo));
    }
    const Operand ao = {{am[0], am[1]}, L.p, L.p, L.ldp, L.stride_p, false};
    ok = ok && fill(maps[2], ao, ao);
    if (!ok) return cuda_fail(cudaErrorInvalidValue);

    const dim3 pre((unsigned)L.parts, (unsigned)B);
    e = with_type(grad_type, [&](auto t) {
        using TG = decltype(t);
        trace_before(st, "muon_norm_kernel");
        cudaError_t r = launch_pdl(muon_norm_kernel<TG>, pre, MN_THREADS, st, pp);
        trace_after(st);
        if (r != cudaSuccess) return r;
        trace_before(st, "muon_scale_kernel");
        r = launch_pdl(muon_scale_kernel<TG>, pre, MN_THREADS, st, pp);
        trace_after(st);
        return r;
    });
    if (e != cudaSuccess) return cuda_fail(e);

    auto launch = [&](GemmParams& g, const Maps& from) {
        for (int h = 0; h < parts; ++h) {
            g.a[h] = from.a[h];
            g.b[h] = from.b[h];
            g.b_half[h] = from.b_half[h];
        }
        g.batch = B;
        g.ctrl = pp.ctrl;
        g.stall = stall;
        g.lift = pp.lift;
        auto cut = [&](int size) {
            g.tiles_m = (int32_t)ceil_div64(g.M, size);
            g.tiles_n = (int32_t)ceil_div64(g.N, size);
            return g.mode <= MU_SQUARE ? (int64_t)g.tiles_m * (g.tiles_m + 1) / 2
                                       : (int64_t)g.tiles_m * g.tiles_n;
        };
        const int64_t kblocks = ceil_div64(g.K, GM_K);
        int64_t tiles = cut(SP_TILE);
        // as many blocks a tile as run at once, each with 64 of K at least (with 128 at
        // least, five steps of 300 x 300 in bf16 take 154 us instead of 139)
        int lg = 0;
        while (lg < 3 && tiles * B <= dev.clusters[lg + 1] && kblocks >= 2 << lg) ++lg;
        const int split = 1 << lg;
        // launches over parts of K that keep the truncated sums short (128 x 28,672 in two
        // parts 417 us; the one pair of blocks that its tile would have 2,090)
        const int64_t parts_k = exact ? ceil_div64(kblocks, (int64_t)split * SP_MAX_SUM) : 1;
        const int64_t pairs_from = !exact        ? MU_PAIR_TILES_11
                                   : parts_k > 1 ? MU_PAIR_TILES_LONG
                                                 : MU_PAIR_TILES_22;
        cudaError_t r = cudaSuccess;
        if (cut(GM_TILE) * B >= pairs_from) {
            tiles = cut(GM_TILE);
            g.tiles = (int32_t)tiles;
            // where the last round would leave half of the pairs idle, its tiles are
            // halved (a half takes three quarters of the time of a whole one)
            const int64_t all = tiles * B, rest = all % pairs;
            g.whole = (int32_t)(2 * rest <= pairs ? all - rest : all);
            const int64_t pieces = 2 * all - g.whole;
            const unsigned grid = 2u * (unsigned)std::min<int64_t>(pieces, pairs);
            trace_before(st, "muon_gemm_kernel");
            r = with_kernel(exact, g.mode, [&](auto pair, auto) {
                return launch_pdl(pair, grid, GM_THREADS, st, g, GM_SMEM);
            });
            trace_after(st);
        } else {
            cut(SP_TILE);
            g.width = SP_TILE;
            // (a short side of at most 64, whose products have one 64 of K and so no split:
            // 64 x 5,000 153 us with tiles of 128 columns, 143 of 64; 64 x 8,192 168 and 159)
            if (g.mode >= MU_UPDATE && split == 1 && 2 * tiles * B <= dev.clusters[0]) {
                g.width = SP_TILE / 2;
                g.tiles_n = (int32_t)ceil_div64(g.N, g.width);
                tiles = (int64_t)g.tiles_m * g.tiles_n;
            }
            g.tiles = (int32_t)tiles;
            g.stages = !exact && tiles * B <= dev.clusters[lg] ? SP_MAX_STAGES : SP_MIN_STAGES;
            // (even parts: each has far more than one 64 for every block of a cluster)
            for (int64_t i = 0; i < parts_k && r == cudaSuccess; ++i) {
                g.k_first = (int32_t)(kblocks * i / parts_k);
                g.k_blocks = (int32_t)(kblocks * (i + 1) / parts_k) - g.k_first;
                g.add = i > 0;
                trace_before(st, "muon_split_kernel");
                r = with_kernel(exact, g.mode, [&](auto, auto kernel) {
                    return launch_clusters(kernel, (unsigned)(tiles * B * split), (unsigned)split,
                                           SP_THREADS, sp_smem(exact, g.stages), st, g);
                });
                trace_after(st);
            }
        }
        return r;
    };
    int cur = 0;
    for (int i = 0; i < steps; ++i) {
        const float* k = coef + 3 * i;
        GemmParams g = {};
        g.drop = drop[i];
        g.drop_next = drop[i + 1];
        g.mode = MU_GRAM;
        g.M = g.N = P;
        g.K = Q;
        g.a_mn = g.b_mn = tall;
        g.alpha = (float)(MU_SA / (S * S));
        g.dst[0] = am[0];
        g.dst[1] = am[1];
        g.ld = L.ldp;
        g.stride = L.stride_p;
        if ((e = launch(g, maps[cur])) != cudaSuccess) return cuda_fail(e);

        g.mode = MU_SQUARE;
        g.K = P;
        g.a_mn = g.b_mn = 0;
        g.alpha = k[2] / MU_SA;
        g.beta = k[1];
        g.src[0] = am[0];
        g.src[1] = am[1];
        g.dst[0] = bm[0];
        g.dst[1] = bm[1];
        if ((e = launch(g, maps[2])) != cudaSuccess) return cuda_fail(e);

        const bool last = i == steps - 1;
        g.mode = last ? MU_LAST : MU_UPDATE;
        g.M = (int32_t)rows;
        g.N = (int32_t)cols;
        g.K = P;
        g.b_mn = !tall;
        g.n_fast = tall;
        g.alpha = last ? (float)(scale / (S * MU_SA)) : 1.0f / MU_SA;
        g.beta = last ? (float)(k[0] * (double)scale / S) : k[0];
        g.src[0] = x[cur][0];
        g.src[1] = x[cur][1];
        g.dst[0] = x[cur ^ 1][0];
        g.dst[1] = x[cur ^ 1][1];
        g.ld = L.ldx;
        g.stride = L.stride_x;
        g.out = out;
        g.out_type = out_type;
        g.ld_out = ld_out;
        g.stride_out = stride_out;
        auto starts_on = [&](int64_t a) {
            return aligned(out, (size_t)a) && ld_out * (int64_t)so % a == 0 &&
                   (B == 1 || stride_out * (int64_t)so % a == 0);
        };
        g.out_align = starts_on(16) ? 16 : starts_on(4) ? 4 : 2;
        if ((e = launch(g, maps[3 + cur])) != cudaSuccess) return cuda_fail(e);
        cur ^= 1;
    }
    return TOPK_EF_OK;
}

}  // extern "C"
