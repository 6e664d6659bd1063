// Host side of layer_norm_grad (include/topk_ef.h): argument checks, workspace layout,
// choice of kernel by row length: norm_grad_kernel -> norm_sum_kernel, for rows past NG_COLS_D
// norm_cols_kernel -> norm_grad_kernel or norm_grad_long_kernel -> norm_sum_kernel.
#include <cuda_runtime.h>

#include <algorithm>

#include "topk_ef.h"
#include "common.cuh"
#include "kernels_norm_grad.cuh"
#include "norm_host.cuh"

using namespace tke;

namespace {

// Blocks that have at least four rows each.
int64_t row_parts(int64_t T) { return std::max<int64_t>(1, ceil_div64(T, 4)); }

// Most partial rows of the column sums: as many blocks as run at once, two of 256 threads an SM
// or one of 512, at 128 registers each; those of the column kernel.
int64_t grad_parts(int64_t T, int64_t D) {
    return std::min(row_parts(T), D > NG_COLS_D ? NL_PARTS : D > 4096 ? SMS : (int64_t)2 * SMS);
}

template <typename TX, typename TD, int G, int V>
cudaError_t launch_grad(const NormGradParams& p, int32_t& parts, cudaStream_t st) {
    constexpr int block = NORM_BLOCK<G>;
    constexpr size_t ring = (size_t)block / G * NG_SLOTS<TX, TD, G> *
                            (NR_BYTES<TX, G, V> + NR_BYTES<TD, G, V>);
    constexpr size_t smem = std::max(ring, (size_t)G * NR_ELEMS * 4);
    static Resident resident;
    const int most = resident.get(norm_grad_kernel<TX, TD, G, V>, block, smem);
    if (!most) return cudaErrorLaunchOutOfResources;
    const int64_t rows = ceil_div64(p.T, block / G);
    parts = (int32_t)std::min(std::min<int64_t>(most, rows), G < 1024 ? grad_parts(p.T, p.D) : row_parts(p.T));
    trace_before(st, "norm_grad_kernel");
    const cudaError_t e =
        launch_pdl(norm_grad_kernel<TX, TD, G, V>, (unsigned)parts, block, st, p, smem);
    trace_after(st);
    return e;
}

// The column sums by themselves.
template <typename TX, typename TD, int V>
cudaError_t launch_cols(const NormGradParams& p, int32_t& parts, cudaStream_t st) {
    parts = (int32_t)grad_parts(p.T, p.D);
    trace_before(st, "norm_cols_kernel");
    const cudaError_t e =
        launch_pdl(norm_cols_kernel<TX, TD, V>,
                   dim3((unsigned)ceil_div64(p.D, NL_COLS * V), (unsigned)parts), NL_COLS, st, p);
    trace_after(st);
    return e;
}

template <typename TX, typename TD, int V>
cudaError_t grad_by_length(const NormGradParams& p, int32_t& parts, cudaStream_t st) {
    if (p.D <= 128) return launch_grad<TX, TD, 8, V>(p, parts, st);
    if (p.D <= 256) return launch_grad<TX, TD, 16, V>(p, parts, st);
    if (p.D <= 512) return launch_grad<TX, TD, 32, V>(p, parts, st);
    if (p.D <= 1024) return launch_grad<TX, TD, 64, V>(p, parts, st);
    if (p.D <= 2048) return launch_grad<TX, TD, 128, V>(p, parts, st);
    if (p.D <= 4096) return launch_grad<TX, TD, 256, V>(p, parts, st);
    if (p.D <= 8192) return launch_grad<TX, TD, 512, V>(p, parts, st);
    int32_t none = 0;
    return launch_grad<TX, TD, 1024, V>(p, none, st);
}

}  // namespace

extern "C" {

size_t layer_norm_grad_workspace_bytes(int64_t T, int64_t D) {
    if (!norm_sizes_ok(T, D)) return 0;
    return align_up(sizeof(Ctrl)) + align_up((size_t)grad_parts(T, D) * 2 * (size_t)D * 4);
}

int layer_norm_grad(const void* grad_out, int32_t grad_out_type, int64_t ld_grad_out,
                    const void* x, int32_t x_type, int64_t ld_x, const float* mean,
                    const float* rstd, const void* weight, int32_t weight_type, int64_t T,
                    int64_t D, void* grad_x, int64_t ld_grad_x, void* grad_weight,
                    int32_t grad_weight_type, void* grad_bias, int32_t grad_bias_type,
                    int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
    const size_t need = layer_norm_grad_workspace_bytes(T, D);
    const size_t sx = type_size(x_type), sd = type_size(grad_out_type);
    const bool cols = grad_weight || grad_bias;
    if (!need || !sx || !sd || ld_x < D || ld_grad_out < D || ld_grad_x < D)
        return TOPK_EF_ERR_INVALID_ARG;
    if (weight && (!type_size(weight_type) || !pointer_ok(weight, weight_type)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (grad_weight && (!type_size(grad_weight_type) || !pointer_ok(grad_weight, grad_weight_type)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (grad_bias && (!type_size(grad_bias_type) || !pointer_ok(grad_bias, grad_bias_type)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (cols && (grad_weight == grad_bias || !ws || !aligned(ws, ALIGN)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && (!pointer_ok(grad_out, grad_out_type) || !pointer_ok(x, x_type) ||
                  !pointer_ok(grad_x, x_type) || !pointer_ok(mean, TOPK_EF_F32) ||
                  !pointer_ok(rstd, TOPK_EF_F32)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && ((grad_x == x && ld_grad_x != ld_x) ||
                  (grad_x == grad_out && (sx != sd || ld_grad_x != ld_grad_out))))
        return TOPK_EF_ERR_INVALID_ARG;
    // (the column gradients are written after all is read)
    const Region rx = rows_of(x, T, ld_x, D, sx), rd = rows_of(grad_out, T, ld_grad_out, D, sd);
    const Region rg = rows_of(grad_x, T, ld_grad_x, D, sx);
    const Region rw = vector_of(grad_weight, D, type_size(grad_weight_type));
    const Region rb = vector_of(grad_bias, D, type_size(grad_bias_type));
    const Region rs = vector_of(cols ? ws : nullptr, 1, need);
    const Region rm = vector_of(mean, T, 4), rr = vector_of(rstd, T, 4);
    const Region rk = vector_of(weight, D, type_size(weight_type));
    if ((grad_x != x && meet(rg, rx)) || (grad_x != grad_out && meet(rg, rd)) ||
        any_meet({rg, rw, rb, rs}) || any_meet({rg, rs}, {rm, rr, rk}) || any_meet({rs}, {rx, rd}))
        return TOPK_EF_ERR_INVALID_ARG;
    if (cols && ws_bytes < need) return TOPK_EF_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    NormGradParams p = {};
    p.dy = grad_out;
    p.x = x;
    p.mean = mean;
    p.rstd = rstd;
    p.w = weight;
    p.dx = grad_x;
    p.part = cols ? reinterpret_cast<float*>(static_cast<char*>(ws) + align_up(sizeof(Ctrl))) : nullptr;
    p.T = T;
    p.D = D;
    p.ldy = ld_grad_out;
    p.ldx = ld_x;
    p.lddx = ld_grad_x;
    p.w_type = weight_type;
    p.inv_d = 1.0f / (float)D;
    int32_t parts = 0;
    cudaError_t e = cudaSuccess;
    if (T > 0) {
        const bool vec = D % 8 == 0 && rows16(x, ld_x, sx) && rows16(grad_x, ld_grad_x, sx) &&
                         rows16(grad_out, ld_grad_out, sd) && aligned(weight, 16);
        e = with_type(x_type, [&](auto tx) {
            return with_type(grad_out_type, [&](auto td) {
                using TX = decltype(tx);
                using TD = decltype(td);
                // (the sums first: grad_x may be x or grad_out)
                cudaError_t r = cols && D > NG_COLS_D
                                    ? vec ? launch_cols<TX, TD, 4>(p, parts, st) : launch_cols<TX, TD, 1>(p, parts, st)
                                    : cudaSuccess;
                if (r != cudaSuccess) return r;
                if (D <= NM_MAX_D)
                    return vec ? grad_by_length<TX, TD, NORM_GROUP<TX, TD>>(p, parts, st)
                               : grad_by_length<TX, TD, 1>(p, parts, st);
                trace_before(st, "norm_grad_long_kernel");
                r = launch_pdl(norm_grad_long_kernel<TX, TD>, (unsigned)std::min<int64_t>(T, SMS * 4),
                               NL_THREADS, st, p);
                trace_after(st);
                return r;
            });
        });
        if (e != cudaSuccess) return cuda_fail(e);
    }
    if (!cols) return TOPK_EF_OK;
    NormSumParams s = {};
    s.part = p.part;
    s.ctrl = static_cast<Ctrl*>(ws);
    s.out[0] = grad_weight;
    s.out[1] = grad_bias;
    s.type[0] = grad_weight_type;
    s.type[1] = grad_bias_type;
    s.D = D;
    s.parts = parts;
    s.accumulate = accumulate ? 1 : 0;
    trace_before(st, "norm_sum_kernel");
    e = launch_pdl(norm_sum_kernel, dim3((unsigned)ceil_div64(D, 32), 2), 32 * NS_WARPS, st, s);
    trace_after(st);
    return e == cudaSuccess ? TOPK_EF_OK : cuda_fail(e);
}

}  // extern "C"
