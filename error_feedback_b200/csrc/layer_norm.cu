// Host side of layer_norm (include/topk_ef.h): argument checks, choice of kernel by row
// length: norm_kernel, norm_long_kernel for rows past NM_MAX_D.
#include <cuda_runtime.h>

#include <algorithm>

#include "topk_ef.h"
#include "common.cuh"
#include "norm_host.cuh"

using namespace tke;

namespace {

template <typename TX, typename TY, int G, int V>
cudaError_t launch_norm(const NormParams& p, cudaStream_t st) {
    constexpr int block = NORM_BLOCK<G>;
    constexpr size_t smem = (size_t)block / G * NR_SLOTS<TX, G> * NR_BYTES<TX, G, V>;
    static Resident resident;
    const int most = resident.get(norm_kernel<TX, TY, G, V>, block, smem);
    if (!most) return cudaErrorLaunchOutOfResources;
    const int64_t rows = ceil_div64(p.T, block / G);
    trace_before(st, "norm_kernel");
    const cudaError_t e = launch_pdl(norm_kernel<TX, TY, G, V>,
                                     (unsigned)std::min<int64_t>(most, rows), block, st, p, smem);
    trace_after(st);
    return e;
}

template <typename TX, typename TY, int V>
cudaError_t norm_by_length(const NormParams& p, cudaStream_t st) {
    if (p.D <= 128) return launch_norm<TX, TY, 8, V>(p, st);
    if (p.D <= 256) return launch_norm<TX, TY, 16, V>(p, st);
    if (p.D <= 512) return launch_norm<TX, TY, 32, V>(p, st);
    if (p.D <= 1024) return launch_norm<TX, TY, 64, V>(p, st);
    if (p.D <= 2048) return launch_norm<TX, TY, 128, V>(p, st);
    if (p.D <= 4096) return launch_norm<TX, TY, 256, V>(p, st);
    if (p.D <= 8192) return launch_norm<TX, TY, 512, V>(p, st);
    return launch_norm<TX, TY, 1024, V>(p, st);
}

}  // namespace

extern "C" {

int layer_norm(const void* x, int32_t x_type, int64_t ld_x, const void* weight,
               int32_t weight_type, const void* bias, int32_t bias_type, int64_t T, int64_t D,
               float eps, void* out, int32_t out_type, int64_t ld_out, float* mean, float* rstd,
               void* stream) {
    const size_t sx = type_size(x_type), so = type_size(out_type);
    if (!norm_sizes_ok(T, D) || !sx || !so || ld_x < D || ld_out < D || !(eps >= 0.0f))
        return TOPK_EF_ERR_INVALID_ARG;
    if (weight && (!type_size(weight_type) || !pointer_ok(weight, weight_type)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (bias && (!type_size(bias_type) || !pointer_ok(bias, bias_type)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (!aligned(mean, 4) || !aligned(rstd, 4)) return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && (!pointer_ok(x, x_type) || !pointer_ok(out, out_type)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && out == x && (sx != so || ld_x != ld_out)) return TOPK_EF_ERR_INVALID_ARG;
    if (T == 0) return TOPK_EF_OK;
    const Region rx = rows_of(x, T, ld_x, D, sx), ro = rows_of(out, T, ld_out, D, so);
    const Region rm = vector_of(mean, T, 4), rr = vector_of(rstd, T, 4);
    if ((out != x && meet(ro, rx)) || any_meet({rm, rr}, {rx}) || any_meet({ro, rm, rr}) ||
        any_meet({ro, rm, rr}, {vector_of(weight, D, type_size(weight_type)), vector_of(bias, D, type_size(bias_type))}))
        return TOPK_EF_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    NormParams p = {};
    p.x = x;
    p.w = weight;
    p.b = bias;
    p.y = out;
    p.mean = mean;
    p.rstd = rstd;
    p.T = T;
    p.D = D;
    p.ldx = ld_x;
    p.ldy = ld_out;
    p.w_type = weight_type;
    p.b_type = bias_type;
    p.eps = eps;
    p.inv_d = 1.0f / (float)D;
    const bool vec = D % 8 == 0 && rows16(x, ld_x, sx) && rows16(out, ld_out, so) &&
                     aligned(weight, 16) && aligned(bias, 16);
    const cudaError_t e = with_type(x_type, [&](auto tx) {
        return with_type(out_type, [&](auto to) {
            using TX = decltype(tx);
            using TO = decltype(to);
            if (D <= NM_MAX_D)
                return vec ? norm_by_length<TX, TO, NORM_GROUP<TX, TO>>(p, st)
                           : norm_by_length<TX, TO, 1>(p, st);
            trace_before(st, "norm_long_kernel");
            const cudaError_t r = launch_pdl(norm_long_kernel<TX, TO>,
                                             (unsigned)std::min<int64_t>(T, SMS * 4), NL_THREADS, st, p);
            trace_after(st);
            return r;
        });
    });
    return e == cudaSuccess ? TOPK_EF_OK : cuda_fail(e);
}

}  // extern "C"
