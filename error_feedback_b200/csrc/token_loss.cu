// Host side of token_logprobs, token_logprobs_grad and distill_loss
// (include/topk_ef.h): argument checks, the blocks of a row.  One kernel a
// call; the status word is written by a block that checks the ids of a short list,
// or cleared before the kernel whose blocks check a long one.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "topk_ef.h"
#include "common.cuh"
#include "host.cuh"
#include "kernels_logits.cuh"

using namespace tke;

namespace {

constexpr int64_t SCAN_IDS = 8192;         // ids that one block checks
constexpr int SMS = 148;
constexpr int64_t LEAST_LINES = 32;        // lines of a block of a cluster
// Bytes of logits that L2 holds besides what is written (2,048 x 131,072 bf16, 114 MB: 255 us
// one block a row, 239 two).
constexpr int64_t GRAD_L2 = (int64_t)80 << 20;
constexpr int64_t ROUND = SMS * 3;         // blocks of eight warps that run at once
// Warps of a row: fewer once there are more rows than blocks that run at once, so that more
// of them overlap.  (1,024 x 1,000 bf16, top 20: one warp 9.5 us, four 14.1; 600 x 1,000: both
// 9.5; 1,024 x 8,000: 18.2 and 12.6, 2,048 x 8,000: 19.7 and 21.4.  2,048 x 1,000: four 21.3,
// eight 34.1.)
int row_warps(int64_t T, int64_t lines) {
    if (T <= ROUND) return 8;
    if (T > (lines <= 64 ? 2 : 4) * ROUND && lines <= LG_SMALL) return 1;
    return lines <= 256 ? 4 : 8;
}
// token_logprobs' too, where rows are many.  With a top, since others read while one selects, if
// the last round is as full by four as by eight: 4,096 x 131,072 bf16, top 20, 209 us by four and
// 233 by eight, 1,024 rows 68 and 61.  Short of 1,024 lines it need not be (2,048 x 64,000: 65 and
// 70); more than 4,608 take shared memory from blocks of four (1,776 x 400,000: 288 and 254).
// Without a top, when four of eight or eight of four run at once on an SM: rows of up to 960 lines
// (16,384 x 32,000: 189 and 234; 1,333 x 20,000: 16.5 and 19.7; 900 x 30,000 fp32: 21.5 and 22.8),
// longer ones if they are more than those blocks and the last round is as full (2,048 x 64,000: 50.0
// and 52.3; 1,400 x 131,072: 72 and 66, 900: 54.5 and 45.6) or one of many (4,096 x 131,072: 178.4
// and 181.6).
int logprob_warps(int64_t T, int64_t lines, bool top) {
    if (T < 2 * ROUND || lines <= 256) return row_warps(T, lines);
    const int64_t at_once = top ? ROUND : SMS * 4;     // blocks of eight
    const bool even = ceil_div64(T, 2 * at_once) * 2 == ceil_div64(T, at_once);
    if (top) return lines <= 1024 || (lines <= 4608 && even) ? 4 : row_warps(T, lines);
    return lines <= 960 || (T > 2 * at_once && (even || T > 5 * at_once)) ? 4 : row_warps(T, lines);
}

bool sizes_ok(int64_t T, int64_t V) {
    return T >= 0 && T <= MAX_N && V >= 1 && V <= (int64_t)1 << 24;
}
bool pointer_ok(const void* p, size_t size) { return p && aligned(p, size); }
bool scale_ok(float s) { return s >= 1e-30f && s <= 1e30f; }

// Most 128-byte lines that a row touches.
int64_t most_lines(const void* z, int64_t ld, int64_t V, size_t size) {
    const bool whole = (uintptr_t)z % LG_LINE == 0 && (size_t)ld * size % LG_LINE == 0;
    return whole ? ceil_div64(V * (int64_t)size, LG_LINE) : (V * (int64_t)size + LG_LINE - 2) / LG_LINE + 1;
}

// Blocks of a row's cluster: as many as run at once with `most` of the call's (a second round
// of blocks would take as long as the first: 64 x 32,768 bf16 11.8 us with eight, 6.7 with four).
int row_blocks(int64_t T, int64_t lines, int64_t most) {
    int c = 1;
    while (c < 16 && T * 2 * c <= most && lines / (2 * c) >= LEAST_LINES) c *= 2;
    return c;
}

// Lets a kernel have clusters of 16 and `smem` bytes, once for each device.
template <typename K>
cudaError_t allow(K kernel, std::atomic<uint64_t>& done, size_t smem) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev >= 64 || (done.load() >> dev & 1)) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && smem)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) done.fetch_or(1ull << dev);
    return e;
}

// Rows of z and of out that start alike within their 128-byte lines.
bool same_lines(const void* a, int64_t lda, const void* b, int64_t ldb, size_t size) {
    return (uintptr_t)a % LG_LINE == (uintptr_t)b % LG_LINE &&
           (size_t)(lda - ldb) * size % LG_LINE == 0;
}

template <int W, typename T, bool ENTROPY, bool TOP>
cudaError_t launch_logprob(const LogprobParams& p, size_t smem, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = logprob_kernel<W, T, ENTROPY, TOP>;
    cudaError_t e = allow(kernel, done, TOP ? TL_MAX_LINES * 4 : 0);
    if (e != cudaSuccess) return e;
    const int64_t rows = ceil_div64(p.T, Team<W>::TEAMS);
    trace_before(st, "logprob_kernel");
    e = launch_clusters(kernel, (unsigned)((rows + p.scan) * p.blocks), (unsigned)p.blocks,
                        Team<W>::BLOCK, smem, st, p);
    trace_after(st);
    return e;
}

template <typename T, bool ENTROPY, bool TOP>
cudaError_t logprob_by_length(const LogprobParams& p, int warps, size_t smem, cudaStream_t st) {
    return warps == 1   ? launch_logprob<1, T, ENTROPY, TOP>(p, smem, st)
           : warps == 4 ? launch_logprob<4, T, ENTROPY, TOP>(p, smem, st)
                        : launch_logprob<8, T, ENTROPY, TOP>(p, smem, st);
}

template <int W, typename T, typename TO, bool SAME>
cudaError_t launch_distill(const DistillParams& p, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const auto kernel = distill_kernel<W, T, TO, SAME>;
    cudaError_t e = allow(kernel, done, 0);
    if (e != cudaSuccess) return e;
    const int64_t rows = ceil_div64(p.T, Team<W>::TEAMS);
    trace_before(st, "distill_kernel");
    e = launch_clusters(kernel, (unsigned)((rows + p.scan) * p.blocks), (unsigned)p.blocks,
                        Team<W>::BLOCK, 0, st, p);
    trace_after(st);
    return e;
}

template <typename T, typename TO, bool SAME>
cudaError_t distill_by_length(const DistillParams& p, int warps, cudaStream_t st) {
    return warps == 1   ? launch_distill<1, T, TO, SAME>(p, st)
           : warps == 4 ? launch_distill<4, T, TO, SAME>(p, st)
                        : launch_distill<8, T, TO, SAME>(p, st);
}

}  // namespace

extern "C" {

size_t token_logprobs_workspace_bytes(void) { return align_up(sizeof(Ctrl)); }

int token_logprobs(const void* logits, int32_t logits_type, int64_t ld_logits, const void* ids,
                   int32_t id_bytes, int64_t T, int64_t V, float scale, int64_t padding_idx,
                   int32_t top, float* logprob, float* entropy, float* lse, int32_t* top_ids,
                   float* top_logprobs, void* ws, size_t ws_bytes, void* stream) {
    const size_t sz = type_size(logits_type);
    if (!sizes_ok(T, V) || !sz || ld_logits < V || !scale_ok(scale) || top < 0 || top > TL_MAX_TOP ||
        !ws || !aligned(ws, ALIGN))
        return TOPK_EF_ERR_INVALID_ARG;
    const int64_t lines = most_lines(logits, ld_logits, V, sz);
    if (top > 0 && most_lines(nullptr, 1, V, sz) > TL_MAX_LINES) return TOPK_EF_ERR_INVALID_ARG;
    if (ids && ((id_bytes != 4 && id_bytes != 8) || !aligned(ids, id_bytes)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (!ids && logprob) return TOPK_EF_ERR_INVALID_ARG;
    if (!aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(top_ids, 4) ||
        !aligned(top_logprobs, 4))
        return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && !pointer_ok(logits, sz)) return TOPK_EF_ERR_INVALID_ARG;
    const std::initializer_list<Region> writes = {
        vector_of(logprob, T, 4), vector_of(entropy, T, 4), vector_of(lse, T, 4), vector_of(top_ids, T * top, 4),
        vector_of(top_logprobs, T * top, 4), vector_of(ws, 1, token_logprobs_workspace_bytes())};
    if (any_meet(writes) || any_meet(writes, {rows_of(logits, T, ld_logits, V, sz), vector_of(ids, T, id_bytes)}))
        return TOPK_EF_ERR_INVALID_ARG;
    if (ws_bytes < token_logprobs_workspace_bytes()) return TOPK_EF_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LogprobParams p = {};
    p.z = logits;
    p.ids = ids;
    p.logprob = logprob;
    p.entropy = entropy;
    p.lse = lse;
    p.top_ids = top_ids;
    p.top_logprobs = top_logprobs;
    p.ctrl = static_cast<Ctrl*>(ws);
    p.T = T;
    p.V = V;
    p.ldz = ld_logits;
    p.padding = padding_idx;
    p.id64 = id_bytes == 8;
    p.top = top_ids || top_logprobs ? top : 0;
    const int warps = logprob_warps(T, lines, p.top > 0);
    p.blocks = warps < 8 ? 1 : row_blocks(T, lines, ROUND);
    p.scan = T <= SCAN_IDS;
    p.scale = scale;
    p.c = (float)((double)scale * 1.4426950408889634);
    if (!p.scan) {
        const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(Ctrl), st);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    // the groups' largest values: of lines, or of the chunks of a block's rows
    const size_t smem = !p.top       ? 0
                        : warps == 1 ? Team<1>::TEAMS * LG_SMALL * 4 * sizeof(float)
                                     : ((size_t)lines * 4 + 15) / 16 * 16;
    const cudaError_t e = with_type(logits_type, [&](auto t) {
        using TZ = decltype(t);
        if (p.top)
            return entropy ? logprob_by_length<TZ, true, true>(p, warps, smem, st)
                           : logprob_by_length<TZ, false, true>(p, warps, smem, st);
        return entropy ? logprob_by_length<TZ, true, false>(p, warps, smem, st)
                       : logprob_by_length<TZ, false, false>(p, warps, smem, st);
    });
    return e == cudaSuccess ? TOPK_EF_OK : cuda_fail(e);
}

int token_logprobs_grad(const void* logits, int32_t logits_type, int64_t ld_logits,
                        const void* ids, int32_t id_bytes, int64_t T, int64_t V, float scale,
                        int64_t padding_idx, const float* lse, const float* entropy,
                        const float* grad_logprob, const float* grad_entropy, void* grad_logits,
                        int32_t grad_logits_type, int64_t ld_grad_logits, void* ws,
                        size_t ws_bytes, void* stream) {
    const size_t sz = type_size(logits_type), so = type_size(grad_logits_type);
    if (!sizes_ok(T, V) || !sz || !so || ld_logits < V || ld_grad_logits < V || !scale_ok(scale) ||
        !ws || !aligned(ws, ALIGN))
        return TOPK_EF_ERR_INVALID_ARG;
    if (ids && ((id_bytes != 4 && id_bytes != 8) || !aligned(ids, id_bytes)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (!ids && grad_logprob) return TOPK_EF_ERR_INVALID_ARG;
    if (!aligned(entropy, 4) || !aligned(grad_logprob, 4) || !aligned(grad_entropy, 4) ||
        (grad_entropy && !entropy))
        return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && (!pointer_ok(logits, sz) || !pointer_ok(grad_logits, so) || !pointer_ok(lse, 4)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && grad_logits == logits && (sz != so || ld_logits != ld_grad_logits))
        return TOPK_EF_ERR_INVALID_ARG;
    const Region rz = rows_of(logits, T, ld_logits, V, sz), rg = rows_of(grad_logits, T, ld_grad_logits, V, so);
    const Region rs = vector_of(ws, 1, token_logprobs_workspace_bytes());
    if ((grad_logits != logits && meet(rg, rz)) || meet(rs, rz) || meet(rs, rg) ||
        any_meet({rg, rs}, {vector_of(ids, T, id_bytes), vector_of(lse, T, 4), vector_of(entropy, T, 4),
                            vector_of(grad_logprob, T, 4), vector_of(grad_entropy, T, 4)}))
        return TOPK_EF_ERR_INVALID_ARG;
    if (ws_bytes < token_logprobs_workspace_bytes()) return TOPK_EF_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LogprobGradParams p = {};
    p.z = logits;
    p.ids = ids;
    p.lse = lse;
    p.entropy = entropy;
    p.g = grad_logprob;
    p.h = grad_entropy;
    p.dz = grad_logits;
    p.ctrl = static_cast<Ctrl*>(ws);
    p.T = T;
    p.V = V;
    p.ldz = ld_logits;
    p.lddz = ld_grad_logits;
    p.padding = padding_idx;
    p.id64 = id_bytes == 8;
    p.scan = T <= SCAN_IDS;
    p.scale = scale;
    p.c = (float)((double)scale * 1.4426950408889634);
    p.parts = (int32_t)std::min(ceil_div64(most_lines(logits, ld_logits, V, sz), LD_LINES),
                                std::max<int64_t>(1, MAX_N / (T + 1)));
    if (!p.scan) {
        const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(Ctrl), st);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    const unsigned grid = (unsigned)(ceil_div64(T * p.parts, LD_WARPS) + p.scan);
    const bool same = sz == so && same_lines(logits, ld_logits, grad_logits, ld_grad_logits, sz);
    trace_before(st, "logprob_grad_kernel");
    const cudaError_t e = with_type(logits_type, [&](auto t) {
        return with_type(grad_logits_type, [&](auto to) {
            using TZ = decltype(t);
            using TO = decltype(to);
            if constexpr (sizeof(TZ) == sizeof(TO))
                if (same)
                    return p.h ? launch_pdl(logprob_grad_kernel<TZ, TO, true, true>, grid, LD_THREADS, st, p)
                               : launch_pdl(logprob_grad_kernel<TZ, TO, true, false>, grid, LD_THREADS, st, p);
            return p.h ? launch_pdl(logprob_grad_kernel<TZ, TO, false, true>, grid, LD_THREADS, st, p)
                       : launch_pdl(logprob_grad_kernel<TZ, TO, false, false>, grid, LD_THREADS, st, p);
        });
    });
    trace_after(st);
    return e == cudaSuccess ? TOPK_EF_OK : cuda_fail(e);
}

size_t distill_loss_workspace_bytes(void) { return align_up(sizeof(Ctrl)); }

int distill_loss(const void* logits, int32_t logits_type, int64_t ld_logits,
                 const void* teacher_ids, int32_t id_bytes, const void* teacher_logits,
                 int32_t teacher_type, int64_t T, int64_t V, int32_t K, float scale,
                 const float* weight, float* loss, void* grad_logits, int32_t grad_logits_type,
                 int64_t ld_grad_logits, void* ws, size_t ws_bytes, void* stream) {
    const size_t sz = type_size(logits_type), so = type_size(grad_logits_type);
    const size_t st_ = type_size(teacher_type);
    if (!sizes_ok(T, V) || !sz || !st_ || ld_logits < V || !scale_ok(scale) || K < 0 ||
        K > DL_MAX_K || !ws || !aligned(ws, ALIGN))
        return TOPK_EF_ERR_INVALID_ARG;
    if (grad_logits && (!so || ld_grad_logits < V || !aligned(grad_logits, so)))
        return TOPK_EF_ERR_INVALID_ARG;
    if ((id_bytes != 4 && id_bytes != 8) || !aligned(weight, 4) || !aligned(loss, 4))
        return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && !pointer_ok(logits, sz)) return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && K > 0 && (!pointer_ok(teacher_ids, id_bytes) || !pointer_ok(teacher_logits, st_)))
        return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && grad_logits == logits && (sz != so || ld_logits != ld_grad_logits))
        return TOPK_EF_ERR_INVALID_ARG;
    const Region rz = rows_of(logits, T, ld_logits, V, sz);
    const Region rg = rows_of(grad_logits, T, ld_grad_logits, V, so);
    const Region rl = vector_of(loss, T, 4), rw = vector_of(weight, T, 4);
    const Region rs = vector_of(ws, 1, distill_loss_workspace_bytes());
    const Region ri = vector_of(teacher_ids, T * K, id_bytes), rt = vector_of(teacher_logits, T * K, st_);
    // (a row's weight is read before its loss is written)
    if ((grad_logits != logits && meet(rg, rz)) || (loss != weight && meet(rl, rw)) || meet(rg, rl) || meet(rg, rs) ||
        meet(rl, rs) || meet(rl, rz) || meet(rs, rz) || meet(rg, rw) || meet(rs, rw) || meet(rg, ri) ||
        meet(rl, ri) || meet(rs, ri) || meet(rg, rt) || meet(rl, rt) || meet(rs, rt))
        return TOPK_EF_ERR_INVALID_ARG;
    if (ws_bytes < distill_loss_workspace_bytes()) return TOPK_EF_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    DistillParams p = {};
    p.z = logits;
    p.ids = teacher_ids;
    p.teacher = teacher_logits;
    p.weight = weight;
    p.loss = loss;
    p.dz = grad_logits;
    p.ctrl = static_cast<Ctrl*>(ws);
    p.T = T;
    p.V = V;
    p.ldz = ld_logits;
    p.lddz = ld_grad_logits;
    p.id64 = id_bytes == 8;
    p.teacher_type = teacher_type;
    p.K = K;
    const bool same = grad_logits && sz == so &&
                      same_lines(logits, ld_logits, grad_logits, ld_grad_logits, sz);
    const int64_t lines = most_lines(logits, ld_logits, V, sz);
    const int warps = row_warps(T, lines);
    p.blocks = warps < 8 ? 1 : row_blocks(T, lines, ROUND);
    // rows that blocks are at should fit L2 until their gradient is written
    if (grad_logits && warps == 8)
        while (p.blocks < 4 && lines * LG_LINE * (ROUND / p.blocks) > GRAD_L2) p.blocks *= 2;
    p.scan = T * std::max(K, 1) <= SCAN_IDS;
    p.scale = scale;
    p.c = (float)((double)scale * 1.4426950408889634);
    if (!p.scan) {
        const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(Ctrl), st);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    const cudaError_t e = with_type(logits_type, [&](auto t) {
        return with_type(grad_logits ? grad_logits_type : logits_type, [&](auto to) {
            using TZ = decltype(t);
            using TO = decltype(to);
            if constexpr (sizeof(TZ) == sizeof(TO))
                if (same) return distill_by_length<TZ, TO, true>(p, warps, st);
            return distill_by_length<TZ, TO, false>(p, warps, st);
        });
    });
    return e == cudaSuccess ? TOPK_EF_OK : cuda_fail(e);
}

}  // extern "C"
