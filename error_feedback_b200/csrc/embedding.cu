// Host side of embedding_lookup, embedding_grad and embedding_grad_rows
// (include/topk_ef.h): argument checks, workspace layout, launch sequences.
//
//   embedding_lookup:     lookup_kernel
//   embedding_grad*:      a few tokens: grad_direct_kernel alone; else
//                         rank_kernel (short lists), or per 9-bit digit of the id (sort_count_kernel ->
//                         [sort_prefix_kernel, many tiles] -> sort_scatter_kernel)
//                         -> grad_sum_kernel -> grad_combine_kernel
#include <cuda_runtime.h>

#include <algorithm>

#include "topk_ef.h"
#include "common.cuh"
#include "host.cuh"
#include "kernels_embedding.cuh"

using namespace tke;

namespace {

bool rows16(const void* p, int64_t ld, size_t size) {
    return aligned(p, 16) && (size_t)ld * size % 16 == 0;
}

// ids, rows and columns that every call accepts
bool sizes_ok(int64_t T, int64_t V, int64_t D) {
    return T >= 0 && T <= MAX_N && V >= 0 && V <= MAX_N && D >= 0 && D <= (int64_t)1 << 24;
}

// ------------------------------------------------------------------ gradient

// Positions of one tile of the sum.  Short lists take short tiles, so that
// one wave of blocks has work; long ones amortise the partial rows (at most
// two fp32 rows per tile) over more rows read.
int32_t tile_positions(int64_t T) { return T <= 4096 ? 8 : T <= 262144 ? 32 : EG_MAX_C; }

struct GLayout {
    size_t ctrl, list_count, bitmap, zero_end, word_prefix, totals, counts, key[2], pos[2], list[2],
        head, tail, total;
    int64_t sort_tiles, tiles, Dp;
    int32_t C;
};

GLayout grad_layout(int64_t T, int64_t V, int64_t D) {
    GLayout L;
    L.C = tile_positions(T);
    L.sort_tiles = ceil_div64(T, ES_TILE);
    L.tiles = ceil_div64(T, L.C);
    L.Dp = ceil_div64(D, 8) * 8;
    const size_t words = (size_t)ceil_div64(V, 32) * 4;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes);
        return at;
    };
    L.ctrl = take(sizeof(Ctrl));
    L.list_count = take(2 * sizeof(uint32_t));
    L.bitmap = take(words);
    L.zero_end = o;
    L.word_prefix = take(words);
    L.totals = take(ES_BINS * 4);
    L.counts = take((size_t)L.sort_tiles * ES_BINS * 4);
    for (int i = 0; i < 2; ++i) {
        L.key[i] = take((size_t)T * 4);
        L.pos[i] = take((size_t)T * 4);
    }
    L.list[0] = take((size_t)L.tiles * 16);
    L.list[1] = take(((size_t)L.tiles / EC_LONG + 1) * 16);
    L.head = take((size_t)L.tiles * L.Dp * 4);
    L.tail = take((size_t)L.tiles * L.Dp * 4);
    L.total = o;
    return L;
}

// Units of zeros that a scattering and a counting kernel write besides: about
// what memory takes in the time that they need anyway.  (None: 30,011 x 1,001 fp32 99
// us instead of 93, 32,768 x 4,096 into 131,072 rows 390 instead of 383; half as
// many: 98 and 388; twice as many: 94 and 380.)
constexpr int64_t ES_SCATTER_UNITS = 1200, ES_COUNT_UNITS = 400;

template <typename TI>
cudaError_t launch_sort_pass(SortParams& sp, bool first, Fill& zeros, int64_t& units,
                             cudaStream_t st) {
    // takes up to `most` units for a launch whose own blocks are the first `blocks`
    auto with_units = [&](int blocks, int64_t most) {
        const int64_t n = std::min(units, most);
        sp.fill = zeros;
        sp.fill_from = blocks;
        zeros.first += n;
        units -= n;
        return blocks + (int)n;
    };
    // (the first count sees to the bitmap that says which rows stay out)
    int grid = with_units(sp.tiles, first ? 0 : ES_COUNT_UNITS);
    trace_before(st, "sort_count_kernel");
    cudaError_t e = first ? launch_pdl(sort_count_kernel<TI, true>, grid, ES_THREADS, st, sp)
                          : launch_pdl(sort_count_kernel<TI, false>, grid, ES_THREADS, st, sp);
    trace_after(st);
    if (e != cudaSuccess) return e;
    sp.scanned = sp.tiles > ES_SCAN_TILES;
    if (sp.scanned) {
        trace_before(st, "sort_prefix_kernel");
        e = launch_pdl(sort_prefix_kernel, ES_BINS / 32, 1024, st, sp);
        trace_after(st);
        if (e != cudaSuccess) return e;
    }
    grid = with_units(sp.tiles + (first && sp.word_prefix ? 1 : 0), ES_SCATTER_UNITS);
    trace_before(st, "sort_scatter_kernel");
    e = first ? launch_pdl(sort_scatter_kernel<TI, true>, grid, ES_THREADS, st, sp)
              : launch_pdl(sort_scatter_kernel<TI, false>, grid, ES_THREADS, st, sp);
    trace_after(st);
    return e;
}

int grad_call(const void* dy, int32_t dy_type, int64_t ld_dy, const void* ids, int32_t id_bytes,
              int64_t T, int64_t V, int64_t D, float scale, int64_t padding, void* out,
              int32_t out_type, int64_t ld_out, int32_t accumulate, int32_t* out_rows,
              int32_t* out_count, bool rows, void* ws, size_t ws_bytes, void* stream) {
    const size_t need = embedding_grad_workspace_bytes(T, V, D);
    const size_t sd = type_size(dy_type), so = type_size(out_type);
    if (need == 0 || !ws || !aligned(ws, ALIGN) || !sd || !so) return TOPK_EF_ERR_INVALID_ARG;
    if ((id_bytes != 4 && id_bytes != 8) || ld_dy < D || ld_out < D)
        return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && (!ids || !aligned(ids, id_bytes))) return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && D > 0 && (!dy || !aligned(dy, sd))) return TOPK_EF_ERR_INVALID_ARG;
    const bool writes = D > 0 && V > 0 && (T > 0 || (!rows && !accumulate));
    if (writes && (!out || !aligned(out, so))) return TOPK_EF_ERR_INVALID_ARG;
    if (writes && T > 0 && out == dy) return TOPK_EF_ERR_INVALID_ARG;
    if (rows && (!out_count || !aligned(out_count, 4) ||
                 (T > 0 && V > 0 && (!out_rows || !aligned(out_rows, 4)))))
        return TOPK_EF_ERR_INVALID_ARG;
    if (ws_bytes < need) return TOPK_EF_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const GLayout L = grad_layout(T, V, D);
    char* w = static_cast<char*>(ws);
    const bool direct = T > 0 && T <= DR_MAX, brief = T > 0 && T <= SR_MAX;
    cudaError_t e = cudaSuccess;
    if (!brief) e = cudaMemsetAsync(w, 0, L.zero_end, st);
    if (e == cudaSuccess && rows && T == 0) e = cudaMemsetAsync(out_count, 0, 4, st);
    if (e != cudaSuccess) return cuda_fail(e);

    SortParams sp = {};
    sp.ids = ids;
    sp.counts = reinterpret_cast<uint32_t*>(w + L.counts);
    sp.totals = reinterpret_cast<uint32_t*>(w + L.totals);
    const bool fill = !rows && !accumulate && V > 0 && D > 0;
    sp.bitmap = rows || fill ? reinterpret_cast<uint32_t*>(w + L.bitmap) : nullptr;
    sp.word_prefix = rows ? reinterpret_cast<uint32_t*>(w + L.word_prefix) : nullptr;
    sp.out_count = out_count;
    sp.ctrl = reinterpret_cast<Ctrl*>(w + L.ctrl);
    sp.T = T;
    sp.V = V;
    sp.padding = padding;
    sp.tiles = (int32_t)L.sort_tiles;
    // the dense gradient's zeros, in units
    Fill zeros = {};
    int64_t units = 0;
    if (fill) {
        zeros.out = static_cast<char*>(out);
        zeros.bitmap = brief ? nullptr : sp.bitmap;
        zeros.V = V;
        zeros.row_bytes = D * (int64_t)so;
        zeros.stride_bytes = ld_out * (int64_t)so;
        zeros.size = (int32_t)so;
        zeros.rows = std::max<int64_t>(EG_THREADS / 32, FILL_BYTES / zeros.row_bytes);
        if (direct) zeros.rows = std::min<int64_t>(zeros.rows, DR_FILL_ROWS);
        units = ceil_div64(V, zeros.rows);
    }
    int cur = 0;
    if (direct) {
        // (launched below)
    } else if (brief) {
        RankParams rp = {};
        rp.ids = ids;
        rp.key = reinterpret_cast<uint32_t*>(w + L.key[0]);
        rp.pos = reinterpret_cast<uint32_t*>(w + L.pos[0]);
        rp.list_count = reinterpret_cast<uint32_t*>(w + L.list_count);
        rp.ctrl = sp.ctrl;
        rp.T = T;
        rp.V = V;
        rp.padding = padding;
        rp.rank_blocks = (int32_t)ceil_div64(T, SR_KEYS);
        rp.fill = zeros;
        const int64_t blocks = rp.rank_blocks + units;
        if (blocks > MAX_N) return TOPK_EF_ERR_INVALID_ARG;
        trace_before(st, "rank_kernel");
        e = id_bytes == 8 ? launch_pdl(rank_kernel<int64_t>, (unsigned)blocks, SR_THREADS, st, rp)
                          : launch_pdl(rank_kernel<int32_t>, (unsigned)blocks, SR_THREADS, st, rp);
        trace_after(st);
        if (e != cudaSuccess) return cuda_fail(e);
        sp.word_prefix = nullptr;
        units = 0;
    } else if (T > 0) {
        int bits = 1;
        while (bits < 32 && ((uint64_t)V >> bits) != 0) ++bits;
        const int passes = (bits + ES_BITS - 1) / ES_BITS;
        for (int i = 0; i < passes; ++i) {
            sp.shift = i * ES_BITS;
            sp.key_in = reinterpret_cast<uint32_t*>(w + L.key[cur]);
            sp.pos_in = reinterpret_cast<uint32_t*>(w + L.pos[cur]);
            cur = i == 0 ? 0 : cur ^ 1;
            sp.key_out = reinterpret_cast<uint32_t*>(w + L.key[cur]);
            sp.pos_out = reinterpret_cast<uint32_t*>(w + L.pos[cur]);
            e = id_bytes == 8 ? launch_sort_pass<int64_t>(sp, i == 0, zeros, units, st)
                              : launch_sort_pass<int32_t>(sp, i == 0, zeros, units, st);
            if (e != cudaSuccess) return cuda_fail(e);
        }
    }

    GradParams p = {};
    p.dy = dy;
    p.out = out;
    p.key = reinterpret_cast<uint32_t*>(w + L.key[cur]);
    p.pos = reinterpret_cast<uint32_t*>(w + L.pos[cur]);
    p.bitmap = reinterpret_cast<uint32_t*>(w + L.bitmap);
    p.word_prefix = sp.word_prefix;
    p.out_rows = out_rows;
    p.sparse = rows;
    p.out_count = out_count;
    p.head = reinterpret_cast<float*>(w + L.head);
    p.tail = reinterpret_cast<float*>(w + L.tail);
    for (int i = 0; i < 2; ++i) p.list[i] = reinterpret_cast<uint4*>(w + L.list[i]);
    p.list_count = reinterpret_cast<uint32_t*>(w + L.list_count);
    p.T = T;
    p.V = V;
    p.D = D;
    p.Dp = L.Dp;
    p.ld_dy = ld_dy;
    p.ld_out = ld_out;
    p.tiles = L.tiles;
    p.C = L.C;
    p.slabs = (int32_t)std::max<int64_t>(1, ceil_div64(D, EG_COLS));
    p.sum_blocks = L.tiles * p.slabs;
    p.accumulate = accumulate ? 1 : 0;
    p.scale = scale;
    if (direct) {
        DirectParams dp = {};
        dp.ids = ids;
        dp.ctrl = sp.ctrl;
        dp.padding = padding;
        dp.id64 = id_bytes == 8;
        p.slabs = (int32_t)std::max<int64_t>(1, ceil_div64(D, DR_COLS));
        p.sum_blocks = T * p.slabs;
        p.fill = zeros;
        dp.g = p;
        const int64_t blocks = p.sum_blocks + units;
        if (blocks > MAX_N) return TOPK_EF_ERR_INVALID_ARG;
        const bool vec = rows16(dy, ld_dy, sd) && rows16(out, ld_out, so);
        trace_before(st, "grad_direct_kernel");
        e = with_type(dy_type, [&](auto td) {
            return with_type(out_type, [&](auto to) {
                using TD = decltype(td);
                using TO = decltype(to);
                return vec ? launch_pdl(grad_direct_kernel<TD, TO, true>, (unsigned)blocks,
                                        DR_THREADS, st, dp)
                           : launch_pdl(grad_direct_kernel<TD, TO, false>, (unsigned)blocks,
                                        DR_THREADS, st, dp);
            });
        });
        trace_after(st);
        return e == cudaSuccess ? TOPK_EF_OK : cuda_fail(e);
    }
    p.fill = zeros;
    const int64_t grid = p.sum_blocks + units;
    if (grid > MAX_N) return TOPK_EF_ERR_INVALID_ARG;
    if (grid == 0) return TOPK_EF_OK;
    const bool vec = rows16(dy, ld_dy, sd) && rows16(out, ld_out, so);
    e = with_type(dy_type, [&](auto td) {
        return with_type(out_type, [&](auto to) {
            using TD = decltype(td);
            using TO = decltype(to);
            trace_before(st, "grad_sum_kernel");
            cudaError_t r =
                vec ? launch_pdl(grad_sum_kernel<TD, TO, true>, (unsigned)grid, EG_THREADS, st, p)
                    : launch_pdl(grad_sum_kernel<TD, TO, false>, (unsigned)grid, EG_THREADS, st, p);
            trace_after(st);
            if (r != cudaSuccess || L.tiles < 2) return r;
            // runs that cross tiles, and the columns of each that a block takes
            const int64_t most = (L.tiles - 1) * ceil_div64(D, EC_LONG_COLS);
            const int gc = (int)std::min<int64_t>(148 * 4, std::max<int64_t>(1, most));
            trace_before(st, "grad_combine_kernel");
            r = launch_pdl(grad_combine_kernel<TO>, gc, EC_THREADS, st, p);
            trace_after(st);
            return r;
        });
    });
    return e == cudaSuccess ? TOPK_EF_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

size_t embedding_lookup_workspace_bytes(void) { return align_up(sizeof(Ctrl)); }

int embedding_lookup(const void* weight, int32_t weight_type, int64_t ld_weight, const void* ids,
                     int32_t id_bytes, int64_t T, int64_t V, int64_t D, float scale, void* out,
                     int32_t out_type, int64_t ld_out, void* ws, size_t ws_bytes, void* stream) {
    const size_t sw = type_size(weight_type), so = type_size(out_type);
    if (!sizes_ok(T, V, D) || !sw || !so || (id_bytes != 4 && id_bytes != 8) || ld_weight < D ||
        ld_out < D || !ws || !aligned(ws, ALIGN))
        return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && (!ids || !aligned(ids, id_bytes))) return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && D > 0 && (!out || !aligned(out, so) || (V > 0 && (!weight || !aligned(weight, sw)))))
        return TOPK_EF_ERR_INVALID_ARG;
    if (T > 0 && V > 0 && D > 0 && out == weight) return TOPK_EF_ERR_INVALID_ARG;
    if (ws_bytes < embedding_lookup_workspace_bytes()) return TOPK_EF_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LookupParams p = {};
    p.w = weight;
    p.ids = ids;
    p.out = out;
    p.ctrl = static_cast<Ctrl*>(ws);
    p.T = T;
    p.V = V;
    p.D = D;
    p.ldw = ld_weight;
    p.ldo = ld_out;
    p.chunks = (int32_t)std::max<int64_t>(1, ceil_div64(D, LK_COLS));
    p.items = T * p.chunks;
    p.scan = T <= LK_SCAN_T;
    p.scale = scale;
    // a short list's ids are checked by one more block, which writes the
    // status; a long list's by the warps that read them, into a cleared word
    if (!p.scan) {
        const cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(Ctrl), st);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    const int64_t want = std::min<int64_t>(ceil_div64(p.items, LK_THREADS / 32), MAX_N / 2);
    const int grid = (int)std::max<int64_t>(1, want) + (p.scan ? 1 : 0);
    const bool vec = rows16(weight, ld_weight, sw) && rows16(out, ld_out, so);
    trace_before(st, "lookup_kernel");
    const cudaError_t e = with_type(weight_type, [&](auto tw) {
        return with_type(out_type, [&](auto to) {
            using TW = decltype(tw);
            using TO = decltype(to);
            if (id_bytes == 8)
                return vec ? launch_pdl(lookup_kernel<TW, TO, int64_t, true>, grid, LK_THREADS, st, p)
                           : launch_pdl(lookup_kernel<TW, TO, int64_t, false>, grid, LK_THREADS, st, p);
            return vec ? launch_pdl(lookup_kernel<TW, TO, int32_t, true>, grid, LK_THREADS, st, p)
                       : launch_pdl(lookup_kernel<TW, TO, int32_t, false>, grid, LK_THREADS, st, p);
        });
    });
    trace_after(st);
    return e == cudaSuccess ? TOPK_EF_OK : cuda_fail(e);
}

size_t embedding_grad_workspace_bytes(int64_t T, int64_t V, int64_t D) {
    return sizes_ok(T, V, D) ? grad_layout(T, V, D).total : 0;
}

int embedding_grad(const void* grad_out, int32_t grad_out_type, int64_t ld_grad_out,
                   const void* ids, int32_t id_bytes, int64_t T, int64_t V, int64_t D, float scale,
                   int64_t padding_idx, void* grad_weight, int32_t grad_weight_type,
                   int64_t ld_grad_weight, int32_t accumulate, void* ws, size_t ws_bytes,
                   void* stream) {
    return grad_call(grad_out, grad_out_type, ld_grad_out, ids, id_bytes, T, V, D, scale,
                     padding_idx, grad_weight, grad_weight_type, ld_grad_weight, accumulate,
                     nullptr, nullptr, false, ws, ws_bytes, stream);
}

int embedding_grad_rows(const void* grad_out, int32_t grad_out_type, int64_t ld_grad_out,
                        const void* ids, int32_t id_bytes, int64_t T, int64_t V, int64_t D,
                        float scale, int64_t padding_idx, int32_t* out_rows, void* out_val,
                        int32_t out_val_type, int64_t ld_out_val, int32_t* out_count, void* ws,
                        size_t ws_bytes, void* stream) {
    return grad_call(grad_out, grad_out_type, ld_grad_out, ids, id_bytes, T, V, D, scale,
                     padding_idx, out_val, out_val_type, ld_out_val, 0, out_rows, out_count, true,
                     ws, ws_bytes, stream);
}

}  // extern "C"
