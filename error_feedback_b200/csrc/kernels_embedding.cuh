// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   lookup:  out[t, :] = round(scale * W[id_t, :])
//   grad:    g[v, :]   = (accumulate ? g[v, :] : 0) + scale * sum_{t: id_t = v} dy[t, :]
//
// The gradient sorts the positions by id (stable, so the positions of one id
// stay in ascending order), cuts the sorted list into tiles of `C` positions
// and sums runs of equal ids inside each tile; a run that crosses tiles
// leaves one fp32 partial row per tile, which a last kernel adds in tile
// order.  The work of a tile does not depend on how often an id occurs, and
// the order of every sum is a function of the sizes alone: no floating-point
// atomics, results bit-identical from run to run.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "elements.cuh"

namespace tke {

// ------------------------------------------------------------------- lookup

constexpr int LK_THREADS = 128;
constexpr int LK_COLS = 1024;          // columns of one warp's item
constexpr int64_t LK_SCAN_T = 8192;    // up to here one block checks every id

struct LookupParams {
    const void* w;
    const void* ids;
    void* out;
    Ctrl* ctrl;
    int64_t T, V, D, ldw, ldo;
    int64_t items;                 // T * ceil(D / LK_COLS)
    int32_t chunks;                // ceil(D / LK_COLS)
    int32_t scan;                  // the last block checks the ids and writes the status
    float scale;
};

// One warp per (token, LK_COLS columns): bound by the bytes of the rows read
// and written (16,384 rows of 4,096 bf16: 37 us, 5.1 TB/s).  VEC: rows start on
// 16-byte boundaries on both sides.
template <typename TW, typename TO, typename TI, bool VEC>
__global__ void __launch_bounds__(LK_THREADS) lookup_kernel(const LookupParams p) {
    pdl_launch();
    pdl_wait();
    const TI* ids = static_cast<const TI*>(p.ids);
    int nblocks = (int)gridDim.x;
    if (p.scan) {
        --nblocks;
        if ((int)blockIdx.x == nblocks) {
            int bad = 0;
            for (int64_t t = threadIdx.x; t < p.T; t += LK_THREADS) {
                const int64_t id = (int64_t)ids[t];
                bad |= (id < 0 || id >= p.V);
            }
            bad = __syncthreads_or(bad);
            if (threadIdx.x == 0) {
                p.ctrl->path_small = 0;
                p.ctrl->status = bad ? ST_BAD_INPUT : 0u;
            }
            return;
        }
    }
    const TW* w = static_cast<const TW*>(p.w);
    TO* out = static_cast<TO*>(p.out);
    const int lane = (int)lane_id();
    const int64_t stride = (int64_t)nblocks * (LK_THREADS / 32);
    for (int64_t it = (int64_t)blockIdx.x * (LK_THREADS / 32) + warp_id(); it < p.items;
         it += stride) {
        const int64_t t = it / p.chunks;
        const int64_t c0 = (it - t * p.chunks) * LK_COLS;
        const int64_t id = (int64_t)ids[t];
        const bool ok = id >= 0 && id < p.V;
        if (!ok && !p.scan && lane == 0) atomicOr(&p.ctrl->status, ST_BAD_INPUT);
        const TW* src = w + (ok ? id : 0) * p.ldw;
        TO* dst = out + t * p.ldo;
        if (VEC) {
            Vec8<TW> v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t c = c0 + j * 256 + lane * 8;
                if (ok && c + 8 <= p.D) v[j] = load8(src + c);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t c = c0 + j * 256 + lane * 8;
                if (c + 8 <= p.D) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = ok ? p.scale * elem8(v[j], e) : 0.0f;
                    store8(dst + c, x);
                } else {
                    for (int64_t k = c; k < p.D; ++k)
                        dst[k] = from_f32<TO>(ok ? p.scale * to_f32(src[k]) : 0.0f);
                }
            }
        } else {
            // rows that start anywhere: one element a lane.  (Groups of four, aligned
            // in the output and shifted into place from aligned loads, take more
            // instructions than they save: 43 against 28 us for 30,011 rows of 1,001
            // fp32 to bf16.)
            const TW* s = src + c0 + lane;
            TO* d = dst + c0 + lane;
            const int n = (int)min((int64_t)LK_COLS, p.D - c0);
            int c = 0;
            for (; c + 256 <= n; c += 256) {
                TW v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (ok) v[j] = s[c + j * 32];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    d[c + j * 32] = from_f32<TO>(ok ? p.scale * to_f32(v[j]) : 0.0f);
            }
            TW v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (ok && c + j * 32 + lane < n) v[j] = s[c + j * 32];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j * 32 + lane < n)
                    d[c + j * 32] = from_f32<TO>(ok ? p.scale * to_f32(v[j]) : 0.0f);
        }
    }
}

// ------------------------------------------------- zeros of a dense gradient

// Rows of a dense gradient that no position names are written as zeros, in
// units of about 32 KB that any block of a call may take: the blocks of the
// sort, which leaves memory idle, take the first ones, the sums' the others.
constexpr int64_t FILL_BYTES = 32768;

struct Fill {
    char* out;
    const uint32_t* bitmap;        // ids that occur; null: every row is written
    int64_t V, row_bytes, stride_bytes;
    int64_t rows;                  // of one unit
    int64_t first;                 // unit of this launch's first filling block
    int32_t size;                  // of an element
};

__device__ __forceinline__ void zero_row(char* dst, int64_t bytes, int size, int lane) {
    int64_t done = 0;
    if ((uintptr_t)dst % 16 == 0) {
        done = bytes / 16;
        for (int64_t c = lane; c < done; c += 32)
            reinterpret_cast<uint4*>(dst)[c] = make_uint4(0, 0, 0, 0);
        done *= 16;
    }
    if (size == 4) {
        for (int64_t c = done / 4 + lane; c < bytes / 4; c += 32) reinterpret_cast<uint32_t*>(dst)[c] = 0;
    } else {
        for (int64_t c = done / 2 + lane; c < bytes / 2; c += 32) reinterpret_cast<uint16_t*>(dst)[c] = 0;
    }
}

// The unit of the `block`-th filling block of a launch.
__device__ __forceinline__ void fill_unit(const Fill& f, int64_t block) {
    const int64_t r0 = (f.first + block) * f.rows, r1 = min(f.V, r0 + f.rows);
    for (int64_t v = r0 + warp_id(); v < r1; v += blockDim.x / 32)
        if (!f.bitmap || !(f.bitmap[v >> 5] >> (v & 31) & 1u))
            zero_row(f.out + v * f.stride_bytes, f.row_bytes, f.size, (int)lane_id());
}

// ----------------------------------------------------- sort of the positions

// Least-significant-digit radix sort of (key, position), 9 bits a pass:
// counting and scattering kernels over tiles of 2,048 keys.  A key is the id,
// or V (which sorts last) for the padding id and for ids outside [0, V).  Bound by
// latency: the four launches for 131,072 positions take 30 us, each a chain of a
// few dependent loads in 64 blocks.
constexpr int ES_BITS = 9;
constexpr int ES_BINS = 1 << ES_BITS;
constexpr int ES_THREADS = 512;
constexpr int ES_WARPS = ES_THREADS / 32;
constexpr int ES_TILE = 2048;
constexpr int ES_ROUNDS = ES_TILE / ES_THREADS;     // keys per thread
constexpr int ES_WORDS = 256;
constexpr int ES_SCAN_TILES = 64;                   // more tiles: prefixes by their own kernel
static_assert(ES_BINS == ES_THREADS, "one thread per bin");

struct SortParams {
    const void* ids;               // first pass
    const uint32_t* key_in;        // later passes
    const uint32_t* pos_in;
    uint32_t* key_out;
    uint32_t* pos_out;
    uint32_t* counts;              // [tiles][ES_BINS]
    uint32_t* totals;              // [ES_BINS], when the prefixes are scanned ahead
    uint32_t* bitmap;              // ids that occur (first pass), or null
    uint32_t* word_prefix;         // ids that occur below each bitmap word (first pass), or null
    int32_t* out_count;            // their number (with word_prefix)
    Ctrl* ctrl;
    int64_t T, V, padding;
    int32_t tiles, shift, scanned;
    int32_t fill_from;             // blocks from this one on write zeros
    Fill fill;
};

template <typename TI>
__device__ __forceinline__ uint32_t sort_key(const TI* ids, int64_t t, int64_t V, int64_t padding,
                                             bool& bad) {
    const int64_t id = (int64_t)ids[t];
    const bool out = id < 0 || id >= V;
    bad = out && id != padding;
    return (out || id == padding) ? (uint32_t)V : (uint32_t)id;
}

__device__ __forceinline__ void set_bits(uint32_t* word, uint32_t bits) {
    if ((__ldcg(word) & bits) != bits) atomicOr(word, bits);
}

// Frequent ids would have every block set the same few words at once: each
// block gathers its bits in shared memory first, one word to a slot (a word
// whose slot another has taken goes to memory directly).
template <typename TI, bool FIRST>
__global__ void __launch_bounds__(ES_THREADS) sort_count_kernel(const SortParams p) {
    __shared__ uint32_t hist[ES_BINS];
    __shared__ uint32_t s_word[ES_WORDS], s_bits[ES_WORDS];
    pdl_launch();
    hist[threadIdx.x] = 0;
    if (FIRST && threadIdx.x < ES_WORDS) {
        s_word[threadIdx.x] = 0xFFFFFFFFu;
        s_bits[threadIdx.x] = 0;
    }
    pdl_wait();
    if (!FIRST && (int)blockIdx.x >= p.fill_from) {
        fill_unit(p.fill, (int)blockIdx.x - p.fill_from);
        return;
    }
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * ES_TILE;
#pragma unroll
    for (int r = 0; r < ES_ROUNDS; ++r) {
        const int64_t t = base + r * ES_THREADS + threadIdx.x;
        uint32_t key = 0;
        if (t < p.T) {
            if (FIRST) {
                bool bad;
                key = sort_key(static_cast<const TI*>(p.ids), t, p.V, p.padding, bad);
                if (bad) atomicOr(&p.ctrl->status, ST_BAD_INPUT);
                if (p.bitmap && key < (uint32_t)p.V) {
                    const uint32_t word = key >> 5, bit = 1u << (key & 31);
                    volatile uint32_t* slot = &s_word[word % ES_WORDS];
                    if (*slot == 0xFFFFFFFFu)
                        atomicCAS(&s_word[word % ES_WORDS], 0xFFFFFFFFu, word);
                    if (*slot == word) {
                        volatile uint32_t* bits = &s_bits[word % ES_WORDS];
                        if (!(*bits & bit)) atomicOr(&s_bits[word % ES_WORDS], bit);
                    } else {
                        set_bits(&p.bitmap[word], bit);
                    }
                }
            } else {
                key = p.key_in[t];
            }
        }
        // (frequent ids share their digits: one add for the lanes of a bin)
        warp_agg_inc(hist, (key >> p.shift) & (ES_BINS - 1), t < p.T);
    }
    __syncthreads();
    if (FIRST && p.bitmap && threadIdx.x < ES_WORDS && s_bits[threadIdx.x])
        set_bits(&p.bitmap[s_word[threadIdx.x]], s_bits[threadIdx.x]);
    p.counts[(int64_t)blockIdx.x * ES_BINS + threadIdx.x] = hist[threadIdx.x];
}

// counts -> exclusive prefixes over the tiles (in place) and totals, per bin;
// one block per 32 bins, its 32 warps over ranges of tiles.
__global__ void __launch_bounds__(1024) sort_prefix_kernel(const SortParams p) {
    __shared__ uint32_t part[32][33];
    pdl_launch();
    pdl_wait();
    const int bin = (int)blockIdx.x * 32 + (int)lane_id();
    const int per = (p.tiles + 31) / 32;
    const int t0 = min(p.tiles, (int)warp_id() * per), t1 = min(p.tiles, t0 + per);
    uint32_t s = 0;
    for (int t = t0; t < t1; ++t) s += p.counts[(int64_t)t * ES_BINS + bin];
    part[warp_id()][lane_id()] = s;
    __syncthreads();
    uint32_t run = 0;
    for (int w = 0; w < (int)warp_id(); ++w) run += part[w][lane_id()];
    for (int t = t0; t < t1; ++t) {
        const uint32_t c = p.counts[(int64_t)t * ES_BINS + bin];
        p.counts[(int64_t)t * ES_BINS + bin] = run;
        run += c;
    }
    if (warp_id() == 31) p.totals[bin] = run;
}

// Number of ids that occur below every 32-id word of the bitmap, and in all.
__device__ __forceinline__ void bitmap_prefix(const SortParams& p, uint32_t* s_red) {
    const int64_t words = ceil_div64(p.V, 32);
    constexpr int PER = 8;
    uint32_t run = 0;
    for (int64_t w0 = 0; w0 < words; w0 += ES_THREADS * PER) {
        const int64_t w = w0 + (int64_t)threadIdx.x * PER;
        uint32_t c[PER], sum = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            c[j] = w + j < words ? (uint32_t)__popc(__ldcg(&p.bitmap[w + j])) : 0u;
            sum += c[j];
        }
        uint32_t tot;
        uint32_t ex = run + block_excl_scan(sum, s_red, &tot);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (w + j < words) p.word_prefix[w + j] = ex;
            ex += c[j];
        }
        run += tot;
    }
    if (threadIdx.x == 0) *p.out_count = (int32_t)run;
}

// Stable scatter of one tile: the place of a key is the number of keys with a
// smaller digit, plus those of the same digit in earlier tiles, in earlier
// warps (each warp has a contiguous 128 keys) and earlier in this warp.
template <typename TI, bool FIRST>
__global__ void __launch_bounds__(ES_THREADS) sort_scatter_kernel(const SortParams p) {
    __shared__ __align__(16) uint32_t hist[ES_WARPS][ES_BINS];
    __shared__ uint32_t s_red[33];
    pdl_launch();
    const int tid = (int)threadIdx.x, lane = (int)lane_id(), warp = (int)warp_id();
    pdl_wait();
    if ((int)blockIdx.x >= p.fill_from) {
        fill_unit(p.fill, (int)blockIdx.x - p.fill_from);
        return;
    }
    if (FIRST && (int)blockIdx.x == p.tiles) {
        bitmap_prefix(p, s_red);
        return;
    }
    const int64_t base = (int64_t)blockIdx.x * ES_TILE + warp * (ES_TILE / ES_WARPS);
    uint32_t key[ES_ROUNDS], pos[ES_ROUNDS], rank[ES_ROUNDS];
#pragma unroll
    for (int r = 0; r < ES_ROUNDS; ++r) {
        const int64_t t = base + r * 32 + lane;
        key[r] = 0;
        pos[r] = (uint32_t)t;
        if (t < p.T) {
            if (FIRST) {
                bool bad;
                key[r] = sort_key(static_cast<const TI*>(p.ids), t, p.V, p.padding, bad);
            } else {
                key[r] = p.key_in[t];
                pos[r] = p.pos_in[t];
            }
        }
    }
    // first place of this thread's bin among this tile's keys
    uint32_t before = 0, total = 0;
    if (p.scanned) {
        before = p.counts[(int64_t)blockIdx.x * ES_BINS + tid];
        total = p.totals[tid];
    } else {
        // each quarter of the block sums every fourth tile, four bins a thread
        const int g = tid >> 7, q = tid & 127;
        uint4 tot = make_uint4(0, 0, 0, 0), bef = tot;
#pragma unroll 16
        for (int t = g; t < p.tiles; t += 4) {
            const uint4 c = *reinterpret_cast<const uint4*>(p.counts + t * ES_BINS + 4 * q);
            const uint32_t m = t < (int)blockIdx.x ? 0xFFFFFFFFu : 0u;
            tot.x += c.x;
            tot.y += c.y;
            tot.z += c.z;
            tot.w += c.w;
            bef.x += c.x & m;
            bef.y += c.y & m;
            bef.z += c.z & m;
            bef.w += c.w & m;
        }
        reinterpret_cast<uint4*>(hist[g])[q] = tot;
        reinterpret_cast<uint4*>(hist[4 + g])[q] = bef;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            total += hist[i][tid];
            before += hist[4 + i][tid];
        }
    }
    uint32_t all;
    before += block_excl_scan(total, s_red, &all);
#pragma unroll
    for (int w = 0; w < ES_WARPS; ++w) hist[w][tid] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ES_ROUNDS; ++r) {
        const bool live = base + r * 32 + lane < p.T;
        const uint32_t act = __ballot_sync(0xFFFFFFFFu, live);
        if (live) {
            const uint32_t d = (key[r] >> p.shift) & (ES_BINS - 1);
            const uint32_t peers = __match_any_sync(act, d);
            const int leader = __ffs(peers) - 1;
            uint32_t had = 0;
            if (lane == leader) {
                had = hist[warp][d];
                hist[warp][d] = had + (uint32_t)__popc(peers);
            }
            had = __shfl_sync(peers, had, leader);
            rank[r] = had + (uint32_t)__popc(peers & ((1u << lane) - 1u));
        }
        __syncwarp();
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < ES_WARPS; ++w) {
        const uint32_t c = hist[w][tid];
        hist[w][tid] = before;
        before += c;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ES_ROUNDS; ++r) {
        if (base + r * 32 + lane < p.T) {
            const uint32_t at = hist[warp][(key[r] >> p.shift) & (ES_BINS - 1)] + rank[r];
            p.key_out[at] = key[r];
            p.pos_out[at] = pos[r];
        }
    }
}

// ------------------------------------------------------------- short lists

// Up to SR_MAX positions are sorted by one kernel: every block counts, for
// its own keys, the keys that come before them among all (the whole list is
// read by every block; T^2 comparisons over all SMs; 2,048 positions in 4 us,
// where the radix sort's four launches take 20).  Whole calls by ranking and by
// radix, row-sparse, 768 columns: 18 and 37 us for 2,048 positions, 23 and 40 for
// 4,096, 42 and 50 for 8,192, where the list fills a block's static shared memory.
// Blocks after the ranking ones write the zeros of a dense gradient in the meantime.
constexpr int SR_THREADS = 512;
constexpr int SR_MAX = 8192;
constexpr int SR_SHARE = 16;           // threads of one key
constexpr int SR_KEYS = SR_THREADS / SR_SHARE;

struct RankParams {
    const void* ids;
    uint32_t* key;                 // sorted
    uint32_t* pos;
    uint32_t* list_count;
    Ctrl* ctrl;
    int64_t T, V, padding;
    int32_t rank_blocks;
    Fill fill;
};

template <typename TI>
__global__ void __launch_bounds__(SR_THREADS) rank_kernel(const RankParams p) {
    __shared__ __align__(16) uint32_t s_key[SR_MAX];
    pdl_launch();
    pdl_wait();
    const int tid = (int)threadIdx.x;
    if ((int)blockIdx.x >= p.rank_blocks) {
        fill_unit(p.fill, (int)blockIdx.x - p.rank_blocks);
        return;
    }
    const int T = (int)p.T, T4 = (T + 3) / 4;
    int bad_any = 0;
#pragma unroll 8
    for (int t = tid; t < T4 * 4; t += SR_THREADS) {
        bool bad = false;
        s_key[t] = t < T ? sort_key(static_cast<const TI*>(p.ids), t, p.V, p.padding, bad)
                         : 0xFFFFFFFFu;
        bad_any |= bad;
    }
    bad_any = __syncthreads_or(bad_any);
    if (blockIdx.x == 0 && tid == 0) {
        p.ctrl->path_small = 0;
        p.ctrl->status = bad_any ? ST_BAD_INPUT : 0u;
        p.list_count[0] = p.list_count[1] = 0;
    }
    // neighbouring threads share a key and take turns at the quadruples
    const int t = (int)blockIdx.x * SR_KEYS + tid / SR_SHARE, turn = tid % SR_SHARE;
    const uint32_t mine = t < T ? s_key[t] : 0;
    const uint4* all = reinterpret_cast<const uint4*>(s_key);
    uint32_t before = 0;
    // earlier positions come first among equals: key <= mine there, key < mine after
    const int split = min(t, T) / 4;
#pragma unroll 4
    for (int j = turn; j < split; j += SR_SHARE) {
        const uint4 k = all[j];
        before += (k.x <= mine) + (k.y <= mine) + (k.z <= mine) + (k.w <= mine);
    }
    if (turn < 4) {
        const int j = split * 4 + turn;
        if (j < T) before += j < t ? s_key[j] <= mine : s_key[j] < mine;
    }
#pragma unroll 4
    for (int j = split + 1 + turn; j < T4; j += SR_SHARE) {
        const uint4 k = all[j];
        before += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
    }
#pragma unroll
    for (int o = 1; o < SR_SHARE; o <<= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    if (t < T && turn == 0) {
        p.key[before] = mine;
        p.pos[before] = (uint32_t)t;
    }
}

// ------------------------------------------------------------------ the sums

constexpr int EG_THREADS = 128;
constexpr int EG_COLS = EG_THREADS * 8;    // columns of one block
constexpr int EG_MAX_C = 128;              // positions of one tile, at most
constexpr int EC_LONG = 16;                // a run over more tiles is added up by a whole block

struct GradParams {
    const void* dy;
    void* out;
    const uint32_t* key;           // sorted
    const uint32_t* pos;
    const uint32_t* bitmap;
    const uint32_t* word_prefix;   // row-sparse output: ordinals
    int32_t* out_rows;             // row-sparse output
    float* head;                   // [tiles][Dp]: run continued from the tile before
    float* tail;                   // [tiles][Dp]: run begun here that goes on in the next
    int32_t* out_count;            // (short list)
    uint4* list[2];                // tile whose tail goes on, the tail's row of out, its key:
    uint32_t* list_count;          //   short runs, long runs (EC_LONG tiles or more after it)
    int64_t T, V, D, Dp, ld_dy, ld_out;
    int64_t tiles;
    int64_t sum_blocks;            // tiles * slabs; the blocks after them fill with zeros
    int32_t slabs, C;
    int32_t accumulate, sparse;
    float scale;
    Fill fill;
};

// Row of the row-sparse output that holds `key`.
__device__ __forceinline__ int64_t ordinal(const GradParams& p, uint32_t key) {
    const uint32_t word = p.bitmap[key >> 5];
    return (int64_t)p.word_prefix[key >> 5] + __popc(word & ((1u << (key & 31)) - 1u));
}

// One block per (tile of C sorted positions, EG_COLS columns); thread j has 8
// columns: consecutive ones (VEC: rows on 16-byte boundaries), else one in
// every EG_THREADS.  Bound by the rows of dy read and the rows written: 131,072
// rows of 1,024 bf16 in 69 us, 5.4 TB/s.
template <typename TD, typename TO, bool VEC>
__global__ void __launch_bounds__(EG_THREADS, VEC && sizeof(TD) == 2 ? 10 : 8) grad_sum_kernel(const GradParams p) {
    __shared__ uint32_t s_key[EG_MAX_C + 2], s_pos[EG_MAX_C];
    __shared__ uint32_t s_red[33];
    pdl_launch();
    pdl_wait();
    const int tid = (int)threadIdx.x;
    if ((int64_t)blockIdx.x >= p.sum_blocks) {
        fill_unit(p.fill, (int64_t)blockIdx.x - p.sum_blocks);
        return;
    }
    const int64_t tile = (int64_t)blockIdx.x / p.slabs;
    const int64_t slab = (int64_t)blockIdx.x - tile * p.slabs;
    const int64_t start = tile * p.C;
    const int n = (int)min((int64_t)p.C, p.T - start);
    const uint32_t none = (uint32_t)p.V;       // key of positions that do not count
    for (int i = tid; i < n + 2; i += EG_THREADS) {
        const int64_t t = start + i - 1;
        s_key[i] = (t >= 0 && t < p.T) ? p.key[t] : 0xFFFFFFFFu;
        if (i < n) s_pos[i] = p.pos[start + i];
    }
    __syncthreads();
    // row-sparse output: the rows of this tile's runs follow one another
    int64_t row = 0;
    if (p.sparse) {
        if (p.word_prefix) {
            if (s_key[1] != none) row = ordinal(p, s_key[1]);
        } else {
            // short list: runs that begin before this tile, by counting
            uint32_t heads = 0;
#pragma unroll 8
            for (int t = tid; t <= (int)start; t += EG_THREADS)
                heads += t == 0 || p.key[t] != p.key[t - 1];
            row = (int64_t)block_sum(heads, s_red) - 1;
        }
    }
    const TD* dy = static_cast<const TD*>(p.dy);
    const int64_t c0 = slab * EG_COLS + (VEC ? tid * 8 : tid);
    auto col = [&](int j) { return c0 + (VEC ? j : j * EG_THREADS); };
    const bool whole = col(7) < p.D;
    float acc[8] = {};

    auto flush = [&](int i, bool first, bool goes_on) {   // the run that ends at position i
        const uint32_t k = s_key[i + 1];
        const bool from_before = first && s_key[0] == k;
        if (from_before || goes_on) {
            float* part = (from_before ? p.head : p.tail) + tile * p.Dp;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (whole || col(j) < p.D) part[col(j)] = acc[j];
            if (!from_before && slab == 0 && tid == 0) {
                const int64_t far = tile + EC_LONG;
                const int l = far < p.tiles && p.key[far * p.C] == k;
                p.list[l][atomicAdd(p.list_count + l, 1u)] =
                    make_uint4((uint32_t)tile, p.sparse ? (uint32_t)row : k, k, 0u);
            }
        } else {
            if (!p.sparse) row = k;
            TO* dst = static_cast<TO*>(p.out) + row * p.ld_out;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = p.scale * acc[j];
            if (VEC && whole) {
                if (p.accumulate) {
                    const Vec8<TO> o = load8(dst + c0);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] += elem8(o, j);
                }
                store8(dst + c0, y);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col(j) < p.D)
                        dst[col(j)] = from_f32<TO>(p.accumulate ? to_f32(dst[col(j)]) + y[j] : y[j]);
            }
        }
        if (p.sparse && !from_before && slab == 0 && tid == 0) p.out_rows[row] = (int32_t)k;
        ++row;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    };

    bool first = true;
    int i = 0;
    constexpr int U = 4;                       // rows in flight
    for (; i < n; i += U) {
        if (s_key[i + 1] == none) break;
        Vec8<TD> v[U];
        TD sv[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u >= n || s_key[i + u + 1] == none) continue;
            const TD* src = dy + (int64_t)s_pos[i + u] * p.ld_dy;
            if (VEC) {
                if (whole) {
                    v[u] = load8(src + c0);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        reinterpret_cast<TD*>(&v[u])[j] =
                            col(j) < p.D ? src[col(j)] : from_f32<TD>(0.0f);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sv[u][j] = col(j) < p.D ? src[col(j)] : from_f32<TD>(0.0f);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u >= n || s_key[i + u + 1] == none) continue;
            if (i + u > 0 && s_key[i + u + 1] != s_key[i + u]) {
                flush(i + u - 1, first, false);
                first = false;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += VEC ? elem8(v[u], j) : to_f32(sv[u][j]);
        }
    }
    // the last run of positions that count
    int m = n;
    while (m > 0 && s_key[m] == none) --m;
    if (m > 0) flush(m - 1, first, s_key[m] == s_key[m + 1]);
    // short list: the last run's block knows how many there are
    if (p.sparse && !p.word_prefix && slab == 0 && tid == 0 &&
        (m == n ? start + n == p.T : (m > 0 || start == 0 || s_key[0] != none)))
        *p.out_count = (int32_t)row;
}

constexpr int EC_THREADS = 512;
constexpr int EC_WARPS = EC_THREADS / 32;
constexpr int EC_COLS = 512;           // columns of a warp with a short run: 32 lanes x 4 x float4
constexpr int EC_LONG_COLS = 128;      // columns of a block with a long run: 32 lanes x float4

// The sum of partial rows [j0, j1) of the run that begins in `tile`: its tail,
// then the heads of the following tiles.
template <int N>
__device__ __forceinline__ void add_parts(const GradParams& p, int64_t tile, int64_t j0, int64_t j1,
                                          int64_t c, float4* s) {
#pragma unroll
    for (int u = 0; u < N; ++u) s[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll (N == 1 ? 8 : 4)
    for (int64_t j = j0; j < j1; ++j) {
        const float* part = (j == 0 ? p.tail : p.head) + (tile + j) * p.Dp + c;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            if (c + u * 128 >= p.D) continue;
            const float4 x = *reinterpret_cast<const float4*>(part + u * 128);
            s[u].x += x.x;
            s[u].y += x.y;
            s[u].z += x.z;
            s[u].w += x.w;
        }
    }
}

template <typename TO, int N>
__device__ __forceinline__ void put_row(const GradParams& p, int64_t row, int64_t c, const float4* s) {
    TO* dst = static_cast<TO*>(p.out) + row * p.ld_out + c;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const float y[4] = {p.scale * s[u].x, p.scale * s[u].y, p.scale * s[u].z, p.scale * s[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = u * 128 + j;
            if (c + k < p.D) dst[k] = from_f32<TO>(p.accumulate ? to_f32(dst[k]) + y[j] : y[j]);
        }
    }
}

// Number of tiles that the run of key k touches from `tile` on, by probes of the
// first keys of tiles, one per thread at a time: first of the next tiles, then
// ever finer between the last hit and the first miss.  BLOCK: by the whole
// block, else by a warp.
template <bool BLOCK>
__device__ __forceinline__ int64_t run_tiles(const GradParams& p, int64_t tile, uint32_t k) {
    constexpr int W = BLOCK ? EC_THREADS : 32;
    const int id = BLOCK ? (int)threadIdx.x : (int)lane_id();
    int64_t hit = tile, miss = p.tiles;
    for (int64_t step = 1; miss - hit > 1;) {
        const int64_t at = hit + (id + 1) * step;
        const bool in = at < miss && p.key[at * p.C] == k;
        const int n = BLOCK ? __syncthreads_count(in)            // (hits come first)
                            : __popc(__ballot_sync(0xFFFFFFFFu, in));
        if (n < W) miss = min(miss, hit + (n + 1) * step);
        hit += n * step;
        step = max((int64_t)1, (miss - hit) / W);
    }
    return hit - tile + 1;
}

// Adds the partial rows of every run that crosses tiles, in tile order.  Long
// runs (a frequent id): a block takes 128 columns, its warps contiguous parts
// of the run, and their sums are added in order.  Short ones, two or three
// partial rows as a rule: a warp takes 512 columns.  Bound by latency (list, key,
// probes, partial rows): 16 us for 1,407 runs of up to 242 partial rows.
template <typename TO>
__global__ void __launch_bounds__(EC_THREADS) grad_combine_kernel(const GradParams p) {
    __shared__ float4 s_part[EC_WARPS][32];
    pdl_launch();
    pdl_wait();
    const int lane = (int)lane_id(), warp = (int)warp_id();
    const int64_t long_slabs = ceil_div64(p.D, EC_LONG_COLS);
    const int64_t long_items = (int64_t)p.list_count[1] * long_slabs;
    for (int64_t it = blockIdx.x; it < long_items; it += gridDim.x) {
        const int64_t run = it / long_slabs, c = (it - run * long_slabs) * EC_LONG_COLS + lane * 4;
        const uint4 entry = p.list[1][run];
        const int64_t parts = run_tiles<true>(p, entry.x, entry.z), per = ceil_div64(parts, EC_WARPS);
        float4 s;
        add_parts<1>(p, entry.x, min(parts, warp * per), min(parts, (warp + 1) * per), c, &s);
        s_part[warp][lane] = s;
        __syncthreads();
        if (warp == 0) {
            const int used = (int)ceil_div64(parts, per);
            for (int q = 1; q < used; ++q) {
                const float4 x = s_part[q][lane];
                s.x += x.x;
                s.y += x.y;
                s.z += x.z;
                s.w += x.w;
            }
            put_row<TO, 1>(p, entry.y, c, &s);
        }
        __syncthreads();
    }
    const int64_t slabs = ceil_div64(p.D, EC_COLS);
    const int64_t items = (int64_t)p.list_count[0] * slabs;
    // (from the last block on: the first ones have had the long runs)
    for (int64_t it = (int64_t)(gridDim.x - 1 - blockIdx.x) * EC_WARPS + warp; it < items;
         it += (int64_t)gridDim.x * EC_WARPS) {
        const int64_t run = it / slabs, c = (it - run * slabs) * EC_COLS + lane * 4;
        const uint4 entry = p.list[0][run];
        float4 s[4];
        add_parts<4>(p, entry.x, 0, run_tiles<false>(p, entry.x, entry.z), c, s);
        put_row<TO, 4>(p, entry.y, c, s);
    }
}

// -------------------------------------------------- a few tokens: one kernel

// Up to DR_MAX positions: a block per (position, DR_COLS columns).  Every block
// reads the whole list; the block of an id's first position sums the id's rows:
// the warps take contiguous parts of them, and their sums are added in order.
// One launch of independent blocks instead of three chained ones: 500 positions
// of 1,024 columns in 6.2 us on the GPU against 15.  Whole calls by one kernel (with
// room for 1,024 positions) and by three, at 512, 768 and 1,024 positions: added to
// rows of 1,024 columns 8, 11 and 14 us against 15, 16 and 17, to rows of 4,096 23,
// 33 and 43 against 17, 18 and 19, row-sparse with 768 columns 12, 18 and 25 against
// 13, 14 and 14.
constexpr int DR_THREADS = 128;
constexpr int DR_WARPS = DR_THREADS / 32;
constexpr int DR_MAX = 512;
constexpr int DR_COLS = 256;
constexpr int DR_TABLE = 2 * DR_MAX;       // distinct ids, open addressing
constexpr int DR_FILL_ROWS = 2048;         // rows of one fill block, at most

struct DirectParams {
    GradParams g;                  // (dy, out, out_rows, out_count, sizes, strides, scale)
    const void* ids;
    Ctrl* ctrl;
    int64_t padding;
    int32_t id64;
};

template <typename TD, typename TO, bool VEC>
__global__ void __launch_bounds__(DR_THREADS) grad_direct_kernel(const DirectParams p) {
    __shared__ uint32_t s_key[DR_MAX], s_same[DR_MAX / 32], s_list[DR_MAX], s_red[33];
    __shared__ uint32_t s_table[DR_TABLE];
    __shared__ __align__(16) float s_part[DR_WARPS][DR_COLS];
    __shared__ int s_n;
    pdl_launch();
    const int tid = (int)threadIdx.x, lane = (int)lane_id(), warp = (int)warp_id();
    const GradParams& g = p.g;
    const int T = (int)g.T;
    const uint32_t none = (uint32_t)g.V;
    pdl_wait();
    int bad_any = 0;
#pragma unroll
    for (int j = 0; j < DR_MAX / DR_THREADS; ++j) {
        const int i = j * DR_THREADS + tid;
        bool bad = false;
        uint32_t k = none;
        if (i < T)
            k = p.id64 ? sort_key(static_cast<const int64_t*>(p.ids), i, g.V, p.padding, bad)
                       : sort_key(static_cast<const int32_t*>(p.ids), i, g.V, p.padding, bad);
        s_key[i] = k;
        bad_any |= bad;
    }
    if (g.sparse)
        for (int i = tid; i < DR_TABLE; i += DR_THREADS) s_table[i] = none;
    bad_any = __syncthreads_or(bad_any);

    if ((int64_t)blockIdx.x >= g.sum_blocks) {
        // rows of a dense gradient that no position names
        __shared__ uint32_t s_named[DR_FILL_ROWS / 32];
        for (int i = tid; i < DR_FILL_ROWS / 32; i += DR_THREADS) s_named[i] = 0;
        __syncthreads();
        const int64_t r0 = ((int64_t)blockIdx.x - g.sum_blocks) * g.fill.rows;
        const int64_t r1 = min(g.V, r0 + g.fill.rows);
        for (int i = tid; i < T; i += DR_THREADS) {
            const int64_t k = s_key[i];
            if (k >= r0 && k < r1) atomicOr(&s_named[(k - r0) >> 5], 1u << ((k - r0) & 31));
        }
        __syncthreads();
        for (int64_t v = r0 + warp; v < r1; v += DR_WARPS)
            if (!(s_named[(v - r0) >> 5] >> ((v - r0) & 31) & 1u))
                zero_row(g.fill.out + v * g.fill.stride_bytes, g.fill.row_bytes, g.fill.size, lane);
        return;
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.ctrl->path_small = 0;
        p.ctrl->status = bad_any ? ST_BAD_INPUT : 0u;
    }
    const int t = (int)(blockIdx.x / (unsigned)g.slabs);
    const int slab = (int)(blockIdx.x - (unsigned)t * (unsigned)g.slabs);
    const uint32_t mine = s_key[t];
    int earlier = 0;
#pragma unroll
    for (int j = 0; j < DR_MAX / DR_THREADS; ++j) {
        const int i = j * DR_THREADS + tid;
        const bool same = i < T && s_key[i] == mine;
        earlier |= same && i < t;
        const uint32_t word = __ballot_sync(0xFFFFFFFFu, same);
        if (lane == 0) s_same[i >> 5] = word;
    }
    earlier = __syncthreads_or(earlier);
    const bool counts = g.sparse && blockIdx.x == 0;     // writes the number of ids
    const bool sums = !earlier && mine != none;
    if (!sums && !counts) return;

    // row-sparse output: ids below this one, and in all, by a table of distinct ids
    int64_t row = mine;
    if (g.sparse) {
        for (int i = tid; i < T; i += DR_THREADS) {
            const uint32_t k = s_key[i];
            if (k == none) continue;
            uint32_t at = (k * 2654435761u) >> 16 & (DR_TABLE - 1);
            for (;; at = (at + 1) & (DR_TABLE - 1)) {       // (never full)
                const uint32_t was = atomicCAS(&s_table[at], none, k);
                if (was == none || was == k) break;
            }
        }
        __syncthreads();
        uint32_t below = 0, all = 0;
        for (int i = tid; i < DR_TABLE; i += DR_THREADS) {
            all += s_table[i] != none;
            below += s_table[i] < mine;                     // (none is above every id)
        }
        row = block_sum(below, s_red);
        all = block_sum(all, s_red);
        if (counts && tid == 0) *g.out_count = (int32_t)all;
        if (!sums) return;
        if (slab == 0 && tid == 0) g.out_rows[row] = (int32_t)mine;
    }
    if (warp == 0) {
        const uint32_t word = lane < DR_MAX / 32 ? s_same[lane] : 0;
        uint32_t at = warp_incl_scan((uint32_t)__popc(word));
        if (lane == 31) s_n = (int)at;
        at -= __popc(word);
        for (uint32_t w = word; w; w &= w - 1) s_list[at++] = lane * 32 + __ffs(w) - 1;
    }
    __syncthreads();
    const int n = s_n, per = (n + DR_WARPS - 1) / DR_WARPS;
    const int i0 = min(n, warp * per), i1 = min(n, i0 + per);
    const TD* dy = static_cast<const TD*>(g.dy);
    const int64_t c0 = (int64_t)slab * DR_COLS + (VEC ? lane * 8 : lane);
    auto col = [&](int j) { return c0 + (VEC ? j : j * 32); };
    const bool whole = col(7) < g.D;
    float acc[8] = {};
    constexpr int U = 4;                                    // rows in flight
    for (int i = i0; i < i1; i += U) {
        Vec8<TD> v[U];
        TD sv[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u >= i1) continue;
            const TD* src = dy + (int64_t)s_list[i + u] * g.ld_dy;
            if (VEC && whole) {
                v[u] = load8(src + c0);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) sv[u][j] = col(j) < g.D ? src[col(j)] : from_f32<TD>(0.0f);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u >= i1) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += VEC && whole ? elem8(v[u], j) : to_f32(sv[u][j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s_part[warp][VEC ? lane * 8 + j : lane + j * 32] = acc[j];
    __syncthreads();
    if (warp != 0) return;
    const int used = (n + per - 1) / per;
    for (int w = 1; w < used; ++w)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += s_part[w][VEC ? lane * 8 + j : lane + j * 32];
    TO* dst = static_cast<TO*>(g.out) + row * g.ld_out;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = g.scale * acc[j];
    if (VEC && whole) {
        if (g.accumulate) {
            const Vec8<TO> o = load8(dst + c0);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] += elem8(o, j);
        }
        store8(dst + c0, y);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col(j) < g.D)
                dst[col(j)] = from_f32<TO>(g.accumulate ? to_f32(dst[col(j)]) + y[j] : y[j]);
    }
}

}  // namespace tke
