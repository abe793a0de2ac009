// attn_seq.cuh -- sequences over a paged cache as the attention kernels see
// them: their work as one list of key tiles, cut into equal runs.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attn_common.cuh"
#include "fb_internal.cuh"
#include "tensor_core.cuh"

namespace fb {

struct TreeArgs {
    const void *q, *kc, *vc;
    void *out;
    float *lse;
    const int32_t *table, *lens, *cu;
    const uint64_t *mask;
    float *part, *part_ml;
    int4 *records;
    unsigned int *errors;
    int n, T, Hkv, group, ldq, ldo, table_width, ld_table, max_draft, pages, page_shift;
    int whole;   // items are not cut: a run is of items
    int tile_tokens;   // drafted tokens of a tensor-core tile: 128 / group of them, whole groups of rows
    float scale_log2;
};

constexpr int kMinTiles = 2;       // key tiles of a run, at least
constexpr int kTreeTileRows = 256; // rows of an item on the tensor cores: two tiles of 128

// The drafted token of row `local` of tile s of a block of two (-1: none); its head in the group is local % group.
__device__ __forceinline__ int tile_token(const TreeArgs &a, int block, int s, int local, int m) {
    const int t = local / a.group, token = (2 * block + s) * a.tile_tokens + t;
    return t < a.tile_tokens && token < m ? token : -1;
}

// One sequence: its tokens, its keys and its work.
struct Seq {
    int first, m, len, tiles, row_tiles;
    bool too_many;
};

// In row tiles of ROWS and key tiles of KEYS.
template <int ROWS, int KEYS>
__device__ __forceinline__ Seq sequence(const TreeArgs &a, int s) {
    Seq q;
    int first = s, end = s + 1;
    if (a.cu) {
        first = min(max(a.cu[s], 0), a.T);
        end = min(max(a.cu[s + 1], first), a.T);
    }
    q.first = first;
    q.too_many = end - first > a.max_draft;
    q.m = min(end - first, a.max_draft);
    // more committed keys than the table has room for: one beyond it is enough to make every row NaN
    const int64_t room = min(((int64_t)a.table_width << a.page_shift) + 1, (int64_t)INT32_MAX - 256);
    q.len = (int)min((int64_t)max(a.lens[s], 0), room);
    q.tiles = max(1, (q.len + q.m + KEYS - 1) / KEYS);
    if constexpr (ROWS == kTreeTileRows) q.row_tiles = (q.m + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
    else q.row_tiles = (q.m * a.group + ROWS - 1) / ROWS;
    return q;
}

// A place in the list of key tiles.
struct Cursor {
    Seq q;
    int s, item, kt;   // item = key head * row tiles + row tile
    int64_t pos;       // behind the run's beginning
};

template <int ROWS, int KEYS, int kPiece>
__device__ __forceinline__ void step(const TreeArgs &a, Cursor &c) {
    if (!a.whole) ++c.pos;
    if (++c.kt < c.q.tiles) return;
    c.kt = 0;
    c.pos += a.whole ? 1 : kPiece;
    if (++c.item < c.q.row_tiles * a.Hkv) return;
    c.item = 0;
    do {
        if (++c.s >= a.n) return;
        c.q = sequence<ROWS, KEYS>(a, c.s);
    } while (c.q.row_tiles == 0);
}

// What a warp has to do of the whole list: `run` tiles for each CTA of the grid (an item counting kPiece
// more, for what starting and ending it costs), this one's from `begin` on, `span` of them.
struct Run {
    int64_t run, begin, span;
};
template <int ROWS, int KEYS, int kPiece>
__device__ __forceinline__ Run find_run(const TreeArgs &a, Cursor &at) {
    const int lane = threadIdx.x % 32;
    auto weight = [&](int s) {
        const Seq q = sequence<ROWS, KEYS>(a, s);
        if (q.too_many && blockIdx.x == 0) atomicOr(a.errors, kErrorInput);
        return (int64_t)q.row_tiles * a.Hkv * (a.whole ? 1 : q.tiles + kPiece);
    };
    int64_t total = 0;
    for (int s = lane; s < a.n; s += 32) total += weight(s);
#pragma unroll
    for (int x = 16; x; x >>= 1) total += __shfl_xor_sync(~0u, total, x);
    Run r;
    r.run = max((total + gridDim.x - 1) / gridDim.x, (int64_t)(a.whole ? 1 : kMinTiles + kPiece));
    r.begin = r.run * blockIdx.x, r.span = min(r.run, total - r.begin);
    if (r.span <= 0) return r;
    int64_t before = 0;
    int base = 0;
    for (; base < a.n; base += 32) {
        const int64_t w = base + lane < a.n ? weight(base + lane) : 0;
        int64_t upto = w;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, upto, x);
            if (lane >= x) upto += y;
        }
        const unsigned past = __ballot_sync(~0u, before + upto > r.begin);
        if (past) {
            const int l = __ffs(past) - 1;
            at.s = base + l;
            before += __shfl_sync(~0u, upto - w, l);
            break;
        }
        before += __shfl_sync(~0u, upto, 31);
    }
    if (base >= a.n) {   // only if the lengths changed under the call: no work, rather than a search without end
        r.span = 0;
        return r;
    }
    at.q = sequence<ROWS, KEYS>(a, at.s);
    if (a.whole) {
        at.item = (int)(r.begin - before);
        at.kt = 0, at.pos = 0;
        return r;
    }
    const int length = at.q.tiles + kPiece;
    at.item = (int)((r.begin - before) / length);
    at.kt = (int)((r.begin - before) % length) - kPiece;   // an item's tiles come behind its start
    at.pos = at.kt < 0 ? -at.kt : 0;
    at.kt = max(at.kt, 0);
    return r;
}

// Values of 16 bits, in pairs.
template <typename E>
__device__ __forceinline__ bool not_finite(uint32_t two) {
    constexpr uint32_t e = std::is_same_v<E, __half> ? 0x7C00u : 0x7F80u;
    return (two & e) == e || (two >> 16 & e) == e;
}
template <typename E>
__device__ __forceinline__ uint32_t finite_part(uint32_t two) {
    constexpr uint32_t e = std::is_same_v<E, __half> ? 0x7C00u : 0x7F80u;
    if ((two & e) == e) two &= 0xFFFF0000u;
    if ((two >> 16 & e) == e) two &= 0x0000FFFFu;
    return two;
}

// Trees with many rows a key head, on the tensor cores: pages of at least 8 rows, groups of at most 128; one CTA
// an SM, partial results of kTreeTileRows rows.
cudaError_t launch_tree_tiles(const TreeArgs &a, const fb_kv_cache &cache, bool pdl, cudaStream_t s);

// [page][head][row][D] in boxes of 64 columns and `rows` rows of a page.
inline bool cache_map(CUtensorMap *map, void *base, const fb_kv_cache &c, int rows) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t row = (cuuint64_t)c.D * 2, head = row * c.page_size;
    const cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)c.page_size, (cuuint64_t)c.Hkv, (cuuint64_t)c.pages};
    const cuuint64_t strides[3] = {row, head, head * c.Hkv};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, steps[4] = {1, 1, 1, 1};
    return f(map, c.t == FB_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims,
             strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace fb
