// attn_tiles.cuh -- attention on the tensor cores in tiles of 128 queries and 128
// keys: of packed prompts, and of drafted trees over a paged cache.
//
//   out_i = sum_j exp(scale q_i.k_j - m_i) v_j / sum_j exp(scale q_i.k_j - m_i)
//
// over the keys j that row i sees, in one pass over the keys with a running maximum m and sum.  An item is 256
// queries of one head (of one key head, over a cache): two tiles of 128 rows that share every tile of 128 keys
// and take turns, so that the tensor cores multiply for one while the other's
// exponentials are taken.  Per 128 keys and 256 queries the products take 4 x
// 128 x 128 x D multiply-adds, 2,048 cycles of one SM at D = 128, and the 32,768
// exponentials just as many of its special-function units: both bound the
// kernel, and everything else has to fit beside them.
//
//   warps 0-3, 4-7   one tile of queries each, one row a thread: scores from
//                    tensor memory, maximum, exponentials, sum, rounded weights
//                    back over the scores; at the end the output
//   warp 8           finds the items and issues the copies (queries once, keys
//                    and values through a ring of tiles)
//   warp 9           issues the products: S = Q K^T from shared memory, O += P V
//                    with P from tensor memory
//   warps 10, 11     clear infinities and NaN from the value tiles that some row
//                    of the item must not see (those on the diagonal, or with drafted keys): a weight
//                    of zero would not stop them.  They note the rows, and the
//                    rows that do see them add them at the end.
//
// Tensor memory: two score tiles of 128 columns, each overwritten by its
// weights (64 columns), and two outputs of D columns.  The products are issued
// by one thread and complete in order, so a new score tile may be asked for as
// soon as the product that reads the old weights has been issued.  The weights
// come in two halves, so that the product starts before the second is there.
//
// Measured (16,384 tokens, 32 heads over 8 of 128, bf16): 1.69 ms, 1.30 PFLOP/s (once after a rest; back to back the
// power cap makes it 1.93), tensor cores 66% busy; a step of 128 keys and 256 queries takes 3,250 cycles:
// the chain of one tile (scores, 1,950 cycles of softmax, product, scores) is
// what two tiles in turn do not quite hide.  K and V come from L2 (5.5 GB a
// launch), not from HBM.
//
// The outputs are rescaled only when a row's maximum has grown by more than
// 2^8 since the last time (exact all the same: the sum carries the same factor,
// and weights that much larger fit either type), which few tiles need.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "attn_common.cuh"
#include "attn_seq.cuh"
#include "fb_internal.cuh"
#include "tensor_core.cuh"

namespace fb {

constexpr int kTile = 128;                 // queries of a tile, keys of a tile
constexpr int kBlock = 2 * kTile;          // queries of an item
constexpr int kTileThreads = 384;
constexpr int kColumns = 512;              // all of tensor memory
constexpr int kItems = 2;                  // items known at a time
constexpr int kItemReaders = 8 + 1 + 2;    // warps that read an item
// Registers a thread: at the launch, then of the softmax warps and of the others; the shares of the
// eight and the four warps add up to the launch's.
constexpr int kLaunchRegisters = 168, kManyRegisters = 208, kFewRegisters = 88;
static_assert(8 * kManyRegisters + 4 * kFewRegisters == 12 * kLaunchRegisters, "registers are moved, not made");

template <int D>
constexpr int kTileBytes = kTile * D * 2;
template <int D>
constexpr int kRing = D == 128 ? 5 : 8;    // key and value tiles in shared memory, beside the queries
template <int D>
constexpr int kSmemBytes = (2 + kRing<D>) * kTileBytes<D> + 1024;

struct PromptArgs {
    const void *v;
    void *out;
    float *lse;
    const int32_t *cu;
    unsigned int *errors;
    int n, T, Hq, group, ldv, ldo;
    float scale_log2;
};

// Few items for the CTAs: an item is one tile of queries, and the two tiles' places take its key tiles in turn
// (even ones, odd ones), which halves the longest item; their results are joined in tensor memory at the end.
struct SplitArgs : PromptArgs {};

struct Item {
    int n[2];                      // tiles of keys that the two query tiles meet; n[0] 0: no more items
    int first, len, block, head;   // the sequence's first token and (committed) length; the block of 256 rows; the
                                   // query head, or over a cache the key head
    int clean_from;                // first of the item's key tiles in which some row must not see some key
    int seq, m, kt0, piece;        // over a cache: sequence, drafted tokens, first key tile, place of a partial result (-1)
    uint32_t odd[2][4];            // rows of the tiles from there on whose values are not all finite
};

struct Barriers {
    uint64_t q_full[2], q_free[2];          // the query tiles
    uint64_t full[8], free_[8], clean[8], ask[8];   // the ring
    uint64_t s_full[2], p_full[2][2], o_full[2];   // the weights by halves of the keys
    uint64_t item_full[kItems], item_free[kItems];
    uint64_t merge_full, merge_free;        // the second half of a split item there, read
    uint64_t done;
};

static_assert(kBlock == kTreeTileRows, "the join reads the blocks' rows");

// What starting and ending an item costs, in key tiles.
constexpr int kTilePiece = 3;

// Args: PromptArgs or SplitArgs for packed prompts, TreeArgs for drafted trees over a paged cache (rows: the drafted tokens
// times the query heads of a key head).
template <typename E, int D, typename Args>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const Args a, const __grid_constant__ CUtensorMap q_map,
                  const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    constexpr int R = kRing<D>;
    constexpr bool kCache = std::is_same_v<Args, TreeArgs>, kSplit = std::is_same_v<Args, SplitArgs>;
    constexpr int kRows = kSplit ? kTile : kBlock;   // of an item
    constexpr bool kBf16 = std::is_same_v<E, __nv_bfloat16>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Barriers bars;
    __shared__ Item items[kItems];
    __shared__ float2 merge_ml[kSplit ? kTile : 1];   // maxima and sums of the second half
    __shared__ uint32_t tmem_at;
    __shared__ int gave_up_word;
    volatile int *gave_up = &gave_up_word;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t tiles = (smem_address(smem_raw) + 1023) & ~1023u;   // q0, q1, ring
    const uint32_t ring = tiles + 2 * kTileBytes<D>;
    auto bar = [&](const uint64_t &b) { return smem_address(&b); };
    auto wait = [&](const uint64_t &b, uint32_t parity) { return barrier_wait(smem_address(&b), parity, gave_up); };
    // the same for all 32 lanes, which go on or give up together
    auto warp_wait = [&](const uint64_t &b, uint32_t parity) { return (bool)__all_sync(~0u, wait(b, parity)); };

    if (tid == 0) {
        gave_up_word = 0;
        for (int i = 0; i < 2; ++i) {
            barrier_init(bar(bars.q_full[i]), 1), barrier_init(bar(bars.q_free[i]), 1);
            barrier_init(bar(bars.p_full[i][0]), 4), barrier_init(bar(bars.p_full[i][1]), 4);
            barrier_init(bar(bars.s_full[i]), 1), barrier_init(bar(bars.o_full[i]), 1);
        }
        for (int i = 0; i < R; ++i) {
            barrier_init(bar(bars.full[i]), 1), barrier_init(bar(bars.free_[i]), 1);
            barrier_init(bar(bars.clean[i]), 2), barrier_init(bar(bars.ask[i]), 1);
        }
        for (int i = 0; i < kItems; ++i)
            barrier_init(bar(bars.item_full[i]), 1), barrier_init(bar(bars.item_free[i]), kItemReaders);
        barrier_init(bar(bars.merge_full), 4), barrier_init(bar(bars.merge_free), 4);
        barrier_init(bar(bars.done), 1);
        barrier_inits_done();
    }
    if (warp == 9) tmem_alloc(smem_address(&tmem_at), kColumns);
    tensor_fence_before();
    __syncthreads();
    tensor_fence_after();
    const uint32_t tmem = tmem_at;
    wait_for_previous_kernel();

    // Registers move by warpgroups: the four warps of one execute the same instruction, before their roles part.
    if (warp >= 8) {
        give_registers<kFewRegisters>();
        if (warp == 8) {
            // ---- items and copies -----------------------------------------------------
            if constexpr (kCache) {
                // A run of the list of key tiles, piece by piece.  The whole warp takes part: each lane looks up the
                // page of its box (page_size keys, at most a tile) and copies it.
                Cursor c;
                const Run r = find_run<kBlock, kTile, kTilePiece>(a, c);
                if (lane == 0) a.records[blockIdx.x] = make_int4(0, 0, 0, 0);
                const int box = min(1 << a.page_shift, kTile), boxes = kTile / box;
                uint32_t loads = 0, q_uses[2] = {0, 0};
                bool more = r.span > 0;
                for (uint32_t count = 0;; ++count) {
                    const int slot = count % kItems;
                    if (!warp_wait(bars.item_free[slot], (count / kItems & 1) ^ 1)) break;
                    Item it = {};
                    int kt1 = 0, hk = 0;
                    if (more) {
                        const Seq &q = c.q;
                        const int rt = c.item % q.row_tiles;
                        hk = c.item / q.row_tiles;
                        kt1 = (int)min((int64_t)q.tiles, c.kt + r.span - c.pos);
                        const bool whole = c.kt == 0 && kt1 == q.tiles;
                        it.n[0] = kt1 - c.kt, it.n[1] = (2 * rt + 1) * a.tile_tokens < q.m ? kt1 - c.kt : 0;
                        it.first = q.first, it.len = q.len, it.block = rt, it.head = hk;
                        it.clean_from = max(q.len / kTile - c.kt, 0);
                        it.seq = c.s, it.m = q.m, it.kt0 = c.kt;
                        it.piece = whole ? -1 : 2 * (int)blockIdx.x + (c.kt == 0 ? 1 : 0);
                        if (!whole && c.kt == 0 && lane == 0) {
                            // where a cut item begins, the join learns where it lies and in which CTA it ends
                            const int64_t end = c.pos + q.tiles;
                            a.records[blockIdx.x] = make_int4((int)((r.begin + end - 1) / r.run) + 1, q.first, c.item,
                                                              q.m | q.row_tiles << 16);
                        }
                    }
                    if (lane == 0) {
                        items[slot] = it;
                        barrier_arrive(bar(bars.item_full[slot]));
                    }
                    __syncwarp();
                    if (!more) break;
                    const int keys = it.len + it.m;
                    auto load_query = [&](int s) {
                        if (!warp_wait(bars.q_free[s], (q_uses[s] & 1) ^ 1)) return false;
                        ++q_uses[s];
                        if (lane == 0) {
                            barrier_expect(bar(bars.q_full[s]), a.tile_tokens * a.group * D * 2);
                            for (int x = 0; x < D / 64; ++x)
                                tile_copy(tiles + s * kTileBytes<D> + x * (kTile * 128), &q_map, 64 * x, hk * a.group,
                                          it.first + (2 * it.block + s) * a.tile_tokens, bar(bars.q_full[s]));
                        }
                        __syncwarp();
                        return true;
                    };
                    auto load_ring = [&](const CUtensorMap *map, int j, bool ask) {
                        const int place = loads % R, p = (it.kt0 + j) * kTile + lane * box;
                        const bool wanted = lane < boxes && p < keys;
                        const int at = p >> a.page_shift;
                        const int page = wanted && at < a.table_width ? a.table[(size_t)it.seq * a.ld_table + at] : -1;
                        const bool good = wanted && page >= 0 && page < a.pages;
                        if (!warp_wait(bars.free_[place], (loads / R & 1) ^ 1)) return false;
                        ++loads;
                        const uint32_t to = ring + place * kTileBytes<D> + lane * box * 128, full = bar(bars.full[place]);
                        const uint32_t bytes = __popc(__ballot_sync(~0u, good)) * box * D * 2;
                        if (wanted && !good) {   // no such page: the rows that see it become NaN
                            atomicOr(a.errors, kErrorInput);
                            for (int x = 0; x < D / 64; ++x)
                                for (int i = 0; i < box * 128; i += 16)
                                    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(to + x * (kTile * 128) + i),
                                                 "r"(0x7FFF7FFFu)
                                                 : "memory");
                            writes_before_async();
                        }
                        __syncwarp();
                        if (lane == 0) {
                            if (bytes) barrier_expect(full, bytes);
                            else barrier_arrive(full);
                        }
                        __syncwarp();
                        if (good)
                            for (int x = 0; x < D / 64; ++x)
                                tile_copy4(to + x * (kTile * 128), map, 64 * x, p & ((1 << a.page_shift) - 1), hk, page, full);
                        if (ask && lane == 0) barrier_arrive(bar(bars.ask[place]));
                        __syncwarp();
                        return true;
                    };
                    const int n = it.n[0];
                    bool ok = load_query(0) && load_ring(&k_map, 0, false) && (it.n[1] == 0 || load_query(1));
                    for (int j = 0; ok && j < n; ++j)
                        ok = (j == 0 || load_ring(&k_map, j, false)) && load_ring(&v_map, j, j >= it.clean_from);
                    if (!ok) break;
                    c.kt += n - 1, c.pos += n - 1;
                    step<kBlock, kTile, kTilePiece>(a, c);
                    more = c.pos < r.span;
                }
            } else {
                // Sequences are taken 32 at a time, one a lane.  Their items come longest first: by the block's
                // place in its sequence, falling, then by sequence, then by head.  Every other round of CTAs runs
                // backwards, which evens out what a CTA gets.
                int64_t before = 0, chunk = 0;           // items of the chunks before, items of this one
                int64_t level_before = 0;                // items of the chunk's levels before
                int base = -32, first = 0, len = 0, blocks = 0, level = 0;
                uint32_t loads = 0, q_uses[2] = {0, 0};
                for (uint32_t count = 0;; ++count) {
                    const int64_t want = (int64_t)count * gridDim.x + (count & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                    while (base < a.n && want >= before + chunk) {
                        before += chunk;
                        base += 32;
                        first = len = 0;
                        if (base + lane < a.n) {
                            first = min(max(a.cu[base + lane], 0), a.T);
                            len = min(max(a.cu[base + lane + 1], first), a.T) - first;
                        }
                        blocks = (len + kRows - 1) / kRows;
                        chunk = (int64_t)__reduce_add_sync(~0u, blocks) * a.Hq;
                        level = __reduce_max_sync(~0u, blocks) - 1;
                        level_before = 0;
                    }
                    Item it = {};
                    if (base < a.n) {
                        uint32_t there = __ballot_sync(~0u, blocks > level);
                        while (want - before >= level_before + (int64_t)__popc(there) * a.Hq) {
                            level_before += (int64_t)__popc(there) * a.Hq;
                            there = __ballot_sync(~0u, blocks > --level);
                        }
                        const int i = (int)(want - before - level_before);
                        for (int k = i / a.Hq; k > 0; --k) there &= there - 1;
                        const int src = __ffs(there) - 1;
                        it.first = __shfl_sync(~0u, first, src), it.len = __shfl_sync(~0u, len, src);
                        it.head = i % a.Hq;
                        it.block = level;
                        if (kSplit) {
                            it.n[0] = (level + 2) / 2, it.n[1] = (level + 1) / 2;
                            it.clean_from = level;
                        } else {
                            it.n[0] = 2 * level + 1;
                            it.n[1] = level * kBlock + kTile < it.len ? 2 * level + 2 : 0;
                            it.clean_from = 2 * level;
                        }
                    }
                    const int slot = count % kItems;
                    bool ok = true;
                    if (lane == 0) {
                        ok = wait(bars.item_free[slot], (count / kItems & 1) ^ 1);
                        if (ok) {
                            items[slot] = it;
                            barrier_arrive(bar(bars.item_full[slot]));
                        }
                        if (ok && it.n[0] > 0) {
                            const int hk = it.head / a.group, n1 = it.n[1], n = max(it.n[0], n1);
                            auto load_query = [&](int s) {
                                if (!wait(bars.q_free[s], (q_uses[s] & 1) ^ 1)) return false;
                                ++q_uses[s];
                                barrier_expect(bar(bars.q_full[s]), kTileBytes<D>);
                                for (int c = 0; c < D / 64; ++c)
                                    tile_copy(tiles + s * kTileBytes<D> + c * (kTile * 128), &q_map, 64 * c, it.head,
                                              it.first + it.block * kRows + s * kTile, bar(bars.q_full[s]));
                                return true;
                            };
                            auto load_ring = [&](const CUtensorMap *map, int tile, bool ask) {
                                const int place = loads % R;
                                if (!wait(bars.free_[place], (loads / R & 1) ^ 1)) return false;
                                ++loads;
                                barrier_expect(bar(bars.full[place]), kTileBytes<D>);
                                for (int c = 0; c < D / 64; ++c)
                                    tile_copy(ring + place * kTileBytes<D> + c * (kTile * 128), map, 64 * c, hk,
                                              it.first + tile * kTile, bar(bars.full[place]));
                                if (ask) barrier_arrive(bar(bars.ask[place]));
                                return true;
                            };
                            if (kSplit) {   // the keys two tiles ahead of the values
                                const int all = it.n[0] + n1;
                                ok = load_query(0) && load_ring(&k_map, 0, false) && (all == 1 || load_ring(&k_map, 1, false));
                                for (int j = 0; ok && j < all; ++j)
                                    ok = load_ring(&v_map, j, j == all - 1) && (j + 2 >= all || load_ring(&k_map, j + 2, false));
                            } else {
                                ok = load_query(0) && load_ring(&k_map, 0, false) && (n1 == 0 || load_query(1));
                                for (int j = 0; ok && j < n; ++j)
                                    ok = (j == 0 || load_ring(&k_map, j, false)) && load_ring(&v_map, j, j >= it.clean_from);
                            }
                        }
                    }
                    if (!__shfl_sync(~0u, (int)ok, 0) || it.n[0] == 0) break;
                }
            }
        } else if (warp == 9) {
            // ---- products ---------------------------------------------------------------
            // The whole warp walks through the waits, so that addresses and control are uniform; one thread issues.
            constexpr uint32_t kScores = mma_word(kBf16, kTile, kTile, false), kValues = mma_word(kBf16, kTile, D, true);
            const bool leader = elected();
            struct Place {
                uint32_t at, phase;
                __device__ void next() {
                    if (++at == R) at = 0, phase ^= 1;
                }
            };
            Place place = {0, 0};
            uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0}, clean_phase = 0;   // clean_phase: a bit a place
            auto scores = [&](int s, uint32_t at) {
                const uint32_t q = tile_descriptor(tiles + (kSplit ? 0 : s) * kTileBytes<D>, 16);
                const uint32_t k = tile_descriptor(ring + at * kTileBytes<D>, 16);
                if (leader) {
    #pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const uint32_t step = (x / 4 * (kTile * 128) + x % 4 * 32) / 16;
                        mma_shared(tmem + s * kTile, q + step, k + step, kScores, x > 0);
                    }
                    mma_commit(bar(bars.s_full[s]));
                }
            };
            auto values = [&](int s, uint32_t at, int h, bool add) {   // with one half of the keys
                const uint32_t v = tile_descriptor(ring + at * kTileBytes<D> + h * (kTile / 2 * 128), kTile * 128);
                if (leader) {
    #pragma unroll
                    for (int x = 0; x < kTile / 32; ++x)
                        mma_tensor(tmem + 2 * kTile + s * D, tmem + s * kTile + h * 32 + x * 8, v + x * (2048 / 16), kValues,
                                   add || x > 0);
                }
            };
            auto commit = [&](uint64_t &b) {
                if (leader) mma_commit(bar(b));
            };
            auto run = [&]() {
                for (uint32_t count = 0;; ++count) {
                    const int slot = count % kItems;
                    if (!warp_wait(bars.item_full[slot], count / kItems & 1)) return;
                    const int n0 = __shfl_sync(~0u, items[slot].n[0], 0), n1 = __shfl_sync(~0u, items[slot].n[1], 0);
                    const int n = max(n0, n1), clean_from = __shfl_sync(~0u, items[slot].clean_from, 0);
                    __syncwarp();
                    if (leader) barrier_arrive(bar(bars.item_free[slot]));
                    if (n0 == 0) return;
                    if constexpr (kSplit) {
                        const int all = n0 + n1;
                        if (!warp_wait(bars.q_full[0], q_phase[0])) return;
                        q_phase[0] ^= 1;
    #pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            if (s >= all) continue;
                            if (!warp_wait(bars.full[place.at], place.phase)) return;
                            tensor_fence_after();
                            scores(s, place.at);
                            commit(bars.free_[place.at]);
                            place.next();
                        }
                        if (all <= 2) commit(bars.q_free[0]);
                        for (int t0 = 0; t0 < all; t0 += 2) {
    #pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                const int t = t0 + s;
                                if (t >= all) continue;
                                const bool more = t + 2 < all;
                                const Place v = place;
                                place.next();
                                const Place k = place;   // the keys two tiles on
                                if (more) place.next();
                                if (!warp_wait(bars.full[v.at], v.phase)) return;
                                if (t == all - 1) {
                                    if (!warp_wait(bars.clean[v.at], clean_phase >> v.at & 1)) return;
                                    clean_phase ^= 1u << v.at;
                                }
                                if (more && !warp_wait(bars.full[k.at], k.phase)) return;
    #pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    if (!warp_wait(bars.p_full[s][h], p_phase[s])) return;
                                    tensor_fence_after();
                                    values(s, v.at, h, t0 > 0 || h > 0);
                                }
                                p_phase[s] ^= 1;
                                if (more) {
                                    scores(s, k.at);
                                    if (t + 3 == all) commit(bars.q_free[0]);
                                } else {
                                    commit(bars.o_full[s]);
                                }
                                commit(bars.free_[v.at]);
                                if (more) commit(bars.free_[k.at]);
                            }
                        }
                        continue;
                    }
                    if (!warp_wait(bars.full[place.at], place.phase)) return;
    #pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int ns = s ? n1 : n0;
                        if (ns == 0) continue;
                        if (!warp_wait(bars.q_full[s], q_phase[s])) return;
                        q_phase[s] ^= 1;
                        tensor_fence_after();
                        scores(s, place.at);
                        if (ns == 1) commit(bars.q_free[s]);
                    }
                    commit(bars.free_[place.at]);
                    place.next();
                    for (int j = 0; j < n; ++j) {
                        const Place v = place;
                        place.next();
                        const Place k = place;   // the next keys
                        if (j + 1 < n) place.next();
                        if (!warp_wait(bars.full[v.at], v.phase)) return;
                        if (j >= clean_from) {
                            if (!warp_wait(bars.clean[v.at], clean_phase >> v.at & 1)) return;
                            clean_phase ^= 1u << v.at;
                        }
                        if (j + 1 < n && !warp_wait(bars.full[k.at], k.phase)) return;
    #pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const int ns = s ? n1 : n0;
                            if (j >= ns) continue;
    #pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (!warp_wait(bars.p_full[s][h], p_phase[s])) return;
                                tensor_fence_after();
                                values(s, v.at, h, j > 0 || h > 0);
                            }
                            p_phase[s] ^= 1;
                            if (j + 1 == ns) {
                                commit(bars.o_full[s]);
                            } else {
                                scores(s, k.at);
                                if (j + 2 == ns) commit(bars.q_free[s]);
                            }
                        }
                        commit(bars.free_[v.at]);
                        if (j + 1 < n) commit(bars.free_[k.at]);
                    }
                }
            };
            run();
            commit(bars.done);   // no arrival of a commit is under way when the CTA's memory goes
            warp_wait(bars.done, 0);
        } else {
            // ---- values that are not finite, in the tiles on the diagonal ------------------
            uint32_t loads = 0, asks = 0;
            bool ok = true;
            for (uint32_t count = 0; ok; ++count) {
                const int slot = count % kItems;
                ok = warp_wait(bars.item_full[slot], count / kItems & 1);
                if (!ok) break;
                const int n0 = items[slot].n[0], n1 = items[slot].n[1], n = kSplit ? n0 + n1 : max(n0, n1);
                const int from = items[slot].clean_from;
                // keys of the tile, counted from the first tile looked at
                const int keys = items[slot].len + items[slot].m - (kCache ? items[slot].len / kTile : from) * kTile;
                const int skip = kCache ? items[slot].kt0 + from - items[slot].len / kTile : 0;
                for (int j = from; ok && j < n; ++j) {
                    const uint32_t i = loads + 2 * j + 1;
                    const int place = i % R;
                    ok = warp_wait(bars.ask[place], asks >> place & 1) && warp_wait(bars.full[place], i / R & 1);
                    if (!ok) break;
                    asks ^= 1u << place;
                    const uint32_t at = ring + place * kTileBytes<D>;
    #pragma unroll 4
                    for (int c = tid - 320; c < kTileBytes<D> / 16; c += 64) {
                        uint32_t w[4];
                        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                     : "r"(at + c * 16)
                                     : "memory");
                        // a half whose magnitude reaches the exponent of infinity carries into its sign bit
                        constexpr uint32_t kStep = kBf16 ? 0x00800080u : 0x04000400u;
                        uint32_t odd = 0;
    #pragma unroll
                        for (int x = 0; x < 4; ++x) odd |= (w[x] & 0x7FFF7FFFu) + kStep;
                        if (odd & 0x80008000u) {
                            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + c * 16), "r"(finite_part<E>(w[0])),
                                         "r"(finite_part<E>(w[1])), "r"(finite_part<E>(w[2])), "r"(finite_part<E>(w[3]))
                                         : "memory");
                            const int row = c / 8 % kTile;
                            const int tile = j - from + skip;   // 0 or 1
                            if (tile * kTile + row < keys) atomicOr(&items[slot].odd[tile][row / 32], 1u << row % 32);
                        }
                    }
                    writes_before_async();
                    __syncwarp();
                    if (lane == 0) barrier_arrive(bar(bars.clean[place]));
                }
                loads += 2 * n;
                __syncwarp();
                if (lane == 0) barrier_arrive(bar(bars.item_free[slot]));
                if (n0 == 0) break;
            }
        }
    } else {
        // ---- softmax and output: one row a thread ----------------------------------------
        take_registers<kManyRegisters>();
        const int s = warp / 4, local = tid % kTile;
        const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t s_at = tmem + lanes + s * kTile, o_at = tmem + lanes + 2 * kTile + s * D;
        const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
        uint32_t s_uses = 0, o_uses = 0, merges = 0;
        const int heads = [&] {
            if constexpr (kCache) return a.Hkv * a.group;
            else return a.Hq;
        }();
        bool ok = true;
        for (uint32_t count = 0; ok; ++count) {
            const int slot = count % kItems;
            ok = warp_wait(bars.item_full[slot], count / kItems & 1);
            if (!ok) break;
            if (items[slot].n[0] == 0) break;
            const int n = items[slot].n[s], clean_from = items[slot].clean_from;
            int row;                 // of the sequence; over a cache the row's drafted token, -1 where there is none
            uint64_t bits = 0;       // over a cache: the drafted tokens that the row sees
            if constexpr (kCache) {
                const int m = items[slot].m;
                row = tile_token(a, items[slot].block, s, local, m);
                if (row >= 0) bits = a.mask ? a.mask[items[slot].first + row] : ~0ull >> (63 - row);
                if (m < 64) bits &= (1ull << m) - 1;
            } else {
                row = items[slot].block * kRows + (kSplit ? 0 : s * kTile) + local;
            }
            float m = -INFINITY, l = 0.0f;   // m: what the weights so far are relative to, from a (scaled) maximum
            for (int j = 0; j < n; ++j) {
                ok = warp_wait(bars.s_full[s], s_uses++ & 1);
                if (!ok) break;
                tensor_fence_after();
                uint32_t x[4][32];
                // some row must not see some key (of a split item, the last tile alone lies on the diagonal)
                const bool diagonal = kCache ? j >= clean_from : j == n - 1 && (!kSplit || s == (clean_from & 1));
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_load32(x[c], s_at + 32 * c);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_wait32(x[c]);
                if (diagonal) {
                    if constexpr (kCache) {
                        // the keys before `draft` are committed, from there on the row's bits say
                        const int draft = items[slot].len - (items[slot].kt0 + j) * kTile;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int d = draft - 32 * c;   // of this part's 32 keys
                            const uint32_t sees = d >= 32    ? ~0u
                                                  : d >= 0   ? (uint32_t)(bits << d) | ((1u << d) - 1)
                                                  : d > -64  ? (uint32_t)(bits >> -d)
                                                             : 0u;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(sees >> i & 1)) x[c][i] = 0xFF800000u;
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (32 * c + i > local) x[c][i] = 0xFF800000u;
                    }
                }
                // The first weights are computed from the maximum so far while the new one is looked for: it
                // seldom asks for a change, and the exponentials' unit need not wait for it.
                uint64_t sum[2];
                uint32_t p[16];
                auto weights = [&](int c, float ref) {
                    const uint64_t ref2 = pair(-ref, -ref);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float lo, hi;
                        unpair(fma2(pair(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])), scale2, ref2), lo, hi);
                        lo = exp2_approx(lo), hi = exp2_approx(hi);
                        const uint64_t both = pair(lo, hi);
                        sum[i % 2] = c == 0 && i < 2 ? both : add2(sum[i % 2], both);
                        p[i] = pack2<E>(lo, hi);
                    }
                };
                weights(0, m == -INFINITY ? 0.0f : m);
                float top[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    top[c] = max3(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]), __uint_as_float(x[c][2]));
#pragma unroll
                    for (int i = 3; i < 31; i += 2)
                        top[c] = max3(top[c], __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
                    top[c] = max3(top[c], __uint_as_float(x[c][31]), __uint_as_float(x[c][31]));
                }
                const float mn = max3(max3(top[0], top[1], top[2]), top[3], top[3]) * a.scale_log2 - kHeadroomLog2<E>;
                if (!(mn < INFINITY)) l = NAN;   // a score that is NaN or infinite: the row has no weights
                const bool grown = mn > m + kRescaleLog2;   // also the first finite score of the row
                if (__any_sync(~0u, grown)) {
                    const float f = grown ? exp2_approx(m - mn) : 1.0f;
                    if (grown) m = mn;
                    l *= f;
                    if (j > 0) {   // the product before is complete: this tile's scores were issued behind it
                        const uint64_t f2 = pair(f, f);
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_load16(o, o_at + c);
                            tmem_wait16(o);
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                float lo, hi;
                                unpair(mul2(pair(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), f2), lo, hi);
                                o[i] = __float_as_uint(lo), o[i + 1] = __float_as_uint(hi);
                            }
                            tmem_store16(o_at + c, o);
                        }
                    }
                    weights(0, m == -INFINITY ? 0.0f : m);
                }
                const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c > 0) weights(c, ref);
                    tmem_store16(s_at + 16 * c, p);
                    if (c % 2) {
                        tmem_stores_done();
                        tensor_fence_before();
                        __syncwarp();
                        if (lane == 0) barrier_arrive(bar(bars.p_full[s][c / 2]));
                    }
                }
                float lo, hi;
                unpair(add2(sum[0], sum[1]), lo, hi);
                l += lo + hi;
            }
            bool second = false;   // a split item's second half, to be joined to the first
            if constexpr (kSplit) {
                if (ok && n > 0 && s == 1) {
                    merge_ml[local] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) barrier_arrive(bar(bars.merge_full));
                    ok = warp_wait(bars.merge_free, merges++ & 1);   // its outputs stay until they have been read
                    if (!ok) break;
                }
                second = s == 0 && items[slot].n[1] > 0;
                if (ok && second) {
                    ok = warp_wait(bars.o_full[1], merges & 1) && warp_wait(bars.merge_full, merges & 1);
                    ++merges;
                    if (!ok) break;
                }
            }
            if (ok && n > 0 && !(kSplit && s == 1)) {
                ok = warp_wait(bars.o_full[s], o_uses++ & 1);
                if (!ok) break;
                tensor_fence_after();
                const Item &it = items[slot];
                const int first = it.first;
                int token, head, hk;
                bool mine;
                if constexpr (kCache) {
                    token = first + row, hk = it.head, head = hk * a.group + local % a.group;
                    mine = row >= 0;
                } else {
                    token = first + row, head = it.head, hk = head / a.group;
                    mine = row < it.len;
                }
                const bool partial = kCache && it.piece >= 0;
                float f0 = 1.0f, f1 = 0.0f;   // of the halves of a split item
                if (kSplit && second) {
                    const float2 other = merge_ml[kSplit ? local : 0];
                    const float best = fmaxf(m, other.x), ref = best == -INFINITY ? 0.0f : best;
                    f0 = exp2_approx(m - ref), f1 = exp2_approx(other.x - ref);
                    l = l * f0 + other.y * f1, m = ref;
                }
                const float inv = partial ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
                uint32_t odd = 0;
#pragma unroll
                for (int t = 0; t < 8; ++t) odd |= it.odd[t / 4][t % 4];
                E *out = (E *)a.out + (size_t)token * a.ldo + (size_t)head * D;
#pragma unroll 1   // little code: the tiles' own stays near
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_load32(o, o_at + c);
                    tmem_wait32(o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * (kSplit ? f0 * inv : inv));
                    if (kSplit && second) {
                        uint32_t o1[32];
                        tmem_load32(o1, o_at + D + c);
                        tmem_wait32(o1);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), f1 * inv, __uint_as_float(o[i])));
                    }
                    for (int t = 0; odd && t < 2; ++t)
                        for (int w = 0; w < 4; ++w)
                            for (uint32_t rows = it.odd[t][w]; rows; rows &= rows - 1) {
                                const E *v = nullptr;
                                if constexpr (kCache) {
                                    const int key = (it.len / kTile + t) * kTile + 32 * w + __ffs(rows) - 1, d = key - it.len;
                                    if (d >= 0 && !(bits >> d & 1)) continue;
                                    const int at = key >> a.page_shift;
                                    const int page = at < a.table_width ? a.table[(size_t)it.seq * a.ld_table + at] : -1;
                                    if (page >= 0 && page < a.pages)
                                        v = (const E *)a.vc + ((((size_t)page * a.Hkv + hk) << a.page_shift) +
                                                               (key & ((1 << a.page_shift) - 1))) * D + c;
                                } else {
                                    const int key = (kRows / kTile * it.block + t) * kTile + 32 * w + __ffs(rows) - 1;
                                    if (key > row) continue;
                                    v = (const E *)a.v + (size_t)(first + key) * a.ldv + (size_t)hk * D + c;
                                }
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const float f = v ? (float)v[i] : NAN;
                                    if (!isfinite(f)) o[i] = __float_as_uint(__uint_as_float(o[i]) + f);
                                }
                            }
                    if (kCache && partial && mine) {
                        if constexpr (kCache) {
                            // rows side by side, so that a warp writes whole lines
                            float4 *part = reinterpret_cast<float4 *>(a.part) +
                                           ((size_t)it.piece * (D / 4) + c / 4) * kBlock + s * kTile + local;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                part[(size_t)i * kBlock] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                                       __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                        }
                    } else if (mine) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint4 r;
                            r.x = pack2<E>(__uint_as_float(o[8 * i]), __uint_as_float(o[8 * i + 1]));
                            r.y = pack2<E>(__uint_as_float(o[8 * i + 2]), __uint_as_float(o[8 * i + 3]));
                            r.z = pack2<E>(__uint_as_float(o[8 * i + 4]), __uint_as_float(o[8 * i + 5]));
                            r.w = pack2<E>(__uint_as_float(o[8 * i + 6]), __uint_as_float(o[8 * i + 7]));
                            *reinterpret_cast<uint4 *>(out + c + 8 * i) = r;
                        }
                    }
                }
                tensor_fence_before();
                if (kSplit && second) {
                    __syncwarp();
                    if (lane == 0) barrier_arrive(bar(bars.merge_free));
                }
                if (partial && mine) {
                    if constexpr (kCache)
                        *reinterpret_cast<float2 *>(a.part_ml + ((size_t)it.piece * kBlock + s * kTile + local) * 2) = make_float2(m, l);
                } else if (a.lse && mine) {
                    a.lse[(size_t)token * heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
                }
            }
            __syncwarp();
            if (lane == 0) barrier_arrive(bar(bars.item_free[slot]));
        }
    }
    __syncthreads();
    if (gave_up_word) {
        outlast_copies();
        if (tid == 0) atomicOr(a.errors, kErrorWait);
        __syncthreads();
    }
    if (warp == 9) tmem_free(tmem, kColumns);
}

// ---- host ---------------------------------------------------------------------------

// [token][head][D] in boxes of 64 columns, `heads` heads and `tokens` tokens.
inline bool head_map(CUtensorMap *map, const void *base, fb_dtype t, int T, int H, int D, int ld, int heads, int tokens) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens}, steps[3] = {1, 1, 1};
    return f(map, t == FB_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
             strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether the compiler gave the kernel the registers that its warps' shares add up to.
template <auto Kernel>
bool registers_as_planned() {
    static std::atomic<int> registers{0};
    if (!registers.load(std::memory_order_relaxed)) {
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, Kernel) != cudaSuccess) return false;
        registers.store(attr.numRegs, std::memory_order_relaxed);
    }
    return registers.load(std::memory_order_relaxed) == kLaunchRegisters;
}

}  // namespace fb
