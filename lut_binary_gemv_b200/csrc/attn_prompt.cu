// attn_prompt.cu -- causal attention of packed prompts on the tensor cores.
//
//   out_i = sum_{j <= i} exp(scale q_i.k_j - m_i) v_j / sum_{j <= i} exp(scale q_i.k_j - m_i)
//
// in one pass over the keys with a running maximum m and sum.  An item is 256
// queries of one head: two tiles of 128 rows that share every tile of 128 keys
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
//                    of the item must not see (those on the diagonal): a weight
//                    of zero would not stop them.  They note the rows, and the
//                    rows that do see them add them at the end.
//
// Tensor memory: two score tiles of 128 columns, each overwritten by its
// weights (64 columns), and two outputs of D columns.  The products are issued
// by one thread and complete in order, so a new score tile may be asked for as
// soon as the product that reads the old weights has been issued.
//
// The outputs are rescaled only when a row's maximum has grown by more than
// 2^8 since the last time (exact all the same: the sum carries the same factor,
// and weights up to 2^8 lose nothing in either type), which few tiles need.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "attn_common.cuh"
#include "fb_internal.cuh"
#include "tensor_core.cuh"

namespace fb {
namespace {

constexpr int kTile = 128;                 // queries of a tile, keys of a tile
constexpr int kBlock = 2 * kTile;          // queries of an item
constexpr int kThreads = 384;
constexpr int kColumns = 512;              // all of tensor memory
constexpr int kItems = 2;                  // items known at a time
constexpr int kItemReaders = 8 + 1 + 2;    // warps that read an item
// Registers a thread: at the launch, then of the softmax warps and of the others; the shares of the
// eight and the four warps add up to the launch's.
constexpr int kLaunchRegisters = 168, kManyRegisters = 208, kFewRegisters = 88;
static_assert(8 * kManyRegisters + 4 * kFewRegisters == 12 * kLaunchRegisters, "registers are moved, not made");
constexpr float kRescaleLog2 = 8.0f;

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

struct Item {
    int first, len, block, head;   // the sequence's first token and length; head < 0: no more items
    uint32_t odd[2][4];            // rows of the two diagonal tiles whose values are not all finite
};

struct Barriers {
    uint64_t q_full[2], q_free[2];          // the query tiles
    uint64_t full[8], free_[8], clean[8], ask[8];   // the ring
    uint64_t s_full[2], p_full[2][2], o_full[2];   // the weights by halves of the keys
    uint64_t item_full[kItems], item_free[kItems];
    uint64_t done;
};

// Tiles of keys that query tile s of block b meets (0 where it has no rows).
__device__ __forceinline__ int key_tiles(const Item &it, int s) {
    return it.block * kBlock + s * kTile < it.len ? 2 * it.block + s + 1 : 0;
}

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

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap q_map,
                  const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    constexpr int R = kRing<D>;
    constexpr bool kBf16 = std::is_same_v<E, __nv_bfloat16>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Barriers bars;
    __shared__ Item items[kItems];
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
        barrier_init(bar(bars.done), 1);
        barrier_inits_done();
    }
    if (warp == 9) tmem_alloc(smem_address(&tmem_at), kColumns);
    tensor_fence_before();
    __syncthreads();
    tensor_fence_after();
    const uint32_t tmem = tmem_at;
    wait_for_previous_kernel();

    if (warp == 8) {
        // ---- items and copies -----------------------------------------------------
        give_registers<kFewRegisters>();
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
                blocks = (len + kBlock - 1) / kBlock;
                chunk = (int64_t)__reduce_add_sync(~0u, blocks) * a.Hq;
                level = __reduce_max_sync(~0u, blocks) - 1;
                level_before = 0;
            }
            Item it;
            it.head = -1, it.first = it.len = it.block = 0;
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
            }
            const int slot = count % kItems;
            bool ok = true;
            if (lane == 0) {
                ok = wait(bars.item_free[slot], (count / kItems & 1) ^ 1);
                if (ok) {
                    items[slot].first = it.first, items[slot].len = it.len;
                    items[slot].block = it.block, items[slot].head = it.head;
                    for (int t = 0; t < 8; ++t) items[slot].odd[t / 4][t % 4] = 0;
                    barrier_arrive(bar(bars.item_full[slot]));
                }
                if (ok && it.head >= 0) {
                    const int hk = it.head / a.group, n0 = key_tiles(it, 0), n1 = key_tiles(it, 1), n = max(n0, n1);
                    auto load_query = [&](int s) {
                        if (!wait(bars.q_free[s], (q_uses[s] & 1) ^ 1)) return false;
                        ++q_uses[s];
                        barrier_expect(bar(bars.q_full[s]), kTileBytes<D>);
                        for (int c = 0; c < D / 64; ++c)
                            tile_copy(tiles + s * kTileBytes<D> + c * (kTile * 128), &q_map, 64 * c, it.head,
                                      it.first + it.block * kBlock + s * kTile, bar(bars.q_full[s]));
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
                    ok = load_query(0) && load_ring(&k_map, 0, false) && (n1 == 0 || load_query(1));
                    for (int j = 0; ok && j < n; ++j)
                        ok = (j == 0 || load_ring(&k_map, j, false)) && load_ring(&v_map, j, j >= n0 - 1);
                }
            }
            if (!__shfl_sync(~0u, (int)ok, 0) || it.head < 0) break;
        }
    } else if (warp == 9) {
        // ---- products ---------------------------------------------------------------
        give_registers<kFewRegisters>();
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
            const uint32_t q = tile_descriptor(tiles + s * kTileBytes<D>, 16);
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
                const int head = items[slot].head;
                const int n0 = __shfl_sync(~0u, key_tiles(items[slot], 0), 0), n1 = __shfl_sync(~0u, key_tiles(items[slot], 1), 0);
                const int n = max(n0, n1);
                __syncwarp();
                if (leader) barrier_arrive(bar(bars.item_free[slot]));
                if (head < 0) return;
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
                    if (j >= n0 - 1) {
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
    } else if (warp >= 10) {
        // ---- values that are not finite, in the tiles on the diagonal ------------------
        give_registers<kFewRegisters>();
        uint32_t loads = 0, asks = 0;
        bool ok = true;
        for (uint32_t count = 0; ok; ++count) {
            const int slot = count % kItems;
            ok = warp_wait(bars.item_full[slot], count / kItems & 1);
            if (!ok) break;
            const int head = items[slot].head, block = items[slot].block, len = items[slot].len;
            const int n0 = key_tiles(items[slot], 0), n = max(n0, key_tiles(items[slot], 1));
            for (int j = n0 - 1; ok && head >= 0 && j < n; ++j) {
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
                        if (j * kTile + row < len) atomicOr(&items[slot].odd[j - 2 * block][row / 32], 1u << row % 32);
                    }
                }
                writes_before_async();
                __syncwarp();
                if (lane == 0) barrier_arrive(bar(bars.clean[place]));
            }
            loads += 2 * n;
            __syncwarp();
            if (lane == 0) barrier_arrive(bar(bars.item_free[slot]));
            if (head < 0) break;
        }
    } else {
        // ---- softmax and output: one row a thread ----------------------------------------
        take_registers<kManyRegisters>();
        const int s = warp / 4, local = tid % kTile;
        const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t s_at = tmem + lanes + s * kTile, o_at = tmem + lanes + 2 * kTile + s * D;
        const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
        uint32_t s_uses = 0, o_uses = 0;
        bool ok = true;
        for (uint32_t count = 0; ok; ++count) {
            const int slot = count % kItems;
            ok = warp_wait(bars.item_full[slot], count / kItems & 1);
            if (!ok) break;
            const int head = items[slot].head, n = key_tiles(items[slot], s);
            if (head < 0) break;
            const int row = items[slot].block * kBlock + s * kTile + local;
            float m = -INFINITY, l = 0.0f;   // m: the (scaled) maximum that the weights so far are relative to
            for (int j = 0; j < n; ++j) {
                ok = warp_wait(bars.s_full[s], s_uses++ & 1);
                if (!ok) break;
                tensor_fence_after();
                uint32_t x[4][32];
                const bool diagonal = j == n - 1;
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_load32(x[c], s_at + 32 * c);
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_wait32(x[c]);
                if (diagonal) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * c + i > local) x[c][i] = 0xFF800000u;
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
                const float mn = max3(max3(top[0], top[1], top[2]), top[3], top[3]) * a.scale_log2;
                if (!(mn < INFINITY)) l = NAN;   // a score that is NaN or infinite: the row has no weights
                const bool grown = mn > m + kRescaleLog2;   // also the first finite score of the row
                if (__any_sync(~0u, grown)) {
                    const float f = grown ? exp2_approx(m - mn) : 1.0f;
                    if (grown) m = mn;
                    l *= f;
                    if (j > 0) {   // the product before is complete: this tile's scores were issued behind it
                        const uint64_t f2 = pair(f, f);
#pragma unroll
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
            if (ok && n > 0) {
                ok = warp_wait(bars.o_full[s], o_uses++ & 1);
                if (!ok) break;
                tensor_fence_after();
                const Item &it = items[slot];
                const int first = it.first;
                const bool mine = row < it.len;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                E *out = (E *)a.out + (size_t)(first + row) * a.ldo + (size_t)head * D;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_load32(o, o_at + c);
                    tmem_wait32(o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
                    for (int t = 0; t <= s; ++t)
                        for (int w = 0; w < 4; ++w)
                            for (uint32_t bits = it.odd[t][w]; bits; bits &= bits - 1) {
                                const int key = (2 * it.block + t) * kTile + 32 * w + __ffs(bits) - 1;
                                if (key > row) continue;
                                const E *v = (const E *)a.v + (size_t)(first + key) * a.ldv + (size_t)(head / a.group) * D + c;
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const float f = (float)v[i];
                                    if (!isfinite(f)) o[i] = __float_as_uint(__uint_as_float(o[i]) + f);
                                }
                            }
                    if (mine) {
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
                if (a.lse && mine)
                    a.lse[(size_t)(first + row) * a.Hq + head] =
                        l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
            }
            __syncwarp();
            if (lane == 0) barrier_arrive(bar(bars.item_free[slot]));
        }
    }
    __syncthreads();
    if (gave_up_word) {
        // copies and products that were under way land in this CTA's memory: give them time before it is reused
        const uint64_t start = now_ns();
        while (now_ns() - start < 20000000ull) __nanosleep(1000);
        if (tid == 0) atomicOr(a.errors, 4u);
        __syncthreads();
    }
    if (warp == 9) tmem_free(tmem, kColumns);
}

// ---- host ---------------------------------------------------------------------------

// [token][head][D] in boxes of 64 columns, one head and a tile of tokens.
bool head_map(CUtensorMap *map, void *base, fb_dtype t, int T, int H, int D, int ld) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kTile}, steps[3] = {1, 1, 1};
    return f(map, t == FB_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims,
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

template <typename E, int D>
cudaError_t launch_prompt(const PromptArgs &a, const fb_heads &in, bool pdl, cudaStream_t s) {
    CUtensorMap q, k, v;
    if (!head_map(&q, in.q, in.t, in.T, in.Hq, D, in.ldq) || !head_map(&k, in.k, in.t, in.T, in.Hkv, D, in.ldk) ||
        !head_map(&v, in.v, in.t, in.T, in.Hkv, D, in.ldv))
        return cudaErrorInvalidValue;
    auto kernel = prompt_kernel<E, D>;
    if (!registers_as_planned<prompt_kernel<E, D>>()) return cudaErrorInvalidValue;   // a warp would wait for registers for good
    cudaError_t e = allow_shared<prompt_kernel<E, D>>(kSmemBytes<D>);
    if (e != cudaSuccess) return e;
    // one CTA an SM, no more than there can be items
    const int64_t most = ((int64_t)(in.T + kBlock - 1) / kBlock + (a.n < in.T ? a.n : in.T)) * in.Hq;
    const int ctas = (int)(most < sm_count() ? most : sm_count());
    return launch(kernel, dim3(ctas), dim3(kThreads), kSmemBytes<D>, s, pdl, a, q, k, v);
}

}  // namespace
}  // namespace fb

using namespace fb;

extern "C" fb_status fb_attn_prompt(const fb_heads *in, const int32_t *cu_seqlens, int n, float scale, void *out,
                                    int ldo, float *lse, unsigned flags, void *stream) {
    if (!in || (flags & ~FB_GEMV_PDL) || !valid_heads(*in) || !in->q || !in->k || !in->v || !out || !cu_seqlens ||
        n < 1 || n > kMaxTokens || ldo < in->Hq * in->D || !(scale > 0.0f) || scale > 3e38f)
        return FB_ERR_INVALID_VALUE;
    if (in->t == FB_F32 || (in->D != 64 && in->D != 128)) return FB_ERR_UNSUPPORTED;
    if (!aligned(in->q, 16) || !aligned(in->k, 16) || !aligned(in->v, 16) || !aligned(out, 16) || in->ldq % 8 ||
        in->ldk % 8 || in->ldv % 8 || ldo % 8 || !aligned(cu_seqlens, 4) || !aligned(lse, 4))
        return FB_ERR_MISALIGNED;
    PromptArgs a = {};
    a.v = in->v, a.out = out, a.lse = lse, a.cu = cu_seqlens, a.n = n;
    a.errors = (unsigned int *)attn_errors_address();
    a.T = in->T, a.Hq = in->Hq, a.group = in->Hq / in->Hkv, a.ldv = in->ldv, a.ldo = ldo;
    a.scale_log2 = scale * 1.44269504089f;
    if (!a.errors) return FB_ERR_CUDA;
    const bool pdl = flags & FB_GEMV_PDL;
    cudaStream_t s = as_stream(stream);
    if (in->t == FB_F16)
        return status_of(in->D == 64 ? launch_prompt<__half, 64>(a, *in, pdl, s)
                                     : launch_prompt<__half, 128>(a, *in, pdl, s));
    return status_of(in->D == 64 ? launch_prompt<__nv_bfloat16, 64>(a, *in, pdl, s)
                                 : launch_prompt<__nv_bfloat16, 128>(a, *in, pdl, s));
}
