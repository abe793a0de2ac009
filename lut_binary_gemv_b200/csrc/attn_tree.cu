// attn_tree.cu -- attention of single tokens and of trees of drafted tokens
// over a paged cache.
//
//   out_i = sum_j p_ij v_j over the committed keys and the drafted keys whose
//   bit is set in the token's mask, p the softmax of scale q_i.k_j.
//
// A key and its value are read once for the rows that share them (the drafted
// tokens times the query heads of a key head), so for few rows the kernel is
// bound by HBM and everything serves the stream of keys:
//
//  * The work is the list of (sequence, key head, row tile, tile of 64 keys),
//    cut into one equal run of key tiles for each resident CTA, whatever the
//    lengths: a long sequence spreads over many CTAs and a CTA takes many short
//    ones.  Each CTA finds its run from the lengths on the device.  A sequence
//    cut by a run's end leaves its running maximum, sum and unnormalised output
//    in the workspace (a CTA has at most two such pieces, its first and its
//    last), and join_kernel joins them in order, so results do not depend on
//    timing.
//  * Of a tile, each warp owns 16 keys for all rows (up to 32 of them): one
//    thread asks for them with tiled copies two tiles ahead, across the ends of
//    sequences, and the warp needs no CTA barrier until the piece ends.  (Pages
//    of fewer than 16 rows are copied row by row.)
//  * Scores and outputs are m16n8k16 products with fp32 accumulators; the
//    weights stay in registers between the two.
//  * From 33 rows a key head on, the tensor-core tiles of attn_tiles.cuh are
//    faster at every size measured (8 sequences of 4,000 keys and 40 rows: 43
//    us against 83; at 32 rows 43 against 40), with the same runs and join.
//    Pages of fewer than 8 rows, or groups of more than 128 query heads, stay
//    here: two warps share 32 keys and split 64 rows.
//
// Measured (bf16, 64 heads over 8 of 128): one token over 131,071 keys 95 us,
// 5.65 TB/s, of which the join takes 5; 32 conversations of 1 to 15,000 keys 82
// us, 5.7 TB/s.  Counting the pieces' cost in the runs took the latter from 119
// to 105 us and drafted trees of 1 to 31 tokens from 171 to 62.
//
// A tile that reaches into the drafted keys may hold infinities or NaN that
// some rows must not see, and a weight of zero does not stop them: such values
// are added to the rows that see them and cleared before the product.
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
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTileKeys = 64;      // keys of a tile, 16 loaded by each warp
constexpr int kCtasPerSm = 2;
__device__ unsigned int g_attn_errors;

constexpr int kWholeKeys = 512;    // tables of no more keys: items are not cut (the host does not know the lengths)

// What starting and ending a piece costs, in key tiles.
template <int MT>
constexpr int kPieceTiles = MT == 1 ? 3 : 8;

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
template <typename E>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same_v<E, __half>)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of a 16-byte chunk in a block of 16 rows: columns in groups of 64
// (128 bytes a row), the chunk's index turned by the row, as the tiled copies
// put it; the eight rows of a matrix load lie in eight different groups of banks.
__device__ __forceinline__ int chunk_at(int row, int chunk) {
    return (chunk >> 3) * 2048 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

template <int D>
constexpr int kStages = 384 / D;   // 96 KB of tiles a CTA, two CTAs an SM
template <int D>
constexpr int kSlice = 16 * D * 4;  // a warp's share of a tile's place: 16 keys, then their values
template <int D>
constexpr int kStageBytes = kWarps * kSlice<D>;

template <int D, int ROWS>
constexpr int tree_smem_bytes() {
    return kStages<D> * kStageBytes<D> + ROWS * D * 2;
}

// WR row warps times WK key warps; MT row tiles of 16 a warp; kTiled: pages of at least 16 rows.
template <typename E, int D, int WR, int WK, int MT, bool kTiled>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    tree_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    static_assert(WR * WK == kWarps, "four warps");
    constexpr int ROWS = WR * MT * 16, kPiece = kPieceTiles<MT>;
    constexpr int KW = kTileKeys / WK;      // keys a warp multiplies
    constexpr int NT = KW / 8;              // 8-key columns of its scores
    constexpr int CH = D / 8;               // 16-byte chunks of a row
    constexpr int S = kStages<D>;
    constexpr int kHalf = kSlice<D> / 2;    // from a slice's keys to its values
    constexpr bool kOwnKeys = WK == kWarps; // a warp multiplies the keys it loads, and no others
    constexpr bool kQueriesHeld = MT == 1;  // the queries stay in registers
    constexpr bool kTwoParts = MT == 1;     // the weights as two operands
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[S][kWarps];
    __shared__ uint64_t s_mask[ROWS];
    __shared__ float s_ml[2][kWarps][MT * 16];
    __shared__ int gave_up_word;
    volatile int *gave_up = &gave_up_word;

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int wr = warp % WR, wk = warp / WR;
    const uint32_t stages = smem_address(smem), q_at = stages + S * kStageBytes<D>;

    if (tid == 0) {
        gave_up_word = 0;
        for (int i = 0; i < S * kWarps; ++i) barrier_init(smem_address(&full[i / kWarps][i % kWarps]), 1);
        barrier_inits_done();
    }
    __syncthreads();
    wait_for_previous_kernel();

    // ---- this CTA's run of key tiles -----------------------------------------
    Cursor at;
    const Run r = find_run<ROWS, kTileKeys, kPiece>(a, at);
    if (tid == 0 && !a.whole) a.records[blockIdx.x] = make_int4(0, 0, 0, 0);
    asm volatile("griddepcontrol.launch_dependents;");   // the join may be made ready; it waits for the end of this grid
    if (r.span <= 0) return;
    const int64_t span = r.span;

    // ---- loading: each warp brings in keys 16 warp .. 16 warp + 15 of a tile ----
    Cursor ahead = at;
    int load_stage = 0;
    bool lost = false;   // a wait was given up: no more copies, whose places may still be awaiting the last ones
    // the page of a key position of the cursor's sequence (-1 beyond the table)
    auto page_of = [&](int p) {
        const int slot = p >> a.page_shift;
        return p < ahead.q.len + ahead.q.m && slot < a.table_width ? a.table[(size_t)ahead.s * a.ld_table + slot] : -1;
    };
    int page = page_of(ahead.kt * kTileKeys + 16 * warp + (kTiled ? 0 : lane % 16));   // looked up a tile early
    auto load_tile = [&]() {
        if (ahead.pos < span && !lost) {
            const int hk = ahead.item / ahead.q.row_tiles, keys = ahead.q.len + ahead.q.m;
            const uint32_t k_at = stages + load_stage * kStageBytes<D> + warp * kSlice<D>, v_at = k_at + kHalf;
            const int p0 = ahead.kt * kTileKeys + 16 * warp;
            if constexpr (kTiled) {
                const uint32_t bar = smem_address(&full[load_stage][warp]);
                const bool good = page >= 0 && page < a.pages;
                if (p0 < keys && !good) {   // no such page: the rows that see it become NaN
                    for (int i = lane; i < kSlice<D> / 16; i += 32)
                        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(k_at + 16 * i), "r"(0x7FFF7FFFu) : "memory");
                    writes_before_async();
                    __syncwarp();
                }
                if (lane == 0) {
                    if (p0 < keys && good) {
                        const int row = p0 & ((1 << a.page_shift) - 1);
                        barrier_expect(bar, kSlice<D>);
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            tile_copy4(k_at + c * 2048, &k_map, 64 * c, row, hk, page, bar);
                            tile_copy4(v_at + c * 2048, &v_map, 64 * c, row, hk, page, bar);
                        }
                    } else {
                        if (p0 < keys) atomicOr(a.errors, kErrorInput);
                        barrier_arrive(bar);
                    }
                }
                __syncwarp();
            } else {
                // lane r (and r + 16) has the row of key r: its element offset, -1 behind the keys, -2 on a bad page
                int64_t off = -1;
                const int p = p0 + lane % 16;
                if (p < keys) {
                    if (page >= 0 && page < a.pages) {
                        off = ((((int64_t)page * a.Hkv + hk) << a.page_shift) + (p & ((1 << a.page_shift) - 1))) * D;
                    } else {
                        off = -2;
                        atomicOr(a.errors, kErrorInput);
                    }
                }
                const int chunk = lane % CH;
#pragma unroll
                for (int i = 0; i < 16 * CH / 32; ++i) {
                    const int r = i * (32 / CH) + lane / CH;
                    const int64_t o = __shfl_sync(~0u, off, r);
                    const int d = chunk_at(r, chunk);
                    if (o == -2) {
                        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(k_at + d), "r"(0x7FFF7FFFu) : "memory");
                        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(v_at + d), "r"(0x7FFF7FFFu) : "memory");
                    } else {
                        const int64_t e = o < 0 ? 0 : o + chunk * 8;
                        copy16(k_at + d, (const E *)a.kc + e, o >= 0);
                        copy16(v_at + d, (const E *)a.vc + e, o >= 0);
                    }
                }
            }
            step<ROWS, kTileKeys, kPiece>(a, ahead);
            if (ahead.pos < span) {
                page = page_of(ahead.kt * kTileKeys + 16 * warp + (kTiled ? 0 : lane % 16));
            }
        }
        if (!kTiled) copies_close();
        load_stage = load_stage + 1 == S ? 0 : load_stage + 1;
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) load_tile();

    // ---- the pieces -------------------------------------------------------------
    int stage = 0, last_stage = 0;
    uint32_t phase = 0;
    while (at.pos < span) {
        const Seq q = at.q;
        const int hk = at.item / q.row_tiles, rt = at.item % q.row_tiles;
        const int kt0 = at.kt, kt1 = a.whole ? q.tiles : (int)min((int64_t)q.tiles, at.kt + span - at.pos);
        const int64_t item_end = at.pos - kt0 + q.tiles;
        const int rows = min(ROWS, q.m * a.group - rt * ROWS);

        // the rows' queries and masks (row r: token r / group, head r % group of the key head's)
        __syncthreads();
        for (int i = tid; i < ROWS * CH; i += kThreads) {
            const int r = i / CH, c = i % CH, rr = rt * ROWS + r;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                const int token = q.first + rr / a.group, h = hk * a.group + rr % a.group;
                v = *reinterpret_cast<const uint4 *>((const E *)a.q + (size_t)token * a.ldq + (size_t)h * D + c * 8);
            }
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(q_at + r / 16 * kHalf + chunk_at(r % 16, c)), "r"(v.x),
                         "r"(v.y), "r"(v.z), "r"(v.w)
                         : "memory");
        }
        if (tid < ROWS) {
            const int i = (rt * ROWS + tid) / a.group;
            uint64_t bits = 0;
            if (tid < rows) bits = a.mask ? a.mask[q.first + i] : ~0ull >> (63 - i);
            s_mask[tid] = q.m < 64 ? bits & ((1ull << q.m) - 1) : bits;
        }
        __syncthreads();
        auto queries = [&](int t, int d, uint32_t (&r)[4]) {
            ldmatrix4(r, q_at + (wr * MT + t) * kHalf + chunk_at(lane % 16, 2 * d + lane / 16));
        };
        uint32_t held[kQueriesHeld ? D / 16 : 1][4];
        if constexpr (kQueriesHeld) {
#pragma unroll
            for (int d = 0; d < D / 16; ++d) queries(0, d, held[d]);
        }

        float o[MT][D / 8][4] = {};
        float m[MT][2], l[MT][2];   // m: what the weights so far are relative to, from a (scaled) maximum
#pragma unroll
        for (int t = 0; t < MT; ++t) m[t][0] = m[t][1] = -INFINITY, l[t][0] = l[t][1] = 0.0f;

        for (int kt = kt0; kt < kt1; ++kt) {
            bool there = true;
            if constexpr (kTiled) {
                if (kOwnKeys) {
                    there = barrier_wait(smem_address(&full[stage][warp]), phase, gave_up);
                } else {
                    for (int i = 0; i < KW / 16; ++i) there &= barrier_wait(smem_address(&full[stage][wk * (KW / 16) + i]), phase, gave_up);
                }
            } else {
                copies_wait<S - 2>();
            }
            if (kOwnKeys) {
                __syncwarp();
                if (kTiled) lost |= !__all_sync(~0u, there);
            } else {
                lost |= !__syncthreads_and(there);
            }
            load_tile();   // into the place of the tile before, which its readers have left
            const uint32_t keys_at = stages + stage * kStageBytes<D> + wk * (KW / 16) * kSlice<D>, values_at = keys_at + kHalf;

            float s[MT][NT][4] = {};
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                uint32_t qa[MT][4];
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if constexpr (kQueriesHeld) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) qa[t][x] = held[d][x];
                    } else {
                        queries(t, d, qa[t]);
                    }
                }
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t kb[4];
                    ldmatrix4(kb, keys_at + j / 2 * kSlice<D> + chunk_at(lane % 8 + (lane / 16) * 8, 2 * d + (lane / 8) % 2));
#pragma unroll
                    for (int t = 0; t < MT; ++t) mma<E>(s[t][j], qa[t], kb[0], kb[1]), mma<E>(s[t][j + 1], qa[t], kb[2], kb[3]);
                }
            }

            const int tile_key = kt * kTileKeys, key0 = wk * KW;
            const bool partly = tile_key + kTileKeys > q.len;   // some keys are drafted, or behind the last
            if (partly) {
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint64_t bits = s_mask[(wr * MT + t) * 16 + half * 8 + lane / 4];
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int dj = tile_key + key0 + 8 * j + 2 * (lane % 4) + e - q.len;
                                const bool sees = dj < 0 || (dj < 64 && (bits >> dj & 1));
                                if (!sees) s[t][j][2 * half + e] = -INFINITY;
                            }
                    }
            }

            // The outputs are rescaled only when a row's maximum has grown by more than 2^8 since the last time:
            // the sum carries the same factor, and weights that much larger fit either type.
            float top[MT][2];
            bool grown = false;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float x = -INFINITY;
#pragma unroll
                    for (int j = 0; j < NT; ++j) x = fmaxf(x, fmaxf(s[t][j][2 * half], s[t][j][2 * half + 1]));
                    x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(~0u, x, 2));
                    top[t][half] = x * a.scale_log2 - kHeadroomLog2<E>;
                    grown |= top[t][half] > m[t][half] + kRescaleLog2;   // also the first finite score of a row
                }
            if (__any_sync(~0u, grown)) {
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const bool up = top[t][half] > m[t][half] + kRescaleLog2;
                        const float f = up ? exp2_approx(m[t][half] - top[t][half]) : 1.0f;
                        if (up) m[t][half] = top[t][half];
                        l[t][half] *= f;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) o[t][j][2 * half] *= f, o[t][j][2 * half + 1] *= f;
                    }
            }
            // For up to 16 rows the weights meet the values as two operands, the rounded weight and what the rounding
            // left: beside the stream of keys the second product costs nothing there, and the weights lose no more
            // than 2^-16 of their size (fp16: or 2^-32 of the largest).  For more rows it would cost 12%; there they
            // are rounded once.
            uint32_t pa[MT][NT / 2][4], pr[MT][NT / 2][4];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float ref = m[t][half] == -INFINITY ? 0.0f : m[t][half];
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const float p0 = exp2_approx(fmaf(s[t][j][2 * half], a.scale_log2, -ref));
                        const float p1 = exp2_approx(fmaf(s[t][j][2 * half + 1], a.scale_log2, -ref));
                        sum += p0 + p1;
                        const uint32_t near = pack2<E>(p0, p1);
                        pa[t][j / 2][(j % 2) * 2 + half] = near;
                        if constexpr (kTwoParts) {
                            const float2 had = unpack2<E>(near);
                            pr[t][j / 2][(j % 2) * 2 + half] = pack2<E>(p0 - had.x, p1 - had.y);
                        }
                    }
                    l[t][half] += sum;
                }

            if (partly) {
                // the warp that loaded the values clears those behind the keys (they may be anything) and
                // looks for others that are not finite
                const uint32_t own = stages + stage * kStageBytes<D> + warp * kSlice<D> + kHalf;
                const int there = q.len + q.m - tile_key - 16 * warp;   // rows of its 16 that are keys
                bool odd = false;
                for (int i = lane; i < kHalf / 16; i += 32) {
                    if (i / 8 % 16 >= there) {
                        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(own + 16 * i), "r"(0) : "memory");
                        continue;
                    }
                    uint4 v;
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(own + 16 * i) : "memory");
                    odd |= not_finite<E>(v.x) || not_finite<E>(v.y) || not_finite<E>(v.z) || not_finite<E>(v.w);
                }
                writes_before_async();
                if (kOwnKeys) __syncwarp();   // other lanes read the cleared rows, and a vote orders no memory
                odd = kOwnKeys ? __any_sync(~0u, odd) : __syncthreads_or(odd);
                if (odd) {
                    for (int kk = 0; kk < KW; ++kk) {
                        const int dj = tile_key + key0 + kk - q.len;
#pragma unroll
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const uint64_t bits = s_mask[(wr * MT + t) * 16 + half * 8 + lane / 4];
                                if (!(dj < 0 || (dj < 64 && (bits >> dj & 1)))) continue;
#pragma unroll
                                for (int j = 0; j < D / 8; ++j) {
                                    uint32_t v;
                                    asm volatile("ld.shared.b32 %0, [%1];"
                                                 : "=r"(v)
                                                 : "r"(values_at + kk / 16 * kSlice<D> + chunk_at(kk % 16, j) + 4 * (lane % 4))
                                                 : "memory");
                                    if (not_finite<E>(v)) {
                                        const float2 f = unpack2<E>(v ^ finite_part<E>(v));
                                        o[t][j][2 * half] += f.x, o[t][j][2 * half + 1] += f.y;
                                    }
                                }
                            }
                    }
                    if (kOwnKeys) __syncwarp();
                    else __syncthreads();
                    for (int i = lane; i < kHalf / 4; i += 32) {
                        uint32_t v;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(own + 4 * i) : "memory");
                        if (not_finite<E>(v)) asm volatile("st.shared.b32 [%0], %1;" ::"r"(own + 4 * i), "r"(finite_part<E>(v)) : "memory");
                    }
                    writes_before_async();
                    if (kOwnKeys) __syncwarp();
                    else __syncthreads();
                }
            }

#pragma unroll
            for (int c = 0; c < NT / 2; ++c)
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    uint32_t vb[4];
                    ldmatrix4_trans(vb, values_at + c * kSlice<D> + chunk_at(lane % 16, 2 * d + lane / 16));
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        mma<E>(o[t][2 * d], pa[t][c], vb[0], vb[1]), mma<E>(o[t][2 * d + 1], pa[t][c], vb[2], vb[3]);
                        if constexpr (kTwoParts)
                            mma<E>(o[t][2 * d], pr[t][c], vb[0], vb[1]), mma<E>(o[t][2 * d + 1], pr[t][c], vb[2], vb[3]);
                    }
                }

            last_stage = stage;
            if (++stage == S) stage = 0, phase ^= 1;
            step<ROWS, kTileKeys, kPiece>(a, at);
        }

        // ---- join the key warps through the last tile's place (free until the next tile is
        // asked for, behind the next piece's first barrier): 16 rows a warp at a time ----
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                l[t][half] += __shfl_xor_sync(~0u, l[t][half], 1);
                l[t][half] += __shfl_xor_sync(~0u, l[t][half], 2);
                if (lane % 4 == 0) {
                    s_ml[0][warp][t * 16 + half * 8 + lane / 4] = m[t][half];
                    s_ml[1][warp][t * 16 + half * 8 + lane / 4] = l[t][half];
                }
            }
        const bool whole = kt0 == 0 && kt1 == q.tiles;
        const size_t piece = 2 * (size_t)blockIdx.x + (kt0 == 0 ? 1 : 0);
        uint8_t *join = smem + last_stage * kStageBytes<D>;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            __syncthreads();   // all warps are done with the tile (or with the rows before)
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    const int r = half * 8 + lane / 4, c = 2 * j + (lane % 4) / 2;
                    *reinterpret_cast<float2 *>(join + warp * kSlice<D> + r * D * 4 + ((c ^ (r & 7) * 2) << 4) + (lane % 2) * 8) =
                        make_float2(o[t][j][2 * half], o[t][j][2 * half + 1]);
                }
            writes_before_async();
            __syncthreads();
            // warp (wr, wk) takes the columns wk of WK of its row warp's 16 rows, four at a time
            constexpr int CW = D / 4 / WK;                     // chunks of four columns a warp joins
            for (int i = lane; i < 16 * CW; i += 32) {
                const int r = i / CW, c = wk * CW + i % CW, row = (wr * MT + t) * 16 + r;
                if (row >= rows) continue;
                float best = -INFINITY;
#pragma unroll
                for (int x = 0; x < WK; ++x) best = fmaxf(best, s_ml[0][x * WR + wr][t * 16 + r]);
                const float ref = best == -INFINITY ? 0.0f : best;
                float4 y = make_float4(0, 0, 0, 0);
                float sum = 0.0f;
#pragma unroll
                for (int x = 0; x < WK; ++x) {
                    const int w = x * WR + wr;
                    const float f = exp2_approx(s_ml[0][w][t * 16 + r] - ref);
                    const float4 v = *reinterpret_cast<const float4 *>(join + w * kSlice<D> + r * D * 4 + ((c ^ (r & 7) * 2) << 4));
                    sum = fmaf(f, s_ml[1][w][t * 16 + r], sum);
                    y.x = fmaf(f, v.x, y.x), y.y = fmaf(f, v.y, y.y), y.z = fmaf(f, v.z, y.z), y.w = fmaf(f, v.w, y.w);
                }
                if (whole) {
                    const int rr = rt * ROWS + row, token = q.first + rr / a.group, h = hk * a.group + rr % a.group;
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    uint2 packed;
                    packed.x = pack2<E>(y.x * inv, y.y * inv), packed.y = pack2<E>(y.z * inv, y.w * inv);
                    *reinterpret_cast<uint2 *>((E *)a.out + (size_t)token * a.ldo + (size_t)h * D + 4 * c) = packed;
                    if (a.lse && c == 0)
                        a.lse[(size_t)token * a.Hkv * a.group + h] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.69314718056f;
                } else {
                    *reinterpret_cast<float4 *>(a.part + (piece * ROWS + row) * D + 4 * c) = y;
                    if (c == 0) *reinterpret_cast<float2 *>(a.part_ml + (piece * ROWS + row) * 2) = make_float2(best, sum);
                }
            }
        }
        // the CTA where a cut sequence begins tells the join where it lies and in which CTA it ends
        if (!whole && kt0 == 0 && tid == 0) {
            a.records[blockIdx.x] = make_int4((int)((r.begin + item_end - 1) / r.run) + 1, q.first, hk * q.row_tiles + rt, rows | q.row_tiles << 16);
        }
    }
    if (!kTiled) copies_wait<0>();
    if (lost) {
        outlast_copies();
        if (lane == 0) atomicOr(a.errors, kErrorWait);
    }
}

// Joins the pieces of the cut items: block x the one that begins in CTA x.  A thread takes four columns of a row;
// where an item has fewer of them than the block threads, several share its pieces.  Several pieces are asked
// for before the first is used.  The order is fixed, so results do not depend on timing.
// The tensor-core tiles leave their rows side by side (a thread a row), the others their columns.
template <int ROWS>
constexpr int kJoinThreads = ROWS == kTreeTileRows ? 128 : 512;

template <typename E, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads<ROWS>) join_kernel(const TreeArgs a) {
    constexpr bool kRowsBeside = ROWS == kTreeTileRows;
    constexpr int CH = D / 4, kBlockThreads = kJoinThreads<ROWS>, kAtOnce = kRowsBeside ? 4 : 8;
    __shared__ float4 s_y[kBlockThreads];
    __shared__ float2 s_ml[kBlockThreads];
    wait_for_previous_kernel();
    const int4 rec = a.records[blockIdx.x];
    const int row_tiles = rec.w >> 16, rows = rec.w & 0xFFFF;   // tensor-core tiles: the drafted tokens
    if (rec.x == 0) return;
    const int first = blockIdx.x, last = rec.x - 1, tid = threadIdx.x;
    const int units = kRowsBeside ? ROWS * CH : rows * CH;
    // threads that share a unit: as many as fit, a power of two, no more than there are pieces
    int shares = 1;
    while (!kRowsBeside && 2 * shares * units <= kBlockThreads && 2 * shares <= last - first + 1) shares *= 2;
    const int at_once = shares > 1 ? units : kBlockThreads;   // units a pass
    for (int u0 = blockIdx.y * at_once; u0 < units; u0 += gridDim.y * at_once) {
        const int unit = u0 + tid % at_once, share = tid / at_once;
        const int row = kRowsBeside ? unit % ROWS : unit / CH, c = kRowsBeside ? unit / ROWS : unit % CH;
        const int hk = rec.z / row_tiles, rt = rec.z % row_tiles, rr = rt * ROWS + row;
        const int token = kRowsBeside ? tile_token(a, rt, row / 128, row % 128, rows) : rr / a.group;
        const int h = hk * a.group + (kRowsBeside ? row % 128 : rr) % a.group;
        const bool mine = unit < units && share < shares && (kRowsBeside ? token >= 0 : row < rows);
        float top = -INFINITY, sum = 0.0f;
        float4 y = make_float4(0, 0, 0, 0);
        for (int x0 = first + share; mine && x0 <= last; x0 += kAtOnce * shares) {
            float2 ml[kAtOnce];
            float4 v[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int x = x0 + i * shares;
                ml[i] = make_float2(-INFINITY, 0.0f), v[i] = make_float4(0, 0, 0, 0);
                if (x > last) continue;
                const size_t piece = 2 * (size_t)x + (x == first ? 1 : 0);
                ml[i] = *reinterpret_cast<const float2 *>(a.part_ml + (piece * ROWS + row) * 2);
                v[i] = reinterpret_cast<const float4 *>(a.part)[kRowsBeside ? (piece * CH + c) * ROWS + row : (piece * ROWS + row) * CH + c];
            }
            float best = top;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) best = fmaxf(best, ml[i].x);
            const float ref = best == -INFINITY ? 0.0f : best, f = exp2_approx(top - ref);
            top = best, sum *= f, y.x *= f, y.y *= f, y.z *= f, y.w *= f;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const float g = exp2_approx(ml[i].x - ref);
                sum = fmaf(g, ml[i].y, sum);
                y.x = fmaf(g, v[i].x, y.x), y.y = fmaf(g, v[i].y, y.y), y.z = fmaf(g, v[i].z, y.z), y.w = fmaf(g, v[i].w, y.w);
            }
        }
        if (shares > 1) {   // one pass: the block's threads meet once
            s_ml[tid] = make_float2(top, sum), s_y[tid] = y;
            __syncthreads();
            if (share == 0) {
                float best = -INFINITY;
                for (int i = 0; i < shares; ++i) best = fmaxf(best, s_ml[tid + i * units].x);
                const float ref = best == -INFINITY ? 0.0f : best;
                top = best, sum = 0.0f, y = make_float4(0, 0, 0, 0);
                for (int i = 0; i < shares; ++i) {
                    const float g = exp2_approx(s_ml[tid + i * units].x - ref);
                    const float4 v = s_y[tid + i * units];
                    sum = fmaf(g, s_ml[tid + i * units].y, sum);
                    y.x = fmaf(g, v.x, y.x), y.y = fmaf(g, v.y, y.y), y.z = fmaf(g, v.z, y.z), y.w = fmaf(g, v.w, y.w);
                }
            }
        }
        if (!mine || share > 0) continue;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint2 packed;
        packed.x = pack2<E>(y.x * inv, y.y * inv), packed.y = pack2<E>(y.z * inv, y.w * inv);
        *reinterpret_cast<uint2 *>((E *)a.out + (size_t)(rec.y + token) * a.ldo + (size_t)h * D + 4 * c) = packed;
        if (a.lse && c == 0)
            a.lse[(size_t)(rec.y + token) * a.Hkv * a.group + h] =
                sum == 0.0f ? -INFINITY : ((top == -INFINITY ? 0.0f : top) + log2f(sum)) * 0.69314718056f;
    }
}

// How a call is cut: the rows of a piece, by the rows that a key head has at most, and the CTAs.
struct Shape {
    int rows, ctas;
    bool tiles;   // on the fifth-generation tensor cores
    bool whole;   // items are not cut: where every sequence is short, that gains less than the second launch costs
};
Shape shape_of(int Hq, const fb_kv_cache &c, int max_draft, int table_width) {
    const int group = Hq / c.Hkv, most = max_draft * group;
    if (most > 32 && group <= 128 && c.page_size >= 8) return {kTreeTileRows, sm_count(), true, false};
    return {most <= 16 ? 16 : most <= 32 ? 32 : 64, sm_count() * kCtasPerSm, false,
            (int64_t)table_width * c.page_size <= kWholeKeys};
}

// The workspace: the pieces' outputs, their maxima and sums, a record a CTA.
struct Workspace {
    size_t ml, records, bytes;
};
Workspace workspace(const Shape &sh, int D) {
    const size_t pieces = 2 * (size_t)sh.ctas;
    Workspace w;
    w.ml = pieces * sh.rows * D * sizeof(float);
    w.records = w.ml + pieces * sh.rows * 2 * sizeof(float);
    w.bytes = w.records + sh.ctas * sizeof(int4);
    return w;
}

template <typename E, int D, int ROWS>
cudaError_t launch_join(const TreeArgs &a, int ctas, cudaStream_t s) {
    const int passes = ROWS == kTreeTileRows ? ROWS * D / 4 / kJoinThreads<ROWS> : 1;
    return launch(join_kernel<E, D, ROWS>, dim3(ctas, passes), dim3(kJoinThreads<ROWS>), 0, s, true, a);
}

template <typename E, int D, int WR, int WK, int MT, bool kTiled>
cudaError_t launch_tree(const TreeArgs &a, const fb_kv_cache &cache, bool pdl, cudaStream_t s) {
    constexpr int ROWS = WR * MT * 16, smem = tree_smem_bytes<D, ROWS>();
    CUtensorMap k = {}, v = {};
    if (kTiled && (!cache_map(&k, cache.k, cache, 16) || !cache_map(&v, cache.v, cache, 16))) return cudaErrorInvalidValue;
    cudaError_t e = allow_shared<tree_kernel<E, D, WR, WK, MT, kTiled>>(smem);
    if (e != cudaSuccess) return e;
    const dim3 grid(sm_count() * kCtasPerSm);
    e = launch(tree_kernel<E, D, WR, WK, MT, kTiled>, grid, dim3(kThreads), smem, s, pdl, a, k, v);
    if (e != cudaSuccess) return e;
    return a.whole ? cudaSuccess : launch_join<E, D, ROWS>(a, grid.x, s);
}

template <typename E, int D, int WR, int WK, int MT>
cudaError_t launch_tree_pages(const TreeArgs &a, const fb_kv_cache &cache, bool pdl, cudaStream_t s) {
    return cache.page_size >= 16 ? launch_tree<E, D, WR, WK, MT, true>(a, cache, pdl, s)
                                 : launch_tree<E, D, WR, WK, MT, false>(a, cache, pdl, s);
}

template <typename E, int D>
cudaError_t launch_tree_rows(const TreeArgs &a, const fb_kv_cache &cache, const Shape &sh, bool pdl, cudaStream_t s) {
    if (sh.tiles) {
        const cudaError_t e = launch_tree_tiles(a, cache, pdl, s);
        return e != cudaSuccess ? e : launch_join<E, D, kTreeTileRows>(a, sh.ctas, s);
    }
    const int rows = sh.rows;
    if (rows == 16) return launch_tree_pages<E, D, 1, 4, 1>(a, cache, pdl, s);
    if (rows == 32) return launch_tree_pages<E, D, 1, 4, 2>(a, cache, pdl, s);
    return launch_tree_pages<E, D, 2, 2, 2>(a, cache, pdl, s);
}

}  // namespace

void *attn_errors_address() {
    static std::atomic<void *> cached[64];   // by device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    void *p = cached[dev].load(std::memory_order_relaxed);
    if (!p) {
        if (cudaGetSymbolAddress(&p, g_attn_errors) != cudaSuccess) return nullptr;
        cached[dev].store(p, std::memory_order_relaxed);
    }
    return p;
}

}  // namespace fb

using namespace fb;

extern "C" size_t fb_attn_tree_workspace_bytes(int Hq, const fb_kv_cache *cache, int max_draft, int table_width) {
    if (!cache || !valid_cache(*cache) || Hq < 1 || Hq > kMaxHeads || Hq % cache->Hkv ||
        (cache->D != 64 && cache->D != 128) || max_draft < 1 || max_draft > 64 || table_width < 1)
        return 0;
    const Shape sh = shape_of(Hq, *cache, max_draft, table_width);
    return sh.whole ? 0 : workspace(sh, cache->D).bytes;
}

extern "C" fb_status fb_attn_tree(const void *q, int ldq, int T, int Hq, const fb_kv_cache *cache,
                                  const int32_t *page_table, int table_width, int ld_table, const int32_t *lens,
                                  const int32_t *cu_draft, int n, int max_draft, const uint64_t *mask, float scale,
                                  void *out, int ldo, float *lse, void *ws, size_t ws_bytes, unsigned flags,
                                  void *stream) {
    if (!q || !cache || !page_table || !lens || !out || (flags & ~FB_GEMV_PDL) || !valid_cache(*cache) || T < 1 ||
        T > kMaxTokens || Hq < 1 || Hq > kMaxHeads || Hq % cache->Hkv || n < 1 || n > 65536 || table_width < 1 ||
        ld_table < table_width ||
        max_draft < 1 || max_draft > 64 || (!cu_draft && T != n) || !(scale > 0.0f) || scale > 1e38f || out == q)
        return FB_ERR_INVALID_VALUE;
    const int D = cache->D;
    if (ldq < (int64_t)Hq * D || ldo < (int64_t)Hq * D) return FB_ERR_INVALID_VALUE;
    if (D != 64 && D != 128) return FB_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache->k, 16) || !aligned(cache->v, 16) || ldq % 8 ||
        ldo % 8 || !aligned(page_table, 4) || !aligned(lens, 4) || !aligned(cu_draft, 4) || !aligned(mask, 8) ||
        !aligned(lse, 4))
        return FB_ERR_MISALIGNED;
    const int group = Hq / cache->Hkv;
    const Shape sh = shape_of(Hq, *cache, max_draft, table_width);
    const Workspace w = workspace(sh, D);
    if (!sh.whole && (!ws || !aligned(ws, 16) || ws_bytes < w.bytes)) return FB_ERR_WORKSPACE;
    TreeArgs a = {};
    a.q = q, a.kc = cache->k, a.vc = cache->v, a.out = out, a.lse = lse;
    a.table = page_table, a.lens = lens, a.cu = cu_draft, a.mask = mask;
    if (!sh.whole)
        a.part = (float *)ws, a.part_ml = (float *)((char *)ws + w.ml), a.records = (int4 *)((char *)ws + w.records);
    a.n = n, a.T = T, a.Hkv = cache->Hkv, a.group = group, a.ldq = ldq, a.ldo = ldo;
    a.table_width = table_width, a.ld_table = ld_table, a.max_draft = max_draft;
    a.pages = cache->pages, a.page_shift = log2_of(cache->page_size);
    a.scale_log2 = scale * 1.44269504089f;
    a.errors = (unsigned int *)attn_errors_address();
    if (!a.errors) return FB_ERR_CUDA;
    a.whole = sh.whole;
    a.tile_tokens = group <= 128 ? 128 / group : 0;
    const bool pdl = flags & FB_GEMV_PDL;
    cudaStream_t s = as_stream(stream);
    if (cache->t == FB_F16)
        return status_of(D == 64 ? launch_tree_rows<__half, 64>(a, *cache, sh, pdl, s)
                                 : launch_tree_rows<__half, 128>(a, *cache, sh, pdl, s));
    return status_of(D == 64 ? launch_tree_rows<__nv_bfloat16, 64>(a, *cache, sh, pdl, s)
                             : launch_tree_rows<__nv_bfloat16, 128>(a, *cache, sh, pdl, s));
}

extern "C" fb_status fb_attn_errors(unsigned int *flags, int clear) {
    if (!flags) return FB_ERR_INVALID_VALUE;
    if (cudaDeviceSynchronize() != cudaSuccess) return FB_ERR_CUDA;
    void *word = attn_errors_address();
    if (!word || cudaMemcpy(flags, word, sizeof(unsigned int), cudaMemcpyDeviceToHost) != cudaSuccess)
        return FB_ERR_CUDA;
    const unsigned int zero = 0;
    if (clear && cudaMemcpy(word, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess) return FB_ERR_CUDA;
    return FB_OK;
}
