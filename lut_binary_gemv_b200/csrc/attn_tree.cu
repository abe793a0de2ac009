// attn_tree.cu -- attention of single tokens and of trees of drafted tokens
// over a paged cache.
//
//   out_i = sum_j p_ij v_j over the committed keys and the drafted keys whose
//   bit is set in the token's mask, p the softmax of scale q_i.k_j.
//
// One warp a row: right for every case, bound by re-reading the keys for
// every row and by one warp's walk along a long cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "fb_internal.cuh"

namespace fb {
namespace {

constexpr int kThreads = 128;

__device__ unsigned int g_attn_errors;

struct TreeArgs {
    const void *q, *kc, *vc;
    void *out;
    float *lse;
    const int32_t *table, *lens, *cu;
    const uint64_t *mask;
    int n, T, Hq, Hkv, ldq, ldo, table_width, ld_table, max_draft, pages, page_shift;
    float scale;
};

template <typename E, int D>
__global__ void __launch_bounds__(kThreads) tree_rows_kernel(const TreeArgs a) {
    wait_for_previous_kernel();
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x % 32, i = (int)(row / a.Hq), h = (int)(row % a.Hq);
    if (i >= a.T) return;
    int seq = i, first = i, m_s = 1;
    if (a.cu) {
        int lo = 0, hi = a.n;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (mid < a.n && a.cu[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        seq = lo, first = max(a.cu[lo], 0);
        const int end = min(a.cu[lo + 1], a.T);
        if (i < first || i >= end) return;
        m_s = end - first;
        if (m_s > a.max_draft) {
            m_s = a.max_draft;
            if (lane == 0) atomicOr(&g_attn_errors, 2u);
            if (i - first >= m_s) return;
        }
    }
    const int len = max(a.lens[seq], 0), d = i - first;
    const uint64_t bits = a.mask ? a.mask[i] : ~0ull >> (63 - d);
    constexpr int P = D / 64;
    const E *q = (const E *)a.q + (size_t)i * a.ldq + (size_t)h * D;
    const int hk = h / (a.Hq / a.Hkv);
    float2 qv[P], o[P] = {};
    for (int p = 0; p < P; ++p) qv[p] = unpack2<E>(((const uint32_t *)q)[32 * p + lane]);
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = 0; j < (int64_t)len + m_s; ++j) {
        if (j >= len && !(bits >> (j - len) & 1)) continue;
        const int64_t slot = j >> a.page_shift;
        const int page = slot < a.table_width ? a.table[(size_t)seq * a.ld_table + slot] : -1;
        if (page < 0 || page >= a.pages) {
            if (lane == 0) atomicOr(&g_attn_errors, 2u);
            l = NAN;
            break;
        }
        const size_t at = ((((size_t)page * a.Hkv + hk) << a.page_shift) + (j - (slot << a.page_shift))) * D;
        const uint32_t *k = (const uint32_t *)((const E *)a.kc + at), *v = (const uint32_t *)((const E *)a.vc + at);
        float s = 0.0f;
        for (int p = 0; p < P; ++p) {
            const float2 kv = unpack2<E>(k[32 * p + lane]);
            s = fmaf(qv[p].x, kv.x, fmaf(qv[p].y, kv.y, s));
        }
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
        s *= a.scale;
        const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.0f : expf(m - mn), w = expf(s - mn);
        l = l * f + w, m = mn;
        for (int p = 0; p < P; ++p) {
            const float2 vv = unpack2<E>(v[32 * p + lane]);
            o[p].x = o[p].x * f + w * vv.x, o[p].y = o[p].y * f + w * vv.y;
        }
    }
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t *out = (uint32_t *)((E *)a.out + (size_t)i * a.ldo + (size_t)h * D);
    for (int p = 0; p < P; ++p) out[32 * p + lane] = pack2<E>(o[p].x * r, o[p].y * r);
    if (a.lse && lane == 0) a.lse[(size_t)i * a.Hq + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

void *attn_errors_address() {
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_attn_errors) == cudaSuccess ? p : nullptr;
}

}  // namespace fb

using namespace fb;

extern "C" size_t fb_attn_tree_workspace_bytes(int Hq, int Hkv, int D, int max_draft) {
    if (Hq < 1 || Hq > kMaxHeads || Hkv < 1 || Hq % Hkv || (D != 64 && D != 128) || max_draft < 1 || max_draft > 64)
        return 0;
    return 16;
}

extern "C" fb_status fb_attn_tree(const void *q, int ldq, int T, int Hq, const fb_kv_cache *cache,
                                  const int32_t *page_table, int table_width, int ld_table, const int32_t *lens,
                                  const int32_t *cu_draft, int n, int max_draft, const uint64_t *mask, float scale,
                                  void *out, int ldo, float *lse, void *ws, size_t ws_bytes, unsigned flags,
                                  void *stream) {
    if (!q || !cache || !page_table || !lens || !out || (flags & ~FB_GEMV_PDL) || !valid_cache(*cache) || T < 1 ||
        T > kMaxTokens || Hq < 1 || Hq > kMaxHeads || Hq % cache->Hkv || n < 1 || n > 65536 || table_width < 1 ||
        ld_table < table_width ||
        max_draft < 1 || max_draft > 64 || (!cu_draft && T != n) || !(scale > 0.0f) || scale > 3e38f)
        return FB_ERR_INVALID_VALUE;
    const int D = cache->D;
    if (ldq < (int64_t)Hq * D || ldo < (int64_t)Hq * D) return FB_ERR_INVALID_VALUE;
    if (D != 64 && D != 128) return FB_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache->k, 16) || !aligned(cache->v, 16) || ldq % 8 ||
        ldo % 8 || !aligned(page_table, 4) || !aligned(lens, 4) || !aligned(cu_draft, 4) || !aligned(mask, 8) ||
        !aligned(lse, 4))
        return FB_ERR_MISALIGNED;
    if (!ws || !aligned(ws, 16) || ws_bytes < fb_attn_tree_workspace_bytes(Hq, cache->Hkv, D, max_draft))
        return FB_ERR_WORKSPACE;
    TreeArgs a = {q,  cache->k, cache->v,   out, lse, page_table, lens,     cu_draft,  mask,        n,
                  T,  Hq,       cache->Hkv, ldq, ldo, table_width, ld_table, max_draft, cache->pages, log2_of(cache->page_size), scale};
    const int64_t rows = (int64_t)T * Hq;
    const dim3 grid((unsigned)((rows + 3) / 4)), block(kThreads);
    const bool pdl = flags & FB_GEMV_PDL, half = cache->t == FB_F16;
    cudaStream_t s = as_stream(stream);
    if (D == 64)
        return status_of(half ? launch(tree_rows_kernel<__half, 64>, grid, block, 0, s, pdl, a)
                              : launch(tree_rows_kernel<__nv_bfloat16, 64>, grid, block, 0, s, pdl, a));
    return status_of(half ? launch(tree_rows_kernel<__half, 128>, grid, block, 0, s, pdl, a)
                          : launch(tree_rows_kernel<__nv_bfloat16, 128>, grid, block, 0, s, pdl, a));
}
