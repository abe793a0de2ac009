// attn_prompt.cu -- causal attention of packed prompts.
//
//   out_i = sum_{j <= i} exp(scale q_i.k_j - m_i) v_j / sum_{j <= i} exp(scale q_i.k_j - m_i)
//
// over the tokens j of i's sequence, in one pass over the keys with the
// running maximum m and sum.  One warp a row: right for every case, bound by
// re-reading the keys for every row.
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

struct PromptArgs {
    const void *q, *k, *v;
    void *out;
    float *lse;
    const int32_t *cu;
    int n, T, Hq, Hkv, ldq, ldk, ldv, ldo;
    float scale;
};

template <typename E, int D>
__global__ void __launch_bounds__(kThreads) prompt_rows_kernel(const PromptArgs a) {
    wait_for_previous_kernel();
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x % 32, i = (int)(row / a.Hq), h = (int)(row % a.Hq);
    if (i >= a.T) return;
    // the last sequence that starts at or before token i, if it holds i
    int lo = 0, hi = a.n;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (mid < a.n && a.cu[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    const int first = max(a.cu[lo], 0);
    if (i < first || i >= a.cu[lo + 1]) return;
    constexpr int P = D / 64;
    const E *q = (const E *)a.q + (size_t)i * a.ldq + (size_t)h * D;
    const int hk = h / (a.Hq / a.Hkv);
    float2 qv[P], o[P] = {};
    for (int p = 0; p < P; ++p) qv[p] = unpack2<E>(((const uint32_t *)q)[32 * p + lane]);
    float m = -INFINITY, l = 0.0f;
    for (int j = first; j <= i; ++j) {
        const uint32_t *k = (const uint32_t *)((const E *)a.k + (size_t)j * a.ldk + (size_t)hk * D);
        const uint32_t *v = (const uint32_t *)((const E *)a.v + (size_t)j * a.ldv + (size_t)hk * D);
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
    uint32_t *out = (uint32_t *)((E *)a.out + (size_t)i * a.ldo + (size_t)h * D);
    for (int p = 0; p < P; ++p) out[32 * p + lane] = pack2<E>(o[p].x / l, o[p].y / l);
    if (a.lse && lane == 0) a.lse[(size_t)i * a.Hq + h] = m + logf(l);
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
    PromptArgs a = {in->q, in->k, in->v, out,     lse,     cu_seqlens, n,  in->T,
                    in->Hq, in->Hkv, in->ldq, in->ldk, in->ldv, ldo, scale};
    const int64_t rows = (int64_t)in->T * in->Hq;
    const dim3 grid((unsigned)((rows + 3) / 4)), block(kThreads);
    const bool pdl = flags & FB_GEMV_PDL, half = in->t == FB_F16;
    cudaStream_t s = as_stream(stream);
    if (in->D == 64)
        return status_of(half ? launch(prompt_rows_kernel<__half, 64>, grid, block, 0, s, pdl, a)
                              : launch(prompt_rows_kernel<__nv_bfloat16, 64>, grid, block, 0, s, pdl, a));
    return status_of(half ? launch(prompt_rows_kernel<__half, 128>, grid, block, 0, s, pdl, a)
                          : launch(prompt_rows_kernel<__nv_bfloat16, 128>, grid, block, 0, s, pdl, a));
}
