// attn_prompt.cu -- causal attention of packed prompts (the kernel: attn_tiles.cuh).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "attn_tiles.cuh"
#include "fb_internal.cuh"

namespace fb {
namespace {

// Up to this many full items for ten SMs, items are split.  Measured, split and not: 150 items, the longest of
// 12,066 keys, 95 and 148 us; 75 items of up to 3,431 keys 30 and 47; 128 even items of 1,000 25 and 23; 256 even
// items of 4,096 92 and 71 (each key tile then serves half as many queries).  The host knows the total of tokens and
// not the lengths, so few even items are split too.
constexpr int kSplitItems = 11;


template <typename E, int D, typename Args>
cudaError_t launch_items(const Args &a, int64_t most, const fb_heads &in, bool pdl, cudaStream_t s) {
    CUtensorMap q, k, v;
    if (!head_map(&q, in.q, in.t, in.T, in.Hq, D, in.ldq, 1, kTile) ||
        !head_map(&k, in.k, in.t, in.T, in.Hkv, D, in.ldk, 1, kTile) ||
        !head_map(&v, in.v, in.t, in.T, in.Hkv, D, in.ldv, 1, kTile))
        return cudaErrorInvalidValue;
    // a warp would wait for registers for good
    if (!registers_as_planned<tile_kernel<E, D, Args>>()) return cudaErrorInvalidValue;
    const cudaError_t e = allow_shared<tile_kernel<E, D, Args>>(kSmemBytes<D>);
    if (e != cudaSuccess) return e;
    // one CTA an SM, no more than there can be items
    const int ctas = (int)(most < sm_count() ? most : sm_count());
    return launch(tile_kernel<E, D, Args>, dim3(ctas), dim3(kTileThreads), kSmemBytes<D>, s, pdl, a, q, k, v);
}

// Items of 256 queries where they go round the SMs, else of 128, split over their keys.
template <typename E, int D>
cudaError_t launch_prompt(const PromptArgs &a, const fb_heads &in, bool pdl, cudaStream_t s) {
    const int64_t n = a.n < in.T ? a.n : in.T, blocks = (in.T + kBlock - 1) / kBlock;
    if (blocks * in.Hq * 10 <= kSplitItems * (int64_t)sm_count())
        return launch_items<E, D>(SplitArgs{a}, ((in.T + kTile - 1) / kTile + n) * in.Hq, in, pdl, s);
    return launch_items<E, D>(a, (blocks + n) * in.Hq, in, pdl, s);
}

}  // namespace
}  // namespace fb

using namespace fb;

extern "C" fb_status fb_attn_prompt(const fb_heads *in, const int32_t *cu_seqlens, int n, float scale, void *out,
                                    int ldo, float *lse, unsigned flags, void *stream) {
    if (!in || (flags & ~FB_GEMV_PDL) || !valid_heads(*in) || !in->q || !in->k || !in->v || !out || !cu_seqlens ||
        n < 1 || n > kMaxTokens || ldo < in->Hq * in->D || !(scale > 0.0f) || scale > 1e38f ||
        out == in->q || out == in->k || out == in->v)
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
