// attn_tree_tiles.cu -- drafted trees with many rows a key head on the tensor
// cores (the kernel: attn_tiles.cuh; the rest of fb_attn_tree: attn_tree.cu).
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

template <typename E, int D>
cudaError_t launch_tiles(const TreeArgs &a, const fb_kv_cache &cache, bool pdl, cudaStream_t s) {
    CUtensorMap q, k, v;
    const int rows = cache.page_size < kTile ? cache.page_size : kTile;
    if (!head_map(&q, a.q, cache.t, a.T, a.Hkv * a.group, D, a.ldq, a.group, a.tile_tokens) ||
        !cache_map(&k, cache.k, cache, rows) || !cache_map(&v, cache.v, cache, rows))
        return cudaErrorInvalidValue;
    if (!registers_as_planned<tile_kernel<E, D, TreeArgs>>()) return cudaErrorInvalidValue;
    const cudaError_t e = allow_shared<tile_kernel<E, D, TreeArgs>>(kSmemBytes<D>);
    if (e != cudaSuccess) return e;
    return launch(tile_kernel<E, D, TreeArgs>, dim3(sm_count()), dim3(kTileThreads), kSmemBytes<D>, s, pdl, a, q, k, v);
}

}  // namespace

// One CTA an SM, pieces of 256 rows.
cudaError_t launch_tree_tiles(const TreeArgs &a, const fb_kv_cache &cache, bool pdl, cudaStream_t s) {
    if (cache.t == FB_F16)
        return cache.D == 64 ? launch_tiles<__half, 64>(a, cache, pdl, s) : launch_tiles<__half, 128>(a, cache, pdl, s);
    return cache.D == 64 ? launch_tiles<__nv_bfloat16, 64>(a, cache, pdl, s)
                         : launch_tiles<__nv_bfloat16, 128>(a, cache, pdl, s);
}

}  // namespace fb
