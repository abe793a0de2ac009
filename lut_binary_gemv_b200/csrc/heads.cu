// heads.cu -- between the q/k/v projections and the attention: the norm of
// each query and key head, the rotation by position, the conversion, and the
// write into the paged cache, in one pass over the heads.
//
//   x' = x * w / sqrt(mean(x^2) + eps);  (a, b) -> (a cos t - b sin t, b cos t + a sin t),
//   t = pos * inv_freq[pair]
//
// The work is one read and one write of every element (a dozen operations
// each): bytes bound long prompts, the launch and one dependent chain of
// loads bound single tokens.  A thread owns 16 elements of a head as two
// vectors of 8: both halves of 8 pairs, so a rotation never leaves the
// thread, and a head's sum of squares is log2(D/16) shuffles.  A block takes
// one token: its angles are computed once (one thread a pair) and shared by
// all its heads.  The angle is reduced in turns in fp64 (pos * inv_freq /
// 2 pi minus its integer), which keeps the error of a position of a million
// at 1e-10 turns, where fp32 would be off by a hundredth of a turn.
// Measured: 16,384 tokens of 64 + 2 x 8 heads of 128, bf16, 116 us, 5.8 TB/s of
// the 6.5 of a copy (blocks of 128 threads 125 us, angles and weights kept in
// registers at half the occupancy 152 us); one token 2.6 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_common.cuh"
#include "fb_internal.cuh"

namespace fb {
namespace {

constexpr int kThreads = 64;

struct RotateArgs {
    const void *q, *k, *v;
    void *qo, *ko, *vo, *kc, *vc;
    int ldq, ldk, ldv, ldqo, ldko, ldvo;
    const int32_t *pos, *slots;
    const double *inv_freq;
    const float *wq, *wk;
    float eps;
    int Hq, Hkv, D, rot, page_shift, neighbours;
    int64_t n_slots;
};

// 8 consecutive elements, as loaded.
template <typename T>
struct Vec8 {
    uint4 r[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T *p) {
    Vec8<T> v;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v.r[i] = reinterpret_cast<const uint4 *>(p)[i];
    return v;
}
__device__ __forceinline__ void widen(const Vec8<float> &v, float *f) {
    const float *s = reinterpret_cast<const float *>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = s[i];
}
__device__ __forceinline__ void widen(const Vec8<__half> &v, float *f) {
    const __half2 *s = reinterpret_cast<const __half2 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __half22float2(s[i]);
        f[2 * i] = t.x, f[2 * i + 1] = t.y;
    }
}
__device__ __forceinline__ void widen(const Vec8<__nv_bfloat16> &v, float *f) {
    const __nv_bfloat162 *s = reinterpret_cast<const __nv_bfloat162 *>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __bfloat1622float2(s[i]);
        f[2 * i] = t.x, f[2 * i + 1] = t.y;
    }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float *f) {
    uint4 r;
    r.x = pack2<T>(f[0], f[1]), r.y = pack2<T>(f[2], f[3]);
    r.z = pack2<T>(f[4], f[5]), r.w = pack2<T>(f[6], f[7]);
    *reinterpret_cast<uint4 *>(p) = r;
}

// GL lanes share a head (the power of two at or above D / 16).
template <typename TI, typename TO, int GL>
__global__ void __launch_bounds__(kThreads, 16) rotate_kernel(const RotateArgs a) {
    __shared__ float s_cos[128], s_sin[128];
    constexpr int kGroups = kThreads / GL;
    const int tid = threadIdx.x, u = tid % GL, token = blockIdx.x;
    const int heads = a.Hq + 2 * a.Hkv;
    const bool in_head = 16 * u < a.D, turns = 16 * u < a.rot;
    const bool halves = turns && !a.neighbours;
    // the thread's two vectors in a rotated head, and in a value head
    const int o0 = halves ? 8 * u : 16 * u, o1 = halves ? a.rot / 2 + 8 * u : 16 * u + 8;

    wait_for_previous_kernel();

    int64_t slot = -1;
    if (a.kc) {
        slot = a.slots[token];
        if (slot >= a.n_slots) slot = -1;
    }
    const int64_t page = slot >> a.page_shift, row = slot - (page << a.page_shift);

    auto source = [&](int h) -> const TI * {
        if (h < a.Hq) return (const TI *)a.q + (size_t)token * a.ldq + (size_t)h * a.D;
        h -= a.Hq;
        if (h < a.Hkv) return (const TI *)a.k + (size_t)token * a.ldk + (size_t)h * a.D;
        return (const TI *)a.v + (size_t)token * a.ldv + (size_t)(h - a.Hkv) * a.D;
    };
    const int step = kGroups * gridDim.y;
    int h = blockIdx.y * kGroups + tid / GL;
    Vec8<TI> x0 = {}, x1 = {};
    auto fetch = [&](int h) {
        if (h < heads && in_head) {
            const TI *s = source(h);
            const bool value = h >= a.Hq + a.Hkv;
            x0 = load8(s + (value ? 16 * u : o0));
            x1 = load8(s + (value ? 16 * u + 8 : o1));
        }
    };
    fetch(h);   // the first head's loads are under way while the angles are computed

    for (int p = tid; p < a.rot / 2; p += kThreads) {
        const double turn = (double)a.pos[token] * (a.inv_freq[p] * 0.15915494309189533577);   // 1 / (2 pi)
        sincospif(2.0f * (float)(turn - rint(turn)), &s_sin[p], &s_cos[p]);
    }
    __syncthreads();
    for (int h0 = blockIdx.y * kGroups; h0 < heads; h0 += step, h += step) {   // the same trips for a whole warp
        const bool active = h < heads && in_head;
        float f[16];
        widen(x0, f), widen(x1, f + 8);
        fetch(h + step);
        const int kd = h < a.Hq ? 0 : h < a.Hq + a.Hkv ? 1 : 2;   // queries, keys, values
        const float *wp = kd == 0 ? a.wq : kd == 1 ? a.wk : nullptr;
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
        if (!active) ss = 0.0f;
#pragma unroll
        for (int m = GL / 2; m; m >>= 1) ss += __shfl_xor_sync(~0u, ss, m);
        if (!active) continue;
        if (wp) {
            const float r = rsqrtf(ss / (float)a.D + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= r * wp[o0 + i], f[8 + i] *= r * wp[o1 + i];
        }
        int p0 = 16 * u, p1 = 16 * u + 8;
        if (kd < 2) {
            p0 = o0, p1 = o1;
            if (halves) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = f[i], y = f[8 + i], c = s_cos[8 * u + i], s = s_sin[8 * u + i];
                    f[i] = x * c - y * s, f[8 + i] = y * c + x * s;
                }
            } else if (turns) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = f[2 * i], y = f[2 * i + 1], c = s_cos[8 * u + i], s = s_sin[8 * u + i];
                    f[2 * i] = x * c - y * s, f[2 * i + 1] = y * c + x * s;
                }
            }
        }
        auto put = [&](TO *d) { store8(d + p0, f), store8(d + p1, f + 8); };
        if (kd == 0) {
            if (a.qo) put((TO *)a.qo + (size_t)token * a.ldqo + (size_t)h * a.D);
        } else {
            const int hk = h - a.Hq - (kd == 2 ? a.Hkv : 0);
            void *o = kd == 1 ? a.ko : a.vo;
            if (o) put((TO *)o + (size_t)token * (kd == 1 ? a.ldko : a.ldvo) + (size_t)hk * a.D);
            if (slot >= 0)
                put((TO *)(kd == 1 ? a.kc : a.vc) + (((page * a.Hkv + hk) << a.page_shift) + row) * a.D);
        }
    }
}

template <typename TI, typename TO>
cudaError_t launch_rotate(const RotateArgs &a, int T, bool pdl, cudaStream_t s) {
    const int units = a.D / 16, heads = a.Hq + 2 * a.Hkv;
    const int GL = units <= 1 ? 1 : units <= 2 ? 2 : units <= 4 ? 4 : units <= 8 ? 8 : 16;
    // one block a token, more where the tokens alone would leave SMs idle
    const int want = ceil_div(4 * sm_count(), T), most = ceil_div(heads, kThreads / GL);
    const dim3 grid(T, want < most ? want : most), block(kThreads);
    switch (GL) {
        case 1: return launch(rotate_kernel<TI, TO, 1>, grid, block, 0, s, pdl, a);
        case 2: return launch(rotate_kernel<TI, TO, 2>, grid, block, 0, s, pdl, a);
        case 4: return launch(rotate_kernel<TI, TO, 4>, grid, block, 0, s, pdl, a);
        case 8: return launch(rotate_kernel<TI, TO, 8>, grid, block, 0, s, pdl, a);
        default: return launch(rotate_kernel<TI, TO, 16>, grid, block, 0, s, pdl, a);
    }
}

// T rows of `width` bytes, `pitch` bytes apart.
struct Rows {
    const void *at;
    int64_t pitch, width;
};
inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && a < 0); }
// Whether two sets of rows share a byte: exactly where the pitches agree (slices of one buffer lie between each
// other's rows), else by what they span.
bool overlap(const Rows &a, const Rows &b, int64_t T) {
    if (!a.at || !b.at) return false;
    const int64_t d = (int64_t)((uintptr_t)b.at - (uintptr_t)a.at), last = T - 1;
    if (T == 1 || a.pitch != b.pitch) return d < last * a.pitch + a.width && -d < last * b.pitch + b.width;
    // row i of a meets row i + k of b where -b.width < d + k * pitch < a.width
    const int64_t k0 = floor_div(-b.width - d, a.pitch) + 1, k1 = -floor_div(d - a.width, a.pitch) - 1;
    return k0 <= k1 && k0 <= last && k1 >= -last;
}

// An output may be its own input, row for row, and meets no other input or output.
bool outputs_apart(const fb_heads &in, const fb_heads &out) {
    const int64_t ei = dtype_size(in.t), eo = dtype_size(out.t), wq = (int64_t)in.Hq * in.D, wk = (int64_t)in.Hkv * in.D;
    const Rows i[3] = {{in.q, in.ldq * ei, wq * ei}, {in.k, in.ldk * ei, wk * ei}, {in.v, in.ldv * ei, wk * ei}};
    const Rows o[3] = {{out.q, out.ldq * eo, wq * eo}, {out.k, out.ldk * eo, wk * eo}, {out.v, out.ldv * eo, wk * eo}};
    for (int x = 0; x < 3; ++x)
        for (int y = 0; y < 3; ++y) {
            const bool same = x == y && o[x].at == i[y].at && in.t == out.t && (o[x].pitch == i[y].pitch || in.T == 1);
            if ((!same && overlap(o[x], i[y], in.T)) || (y > x && overlap(o[x], o[y], in.T))) return false;
        }
    return true;
}

template <typename TO>
cudaError_t launch_rotate_to(fb_dtype t, const RotateArgs &a, int T, bool pdl, cudaStream_t s) {
    if (t == FB_F32) return launch_rotate<float, TO>(a, T, pdl, s);
    if (t == FB_F16) return launch_rotate<__half, TO>(a, T, pdl, s);
    return launch_rotate<__nv_bfloat16, TO>(a, T, pdl, s);
}

}  // namespace
}  // namespace fb

using namespace fb;

extern "C" fb_status fb_qk_norm_rope(const fb_heads *in, const fb_heads *out, const int32_t *pos,
                                     const double *inv_freq, int rot, const float *q_weight, const float *k_weight,
                                     float eps, const fb_kv_cache *cache, const int32_t *slots, unsigned flags,
                                     void *stream) {
    if (!in || !out || (flags & ~(FB_GEMV_PDL | FB_ROPE_NEIGHBOURS)) || !(eps >= 0.0f) || eps > 3e38f)
        return FB_ERR_INVALID_VALUE;
    if (!valid_heads(*in) || !in->q || !in->k || !in->v || out->T != in->T || out->Hq != in->Hq ||
        out->Hkv != in->Hkv || out->D != in->D || !dtype_size(out->t))
        return FB_ERR_INVALID_VALUE;
    const int D = in->D;
    if (rot < 0 || rot > D || (rot > 0 && (!pos || !inv_freq))) return FB_ERR_INVALID_VALUE;
    if ((out->q && out->ldq < in->Hq * D) || (out->k && out->ldk < in->Hkv * D) || (out->v && out->ldv < in->Hkv * D))
        return FB_ERR_INVALID_VALUE;
    if (cache && (!valid_cache(*cache) || cache->t != out->t || cache->Hkv != in->Hkv || cache->D != D || !slots))
        return FB_ERR_INVALID_VALUE;
    if (out->t == FB_F32 || D % 16 || D > 256 || rot % 16) return FB_ERR_UNSUPPORTED;
    const int ei = dtype_size(in->t), eo = dtype_size(out->t);
    if (!aligned(in->q, 16) || !aligned(in->k, 16) || !aligned(in->v, 16) || in->ldq * (int64_t)ei % 16 ||
        in->ldk * (int64_t)ei % 16 || in->ldv * (int64_t)ei % 16 || !aligned(out->q, 16) || !aligned(out->k, 16) ||
        !aligned(out->v, 16) || (out->q && out->ldq * (int64_t)eo % 16) || (out->k && out->ldk * (int64_t)eo % 16) ||
        (out->v && out->ldv * (int64_t)eo % 16) || !aligned(pos, 4) || !aligned(inv_freq, 8) ||
        !aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(slots, 4) ||
        (cache && (!aligned(cache->k, 16) || !aligned(cache->v, 16))))
        return FB_ERR_MISALIGNED;
    if (!outputs_apart(*in, *out)) return FB_ERR_INVALID_VALUE;
    RotateArgs a = {};
    a.q = in->q, a.k = in->k, a.v = in->v;
    a.qo = out->q, a.ko = out->k, a.vo = out->v;
    a.ldq = in->ldq, a.ldk = in->ldk, a.ldv = in->ldv;
    a.ldqo = out->ldq, a.ldko = out->ldk, a.ldvo = out->ldv;
    a.pos = pos, a.inv_freq = inv_freq, a.wq = q_weight, a.wk = k_weight, a.eps = eps;
    a.Hq = in->Hq, a.Hkv = in->Hkv, a.D = D, a.rot = rot;
    a.neighbours = (flags & FB_ROPE_NEIGHBOURS) != 0;
    if (cache) {
        a.kc = cache->k, a.vc = cache->v, a.slots = slots;
        a.page_shift = log2_of(cache->page_size);
        a.n_slots = (int64_t)cache->pages * cache->page_size;
    }
    const bool pdl = flags & FB_GEMV_PDL;
    return status_of(out->t == FB_F16 ? launch_rotate_to<__half>(in->t, a, in->T, pdl, as_stream(stream))
                                      : launch_rotate_to<__nv_bfloat16>(in->t, a, in->T, pdl, as_stream(stream)));
}
