// attn_common.cuh -- what the attention calls share: argument checks of
// heads and caches, packing of value pairs, the programmatic-launch wait.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fb_internal.cuh"

namespace fb {

constexpr int kMaxTokens = 1 << 24;
constexpr int kMaxHeads = 1024;

// Outputs are rescaled only when a row's maximum has grown by more than 2^8 since
// the last time: the sum carries the same factor, and weights that much larger
// fit either type.
constexpr float kRescaleLog2 = 8.0f;
// What a row's weights are relative to lies this many powers of two below its
// maximum: fp16 holds weights from 2^-14 in full and drops them below 2^-25, so
// its largest stands at 2^7, and at no more than 2^15 after a growth that asks
// for no rescaling.  The sum, its logarithm and the joins carry the factor.
// bf16 has fp32's range and needs none.
template <typename E>
constexpr float kHeadroomLog2 = std::is_same_v<E, __half> ? 7.0f : 0.0f;

// Device address of the word in which the attention kernels raise the bits of
// fb_attn_errors, on the current device (null on a CUDA error).
void *attn_errors_address();
constexpr unsigned kErrorInput = 1u, kErrorWait = 2u;

inline int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

inline bool valid_heads(const fb_heads &h) {
    return dtype_size(h.t) && h.T >= 1 && h.T <= kMaxTokens && h.Hq >= 1 && h.Hq <= kMaxHeads && h.Hkv >= 1 &&
           h.Hq % h.Hkv == 0 && h.D >= 1 && h.D <= 65536 && h.ldq >= h.Hq * h.D && h.ldk >= h.Hkv * h.D &&
           h.ldv >= h.Hkv * h.D;
}

inline bool valid_cache(const fb_kv_cache &c) {
    return c.k && c.v && (c.t == FB_F16 || c.t == FB_BF16) && c.pages >= 1 && c.Hkv >= 1 && c.Hkv <= kMaxHeads &&
           c.D >= 1 && c.D <= 65536 && c.page_size >= 1 && c.page_size <= 1024 &&
           (c.page_size & (c.page_size - 1)) == 0 && (int64_t)c.pages * c.page_size < ((int64_t)1 << 31);
}

// Two fp32 values rounded to T, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
}

// 2^x by the special-function unit (2 ulp; results below 2^-126 are zero).
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Programmatic dependent launch: returns once the previous kernel of the
// stream has completed (at once for an ordinary launch).
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace fb
