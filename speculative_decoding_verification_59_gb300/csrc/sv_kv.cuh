// Device helpers of the cache and attention calls: packed bf16 and e4m3
// conversions, and the place of a cached position.
#pragma once

#include "sv_common.cuh"
#include "sv_kv.h"

namespace sv {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two floats rounded to bf16, lo in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two floats rounded to e4m3 (saturating, NaN kept), lo in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 values as fp16 pairs (exact), low byte in the low half.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
    return r;
}
__device__ __forceinline__ void f16x2_to_f32(uint32_t w, float* lo, float* hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(*lo), "=f"(*hi)
        : "r"(w));
}

// Eight bf16 values of a 16-byte vector as floats.
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf_lo(u4_get(w, i));
        x[2 * i + 1] = bf_hi(u4_get(w, i));
    }
}

// The page and slot of position t of sequence b; false when t lies past the
// table or the page it names is none of the cache's.
__device__ __forceinline__ bool cache_place(const spec_kv_cache_t& c, int b, int t, int* page, int* slot) {
    const int p = t / c.page_size;
    if (t < 0 || p >= c.max_pages) return false;
    *slot = t - p * c.page_size;
    *page = __ldg(c.block_table + (size_t)b * c.max_pages + p);
    return (unsigned)*page < (unsigned)c.num_pages;
}

__device__ __forceinline__ int64_t entry_off(const spec_kv_cache_t& c, int page, int slot, int head) {
    return (int64_t)page * c.page_stride + (int64_t)slot * c.token_stride + (int64_t)head * c.head_stride;
}
__device__ __forceinline__ int64_t scale_off(const spec_kv_cache_t& c, int page, int slot, int head) {
    return (int64_t)page * c.scale_page_stride + (int64_t)slot * c.scale_token_stride +
           (int64_t)head * c.scale_head_stride;
}

__device__ __forceinline__ void raise_error(int32_t* err, int bits) {
    if (err) atomicOr(err, bits);
}

}  // namespace sv
