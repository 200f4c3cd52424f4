// The row operators of the target model's dense side: the residual's addition
// with the root-mean-square norm, the gated activation, and the rounding to 8
// bits that both can end in (and that stands alone for other rows and for
// weights).  A block of 128 elements shares a scale:
//   scale = max(max |y|, 1e-20) / 448,   q = e4m3(y * (448 / max(max |y|, 1e-20))).
// All in fp32, rounded once.  A thread works on vectors of 8 elements, so 16
// neighbouring lanes hold a block and find its largest element in four shuffles.
// Memory bounds all of them from some 256 rows of 4096 on, the launch below that.
#include "sv_kv.cuh"
#include "sv_linear.h"

namespace sv {

// (No read-only loads: the sum may be written where the residual was read.)
__device__ __forceinline__ uint4 ld16(const char* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
// Vector i of 8 elements at p: 16 bytes of bf16 or 32 of fp32.
__device__ __forceinline__ void load8(const char* p, int64_t i, bool f32, float (&x)[8]) {
    if (f32) {
        const uint4 a = ld16(p + i * 32), b = ld16(p + i * 32 + 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j] = __uint_as_float(u4_get(a, j));
            x[4 + j] = __uint_as_float(u4_get(b, j));
        }
    } else {
        unpack8(ld16(p + i * 16), x);
    }
}
__device__ __forceinline__ void store8(char* p, int64_t i, bool f32, const float (&x)[8]) {
    if (f32) {
        float4* q = reinterpret_cast<float4*>(p + i * 32);
        q[0] = make_float4(x[0], x[1], x[2], x[3]);
        q[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4*>(p + i * 16) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
}
__device__ __forceinline__ float top8(const float (&x)[8]) {
    float m = fabsf(x[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
    return m;
}
__device__ __forceinline__ void store8_e4m3(char* p, int64_t i, float top, const float (&x)[8]) {
    const float f = kFp8Max / top;
    *reinterpret_cast<uint2*>(p + i * 8) = make_uint2(pack_e4m3(x[0] * f, x[1] * f) | pack_e4m3(x[2] * f, x[3] * f) << 16,
                                                     pack_e4m3(x[4] * f, x[5] * f) | pack_e4m3(x[6] * f, x[7] * f) << 16);
}
// Vector v of row r to 8 bits; all 16 lanes of a block take part, those without a vector
// (have false) with x all zero.
__device__ __forceinline__ void put_e4m3(char* out, float* scale, int64_t scale_stride, int64_t r, int nv, int v, bool have, const float (&x)[8]) {
    float m = top8(x);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = fmaxf(m, kFp8AmaxFloor);
    if (!have) return;
    store8_e4m3(out, r * nv + v, m, x);
    if ((v & 15) == 0) scale[(v >> 4) * scale_stride + r] = m / kFp8Max;
}

// ---- residual and norm ---------------------------------------------------------------
// A row is a group of TPR threads, VPT vectors each, held in registers between the
// two uses.  MORE: longer rows, read once more for the second (from L2, mostly).
struct RowFormat {
    bool xf, sf;                       // x and the residual are fp32
    int out;                           // spec_dtype_t
};
template <int VPT, bool MORE>
__global__ void __launch_bounds__(512) add_norm_kernel(const NormArgs a, const RowFormat f, int tpr) {
    __shared__ float part[2][16];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, in_row = threadIdx.x & (tpr - 1), nv = a.dim / 8;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = row < a.rows;
    const char* x = a.x + row * a.xs * (f.xf ? 4 : 2);
    const char* res = a.res + row * a.rs * (f.sf ? 4 : 2);
    char* sum = a.sum + row * a.ss * (f.sf ? 4 : 2);
    pdl_wait();
    float h[VPT][8];
    // VPT vectors from vector v0 on (those past the row zero), the residual added
    auto fetch = [&](int v0) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = v0 + j * tpr;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[j][e] = 0.f;
            if (live && v < nv) load8(x, v, f.xf, h[j]);
        }
        if (!a.res) return;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = v0 + j * tpr;
            float r[8];
            if (live && v < nv) {
                load8(res, v, f.sf, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[j][e] += r[e];
            }
        }
    };
    float ss = 0.f;
    for (int v0 = in_row; v0 < (MORE ? nv : tpr); v0 += VPT * tpr) {
        fetch(v0);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(h[j][e], h[j][e], ss);
    }
    ss = warp_sum(ss);
    if (tpr > 32) {
        if ((threadIdx.x & 31) == 0) part[0][warp] = ss;
        __syncthreads();
        const int first = (threadIdx.x / tpr) * (tpr / 32);
        ss = 0.f;
        for (int i = 0; i < tpr / 32; ++i) ss += part[0][first + i];
    }
    const float inv = rsqrtf(ss / (float)a.dim + a.eps);
    // (all lanes stay: a block's 16 find its largest element together)
    for (int v0 = in_row; v0 - in_row < (MORE ? nv : 1); v0 += VPT * tpr) {
        if (MORE) fetch(v0);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = v0 + j * tpr;
            const bool have = live && v < nv;
            if (have && a.sum) store8(sum, v, f.sf, h[j]);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = h[j][e] * inv;
            if (have && a.w) {
                float w[8];
                unpack8(*(reinterpret_cast<const uint4*>(a.w) + v), w);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= w[e];
            }
            if (f.out == SPEC_DTYPE_E4M3) put_e4m3(a.out, a.scale, a.scale_stride, row, nv, v, have, y);
            else if (have) store8(a.out, row * nv + v, f.out == SPEC_DTYPE_F32, y);
        }
    }
}

cudaError_t launch_add_norm(const NormArgs& a, spec_dtype_t x, spec_dtype_t sum, spec_dtype_t out, cudaStream_t st) {
    const RowFormat f{x == SPEC_DTYPE_F32, sum == SPEC_DTYPE_F32, (int)out};
    const int nv = a.dim / 8;
    const int vpt = nv <= 512 ? 1 : nv <= 1024 ? 2 : 4;
    int tpr = 32;
    while (tpr < 512 && tpr * vpt < nv) tpr *= 2;
    const int threads = tpr < 128 ? 128 : tpr;
    const dim3 grid((unsigned)(((long long)a.rows + threads / tpr - 1) / (threads / tpr)));
    if (nv > 512 * 4) return launch_pdl(add_norm_kernel<4, true>, grid, threads, 0, st, a, f, tpr);
    if (vpt == 1) return launch_pdl(add_norm_kernel<1, false>, grid, threads, 0, st, a, f, tpr);
    if (vpt == 2) return launch_pdl(add_norm_kernel<2, false>, grid, threads, 0, st, a, f, tpr);
    return launch_pdl(add_norm_kernel<4, false>, grid, threads, 0, st, a, f, tpr);
}

// ---- gated activation, rounding of rows ----------------------------------------------
// x / (1 + e^-x); the tanh form of GELU is x over 1 + e^(-2u), u = sqrt(2 / pi) (x + 0.044715 x^3),
// since (1 + tanh u) / 2 = 1 / (1 + e^(-2u)).
__device__ __forceinline__ float activate(float x, int act) {
    const float t = act == SPEC_ACT_SILU ? x : 1.5957691216057308f * x * fmaf(0.044715f * x, x, 1.f);
    return __fdividef(x, 1.f + __expf(-t));
}

constexpr int kActThreads = 256, kActVectors = 2;
// Vectors are counted with every row filled up to whole blocks, so that a block's 16 lanes
// stand side by side.
__global__ void __launch_bounds__(kActThreads) act_kernel(const ActArgs a, bool f32, int out, unsigned per_row, unsigned total) {
    pdl_trigger();
    const int elt = f32 ? 4 : 2, nv = a.dim / 8;
    float g[kActVectors][8], u[kActVectors][8];
    unsigned row[kActVectors], v[kActVectors];
    bool have[kActVectors];
    pdl_wait();
#pragma unroll
    for (int k = 0; k < kActVectors; ++k) {
        const unsigned i = (blockIdx.x * kActVectors + k) * kActThreads + threadIdx.x;
        row[k] = i / per_row;
        v[k] = i - row[k] * per_row;
        have[k] = i < total && (int)v[k] < nv;
#pragma unroll
        for (int e = 0; e < 8; ++e) g[k][e] = u[k][e] = 0.f;
        if (!have[k]) continue;
        load8(a.gate + (int64_t)row[k] * a.gs * elt, v[k], f32, g[k]);
        if (a.up) load8(a.up + (int64_t)row[k] * a.us * elt, v[k], f32, u[k]);
    }
#pragma unroll
    for (int k = 0; k < kActVectors; ++k) {
        if (a.up) {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[k][e] = activate(g[k][e], a.act) * u[k][e];
        }
        if (out == SPEC_DTYPE_E4M3) put_e4m3(a.out, a.scale, a.scale_stride, row[k], nv, (int)v[k], have[k], g[k]);
        else if (have[k]) store8(a.out, (int64_t)row[k] * nv + v[k], out == SPEC_DTYPE_F32, g[k]);
    }
}

cudaError_t launch_act(const ActArgs& a, spec_dtype_t in, spec_dtype_t out, cudaStream_t st) {
    const unsigned per_row = (unsigned)(a.dim / 8 + 15) / 16 * 16;
    const unsigned total = per_row * (unsigned)a.rows;         // (checked below 2^31)
    const unsigned per = kActThreads * kActVectors;
    return launch_pdl(act_kernel, dim3((total + per - 1) / per), kActThreads, 0, st, a, in == SPEC_DTYPE_F32, (int)out, per_row, total);
}

// ---- rounding of weights -------------------------------------------------------------
// A CTA a block of 128 x 128: 16 lanes a row, 16 rows at a time.
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const TileQuantArgs a, bool f32, int tiles_n) {
    __shared__ float part[8];
    pdl_trigger();
    const int ti = blockIdx.x / tiles_n, tb = blockIdx.x - ti * tiles_n, nv = a.dim / 8;
    const int v = tb * 16 + (threadIdx.x & 15), r0 = ti * kScaleBlock + (threadIdx.x >> 4);
    float x[8][8], m = 0.f;
    pdl_wait();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] = 0.f;
        if (v < nv && r0 + 16 * k < a.rows) load8(a.x + (int64_t)(r0 + 16 * k) * a.xs * (f32 ? 4 : 2), v, f32, x[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, top8(x[k]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = kFp8AmaxFloor;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, part[i]);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (v < nv && r0 + 16 * k < a.rows) store8_e4m3(a.out, (int64_t)(r0 + 16 * k) * nv + v, m, x[k]);
    if (threadIdx.x == 0) a.scale[(int64_t)ti * a.scale_stride + tb] = m / kFp8Max;
}

cudaError_t launch_quantize_tiles(const TileQuantArgs& a, spec_dtype_t in, cudaStream_t st) {
    const int tiles_n = scale_blocks(a.dim);
    const long long tiles = (long long)scale_blocks(a.rows) * tiles_n;
    if (tiles >= (1LL << 31)) return cudaErrorInvalidValue;
    return launch_pdl(quantize_tiles_kernel, dim3((unsigned)tiles), 256, 0, st, a, in == SPEC_DTYPE_F32, tiles_n);
}

}  // namespace sv
