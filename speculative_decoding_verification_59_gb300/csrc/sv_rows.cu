// The row operators of the target model's dense side: the residual's addition
// with the root-mean-square norm, the gated activation, and the rounding to 8
// bits that both can end in (and that stands alone for other rows and for
// weights).  A block of 128 elements shares a scale:
//   scale = max(max |y|, 1e-20) / 448,   q = e4m3(y * (448 / max(max |y|, 1e-20))).
// All in fp32, rounded once.  A thread works on vectors of 8 elements, so 16
// neighbouring lanes hold a block and find its largest element in four shuffles.
// Memory bounds all of them from some 1000 rows of 4096 on (a copy: 6.8 TB/s), a launch and one
// dependent load below that.
#include "sv_kv.cuh"
#include "sv_linear.h"

namespace sv {

// (No read-only loads: the sum may be written where the residual was read.)
__device__ __forceinline__ uint4 ld16(const char* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
// A vector of 8 elements as it lies in memory, 16 bytes of bf16 or 32 of fp32: kept so until it is
// used, it takes half the registers, and more loads are under way.
template <bool F32>
struct Raw8 {
    uint4 w[F32 ? 2 : 1];
    // vector i at p; zeros without `have`
    __device__ __forceinline__ void load(const char* p, int64_t i, bool have) {
#pragma unroll
        for (int k = 0; k < (F32 ? 2 : 1); ++k) {
            w[k] = make_uint4(0u, 0u, 0u, 0u);
            if (have) w[k] = ld16(p + i * (F32 ? 32 : 16) + k * 16);
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(u4_get(w[j >> 2], j & 3));
        } else {
            unpack8(w[0], x);
        }
    }
};
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
// x f, rounded.
__device__ __forceinline__ void store8_e4m3(char* p, int64_t i, float f, const float (&x)[8]) {
    const f32x2 f2 = f2_pack(f, f);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) f2_unpack(f2_mul(f2_pack(x[j], x[j + 1]), f2), y[j], y[j + 1]);
    *reinterpret_cast<uint2*>(p + i * 8) =
        make_uint2(pack_e4m3(y[0], y[1]) | pack_e4m3(y[2], y[3]) << 16, pack_e4m3(y[4], y[5]) | pack_e4m3(y[6], y[7]) << 16);
}
// Vector i of an output to 8 bits; all 16 lanes of a block take part, those without a vector
// (have false) with x all zero.  The block's largest magnitude.  SCALED: of x `times`, a factor of the whole
// row, which the scale takes up: q is rounded from x, not from a product rounded before.
template <bool SCALED>
__device__ __forceinline__ float put_e4m3(char* out, int64_t i, bool have, const float (&x)[8], float times) {
    float m = top8(x);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!SCALED) {
        m = fmaxf(m, kFp8AmaxFloor);
        if (have) store8_e4m3(out, i, kFp8Max / m, x);
        return m;
    }
    const float top = m * times;
    const bool above = top > kFp8AmaxFloor;
    if (have) store8_e4m3(out, i, kFp8Max / (above ? m : kFp8AmaxFloor) * (above ? 1.f : times), x);
    return above ? top : kFp8AmaxFloor;
}

// ---- residual and norm ---------------------------------------------------------------
// A row is a group of TPR threads, VPT vectors each, held in registers between the
// two uses.  MORE: longer rows, read once more for the second (from L2, mostly).  WIDE: rows of 512
// threads, and registers for two of them on an SM, so that one's loads cover the other's sums (2000 rows
// of 12000 to e4m3: 39 us for 54; rows of 4096, several a CTA, 42.0 for 43.2 to e4m3, but 65.4 for 62.4
// with an fp32 residual).
template <bool XF, bool SF, int VPT, bool WIDE, bool MORE>
__global__ void __launch_bounds__(512, VPT == 4 && (WIDE || !(XF || SF)) ? 2 : 1) add_norm_kernel(const NormArgs a, int out, int tpr) {
    __shared__ float part[16];
    pdl_trigger();
    const int warp = threadIdx.x >> 5, in_row = threadIdx.x & (tpr - 1), nv = a.dim / 8;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = row < a.rows;
    const char* x = a.x + row * a.xs * (XF ? 4 : 2);
    const char* res = a.res + row * a.rs * (SF ? 4 : 2);
    char* sum = a.sum + row * a.ss * (SF ? 4 : 2);
    pdl_wait();
    float h[VPT][8];
    // VPT vectors from vector v0 on (those past the row zero), the residual added
    auto fetch = [&](int v0) {
        Raw8<XF> p[VPT];
        Raw8<SF> q[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) p[j].load(x, v0 + j * tpr, live && v0 + j * tpr < nv);
#pragma unroll
        for (int j = 0; j < VPT; ++j) q[j].load(res, v0 + j * tpr, a.res && live && v0 + j * tpr < nv);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float r[8];
            p[j].get(h[j]);
            q[j].get(r);
            if (a.res) {
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    f2_unpack(f2_add(f2_pack(h[j][e], h[j][e + 1]), f2_pack(r[e], r[e + 1])), h[j][e], h[j][e + 1]);
            }
        }
    };
    f32x2 pair = 0;
    for (int v0 = in_row; v0 < (MORE ? nv : tpr); v0 += VPT * tpr) {
        fetch(v0);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const f32x2 x2 = f2_pack(h[j][e], h[j][e + 1]);
                pair = f2_fma(x2, x2, pair);
            }
    }
    float ss, odd;
    f2_unpack(pair, ss, odd);
    ss = warp_sum(ss + odd);
    if (tpr > 32) {
        if ((threadIdx.x & 31) == 0) part[warp] = ss;
        __syncthreads();
        const int first = (threadIdx.x / tpr) * (tpr / 32);
        ss = 0.f;
        for (int i = 0; i < tpr / 32; ++i) ss += part[first + i];
    }
    const float inv = rsqrtf(ss / (float)a.dim + a.eps);
    const bool fp8 = out == SPEC_DTYPE_E4M3;
    // (all lanes stay: a block's 16 find its largest element together)
    for (int v0 = in_row; v0 - in_row < (MORE ? nv : 1); v0 += VPT * tpr) {
        if (MORE) fetch(v0);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = v0 + j * tpr;
            const bool have = live && v < nv;
            if (have && a.sum) store8(sum, v, SF, h[j]);
            float y[8], w[8];
            if (a.w) unpack8(have ? *(reinterpret_cast<const uint4*>(a.w) + v) : make_uint4(0u, 0u, 0u, 0u), w);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                f32x2 y2 = f2_pack(h[j][e], h[j][e + 1]);
                if (!fp8) y2 = f2_mul(y2, f2_pack(inv, inv));
                if (a.w) y2 = f2_mul(y2, f2_pack(w[e], w[e + 1]));
                f2_unpack(y2, y[e], y[e + 1]);
            }
            if (fp8) {
                const float m = put_e4m3<true>(a.out, row * nv + v, have, y, inv);
                if (have && (v & 15) == 0) a.scale[(v >> 4) * a.scale_stride + row] = m / kFp8Max;
            } else if (have) store8(a.out, row * nv + v, out == SPEC_DTYPE_F32, y);
        }
    }
}

template <bool XF, bool SF>
static cudaError_t launch_add_norm_t(const NormArgs& a, int out, int sms, cudaStream_t st) {
    const int nv = a.dim / 8;
    // Few rows: as many threads a row as it has vectors (the time is one row's).  More: two or four
    // vectors a thread, so that an SM holds more rows' loads under way (rows of 4096, one / two / four
    // a thread: 512 rows 5.9 / 4.5 / 5.5 us, 8192 of an fp32 residual 87 / 61.5 / 62, 8192 to e4m3
    // 71.6 / 47.5 / 45.8, since down to 41.7: 6.4 TB/s with the fp32 residual, 5.7 to e4m3, 2.2 us for a row.  Between
    // them less: 512 rows with a bf16 residual to e4m3 5.2 us, 2.8 TB/s, 1152 rows 9.4, 3.5, 2000 of 12000 38.7, 4.4.)
    int vpt = nv > 1024 ? 4 : a.rows <= 2 * sms ? (nv > 512 ? 2 : 1) : a.rows <= 32 * sms ? 2 : 4;
    while (vpt > 1 && nv <= 32 * (vpt / 2)) vpt /= 2;
    int tpr = 32;
    while (tpr < 512 && tpr * vpt < nv) tpr *= 2;
    const int threads = tpr < 128 ? 128 : tpr;
    const dim3 grid((unsigned)(((long long)a.rows + threads / tpr - 1) / (threads / tpr)));
    if (nv > 512 * 4) return launch_pdl(add_norm_kernel<XF, SF, 4, true, true>, grid, threads, 0, st, a, out, tpr);
    if (vpt == 1) return launch_pdl(add_norm_kernel<XF, SF, 1, false, false>, grid, threads, 0, st, a, out, tpr);
    if (vpt == 2) return launch_pdl(add_norm_kernel<XF, SF, 2, false, false>, grid, threads, 0, st, a, out, tpr);
    if (tpr == 512) return launch_pdl(add_norm_kernel<XF, SF, 4, true, false>, grid, threads, 0, st, a, out, tpr);
    return launch_pdl(add_norm_kernel<XF, SF, 4, false, false>, grid, threads, 0, st, a, out, tpr);
}

cudaError_t launch_add_norm(const NormArgs& a, spec_dtype_t x, spec_dtype_t sum, spec_dtype_t out, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    const bool xf = x == SPEC_DTYPE_F32, sf = a.res && sum == SPEC_DTYPE_F32;
    if (xf) return sf ? launch_add_norm_t<true, true>(a, (int)out, di.sm_count, st) : launch_add_norm_t<true, false>(a, (int)out, di.sm_count, st);
    return sf ? launch_add_norm_t<false, true>(a, (int)out, di.sm_count, st) : launch_add_norm_t<false, false>(a, (int)out, di.sm_count, st);
}

// ---- gated activation, rounding of rows ----------------------------------------------
// x / (1 + e^-x); the tanh form of GELU is x over 1 + e^(-2u), u = sqrt(2 / pi) (x + 0.044715 x^3),
// since (1 + tanh u) / 2 = 1 / (1 + e^(-2u)).  Power and reciprocal are the special-function unit's
// (2 and 1 units in the last place); past e^88 the reciprocal is zero, and so is the result.
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// act(x) y, pairwise.
template <int ACT>
__device__ __forceinline__ void gate8(float (&x)[8], const float (&y)[8]) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const f32x2 v = f2_pack(x[j], x[j + 1]);
        f32x2 t = f2_mul(v, f2_pack(-1.4426950408889634f, -1.4426950408889634f));       // -log2 e
        if constexpr (ACT == SPEC_ACT_GELU_TANH) {
            // -2 sqrt(2 / pi) log2 e (x + 0.044715 x^3)
            const f32x2 c = f2_fma(f2_mul(v, v), f2_pack(0.044715f, 0.044715f), f2_pack(1.f, 1.f));
            t = f2_mul(f2_mul(v, c), f2_pack(-2.3022081986f, -2.3022081986f));
        }
        float a, b;
        f2_unpack(t, a, b);
        f2_unpack(f2_add(f2_pack(ex2_approx(a), ex2_approx(b)), f2_pack(1.f, 1.f)), a, b);
        f2_unpack(f2_mul(f2_mul(v, f2_pack(rcp_approx(a), rcp_approx(b))), f2_pack(y[j], y[j + 1])), x[j], x[j + 1]);
    }
}

// A CTA takes RT rows and, 16 lanes a block, 16 / RT blocks of them at a time, V times.  Many rows: 16
// rows of one block, whose scales then leave together in one line (a scale of 4 bytes by itself
// costs a sector: 39.4 us for 33 at 16384 rows of 4096).  Activation of 4000 x 12288 bf16 to e4m3: 38.5 us,
// 6.4 TB/s; of 1152: 12.3, 5.8 (issue slots are 60 % busy; with divisions and single arithmetic, 82 %,
// 15.1); to bf16 4000 take 43.4, 6.8.  7 rows: 1.5.  Rounding of 16384 x 4096: 33.1, 6.1; of 1152: 4.2.
constexpr int kActThreads = 256;
template <bool F32, int ACT, int RT, int V>
__global__ void __launch_bounds__(kActThreads) act_kernel(const ActArgs a, int out, int chunks) {
    constexpr bool GATED = ACT != kActNone;
    constexpr int BT = 16 / RT;                           // blocks at a time
    __shared__ float top[RT > 1 ? V : 1][16];
    pdl_trigger();
    const int nv = a.dim / 8, group = blockIdx.x / chunks, chunk = blockIdx.x - group * chunks;
    const int slot = threadIdx.x >> 4;
    const int64_t row0 = (int64_t)group * RT, row = row0 + slot / BT;
    const int v0 = (chunk * BT * V + slot % BT) * 16 + (threadIdx.x & 15);
    const bool live = row < a.rows;
    Raw8<F32> g[V], u[V];
    pdl_wait();
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int v = v0 + k * BT * 16;
        g[k].load(a.gate + row * a.gs * (F32 ? 4 : 2), v, live && v < nv);
        if (GATED) u[k].load(a.up + row * a.us * (F32 ? 4 : 2), v, live && v < nv);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int v = v0 + k * BT * 16;
        const bool have = live && v < nv;
        float x[8];
        g[k].get(x);
        if (GATED) {
            float y[8];
            u[k].get(y);
            gate8<ACT>(x, y);
        }
        if (out == SPEC_DTYPE_E4M3) {
            const float m = put_e4m3<false>(a.out, row * nv + v, have, x, 1.f);
            if (RT > 1) {
                if ((threadIdx.x & 15) == 0) top[RT > 1 ? k : 0][slot] = m;
            } else if ((threadIdx.x & 15) == 0 && have) {
                a.scale[(v >> 4) * a.scale_stride + row] = m / kFp8Max;
            }
        } else if (have) {
            store8(a.out, row * nv + v, out == SPEC_DTYPE_F32, x);
        }
    }
    if (RT > 1 && out == SPEC_DTYPE_E4M3) {
        __syncthreads();
        if (threadIdx.x < 16 * V) {
            const int k = threadIdx.x >> 4, r = threadIdx.x & 15, b = chunk * V + k;
            if (row0 + r < a.rows && b * 16 < nv) a.scale[b * a.scale_stride + row0 + r] = top[RT > 1 ? k : 0][r] / kFp8Max;
        }
    }
}

template <bool F32, int ACT>
static cudaError_t launch_act_t(const ActArgs& a, int out, int sms, cudaStream_t st) {
    // 16 rows and three blocks of them a CTA where that gives every SM one, else a row's blocks side by side.  (Two, three, four,
    // six, in one run: activation of 1152 x 12288 12.7 / 12.5 / 12.8 / 13.8 us, rounding of 1152 x 4096 4.35 / 3.85 / 4.05 /
    // 4.5, of 16384 37.7 / 33.5 / 33.2 / 34.6.)
    const long long blocks = scale_blocks(a.dim), groups = ((long long)a.rows + 15) / 16;
    if ((blocks + 2) / 3 * groups >= sms) {
        const long long chunks = (blocks + 2) / 3;
        return launch_pdl(act_kernel<F32, ACT, 16, 3>, dim3((unsigned)(chunks * groups)), kActThreads, 0, st, a, out, (int)chunks);
    }
    const long long chunks = (blocks + 15) / 16;
    return launch_pdl(act_kernel<F32, ACT, 1, 1>, dim3((unsigned)(chunks * a.rows)), kActThreads, 0, st, a, out, (int)chunks);
}

cudaError_t launch_act(const ActArgs& a, spec_dtype_t in, spec_dtype_t out, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    const int sms = di.sm_count;
    const int o = (int)out;
    if (in == SPEC_DTYPE_F32)
        return a.act == SPEC_ACT_SILU        ? launch_act_t<true, SPEC_ACT_SILU>(a, o, sms, st)
               : a.act == SPEC_ACT_GELU_TANH ? launch_act_t<true, SPEC_ACT_GELU_TANH>(a, o, sms, st)
                                             : launch_act_t<true, kActNone>(a, o, sms, st);
    return a.act == SPEC_ACT_SILU        ? launch_act_t<false, SPEC_ACT_SILU>(a, o, sms, st)
           : a.act == SPEC_ACT_GELU_TANH ? launch_act_t<false, SPEC_ACT_GELU_TANH>(a, o, sms, st)
                                         : launch_act_t<false, kActNone>(a, o, sms, st);
}

// ---- rounding of weights -------------------------------------------------------------
// A CTA a block of 128 x 128: 16 lanes a row, 16 rows at a time.  24576 x 4096 bf16: 45.5 us, 6.6 TB/s,
// with four CTAs an SM; 55 with the two that more registers leave; two blocks side by side, so that
// rows are read 512 bytes at a time: 64.
template <bool F32>
__global__ void __launch_bounds__(256, F32 ? 3 : 4) quantize_tiles_kernel(const TileQuantArgs a, int tiles_n) {
    constexpr int VECTORS = 8, STEP = 16;
    __shared__ float part[8];
    pdl_trigger();
    const int ti = blockIdx.x / tiles_n, tb = blockIdx.x - ti * tiles_n, nv = a.dim / 8;
    const int v = tb * 16 + (threadIdx.x & 15), r0 = ti * kScaleBlock + (threadIdx.x >> 4);
    Raw8<F32> x[VECTORS];
    float m = 0.f;
    pdl_wait();
#pragma unroll
    for (int k = 0; k < VECTORS; ++k)
        x[k].load(a.x + (int64_t)(r0 + STEP * k) * a.xs * (F32 ? 4 : 2), v, v < nv && r0 + STEP * k < a.rows);
#pragma unroll
    for (int k = 0; k < VECTORS; ++k) {
        float y[8];
        x[k].get(y);
        m = fmaxf(m, top8(y));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = kFp8AmaxFloor;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, part[i]);
#pragma unroll
    for (int k = 0; k < VECTORS; ++k) {
        float y[8];
        x[k].get(y);
        if (v < nv && r0 + STEP * k < a.rows) store8_e4m3(a.out, (int64_t)(r0 + STEP * k) * nv + v, kFp8Max / m, y);
    }
    if (threadIdx.x == 0) a.scale[(int64_t)ti * a.scale_stride + tb] = m / kFp8Max;
}

cudaError_t launch_quantize_tiles(const TileQuantArgs& a, spec_dtype_t in, cudaStream_t st) {
    const int tiles_n = scale_blocks(a.dim);
    const long long tiles = (long long)scale_blocks(a.rows) * tiles_n;
    if (tiles >= (1LL << 31)) return cudaErrorInvalidValue;
    return in == SPEC_DTYPE_F32 ? launch_pdl(quantize_tiles_kernel<true>, dim3((unsigned)tiles), 256, 0, st, a, tiles_n)
                                : launch_pdl(quantize_tiles_kernel<false>, dim3((unsigned)tiles), 256, 0, st, a, tiles_n);
}

}  // namespace sv
