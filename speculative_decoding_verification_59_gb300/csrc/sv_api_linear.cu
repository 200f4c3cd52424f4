// The C ABI of the target model's dense side: argument validation and
// dispatch.  Declarations and contracts are in include/spec_verify.h.
#include <math.h>
#include <stdlib.h>

#include "sv_linear.h"

namespace sv {

static spec_status_t status_of(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }
static bool floats(spec_dtype_t t) { return t == SPEC_DTYPE_F32 || t == SPEC_DTYPE_BF16; }
static bool types(spec_dtype_t t) { return floats(t) || t == SPEC_DTYPE_E4M3; }
static int bytes_of(spec_dtype_t t) { return t == SPEC_DTYPE_F32 ? 4 : t == SPEC_DTYPE_BF16 ? 2 : 1; }

// Rows that are read or written in pieces of 16 bytes.
static bool row_aligned(const void* p, spec_dtype_t t, int64_t stride) {
    return is_aligned(p, 16) && stride * bytes_of(t) % 16 == 0;
}
// An output with contiguous rows of dim elements, and its scales: `steps` strides of at least `least`
// apart (of one, none is used, and 0 may stand there).
static spec_status_t check_out(const void* out, spec_dtype_t t, int dim, const float* scale, int64_t scale_stride, int64_t least, int steps) {
    if (!out) return SPEC_ERR_INVALID_ARG;
    if (t == SPEC_DTYPE_E4M3 && (!scale || (scale_stride < least && (scale_stride != 0 || steps > 1)))) return SPEC_ERR_INVALID_ARG;
    if (dim % (t == SPEC_DTYPE_E4M3 ? 16 : 8)) return SPEC_ERR_MISALIGNED;
    if (!is_aligned(out, 16) || (t == SPEC_DTYPE_E4M3 && !is_aligned(scale, 4))) return SPEC_ERR_MISALIGNED;
    return SPEC_OK;
}
// Rows and elements that the kernels' indexes hold (whole blocks of a row: under 2^31 vectors of 8).
static bool sizes_fit(int rows, int dim) { return rows >= 0 && dim >= 1 && (long long)rows * (scale_blocks(dim) * 16LL) < (1LL << 31); }

}  // namespace sv

using namespace sv;

extern "C" {

spec_status_t spec_add_norm(const void* x, spec_dtype_t x_dtype, int64_t x_stride, const void* residual, spec_dtype_t sum_dtype,
                            int64_t residual_stride, const void* weight, float eps, int rows, int dim, void* sum_out,
                            int64_t sum_stride, void* out, spec_dtype_t out_dtype, float* out_scale, int64_t scale_stride,
                            cudaStream_t stream) {
    if (!floats(x_dtype) || (residual && !floats(sum_dtype)) || !types(out_dtype)) return SPEC_ERR_UNSUPPORTED_DTYPE;
    if (!sizes_fit(rows, dim) || !(eps >= 0.f) || !isfinite(eps) || (sum_out && !residual)) return SPEC_ERR_INVALID_ARG;
    if (rows == 0) return SPEC_OK;
    if (!x) return SPEC_ERR_INVALID_ARG;
    const spec_status_t s = check_out(out, out_dtype, dim, out_scale, scale_stride, rows, scale_blocks(dim));
    if (s != SPEC_OK) return s;
    if (!row_aligned(x, x_dtype, x_stride) || (residual && !row_aligned(residual, sum_dtype, residual_stride)) ||
        (sum_out && !row_aligned(sum_out, sum_dtype, sum_stride)) || !is_aligned(weight, 16))
        return SPEC_ERR_MISALIGNED;
    if (sum_out && rows > 1 && llabs(sum_stride) < dim) return SPEC_ERR_INVALID_ARG;       // rows of it that overlap
    NormArgs a = {};
    a.x = static_cast<const char*>(x);
    a.res = static_cast<const char*>(residual);
    a.w = static_cast<const char*>(weight);
    a.xs = x_stride;
    a.rs = residual_stride;
    a.ss = sum_stride;
    a.sum = static_cast<char*>(sum_out);
    a.out = static_cast<char*>(out);
    a.scale = out_scale;
    a.scale_stride = scale_stride;
    a.eps = eps;
    a.rows = rows;
    a.dim = dim;
    return status_of(launch_add_norm(a, x_dtype, sum_dtype, out_dtype, stream));
}

spec_status_t spec_gated_act(const void* gate, const void* up, spec_dtype_t dtype, int64_t gate_stride, int64_t up_stride, spec_act_t act,
                             int rows, int dim, void* out, spec_dtype_t out_dtype, float* out_scale, int64_t scale_stride,
                             cudaStream_t stream) {
    if (!floats(dtype) || !types(out_dtype)) return SPEC_ERR_UNSUPPORTED_DTYPE;
    if (!sizes_fit(rows, dim) || (act != SPEC_ACT_SILU && act != SPEC_ACT_GELU_TANH)) return SPEC_ERR_INVALID_ARG;
    if (rows == 0) return SPEC_OK;
    if (!gate || !up) return SPEC_ERR_INVALID_ARG;
    const spec_status_t s = check_out(out, out_dtype, dim, out_scale, scale_stride, rows, scale_blocks(dim));
    if (s != SPEC_OK) return s;
    if (!row_aligned(gate, dtype, gate_stride) || !row_aligned(up, dtype, up_stride)) return SPEC_ERR_MISALIGNED;
    const ActArgs a{static_cast<const char*>(gate), static_cast<const char*>(up), gate_stride, up_stride, static_cast<char*>(out),
                    out_scale, scale_stride, rows, dim, (int)act};
    return status_of(launch_act(a, dtype, out_dtype, stream));
}

spec_status_t spec_quantize_e4m3(const void* x, spec_dtype_t dtype, int64_t x_stride, int rows, int dim, int block_rows, void* out,
                                 float* out_scale, int64_t scale_stride, cudaStream_t stream) {
    if (!floats(dtype)) return SPEC_ERR_UNSUPPORTED_DTYPE;
    if (!sizes_fit(rows, dim) || (block_rows != 1 && block_rows != kScaleBlock)) return SPEC_ERR_INVALID_ARG;
    if (rows == 0) return SPEC_OK;
    if (!x) return SPEC_ERR_INVALID_ARG;
    const int blocks = scale_blocks(dim);
    const spec_status_t s = block_rows == 1 ? check_out(out, SPEC_DTYPE_E4M3, dim, out_scale, scale_stride, rows, blocks)
                                            : check_out(out, SPEC_DTYPE_E4M3, dim, out_scale, scale_stride, blocks, scale_blocks(rows));
    if (s != SPEC_OK) return s;
    if (!row_aligned(x, dtype, x_stride)) return SPEC_ERR_MISALIGNED;
    if (block_rows == 1) {
        const ActArgs a{static_cast<const char*>(x), nullptr, x_stride, 0, static_cast<char*>(out), out_scale, scale_stride, rows, dim,
                        kActNone};
        return status_of(launch_act(a, dtype, SPEC_DTYPE_E4M3, stream));
    }
    const TileQuantArgs a{static_cast<const char*>(x), x_stride, static_cast<char*>(out), out_scale, scale_stride, rows, dim};
    return status_of(launch_quantize_tiles(a, dtype, stream));
}

size_t spec_matmul_workspace_size(int M, int N, int K) {
    if (M < 0 || N < 0 || K < 1) return 0;
    return matmul_workspace_size(M, N, K);
}

spec_status_t spec_matmul_plan(int M, int N, int K, int sms, const int32_t* clusters, int32_t* plan) {
    if (M < 1 || N < 1 || K < 1 || sms < 0 || sms == 1 || (sms > 0 && !clusters) || !plan) return SPEC_ERR_INVALID_ARG;
    if (K > INT32_MAX - 256 || M > INT32_MAX - 256 || N > INT32_MAX - 256) return SPEC_ERR_INVALID_ARG;
    int out[5];
    const cudaError_t e = matmul_plan(M, N, K, sms, clusters, out);
    if (e != cudaSuccess) return e == cudaErrorInvalidValue ? SPEC_ERR_INVALID_ARG : SPEC_ERR_CUDA;
    for (int i = 0; i < 5; ++i) plan[i] = out[i];
    return SPEC_OK;
}

spec_status_t spec_matmul_e4m3(const void* x, int64_t x_stride, const float* x_scale, int64_t x_scale_stride, const void* w,
                               int64_t w_stride, const float* w_scale, int64_t w_scale_stride, int M, int N, int K, void* out,
                               spec_dtype_t out_dtype, int64_t out_stride, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
    if (!floats(out_dtype)) return SPEC_ERR_UNSUPPORTED_DTYPE;
    if (M < 0 || N < 0 || K < 1) return SPEC_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SPEC_OK;
    if (!x || !x_scale || !w || !w_scale || !out || !workspace) return SPEC_ERR_INVALID_ARG;
    const int blocks = scale_blocks(K), rows = scale_blocks(N);
    if ((M > 1 && x_stride < K) || (N > 1 && w_stride < K) || (M > 1 && out_stride < N) || (blocks > 1 && x_scale_stride < M) ||
        (rows > 1 && w_scale_stride < blocks))
        return SPEC_ERR_INVALID_ARG;
    if (K > INT32_MAX - 256 || M > INT32_MAX - 256 || N > INT32_MAX - 256 || x_stride >= (1LL << 40) || w_stride >= (1LL << 40) || x_scale_stride >= (1LL << 38))
        return SPEC_ERR_INVALID_ARG;
    const bool few = M > 1 && M <= kMmFew;     // rows whose scales a TMA load brings
    if (!is_aligned(x, 16) || !is_aligned(w, 16) || !is_aligned(x_scale, few ? 16 : 4) || (M > 1 && x_stride % 16) ||
        (N > 1 && w_stride % 16) || (few && blocks > 1 && x_scale_stride % 4) || !is_aligned(w_scale, 4) ||
        !is_aligned(out, bytes_of(out_dtype)) || !is_aligned(workspace, 256))
        return SPEC_ERR_MISALIGNED;
    if (workspace_bytes < matmul_workspace_size(M, N, K)) return SPEC_ERR_WORKSPACE_TOO_SMALL;
    MatmulArgs a = {};
    a.x = static_cast<const char*>(x);
    a.w = static_cast<const char*>(w);
    a.xld = M > 1 ? x_stride : ((int64_t)K + 15) / 16 * 16;    // (of one row no stride is used)
    a.wld = N > 1 ? w_stride : ((int64_t)K + 15) / 16 * 16;
    a.xscale = x_scale;
    a.wscale = w_scale;
    a.xs_stride = blocks > 1 ? x_scale_stride : ((int64_t)M + 3) / 4 * 4;
    a.ws_stride = w_scale_stride;
    a.M = M;
    a.N = N;
    a.K = K;
    a.out = static_cast<char*>(out);
    a.old = M > 1 ? out_stride : ((int64_t)N + 7) / 8 * 8;
    a.f32 = out_dtype == SPEC_DTYPE_F32;
    a.ws = static_cast<char*>(workspace);
    return status_of(launch_matmul(a, stream));
}

}  // extern "C"
