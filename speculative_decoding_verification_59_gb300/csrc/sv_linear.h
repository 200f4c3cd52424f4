// Internal declarations of the target model's dense side: 8-bit rows and
// weights with a scale for each block of 128 elements, the operators that make
// them and their product.  The C ABI in sv_api_linear.cu checks the arguments.
#pragma once

#include "sv_kv.h"

namespace sv {

constexpr int kScaleBlock = 128;       // elements of a row, or rows and columns of a weight, that share a scale
inline int scale_blocks(int n) { return (n - 1) / kScaleBlock + 1; }

struct NormArgs {
    const char *x, *res, *w;           // res, w nullable
    int64_t xs, rs, ss;                // elements between rows: x, residual, sum
    char *sum, *out;                   // sum nullable
    float* scale;                      // E4M3 output: block b of row r at b * scale_stride + r
    int64_t scale_stride;
    float eps;
    int rows, dim;
};
cudaError_t launch_add_norm(const NormArgs& a, spec_dtype_t x, spec_dtype_t sum, spec_dtype_t out, cudaStream_t st);

struct ActArgs {
    const char *gate, *up;             // up null: the values themselves (rounding rows to 8 bits)
    int64_t gs, us;                    // elements between rows
    char* out;
    float* scale;
    int64_t scale_stride;
    int rows, dim, act;
};
constexpr int kActNone = -1;
cudaError_t launch_act(const ActArgs& a, spec_dtype_t in, spec_dtype_t out, cudaStream_t st);

// Blocks of 128 x 128; scale of block (i, b) at i * scale_stride + b.
struct TileQuantArgs {
    const char* x;
    int64_t xs;
    char* out;
    float* scale;
    int64_t scale_stride;
    int rows, dim;
};
cudaError_t launch_quantize_tiles(const TileQuantArgs& a, spec_dtype_t in, cudaStream_t st);

constexpr int kMmFew = 64;             // rows that the transposed product takes
struct MatmulArgs {
    const char *x, *w;                 // e4m3
    int64_t xld, wld;                  // bytes between rows
    const float *xscale, *wscale;
    int64_t xs_stride, ws_stride;      // x: from block to block; w: from block row to block row
    int M, N, K;
    char* out;
    int64_t old;                       // elements between rows of out
    int f32;
    char* ws;
};
size_t matmul_workspace_size(int M, int N, int K);
cudaError_t launch_matmul(const MatmulArgs& a, cudaStream_t st);
// spec_matmul_plan's entries.
cudaError_t matmul_plan(int M, int N, int K, int sms, const int* clusters, int (&out)[5]);

}  // namespace sv
