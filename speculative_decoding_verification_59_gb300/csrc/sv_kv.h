// Internal declarations of the cache and attention calls and of the token
// log-probabilities: host-side launch entry points (the C ABI in sv_api_kv.cu
// checks the arguments) and what their sizes are derived from.
#pragma once

#include "sv_internal.h"

namespace sv {

constexpr int kMaxNewChain = 257;      // new positions per sequence, chains
constexpr int kMaxNewTree = 64;        // trees: one ancestor bit per node in a 64-bit word
constexpr int kMaxGroup = 64;          // query heads per cached head
constexpr float kFp8Max = 448.f;       // largest finite e4m3 value
constexpr float kFp8AmaxFloor = 1e-20f;

struct AppendArgs {
    spec_kv_cache_t c;
    const char *q, *k, *v;                 // bf16
    int64_t qs, ks, vs;                    // bytes between tokens
    const char *qw, *kw;
    float eps;
    const float* rope;
    int rope_rows, rot, inter;
    const int32_t *ctx, *newl, *pos;
    int B, N, Hq;
    char* q_out;
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t st);

cudaError_t launch_kv_read(const spec_kv_cache_t& c, const int32_t* starts, const int32_t* counts, int B, int T,
                           bool f32, void* out_k, void* out_v, cudaStream_t st);
cudaError_t launch_kv_compact(const spec_kv_cache_t& c, const int32_t* ctx, const int32_t* path,
                              const int32_t* acc, int B, int N, cudaStream_t st);

struct AttendArgs {
    spec_kv_cache_t c;
    const char* q;                         // bf16
    int64_t qs;                            // bytes between tokens
    const int32_t *ctx, *newl, *par;
    float scale;
    int B, N, Hq, G;                       // G query heads per cached head
    uint32_t g_mul;                        // ceil(2^32 / G), for G > 1: R / G = mulhi(R, g_mul), R < 2^32 / G
    int page_shift;                        // log2(page_size), -1 when it is no power of two
    int whole;                             // units are dealt whole, not by tiles (set at the launch)
    char* out;                             // bf16
    float* lse;
    char* ws;
};
size_t attend_workspace_size(int B, int N, int Hq, int Hkv, int D);
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st);

// The merge keeps two bytes for each 4 KB chunk of a row in shared memory.
constexpr int kMaxLogprobVocab = 1 << 23;
size_t logprobs_workspace_size(int rows, int V, int K);
cudaError_t launch_logprobs(const void* z, spec_dtype_t dt, const int32_t* tok, float T, int rows, int V, int K,
                            float* lp, float* ent, int32_t* ti, float* tl, void* ws, cudaStream_t st);

}  // namespace sv
