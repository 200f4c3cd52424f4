// The C ABI of the cache, attention and log-probability calls: argument
// validation and dispatch.  Declarations and contracts are in
// include/spec_verify.h.
#include <math.h>

#include "sv_kv.h"

namespace sv {

static spec_status_t status_of(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

// The cache description of a call on B > 0 sequences.
static spec_status_t check_cache(const spec_kv_cache_t* c) {
    if (!c) return SPEC_ERR_INVALID_ARG;
    if (c->dtype != SPEC_DTYPE_BF16 && c->dtype != SPEC_DTYPE_E4M3) return SPEC_ERR_UNSUPPORTED_DTYPE;
    if (!c->k || !c->v || !c->block_table) return SPEC_ERR_INVALID_ARG;
    if (c->dtype == SPEC_DTYPE_E4M3 && (!c->k_scale || !c->v_scale)) return SPEC_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return SPEC_ERR_INVALID_ARG;
    if (c->layers < 1 || c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1 || c->kv_heads < 1)
        return SPEC_ERR_INVALID_ARG;
    if ((long long)c->max_pages * c->page_size >= (1LL << 31) - 4096) return SPEC_ERR_INVALID_ARG;
    const int64_t per = c->dtype == SPEC_DTYPE_E4M3 ? 16 : 8;      // elements in 16 bytes
    if (!is_aligned(c->block_table, 4) || !is_aligned(c->k_scale, 4) || !is_aligned(c->v_scale, 4))
        return SPEC_ERR_MISALIGNED;
    if (!is_aligned(c->k, 16) || !is_aligned(c->v, 16)) return SPEC_ERR_MISALIGNED;
    if (c->page_stride % per || c->token_stride % per || c->head_stride % per || c->layer_stride % per)
        return SPEC_ERR_MISALIGNED;
    return SPEC_OK;
}

}  // namespace sv

using namespace sv;

extern "C" {

spec_status_t spec_kv_append(const spec_kv_cache_t* cache, const void* q, const void* k,
                             const void* v, int64_t q_token_stride, int64_t k_token_stride,
                             int64_t v_token_stride, const void* q_weight, const void* k_weight,
                             float eps, const float* rope, int rope_rows, int rot_dim,
                             int interleaved, const int32_t* context_lens,
                             const int32_t* new_lens, const int32_t* positions, int B, int N,
                             int q_heads, void* q_out, cudaStream_t stream) {
    if (B < 0 || N < 1 || q_heads < 0) return SPEC_ERR_INVALID_ARG;
    if (B == 0) return SPEC_OK;
    const spec_status_t s = check_cache(cache);
    if (s != SPEC_OK) return s;
    if (!k || !v || !context_lens || (q_heads > 0 && (!q || !q_out))) return SPEC_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 16 || (rot_dim > 0 && (!rope || rope_rows < 1)))
        return SPEC_ERR_INVALID_ARG;
    if ((q_weight || k_weight) && !(eps >= 0.f && isfinite(eps))) return SPEC_ERR_INVALID_ARG;
    if ((long long)B * N >= (1LL << 31) || (long long)B * N * ((long long)q_heads + 2LL * cache->kv_heads) >= (1LL << 31))
        return SPEC_ERR_INVALID_ARG;
    if (!is_aligned(k, 16) || !is_aligned(v, 16) || k_token_stride % 8 || v_token_stride % 8 ||
        (q_heads > 0 && (!is_aligned(q, 16) || !is_aligned(q_out, 16) || q_token_stride % 8)) ||
        (q_weight && !is_aligned(q_weight, 16)) || (k_weight && !is_aligned(k_weight, 16)) ||
        (rot_dim > 0 && !is_aligned(rope, 16)))
        return SPEC_ERR_MISALIGNED;
    AppendArgs a = {};
    a.c = *cache;
    a.q = static_cast<const char*>(q);
    a.k = static_cast<const char*>(k);
    a.v = static_cast<const char*>(v);
    a.qs = 2 * q_token_stride;
    a.ks = 2 * k_token_stride;
    a.vs = 2 * v_token_stride;
    a.qw = static_cast<const char*>(q_weight);
    a.kw = static_cast<const char*>(k_weight);
    a.eps = eps;
    a.rope = rope;
    a.rope_rows = rope_rows;
    a.rot = rot_dim;
    a.inter = interleaved != 0;
    a.ctx = context_lens;
    a.newl = new_lens;
    a.pos = positions;
    a.B = B;
    a.N = N;
    a.Hq = q_heads;
    a.q_out = static_cast<char*>(q_out);
    return status_of(launch_append(a, stream));
}

spec_status_t spec_kv_read(const spec_kv_cache_t* cache, const int32_t* starts,
                           const int32_t* counts, int B, int T, spec_dtype_t out_dtype,
                           void* out_k, void* out_v, cudaStream_t stream) {
    if (out_dtype != SPEC_DTYPE_F32 && out_dtype != SPEC_DTYPE_BF16) return SPEC_ERR_UNSUPPORTED_DTYPE;
    if (B < 0 || T < 0) return SPEC_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return SPEC_OK;
    const spec_status_t s = check_cache(cache);
    if (s != SPEC_OK) return s;
    if (!out_k || !out_v || B > 65535 || (long long)T * cache->kv_heads >= (1LL << 31)) return SPEC_ERR_INVALID_ARG;
    if (!is_aligned(out_k, 16) || !is_aligned(out_v, 16)) return SPEC_ERR_MISALIGNED;
    return status_of(launch_kv_read(*cache, starts, counts, B, T, out_dtype == SPEC_DTYPE_F32, out_k, out_v, stream));
}

spec_status_t spec_kv_compact(const spec_kv_cache_t* cache, const int32_t* context_lens,
                              const int32_t* path_nodes, const int32_t* num_accepted, int B,
                              int N, cudaStream_t stream) {
    if (B < 0 || N < 1 || N > 1024) return SPEC_ERR_INVALID_ARG;
    if (B == 0) return SPEC_OK;
    const spec_status_t s = check_cache(cache);
    if (s != SPEC_OK) return s;
    if (!context_lens || !path_nodes || !num_accepted || B > 65535) return SPEC_ERR_INVALID_ARG;
    if ((long long)cache->layers * cache->kv_heads >= (1LL << 31) / (2 * 256 * 2 / 16)) return SPEC_ERR_INVALID_ARG;
    return status_of(launch_kv_compact(*cache, context_lens, path_nodes, num_accepted, B, N, stream));
}

size_t spec_attention_workspace_size(int B, int N, int q_heads, int kv_heads, int head_dim) {
    if (B < 0 || N < 1 || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads) return 0;
    if (N > kMaxNewChain || q_heads / kv_heads > kMaxGroup) return 0;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    return attend_workspace_size(B, N, q_heads, kv_heads, head_dim);
}

spec_status_t spec_paged_attention(const spec_kv_cache_t* cache, const void* q,
                                   int64_t q_token_stride, const int32_t* context_lens,
                                   const int32_t* new_lens, const int32_t* parents, float scale,
                                   int B, int N, int q_heads, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (B < 0 || N < 1 || N > (parents ? kMaxNewTree : kMaxNewChain) || !isfinite(scale)) return SPEC_ERR_INVALID_ARG;
    if (B == 0) return SPEC_OK;
    const spec_status_t s = check_cache(cache);
    if (s != SPEC_OK) return s;
    const int Hkv = cache->kv_heads;
    if (q_heads < Hkv || q_heads % Hkv || q_heads / Hkv > kMaxGroup) return SPEC_ERR_INVALID_ARG;
    if (!q || !context_lens || !out || !workspace) return SPEC_ERR_INVALID_ARG;
    if ((long long)B * N >= (1LL << 31) || (long long)B * N * q_heads >= (1LL << 31)) return SPEC_ERR_INVALID_ARG;
    if (!is_aligned(q, 16) || !is_aligned(out, 16) || q_token_stride % 8 || !is_aligned(workspace, 256))
        return SPEC_ERR_MISALIGNED;
    if (workspace_bytes < attend_workspace_size(B, N, q_heads, Hkv, cache->head_dim))
        return SPEC_ERR_WORKSPACE_TOO_SMALL;
    AttendArgs a = {};
    a.c = *cache;
    a.q = static_cast<const char*>(q);
    a.qs = 2 * q_token_stride;
    a.ctx = context_lens;
    a.newl = new_lens;
    a.par = parents;
    a.scale = scale;
    a.B = B;
    a.N = N;
    a.Hq = q_heads;
    a.G = q_heads / Hkv;
    a.g_mul = (uint32_t)(((1ull << 32) + (uint64_t)a.G - 1) / (uint64_t)a.G);
    a.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (cache->page_size == 1 << i) a.page_shift = i;
    a.out = static_cast<char*>(out);
    a.lse = lse;
    a.ws = static_cast<char*>(workspace);
    return status_of(launch_attend(a, stream));
}

size_t spec_logprobs_workspace_size(int rows, int V, int K) {
    if (rows < 0 || V < 1 || V > kMaxLogprobVocab || K < 0 || K > 8) return 0;
    return logprobs_workspace_size(rows, V, K);
}

spec_status_t spec_token_logprobs(const void* logits, spec_dtype_t dtype, const int32_t* tokens,
                                  float temperature, int rows, int V, int K, float* out_logprob,
                                  float* out_entropy, int32_t* out_top_idx,
                                  float* out_top_logprob, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
    if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return SPEC_ERR_UNSUPPORTED_DTYPE;
    if (rows < 0 || V < 1 || V > kMaxLogprobVocab || K < 0 || K > 8) return SPEC_ERR_INVALID_ARG;
    if (!(temperature >= 1e-20f) || !isfinite(temperature)) return SPEC_ERR_INVALID_ARG;
    if ((long long)rows * ((long long)nseg(V, elt_size(dtype)) + 1) >= (1LL << 31)) return SPEC_ERR_INVALID_ARG;
    if (rows == 0) return SPEC_OK;
    if (!logits || !tokens || !out_logprob || (K > 0 && (!out_top_idx || !out_top_logprob)) || !workspace)
        return SPEC_ERR_INVALID_ARG;
    if (!is_aligned(logits, 16) || !is_aligned(workspace, 256)) return SPEC_ERR_MISALIGNED;
    if (workspace_bytes < logprobs_workspace_size(rows, V, K)) return SPEC_ERR_WORKSPACE_TOO_SMALL;
    return status_of(launch_logprobs(logits, dtype, tokens, temperature, rows, V, K, out_logprob, out_entropy,
                                     out_top_idx, out_top_logprob, workspace, stream));
}

}  // extern "C"
