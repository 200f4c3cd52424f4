/*
 * spec_verify.h - C ABI of the GB300 (sm_103a) speculative-decoding
 * verification library (libspecverify.so).
 *
 * The operation is the target-model verification step of speculative
 * decoding as defined in:
 *   [SD]     "Speculative decoding: guess a few tokens first - why the answer
 *            stays the same" (explainer blog).  Section "What happens in one
 *            round": the target scores all gamma drafts (plus one position)
 *            in one batch, drafts are checked left to right and accepted with
 *            probability min(1, p_i(x_i)/q_i(x_i)), the first rejection voids
 *            the rest and is replaced by a sample from the residual; when all
 *            drafts are accepted a bonus token is sampled from the next
 *            position.  Section "Why fixing wrong guesses does not leave the
 *            target distribution": residual p'(x) = norm(max(0, p(x) - q(x))).
 *            The greedy paragraph: accept while the draft equals the target
 *            argmax, replace the first mismatch by the target token.
 *   [AdaPLD] "AdaPLD: adaptive retrieval and reuse for efficient model-free
 *            speculative decoding", section 3.3 "Tree construction and
 *            verification" and Algorithm 1 (BuildDraftTree / VerifyAndAccept):
 *            a draft tree (main chain plus top-K branches) verified by the
 *            target in one pass.
 *
 * Conventions shared by every call
 *   - Every pointer is a DEVICE pointer owned by the caller; the library never
 *     allocates and keeps no per-call state.  Calls are asynchronous on
 *     `stream`; results are valid once the stream reaches them.  The
 *     library's kernels are launched with programmatic dependent launch: a
 *     call's first kernel may start while the kernel before it on `stream`
 *     finishes, and may then prefetch logits into L2, but it reads the
 *     inputs and the workspace only after that kernel has completed.  Inputs
 *     written by the kernel just before the call on the same stream are
 *     therefore read as written.
 *   - Logits are row-major with V contiguous, dtype SPEC_DTYPE_F32 or
 *     SPEC_DTYPE_BF16.  Logit base pointers must be 16-byte aligned
 *     (SPEC_ERR_MISALIGNED otherwise).  V need not be a multiple of anything.
 *     -inf logits are legal (masked tokens); NaN/+inf logits are undefined.
 *   - `workspace` is caller-owned device scratch of at least
 *     spec_verify_workspace_size() bytes, 256-byte aligned.  Its first 4
 *     bytes are the device error word (below): zero-fill the workspace once
 *     (spec_verify_workspace_init) so that word starts clear.  Everything
 *     else in it is rewritten by each call before it is read, so one
 *     workspace serves calls of any mode and size in turn.  Calls that share
 *     a workspace must be ordered on the device (same stream, or events);
 *     overlapping calls on one workspace race.
 *   - Host-side argument checks return immediately without touching the
 *     device.  Bad input that only the device can see (a draft token outside
 *     [0, V), a row with every logit -inf, a malformed tree) marks that
 *     sequence with num_accepted = -1 and every output token -1, and sets a
 *     bit in the workspace error word (see spec_verify_read_error).
 *   - B = 0 is an empty batch: SPEC_OK, nothing is launched.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SPEC_OK = 0,
    SPEC_ERR_INVALID_ARG = 1,          /* null pointer, negative size, bad temperature */
    SPEC_ERR_UNSUPPORTED_DTYPE = 2,
    SPEC_ERR_MISALIGNED = 3,           /* logits or workspace not aligned as required */
    SPEC_ERR_WORKSPACE_TOO_SMALL = 4,
    SPEC_ERR_CUDA = 5,                 /* a CUDA runtime call or launch failed */
    SPEC_ERR_DEVICE_INPUT = 6,         /* reported by spec_verify_read_error only */
    SPEC_ERR_EXCEEDS_STATIC_SCRATCH = 7 /* spec_verify_sample_noalloc: the problem needs more than
                                           SPEC_VERIFY_NOALLOC_SCRATCH_BYTES of scratch */
} spec_status_t;

/* SPEC_DTYPE_E4M3 (8-bit floats: 4 exponent bits, 3 mantissa bits, largest 448) is a type of
 * cache contents only (spec_kv_cache_t). */
typedef enum { SPEC_DTYPE_F32 = 0, SPEC_DTYPE_BF16 = 1, SPEC_DTYPE_E4M3 = 2 } spec_dtype_t;

/* Bits of the device error word. */
#define SPEC_DEVERR_TOKEN_RANGE  1   /* a draft / node token outside [0, V) */
#define SPEC_DEVERR_EMPTY_ROW    2   /* a logits row whose every entry is -inf (sampling) */
#define SPEC_DEVERR_TREE_PARENT  4   /* parents[0] != -1 or parents[n] not in [0, n) */
#define SPEC_DEVERR_TIMEOUT      8   /* a bounded wait inside a kernel ran out (internal error;
                                        the affected results are not valid) */
#define SPEC_DEVERR_CACHE_RANGE 16   /* a length, position or page id outside the cache, or a
                                        node id outside the tree (cache calls) */

/*
 * Bytes of workspace any of the three verification calls needs for B
 * sequences of `gamma_or_nodes` drafts (chains) or nodes (trees) over a
 * vocabulary of V, for either dtype.  Returns 0 for invalid sizes.
 */
size_t spec_verify_workspace_size(int B, int gamma_or_nodes, int V);

/* Zero-fills a workspace (cudaMemsetAsync on `stream`). */
spec_status_t spec_verify_workspace_init(void* workspace, size_t workspace_bytes,
                                         cudaStream_t stream);

/*
 * Stochastic verification of B independent draft chains ([SD] "What happens in
 * one round", steps 1-4, and the residual of "Why fixing wrong guesses ...").
 *
 *   target_logits [B, gamma+1, V]  target logits z^t; row i scores position i
 *   draft_logits  [B, gamma, V]    draft logits z^d (NULL allowed if gamma == 0)
 *   draft_tokens  [B, gamma] int32 drafted tokens x_0..x_{gamma-1}
 *   uniforms      [B, gamma+1] f32 in [0, 1): u_i decides draft i (accepted iff
 *                                  u_i < p_i(x_i)/q_i(x_i)); u_gamma drives the
 *                                  single final sample (residual or bonus) by
 *                                  inverse CDF in index order
 *   temperature   finite, >= 1e-20; p = softmax(z^t / T), q = softmax(z^d / T)
 *   0 <= gamma <= 256, 1 <= V <= 2097152, B >= 0.  (The final sample scans
 *   the 8192-element chunk totals of a row in one 256-thread CTA, hence the
 *   bound on V; larger V returns SPEC_ERR_INVALID_ARG.)
 * Outputs (device):
 *   out_tokens       [B, gamma+1] int32: the k accepted drafts, the final
 *                    token, then -1
 *   out_num_accepted [B] int32: k in [0, gamma] (emitted tokens = k + 1)
 *   out_logprobs     [B, gamma, 2] f32, nullable: ln p_i(x_i), ln q_i(x_i)
 *
 * A streaming pass over every logit row (row max and sum-exp partials) is
 * followed by two kernels: the accept decisions, then the chunk sums of the
 * exponentials and of the residual weights of the one rejected (or bonus)
 * row pair, in which the last chunk of each sequence to finish runs the
 * inverse-CDF search.
 */
spec_status_t spec_verify_sample(const void* target_logits, const void* draft_logits,
                                 spec_dtype_t dtype, const int32_t* draft_tokens,
                                 const float* uniforms, float temperature, int B, int gamma,
                                 int V, int32_t* out_tokens, int32_t* out_num_accepted,
                                 float* out_logprobs, void* workspace, size_t workspace_bytes,
                                 cudaStream_t stream);

/*
 * Lazy (early-exit) stochastic verification ([SD] "What happens in one
 * round", step 3: the first rejection discards every later draft, so a
 * position's rows are only needed while every earlier draft was accepted).
 * Same arguments, workspace and outputs as spec_verify_sample, with the same
 * tokens and accept counts.  The positions are streamed in groups of
 * doubling size -- [0, 2), [2, 6), [6, 14), ... -- each group one pass over
 * the GPU for the sequences whose drafts before it were all accepted, so
 * after a rejection at k only the rows of the groups up to k's are read (at
 * most positions 0..2k+1), all 2 gamma + 1 rows when every draft is
 * accepted.  A group runs on to the end (at most 128 positions) when the
 * rows after it, for all B sequences, hold fewer than 96 MB: a pass then
 * costs more than it can save.  spec_verify_set_lazy_split_bytes, or the
 * environment variable SPEC_VERIFY_LAZY_SPLIT_BYTES read once at the first
 * lazy call or groups query of the process, overrides that figure (0: split
 * at every boundary); the outputs do not depend on it.  out_logprobs (nullable)
 * holds the log-probabilities of positions 0..min(k, gamma - 1); later
 * positions, and every position of a bad sequence, are NaN.  Rows whose
 * byte length is not a multiple of 16 take the full pass (every row read)
 * with the same outputs.  Device-side bad-input detection covers the rows
 * decided: positions 0..k.
 */
spec_status_t spec_verify_sample_lazy(const void* target_logits, const void* draft_logits,
                                      spec_dtype_t dtype, const int32_t* draft_tokens,
                                      const float* uniforms, float temperature, int B, int gamma,
                                      int V, int32_t* out_tokens, int32_t* out_num_accepted,
                                      float* out_logprobs, void* workspace, size_t workspace_bytes,
                                      cudaStream_t stream);

/*
 * The position groups that spec_verify_sample_lazy streams for B sequences of
 * gamma drafts over V logits of the given dtype ([SD] "What happens in one
 * round", step 3, read as in spec_verify_sample_lazy): writes the groups'
 * upper ends, exclusive, to ends[0 .. count) in ascending order (group g
 * covers positions ends[g-1] .. ends[g]-1, from 0; the last end is gamma + 1)
 * and returns count, at most 8.  The sizes double from 2 -- [0,2), [2,6),
 * [6,14), ... -- and a group runs on to the end (at most 128 positions) when
 * the rows after it, for all B sequences, hold fewer than 96 MB (or the
 * figure set as described for spec_verify_sample_lazy).  Host only, no CUDA
 * call; returns 0 for invalid arguments (B < 1, gamma outside 0..256, V < 1,
 * an unknown dtype, ends NULL).  ends must hold 8 entries.  The groups of a
 * lazy call are those this function returns with the same figure in force.
 */
int spec_verify_lazy_groups(int B, int gamma, int V, spec_dtype_t dtype, int32_t* ends);

/*
 * Sets the figure of spec_verify_sample_lazy's group rule: a group runs on to
 * the end when the rows after it hold fewer than `bytes` (0: split at every
 * boundary; negative: back to the built-in 96 MB).  Process-wide, for calls
 * and queries made afterwards from any thread; it replaces the value of
 * SPEC_VERIFY_LAZY_SPLIT_BYTES.  Host only.
 */
void spec_verify_set_lazy_split_bytes(double bytes);

/*
 * The two halves of spec_verify_sample, for callers that want to overlap or
 * time them separately; spec_verify_sample is exactly _stats then _finish on
 * the same stream with the same arguments and workspace.
 *   _stats:  streams every logit row once and leaves per-row partial
 *            statistics (running max and sum of exponentials) in the
 *            workspace.  Writes no output.
 *   _finish: takes the accept decisions from those statistics and draws the
 *            final token of every sequence (residual after a rejection, bonus
 *            otherwise); writes every output of spec_verify_sample.
 * The workspace and the logits must stay unchanged between the two calls.
 */
spec_status_t spec_verify_sample_stats(const void* target_logits, const void* draft_logits,
                                       spec_dtype_t dtype, float temperature, int B, int gamma,
                                       int V, void* workspace, size_t workspace_bytes,
                                       cudaStream_t stream);
spec_status_t spec_verify_sample_finish(const void* target_logits, const void* draft_logits,
                                        spec_dtype_t dtype, const int32_t* draft_tokens,
                                        const float* uniforms, float temperature, int B,
                                        int gamma, int V, int32_t* out_tokens,
                                        int32_t* out_num_accepted, float* out_logprobs,
                                        void* workspace, size_t workspace_bytes,
                                        cudaStream_t stream);

/*
 * Greedy verification ([SD] greedy paragraph): g_i = argmax_j z^t[b,i,j]
 * (lowest index among equal logits), k = first i with x_i != g_i, else gamma.
 * Draft logits are not needed.
 *   target_logits [B, gamma+1, V], draft_tokens [B, gamma] (NULL if gamma == 0)
 *   out_tokens [B, gamma+1]: x_0..x_{k-1}, g_k, then -1;  out_num_accepted [B]: k
 */
spec_status_t spec_verify_greedy(const void* target_logits, spec_dtype_t dtype,
                                 const int32_t* draft_tokens, int B, int gamma, int V,
                                 int32_t* out_tokens, int32_t* out_num_accepted, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream);

/*
 * Greedy verification of a draft tree ([AdaPLD] 3.3, Algorithm 1).
 *   target_logits [B, N, V]: row n scores the continuation after node n
 *   node_tokens   [B, N] int32: token of node n (node 0, the root, is ignored)
 *   parents       [B, N] int32: parents[0] = -1, 0 <= parents[n] < n
 * A node is accepted when its parent is accepted and its token equals the
 * argmax of the parent's row (the root is accepted).  Result: the longest
 * root path of accepted nodes (ties: lexicographically smallest node ids) and
 * the bonus token argmax(row of the path's last node).
 *   out_path_nodes   [B, N]: path node ids (root excluded), then -1
 *   out_tokens       [B, N]: path tokens, then the bonus token, then -1
 *   out_num_accepted [B]: path length
 */
spec_status_t spec_verify_tree_greedy(const void* target_logits, spec_dtype_t dtype,
                                      const int32_t* node_tokens, const int32_t* parents, int B,
                                      int N, int V, int32_t* out_path_nodes, int32_t* out_tokens,
                                      int32_t* out_num_accepted, void* workspace,
                                      size_t workspace_bytes, cudaStream_t stream);

/*
 * Branch tokens of a draft tree ([AdaPLD] 3.3 "strict hit path" and
 * Algorithm 1: TopKNextTokens(M, x_{<=p*}, K) \ {d_main[1]}): for each of
 * `rows` rows of V logits, the K tokens with the largest logits (larger logit
 * first, lower index first among equal logits, -0.0 equal to +0.0), then the
 * row's excluded token removed from that list when it is in it.  The list
 * keeps its order and is padded with -1 (value -inf), also when V < K.
 *   logits   [rows, V], row-major, 16-byte aligned, bf16 or fp32; -inf
 *            (masked) logits are ordinary values, NaN is undefined
 *   exclude  [rows] int32 (NULL: no exclusion); -1, or any value outside
 *            [0, V), excludes nothing
 *   out_idx  [rows, K] int32
 *   out_val  [rows, K] float (NULL: not written): the logits of out_idx
 * 1 <= K <= 8.  Workspace: spec_topk_workspace_size(rows, V, K) bytes,
 * 256-byte aligned, its first 256 bytes zero-filled once (the error word, as
 * for the verification calls); nothing else is carried between calls.
 */
size_t spec_topk_workspace_size(int rows, int V, int K);
spec_status_t spec_topk_exclude(const void* logits, spec_dtype_t dtype, int rows, int V, int K,
                                const int32_t* exclude, int32_t* out_idx, float* out_val,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Lexical retrieval of a reuse position ([AdaPLD] 3.2 "lexical retrieval
 * stage", 3.3 "strict hit path", Algorithm 1 LexicalRetrieval and d_main):
 * sequence b's context is tokens[b, 0 .. lengths[b]-1] and its query its last
 * w tokens.  A match is a position p with w-1 <= p <= lengths[b]-2 whose
 * window tokens[b, p-w+1 .. p] equals the query.  The pages choose among the
 * matches by hidden-state similarity; here the most recent match p* is the
 * reuse position.
 *   tokens      [B, n_max] int32, 16-byte aligned, n_max a multiple of 4;
 *               entries at or past lengths[b] are ignored
 *   lengths     [B] int32 in 1..n_max (device); another value marks the
 *               sequence bad: out_count -1, every output -1, error bit
 *               SPEC_DEVERR_TOKEN_RANGE
 *   out_count   [B]: number of matches
 *   out_matches [B, max_matches]: the first max_matches match positions in
 *               ascending order, then -1
 *   out_draft   [B, L] (NULL: not written): tokens[b, p*+1 .. min(p*+L,
 *               lengths[b]-1)], then -1; all -1 without a match
 * 1 <= w <= 8, 0 <= L <= 1024, 1 <= max_matches <= 4096.  Workspace:
 * spec_ngram_workspace_size(B, n_max, max_matches) bytes, 256-byte aligned,
 * first 256 bytes zero-filled once (the error word).
 */
size_t spec_ngram_workspace_size(int B, int n_max, int max_matches);
spec_status_t spec_ngram_retrieve(const int32_t* tokens, const int32_t* lengths, int B, int n_max,
                                  int w, int L, int max_matches, int32_t* out_count,
                                  int32_t* out_matches, int32_t* out_draft, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream);

/*
 * Semantic fallback of the reuse-position search ([AdaPLD] 3.2 "semantic
 * fallback stage", Algorithm 1 SemanticFallback): for each sequence b,
 * score(j) = h . H_j / (|h| |H_j|) over its window of W hidden states (the
 * states of the most recent forward steps), then the delta largest scores,
 * larger first, lower window index first among equal scores.  A zero norm
 * gives score 0.  Scores are accumulated in fp32 (|error| ~1e-6).
 *   hidden     [B, W, d] bf16 or fp32, 16-byte aligned, d a multiple of 8
 *              (bf16) or 4 (fp32)
 *   query      [B, d] same dtype, 16-byte aligned
 *   positions  [B, W] int32 (NULL: the window index): the context position of
 *              each window row
 *   out_idx    [B, delta] window rows, -1 padded when W < delta
 *   out_pos    [B, delta] (NULL: not written) their positions, -1 padded
 *   out_score  [B, delta] (NULL: not written) their scores, -inf padded
 * 1 <= delta <= 8, W >= 1.  Workspace: spec_cosine_workspace_size(B, W)
 * bytes, 256-byte aligned.
 */
size_t spec_cosine_workspace_size(int B, int W);
spec_status_t spec_cosine_topk(const void* hidden, const void* query, spec_dtype_t dtype, int B,
                               int W, int d, int delta, const int32_t* positions,
                               int32_t* out_idx, int32_t* out_pos, float* out_score,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * spec_verify_sample for callers that cannot allocate device memory.
 *
 * The source pages have no counterpart to this call; it exists for callers
 * that cannot provide a workspace: a plugin whose host framework owns all
 * device memory in its own pool and passes in only input and output buffers,
 * or a decode loop that must not call cudaMalloc/cudaFree (which can
 * synchronise the device) in the middle of a step.  Arguments, outputs and
 * results are those of spec_verify_sample without the workspace; the same
 * kernels run.  The call allocates nothing and calls no allocating routine.
 *
 * Scratch: a fixed array of SPEC_VERIFY_NOALLOC_SCRATCH_BYTES (8 MiB) that the
 * library places in the device memory of every GPU it is loaded on, held
 * until the process exits.  Problems whose scratch need,
 * spec_verify_workspace_size(B, gamma, V), exceeds it are rejected with
 * SPEC_ERR_EXCEEDS_STATIC_SCRATCH before anything is launched (B = 256
 * sequences of 4 drafts over 128256 fp32 logits need 6.8 MB).
 *
 * The first call on each device, made while that device is current, looks up
 * the array's device address (cudaGetSymbolAddress, which may also load the
 * library's kernels onto that device); make that first call before any stream
 * capture.  The address is kept for the life of the process: after
 * cudaDeviceReset (or any other reset of the device's primary context) in the
 * same process, this entry point must not be called again on that device.  Every call on a device shares the one array, so calls whose work
 * overlaps on the GPU (different streams without ordering, or host threads
 * racing on one device) race on it and give undefined results; order them.
 * Bad input is reported per sequence (num_accepted = -1, tokens -1) only: the
 * device error word of the workspace calls is not readable for this entry.
 */
#define SPEC_VERIFY_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
spec_status_t spec_verify_sample_noalloc(const void* target_logits, const void* draft_logits,
                                         spec_dtype_t dtype, const int32_t* draft_tokens,
                                         const float* uniforms, float temperature, int B,
                                         int gamma, int V, int32_t* out_tokens,
                                         int32_t* out_num_accepted, float* out_logprobs,
                                         cudaStream_t stream);

/* ==========================================================================
 * The target model's side of a verification step.  [SD] "What happens in one
 * round", step 2: the target scores the drafted positions in one pass over
 * its cached context; the source pages leave that pass to the model.  These
 * calls are its cache and attention parts, for chains and for draft trees,
 * and the log-probabilities a server reports about the emitted tokens.
 *
 * A paged key-value cache: position t of sequence b lives in page
 * block_table[b, t / page_size], slot t % page_size.  Entry (page, slot,
 * head) of layer 0 holds head_dim contiguous elements at
 *   k + page * page_stride + slot * token_stride + head * head_stride
 * (strides in elements, the same for v), so token-first and head-first pages,
 * and keys beside values in one tensor, are all described by strides.
 *
 *   dtype BF16: no scales.
 *   dtype E4M3: element = e4m3 value * scale, one fp32 scale for each (page,
 *     slot, head), at k_scale / v_scale with the scale_* strides (elements),
 *     zero or positive as spec_kv_append writes them.
 *
 * head_dim is 64, 128 or 256; page_size, num_pages, max_pages >= 1.  k and v
 * are 16-byte aligned and their strides multiples of 16 bytes
 * (SPEC_ERR_MISALIGNED otherwise).  `layers` and the layer strides matter to
 * spec_kv_compact only; the other calls work on the layer that k and v point
 * to.  `error` (nullable) is a device error word (int32, zeroed by the
 * caller; spec_verify_read_error reads and clears it).
 *
 * New positions: a call brings N positions for each of B sequences, sequence
 * b's at cache positions context_lens[b] .. context_lens[b] + n_b - 1, where
 * n_b is new_lens[b] (NULL: N).  A sequence whose lengths are negative, pass N or pass
 * max_pages * page_size, or whose table names a page outside
 * [0, num_pages) at a position the call reads or writes, sets
 * SPEC_DEVERR_CACHE_RANGE; nothing outside the cache is touched, and what
 * such a sequence gets instead is said at each call.
 * ======================================================================== */
typedef struct {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    const int32_t* block_table;          /* [B, max_pages] */
    int32_t* error;                      /* nullable */
    int64_t page_stride, token_stride, head_stride, layer_stride;
    int64_t scale_page_stride, scale_token_stride, scale_head_stride, scale_layer_stride;
    int32_t dtype;                       /* SPEC_DTYPE_BF16 or SPEC_DTYPE_E4M3 */
    int32_t layers, num_pages, page_size, max_pages, kv_heads, head_dim;
} spec_kv_cache_t;

/*
 * Prepares the new positions' queries and keys and writes keys and values
 * into the cache, in one pass:
 *   y = x * rsqrt(mean(x^2) + eps) * weight       (per head; weight NULL: y = x)
 *   y's first rot_dim elements rotated by the position's angles:
 *     (a, b) -> (a cos - b sin, b cos + a sin) with a, b = y[i], y[i + rot_dim/2]
 *     (interleaved = 0) or y[2i], y[2i+1] (interleaved = 1)
 * for queries and keys; values are stored as they are.  All in fp32, rounded
 * once: to bf16 (q_out, a BF16 cache), or to e4m3 with the row's scale
 * max(max|y|, 1e-20) / 448.
 *   q, k, v      bf16, token i = b * N + n at q + i * q_token_stride (elements; likewise
 *                k, v), heads contiguous: q_heads, kv_heads and kv_heads rows of head_dim.
 *                16-byte aligned, strides multiples of 8.  q and q_out NULL with
 *                q_heads 0: keys and values only
 *   q_weight, k_weight  [head_dim] bf16, nullable
 *   rope         [rope_rows, rot_dim] fp32: the cosines of a position's rot_dim/2 angles,
 *                then their sines; rot_dim a multiple of 16, at most head_dim (0: no rotation,
 *                rope NULL)
 *   positions    [B, N] int32: row of `rope` for each new position (NULL: its cache
 *                position); a draft tree passes context + depth
 *   q_out        [B, N, q_heads, head_dim] bf16
 * Positions n >= n_b are skipped: nothing is written for them.  For a bad
 * sequence, and for a position outside [0, rope_rows), no cache entry is
 * written and q_out is NaN.  B * N * (q_heads + 2 kv_heads) < 2^31.
 */
spec_status_t spec_kv_append(const spec_kv_cache_t* cache, const void* q, const void* k,
                             const void* v, int64_t q_token_stride, int64_t k_token_stride,
                             int64_t v_token_stride, const void* q_weight, const void* k_weight,
                             float eps, const float* rope, int rope_rows, int rot_dim,
                             int interleaved, const int32_t* context_lens,
                             const int32_t* new_lens, const int32_t* positions, int B, int N,
                             int q_heads, void* q_out, cudaStream_t stream);

/*
 * Reads cached positions back as dense rows: out_k, out_v [B, T, kv_heads,
 * head_dim] of out_dtype (BF16 or F32), row t of sequence b holding position
 * starts[b] + t (NULL: t) for t < counts[b] (NULL: T), zeros for the other
 * rows.  E4M3 entries are multiplied by their scale in fp32 and rounded once.
 * A bad sequence's rows are NaN, and so is the row of a bad page.
 * T * kv_heads < 2^31, B <= 65535.
 */
spec_status_t spec_kv_read(const spec_kv_cache_t* cache, const int32_t* starts,
                           const int32_t* counts, int B, int T, spec_dtype_t out_dtype,
                           void* out_k, void* out_v, cudaStream_t stream);

/*
 * Moves the accepted path of a draft tree to the front of its slots, in every
 * layer of the cache: entry context_lens[b] + path_nodes[b, i] goes to
 * context_lens[b] + i + 1 for i < num_accepted[b].  path_nodes [B, N] and
 * num_accepted [B] are spec_verify_tree_greedy's outputs (node n of the tree
 * was appended at position context + n; the root stays where it is), so node
 * ids ascend along the path.  After it the first context_lens[b] + 1 +
 * num_accepted[b] positions are the verified context.  Entries are moved as
 * they are (scales with them); keys were rotated for the node's depth, which
 * is its new distance from the root.  A sequence with num_accepted -1 is
 * skipped; a path that is not ascending in 1..N-1, or that is longer than
 * N-1, sets SPEC_DEVERR_CACHE_RANGE and moves nothing.  1 <= N <= 1024,
 * B <= 65535.
 */
spec_status_t spec_kv_compact(const spec_kv_cache_t* cache, const int32_t* context_lens,
                              const int32_t* path_nodes, const int32_t* num_accepted, int B,
                              int N, cudaStream_t stream);

/*
 * Attention of the new positions over the cache, which already holds them
 * (spec_kv_append): for query head h of position n, with cached head
 * h / (q_heads / kv_heads),
 *   s_t = scale * q . k_t,   out = sum_t softmax(s)_t v_t,   lse = ln sum_t e^(s_t)
 * over the positions t that n sees: every t < context_lens[b], and of the new
 * ones
 *   parents NULL: those up to itself (a chain, N <= 257);
 *   parents [B, N] int32: itself and its ancestors (a tree, N <= 64, while
 *     spec_verify_tree_greedy and spec_kv_compact take 1024;
 *     parents[0] = -1, 0 <= parents[n] < n as there).
 *   q      [B, N, q_heads, head_dim] bf16, token i at q + i * q_token_stride (elements,
 *          a multiple of 8), heads contiguous; 16-byte aligned
 *   out    [B, N, q_heads, head_dim] bf16, contiguous
 *   lse    [B, N, q_heads] fp32, nullable
 * q_heads is a multiple of kv_heads, at most 64 times it, B * N * q_heads
 * < 2^31.  Scores, softmax statistics and sums are fp32.  Before they meet the
 * values, probabilities are rounded: to bf16 with a BF16 cache (against 64 bits
 * that is 2.3e-3 of the result beside 1.7e-3 from its own rounding), to fp16
 * with an E4M3 one (a probability times its position's value scale, the row's
 * largest such product at least 1).  lse knows nothing of that.  Positions n >= n_b give out = 0 and lse =
 * -inf.  The others of a bad sequence (or of a malformed tree,
 * SPEC_DEVERR_TREE_PARENT) give NaN, and where the lengths themselves are bad
 * all N do.  What the masked entries of the cache hold does not matter, NaN and
 * infinities included.
 *
 * Workspace: spec_attention_workspace_size() bytes, 256-byte aligned, of any
 * contents.  Nothing is carried between calls, so calls of any size may use
 * one in turn, but not at the same time.
 */
size_t spec_attention_workspace_size(int B, int N, int q_heads, int kv_heads, int head_dim);
spec_status_t spec_paged_attention(const spec_kv_cache_t* cache, const void* q,
                                   int64_t q_token_stride, const int32_t* context_lens,
                                   const int32_t* new_lens, const int32_t* parents, float scale,
                                   int B, int N, int q_heads, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Log-probabilities of given tokens with the distribution's entropy and its
 * top alternatives, p = softmax(z / T) over each of `rows` rows of V logits:
 *   out_logprob [rows]          ln p(tokens[r])
 *   out_entropy [rows]          -sum p ln p (nats), nullable
 *   out_top_idx [rows, K]       the K largest logits' tokens (larger first, lower index
 *                               first among equal logits, -0.0 equal to +0.0)
 *   out_top_logprob [rows, K]   their ln p
 * 1 <= V <= 8388608, 0 <= K <= 8 (K = 0: no lists, both may be NULL); with V < K the lists are
 * padded with -1 and -inf.  A masked (-inf) logit has ln p = -inf and adds
 * nothing to the entropy.  A token outside [0, V) gives ln p = NaN and sets
 * SPEC_DEVERR_TOKEN_RANGE; a row of -inf alone gives NaN everywhere (list
 * tokens -1) and sets SPEC_DEVERR_EMPTY_ROW, and so does, with SPEC_DEVERR_TIMEOUT, a row
 * of which a wait that ran out has left something unread.  Sums are fp32.  Logits are
 * 16-byte aligned; V and its row length need no alignment.  Workspace:
 * spec_logprobs_workspace_size(rows, V, K) bytes, 256-byte aligned, its first
 * 256 bytes zero-filled once (the error word).
 */
size_t spec_logprobs_workspace_size(int rows, int V, int K);
spec_status_t spec_token_logprobs(const void* logits, spec_dtype_t dtype, const int32_t* tokens,
                                  float temperature, int rows, int V, int K, float* out_logprob,
                                  float* out_entropy, int32_t* out_top_idx,
                                  float* out_top_logprob, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream);

/* ==========================================================================
 * The dense side of the target model's pass: what lies between its cache and
 * attention calls, with weights and rows in 8 bits.  (The source pages leave it
 * to the model, as they do the calls above.)
 *
 * 8-bit values are e4m3 with fp32 scales, one for each block of 128 elements
 * of a row (the last block of a row may be shorter), or for each 128 x 128 elements
 * of a weight:
 *   t = max(max |y| over the block, 1e-20),  q = e4m3(y * (448 / t)),  scale = t / 448,
 * and an element stands for q * scale.  A NaN stays one; the largest element is taken
 * over the others.  A block with an infinity has scale infinity: its infinities are NaN,
 * its other elements 0 times infinity.
 *   rows:    scale of block b of row r at b * scale_stride + r: a block's scales of
 *            neighbouring rows lie side by side, as the product reads them
 *   weights: scale of block (i, b) (rows 128 i on, elements 128 b on) at
 *            i * scale_stride + b
 *
 * Rows of x, gate, up and the residual: row r at r * stride elements, 16-byte
 * aligned, strides multiples of 16 bytes (SPEC_ERR_MISALIGNED otherwise; 0 for one row
 * that all share), bf16 or fp32.  Outputs `out`: contiguous rows of dim elements, bf16, fp32 or e4m3 (then
 * out_scale is needed, with scale_stride >= rows; 0 may stand there for rows of one block).  dim is a
 * multiple of 8, of 16 for an e4m3 output.  rows * (dim rounded up to 128) < 2^34.  Arithmetic is fp32,
 * each output rounded once.  An output may not overlap an input except as said.
 * ======================================================================== */

/*
 * The residual's addition and the root-mean-square norm of its sum:
 *   h = x + residual (NULL: h = x),   sum_out = h in sum_dtype (nullable),
 *   out = h * rsqrt(mean(h^2) + eps) * weight      (h before its rounding; weight NULL: 1)
 *   residual, sum_out  of sum_dtype, strides of their own, sum_out's at least dim; sum_out may be
 *                      the residual, or x of that type, itself (same stride): the residual
 *                      stream in place
 *   weight             [dim] bf16, 16-byte aligned, nullable
 */
spec_status_t spec_add_norm(const void* x, spec_dtype_t x_dtype, int64_t x_stride,
                            const void* residual, spec_dtype_t sum_dtype,
                            int64_t residual_stride, const void* weight, float eps, int rows,
                            int dim, void* sum_out, int64_t sum_stride, void* out,
                            spec_dtype_t out_dtype, float* out_scale, int64_t scale_stride,
                            cudaStream_t stream);

/*
 * out = act(gate) * up:
 *   SPEC_ACT_SILU        x / (1 + e^-x)
 *   SPEC_ACT_GELU_TANH   x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2
 * gate and up have one dtype; halves of one projection's rows are passed with its stride.
 */
typedef enum { SPEC_ACT_SILU = 0, SPEC_ACT_GELU_TANH = 1 } spec_act_t;
spec_status_t spec_gated_act(const void* gate, const void* up, spec_dtype_t dtype,
                             int64_t gate_stride, int64_t up_stride, spec_act_t act, int rows,
                             int dim, void* out, spec_dtype_t out_dtype, float* out_scale,
                             int64_t scale_stride, cudaStream_t stream);

/*
 * Rounds rows (block_rows 1) or a weight (block_rows 128) to 8 bits; scales as above
 * (a weight's scale_stride is at least the number of a row's blocks; 0 may stand there for up to
 * 128 rows).
 */
spec_status_t spec_quantize_e4m3(const void* x, spec_dtype_t dtype, int64_t x_stride, int rows,
                                 int dim, int block_rows, void* out, float* out_scale,
                                 int64_t scale_stride, cudaStream_t stream);

/*
 * The product of 8-bit rows with an 8-bit weight:
 *   out[m, n] = sum over blocks b of  x_scale[m, b] w_scale[n / 128, b]
 *                                     sum over k in b of x[m, k] w[n, k]
 *   x        [M, K] e4m3, w [N, K] e4m3: 16-byte aligned, strides multiples of 16 and at least K
 *            (of a single row none is used)
 *   x_scale  fp32, block b of row m at b * x_scale_stride + m, the stride at least M (of a single
 *            block none is used).  What lies between M and the stride does not matter.  For 2 to 64
 *            rows 16-byte aligned and the stride a multiple of 4; for one row (the last of a prompt,
 *            say) and for more than 64 neither is needed
 *   w_scale  fp32, at (n / 128) * w_scale_stride + b
 *   out      [M, N] bf16 or fp32, row m at m * out_stride (elements, at least N)
 * Any M, N >= 0 and K >= 1, odd ones included; rows whose stride is a multiple of 16 bytes are
 * written fastest.  Sums are fp32: of a block's products in tensor memory, then, scaled,
 * over the blocks, in an order that the sizes and the device decide (its SMs, and the clusters that it
 * holds at once): the same call on the same device gives the same bits.
 * Workspace: spec_matmul_workspace_size() bytes, 256-byte aligned, its first 256 bytes
 * zero-filled once (the error word; a wait that runs out sets SPEC_DEVERR_TIMEOUT there and
 * leaves NaN in the results it concerns).  Calls that share one must not overlap.
 */
size_t spec_matmul_workspace_size(int M, int N, int K);
spec_status_t spec_matmul_e4m3(const void* x, int64_t x_stride, const float* x_scale,
                               int64_t x_scale_stride, const void* w, int64_t w_stride,
                               const float* w_scale, int64_t w_scale_stride, int M, int N, int K,
                               void* out, spec_dtype_t out_dtype, int64_t out_stride,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * How spec_matmul_e4m3 divides a product of these sizes among the SMs: five numbers to plan[],
 *   [0]  the way: one of spec_matmul_way_t
 *   [1]  weight rows of a tile
 *   [2]  CTAs that take a tile (of one contraction) together: 1, or 2 (a pair)
 *   [3]  CTAs or pairs that are launched (few rows: 0)
 *   [4]  parts of a tile's contraction: 1, those of a cluster, or the most that equal shares leave in
 *        a tile (few rows: 0)
 * sms 0: on the current device.  Else on one of `sms` SMs (two at least), of which clusters[0], [1] and [2] clusters of
 * two, four and eight CTAs run at once; host only then, no CUDA call.
 */
typedef enum {
    SPEC_MATMUL_FEW = 0,          /* up to 64 rows: the product transposed */
    SPEC_MATMUL_WHOLE = 1,        /* whole tiles in turn */
    SPEC_MATMUL_CLUSTERS = 2,     /* a cluster's CTAs or pairs share a tile's contraction */
    SPEC_MATMUL_SHARES = 3        /* equal shares of all tiles, joined through the workspace */
} spec_matmul_way_t;
spec_status_t spec_matmul_plan(int M, int N, int K, int sms, const int32_t* clusters, int32_t* plan);

/*
 * Test hook for the kernels' bounded waits (the source pages have no
 * counterpart).  Every wait of the streaming kernels on a shared-memory
 * barrier of their bulk-copy ring gives up after a number of polls (seconds of
 * wall time by default: spec_verify_default_wait_limit()), sets
 * SPEC_DEVERR_TIMEOUT in the workspace error word and lets the kernel return
 * instead of hanging.  spec_verify_set_wait_limit sets that number for every
 * launch made afterwards in the process, from any thread; 0 makes such waits
 * give up without polling, so a test can drive the timeout path without
 * breaking a kernel.  Results of a call whose wait gave up are not valid; the
 * workspace stays usable for later calls.  A kernel's final wait for its own
 * bulk copies in flight always keeps the default bound.  Host only; set it
 * back to the default after the test.
 */
void spec_verify_set_wait_limit(uint32_t polls);
uint32_t spec_verify_default_wait_limit(void);

/*
 * Synchronises `stream`, returns the accumulated SPEC_DEVERR_* bits of the
 * workspace in *code and clears them.  SPEC_OK when the read succeeded (code
 * may still be nonzero).
 */
spec_status_t spec_verify_read_error(void* workspace, cudaStream_t stream, int32_t* code);

/* Static description of a status code. */
const char* spec_verify_status_string(spec_status_t status);

#ifdef __cplusplus
}
#endif
#endif /* SPEC_VERIFY_H */
