// The paged cache's own calls: appending new positions (head norms, rotation
// and quantisation in the same pass), reading positions back, and moving a
// draft tree's accepted path.  All three move each byte once and compute
// little: memory bounds them when they are large (the read; an append long before
// that its instructions), the launch when small.
#include "sv_kv.cuh"

namespace sv {

constexpr int kKvThreads = 256;

// ---- append -------------------------------------------------------------------
// One row (a token's query, key or value head) per D / 8 lanes, 8 elements a
// lane: 16-byte loads, the norm's sum and the row's largest magnitude by
// shuffles among those lanes.  A half-split rotation pairs element i with
// i + rot/2, which another lane holds at the same offset (rot is a multiple
// of 16), so it takes one shuffle per element; an interleaved one pairs a
// lane's own neighbours.
// 512 positions of 48 heads of 128 to an E4M3 cache (11.6 MB): 7.2 us, 1.6 TB/s, of which
// the rotation is 1.4, the norms 0.7 and the launch with its dependent loads (length,
// table entry) over two: a lane has some 200 instructions for its 16 bytes.  Blocks of
// 128 and row arithmetic in 32 bits took it there from 7.5; eight blocks of 256 an SM
// (32 registers) took 7.9.  One position: 2.3.
constexpr int kAppendThreads = 128;

template <int D, bool FP8>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
    pdl_trigger();
    pdl_wait();
    constexpr int L = D / 8;                                  // lanes per row
    const unsigned heads = a.Hq + 2 * a.c.kv_heads;
    const unsigned rows = (unsigned)a.B * a.N * heads;        // below 2^31
    const unsigned r = blockIdx.x * (kAppendThreads / L) + threadIdx.x / L;
    const bool live = r < rows;                               // a row's lanes agree; idle rows keep the shuffles whole
    const int lr = threadIdx.x % L;
    const int tok = live ? (int)(r / heads) : 0;
    const int h = live ? (int)(r - tok * heads) : 0;
    const int b = tok / a.N, n = tok - b * a.N;
    const int kind = h < a.Hq ? 0 : h < a.Hq + a.c.kv_heads ? 1 : 2;   // query, key, value
    const int head = kind == 0 ? h : kind == 1 ? h - a.Hq : h - a.Hq - a.c.kv_heads;

    const int ctx = __ldg(a.ctx + b);
    const int nb = a.newl ? __ldg(a.newl + b) : a.N;
    const char* src = kind == 0 ? a.q + tok * a.qs : kind == 1 ? a.k + tok * a.ks : a.v + tok * a.vs;
    float x[8];
    unpack8(ld_stream16(src + ((size_t)head * D + lr * 8) * 2), x);

    const int cap = a.c.max_pages * a.c.page_size;
    bool bad = ctx < 0 || nb < 0 || nb > a.N || ctx > cap - nb;
    const bool skip = !live || (!bad && n >= nb);
    const int t = bad ? 0 : ctx + n;
    int rp = t;
    if (a.rot > 0 && !bad && !skip) {
        if (a.pos) rp = __ldg(a.pos + tok);
        if ((unsigned)rp >= (unsigned)a.rope_rows) bad = true;
    }
    int page = 0, slot = 0;
    if (!bad && !skip && !cache_place(a.c, b, t, &page, &slot)) bad = true;

    const char* wsrc = kind == 0 ? a.qw : kind == 1 ? a.kw : nullptr;
    if (a.qw || a.kw) {                                       // every lane takes part in the shuffles
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (wsrc) {
            float w[8];
            unpack8(__ldg(reinterpret_cast<const uint4*>(wsrc) + lr), w);
            const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
        }
    }
    if (a.rot > 0) {                                          // and in these
        const int half = a.rot >> 1;
        const bool turn = kind < 2 && lr * 8 < a.rot && !bad && !skip;
        const float* cs = a.rope + (size_t)(turn ? rp : 0) * a.rot;
        if (a.inter) {
            if (turn) {
                const float4 co = __ldg(reinterpret_cast<const float4*>(cs + lr * 4));
                const float4 si = __ldg(reinterpret_cast<const float4*>(cs + half + lr * 4));
                const float c4[4] = {co.x, co.y, co.z, co.w}, s4[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = x[2 * i], q = x[2 * i + 1];
                    x[2 * i] = p * c4[i] - q * s4[i];
                    x[2 * i + 1] = q * c4[i] + p * s4[i];
                }
            }
        } else {
            const bool upper = lr * 8 >= half;
            const int step = half >> 3;                       // lanes between the halves
            const int base = (threadIdx.x & 31) - lr;
            const int other = lr * 8 < a.rot ? base + (upper ? lr - step : lr + step) : (threadIdx.x & 31);
            const int i0 = turn ? (upper ? lr * 8 - half : lr * 8) : 0;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float4 co = __ldg(reinterpret_cast<const float4*>(cs + i0) + v);
                const float4 si = __ldg(reinterpret_cast<const float4*>(cs + half + i0) + v);
                const float c4[4] = {co.x, co.y, co.z, co.w}, s4[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y = __shfl_sync(0xffffffffu, x[4 * v + i], other);
                    if (turn) x[4 * v + i] = upper ? x[4 * v + i] * c4[i] + y * s4[i] : x[4 * v + i] * c4[i] - y * s4[i];
                }
            }
        }
    }
    if (kind == 0) {
        if (skip) return;
        uint4 o;
        if (bad) {
            o = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
            if (lr == 0 && head == 0) raise_error(a.c.error, SPEC_DEVERR_CACHE_RANGE);
        } else {
            o = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        }
        *reinterpret_cast<uint4*>(a.q_out + (((size_t)tok * a.Hq + head) * D + lr * 8) * 2) = o;
        return;
    }
    if constexpr (!FP8) {
        if (skip) return;
        if (bad) {
            if (lr == 0) raise_error(a.c.error, SPEC_DEVERR_CACHE_RANGE);
            return;
        }
        char* dst = static_cast<char*>(kind == 1 ? a.c.k : a.c.v) + 2 * entry_off(a.c, page, slot, head);
        *reinterpret_cast<uint4*>(dst + lr * 16) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
        if (bad && !skip && lr == 0) raise_error(a.c.error, SPEC_DEVERR_CACHE_RANGE);
        if (bad || skip) return;
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
        const unsigned mask = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1u) << ((threadIdx.x & 31) / L * L);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
        // the nearest e4m3 of y / scale: a true division, so that the row's
        // largest element always lands on 448
        const float sc = fmaxf(m, kFp8AmaxFloor) / kFp8Max;
        uint2 o;
        o.x = pack_e4m3(x[0] / sc, x[1] / sc) | pack_e4m3(x[2] / sc, x[3] / sc) << 16;
        o.y = pack_e4m3(x[4] / sc, x[5] / sc) | pack_e4m3(x[6] / sc, x[7] / sc) << 16;
        char* dst = static_cast<char*>(kind == 1 ? a.c.k : a.c.v) + entry_off(a.c, page, slot, head);
        *reinterpret_cast<uint2*>(dst + lr * 8) = o;
        if (lr == 0) (kind == 1 ? a.c.k_scale : a.c.v_scale)[scale_off(a.c, page, slot, head)] = sc;
    }
}

template <int D>
static cudaError_t launch_append_t(const AppendArgs& a, cudaStream_t st) {
    const long long rows = (long long)a.B * a.N * (a.Hq + 2 * a.c.kv_heads);
    const dim3 grid((unsigned)((rows * (D / 8) + kAppendThreads - 1) / kAppendThreads));
    return a.c.dtype == SPEC_DTYPE_E4M3 ? launch_pdl(append_kernel<D, true>, grid, kAppendThreads, 0, st, a)
                                        : launch_pdl(append_kernel<D, false>, grid, kAppendThreads, 0, st, a);
}

cudaError_t launch_append(const AppendArgs& a, cudaStream_t st) {
    return a.c.head_dim == 64 ? launch_append_t<64>(a, st) : a.c.head_dim == 128 ? launch_append_t<128>(a, st)
                                                                                 : launch_append_t<256>(a, st);
}

// ---- read ---------------------------------------------------------------------
struct ReadArgs {
    spec_kv_cache_t c;
    const int32_t *starts, *counts;
    int T;
    char *out_k, *out_v;
};

// A lane takes the same 8 elements of a position's key and of its value, and
// kReadRows rows (position, head) that lie a CTA's width apart, so that its
// loads are all in flight before the first store and the index arithmetic is
// shared.  blockIdx.y is the sequence; the rows run along x.  Outputs are
// stored as data that is not read again soon.  64 x 2048 positions of 8 e4m3
// heads of 128 as bf16 (0.75 GB): 112 us, 6.65 TB/s, 98 % of a plain copy's
// rate; one row a lane with 64-bit divisions took 127 us, and 16 elements a
// lane (whose two 16-byte stores fill half sectors) 130 us.
constexpr int kReadRows = 2;

template <int D, bool FP8, bool F32>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const ReadArgs a) {
    pdl_trigger();
    pdl_wait();
    constexpr int E = 8, L = D / E, R = kKvThreads / L;       // elements of a lane, lanes of a row, rows abreast
    const int H = a.c.kv_heads, lr = threadIdx.x % L, b = blockIdx.y;
    const unsigned rows = (unsigned)a.T * H, row0 = blockIdx.x * (R * kReadRows) + threadIdx.x / L;
    const int start = a.starts ? __ldg(a.starts + b) : 0;
    const int count = a.counts ? __ldg(a.counts + b) : a.T;
    const bool off = start < 0 || count < 0 || count > a.T || start > a.c.max_pages * a.c.page_size - count;
    uint4 wk[kReadRows], wv[kReadRows];
    float sk[kReadRows], sv_[kReadRows];
    bool bad[kReadRows];
#pragma unroll
    for (int u = 0; u < kReadRows; ++u) {
        const unsigned row = row0 + u * R;
        const int t = (int)(row / (unsigned)H), head = (int)(row - (unsigned)t * H);
        wk[u] = wv[u] = make_uint4(0, 0, 0, 0);
        sk[u] = sv_[u] = 0.f;
        bad[u] = off;
        if (row >= rows || off || t >= count) continue;
        int page, slot;
        if (!cache_place(a.c, b, start + t, &page, &slot)) {
            bad[u] = true;
            continue;
        }
        const int64_t at = (entry_off(a.c, page, slot, head) + lr * E) * (FP8 ? 1 : 2);
        if constexpr (!FP8) {
            wk[u] = ld_stream16(static_cast<const char*>(a.c.k) + at);
            wv[u] = ld_stream16(static_cast<const char*>(a.c.v) + at);
        } else {
            const uint2 k2 = __ldcs(reinterpret_cast<const uint2*>(static_cast<const char*>(a.c.k) + at));
            const uint2 v2 = __ldcs(reinterpret_cast<const uint2*>(static_cast<const char*>(a.c.v) + at));
            wk[u].x = k2.x; wk[u].y = k2.y;
            wv[u].x = v2.x; wv[u].y = v2.y;
            const int64_t so = scale_off(a.c, page, slot, head);
            sk[u] = __ldg(a.c.k_scale + so);
            sv_[u] = __ldg(a.c.v_scale + so);
        }
    }
#pragma unroll
    for (int u = 0; u < kReadRows; ++u) {
        const unsigned row = row0 + u * R;
        if (row >= rows) return;
        if (bad[u] && lr == 0) raise_error(a.c.error, SPEC_DEVERR_CACHE_RANGE);
        const size_t o = ((size_t)b * rows + row) * D + lr * E;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint4 w = kv ? wv[u] : wk[u];
            char* out = (kv ? a.out_v : a.out_k) + o * (F32 ? 4 : 2);
            float x[E];
            if constexpr (FP8) {
#pragma unroll
                for (int j = 0; j < E / 2; ++j)
                    f16x2_to_f32(e4m3_to_f16x2(u4_get(w, j / 2) >> 16 * (j & 1)), &x[2 * j], &x[2 * j + 1]);
                const float sc = kv ? sv_[u] : sk[u];
#pragma unroll
                for (int j = 0; j < E; ++j) x[j] *= sc;
            } else {
                unpack8(w, x);
            }
            if (bad[u]) {
#pragma unroll
                for (int j = 0; j < E; ++j) x[j] = CUDART_NAN_F;
            }
            if constexpr (F32) {
#pragma unroll
                for (int j = 0; j < E / 4; ++j)
                    __stcs(reinterpret_cast<float4*>(out) + j, make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]));
            } else {
#pragma unroll
                for (int j = 0; j < E / 8; ++j)
                    __stcs(reinterpret_cast<uint4*>(out) + j,
                           make_uint4(pack_bf16(x[8 * j], x[8 * j + 1]), pack_bf16(x[8 * j + 2], x[8 * j + 3]),
                                      pack_bf16(x[8 * j + 4], x[8 * j + 5]), pack_bf16(x[8 * j + 6], x[8 * j + 7])));
            }
        }
    }
}

template <int D>
static cudaError_t launch_read_t(const ReadArgs& a, int B, bool f32, cudaStream_t st) {
    const bool fp8 = a.c.dtype == SPEC_DTYPE_E4M3;
    const long long per = kKvThreads / (D / 8) * kReadRows;
    const dim3 grid((unsigned)(((long long)a.T * a.c.kv_heads + per - 1) / per), (unsigned)B);
    if (fp8)
        return f32 ? launch_pdl(kv_read_kernel<D, true, true>, grid, kKvThreads, 0, st, a)
                   : launch_pdl(kv_read_kernel<D, true, false>, grid, kKvThreads, 0, st, a);
    return f32 ? launch_pdl(kv_read_kernel<D, false, true>, grid, kKvThreads, 0, st, a)
               : launch_pdl(kv_read_kernel<D, false, false>, grid, kKvThreads, 0, st, a);
}

cudaError_t launch_kv_read(const spec_kv_cache_t& c, const int32_t* starts, const int32_t* counts, int B, int T,
                           bool f32, void* out_k, void* out_v, cudaStream_t st) {
    const ReadArgs a{c, starts, counts, T, static_cast<char*>(out_k), static_cast<char*>(out_v)};
    return c.head_dim == 64 ? launch_read_t<64>(a, B, f32, st) : c.head_dim == 128 ? launch_read_t<128>(a, B, f32, st)
                                                                                   : launch_read_t<256>(a, B, f32, st);
}

// ---- compact ------------------------------------------------------------------
struct CompactArgs {
    spec_kv_cache_t c;
    const int32_t *ctx, *path, *acc;
    int N;
    unsigned cpr;                  // 16-byte chunks of a cache row
    unsigned cols;                 // columns of the cache: layers x {k, v} x heads x cpr
    unsigned scale_cols;           // layers x {k, v} x heads (E4M3)
};

// A path's ids ascend from at least 1, so node i of the path (from 1) lies
// at slot >= i, and slot i is never a later node's: a thread that owns one
// column (layer, k or v, head, 16 bytes) of every slot moves it along the path in
// order, and no two threads touch the same bytes.  blockIdx.y is the
// sequence; the CTA first lists the moves (source and destination offsets),
// which are the same for every column.
// 32 paths of a 36-node tree in 36 layers of 8 heads of 128 bf16 (9.4 MB): 3.7 us, 2.6
// TB/s; one path in 4 layers: 2.4.  The launch and three loads one after the other
// (path, table, entries) bound both.
__global__ void __launch_bounds__(kKvThreads) kv_compact_kernel(const CompactArgs a) {
    extern __shared__ int64_t moves[];                        // per move: source, destination, scales' two
    __shared__ int n_moves, bad;
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.y;
    const int acc = __ldg(a.acc + b), ctx = __ldg(a.ctx + b);
    if (acc == -1) return;
    const int cap = a.c.max_pages * a.c.page_size;
    const bool off = acc < 0 || acc >= a.N || ctx < 0 || ctx > cap - 1 - acc;
    if (threadIdx.x == 0) {
        n_moves = 0;
        bad = off;
    }
    __syncthreads();
    const int32_t* path = a.path + (size_t)b * a.N;
    int first = 0;
    if (!off) {                                               // CTA-uniform
        // the path's form, and how many of its first ids are in place already
        // (ids ascend, so after the first that is not none is)
        bool wrong = false;
        int here = 0;
        for (int i = threadIdx.x; i < acc; i += kKvThreads) {
            const int p = __ldg(path + i), before = i ? __ldg(path + i - 1) : 0;
            wrong |= p <= before || p >= a.N;
            here += p == i + 1;
        }
        if (wrong) bad = 1;
        if (here) atomicAdd(&n_moves, here);
        __syncthreads();
        first = min(n_moves, acc);
        for (int i = first + threadIdx.x; i < acc; i += kKvThreads) {
            int sp, ss, dp, ds;
            if (!cache_place(a.c, b, ctx + __ldg(path + i), &sp, &ss) ||
                !cache_place(a.c, b, ctx + i + 1, &dp, &ds)) {
                bad = 1;
                continue;
            }
            int64_t* m = moves + 4 * (i - first);
            m[0] = entry_off(a.c, sp, ss, 0);
            m[1] = entry_off(a.c, dp, ds, 0);
            m[2] = scale_off(a.c, sp, ss, 0);
            m[3] = scale_off(a.c, dp, ds, 0);
        }
    }
    __syncthreads();
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.x == 0) raise_error(a.c.error, SPEC_DEVERR_CACHE_RANGE);
        return;
    }
    const int n = acc - first;
    if (n == 0) return;
    const int elt = a.c.dtype == SPEC_DTYPE_E4M3 ? 1 : 2;
    const unsigned step = gridDim.x * kKvThreads, H = a.c.kv_heads;
    for (unsigned i = blockIdx.x * kKvThreads + threadIdx.x; i < a.cols; i += step) {
        const unsigned r = i / a.cpr, chunk = i - r * a.cpr, lk = r / H, head = r - lk * H;
        char* base = static_cast<char*>(lk & 1 ? a.c.v : a.c.k) +
                     ((int64_t)(lk >> 1) * a.c.layer_stride + head * a.c.head_stride) * elt + chunk * 16;
        for (int j = 0; j < n; ++j)
            *reinterpret_cast<uint4*>(base + moves[4 * j + 1] * elt) =
                *reinterpret_cast<const uint4*>(base + moves[4 * j] * elt);
    }
    for (unsigned i = blockIdx.x * kKvThreads + threadIdx.x; i < a.scale_cols; i += step) {
        const unsigned lk = i / H, head = i - lk * H;
        float* base = (lk & 1 ? a.c.v_scale : a.c.k_scale) + (int64_t)(lk >> 1) * a.c.scale_layer_stride +
                      head * a.c.scale_head_stride;
        for (int j = 0; j < n; ++j) base[moves[4 * j + 3]] = base[moves[4 * j + 2]];
    }
}

cudaError_t launch_kv_compact(const spec_kv_cache_t& c, const int32_t* ctx, const int32_t* path,
                              const int32_t* acc, int B, int N, cudaStream_t st) {
    CompactArgs a{c, ctx, path, acc, N, 0, 0, 0};
    const bool fp8 = c.dtype == SPEC_DTYPE_E4M3;
    a.cpr = c.head_dim * (fp8 ? 1 : 2) / 16;
    a.cols = (unsigned)c.layers * 2 * c.kv_heads * a.cpr;     // (checked below 2^31)
    a.scale_cols = fp8 ? (unsigned)c.layers * 2 * c.kv_heads : 0;
    long long g = ((long long)a.cols + kKvThreads - 1) / kKvThreads;
    if (g > 1024) g = 1024;
    const size_t smem = (size_t)N * 4 * sizeof(int64_t);      // at most 32 KB
    return launch_pdl(kv_compact_kernel, dim3((unsigned)g, (unsigned)B), kKvThreads, smem, st, a);
}

}  // namespace sv
