// What the attention kernels share: asynchronous copies, the split of the work
// among CTAs, and the join of a split unit's parts.
#pragma once

#include "sv_kv.cuh"

namespace sv {

constexpr int kAttMaxCtas = 512;            // the workspace is sized for this many
// What the join of the parts (attend_join_kernel) knows of the unit that CTA c
// begins and others end: at the head of the workspace, one for each CTA.
struct __align__(16) AttSplit {
    int parts;               // CTAs c .. c + parts - 1 hold one each; 0: no such unit
    int b, hk, r0;           // sequence, cached head, first row of the block
    int rows, nb;            // rows of the block, new positions of the sequence
    int unused[2];
};
constexpr size_t kAttHead = kAttMaxCtas * sizeof(AttSplit);
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The reference m of a row moves only when a score passes it by more than
// this (in powers of two): probabilities stay below 2^8 (E4M3 in sv_attend.cu:
// 2^(kFp16Head + 8)), and the sums are rarely rescaled.
constexpr float kRefSlack = 8.f;

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The lengths of one sequence; bad ones read as empty.
struct SeqLen {
    int ctx, total;          // cached before the call, and with the new positions
    int nb;
    bool bad;
};
__device__ __forceinline__ SeqLen seq_len(const AttendArgs& a, int b) {
    SeqLen s;
    s.ctx = __ldg(a.ctx + b);
    s.nb = a.newl ? __ldg(a.newl + b) : a.N;
    s.bad = s.ctx < 0 || s.nb < 0 || s.nb > a.N || s.ctx > a.c.max_pages * a.c.page_size - s.nb;
    s.total = s.bad || s.nb == 0 ? 0 : s.ctx + s.nb;
    return s;
}

// The new position of row R of a cached head, R / G.
__device__ __forceinline__ int row_position(const AttendArgs& a, int R) {
    return a.G == 1 ? R : (int)__umulhi((uint32_t)R, a.g_mul);
}
// The page index and slot of a position.
__device__ __forceinline__ int page_index(const AttendArgs& a, int pos, int* slot) {
    const int pg = a.page_shift >= 0 ? pos >> a.page_shift : pos / a.c.page_size;
    *slot = pos - pg * a.c.page_size;
    return pg;
}

// a / b, in 32 bits where both fit (a 64-bit division takes some hundred
// cycles, and these stand before a CTA's first load).
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
// The scale of an E4M3 position's values as a factor of its probability: not
// below any that spec_kv_append writes, so that a scale of zero (values of
// zero) leaves the position its weight.
__device__ __forceinline__ float value_scale(float s) { return s < 1e-23f ? 1e-23f : s; }

// Share i of `total` tiles among n CTAs begins at tile i * total / n.
__device__ __forceinline__ long long share_begin(long long total, long long n, long long i) { return quotient(i * total, n); }
// The CTA whose share holds tile t.
__device__ __forceinline__ int share_of(long long total, long long n, long long t) {
    return (int)quotient((t + 1) * n - 1, total);
}

// Floats of one part of a split unit: rows sums of D, then the rows' references
// and totals; a multiple of 16 bytes, as the parts are read and written in
// 16-byte pieces.
__host__ __device__ constexpr size_t part_floats(int rows, int D) { return (size_t)rows * D + (2 * rows + 3) / 4 * 4; }

struct AttPlan {
    int n;                   // CTAs that take part
    long long total;         // tiles of all units (or units, where they are dealt whole)
    int b;                   // sequence of this CTA's first tile
    long long at;            // that sequence's first tile
};

// Sums the tiles of all sequences and finds the sequence of this CTA's first
// tile.  Every thread takes a run of sequences.
template <int TILE, int THREADS>
__device__ __forceinline__ void make_plan(const AttendArgs& a, int units, int grid, AttPlan* out) {
    __shared__ long long sums[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (a.B + THREADS - 1) / THREADS;
    const int b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += a.whole ? 1 : max(1, (seq_len(a, b).total + TILE - 1) / TILE);
    mine *= units;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    const int n = (int)min((long long)grid, total);
    long long at = before + incl - mine;
    const long long first = blockIdx.x < n ? share_begin(total, n, blockIdx.x) : -1;
    if (first >= at && first < at + mine) {
        for (int b = b0; b < b1; ++b) {
            const long long t = (long long)units * (a.whole ? 1 : max(1, (seq_len(a, b).total + TILE - 1) / TILE));
            if (first < at + t) {
                out->b = b;
                out->at = at;
                break;
            }
            at += t;
        }
    }
    if (threadIdx.x == 0) {
        out->n = n;
        out->total = total;
    }
    __syncthreads();
}

// A unit: one row block of one cached head of one sequence, of which the CTA
// has tiles ta .. tb - 1.
struct AttUnit {
    int b, u;                // sequence, unit of the sequence
    int tiles, ta, tb;
    int hk, r0, rows;        // cached head, first row and number of rows
    long long at;            // its first tile among all
    SeqLen sl;
};

// Walks a CTA's share unit by unit.
struct AttWalk {
    long long t, end, seq_at;
    int b;

    __device__ __forceinline__ void init(const AttPlan& p) {
        t = share_begin(p.total, p.n, blockIdx.x);
        end = share_begin(p.total, p.n, blockIdx.x + 1);
        seq_at = p.at;
        b = p.b;
    }
    // The next unit; false at the share's end.
    template <int TILE>
    __device__ __forceinline__ bool next(const AttendArgs& a, int RB, int block_rows, AttUnit* x) {
        const int units = a.c.kv_heads * RB;
        while (t < end) {
            const SeqLen sl = seq_len(a, b);
            const int tiles = max(1, (sl.total + TILE - 1) / TILE), dealt = a.whole ? 1 : tiles;
            if (t >= seq_at + (long long)dealt * units) {       // the share goes on in the next sequence
                seq_at += (long long)dealt * units;
                ++b;
                continue;
            }
            x->b = b;
            x->sl = sl;
            x->tiles = tiles;
            x->u = (int)quotient(t - seq_at, dealt);
            x->at = seq_at + (long long)x->u * dealt;
            x->ta = (int)(t - x->at);
            x->tb = a.whole ? tiles : (int)min((long long)tiles, end - x->at);
            x->hk = x->u / RB;
            x->r0 = (x->u - x->hk * RB) * block_rows;
            x->rows = min(block_rows, a.N * a.G - x->r0);
            t = a.whole ? x->at + 1 : x->at + x->tb;
            return true;
        }
        return false;
    }
};

// Notes for the join which unit, if any, the CTA has begun and others end: the
// last one of its share.  By one thread, its walk at the end.
__device__ __forceinline__ void note_split(const AttendArgs& a, const AttPlan& p, const AttUnit& x) {
    AttSplit s = {};
    if ((int)blockIdx.x < p.n && x.ta == 0 && x.tb < x.tiles)
        s = {share_of(p.total, p.n, x.at + x.tiles - 1) - (int)blockIdx.x + 1, x.b, x.hk, x.r0, x.rows, x.sl.nb, {0, 0}};
    reinterpret_cast<AttSplit*>(a.ws)[blockIdx.x] = s;
}

// Writes elements d .. d + 3 of row r of a finished unit: row r0 + r of cached head
// hk of sequence b, which has nb new positions.  Rows past those are empty, whatever
// else the sequence has, a bad page or a malformed tree (whose total is NaN), unless
// its lengths are bad: then nobody knows which rows they are.
__device__ __forceinline__ void put_row(const AttendArgs& a, int b, int hk, int r0, int nb, bool bad_lengths, int D, int r, int d,
                                        float4 v, float lsum, float mref) {
    const int R = r0 + r, n = row_position(a, R), g = R - n * a.G;
    const size_t row = ((size_t)b * a.N + n) * a.Hq + (size_t)hk * a.G + g;
    const bool empty = n >= nb && !bad_lengths;
    const float f = empty ? 0.f : 1.f / lsum;
    if (empty) v = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<uint2*>(a.out + (row * D + d) * 2) = make_uint2(pack_bf16(v.x * f, v.y * f), pack_bf16(v.z * f, v.w * f));
    if (a.lse && d == 0) a.lse[row] = empty ? kNegInf : (mref + __log2f(lsum)) * kLn2;
}

// Joins the parts that `ctas` CTAs of the call's kernel have left, units of up to
// `units` row blocks of block_rows rows, `tiles` tiles at most (sv_attend.cu).
cudaError_t launch_join(const AttendArgs& a, int ctas, long long units, int block_rows, long long tiles, cudaStream_t st);

// Whether a call deals its units whole: `units` of them, of up to `positions`, to `ctas`.
bool attend_whole(long long units, long long positions, long long ctas);

// The matrix-unit kernel of sv_attend_tc.cu (rows of 128 elements).
cudaError_t launch_attend_tc(const AttendArgs& a, cudaStream_t st);
// Whether that kernel takes a call; capacity: positions that a sequence's row of
// the block table has room for, units: cached heads of all sequences.
bool attend_takes_tc(int N, int G, int D, bool fp8, long long capacity, long long units, int sms);
size_t attend_tc_workspace(int N, int G);

}  // namespace sv
