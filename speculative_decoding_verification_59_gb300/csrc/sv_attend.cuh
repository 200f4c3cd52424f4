// What the attention kernels share: asynchronous copies, the split of the work
// among CTAs, and the join of a split unit's parts.
#pragma once

#include "sv_kv.cuh"

namespace sv {

constexpr int kAttMaxCtas = 512;            // workspace slots are sized for this many
constexpr size_t kAttHead = 4096;           // bytes of the workspace before the parts: counters from 256 on
static_assert(256 + kAttMaxCtas * 4 <= kAttHead, "the counters lie in the zeroed head");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The reference m of a row moves only when a score passes it by more than
// this (in powers of two): sums stay below 2^8 per position, and the sums in
// registers are rarely rescaled.
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
    long long total;         // tiles of all units
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
    for (int b = b0; b < b1; ++b) mine += max(1, (seq_len(a, b).total + TILE - 1) / TILE);
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
            const long long t = (long long)units * max(1, (seq_len(a, b).total + TILE - 1) / TILE);
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
            const int tiles = max(1, (sl.total + TILE - 1) / TILE);
            if (t >= seq_at + (long long)tiles * units) {       // the share goes on in the next sequence
                seq_at += (long long)tiles * units;
                ++b;
                continue;
            }
            x->b = b;
            x->sl = sl;
            x->tiles = tiles;
            x->u = (int)quotient(t - seq_at, tiles);
            x->at = seq_at + (long long)x->u * tiles;
            x->ta = (int)(t - x->at);
            x->tb = (int)min((long long)tiles, end - x->at);
            x->hk = x->u / RB;
            x->r0 = (x->u - x->hk * RB) * block_rows;
            x->rows = min(block_rows, a.N * a.G - x->r0);
            t = x->at + x->tb;
            return true;
        }
        return false;
    }
};

// Writes elements d .. d + 3 of row r of a finished unit.
__device__ __forceinline__ void put_row(const AttendArgs& a, const AttUnit& x, bool bad, int D, int r, int d, float4 v,
                                        float lsum, float mref) {
    const int R = x.r0 + r, n = row_position(a, R), g = R - n * a.G;
    const size_t row = ((size_t)x.b * a.N + n) * a.Hq + (size_t)x.hk * a.G + g;
    const bool empty = n >= x.sl.nb && !bad;
    const float f = empty ? 0.f : 1.f / lsum;
    if (empty) v = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<uint2*>(a.out + (row * D + d) * 2) = make_uint2(pack_bf16(v.x * f, v.y * f), pack_bf16(v.z * f, v.w * f));
    if (a.lse && d == 0) a.lse[row] = empty ? kNegInf : (mref + __log2f(lsum)) * kLn2;
}

// Adds rows ra .. rb - 1 of the parts of a unit that CTAs c0 .. c1 hold, in
// that order, and writes them; by WARPS warps (warp w of them).  A warp takes
// ROWS rows at once, one lane per part for their references and totals, then its
// lanes across the elements: the loads of several rows and parts are in flight
// together (a row and part at a time, the join of 32 rows in 5 parts took 22 us;
// the parts come from L2, about 0.5 us away).
template <int D, int WARPS, int ROWS>
__device__ __forceinline__ void join_rows(const AttendArgs& a, const AttUnit& x, int w, float* slots, size_t slot_floats,
                                          int srows, int c0, int c1, int ra, int rb) {
    constexpr int V = D / 32;                                 // elements of a lane: 2, 4 or 8
    constexpr int V4 = V >= 4 ? V / 4 : 1;
    const int lane = threadIdx.x & 31, parts = c1 - c0 + 1;
    auto part = [&](int p) { return slots + (size_t)(2 * (c0 + p) + (p == 0 ? 1 : 0)) * slot_floats; };
    for (int r0 = ra + w * ROWS; r0 < rb; r0 += WARPS * ROWS) {
        float M[ROWS], L[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) { M[k] = kNegInf; L[k] = 0.f; }
        for (int p0 = 0; p0 < parts; p0 += 32) {
            float m[ROWS];
#pragma unroll
            for (int k = 0; k < ROWS; ++k)
                m[k] = p0 + lane < parts && r0 + k < rb ? __ldcg(part(p0 + lane) + (size_t)srows * D + r0 + k) : kNegInf;
#pragma unroll
            for (int k = 0; k < ROWS; ++k) M[k] = fmaxf(M[k], m[k]);
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            M[k] = warp_max(M[k]);
            if (M[k] == kNegInf) M[k] = 0.f;                  // no part has seen a position
        }
        float v[ROWS][V];
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) v[k][e] = 0.f;
        for (int p0 = 0; p0 < parts; p0 += 32) {
            float f[ROWS];
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                const bool on = p0 + lane < parts && r0 + k < rb;
                const float* q = part(on ? p0 + lane : 0) + (size_t)srows * D + (on ? r0 + k : ra);
                f[k] = on ? ex2_approx(__ldcg(q) - M[k]) : 0.f;
                L[k] = on ? fmaf(f[k], __ldcg(q + srows), L[k]) : L[k];
            }
            const int n = min(32, parts - p0);
#pragma unroll(ROWS == 1 ? 8 : 2)
            for (int p = 0; p < n; ++p) {
                const float* q = part(p0 + p) + (size_t)r0 * D + lane * V;
                float y[ROWS][V];
#pragma unroll
                for (int k = 0; k < ROWS; ++k) {
                    const float* at = q + (r0 + k < rb ? k * D : 0);
                    if constexpr (V == 2) {
                        const float2 t = __ldcg(reinterpret_cast<const float2*>(at));
                        y[k][0] = t.x;
                        y[k][1] = t.y;
                    } else {
#pragma unroll
                        for (int h = 0; h < V4; ++h) {
                            const float4 t = __ldcg(reinterpret_cast<const float4*>(at) + h);
                            y[k][4 * h] = t.x;
                            y[k][4 * h + 1] = t.y;
                            y[k][4 * h + 2] = t.z;
                            y[k][4 * h + 3] = t.w;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < ROWS; ++k) {
                    const float fp = __shfl_sync(0xffffffffu, f[k], p);
#pragma unroll
                    for (int e = 0; e < V; ++e) v[k][e] = fmaf(fp, y[k][e], v[k][e]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            // the lanes' totals in a fixed order
            const float lsum = warp_sum(L[k]);
            if (r0 + k < rb) {
                if constexpr (V == 2) {
                    const float2 o = make_float2(__shfl_down_sync(0xffffffffu, v[k][0], 1), __shfl_down_sync(0xffffffffu, v[k][1], 1));
                    if (!(lane & 1)) put_row(a, x, false, D, r0 + k, lane * 2, make_float4(v[k][0], v[k][1], o.x, o.y), lsum, M[k]);
                } else {
#pragma unroll
                    for (int h = 0; h < V4; ++h)
                        put_row(a, x, false, D, r0 + k, lane * V + 4 * h,
                                make_float4(v[k][4 * h], v[k][4 * h + 1], v[k][4 * h + 2], v[k][4 * h + 3]), lsum, M[k]);
                }
            }
        }
    }
}

// One row a warp while there is a warp for each, else four.
template <int D, int WARPS>
__device__ __forceinline__ void join_parts(const AttendArgs& a, const AttUnit& x, int w, float* slots, size_t slot_floats,
                                           int srows, int c0, int c1, int ra, int rb) {
    if (rb - ra <= WARPS) join_rows<D, WARPS, 1>(a, x, w, slots, slot_floats, srows, c0, c1, ra, rb);
    else join_rows<D, WARPS, 4>(a, x, w, slots, slot_floats, srows, c0, c1, ra, rb);
}

// The matrix-unit kernel of sv_attend_tc.cu (rows of 128 elements).
cudaError_t launch_attend_tc(const AttendArgs& a, cudaStream_t st);
// Whether that kernel takes a call; capacity: positions that a sequence's row of
// the block table has room for.
bool attend_takes_tc(int N, int G, int D, long long capacity);
size_t attend_tc_workspace(int N, int G);

}  // namespace sv
