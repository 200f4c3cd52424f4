// Attention of a few new positions per sequence over the paged cache, split
// over the cache's length, and the join of what was split.
//
// out = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m), s_t = (scale log2 e) q.k_t,
// with the running reference m of a one-pass softmax.  The rows of one cached
// head -- N positions x G query heads -- share every key and value, so they go
// through the matrix units together, up to 32 at a time: one such row block of
// one cached head of one sequence is a unit.
//
// Work split.  A unit's positions are cut into tiles; all units' tiles, laid
// end to end, are dealt to the CTAs in equal contiguous shares, computed on
// the device from the lengths (ragged batches balance, and a captured call
// follows its lengths).  A share may end one unit and begin the next.  (Short units are
// dealt whole.)  A unit
// within one share is written at once; otherwise each CTA leaves its
// unnormalised sum, reference and total in the workspace, and a second small
// kernel adds them in the order of the shares.
//
// Inside a CTA each of the four warps (or pairs of warps, with 16 rows each) takes its
// own slice of every tile and its own running softmax, so these never wait for one
// another while streaming: a warp copies its slices with 16-byte cp.async into a ring of its
// own.  mma.sync (m16n8k16): 16 rows of queries against 8 positions (scores), then
// probabilities against 8 head elements (sums).  An E4M3 cache is widened to
// fp16 (exact) next to the matrix instruction; queries then go in as fp16,
// each row scaled by a power of two, and a position's key scale multiplies
// its score, its value scale its probability (as a summand of the exponent).
// Probabilities then are fp16 too, whose steps end at 2^-24: a row's reference is
// kept kFp16Head below its largest score, where fp16 still holds the largest
// (2^(kFp16Head + kRefSlack)), so that next to nothing is what is lost.
//
// Measured (8 cached heads of 128, bf16, lengths from half of the stated one to all of it):
// 64 sequences x 4 rows over 4000 in 127 us, 6.2 TB/s of the cache's 0.79 GB, memory-bound;
// 4 rows over 1000 in 7.4 us, of which the join is 3 and one tile alone 4.4 (launch, four
// dependent loads); 42 trees x 184 rows over 1782 with heads of 64 in 174 us, bound by
// the matrix instructions and by reading the cache once for every 32 rows.
#include "sv_attend.cuh"

namespace sv {

constexpr int kAttWarps = 4;
constexpr float kFp16Head = 7.f;
// RG = 2: two sets of kAttWarps warps, each with its own rows, over one ring of
// slices for every two warps (256 elements, more than 16 rows: 16 rows are what a
// warp's registers hold, and three stages leave room for one CTA on an SM).
template <int D, int MT, int RG, bool FP8>
struct AttCfg {
    static constexpr int THREADS = kAttWarps * 32 * RG;
    static constexpr int CTAS = RG == 1 ? 2 : 1;               // on an SM
    static constexpr int ELT = FP8 ? 1 : 2;
    static constexpr int ROWB = D * ELT;                       // bytes of a cached row
    static constexpr int CPR = ROWB / 16;                      // 16-byte chunks of it
    static constexpr int ST0 = 4096 / ROWB;
    static constexpr int ST = ST0 < 16 ? 16 : ST0 > 32 ? 32 : ST0;   // positions of a slice
    static constexpr int NT = ST / 8;
    static constexpr int STAGE = 2 * ST * ROWB + (FP8 ? 2 * ST * 4 : 0);
    static constexpr int NS0 = 24576 * RG / (2 * ST * ROWB);
    static constexpr int NS = NS0 < 3 ? 3 : NS0 > 6 ? 6 : NS0;       // stages of a warp's ring
    static constexpr int WROWS = 16 * MT, ROWS = WROWS * RG;    // rows of a warp, of a unit
    static constexpr int TILE = kAttWarps * ST;                // positions of a tile
    static constexpr int OP = D + 8;                           // padded row of the warps' sums
    static constexpr int RING = kAttWarps * NS * STAGE;
    static constexpr int MERGE = kAttWarps * ROWS * OP * 4;   // (a set's warps have its rows)
    // 32 rows of 128 elements: the queries' fragments stay in shared memory (one
    // copy for the four warps), the sums need the registers
    static constexpr bool QSM = MT == 2 && D == 128;
    static constexpr int QOFF = RING > MERGE ? RING : MERGE;
    static constexpr int SMEM = QOFF + (QSM ? MT * (D / 16) * 512 : 0);
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row t in a slice: chunks swizzled so that
// eight consecutive rows' equal chunks lie in eight different bank groups.
template <int CPR>
__device__ __forceinline__ int swz(int t, int c) {
    if constexpr (CPR >= 8) return (t * CPR + (c ^ (t & 7))) * 16;
    else return (t * CPR + (c ^ ((t >> 1) & 3))) * 16;          // CPR = 4: two rows per 128 bytes
}

template <int D, int MT, int RG, bool FP8>
__global__ void __launch_bounds__(AttCfg<D, MT, RG, FP8>::THREADS, AttCfg<D, MT, RG, FP8>::CTAS) attend_kernel(const AttendArgs a) {
    using C = AttCfg<D, MT, RG, FP8>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ AttPlan plan;
    __shared__ unsigned long long anc[2][kMaxNewTree];         // ancestors and itself, by node
    __shared__ short up[2][kMaxNewTree];
    __shared__ float wm[kAttWarps][C::ROWS], wl[kAttWarps][C::ROWS];
    __shared__ int wbad[kAttWarps * RG];
    const int lane = threadIdx.x & 31;
    const int set = RG > 1 ? threadIdx.x / (kAttWarps * 32) : 0, warp = (threadIdx.x >> 5) - set * kAttWarps;
    // the warps that share a ring
    auto ring_sync = [&] {
        if constexpr (RG > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + warp), "n"(RG * 32) : "memory");
        else __syncwarp();
    };
    const int quad = lane & 3, lrow = lane >> 2;
    pdl_trigger();
    pdl_wait();

    const int RT = a.N * a.G;                                  // rows of a cached head
    const int RB = (RT + C::ROWS - 1) / C::ROWS;
    make_plan<C::TILE, C::THREADS>(a, a.c.kv_heads * RB, gridDim.x, &plan);
    AttWalk walk;
    AttUnit un;
    if ((int)blockIdx.x >= plan.n) {
        if (threadIdx.x == 0) note_split(a, plan, un);
        return;
    }
    walk.init(plan);
    int anc_b = -1, tree_bad = 0;
    const float c2 = a.scale * kLog2e;
    float* slots = reinterpret_cast<float*>(a.ws + kAttHead);
    const int srows = min(C::ROWS, RT);
    const size_t slot_floats = part_floats(srows, D);

    while (walk.next<C::TILE>(a, RB, C::ROWS, &un)) {
        const SeqLen& sl = un.sl;
        const int b = un.b, tiles = un.tiles, ta = un.ta, tb = un.tb, hk = un.hk, r0 = un.r0, rows = un.rows;
        __syncthreads();                                        // the unit before is done with shared memory
        if (a.par && anc_b != b) {
            // ancestors by pointer doubling: 2^6 steps cover any path of 64 nodes
            const int n = threadIdx.x;
            int wrong = 0;
            if (n < a.N) {
                const int p = __ldg(a.par + (size_t)b * a.N + n);
                wrong = n < sl.nb && (n == 0 ? p != -1 : (p < 0 || p >= n));
                anc[0][n] = 1ull << n;
                up[0][n] = (short)(wrong || n == 0 || n >= sl.nb ? -1 : p);
            }
            wrong = __syncthreads_or(wrong);
#pragma unroll
            for (int k = 0; k < 6; ++k) {
                if (n < a.N) {
                    const int p = up[k & 1][n];
                    anc[(k + 1) & 1][n] = anc[k & 1][n] | (p >= 0 ? anc[k & 1][p] : 0ull);
                    up[(k + 1) & 1][n] = p >= 0 ? up[k & 1][p] : (short)-1;
                }
                __syncthreads();
            }
            anc_b = b;
            tree_bad = wrong;
            if (wrong && threadIdx.x == 0) raise_error(a.c.error, SPEC_DEVERR_TREE_PARENT);
        }
        if (sl.bad && threadIdx.x == 0) raise_error(a.c.error, SPEC_DEVERR_CACHE_RANGE);

        // ---- the rows' queries as matrix fragments; rows past the unit's are zero
        uint32_t qf[MT][D / 16][4];
        float rs[MT][2];                                        // score factor of the thread's rows
        int rn[MT][2];                                          // their new position
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                const int r = set * C::WROWS + mt * 16 + hrow * 8 + lrow, R = r0 + r;
                const bool on = r < rows;
                const int n = on ? row_position(a, R) : 0, g = on ? R - n * a.G : 0;
                rn[mt][hrow] = n;
                rs[mt][hrow] = c2;
                const char* src = a.q + ((int64_t)b * a.N + n) * a.qs + ((size_t)hk * a.G + g) * D * 2;
                if constexpr (!FP8) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t* p = reinterpret_cast<const uint32_t*>(src + k * 32) + quad;
                        qf[mt][k][hrow] = on ? __ldg(p) : 0u;
                        qf[mt][k][2 + hrow] = on ? __ldg(p + 4) : 0u;
                    }
                } else {
                    // elements 4 quad .. 4 quad + 3 of every 16: the order in which a
                    // widened key row comes out of the matrix load.  Scaled so that
                    // the row's largest is in [2^8, 2^9): fp16 then holds every
                    // element that matters exactly.
                    float mx = 0.f;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint2 w = on ? __ldg(reinterpret_cast<const uint2*>(src + k * 32) + quad) : make_uint2(0u, 0u);
                        qf[mt][k][hrow] = w.x;
                        qf[mt][k][2 + hrow] = w.y;
                        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(bf_lo(w.x)), fabsf(bf_hi(w.x))),
                                             fmaxf(fabsf(bf_lo(w.y)), fabsf(bf_hi(w.y)))));
                    }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const int ex = (int)(__float_as_uint(mx) >> 23);          // 0..255
                    const int sh = ex < 16 || ex > 240 ? 0 : 135 - ex;        // 2^sh
                    const float f = __uint_as_float((uint32_t)(127 + sh) << 23);
                    rs[mt][hrow] = c2 * __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t x = qf[mt][k][hrow], y = qf[mt][k][2 + hrow];
                        qf[mt][k][hrow] = pack_f16(bf_lo(x) * f, bf_hi(x) * f);
                        qf[mt][k][2 + hrow] = pack_f16(bf_lo(y) * f, bf_hi(y) * f);
                    }
                }
            }
        }

        uint4* qsm = reinterpret_cast<uint4*>(smem + C::QOFF);
        if constexpr (C::QSM) {                                 // the warps hold the same fragments
            if (warp == 0) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        qsm[(mt * (D / 16) + k) * 32 + lane] = make_uint4(qf[mt][k][0], qf[mt][k][1], qf[mt][k][2], qf[mt][k][3]);
            }
            __syncthreads();
        }
        auto query = [&](int mt, int k, uint32_t (&q)[4]) {
            if constexpr (C::QSM) {
                const uint4 w = qsm[(mt * (D / 16) + k) * 32 + lane];
                q[0] = w.x; q[1] = w.y; q[2] = w.z; q[3] = w.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) q[e] = qf[mt][k][e];
            }
        };

        float o[MT][D / 8][4];
        float m[MT][2], l[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt][0] = m[mt][1] = kNegInf;
            l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) o[mt][i][0] = o[mt][i][1] = o[mt][i][2] = o[mt][i][3] = 0.f;
        }

        // ---- the warp's slices: positions (tile * 4 + warp) * ST ..., tiles ta .. tb - 1
        unsigned char* ring = smem + (size_t)warp * C::NS * C::STAGE;
        const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
        const int nsl = tb - ta;
        auto slice_at = [&](int i) { return ((ta + i) * kAttWarps + warp) * C::ST; };
        bool lost = false;
        // Lane t finds entry t of the next slice to copy.  Its page id is loaded one
        // slice before it is used, so that nothing waits for the table.
        int page = 0, slot = 0;
        bool want = false;                                      // the lane has a position (whose page is not looked at yet)
        auto locate = [&](int i) {
            const int pos = slice_at(i) + lane;
            want = i < nsl && lane < C::ST && pos < sl.total;
            if (want) {
                const int pg = page_index(a, pos, &slot);
                page = pg < a.c.max_pages ? __ldg(a.c.block_table + (size_t)b * a.c.max_pages + pg) : -1;
            }
        };
        auto copy = [&](int i) {                                // slice i, located before
            if (i < nsl) {
                const uint32_t st = ring_s + (i % C::NS) * C::STAGE;
                constexpr int RP = 32 / C::CPR;                // rows the warp copies at once
                const int ch = lane % C::CPR, sub = lane / C::CPR;
                const bool ok = want && (unsigned)page < (unsigned)a.c.num_pages;
                lost |= want && !ok;
                const int64_t off = ok ? entry_off(a.c, page, slot, hk) : 0;
                const unsigned okm = __ballot_sync(0xffffffffu, ok);
#pragma unroll
                for (int p = 0; p < C::ST / RP; ++p) {
                    if (RG > 1 && p % RG != set) continue;     // (warps of a ring take turns)
                    const int row = p * RP + sub;
                    const int64_t e = __shfl_sync(0xffffffffu, off, row) * C::ELT + ch * 16;
                    const bool in = (okm >> row) & 1u;
                    const uint32_t d = st + swz<C::CPR>(row, ch);
                    cp16(d, static_cast<const char*>(a.c.k) + e, in);
                    cp16(d + C::ST * C::ROWB, static_cast<const char*>(a.c.v) + e, in);
                }
                if constexpr (FP8) {
                    if (lane < C::ST && set == 0) {
                        const uint32_t d = st + 2 * C::ST * C::ROWB + lane * 4;
                        const int64_t soff = ok ? scale_off(a.c, page, slot, hk) : 0;
                        cp4(d, a.c.k_scale + soff, ok);
                        cp4(d + C::ST * 4, a.c.v_scale + soff, ok);
                    }
                }
            }
            cp_commit();
        };
        __syncwarp();
        locate(0);
#pragma unroll 1
        for (int i = 0; i < C::NS - 1; ++i) {
            copy(i);
            locate(i + 1);
        }

#pragma unroll 1
        for (int i = 0; i < nsl; ++i) {
            cp_wait<C::NS - 2>();
            ring_sync();
            copy(i + C::NS - 1);                                // into the stage read last time round
            locate(i + C::NS);
            const uint32_t ks = ring_s + (i % C::NS) * C::STAGE, vs = ks + C::ST * C::ROWB;
            const float* ksc = reinterpret_cast<const float*>(ring + (i % C::NS) * C::STAGE + 2 * C::ST * C::ROWB);
            const int p0 = slice_at(i);
            if (p0 >= sl.total) continue;                       // warp-uniform

            float s[MT][C::NT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < C::NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
            // a matrix load brings 8 positions x 64 bytes of the keys
#pragma unroll
            for (int cg = 0; cg < C::CPR / 4; ++cg) {
                constexpr int KQ = FP8 ? 4 : 2;                 // query fragments that 64 bytes meet
                uint32_t q[MT][KQ][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < KQ; ++j) query(mt, cg * KQ + j, q[mt][j]);
#pragma unroll
                for (int nt = 0; nt < C::NT; ++nt) {
                    uint32_t kf[4];
                    ldsm4(ks + swz<C::CPR>(nt * 8 + (lane & 7), cg * 4 + (lane >> 3)), kf);
#pragma unroll
                    for (int j = 0; j < KQ; ++j) {
                        uint32_t w0, w1;
                        if constexpr (FP8) {
                            w0 = e4m3_to_f16x2(kf[j] & 0xffffu);
                            w1 = e4m3_to_f16x2(kf[j] >> 16);
                        } else {
                            w0 = kf[2 * j];
                            w1 = kf[2 * j + 1];
                        }
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) mma16<FP8>(s[mt][nt], q[mt][j], w0, w1);
                    }
                }
            }
            // scores in powers of two; for E4M3 plus the log of the value's scale
            float vinv[FP8 ? C::NT : 1][2];
#pragma unroll
            for (int nt = 0; nt < C::NT; ++nt) {
                if constexpr (FP8) {
                    const float2 kk = *reinterpret_cast<const float2*>(ksc + nt * 8 + 2 * quad);
                    float2 vv = *reinterpret_cast<const float2*>(ksc + C::ST + nt * 8 + 2 * quad);
                    vv.x = value_scale(vv.x);
                    vv.y = value_scale(vv.y);
                    const float g0 = __log2f(vv.x), g1 = __log2f(vv.y);
                    vinv[nt][0] = 1.f / vv.x;
                    vinv[nt][1] = 1.f / vv.y;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        s[mt][nt][0] = fmaf(s[mt][nt][0], rs[mt][0] * kk.x, g0);
                        s[mt][nt][1] = fmaf(s[mt][nt][1], rs[mt][0] * kk.y, g1);
                        s[mt][nt][2] = fmaf(s[mt][nt][2], rs[mt][1] * kk.x, g0);
                        s[mt][nt][3] = fmaf(s[mt][nt][3], rs[mt][1] * kk.y, g1);
                    }
                } else {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mt][nt][e] *= c2;
                }
            }
            if (p0 + C::ST > sl.ctx) {                          // new positions, or past the end (warp-uniform)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int d = p0 + nt * 8 + 2 * quad + (e & 1) - sl.ctx, n = rn[mt][e >> 1];
                            const bool sees = d < 0 || (d < sl.nb && (a.par ? (anc[0][n] >> (d & 63)) & 1ull : d <= n));
                            if (!sees) s[mt][nt][e] = kNegInf;
                        }
            }
            // ---- running reference
            float mx[MT][2];
            bool grow = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = kNegInf;
#pragma unroll
                    for (int nt = 0; nt < C::NT; ++nt) x = fmaxf(x, fmaxf(s[mt][nt][2 * h], s[mt][nt][2 * h + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    mx[mt][h] = x;
                    grow |= x > m[mt][h] + kRefSlack + (FP8 ? kFp16Head : 0.f);
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float to = FP8 ? mx[mt][h] - kFp16Head : mx[mt][h], mn = to > m[mt][h] ? to : m[mt][h];
                        const float f = m[mt][h] == kNegInf ? 0.f : ex2_approx(m[mt][h] - mn);
                        m[mt][h] = mn;
                        l[mt][h] *= f;
#pragma unroll
                        for (int d = 0; d < D / 8; ++d) {
                            o[mt][d][2 * h] *= f;
                            o[mt][d][2 * h + 1] *= f;
                        }
                    }
            }
            // ---- probabilities, as the next product's fragments
            uint32_t pf[MT][C::NT / 2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const float m0 = m[mt][0] == kNegInf ? 0.f : m[mt][0], m1 = m[mt][1] == kNegInf ? 0.f : m[mt][1];
#pragma unroll
                for (int nt = 0; nt < C::NT; ++nt) {
                    float (&x)[4] = s[mt][nt];
                    x[0] = ex2_approx(x[0] - m0);
                    x[1] = ex2_approx(x[1] - m0);
                    x[2] = ex2_approx(x[2] - m1);
                    x[3] = ex2_approx(x[3] - m1);
                    if constexpr (FP8) {
                        // (a masked position's scale may be anything)
                        l[mt][0] += (x[0] != 0.f ? x[0] * vinv[nt][0] : 0.f) + (x[1] != 0.f ? x[1] * vinv[nt][1] : 0.f);
                        l[mt][1] += (x[2] != 0.f ? x[2] * vinv[nt][0] : 0.f) + (x[3] != 0.f ? x[3] * vinv[nt][1] : 0.f);
                        pf[mt][nt >> 1][2 * (nt & 1)] = pack_f16(x[0], x[1]);
                        pf[mt][nt >> 1][2 * (nt & 1) + 1] = pack_f16(x[2], x[3]);
                    } else {
                        l[mt][0] += x[0] + x[1];
                        l[mt][1] += x[2] + x[3];
                        pf[mt][nt >> 1][2 * (nt & 1)] = pack_bf16(x[0], x[1]);
                        pf[mt][nt >> 1][2 * (nt & 1) + 1] = pack_bf16(x[2], x[3]);
                    }
                }
            }
            if (p0 + C::ST > sl.ctx) {
                // A value that is no number (of a position that some rows mask) times
                // a probability of zero would still spoil the sum.  Such positions
                // are added one by one, to the rows that see them, and taken out of
                // the slice.
                unsigned char* vb = ring + (i % C::NS) * C::STAGE + C::ST * C::ROWB;
                unsigned odd = 0u;                              // bit t: position t holds one
                for (int e = lane; e < C::ST * C::CPR; e += 32) {
                    const int t0 = e / C::CPR;
                    const uint4 w = *reinterpret_cast<const uint4*>(vb + swz<C::CPR>(t0, e % C::CPR));
                    bool x = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t y = u4_get(w, k);
                        if constexpr (FP8) {
#pragma unroll
                            for (int q = 0; q < 32; q += 8) x |= ((y >> q) & 0x7fu) == 0x7fu;
                        } else {
                            x |= (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
                        }
                    }
                    if (x) odd |= 1u << t0;
                }
                odd = __reduce_or_sync(0xffffffffu, odd);
                if (RG > 1 && odd) ring_sync();                 // (all have looked: the same for a ring's warps)
                for (unsigned left = odd; left; left &= left - 1u) {   // warp-uniform, rare
                    const int t0 = __ffs(left) - 1;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float p = 0.f;
#pragma unroll
                            for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (t0 >> 3 == nt && (t0 & 1) == e) p = s[mt][nt][2 * h + e];
                            p = __shfl_sync(0xffffffffu, p, (lane & ~3) | ((t0 & 7) >> 1));
                            if (p > 0.f || p != p) {
#pragma unroll
                                for (int d = 0; d < D / 8; ++d)
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        // the element that o[mt][d][2 h + e] sums
                                        const int el = FP8 ? (d >> 1) * 16 + 4 * quad + 2 * e + (d & 1) : d * 8 + 2 * quad + e;
                                        const unsigned char* q = vb + swz<C::CPR>(t0, el * C::ELT / 16) + el * C::ELT % 16;
                                        float v;
                                        if constexpr (FP8) {
                                            float unused;
                                            f16x2_to_f32(e4m3_to_f16x2(*q), &v, &unused);
                                        } else {
                                            v = __uint_as_float((uint32_t)*reinterpret_cast<const unsigned short*>(q) << 16);
                                        }
                                        o[mt][d][2 * h + e] = fmaf(p, v, o[mt][d][2 * h + e]);
                                    }
                            }
                        }
                }
                if (odd) {
                    ring_sync();
                    for (int e = lane; e < C::ST * C::CPR; e += 32)
                        if ((odd >> (e / C::CPR)) & 1u)
                            *reinterpret_cast<uint4*>(vb + swz<C::CPR>(e / C::CPR, e % C::CPR)) = make_uint4(0u, 0u, 0u, 0u);
                    ring_sync();
                }
            }
            // ---- sums
#pragma unroll
            for (int kk = 0; kk < C::NT / 2; ++kk) {
                if constexpr (!FP8) {
#pragma unroll
                    for (int dg = 0; dg < D / 16; ++dg) {       // 16 positions x 16 elements
                        uint32_t vf[4];
                        ldsm4t(vs + swz<C::CPR>(kk * 16 + (lane & 15), dg * 2 + (lane >> 4)), vf);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            mma16<false>(o[mt][2 * dg], pf[mt][kk], vf[0], vf[1]);
                            mma16<false>(o[mt][2 * dg + 1], pf[mt][kk], vf[2], vf[3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int dg = 0; dg < D / 32; ++dg) {       // 16 positions x 32 elements, in byte pairs
                        uint32_t vf[4];
                        ldsm4t(vs + swz<C::CPR>(kk * 16 + (lane & 15), dg * 2 + (lane >> 4)), vf);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            // even elements of the two positions, then odd ones
                            const uint32_t x = __byte_perm(vf[2 * j], 0, 0x3120), y = __byte_perm(vf[2 * j + 1], 0, 0x3120);
                            const uint32_t e0 = e4m3_to_f16x2(x & 0xffffu), e1 = e4m3_to_f16x2(y & 0xffffu);
                            const uint32_t d0 = e4m3_to_f16x2(x >> 16), d1 = e4m3_to_f16x2(y >> 16);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                mma16<true>(o[mt][4 * dg + 2 * j], pf[mt][kk], e0, e1);
                                mma16<true>(o[mt][4 * dg + 2 * j + 1], pf[mt][kk], d0, d1);
                            }
                        }
                    }
                }
            }
        }
        cp_wait<0>();
        lost = __any_sync(0xffffffffu, lost);
        if (lane == 0) {
            wbad[set * kAttWarps + warp] = lost;
            if (lost) raise_error(a.c.error, SPEC_DEVERR_CACHE_RANGE);
        }

        // ---- join the warps
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = l[mt][h];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (quad == 0) {
                    wm[warp][set * C::WROWS + mt * 16 + h * 8 + lrow] = m[mt][h];
                    wl[warp][set * C::WROWS + mt * 16 + h * 8 + lrow] = x;
                }
            }
        __syncthreads();                                        // the rings are drained
        float* wo = reinterpret_cast<float*>(smem) + (size_t)warp * C::ROWS * C::OP;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = set * C::WROWS + mt * 16 + h * 8 + lrow;
                if (r < rows) {
                    if constexpr (!FP8) {
#pragma unroll
                        for (int d = 0; d < D / 8; ++d)
                            *reinterpret_cast<float2*>(wo + r * C::OP + d * 8 + 2 * quad) = make_float2(o[mt][d][2 * h], o[mt][d][2 * h + 1]);
                    } else {
#pragma unroll
                        for (int g = 0; g < D / 16; ++g)
                            *reinterpret_cast<float4*>(wo + r * C::OP + g * 16 + 4 * quad) =
                                make_float4(o[mt][2 * g][2 * h], o[mt][2 * g + 1][2 * h], o[mt][2 * g][2 * h + 1], o[mt][2 * g + 1][2 * h + 1]);
                    }
                }
            }
        __syncthreads();
        bool bad = sl.bad || tree_bad;
#pragma unroll
        for (int w = 0; w < kAttWarps * RG; ++w) bad |= wbad[w] != 0;
        const bool whole = ta == 0 && tb == tiles;
        const int mine = 2 * (int)blockIdx.x + (ta == 0 ? 1 : 0);
        float* sp = slots + (size_t)mine * slot_floats;
        for (int i = threadIdx.x; i < rows * (D / 4); i += C::THREADS) {
            const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
            float M = kNegInf;
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) M = fmaxf(M, wm[w][r]);
            const float Ms = M == kNegInf ? 0.f : M;
            float L = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) {
                const float f = ex2_approx(wm[w][r] - Ms);
                const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) + (size_t)w * C::ROWS * C::OP + r * C::OP + d);
                L = fmaf(f, wl[w][r], L);
                x.x = fmaf(f, y.x, x.x);
                x.y = fmaf(f, y.y, x.y);
                x.z = fmaf(f, y.z, x.z);
                x.w = fmaf(f, y.w, x.w);
            }
            if (bad) L = CUDART_NAN_F;
            if (whole) {
                put_row(a, b, hk, r0, sl.nb, sl.bad, D, r, d, x, L, M);
            } else {
                __stcg(reinterpret_cast<float4*>(sp + (size_t)r * D + d), x);
                if (d == 0) {
                    __stcg(sp + (size_t)srows * D + r, M);
                    __stcg(sp + (size_t)srows * (D + 1) + r, L);
                }
            }
        }
    }
    if (threadIdx.x == 0) note_split(a, plan, un);
}

// ---- the join -------------------------------------------------------------------
// One row per `per` warps: each takes every per-th part, four at a time (their
// loads under way together), with a running reference; the row's first warp then
// adds the warps' sums in order.  blockIdx.x is the CTA that began the unit, so the
// grid is the attention kernel's times the rows.
// A launch of its own rather than the last CTA of a unit to arrive: that CTA was
// alone with its unit's parts, behind a fence and a counter, and its code weighed on
// the attention kernel's registers.  13 rows x 4 heads over 4749 positions in 38
// parts: 53.0 us then, 18.4 now; 4 rows x 8 heads over 1000: 8.45 and 7.40; 512
// units of 32 rows over up to 4096: 155.9 and 148.8.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const AttendArgs a, int block_rows, int per) {
    constexpr int W = kJoinThreads / 32, V = D / 32, U = 4;   // warps, elements of a lane, parts at a time
    constexpr int VEC = V < 4 ? V : 4;
    __shared__ __align__(16) float sum[W][D];
    __shared__ float ref[W], tot[W];
    pdl_trigger();
    pdl_wait();
    const int4* note = reinterpret_cast<const int4*>(a.ws + blockIdx.x * sizeof(AttSplit));
    const int4 n0 = __ldcg(note), n1 = __ldcg(note + 1);       // parts, b, hk, r0; rows, nb
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = blockIdx.y * (W / per) + warp / per, w = warp % per;
    if (n0.x == 0 || (int)blockIdx.y * (W / per) >= n1.x) return;   // CTA-uniform
    const int srows = min(block_rows, a.N * a.G);
    const size_t slot_floats = part_floats(srows, D);
    const float* slots = reinterpret_cast<const float*>(a.ws + kAttHead);
    float M = kNegInf, L = 0.f, v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.f;
    if (r < n1.x) {
        for (int p = w; p < n0.x; p += U * per) {
            float m[U], l[U], y[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = min(p + u * per, n0.x - 1);
                const float* at = slots + (size_t)(2 * ((int)blockIdx.x + q) + (q == 0 ? 1 : 0)) * slot_floats;
                m[u] = __ldcg(at + (size_t)srows * D + r);
                l[u] = __ldcg(at + (size_t)srows * (D + 1) + r);
                const float* z = at + (size_t)r * D + lane * VEC;
#pragma unroll
                for (int h = 0; h < V / VEC; ++h) {
                    if constexpr (VEC == 2) {
                        const float2 t = __ldcg(reinterpret_cast<const float2*>(z));
                        y[u][0] = t.x;
                        y[u][1] = t.y;
                    } else {
                        const float4 t = __ldcg(reinterpret_cast<const float4*>(z) + 32 * h);
                        y[u][4 * h] = t.x;
                        y[u][4 * h + 1] = t.y;
                        y[u][4 * h + 2] = t.z;
                        y[u][4 * h + 3] = t.w;
                    }
                }
            }
            float mx = M;
#pragma unroll
            for (int u = 0; u < U; ++u) mx = p + u * per < n0.x ? fmaxf(mx, m[u]) : mx;
            const float base = mx == kNegInf ? 0.f : mx;       // (no position seen yet)
            const float f = ex2_approx(M - base);
            M = mx;
            L *= f;
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] *= f;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p + u * per < n0.x) {                      // warp-uniform
                    const float fu = ex2_approx(m[u] - base);
                    L = fmaf(fu, l[u], L);
#pragma unroll
                    for (int e = 0; e < V; ++e) v[e] = fmaf(fu, y[u][e], v[e]);
                }
        }
    }
    if (per > 1) {                                             // the row's warps: CTA-uniform
#pragma unroll
        for (int h = 0; h < V / VEC; ++h)
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum[warp][h * 128 + lane * VEC + e] = v[h * VEC + e];
        if (lane == 0) {
            ref[warp] = M;
            tot[warp] = L;
        }
        __syncthreads();
        if (w > 0) return;
        for (int i = 1; i < per; ++i) M = fmaxf(M, ref[warp + i]);
        const float base = M == kNegInf ? 0.f : M;
        L = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = 0.f;
        for (int i = 0; i < per; ++i) {
            const float f = ex2_approx(ref[warp + i] - base);
            L = fmaf(f, tot[warp + i], L);
#pragma unroll
            for (int h = 0; h < V / VEC; ++h)
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[h * VEC + e] = fmaf(f, sum[warp + i][h * 128 + lane * VEC + e], v[h * VEC + e]);
        }
    }
    if (r >= n1.x) return;                                     // warp-uniform
    const float base = M == kNegInf ? 0.f : M;
    if constexpr (VEC == 2) {
        const float2 o = make_float2(__shfl_down_sync(0xffffffffu, v[0], 1), __shfl_down_sync(0xffffffffu, v[1], 1));
        if (!(lane & 1)) put_row(a, n0.y, n0.z, n0.w, n1.y, false, D, r, lane * 2, make_float4(v[0], v[1], o.x, o.y), L, base);
    } else {
#pragma unroll
        for (int h = 0; h < V / VEC; ++h)
            put_row(a, n0.y, n0.z, n0.w, n1.y, false, D, r, h * 128 + lane * 4,
                    make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]), L, base);
    }
}

// Short units are not worth splitting: the second launch, the parts, CTAs that begin
// two units.  How short depends on how many CTAs would have nothing to do (us whole /
// by tiles; 8 cached heads, 4 rows of 128, but for * 48 rows on the tcgen05 kernel, and for
// + 32 rows of 64): 8 units of 250 positions 6.6 / 6.9, of 380 8.1 / 7.1; 64 of 380 8.6 /
// 9.0 and * 13.3 / 19.7, of 630 11.5 / 10.6; 160 of 500 11.2 / 12.2, + 12.2 / 16.1, but *
// 28.1 / 25.8; 512 of 250 13.5 / 17.0, * 36.8 / 44.7, + 16.3 / 22.6, of 630 28.7 / 29.9, * 70.6
// / 73.2, + 25.9 / 32.7, of 1000 40.8 / 40.4, * 67.6 / 75.0, + 39.1 / 38.1.
// The positions are those that the block table has room for: the host does not know the
// lengths.  The rule does not ask which kernel runs; of these cases that costs
// * 160 units of 500.
bool attend_whole(long long units, long long positions, long long ctas) {
    return positions <= 256 || (positions <= 512 && 4 * units >= ctas) || (positions <= 768 && 2 * units >= 3 * ctas);
}

cudaError_t launch_join(const AttendArgs& a, int ctas, long long units, int block_rows, long long tiles, cudaStream_t st) {
    if (a.whole) return cudaSuccess;                           // no unit is split
    // about four parts a warp
    long long parts = ctas / units + 2;
    if (parts > tiles) parts = tiles;
    const int per = parts > 16 ? 8 : parts > 8 ? 4 : parts > 4 ? 2 : 1;
    const int rows = min(block_rows, a.N * a.G), rpc = kJoinThreads / 32 / per;
    const dim3 grid((unsigned)ctas, (unsigned)((rows + rpc - 1) / rpc));
    return a.c.head_dim == 64    ? launch_pdl(attend_join_kernel<64>, grid, kJoinThreads, 0, st, a, block_rows, per)
           : a.c.head_dim == 128 ? launch_pdl(attend_join_kernel<128>, grid, kJoinThreads, 0, st, a, block_rows, per)
                                 : launch_pdl(attend_join_kernel<256>, grid, kJoinThreads, 0, st, a, block_rows, per);
}

// Rows of a cached head that a unit holds, at most.
static int att_rows(int N, int G) { return N * G <= 16 ? 16 : 32; }   // (16 where elements are 256 and blocks few)

size_t attend_workspace_size(int B, int N, int Hq, int Hkv, int D) {
    // the join's notes, then two parts per CTA, for either kernel
    const int G = Hq / Hkv, rt = N * G, rows = att_rows(N, G);
    const size_t here = kAttHead + align256((size_t)2 * kAttMaxCtas * part_floats(rt < rows ? rt : rows, D) * 4);
    const size_t tc = attend_takes_tc(N, G, D, false, INT64_MAX, 0, 1) ? attend_tc_workspace(N, G) : 0;
    return here > tc ? here : tc;
}

template <int D, int MT, int RG, bool FP8>
static cudaError_t launch_attend_t(const AttendArgs& a, cudaStream_t st) {
    using C = AttCfg<D, MT, RG, FP8>;
    auto kfn = attend_kernel<D, MT, RG, FP8>;
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    static DeviceSlots slots = {};
    int occ = 0;
    e = device_once(slots, &occ, [&](int, int* o) {
        cudaError_t r = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (r != cudaSuccess) return r;
        r = cudaFuncSetAttribute(kfn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (r != cudaSuccess) return r;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(o, kfn, C::THREADS, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    const long long rb = ((long long)a.N * a.G + C::ROWS - 1) / C::ROWS;
    const long long most = ((long long)a.c.max_pages * a.c.page_size + C::TILE - 1) / C::TILE;   // tiles of a unit
    long long g = (long long)di.sm_count * occ;
    if (g > kAttMaxCtas) g = kAttMaxCtas;
    const long long units = (long long)a.B * a.c.kv_heads * rb;
    AttendArgs w = a;
    w.whole = most == 1 || attend_whole(units, (long long)a.c.max_pages * a.c.page_size, g);
    if (g > units * (w.whole ? 1 : most)) g = units * (w.whole ? 1 : most);
    e = launch_pdl(kfn, dim3((unsigned)g), C::THREADS, C::SMEM, st, w);
    return e != cudaSuccess ? e : launch_join(w, (int)g, units, C::ROWS, most, st);
}

template <int D, bool FP8>
static cudaError_t launch_attend_d(const AttendArgs& a, cudaStream_t st) {
    if (att_rows(a.N, a.G) == 16) return launch_attend_t<D, 1, 1, FP8>(a, st);
    if constexpr (D < 256) return launch_attend_t<D, 2, 1, FP8>(a, st);
    // Rows of 256 bf16 by two sets of warps where there are more blocks of 16 rows than
    // SMs, or more than 32 tiles for each SM: 190 us for 270 at 64 x 8 heads x 20 rows over
    // up to 2000, 88 for 118 at 10 x 8 x 285 rows over 69, 80 for 102 at 8 x 8 x 32 rows over
    // up to 8000, but 26.2 for 22.8 at 8 heads x 68 rows over 1930 (40 blocks of 31 tiles).
    // Of E4M3 rows two CTAs fit an SM as it is (202 for 196).
    if constexpr (D == 256 && !FP8) {
        DeviceInfo di;
        const cudaError_t e = device_info(&di);
        if (e != cudaSuccess) return e;
        const long long blocks = (long long)a.B * a.c.kv_heads * ((a.N * a.G + 15) / 16);
        const long long tiles = ((long long)a.c.max_pages * a.c.page_size + 63) / 64;
        if (blocks > di.sm_count || blocks * tiles > 32LL * di.sm_count) return launch_attend_t<D, 1, 2, FP8>(a, st);
    }
    if constexpr (D == 256) return launch_attend_t<D, 1, 1, FP8>(a, st);
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st) {
    const bool f8 = a.c.dtype == SPEC_DTYPE_E4M3;
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    if (attend_takes_tc(a.N, a.G, a.c.head_dim, f8, (long long)a.c.max_pages * a.c.page_size, (long long)a.B * a.c.kv_heads,
                        di.sm_count))
        return launch_attend_tc(a, st);
    switch (a.c.head_dim) {
        case 64: return f8 ? launch_attend_d<64, true>(a, st) : launch_attend_d<64, false>(a, st);
        case 128: return f8 ? launch_attend_d<128, true>(a, st) : launch_attend_d<128, false>(a, st);
        default: return f8 ? launch_attend_d<256, true>(a, st) : launch_attend_d<256, false>(a, st);
    }
}

}  // namespace sv
