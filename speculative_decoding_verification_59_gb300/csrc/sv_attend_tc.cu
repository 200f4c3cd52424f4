// Paged attention on the fifth-generation tensor cores, for heads of 128
// elements: the same units, shares and join as sv_attend.cu, with the two
// products as tcgen05.mma and the accumulators in tensor memory.
//
// Both products are taken transposed, so that the 128 positions of a tile and
// the 128 elements of a head are the 128 rows that the instruction wants, and the
// few query rows its free dimension N (a multiple of 16 up to 144):
//   S^T [positions x rows] = K [positions x 128] Q^T,
//   O^T [elements x rows] += V^T [elements x positions] P^T.
// K and V lie in shared memory as they come from the cache (128-byte swizzled
// rows of 64 elements); V is the transposed operand.  A thread of the softmax
// warps owns one position, that is one lane of tensor memory: its key and value
// scales are scalars, it reads its scores of all rows, and writes its
// probabilities as one row of P.
//
// The warps of a CTA, one CTA per SM, each walking the CTA's share:
//   softmax   4 warps, or two or three times 4 where there are more rows, each 4
//             with their share of them
//   MMA       2 threads: one issues the first product, one the second
//   loaders   4 warps bring the queries, and keys and values into a ring of buffers
//             each.  A tile of old positions whose pages fit it (page sizes that divide
//             128, from 8 on, or are multiples of it) comes by TMA, a box per page;
//             other page sizes, and the tiles with new positions, where stale
//             entries are left out, by the threads' 16-byte cp.async.
// An E4M3 cache is multiplied as it lies (kind::f8f6f4), the other operand split
// into e4m3 terms: two for a query (a bf16 significand has two e4m3 significands'
// bits), the second the rounding of 16 times what the first left over; four for a
// probability, each the rounding of 32 times what the one before left over (at
// most 8, of values up to 2^8), which hold what fp16 does, steps of 2^-24 included.
// The terms are columns of their own: S has two columns a row, O four, weighed 1,
// 2^-5, 2^-10, 2^-15 when they are read.  (Three terms have the significand's bits, but
// no steps below 2^-17, or 2^-19 at 32 times: one score far above thousands of others
// took the weight that those have together.  With references 2^4 below the rows' largest
// scores, three reach 2^-23 of those, but the references then move often: 105.3 us for 95.5
// with four, 91 with three and no such range, at 32 trees of 64 rows over up to 2048;
// 149 / 143.6 / 133 for 64 x 32 rows over up to 4000, 114.5 / 116 / 113.8 for 8 x 32 rows
// over up to 32768.  Widening the cache to fp16 in shared memory moved three times the
// bytes there and bound the kernel: 183 us for 8 x 32768 positions.)
// Scores pass through two buffers in tensor memory, so the next tile's first
// product runs beside this tile's softmax.
//
// The running reference m_r of a row is common to the CTA's positions, so a
// new one would need a maximum over 128 threads for every row and tile.  A tile
// only asks whether any score passes its row's reference by 2^8 (one maximum
// per score, one barrier vote); the rows' maxima, the new references and the
// rescaling of O run when one does: on a unit's first tile, and rarely after.
//
// Measured (lengths from half of the stated one to all of it, 8 cached heads):
//   64 sequences x 32 rows over 4096, bf16: 140 us, 5.8 TB/s of the cache's 812 MB, 86 % of
//     a plain copy's rate.  Memory bounds the tiles; what is left is units' begins and ends.
//   32 trees x 144 rows over 2048, bf16: 97.3 us, 305 TFLOP/s.  A tile's softmax is four
//     dependent steps, together 3900 cycles (the scores' wait 420, scores and vote 1270, P's
//     buffer 410, powers and P 1770: clock reads in a copy of the kernel), and a unit begins
//     and ends in some 13000.  In a seventh of their time warps wait for instructions.
//   8 sequences x 32 rows over 32768, E4M3: 112.4 us, 3.5 TB/s: the same softmax, 2800
//     cycles for a tile that the memory brings in 1400 (400, 790, 450, 1140).
#include <cuda.h>

#include "sv_attend.cuh"
#include "sv_tma.cuh"

namespace sv {

constexpr int kTcTile = 128;
constexpr int kTcD = 128;
// The loaders run at most 6 tiles ahead of the softmax (key buffers and two
// score buffers): scales are held for 7 tiles, what the loaders tell the
// softmax by unit for 8.
constexpr int kTcScaleRing = 7;
constexpr int kTcUnitRing = 8;
// Polls of a wait before it gives up, whatever larger bound is in force: a poll
// sleeps for up to some ten microseconds here, and no wait of this kernel lasts
// longer than the memory takes to answer.
constexpr uint32_t kTcWaitLimit = 1u << 18;
constexpr int kTcMaxCtas = 256;
static_assert(kTcMaxCtas <= kAttMaxCtas, "a note for each");
constexpr float kNoRef = -1e30f;                 // reference of a row that has seen no position

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

template <int CH, int NSM, bool FP8>
struct TcCfg {
    static constexpr int COLS = CH * 16;         // rows of a softmax warpgroup
    static constexpr int RP = NSM * COLS;        // rows of a unit, at most
    static constexpr int BUF = kTcTile * kTcD * (FP8 ? 1 : 2);   // a tile's keys or values
    static constexpr int QT = FP8 ? 2 : 1, PT = FP8 ? 4 : 1;     // terms of a query, of a probability
    static constexpr int PROWS = FP8 ? 128 : 64; // columns of P in 128 bytes
    static constexpr int PB = (PT * RP + PROWS - 1) / PROWS;     // blocks of them
    static constexpr int QB = FP8 || RP == 64 ? 2 : 1;          // units whose queries are held
    // buffers of keys, of values (32 bf16 rows: a third of keys in the place of other
    // queries, 140 us for 143 at 64 x 32 rows over up to 4096)
    static constexpr int KB = FP8 ? 4 : RP > 32 ? 2 : 3;
    static constexpr int VB = FP8 ? (RP > 32 ? 4 : 5) : RP > 64 ? 2 : 3;
    static constexpr int S_COLS = QT * RP;       // columns of tensor memory: scores, sums
    static constexpr int O_AT = 2 * S_COLS, T_COLS = O_AT + PT * RP;
    static constexpr int WORDS = (COLS + 31) / 32;   // a bit for each row of a warpgroup
    // Up to 32 rows the scores stay in registers between the vote and the
    // probabilities, beside as many running totals; beyond, they are read from
    // tensor memory twice.
    static constexpr bool KEEP = CH <= 2;
    static constexpr int SM_THREADS = NSM * 128;
    // loader warps: 4, or 2 where that leaves the softmax's twelve warps 128 registers
    // a thread (18 warps count as 20: 96)
    static constexpr int LW = NSM == 3 ? 2 : 4;
    static constexpr int LOADERS = LW * 32;
    static constexpr int THREADS = SM_THREADS + 64 + LOADERS;
    static constexpr int V_OFF = KB * BUF;
    static constexpr int P_OFF = V_OFF + VB * BUF;
    static constexpr int Q_OFF = P_OFF + PB * 16384;
    static constexpr int QBYTES = RP * 256;      // bf16: two blocks of half rows; E4M3: two terms
    static constexpr int SCALE_OFF = Q_OFF + QB * QBYTES;
    static constexpr int SMEM = SCALE_OFF + (FP8 ? kTcScaleRing * 2 * kTcTile * 4 : 0) + 1024;   // and room to align
    static_assert(SMEM <= 227 * 1024, "dynamic shared memory");
    static_assert(T_COLS <= 512, "tensor memory");
    static constexpr int TMEM = T_COLS <= 64 ? 64 : T_COLS <= 128 ? 128 : T_COLS <= 256 ? 256 : 512;
};

// ---- tcgen05 in inline PTX ------------------------------------------------------
__device__ __forceinline__ void tc_alloc(uint32_t* dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(uint32_t at, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}
template <bool F8>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (F8)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
}
// Arrives on the barrier when every tcgen05.mma issued so far has completed.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 16 columns of the warp's 32 lanes.
__device__ __forceinline__ void tc_ld16(uint32_t at, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// The same, the wait left to the caller (tc_wait_ld, then tc_ld16_done: nothing
// may use the registers before).
__device__ __forceinline__ void tc_ld16_start(uint32_t at, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
          "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(at));
}
__device__ __forceinline__ void tc_ld16_done(float* v) {
    asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}
__device__ __forceinline__ void tc_ld8(uint32_t at, float (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(at));
    tc_wait_ld();
    asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]));
}
__device__ __forceinline__ void tc_st16(uint32_t at, const float (&v)[16]) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
        : "memory");
    tc_wait_st();
}

// The box from `slot` (a multiple of 8) of a page's head (entry `place` of the map)
// into shared memory.
template <bool FP8>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int slot, int place, uint64_t* bar) {
    if constexpr (FP8)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(map), "r"(0), "r"(slot), "r"(place), "r"(smem_addr(bar))
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], [%5];" ::"r"(dst),
            "l"(map), "r"(0), "r"(slot >> 3), "r"(place), "r"(smem_addr(bar))
            : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}

// Shared-memory operand with 128-byte swizzled rows.  K-major (the contraction
// contiguous): sbo is the step between groups of 8 rows.  MN-major: lbo the step
// between blocks of 128 bytes of the other dimension, sbo between groups of 8
// steps of the contraction.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// Instruction descriptor: fp32 accumulators, both operands bf16 (or e4m3),
// M = 128, N = n; ta / tb: that operand is MN-major.
__device__ __forceinline__ uint32_t tc_idesc(bool e4m3, bool ta, bool tb, int n) {
    const uint32_t t = e4m3 ? 0u : 1u;
    return 1u << 4 | t << 7 | t << 10 | (uint32_t)ta << 15 | (uint32_t)tb << 16 | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_any(int id, int threads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}

// Arrives on the barrier when the thread's cp.asyncs so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Byte offset of 16-byte chunk c of row t in a tile: groups of 8 rows, in each the
// 128-byte swizzled rows (bf16: first halves, then second halves, so that a page comes
// in one box: with a box for each half, pages of 16 took 158 us for 64 x 32 rows over
// up to 4096, those of 8 190).
template <bool FP8>
__device__ __forceinline__ int tc_off(int t, int c) {
    if constexpr (FP8) return t * 128 + ((c ^ (t & 7)) << 4);
    else return (t >> 3) * 2048 + (c >> 3) * 1024 + (t & 7) * 128 + (((c & 7) ^ (t & 7)) << 4);
}

// A pair of bf16 values with infinities and NaN set to zero.
__device__ __forceinline__ uint32_t drop_odd_bf16(uint32_t y) {
    if ((y & 0x7f80u) == 0x7f80u) y &= 0xffff0000u;
    if ((y & 0x7f800000u) == 0x7f800000u) y &= 0xffffu;
    return y;
}

// Four e4m3 values with NaN set to zero.
__device__ __forceinline__ uint32_t drop_odd_e4m3(uint32_t y) {
#pragma unroll
    for (int s = 0; s < 32; s += 8)
        if (((y >> s) & 0x7fu) == 0x7fu) y &= ~(0xffu << s);
    return y;
}

// The e4m3 rounding of a pair, which is replaced by sixteen times what that
// leaves over.
__device__ __forceinline__ uint32_t e4m3_term(float& a, float& b) {
    const uint32_t t = pack_e4m3(a, b);
    float x, y;
    f16x2_to_f32(e4m3_to_f16x2(t), &x, &y);
    a = (a - x) * 16.f;
    b = (b - y) * 16.f;
    return t;
}

// The same of a pair of fp16 values (both steps are exact there): their e4m3
// roundings, and 32 times what those leave over.
__device__ __forceinline__ uint32_t e4m3_of_f16x2(uint32_t p) {
    unsigned short t;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(t) : "r"(p));
    return t;
}
__device__ __forceinline__ uint32_t left_over_f16x2(uint32_t p, uint32_t t) {
    uint32_t r;
    asm("{\n\t.reg .b32 d;\n\tsub.f16x2 d, %1, %2;\n\tmul.f16x2 %0, d, %3;\n\t}" : "=r"(r) : "r"(p), "r"(e4m3_to_f16x2(t)), "r"(0x50005000u));
    return r;
}

struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Add {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// Reduces 16 columns over the warp's lanes in 16 shuffles: halving the columns
// a lane still holds at each step.  Both lanes of a pair end with the result
// of column fold_column(lane).
template <typename Op>
__device__ __forceinline__ float fold16(float (&v)[16], int lane, Op op) {
#pragma unroll
    for (int h = 8; h >= 1; h >>= 1) {
        const bool high = lane & (2 * h);
#pragma unroll
        for (int j = 0; j < h; ++j) {
            const float give = high ? v[j] : v[j + h], keep = high ? v[j + h] : v[j];
            v[j] = op(keep, __shfl_xor_sync(0xffffffffu, give, 2 * h));
        }
    }
    return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}
__device__ __forceinline__ int fold_column(int lane) { return lane >> 1; }

template <int CH, int NSM, bool FP8>
__global__ void __launch_bounds__(TcCfg<CH, NSM, FP8>::THREADS, 1) attend_tc_kernel(const AttendArgs a, int block_rows, int rp, int box, int page_places, int head_places, uint32_t limit, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
    using C = TcCfg<CH, NSM, FP8>;
    constexpr int RP = C::RP, KB = C::KB, VB = C::VB;
    extern __shared__ unsigned char smem_raw[];
    __shared__ AttPlan plan;
    __shared__ __align__(8) uint64_t k_full[KB], k_empty[KB], v_full[VB], v_empty[VB], s_full[2], s_free[2], p_full, pv_done,
        q_full[C::QB], q_free[C::QB], drained[2];
    __shared__ __align__(16) float nref[RP], alpha[RP];        // minus the rows' references; the rescaling
    __shared__ float wred[NSM * 4][C::COLS];
    __shared__ short rown[RP];                                  // new position of a row
    __shared__ __align__(16) int rowat[RP];                                   // its row of the output, from the sequence's first
    __shared__ unsigned long long anc[NSM][2][kMaxNewTree];    // trees: ancestors and itself, by node
    __shared__ short up[NSM][2][kMaxNewTree];
    __shared__ uint32_t vis[NSM][kMaxNewTree][C::WORDS];       // trees: the warpgroup's rows that see a node
    __shared__ uint32_t tmem_at;
    __shared__ int unit_bad[NSM][kTcUnitRing];                  // a page that is none
    __shared__ __align__(16) float qinv[4][FP8 ? RP : 4];       // E4M3: by unit, what takes back a row's scaling
    __shared__ int odd_any, tree_bad[NSM];
    unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kMmaWarp = C::SM_THREADS / 32;

    if (tid == 0) {
        for (int i = 0; i < KB; ++i) {
            mbar_init(&k_full[i], C::LOADERS);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < VB; ++i) {
            mbar_init(&v_full[i], C::LOADERS);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(&drained[0], 1);
        mbar_init(&drained[1], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], C::SM_THREADS / 32);
        }
        mbar_init(&p_full, C::SM_THREADS / 32);
        mbar_init(&pv_done, 1);
        for (int i = 0; i < C::QB; ++i) {
            mbar_init(&q_full[i], FP8 ? C::LOADERS / 32 : C::LOADERS);
            mbar_init(&q_free[i], 1);
        }
        mbar_init_fence();
        odd_any = 0;
        for (int i = 0; i < NSM * kTcUnitRing; ++i) unit_bad[0][i] = 0;
    }
    if (warp == kMmaWarp) tc_alloc(&tmem_at, C::TMEM);
    pdl_trigger();
    pdl_wait();
    const int RB = (a.N * a.G + block_rows - 1) / block_rows;
    tc_before();
    make_plan<kTcTile, C::THREADS>(a, a.c.kv_heads * RB, gridDim.x, &plan);   // ends in a barrier
    tc_after();
    const uint32_t tmem = tmem_at;
    AttWalk walk;
    AttUnit un;
    if ((int)blockIdx.x < plan.n) {
        walk.init(plan);
    } else {
        walk.t = walk.end = 0;
        walk.seq_at = 0;
        walk.b = 0;
    }

    if (warp > kMmaWarp + 1) {
        // ================= loaders =================
        const int lt = tid - C::SM_THREADS - 64, lw = lt >> 5;
        constexpr int RS = 4 / C::LW;                          // sets of 32 rows of a warp: rows (h LW + lw) 32 ..
        constexpr int CPR = FP8 ? 8 : 16;                      // 16-byte chunks of a cached row
        constexpr int RPI = 32 / CPR;                          // rows a warp copies at once
        constexpr int PIECES = 32 / RPI;                       // 32 rows: pieces of 16 bytes a thread
        const int ch = lane % CPR, sub = lane / CPR;
        bool ok = true;
        unsigned t = 0;                                        // tiles issued
        unsigned uc = 0;                                       // units
        while (ok && walk.next<kTcTile>(a, RB, block_rows, &un)) {
            // ---- the block table's entries, their loads under way beside the queries'
            auto by_tma = [&](int i) { return box > 0 && (i + 1) * kTcTile <= min(un.sl.ctx, un.sl.total); };
            auto table = [&](int pg) {                          // entry pg of the sequence's row; -1 past it
                return pg < a.c.max_pages ? __ldg(a.c.block_table + (size_t)un.b * a.c.max_pages + pg) : -1;
            };
            // What TMA tiles need of the block table is loaded for 32 boxes at once, a
            // group before it is used: lane l holds box l of the group (a load of
            // its own before each tile cost 1400 cycles a tile).
            const int boxes = box > 0 ? kTcTile / box : 1;      // a tile's: 1, 2, .. 16
            const int group = 32 / boxes;                       // tiles of a group
            auto group_page = [&](int i0) {                     // group of tiles from i0 on
                int slot;
                const int pos = i0 * kTcTile + lane * box;
                return box > 0 && pos + box <= min(un.sl.ctx, un.sl.total) ? table(page_index(a, pos, &slot)) : -1;
            };
            int g0 = un.ta, pages = group_page(g0), pages_next = group_page(g0 + group);
            // The other tiles: lane l finds row l of each of the warp's sets, one tile ahead (E4M3: of
            // every tile, for the scales).
            auto row_page = [&](int i, int h, int* slot) {
                const int pos = i * kTcTile + (h * C::LW + lw) * 32 + lane;
                *slot = 0;
                return pos < un.sl.total ? table(page_index(a, pos, slot)) : -2;      // -2: no position
            };
            auto by_row = [&](int i) { return i < un.tb && (!by_tma(i) || FP8); };
            int rpage[RS], rslot[RS];
#pragma unroll
            for (int h = 0; h < RS; ++h) {
                rpage[h] = -2;
                rslot[h] = 0;
                if (by_row(un.ta)) rpage[h] = row_page(un.ta, h, &rslot[h]);
            }
            // ---- the unit's queries.  bf16: behind its first keys, which wait for nothing that the
            // unit before still has to do, and the thread goes on while the copies are under
            // way (before them and through registers, 144 rows kept the loaders for 8000
            // cycles a unit).  E4M3: through registers, in terms (few rows; among the tiles'
            // code, that of every tile was slower: 133 us for 111 at 8 x 32768 positions, with
            // three terms of the probabilities).
            auto queries = [&] {
                const int qb = (int)(uc % C::QB);
                if (uc >= (unsigned)C::QB && !wait_bounded(&q_free[qb], (uc / C::QB - 1) & 1u, limit)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                unsigned char* qs = smem + C::Q_OFF + qb * C::QBYTES;
                auto query_row = [&](int r) {
                    const int R = un.r0 + r, n = row_position(a, R), g = R - n * a.G;
                    return a.q + ((int64_t)un.b * a.N + n) * a.qs + ((size_t)un.hk * a.G + g) * kTcD * 2;
                };
                if constexpr (!FP8) {
                    const uint32_t to = smem_addr(qs) + (lt >> 3 & 1) * (RP * 128);
#pragma unroll 4
                    for (int r = lt >> 4; r < rp; r += C::LOADERS / 16)
                        cp16(to + r * 128 + (((lt & 7) ^ (r & 7)) << 4), query_row(min(r, un.rows - 1)) + (lt & 15) * 16, r < un.rows);
                    cp_arrive(&q_full[qb]);
                } else {
                    constexpr int QK = 6;                      // loads of a thread in flight
                    for (int i0 = lt; i0 < rp * 16; i0 += C::LOADERS * QK) {
                        uint4 w[QK];
#pragma unroll
                        for (int k = 0; k < QK; ++k) {
                            const int i = i0 + C::LOADERS * k, r = i >> 4;
                            w[k] = r < un.rows ? __ldg(reinterpret_cast<const uint4*>(query_row(r)) + (i & 15)) : make_uint4(0u, 0u, 0u, 0u);
                        }
#pragma unroll
                        for (int k = 0; k < QK; ++k) {
                            const int i = i0 + C::LOADERS * k, r = i >> 4, c16 = i & 15;
                            // the row's 16 lanes find the power of two that brings its largest
                            // element into [2^7, 2^8), and write its two terms
                            float x[8], mx = 0.f;
                            unpack8(w[k], x);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                if (!(fabsf(x[j]) < CUDART_INF_F)) x[j] = CUDART_NAN_F;        // (e4m3 has no infinity)
                                else mx = fmaxf(mx, fabsf(x[j]));
                            }
#pragma unroll
                            for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                            const int ex = (int)(__float_as_uint(mx) >> 23), sh = ex < 24 || ex > 240 ? 0 : 134 - ex;
                            const float f = __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
                            for (int j = 0; j < 8; ++j) x[j] *= f;
                            uint2 term[2];
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                term[q].x = e4m3_term(x[0], x[1]);
                                term[q].x |= e4m3_term(x[2], x[3]) << 16;
                                term[q].y = e4m3_term(x[4], x[5]);
                                term[q].y |= e4m3_term(x[6], x[7]) << 16;
                            }
                            if (r < rp) {
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    const int at = q * rp + r;
                                    *reinterpret_cast<uint2*>(qs + at * 128 + (((c16 >> 1) ^ (at & 7)) << 4) + (c16 & 1) * 8) = term[q];
                                }
                                if (c16 == 0) qinv[uc & 3][r] = __uint_as_float((uint32_t)(127 - sh) << 23);
                            }
                        }
                    }
                    proxy_fence();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&q_full[qb]);
                }
            };

            if constexpr (FP8) queries();

            // ---- the unit's tiles
            for (int i = un.ta; i < un.tb && ok; ++i) {
                const bool tma = by_tma(i);
                int at_page = 0, at_slot = 0;                   // TMA: the lane's box
                bool lost = false;
                if (tma) {
                    if (i == g0 + group) {
                        g0 = i;
                        pages = pages_next;
                        pages_next = group_page(g0 + group);
                    }
                    at_page = __shfl_sync(0xffffffffu, pages, ((i - g0) * boxes + lane) & 31);
                    if (box == kTcTile) page_index(a, i * kTcTile, &at_slot);       // a page may hold several tiles
                    lost = lane < boxes && (unsigned)at_page >= (unsigned)a.c.num_pages;
                    if (lost) at_page = 0;                      // the unit ends as NaN anyway
                }
                int64_t off[RS], so[RS];                        // the lane's rows and scales
                unsigned havem[RS];
                bool scaled[RS];
#pragma unroll
                for (int h = 0; h < RS; ++h) {
                    scaled[h] = (unsigned)rpage[h] < (unsigned)a.c.num_pages;
                    lost |= !tma && !scaled[h] && rpage[h] != -2;
                    off[h] = scaled[h] && !tma ? entry_off(a.c, rpage[h], rslot[h], un.hk) : 0;
                    so[h] = FP8 && scaled[h] ? scale_off(a.c, rpage[h], rslot[h], un.hk) : 0;
                    havem[h] = __ballot_sync(0xffffffffu, scaled[h]);
                    rpage[h] = -2;
                    if (by_row(i + 1)) rpage[h] = row_page(i + 1, h, &rslot[h]);
                }
                if (__any_sync(0xffffffffu, lost) && lane == 0) {
#pragma unroll
                    for (int w = 0; w < NSM; ++w) unit_bad[w][uc % kTcUnitRing] = 1;
                    raise_error(a.c.error, SPEC_DEVERR_CACHE_RANGE);
                }
                for (int kv = 0; kv < 2; ++kv) {
                    if (!FP8 && kv == 1 && i == un.ta) queries();
                    // The buffer, once it is free.  Every warp waits for every buffer of its
                    // kind and arrives for it, the ones that have no part in a TMA tile too: a
                    // barrier tells its last two phases apart, no more, so none may
                    // fall behind or run ahead.
                    const unsigned n = kv ? VB : KB;
                    if (ok && lane == 0 && t >= n) ok = wait_bounded(kv ? &v_empty[t % VB] : &k_empty[t % KB], (t / n - 1) & 1u, limit);
                    const uint32_t dst = smem_addr(smem + (kv ? C::V_OFF + (t % VB) * C::BUF : (t % KB) * C::BUF));
                    uint64_t* bar = kv ? &v_full[t % VB] : &k_full[t % KB];
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    if (tma) {
                        if (lw == kv) {                         // one warp issues the keys, one the values
                            if (lane == 0) mbar_expect(bar, C::BUF);
                            __syncwarp();
                            if (lane < boxes) {
                                const CUtensorMap* map = kv ? &vmap : &kmap;
                                tma_load<FP8>(dst + lane * box * (FP8 ? 128 : 256), map, at_slot, at_page * page_places + un.hk * head_places, bar);
                            }
                            __syncwarp();
                        }
                    } else {
                        const char* base = static_cast<const char*>(kv ? a.c.v : a.c.k);
#pragma unroll
                        for (int h = 0; h < RS; ++h)
#pragma unroll
                            for (int p = 0; p < PIECES; ++p) {
                                const int wr = p * RPI + sub, row = (h * C::LW + lw) * 32 + wr;
                                const int64_t e = __shfl_sync(0xffffffffu, off[h], wr) * (FP8 ? 1 : 2) + ch * 16;
                                cp16(dst + tc_off<FP8>(row, ch), base + e, (havem[h] >> wr) & 1u);
                            }
                    }
                    bool copies = !tma;                         // the threads have copies of their own in flight
                    if constexpr (FP8) {
                        if (kv == 0) {                          // both scales: the softmax wants them with the scores
#pragma unroll
                            for (int h = 0; h < RS; ++h) {
                                const uint32_t at = smem_addr(smem + C::SCALE_OFF) +
                                                    ((t % kTcScaleRing) * 2 * kTcTile + (h * C::LW + lw) * 32 + lane) * 4;
                                cp4(at, a.c.k_scale + so[h], scaled[h]);
                                cp4(at + kTcTile * 4, a.c.v_scale + so[h], scaled[h]);
                            }
                            copies = true;
                        }
                    }
                    if (copies) cp_arrive(bar);                 // when this thread's copies have landed
                    else if (lane == 0) mbar_arrive_n(bar, 32);
                }
                if (!ok) break;
                ++t;
            }
            ++uc;
        }
        // ---- the tiles still in flight
        cp_wait<0>();
        if (!ok) {
            // a wait ran out: do not leave while a box may still be on its way
            raise_error(a.c.error, SPEC_DEVERR_TIMEOUT);
            if (lt == 0) {
                for (unsigned j = t > KB ? t - KB : 0u; j <= t; ++j)
                    wait_bounded(&k_full[j % KB], (j / KB) & 1u, j < t ? kTcWaitLimit : 1u << 8);
                for (unsigned j = t > VB ? t - VB : 0u; j <= t; ++j)
                    wait_bounded(&v_full[j % VB], (j / VB) & 1u, j < t ? kTcWaitLimit : 1u << 8);
            }
        }
    } else if (warp >= kMmaWarp) {
        // ================= the products =================
        // One thread of the first warp issues S = K Q, one of the second O += V P, so that
        // neither waits for the other's operands.  A step of an operand in bytes
        // is a sixteenth of it in its descriptor.
        if (lane == 0) {
            const bool second = warp > kMmaWarp;
            const uint32_t base = smem_addr(smem);
            const uint32_t id = second ? tc_idesc(FP8, true, true, C::PT * rp) : tc_idesc(FP8, false, false, C::QT * rp);
            constexpr uint32_t GROUP = FP8 ? 1024 : 2048;          // 8 positions of a tile
            const uint64_t a_d = second ? tc_desc(base + C::V_OFF, 1024, GROUP) : tc_desc(base, 16, GROUP);
            const uint64_t b_d = second ? tc_desc(base + C::P_OFF, 16384, 1024) : tc_desc(base + C::Q_OFF, 16, 1024);
            bool ok = true;
            unsigned g = 0, uc = 0;                            // tiles, units
            while (ok && walk.next<kTcTile>(a, RB, block_rows, &un)) {
                const unsigned qb = uc % C::QB;
                for (int i = un.ta; i < un.tb && ok; ++i, ++g) {
                    // the threads' own cp.asyncs arrived by themselves, unfenced
                    const bool fence = !(box > 0 && (i + 1) * kTcTile <= min(un.sl.ctx, un.sl.total));
                    if (!second) {
                        if (i == un.ta) ok = wait_bounded(&q_full[qb], (uc / C::QB) & 1u, limit);
                        if (ok) ok = wait_bounded(&k_full[g % KB], (g / KB) & 1u, limit);
                        if (ok && g >= 2) ok = wait_bounded(&s_free[g & 1], ((g >> 1) - 1) & 1u, limit);
                        if (!ok) break;
                        if (fence || i == un.ta) proxy_fence();
                        tc_after();
                        const uint64_t kd = a_d + (g % KB) * (C::BUF / 16), qd = b_d + qb * (C::QBYTES / 16);
                        const uint32_t at = tmem + (g & 1) * C::S_COLS;
#pragma unroll
                        for (int ks = 0; ks < C::BUF / 4096; ++ks)              // 32 bytes of a row at a time
                            tc_mma<FP8>(at, kd + ((ks >> 2) * 64 + (ks & 3) * 2), qd + ((ks >> 2) * (RP * 8) + (ks & 3) * 2), id, ks > 0);
                        tc_commit(&s_full[g & 1]);
                        tc_commit(&k_empty[g % KB]);
                        if (i + 1 == un.tb) tc_commit(&q_free[qb]);
                    } else {
                        ok = wait_bounded(&v_full[g % VB], (g / VB) & 1u, limit);
                        if (ok) ok = wait_bounded(&p_full, g & 1u, limit);
                        if (!ok) break;
                        if (fence) proxy_fence();
                        tc_after();
                        const uint64_t vd = a_d + (g % VB) * (C::BUF / 16);
                        constexpr int VS = 256, PS = FP8 ? 256 : 128;   // 32 (16) positions, in 16 bytes
#pragma unroll
                        for (int ks = 0; ks < (FP8 ? 4 : 8); ++ks)
                            tc_mma<FP8>(tmem + C::O_AT, vd + ks * VS, b_d + ks * PS, id, ks > 0 || i > un.ta);
                        tc_commit(&pv_done);
                        tc_commit(&v_empty[g % VB]);
                    }
                }
                ++uc;
            }
            if (second) {
                while (walk.next<kTcTile>(a, RB, block_rows, &un)) {}          // (a wait ran out)
                note_split(a, plan, un);
            }
            // every product must have ended before tensor memory is given back
            tc_commit(&drained[second]);
            if (!wait_bounded(&drained[second], 0, kTcWaitLimit) || !ok) raise_error(a.c.error, SPEC_DEVERR_TIMEOUT);
        }
        __syncwarp();
    } else {
        // ================= softmax =================
        const int wg = NSM > 1 ? warp >> 2 : 0;
        const int row = tid & 127;                             // position of a tile; element of a head
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        const int c0 = wg * C::COLS;                           // first row of the warpgroup
        const int chunks = min(CH, max(0, (rp - c0 + 15) / 16));
        const int bar = 1 + wg;
        float* slots = reinterpret_cast<float*>(a.ws + kAttHead);
        const int srows = min(block_rows, a.N * a.G);
        const size_t slot_floats = part_floats(srows, kTcD);
        unsigned g = 0, uc = 0;
        int tree_b = -1;
        bool dead = false;                                     // a wait ran out: the same for the warpgroup,
        bool late = false;                                     // once it has voted on this
        float l[CH * 16];
        while (walk.next<kTcTile>(a, RB, block_rows, &un)) {
            const SeqLen& sl = un.sl;
            // ---- the unit's rows, and who sees whom
            named_sync(bar, 128);                              // the unit before is done with the tables
            if (row < C::COLS) {
                const int R = un.r0 + min(c0 + row, un.rows - 1), n = row_position(a, R);
                rown[c0 + row] = (short)n;
                rowat[c0 + row] = n * a.Hq + un.hk * a.G + (R - n * a.G);
                nref[c0 + row] = -kNoRef;
            }
            if (a.par && (tree_b != un.b || RB > 1)) {
                // ancestors by pointer doubling: 2^6 steps cover any path of 64 nodes
                int wrong = 0;
                if (row == 0) tree_bad[wg] = 0;
                if (row < a.N) {
                    const int p = __ldg(a.par + (size_t)un.b * a.N + row);
                    wrong = row < sl.nb && (row == 0 ? p != -1 : (p < 0 || p >= row));
                    anc[wg][0][row] = 1ull << row;
                    up[wg][0][row] = (short)(wrong || row == 0 || row >= sl.nb ? -1 : p);
                }
                named_sync(bar, 128);
                for (int k = 0; k < 6; ++k) {
                    if (row < a.N) {
                        const int p = up[wg][k & 1][row];
                        anc[wg][(k + 1) & 1][row] = anc[wg][k & 1][row] | (p >= 0 ? anc[wg][k & 1][p] : 0ull);
                        up[wg][(k + 1) & 1][row] = p >= 0 ? up[wg][k & 1][p] : (short)-1;
                    }
                    named_sync(bar, 128);
                }
                for (int i = row; i < kMaxNewTree * C::WORDS; i += 128) {
                    const int node = i / C::WORDS, w = i - node * C::WORDS;
                    uint32_t bits = 0u;
                    for (int k = 0; k < 32 && w * 32 + k < C::COLS; ++k)
                        bits |= (uint32_t)((anc[wg][0][rown[c0 + w * 32 + k]] >> node) & 1ull) << k;
                    vis[wg][node][w] = bits;
                }
                if (wrong) {
                    tree_bad[wg] = 1;
                    raise_error(a.c.error, SPEC_DEVERR_TREE_PARENT);
                }
                tree_b = un.b;
            }
            if (sl.bad && tid == 0) raise_error(a.c.error, SPEC_DEVERR_CACHE_RANGE);
            const float c2 = a.scale * kLog2e;
#pragma unroll
            for (int j = 0; j < CH * 16; ++j) l[j] = 0.f;
            named_sync(bar, 128);

            for (int i = un.ta; i < un.tb && !dead; ++i, ++g) {
                const int p0 = i * kTcTile, pos = p0 + row;
                const bool masked = p0 + kTcTile > sl.ctx;     // uniform: new positions, or past the end
                const int d = pos - sl.ctx;
                const bool gone = pos >= sl.total;
                // the warpgroup's rows that see this position, a bit each
                uint32_t sees[C::WORDS];
#pragma unroll
                for (int w = 0; w < C::WORDS; ++w) {
                    sees[w] = gone ? 0u : 0xffffffffu;
                    if (masked && d >= 0 && !gone) {
                        if (a.par) {
                            sees[w] = vis[wg][d & 63][w];
                        } else {                               // a chain: rows d G and up of the cached head
                            const int from = d * a.G - un.r0 - c0 - w * 32;
                            sees[w] = from <= 0 ? 0xffffffffu : from >= 32 ? 0u : 0xffffffffu << from;
                        }
                    }
                }
                bool ok = wait_bounded(&s_full[g & 1], (g >> 1) & 1u, limit);
                ok = __all_sync(0xffffffffu, ok);
                tc_after();
                float f = c2, add = 0.f, vinv = 0.f;
                if constexpr (FP8) {
                    const float* sc = reinterpret_cast<const float*>(smem + C::SCALE_OFF) + (g % kTcScaleRing) * 2 * kTcTile;
                    f = c2 * sc[row];
                    const float vs = value_scale(sc[kTcTile + row]);
                    add = __log2f(vs);
                    vinv = fabsf(vs) < CUDART_INF_F ? 1.f / vs : 0.f;         // (of a masked position it may be anything)
                }
                // The score of the warpgroup's row k in powers of two, plus nr (less its
                // reference).  The tiles that hold new positions, or the end, are masked;
                // the others run without.
                // Two rows an instruction.
                const f32x2 ff = f2_pack(f, f), aa = f2_pack(add, add);
                auto arg = [&](auto mask, float& s0, float& s1, int k, float nr0, float nr1) {
                    f32x2 r = f2_pack(nr0, nr1);
                    if constexpr (FP8) r = f2_add(r, aa);
                    f2_unpack(f2_fma(f2_pack(s0, s1), ff, r), s0, s1);
                    if constexpr (decltype(mask)::value) {
                        if (!((sees[k >> 5] >> (k & 31)) & 1u)) s0 = kNegInf;
                        if (!((sees[k >> 5] >> ((k + 1) & 31)) & 1u)) s1 = kNegInf;
                    }
                };
                const uint32_t s_at = lanes + (g & 1) * C::S_COLS + c0;
                const float* qf = qinv[uc & 3];
                // Reads the scores two chunks (E4M3: a chunk's two terms) at a time, takes them relative to the references
                // and gives them to `use(first row, 16 values)`.
                auto each = [&](auto mask, auto use) {
#pragma unroll
                    for (int cc = 0; cc < CH; cc += FP8 ? 1 : 2) {
                        if (cc < chunks) {
                        float v[2][16];
                        const bool two = !FP8 && cc + 1 < CH; // (a second chunk past the unit's rows is read and left)
                        tc_ld16_start(s_at + cc * 16, v[0]);
                        if (two || FP8) tc_ld16_start(s_at + (FP8 ? rp + cc * 16 : cc * 16 + 16), v[1]);
                        tc_wait_ld();
                        tc_ld16_done(v[0]);
                        if (two || FP8) tc_ld16_done(v[1]);
                        if constexpr (FP8) {                   // the two terms, and the row's scaling
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float4 q = *reinterpret_cast<const float4*>(&qf[c0 + cc * 16 + j]);
                                const f32x2 w = f2_pack(0.0625f, 0.0625f);
                                f2_unpack(f2_mul(f2_fma(f2_pack(v[1][j], v[1][j + 1]), w, f2_pack(v[0][j], v[0][j + 1])), f2_pack(q.x, q.y)),
                                          v[0][j], v[0][j + 1]);
                                f2_unpack(f2_mul(f2_fma(f2_pack(v[1][j + 2], v[1][j + 3]), w, f2_pack(v[0][j + 2], v[0][j + 3])), f2_pack(q.z, q.w)),
                                          v[0][j + 2], v[0][j + 3]);
                            }
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (h == 0 || (two && cc + 1 < chunks)) {
#pragma unroll
                                for (int j = 0; j < 16; j += 4) {
                                    const int k = (cc + h) * 16 + j;
                                    const float4 nr = *reinterpret_cast<const float4*>(&nref[c0 + k]);
                                    arg(mask, v[h][j], v[h][j + 1], k, nr.x, nr.y);
                                    arg(mask, v[h][j + 2], v[h][j + 3], k + 2, nr.z, nr.w);
                                }
                                use((cc + h) * 16, v[h]);
                            }
                        }
                    }
                };
                float x[C::KEEP ? CH * 16 : 1];
                auto score_all = [&](auto mask) {
                    float top = kNegInf;
                    each(mask, [&](int k0, const float (&v)[16]) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            top = fmaxf(top, fmaxf(fmaxf(v[j], v[j + 1]), fmaxf(v[j + 2], v[j + 3])));
                            if constexpr (C::KEEP) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) x[k0 + j + e] = v[j + e];
                            }
                        }
                    });
                    return top;
                };
                // (up to 32 rows all tiles take the masked code: the few instructions it
                // costs are not missed, those of a second copy would be)
                const float top = C::KEEP || masked ? score_all(Yes{}) : score_all(No{});
                const bool first = i == un.ta;
                ok = ok && !late;
                if (named_any(bar, 128, !ok || top > kRefSlack)) {
                    // ---- new references (or a wait that ran out)
                    if (!first && ok) ok = wait_bounded(&pv_done, (g - 1) & 1u, limit);    // O is at rest
                    if (named_any(bar, 128, !ok)) {
                        dead = true;
                        break;
                    }
                    tc_after();
                    for (int ch = 0; ch < chunks; ++ch) {      // the rows' maxima over the warp, 16 at a time
                        float v[16];
                        tc_ld16(s_at + ch * 16, v);
                        if constexpr (FP8) {
                            float u[16];
                            tc_ld16(s_at + rp + ch * 16, u);
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = fmaf(u[j], 0.0625f, v[j]) * qf[c0 + ch * 16 + j];
                        }
                        uint32_t bits = sees[0];
#pragma unroll
                        for (int w = 1; w < C::WORDS; ++w)
                            if (ch >> 1 == w) bits = sees[w];
                        bits = masked ? bits >> (16 * (ch & 1)) : 0xffffu;
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = (bits >> j) & 1u ? (FP8 ? fmaf(v[j], f, add) : v[j] * f) : kNegInf;
                        const float x = fold16(v, lane, Max{});
                        if (!(lane & 1)) wred[warp][ch * 16 + fold_column(lane)] = x;
                    }
                    named_sync(bar, 128);
                    if (row < chunks * 16) {
                        const int w0 = wg * 4;
                        const float x = fmaxf(fmaxf(wred[w0][row], wred[w0 + 1][row]), fmaxf(wred[w0 + 2][row], wred[w0 + 3][row]));
                        const float m = -nref[c0 + row];
                        const bool up = x > m + kRefSlack;
                        nref[c0 + row] = up ? -x : -m;
                        alpha[c0 + row] = !up ? 1.f : m == kNoRef ? 0.f : ex2_approx(m - x);
                    }
                    named_sync(bar, 128);
#pragma unroll
                    for (int ch = 0; ch < CH; ++ch)
                        if (ch < chunks) {
                            if (!first) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) l[ch * 16 + j] *= alpha[c0 + ch * 16 + j];
#pragma unroll 1
                                for (int q = 0; q < C::PT; ++q) {
                                    float v[16];
                                    const uint32_t at = lanes + C::O_AT + q * rp + c0 + ch * 16;
                                    tc_ld16(at, v);
#pragma unroll
                                    for (int j = 0; j < 16; ++j) v[j] *= alpha[c0 + ch * 16 + j];
                                    tc_st16(at, v);
                                }
                            }
                        }
                    if constexpr (C::KEEP) score_all(Yes{});
                }
                // ---- probabilities; P is free once the tile before has been summed
                if (g > 0) ok = wait_bounded(&pv_done, (g - 1) & 1u, limit);
                late = !ok;
                unsigned char* prow = smem + C::P_OFF + row * 128;
                auto weigh = [&](int k0, const float (&v)[16]) {
                    if constexpr (FP8) {
                        uint32_t p[8];
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float y = ex2_approx(v[j]), z = ex2_approx(v[j + 1]);
                            f2_unpack(f2_fma(f2_pack(y, z), f2_pack(vinv, vinv), f2_pack(l[k0 + j], l[k0 + j + 1])), l[k0 + j], l[k0 + j + 1]);
                            p[j >> 1] = pack_f16(y, z);        // to 11 bits; what follows is exact
                        }
#pragma unroll
                        for (int q = 0; q < C::PT; ++q) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint32_t t = e4m3_of_f16x2(p[j]);
                                if (q + 1 < C::PT) p[j] = left_over_f16x2(p[j], t);
                                if (j & 1) w[j >> 1] |= t << 16;
                                else w[j >> 1] = t;
                            }
                            const int c = q * rp + c0 + k0;    // a column of P, a multiple of 16
                            *reinterpret_cast<uint4*>(prow + (c >> 7) * 16384 + ((((c & 127) >> 4) ^ (row & 7)) << 4)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        uint32_t w[8];
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float y = ex2_approx(v[j]), z = ex2_approx(v[j + 1]);
                            f2_unpack(f2_add(f2_pack(l[k0 + j], l[k0 + j + 1]), f2_pack(y, z)), l[k0 + j], l[k0 + j + 1]);
                            w[j >> 1] = pack_bf16(y, z);
                        }
                        const int c = c0 + k0;
                        unsigned char* at = prow + (c >> 6) * 16384;
                        const int k = (c & 63) >> 3;
                        *reinterpret_cast<uint4*>(at + ((k ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4*>(at + (((k + 1) ^ (row & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                };
                if constexpr (C::KEEP) {
#pragma unroll
                    for (int ch = 0; ch < CH; ++ch)
                        if (ch < chunks) {
                            float v[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = x[ch * 16 + j];
                            weigh(ch * 16, v);
                        }
                } else {
                    if (masked) each(Yes{}, weigh);
                    else each(No{}, weigh);
                }
                if (masked && wg == 0) {
                    // A new position's value that is no number, times a row's probability of
                    // zero, would spoil the row's sum: such values are taken out of the tile
                    // here, and given to the rows that see them at the unit's end.
                    // (by all threads, 16 bytes each: a position a thread was 16 rounds of a
                    // few threads, 3000 cycles at every unit's end)
                    late |= !wait_bounded(&v_full[g % VB], (g / VB) & 1u, limit);
                    constexpr int PIECES = C::BUF / 2048;       // of a position
                    const int t0 = max(sl.ctx - p0, 0), n = (min(sl.total - p0, kTcTile) - t0) * PIECES;
                    unsigned char* vb = smem + C::V_OFF + (g % VB) * C::BUF;
#pragma unroll 1
                    for (int e = row; e < n; e += 128) {
                        uint4* at = reinterpret_cast<uint4*>(vb + tc_off<FP8>(t0 + e / PIECES, e % PIECES));
                        uint4 w = *at;
                        const uint4 was = w;
                        w.x = FP8 ? drop_odd_e4m3(w.x) : drop_odd_bf16(w.x);
                        w.y = FP8 ? drop_odd_e4m3(w.y) : drop_odd_bf16(w.y);
                        w.z = FP8 ? drop_odd_e4m3(w.z) : drop_odd_bf16(w.z);
                        w.w = FP8 ? drop_odd_e4m3(w.w) : drop_odd_bf16(w.w);
                        if (w.x != was.x || w.y != was.y || w.z != was.z || w.w != was.w) {
                            odd_any = 1;
                            *at = w;
                        }
                    }
                }
                proxy_fence();
                tc_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s_free[g & 1]);
                    mbar_arrive(&p_full);
                }
            }

            // ---- the unit's end
            bool ok = !dead && !late;
            if (ok) ok = wait_bounded(&pv_done, (g - 1) & 1u, limit);
            dead = named_any(bar, 128, !ok);
            tc_after();
            // totals: over the lanes, then over the four warps
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
                if (ch < chunks) {
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = l[ch * 16 + j];
                    const float x = fold16(v, lane, Add{});
                    if (!(lane & 1)) wred[warp][ch * 16 + fold_column(lane)] = x;
                }
            named_sync(bar, 128);
            const bool bad = sl.bad || (a.par && tree_bad[wg]) || unit_bad[wg][uc % kTcUnitRing] || dead;
            const int mine = min(chunks * 16, un.rows - c0);   // rows of the warpgroup (may be none)
            float lsum = 0.f;
            if (row < mine) {
                const int w0 = wg * 4;
                lsum = (wred[w0][row] + wred[w0 + 1][row]) + (wred[w0 + 2][row] + wred[w0 + 3][row]);
                if (bad) lsum = CUDART_NAN_F;
            }
            const bool whole = un.ta == 0 && un.tb == un.tiles;
            float* sp = slots + (size_t)(2 * (int)blockIdx.x + (un.ta == 0 ? 1 : 0)) * slot_floats;
            if (row < mine) {                                  // thread r: row r's totals
                const int r = c0 + row;
                const float m = -nref[r];
                if (whole) {
                    const bool none = rown[r] >= sl.nb && !sl.bad;         // (as in put_row)
                    alpha[r] = none ? 0.f : 1.f / lsum;
                    if (a.lse) a.lse[(size_t)un.b * a.N * a.Hq + rowat[r]] = none ? kNegInf : (m + __log2f(lsum)) * kLn2;
                } else {
                    // a row that has seen nothing joins with weight zero
                    __stcg(sp + (size_t)srows * kTcD + r, m == kNoRef && !bad ? kNegInf : m);
                    __stcg(sp + (size_t)srows * (kTcD + 1) + r, lsum);
                }
            }
            named_sync(bar, 128);
            if (row == 0) unit_bad[wg][uc % kTcUnitRing] = 0;
            // (a small loop: it runs once a unit, its instructions seldom at hand)
#pragma unroll 1
            for (int k0 = 0; k0 < mine; k0 += 8) {
                float v[8];
                tc_ld8(lanes + C::O_AT + c0 + k0, v);
                if constexpr (FP8) {
#pragma unroll
                    for (int q = 1; q < C::PT; ++q) {
                        float y[8];
                        tc_ld8(lanes + C::O_AT + q * rp + c0 + k0, y);
                        const float f = __uint_as_float((uint32_t)(127 - 5 * q) << 23);        // 2^-5q
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = fmaf(y[k], f, v[k]);
                    }
                }
                if (odd_any) {
                    const int j0 = max(sl.ctx, un.ta * kTcTile), j1 = min(sl.total, un.tb * kTcTile);
                    for (int j = j0; j < j1; ++j) {
                        int page, slot;
                        if (!cache_place(a.c, un.b, j, &page, &slot)) continue;
                        const int64_t off = entry_off(a.c, page, slot, un.hk) + row;
                        float x;
                        if constexpr (FP8) {
                            float unused;
                            f16x2_to_f32(e4m3_to_f16x2(static_cast<const unsigned char*>(a.c.v)[off]), &x, &unused);
                        } else {
                            x = __uint_as_float((uint32_t)static_cast<const unsigned short*>(a.c.v)[off] << 16);
                        }
                        if (fabsf(x) < CUDART_INF_F) continue;
                        const int d = j - sl.ctx;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int n = rown[c0 + k0 + k];
                            if (a.par ? (anc[wg][0][n] >> (d & 63)) & 1ull : d <= n) v[k] += x;
                        }
                    }
                }
                if (whole) {
                    unsigned short* to = reinterpret_cast<unsigned short*>(a.out) + (size_t)un.b * a.N * a.Hq * kTcD + row;
#pragma unroll
                    for (int k = 0; k < 8; k += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(&alpha[c0 + k0 + k]);
                        const int4 at = *reinterpret_cast<const int4*>(&rowat[c0 + k0 + k]);
                        const float f[4] = {w.x, w.y, w.z, w.w};
                        const int r[4] = {at.x, at.y, at.z, at.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (k0 + k + e < mine)
                                to[(int64_t)r[e] * kTcD] =
                                    (unsigned short)(pack_bf16(f[e] == 0.f ? 0.f : v[k + e] * f[e], 0.f) & 0xffffu);
                    }
                } else {
                    float* to = sp + (size_t)(c0 + k0) * kTcD + row;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k0 + k < mine) __stcg(to + k * kTcD, v[k]);
                }
            }
            tc_before();
            ++uc;
        }
        if (dead && row == 0) raise_error(a.c.error, SPEC_DEVERR_TIMEOUT);
        tc_before();
    }
    __syncthreads();
    tc_after();
    if (warp == kMmaWarp) tc_dealloc(tmem, C::TMEM);
}

// Rows of a unit: all of a cached head's, or equal blocks of at most `most`.
static int tc_block_rows(int rt, int most) {
    const int blocks = (rt + most - 1) / most;
    return ((rt + blocks - 1) / blocks + 15) / 16 * 16;
}
constexpr int kTcMostBf16 = 144, kTcMostFp8 = 64;

// Which kernel takes heads of 128 (each side measured on one GB300, 8 cached heads,
// ragged lengths of half to all of the stated one; us here / in sv_attend.cu).
//   16 rows and fewer: one matrix tile of that one's is enough, and its units cost less
//     to begin and end: 78.1 / 73.4 for 64 sequences of 2000 positions, 56.2 / 45.6 of
//     1000, 22.3 / 20.6 for 8 of 4000.
//   17 to 32: this one gains per position what it loses per unit, so the longest context
//     that the block table has room for decides.  bf16, 32 rows: 64.4 / 59.7 for 64
//     sequences of 1000, 12.4 / 13.0 for one, but 80.5 / 90.8 and 13.3 / 19.0 of 2000.  E4M3,
//     where the other reads half the bytes and widens them, per position the two are
//     alike, and this one gains where CTAs share a unit's positions, as long as there are
//     fewer units (sequences x cached heads) than SMs.  32 rows: 14.4 / 14.2 for one
//     sequence of 1000, 16.0 / 16.5 of 2000, 20.4 / 23.2 of 4000, 25.3 / 29.7 for 8 of 2000,
//     115.4 / 117.8 of 32768, 46.3 / 47.6 for 16 of 4000, but 80.2 / 80.1 for 32 and
//     143.6 / 136.2 for 64; 20 rows: 14.4 / 13.6 for one of 1500, 24.8 / 27.0 for 8 of 2000,
//     46.3 / 45.2 for 16 of 4000, 141.9 / 131.4 for 64.
//   More: that one reads the cache once for every 32: 148.5 / 332.3 for 36 rows and 64 of
//     4000, 100.8 / 167.4 of 2000, 51.1 / 49.6 of 300.
// The host does not know the lengths: in a table much wider than its contexts, calls of 17
// to 32 rows come here however short these are.
constexpr long long kTcMinCapacity = 1536;
bool attend_takes_tc(int N, int G, int D, bool fp8, long long capacity, long long units, int sms) {
    return D == kTcD && (N * G > 32 || (N * G > 16 && capacity >= kTcMinCapacity && (!fp8 || units < sms)));
}

size_t attend_tc_workspace(int N, int G) {
    // the largest block of rows that N G or fewer can come in, so that more rows
    // never need less
    const int rt = N * G, rows = rt < kTcMostBf16 ? rt : kTcMostBf16;
    return kAttHead + align256((size_t)2 * kTcMaxCtas * part_floats(rows, kTcD) * 4);
}

// The driver's tensor map encoder (the library links the runtime only).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Where the places of a tensor map lie: a page's head every `unit` elements, at place
// page * pages + head * heads.  Pages that hold whole heads, or heads that hold whole
// pages; 0 for another layout.
struct Places {
    int64_t unit;
    int pages, heads;
};
static Places places_of(const spec_kv_cache_t& c) {
    const int64_t p = c.page_stride, h = c.kv_heads > 1 ? c.head_stride : p;
    if (p < 1 || h < 1) return {};
    const int64_t q = p % h == 0 ? p / h : 1, r = p % h == 0 ? 1 : h % p == 0 ? h / p : 0;
    if (r == 0 || (c.num_pages - 1) * q + (c.kv_heads - 1) * r >= (1ll << 31) || q > INT32_MAX || r > INT32_MAX) return {};
    return {p < h ? p : h, (int)q, (int)r};
}

// A layer's keys (or values) as boxes of `box` slots of a page's head.  E4M3: [place, slot,
// 128 bytes]; bf16: [place, group of 8 slots, half, slot, 128 bytes].
static bool encode_map(CUtensorMap* m, const spec_kv_cache_t& c, void* base, int box, const Places& at) {
    const bool f8 = c.dtype == SPEC_DTYPE_E4M3;
    const int elt = f8 ? 1 : 2;
    const cuuint64_t token = (cuuint64_t)c.token_stride * elt, place = (cuuint64_t)at.unit * elt;
    const cuuint64_t n = (cuuint64_t)(c.num_pages - 1) * at.pages + (cuuint64_t)(c.kv_heads - 1) * at.heads + 1;
    const cuuint64_t groups = (cuuint64_t)c.page_size / 8;
    const cuuint64_t dims8[3] = {128, (cuuint64_t)c.page_size, n}, dims16[5] = {64, 8, 2, groups, n};
    const cuuint64_t strides8[2] = {token, place}, strides16[4] = {token, 128, 8 * token, place};
    const cuuint32_t boxes8[3] = {128, (cuuint32_t)box, 1}, boxes16[5] = {64, 8, 2, (cuuint32_t)box / 8, 1};
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    for (cuuint64_t s : {token, 8 * token, place})
        if (s == 0 || s >= (1ull << 40)) return false;
    return encoder() &&
           encoder()(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f8 ? 3 : 5, base, f8 ? dims8 : dims16,
                     f8 ? strides8 : strides16, f8 ? boxes8 : boxes16, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CH, int NSM, bool FP8>
static cudaError_t launch_tc_t(const AttendArgs& a, int block_rows, int rp, cudaStream_t st) {
    using C = TcCfg<CH, NSM, FP8>;
    auto kfn = attend_tc_kernel<CH, NSM, FP8>;
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    static DeviceSlots slots = {};
    int unused = 0;
    e = device_once(slots, &unused, [&](int, int* o) {
        *o = 1;
        return cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    const long long rb = ((long long)a.N * a.G + block_rows - 1) / block_rows;
    const long long most = ((long long)a.c.max_pages * a.c.page_size + kTcTile - 1) / kTcTile;   // tiles of a unit
    long long g = di.sm_count < kTcMaxCtas ? di.sm_count : kTcMaxCtas;
    const long long units = (long long)a.B * a.c.kv_heads * rb;
    AttendArgs w = a;
    w.whole = most == 1 || attend_whole(units, (long long)a.c.max_pages * a.c.page_size, g);
    if (g > units * (w.whole ? 1 : most)) g = units * (w.whole ? 1 : most);
    // TMA boxes: one page, or 128 of its slots; tiles then begin and end with boxes
    const int ps = a.c.page_size;
    int box = ps % kTcTile == 0 ? kTcTile : ps >= 8 && kTcTile % ps == 0 ? ps : 0;
    CUtensorMap km = {}, vm = {};
    const Places at = places_of(a.c);
    if (at.unit == 0 || (box > 0 && (!encode_map(&km, a.c, a.c.k, box, at) || !encode_map(&vm, a.c, a.c.v, box, at)))) box = 0;
    const uint32_t limit = ring_wait_limit() < kTcWaitLimit ? ring_wait_limit() : kTcWaitLimit;
    e = launch_pdl(kfn, dim3((unsigned)g), C::THREADS, C::SMEM, st, w, block_rows, rp, box, at.pages, at.heads, limit, km, vm);
    return e != cudaSuccess ? e : launch_join(w, (int)g, units, block_rows, most, st);
}

template <bool FP8>
static cudaError_t launch_tc_e(const AttendArgs& a, cudaStream_t st) {
    const int rt = a.N * a.G, br = tc_block_rows(rt, FP8 ? kTcMostFp8 : kTcMostBf16);
    const int rp = br;                                          // a multiple of 16, as N of the products
    // (17 rows or more: blocks of 32 at least)
    // (an E4M3 tile's softmax has more to do, splitting the probabilities, in half the
    // time: two warpgroups from 17 rows on; with one it took 3300 cycles a tile of 32 rows)
    if (rp <= 32) return launch_tc_t<FP8 ? 1 : 2, FP8 ? 2 : 1, FP8>(a, br, rp, st);
    if (rp <= 64) return launch_tc_t<FP8 ? 2 : 4, FP8 ? 2 : 1, FP8>(a, br, rp, st);
    if constexpr (!FP8) return launch_tc_t<3, 3, false>(a, br, rp, st);
    return cudaErrorInvalidValue;                               // (blocks of an 8-bit cache are no larger)
}

cudaError_t launch_attend_tc(const AttendArgs& a, cudaStream_t st) {
    return a.c.dtype == SPEC_DTYPE_E4M3 ? launch_tc_e<true>(a, st) : launch_tc_e<false>(a, st);
}

}  // namespace sv
