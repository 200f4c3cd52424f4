// Products of 8-bit matrices with a scale for each block of 128, on the
// fifth-generation tensor cores:
//   out[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{k in block b} x[m, k] w[n, k].
// The scales change with every 128 elements of the contraction, so an
// accumulator in tensor memory holds one block's products only.  The inner sums
// are fp32 (exact where 24 bits hold them; of products 2^28 apart, off by up to 3 steps of
// 2^-23 of what their magnitudes add up to); the warps that read them add them, times the
// two scales, to running sums in registers, while the next blocks' products run into
// the other accumulators.
//
// Measured (one GB300, random inputs, new every time, bf16 out; bf16 products of cuBLAS reach 1924 TFLOP/s, a
// copy 6.8 TB/s):
//   1 row, N = 6144, K = 4096: 5.9 us, 4.3 TB/s (7.4 with more weights in turn than L2 holds); N = 151936: 90
//     us, 6.9 TB/s.  Memory, and some 2 us from one call's last store to the next one's first load and of the join.
//   512 rows, N = 151936, K = 4096: 265 us, 2.4 PFLOP/s; N = 24576: 47 us, 2.2; 1152 rows, N = 4096, K =
//     12288: 50 us, 2.3.  A step of 256 x 256 x 128 takes a pair 0.4 us, of which the products would
//     take 0.27: the rest is the chain from an accumulator's last product to its next, and what L2 brings (64
//     KB a step and pair, 11 TB/s in all: with half the bytes of both operands left out, the largest
//     took 211 us for 240); and the clock falls to 1.75 GHz under it.  (Constant inputs, which use less power: 240
//     us, 2.65 PFLOP/s.)
#include "sv_common.cuh"
#include "sv_kv.cuh"
#include "sv_linear.h"
#include "sv_tc.cuh"

namespace sv {

constexpr int kMmTile = 128;           // rows of an operand's tile, and elements of the contraction in a step
constexpr int kMmBytes = kMmTile * kMmTile;

// ---- PTX of clusters and pairs ---------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Without an order of memory: that all have come, no more.  (At a kernel's end the release waits for its
// stores to be acknowledged, 0.4 to 0.5 us of every call.)  What other CTAs send or read has to have
// come by then.
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// One lane of a converged warp.  (Loads and products are issued by loops that the whole warp
// runs, so that addresses and descriptors stay in uniform registers: in a branch of one lane
// the four products of a step took 315 cycles to issue.)
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint32_t limit) {
    return __all_sync(0xffffffffu, wait_bounded(bar, parity, limit));
}
// Whether the phase is complete, without waiting: asked a step ahead, the answer (some 100 cycles)
// comes while the step before is issued.
__device__ __forceinline__ bool phase_done(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// The address of a shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
// A scale.  (Not a read-only load, which could move ahead of the wait for the kernel before.)
__device__ __forceinline__ float ld_scale(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
// Four bytes to shared memory, asynchronously (zero without `have`); the arrival of the thread's
// copies so far on a barrier; the wait for all of them.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool have) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(have ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}
// The same from either CTA of a pair, the bytes counted by the barrier at `bar` of the
// cluster's shared memory.
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// A box from shared memory (written through proxy_fence before), as a group of its own; the wait until
// all but N of the thread's groups have been read.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y), "r"(src) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void tma_store_wait() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void map_prefetch(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void pair_alloc(uint32_t* dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t at, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// Arrives on the barrier at this place in both CTAs when the products issued so far have completed.
__device__ __forceinline__ void pair_commit(uint64_t* bar, unsigned short both) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_addr(bar)),
                 "h"(both)
                 : "memory");
}
// ---- few rows ----------------------------------------------------------------------
// Up to 64 rows of x: the product is taken transposed, so that 128 weight rows are the
// rows that the instruction wants and the few rows of x its free dimension T.  The weights are
// read once, which bounds these calls.  A tile of 128 weight rows is shared by a cluster of S CTAs, each
// with its part of the contraction; they add their sums over distributed shared memory, in the order of
// their ranks, each a part of the columns.
//   warp 0     loads: both operands and the rows' scales of BP blocks into a ring, by TMA
//   warp 1     issues the products
//   warps 2-5  running sums: a thread owns a weight row, the rows' scales are read from shared
//              memory, the weights' scale is the tile's
// Handing on a block takes a CTA's warps some 400 cycles of waits and arrivals, 16 KB in 0.2 us.  So two
// CTAs an SM, 100 KB under way each (one with all the ring: 7.0 us for 6.3 at one row, N = 6144, K = 4096,
// 27.5 for 22 at 64 rows, N = 24576), and for up to 16 rows two blocks at a time (one row: 6.26 for 6.48;
// 64 rows so: 24.8 for 23.2).  Equal shares of all tiles' blocks, their parts joined through
// memory, gained nothing here over a cluster or a CTA a tile: 96.8 us for 94.5 at one row, N = 151936.  (These
// pairs of times are from before a kernel's end lost its release, 0.4 to 0.5 us of each: now 5.9 us
// at one row, N = 6144, and 21.7 at 64 rows, N = 24576, where 192 tiles leave 112 of 304 places empty.)  65
// to 128 rows this way: 6.4 us for the 5.6 of pairs at 1000 x 1040, 28.9 for 27.3 at 24576 x 4096, and
// 18.5 for 20.7 only at 4096 x 12288 (single CTAs: 16.8).
template <int T>
struct FewCfg {
    static constexpr int BP = T <= 16 ? 2 : 1;            // blocks at a time
    static constexpr int SCALE = BP * T * 4;
    static constexpr int STAGES = T <= 16 ? 3 : T <= 32 ? 5 : 4;
    static constexpr int COLS = BP * T, TMEM = COLS * STAGES <= 128 ? 128 : 256;   // accumulators: a stage's
    static constexpr int X_AT = BP * kMmBytes, X_BYTES = T * kMmTile, BYTES = kMmBytes + X_BYTES, STAGE = BP * BYTES;
    // Scales have a place more than the operands: an arrival does not wait for what the warp is still
    // reading from shared memory, so a place is written again only when the warps have taken the step
    // after (with as many places as stages, one row's scales in 10^5 came from the next round).  No barrier
    // says that its reads have come by then, the sums do: before the arrival of step i + 1 stand its
    // multiply-adds, each of which adds to what step i's left, which needed step i's scale.  Sums in two sets, or
    // steps whose multiply-adds move behind the next one's arrival, would take that away.
    static constexpr int SCALE_AT = STAGES * STAGE, PLACES = STAGES + 1;
    static constexpr int SMEM = SCALE_AT + PLACES * SCALE + 1024;        // and room to align
    static constexpr int THREADS = 192, CTAS = 2;
    static_assert(CTAS * (SMEM + 2048) <= 228 * 1024 && CTAS * TMEM <= 512 && COLS * STAGES <= TMEM, "what an SM has");
    static_assert(3 * (SMEM + 1024) > 228 * 1024, "no more CTAs than tensor memory has room for");
    static_assert(SCALE % 128 == 0 && T * kMmTile * 4 <= SCALE_AT, "alignment; the sums of a CTA fit the ring");
};

// n (up to 4) neighbouring results from element `at` of out on; wide: rows begin at 16 bytes.
__device__ __forceinline__ void put4(const MatmulArgs& a, int64_t at, int n, bool wide, const float (&v)[4]) {
    if (a.f32) {
        float* to = reinterpret_cast<float*>(a.out) + at;
        if (wide && n == 4) {
            *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) to[e] = v[e];
        }
    } else {
        unsigned short* to = reinterpret_cast<unsigned short*>(a.out) + at;
        const uint2 w = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        if (wide && n == 4) {
            *reinterpret_cast<uint2*>(to) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) to[e] = (unsigned short)((e < 2 ? w.x : w.y) >> 16 * (e & 1));
        }
    }
}

// ANY: one row, whose scales lie anywhere: they are loaded with the tile's and multiplied there, and every place
// holds ones.
template <int T, bool ANY = false>
__global__ void __launch_bounds__(FewCfg<T>::THREADS, FewCfg<T>::CTAS) matmul_few_kernel(const MatmulArgs a, uint32_t limit, int blocks, int S, bool wide,
                                                                          const __grid_constant__ CUtensorMap xmap,
                                                                          const __grid_constant__ CUtensorMap wmap,
                                                                          const __grid_constant__ CUtensorMap smap) {
    using C = FewCfg<T>;
    extern __shared__ unsigned char smem_raw[];
    // done: a step's products are complete; empty: its sums are taken, its stage and accumulator free
    __shared__ __align__(8) uint64_t full[C::STAGES], done[C::STAGES], empty[C::STAGES], drained;
    __shared__ uint32_t tmem_at;
    unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int tile = blockIdx.x / S, rank = blockIdx.x - tile * S;     // (a cluster: S consecutive CTAs)
    const int b0 = (int)((long long)blocks * rank / S), b1 = (int)((long long)blocks * (rank + 1) / S);
    if (warp == 0) {
        if (elect_one()) {
            for (int i = 0; i < C::STAGES; ++i) {
                mbar_init(&full[i], 1);
                mbar_init(&done[i], 1);
                mbar_init(&empty[i], 4);
            }
            mbar_init(&drained, 1);
            mbar_init_fence();
            map_prefetch(&wmap);
            map_prefetch(&xmap);
            if (!ANY) map_prefetch(&smap);
        }
        __syncwarp();
    }
    if (warp == 1) tc_alloc(&tmem_at, C::TMEM);
    if (ANY) {
        for (int i = tid; i < C::PLACES * C::SCALE / 4; i += C::THREADS) reinterpret_cast<float*>(smem + C::SCALE_AT)[i] = 1.f;
    }
    pdl_trigger();
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tmem_at;
    pdl_wait();
    int32_t* error = reinterpret_cast<int32_t*>(a.ws);

    if (warp == 0) {
        bool ok = true;
        unsigned it = 0, s = 0, phase = 0, place = 0;      // step, its stage, how often the ring has come round (mod 2)
        const uint32_t base = smem_addr(smem);
        const bool lead = elect_one();
        for (int b = b0; b < b1; b += C::BP, ++it) {
            if (it >= C::STAGES) {
                ok = wait_warp(&empty[s], phase ^ 1, limit);
                if (!ok) break;
            }
            const uint32_t at = base + s * C::STAGE;
            const bool two = C::BP == 2 && b + 1 < b1;
            if (lead) {
                mbar_arrive_expect_tx(&full[s], (two ? 2 : 1) * C::BYTES + (ANY ? 0 : C::SCALE));
                tma_2d(at, &wmap, b * kMmTile, tile * kMmTile, &full[s]);
                if (two) tma_2d(at + kMmBytes, &wmap, (b + 1) * kMmTile, tile * kMmTile, &full[s]);
                tma_2d(at + C::X_AT, &xmap, b * kMmTile, 0, &full[s]);
                if (two) tma_2d(at + C::X_AT + C::X_BYTES, &xmap, (b + 1) * kMmTile, 0, &full[s]);
                if (!ANY) tma_2d(base + C::SCALE_AT + place * C::SCALE, &smap, 0, b, &full[s]);
            }
            __syncwarp();
            if (++place == C::PLACES) place = 0;
            if (++s == C::STAGES) {
                s = 0;
                phase ^= 1;
            }
        }
        // every copy has landed and every commit has arrived before the CTA ends
        for (unsigned j = it > C::STAGES ? it - C::STAGES : 0; j < it; ++j) {
            const unsigned k = j % C::STAGES, parity = (j / C::STAGES) & 1;
            if (!wait_warp(&full[k], parity, kTcWaitLimit) || !wait_warp(&done[k], parity, limit)) ok = false;
        }
        if (!ok && lane == 0) raise_error(error, SPEC_DEVERR_TIMEOUT);
    } else if (warp == 1) {
        const uint32_t id = tc_idesc(true, false, false, T);
        const uint64_t base = tc_desc(smem_addr(smem), 16, 1024);
        const bool lead = elect_one();
        bool ok = true;
        unsigned it = 0, s = 0, phase = 0;
        for (int b = b0; b < b1; b += C::BP, ++it) {
            ok = wait_warp(&full[s], phase, limit);
            if (!ok) break;
            tc_after();
            const uint64_t wd = base + s * (C::STAGE >> 4), xd = wd + (C::X_AT >> 4);
            const uint32_t to = tmem + s * C::COLS;
            if (lead) {
#pragma unroll
                for (int k = 0; k < 4; ++k) tc_mma<true>(to, wd + 2 * k, xd + 2 * k, id, k > 0);
                if (C::BP == 2 && b + 1 < b1) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc_mma<true>(to + T, wd + (kMmBytes >> 4) + 2 * k, xd + (C::X_BYTES >> 4) + 2 * k, id, k > 0);
                }
                tc_commit(&done[s]);
            }
            __syncwarp();
            if (++s == C::STAGES) {
                s = 0;
                phase ^= 1;
            }
        }
        if (!ok) {
            if (lane == 0) raise_error(error, SPEC_DEVERR_TIMEOUT);
            if (it > 0) {
                if (lead) tc_commit(&drained);
                __syncwarp();
                wait_warp(&drained, 0, kTcWaitLimit);
            }
        }
    }
    const int quad = warp & 3, row = quad * 32 + lane;     // of a tile's weight rows (warps 2 to 5)
    float acc[T];
    if (warp >= 2) {
        const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16);
#pragma unroll
        for (int c = 0; c < T; ++c) acc[c] = 0.f;
        // the tile's scales, 32 blocks at a time, a lane each (one ahead of its use, a load a block
        // held every block up for the memory's answer)
        const float* wsc = a.wscale + (int64_t)tile * a.ws_stride;
        float wl = 0.f;
        bool ok = true;
        unsigned s = 0, phase = 0, place = 0;
        for (int b = b0; b < b1; b += C::BP) {
            if (((b - b0) & 31) == 0 && b + lane < b1) {
                wl = ld_scale(wsc + b + lane);
                if (ANY) wl *= ld_scale(a.xscale + (b + lane) * a.xs_stride);
            }
            const bool two = C::BP == 2 && b + 1 < b1;
            const float wf[2] = {__shfl_sync(0xffffffffu, wl, (b - b0) & 31), __shfl_sync(0xffffffffu, wl, (b - b0 + 1) & 31)};
            ok = wait_warp(&done[s], phase, limit);
            if (!ok) break;
            tc_after();
            const float4* xs = reinterpret_cast<const float4*>(smem + C::SCALE_AT + place * C::SCALE);
            const uint32_t at = from + s * C::COLS;
            float v[2][16];
            tc_ld16_start(at, v[0]);
#pragma unroll
            for (int c = 0; c < C::COLS; c += 16) {
                if (c == T && !two) break;
                float* now = v[(c >> 4) & 1];
                tc_wait_ld();
                tc_ld16_done(now);
                if (c + 16 < C::COLS && (c + 16 != T || two)) tc_ld16_start(at + c + 16, v[((c >> 4) + 1) & 1]);
                const f32x2 w2 = f2_pack(wf[c >= T], wf[c >= T]);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 f = xs[(c + e) >> 2];
                    float* to = acc + (c + e) % T;
                    f2_unpack(f2_fma(f2_pack(now[e], now[e + 1]), f2_mul(f2_pack(f.x, f.y), w2), f2_pack(to[0], to[1])), to[0], to[1]);
                    f2_unpack(f2_fma(f2_pack(now[e + 2], now[e + 3]), f2_mul(f2_pack(f.z, f.w), w2), f2_pack(to[2], to[3])), to[2], to[3]);
                }
            }
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++place == C::PLACES) place = 0;
            if (++s == C::STAGES) {
                s = 0;
                phase ^= 1;
            }
        }
        if (!ok) {                                         // a result that is not valid shows
#pragma unroll
            for (int c = 0; c < T; ++c) acc[c] = CUDART_NAN_F;
            if (lane == 0) raise_error(error, SPEC_DEVERR_TIMEOUT);
        }
    }
    tc_before();
    __syncthreads();                                       // every product is done, the ring is free
    tc_after();
    // ---- the output: the CTAs' sums, [row of x][weight row], through shared memory; a thread takes
    // four neighbouring weight rows of a row of x, a warp 128.  (A weight row a thread, with its sums in registers: 64
    // stores of two bytes each for 64 rows, and as many dependent reads of other CTAs' sums.)
    float* sums = reinterpret_cast<float*>(smem);
    if (warp >= 2) {
#pragma unroll
        for (int c = 0; c < T; ++c)
            if (c < a.M) sums[c * kMmTile + row] = acc[c];
    }
    if (S == 1) __syncthreads();
    else cluster_sync();
    const int rows = (a.M - rank + S - 1) / S;             // of x: this CTA's are rank, rank + S, ...
    const uint32_t from = smem_addr(sums);
    for (int i = tid; i < rows * 32; i += C::THREADS) {
        const int m = rank + (i >> 5) * S, o = (i & 31) * 4;
        const int64_t n = (int64_t)tile * kMmTile + o;
        if (n >= a.N) continue;
        float4 x[8];                                       // all under way at once
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (r >= S) break;
            x[r] = ld_cluster4(cluster_addr(from + (m * kMmTile + o) * 4, S == 1 ? (uint32_t)rank : (uint32_t)r));
        }
        float v[4] = {};
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (r >= S) break;
            v[0] += x[r].x, v[1] += x[r].y, v[2] += x[r].z, v[3] += x[r].w;
        }
        put4(a, (int64_t)m * a.old + n, (int)min((int64_t)4, a.N - n), wide, v);
    }
    if (S > 1) cluster_meet();                             // no CTA ends while another reads its sums
    if (warp == 1) tc_dealloc(tmem, C::TMEM);
}

// ---- shares and parts ----------------------------------------------------------------
// For more rows the steps (blocks of the contraction) of all tiles, end to end, are dealt to pairs of CTAs, or to
// CTAs by themselves: whole tiles, or, to pairs, equal shares that may begin and end inside a tile.  Of a tile in
// several shares, each warp of each pair leaves its part of the sums in the workspace and takes a ticket; the
// one that takes the last adds the parts in their order, whichever that was, and writes the
// output.  Nobody waits for anybody.
struct MmPlan {
    long long tiles, total;            // steps of all tiles
    int pairs, blocks, whole;          // pairs, or single CTAs; blocks: steps of a tile
    int W, tiles_m;                    // a tile's weight rows; tiles of 256 (128) rows of x
    int split;                         // pairs (CTAs) of a cluster
    int pair;                          // CTAs in pairs, or each by itself
    unsigned long long tag;
    // equal shares: the first step of a pair's
    __host__ __device__ __forceinline__ long long begin(int p) const { return total * p / pairs; }
    // (a cluster's pairs share its tile)
    __device__ __forceinline__ long long part_begin(int p) const {
        const int tile = p / split, q = p - tile * split;
        return (long long)tile * blocks + (long long)blocks * q / split;
    }
    // the pair whose (equal) share has step u
    __host__ __device__ __forceinline__ int of(long long u) const { return (int)(((u + 1) * pairs - 1) / total); }
};
// The workspace: error word (256 bytes), a ticket for each pair's last tile, CTA and warp, two parts a pair.
constexpr int kMmMaxPairs = 80;
constexpr size_t kMmTicketAt = 256;
constexpr size_t kMmPartAt = kMmTicketAt + (size_t)kMmMaxPairs * 16 * 8;
constexpr size_t kMmPartBytes = (size_t)256 * 256 * 4;     // of the widest tile

// A tile's parts are those of pairs p0 to p1, the first the last part of its pair.
struct MmParts {
    long long t0;
    int p0, p1;
    __device__ __forceinline__ MmParts(const MmPlan& plan, int tile) {
        t0 = (long long)tile * plan.blocks;
        p0 = plan.of(t0);
        p1 = plan.of(t0 + plan.blocks - 1);
    }
    __device__ __forceinline__ float* part(const MmPlan& plan, char* ws, int p) const {
        return reinterpret_cast<float*>(ws + kMmPartAt + (size_t)(2 * p + (plan.begin(p) < t0)) * kMmPartBytes);
    }
};
// A ticket of those of launch `tag`: how many were taken before.  Whatever the word held, a ticket
// of another launch counts as none; the last to come leaves zero, for a replay of the same launch.
__device__ __forceinline__ unsigned tickets_taken(unsigned long long w, unsigned long long tag) {
    return (w >> 24) == tag ? (unsigned)(w & 0xffffffu) : 0u;
}
__device__ __forceinline__ unsigned take_ticket(unsigned long long* w, unsigned long long tag) {
    unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(w), seen;
    do {
        seen = old;
        old = atomicCAS(w, seen, (seen >> 24) == tag ? seen + 1 : (tag << 24) + 1);
    } while (old != seen);
    return tickets_taken(seen, tag);
}
// The warp's, after what its lanes have written: whether it was the last of n.
__device__ __forceinline__ bool last_ticket(unsigned long long* w, unsigned long long tag, int n, int lane) {
    __threadfence();
    __syncwarp();
    // (votes: a warp that knows that it stays together keeps its counters in uniform registers)
    if (!__any_sync(0xffffffffu, lane == 0 && (int)take_ticket(w, tag) == n - 1)) return false;
    if (lane == 0) *w = 0;
    __threadfence();
    return true;
}

// ---- more rows ---------------------------------------------------------------------
// A pair of CTAs takes 256 rows of x times W weight rows (cta_group::2: each loads its 128
// rows of x and half of the weight rows, and holds its 128 rows' sums), or a CTA by itself 128 times W.  A
// pair brings 64 KB for 256 x 256 x 128, two CTAs 96: 235 us for 267 at 512 x 151936 x 4096.  Single
// ones divide rows and tiles more finely: 1152 rows, 4096 x 12288: 47 us for 58; 128 rows, 24576 x 4096: 23 for
// 28.  Which, and W, of 64, 128, 192 and 256, is chosen by the launch so that the tiles fill them evenly.
//   warp 0      loads
//   warp 1      issues the products (the pair's first CTA, for both)
//   warp 2      brings the scales
//   warps 4-11  running sums, then the tile's output: a thread owns a row of x and a half of the
//               tile's columns
// TWO (W 192 or 256): the halves of the columns are products of their own, each with its
// accumulators, so that the second half's run while the first's are read.  Between an
// accumulator's last product and its next lie a commit, a wake, its reading and an arrival in the other
// CTA, some 1400 cycles in which two accumulators of 256 columns left the tensor cores idle half the
// time (512 x 38912 x 4096: 69 us so, 64 with halves).
struct ManyCfg {
    static constexpr int EW = 8;                           // warps of the sums
    static constexpr int STAGES = 8, NB = 4;               // at most
    static constexpr int COLS = 128;                       // a warp's columns, at most
    static constexpr int X_BYTES = kMmBytes;
    static constexpr int OUT_AT = 185 * 1024;              // two pieces of 32 rows x 64 bytes a warp
    static constexpr int FS = 4;                           // groups of four steps whose scales are held
    static constexpr int F_BYTES = 128 * 16 + 64;          // the rows' four; for each half, those of two blocks of the weights
    static constexpr int F_AT = OUT_AT + EW * 4096;
    static constexpr int SMEM = F_AT + FS * F_BYTES + 1024;
    static constexpr int THREADS = 128 + EW * 32;
    // registers: the launch's share a thread, and how the warpgroups split it
    static constexpr int REGS = 65536 / THREADS / 8 * 8, LESS = 56;
    static constexpr int MORE = (REGS * THREADS - LESS * 128) / (EW * 32) / 8 * 8;
    static constexpr int PART = COLS * 32;                 // floats of a warp's part
    static_assert(SMEM + 512 <= 227 * 1024, "shared memory");
};
// Whether the halves of a tile's columns are products of their own (a pair's product has a
// multiple of 32 columns); stages of a ring; accumulators (of a half, where there are two).
__host__ __device__ constexpr bool two_halves(int W) { return W > 128 && W % 64 == 0; }
// Blocks of the contraction in a step, each with its accumulator: handing a step to the sums takes their warps
// some 300 cycles besides its columns, which 64 columns are not worth (a block of theirs 0.15 us, 0.21 alone;
// of 128 columns 0.245 alone, 0.255 by twos, whose stages are fewer).
__host__ __device__ constexpr int blocks_of(int W) { return W == 64 ? 2 : 1; }
__host__ __device__ constexpr unsigned least(unsigned a, unsigned b) { return a < b ? a : b; }
__host__ __device__ constexpr unsigned stages_of(int W, bool pair) {
    return least(ManyCfg::OUT_AT / (blocks_of(W) * (ManyCfg::X_BYTES + W / (pair ? 2 : 1) * kMmTile)), ManyCfg::STAGES);
}
// (no more than stages: a barrier of products counts two rounds of its stage before the sums have seen one)
__host__ __device__ constexpr unsigned buffers_of(int W, bool pair) { return least(least(512 / (blocks_of(W) * W), ManyCfg::NB), stages_of(W, pair)); }
enum MmMode { kMmWhole, kMmTickets, kMmCluster };
template <int W, MmMode MODE, bool PAIR>
__global__ void __launch_bounds__(ManyCfg::THREADS, 1) matmul_many_kernel(const MatmulArgs a, uint32_t limit, const MmPlan plan,
                                                                         const __grid_constant__ CUtensorMap xmap,
                                                                         const __grid_constant__ CUtensorMap wmap,
                                                                         const __grid_constant__ CUtensorMap omap, bool by_tma, int vec) {
    using C = ManyCfg;
    constexpr bool TWO = two_halves(W);
    constexpr int H = W / 2;
    constexpr bool CROSS = kScaleBlock % H != 0;           // a half's columns may lie in two blocks of the weights
    static_assert(H % 32 == 0 && H <= ManyCfg::COLS, "whole pieces of the output");
    // Whether the sums ask for the next step's products ahead (1152 x 4096 x 12288, then in shares: 58.5 us for 60.5;
    // whole tiles with halves, bound by power: 239 for 236 at 512 x 151936 x 4096).
    constexpr bool PEEK = !TWO || MODE == kMmTickets;
    constexpr int BP = blocks_of(W);
    constexpr int CTAS = PAIR ? 2 : 1, ROWS = CTAS * 128;  // a tile's CTAs and rows of x
    constexpr int OWN = W / CTAS;                          // weight rows that a CTA loads
    constexpr unsigned stages = stages_of(W, PAIR), buffers = buffers_of(W, PAIR);
    constexpr uint32_t block_bytes = C::X_BYTES + OWN * kMmTile, stage_bytes = BP * block_bytes;
    static_assert(stages >= 3, "loads under way");
    static_assert(MODE != kMmTickets || PAIR, "the workspace has tickets and parts for pairs");
    static_assert(BP == 1 || !TWO, "a step's accumulators");
    extern __shared__ unsigned char smem_raw[];
    // done: a step's products (of a half) are complete; after the second half's its stage is free.  (As
    // many as stages: an accumulator's next product waits for the sums, a stage's next load for done, so
    // no phase is passed unseen.)
    __shared__ __align__(8) uint64_t full[C::STAGES], done[2][C::STAGES], t_empty[2][C::NB], f_full[C::FS], f_empty[C::FS], drained;
    __shared__ uint32_t tmem_at;
    __shared__ int failed;
    unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    // (a cluster: pairs of a tile's, where they share it; the first CTA of a pair leads it)
    const uint32_t place = cluster_rank(), rank = PAIR ? place & 1 : 0, leader = place - rank;
    const int pair = blockIdx.x / CTAS, blocks = plan.blocks, tiles_m = plan.tiles_m;
    // The first tile, its first step, and the steps to do.  Whole tiles go to the pairs in turn: those of the
    // same weight rows are taken side by side, and the weights read once.
    int first_tile = pair, first_b = 0;
    long long steps = (plan.tiles - pair + plan.pairs - 1) / plan.pairs * blocks;
    if (MODE != kMmWhole) {
        const long long u0 = MODE == kMmCluster ? plan.part_begin(pair) : plan.begin(pair);
        steps = (MODE == kMmCluster ? plan.part_begin(pair + 1) : plan.begin(pair + 1)) - u0;
        first_tile = (int)(u0 / blocks);
        first_b = (int)(u0 - (long long)first_tile * blocks);
    }
    const int turn = MODE == kMmWhole ? plan.pairs : 1;    // from one tile to the next
    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&done[0][i], 1);
            mbar_init(&done[1][i], 1);
        }
        for (int i = 0; i < C::NB; ++i) {                  // both CTAs' warps
            mbar_init(&t_empty[0][i], CTAS * C::EW / (TWO ? 2 : 1));
            mbar_init(&t_empty[1][i], CTAS * C::EW / 2);
        }
        for (int i = 0; i < C::FS; ++i) {
            mbar_init(&f_full[i], 32);
            mbar_init(&f_empty[i], C::EW);
        }
        mbar_init(&drained, 1);
        mbar_init_fence();
        failed = 0;
        map_prefetch(&xmap);
        map_prefetch(&wmap);
        if (by_tma) map_prefetch(&omap);
    }
    if (warp == 1) {
        if (PAIR) pair_alloc(&tmem_at, 512);
        else tc_alloc(&tmem_at, 512);
    }
    pdl_trigger();
    tc_before();
    cluster_sync();
    tc_after();
    const uint32_t tmem = tmem_at;
    pdl_wait();
    auto fail = [&]() {
        raise_error(reinterpret_cast<int32_t*>(a.ws), SPEC_DEVERR_TIMEOUT);
        failed = 1;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::LESS));
        if (warp == 0) {
            bool ok = true, free = false;
            unsigned it = 0, s = 0, phase = 0;             // step, its stage, how often the ring has come round (mod 2)
            const uint32_t base = smem_addr(smem), bars = cluster_addr(smem_addr(full), leader);
            uint64_t(&last)[C::STAGES] = done[TWO ? 1 : 0];
            const bool lead = elect_one();
            long long left = steps;
            for (int tile = first_tile, b = first_b; ok && left > 0; tile += turn, b = 0) {
                const int tn = tile / tiles_m, m0 = (tile - tn * tiles_m) * ROWS + (int)rank * 128;
                // (a product's columns are half the first CTA's weight rows, half the second's)
                const int n0 = tn * W + (int)rank * (TWO ? H / 2 : H);
                const int end = (int)min((long long)blocks, b + left);
                left -= end - b;
                for (; b < end; b += BP, ++it) {
                    if (it >= stages && !free) {
                        ok = wait_warp(&last[s], phase ^ 1, limit);
                        if (!ok) break;
                    }
                    const uint32_t at = base + s * stage_bytes, bar = bars + s * 8;
                    const unsigned now = s;
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1;
                    }
                    free = phase_done(&last[s], phase ^ 1);
                    if (lead) {
                        const bool all = b + BP <= end;    // (else the step has one block of two)
                        if (rank == 0) mbar_arrive_expect_tx(&full[now], CTAS * (all ? stage_bytes : block_bytes));
#pragma unroll
                        for (int k = 0; k < BP; ++k) {
                            if (k > 0 && !all) break;
                            const uint32_t to = at + k * block_bytes;
                            if constexpr (PAIR) {
                                tma_2d_pair(to, &xmap, (b + k) * kMmTile, m0, bar);
                                tma_2d_pair(to + C::X_BYTES, &wmap, (b + k) * kMmTile, n0, bar);
                                if constexpr (TWO) tma_2d_pair(to + C::X_BYTES + H / 2 * kMmTile, &wmap, (b + k) * kMmTile, n0 + H, bar);
                            } else {
                                tma_2d(to, &xmap, (b + k) * kMmTile, m0, &full[now]);
                                tma_2d(to + C::X_BYTES, &wmap, (b + k) * kMmTile, n0, &full[now]);
                            }
                        }
                    }
                    free = __all_sync(0xffffffffu, free);
                }
            }
            // every copy has landed and every commit has arrived before the CTA ends
            for (unsigned j = it > stages ? it - stages : 0; j < it; ++j) {
                const unsigned k = j % stages, parity = (j / stages) & 1;
                if (rank == 0 && !wait_warp(&full[k], parity, kTcWaitLimit)) ok = false;
                if (!wait_warp(&last[k], parity, limit)) ok = false;
            }
            if (!ok && lane == 0) fail();
        } else if (warp == 1 && rank == 0) {
            const unsigned short both = (unsigned short)(3u << leader);
            const uint32_t id = tc_idesc(true, false, false, TWO ? H : W, ROWS);
            const auto mma = [&](uint32_t d, uint64_t x, uint64_t w, bool add) {
                if constexpr (PAIR) pair_mma(d, x, w, id, add);
                else tc_mma<true>(d, x, w, id, add);
            };
            const auto commit = [&](uint64_t* bar) {
                if constexpr (PAIR) pair_commit(bar, both);
                else tc_commit(bar);
            };
            const uint64_t base = tc_desc(smem_addr(smem), 16, 1024);
            unsigned it = 0, s = 0, phase = 0, t = 0, t_phase = 0;
            const bool lead = elect_one();
            bool ok = true, ready = false;
            // (a barrier's phase before its first counts as complete: no step waits for an accumulator that
            // nothing has used)
            int b = first_b, end = (int)min((long long)blocks, b + steps);
            for (long long left = steps; left > 0; ++it) {
                const int n = BP == 1 ? 1 : min(BP, end - b);      // blocks of the step
                left -= n;
                if constexpr (BP > 1) {
                    b += n;
                    if (b == end) b = 0, end = (int)min((long long)blocks, left);
                }
                if (!ready) {
                    ok = wait_warp(&full[s], phase, limit) && wait_warp(&t_empty[0][t], t_phase ^ 1, limit);
                    if (!ok) break;
                }
                tc_after();
                const uint64_t xd = base + s * (stage_bytes >> 4), wd = xd + (C::X_BYTES >> 4);
                const uint32_t to = tmem + t * (TWO ? H : BP * W);
                const unsigned now = s;
                if constexpr (TWO) {
                    const bool second = phase_done(&t_empty[1][t], t_phase ^ 1);
                    if (lead) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma(to, xd + 2 * k, wd + 2 * k, k > 0);
                        commit(&done[0][now]);
                    }
                    if (!__all_sync(0xffffffffu, second)) {
                        ok = wait_warp(&t_empty[1][t], t_phase ^ 1, limit);
                        if (!ok) {
                            ++it;                          // (products have been issued)
                            break;
                        }
                    }
                    tc_after();
                }
                if (++s == stages) {
                    s = 0;
                    phase ^= 1;
                }
                if (++t == buffers) {
                    t = 0;
                    t_phase ^= 1;
                }
                const bool next = phase_done(&full[s], phase) & phase_done(&t_empty[0][t], t_phase ^ 1);
                if (lead) {
                    const uint64_t wd2 = TWO ? wd + (OWN / 2 * kMmTile >> 4) : wd;
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma(to + (TWO ? 256 : 0), xd + 2 * k, wd2 + 2 * k, k > 0);
                    if (BP > 1 && n > 1) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma(to + W, xd + (block_bytes >> 4) + 2 * k, wd + (block_bytes >> 4) + 2 * k, k > 0);
                    }
                    commit(&done[TWO ? 1 : 0][now]);
                }
                ready = __all_sync(0xffffffffu, next);
            }
            // the other CTA's last arrivals have come (t and t_phase: the next step's)
            for (unsigned j = 0; ok && j < buffers && j < it; ++j) {
                if (t == 0) t_phase ^= 1;
                t = t == 0 ? buffers - 1 : t - 1;
                ok = wait_warp(&t_empty[0][t], t_phase, kTcWaitLimit) && (!TWO || wait_warp(&t_empty[1][t], t_phase, kTcWaitLimit));
            }
            if (!ok) {
                if (lane == 0) fail();
                if (it > 0) {
                    if (lead) commit(&drained);
                    __syncwarp();
                    wait_warp(&drained, 0, kTcWaitLimit);
                }
            }
        } else if (warp == 2) {
            // Scales, four steps at a time, by asynchronous copies some groups ahead of the sums.  (Loaded
            // through registers by the threads of the sums, four steps ahead, they held each
            // step up by 600 to 700 cycles.)
            unsigned gi = 0;
            bool ok = true;
            long long left = steps;
            for (int tile = first_tile, at = first_b; ok && left > 0; tile += turn, at = 0) {
                const int end = (int)min((long long)blocks, at + left);
                left -= end - at;
                const int tn = tile / tiles_m, m0 = (tile - tn * tiles_m) * ROWS + (int)rank * 128;
                // the first 16 lanes: a half's first or second 128-block of the weights, and a step of the four
                const int wrow = min((tn * W + (lane >> 3 & 1) * H) / kScaleBlock + (lane >> 2 & 1), (a.N - 1) / kScaleBlock);
                const float* wsc = a.wscale + (int64_t)wrow * a.ws_stride;
                for (int b4 = at; b4 < end; b4 += 4, ++gi) {
                    const unsigned s = gi % C::FS;
                    if (gi >= C::FS) ok = wait_warp(&f_empty[s], (gi / C::FS - 1) & 1, limit);
                    if (!ok) break;
                    const uint32_t to = smem_addr(smem + C::F_AT + s * C::F_BYTES);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int m = m0 + r * 32 + lane;
                            const bool have = m < a.M && b4 + j < end;
                            copy4(to + (r * 32 + lane) * 16 + j * 4, have ? a.xscale + (int64_t)(b4 + j) * a.xs_stride + m : a.xscale, have);
                        }
                    if (lane < 16) {
                        const int b = b4 + (lane & 3);
                        copy4(to + 128 * 16 + lane * 4, b < end ? wsc + b : wsc, b < end);
                    }
                    copies_arrive(&f_full[s]);
                }
            }
            copies_done();
            if (!ok && lane == 0) fail();
        }
        __syncwarp();
        if (MODE == kMmCluster) cluster_sync();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::MORE));
        const int part = (warp - 4) >> 2, quad = warp & 3, half = TWO ? part : 0;
        const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + (TWO ? part * 256 : part * H), step = TWO ? H : BP * W;
        unsigned char* const pieces = smem + C::OUT_AT + (warp - 4) * 4096;
        const uint32_t t_free = cluster_addr(smem_addr(t_empty[half]), leader);
        unsigned gi = 0, s = 0, phase = 0, t = 0, stored = 0;
        bool ok = true, there = false;
        long long left = steps;
        float acc[C::COLS];
        auto output = [&](int tile, int lo, int hi) {      // of the warp's columns lo to hi
            const int tn = tile / tiles_m, m0 = (tile - tn * tiles_m) * ROWS + (int)rank * 128 + quad * 32;
            const int n0 = tn * W + part * H;
            // ---- the tile's output, in pieces of 64 bytes of the warp's 32 rows: by TMA where the rows are
            // aligned, else through the same place and registers, `vec` bytes a lane
            if (m0 >= a.M) return;
            auto piece = [&](unsigned char* at_, int r, int c) { return reinterpret_cast<uint4*>(at_ + r * 64 + ((c ^ (r >> 1 & 3)) << 4)); };
            auto send = [&](unsigned char* from_, int n) {
                if (by_tma) {
                    proxy_fence();
                    __syncwarp();
                    if (lane == 0) tma_store_2d(&omap, n, m0, smem_addr(from_));
                    ++stored;
                    return;
                }
                __syncwarp();
                const int elt = a.f32 ? 4 : 2, at_ = lane * vec & 63, step_ = vec / 2;          // rows at a time
                const bool have = n + at_ / elt < a.N;
                char* to = a.out + ((int64_t)(m0 + lane * vec / 64) * a.old + n) * elt + at_;
#pragma unroll 4
                for (int r = lane * vec / 64; r < 32; r += step_, to += (int64_t)step_ * a.old * elt) {
                    const unsigned char* x = reinterpret_cast<unsigned char*>(piece(from_, r, at_ >> 4)) + (at_ & 15);
                    if (!have || m0 + r >= a.M) continue;
                    if (vec == 8) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(x);
                    else if (vec == 4) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(x);
                    else *reinterpret_cast<unsigned short*>(to) = *reinterpret_cast<const unsigned short*>(x);
                }
                __syncwarp();
            };
            // (a piece's place is free again when the last store but one has been read)
            auto place = [&]() {
                if (by_tma) {
                    if (lane == 0) tma_store_wait<1>();
                    __syncwarp();
                }
                return pieces + (stored & 1) * 2048;
            };
            if (a.f32) {
#pragma unroll
                for (int c0 = 0; c0 < H; c0 += 16) {
                    if (n0 + c0 >= a.N) break;
                    if (MODE == kMmCluster && (c0 < lo || c0 >= hi)) continue;
                    unsigned char* to = place();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float* x = acc + c0 + 4 * c;
                        *piece(to, lane, c) =
                            make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
                    }
                    send(to, n0 + c0);
                }
            } else {
#pragma unroll
                for (int c0 = 0; c0 < H; c0 += 32) {
                    if (n0 + c0 >= a.N) break;
                    if (MODE == kMmCluster && (c0 < lo || c0 >= hi)) continue;
                    unsigned char* to = place();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float* x = acc + c0 + 8 * c;
                        *piece(to, lane, c) =
                            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
                    }
                    send(to, n0 + c0);
                }
            }
        };
        for (int tile = first_tile, at = first_b; left > 0; tile += turn, at = 0) {
            const int end = (int)min((long long)blocks, at + left);
            left -= end - at;
            const int n0 = tile / tiles_m * W + part * H;
            const int split = (n0 / kScaleBlock + 1) * kScaleBlock - n0;     // columns of the first block
#pragma unroll
            for (int c = 0; c < C::COLS; ++c) acc[c] = 0.f;
            for (int b4 = at; ok && b4 < end; b4 += 4, ++gi) {
                const unsigned char* scales = smem + C::F_AT + gi % C::FS * C::F_BYTES;
                ok = wait_warp(&f_full[gi % C::FS], (gi / C::FS) & 1, limit);
                if (!ok) break;
                const float4 fx = *reinterpret_cast<const float4*>(scales + (quad * 32 + lane) * 16);
                const float4 fw = *reinterpret_cast<const float4*>(scales + 128 * 16 + part * 32);
                const float4 fv = CROSS ? *reinterpret_cast<const float4*>(scales + 128 * 16 + part * 32 + 16) : fw;
                const float f[4] = {fx.x * fw.x, fx.y * fw.y, fx.z * fw.z, fx.w * fw.w};
                const float g[4] = {fx.x * fv.x, fx.y * fv.y, fx.z * fv.z, fx.w * fv.w};
                // the group before has been taken; this one may still be on its way from shared memory
                if (lane == 0 && gi > 0) mbar_arrive(&f_empty[(gi - 1) % C::FS]);
#pragma unroll
                for (int j = 0; j < 4; j += BP) {
                    if (!ok || b4 + j >= end) continue;
                    if (!PEEK || !there) ok = wait_warp(&done[half][s], phase, limit);
                    if (!ok) continue;
                    tc_after();
                    constexpr int L = 16;                  // columns a load
                    const uint32_t at_ = from + t * step;
                    const bool all = b4 + j + BP <= end;
                    float v[2][L];
                    tc_ld16_start(at_, v[0]);
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1;
                    }
#pragma unroll
                    for (int c = 0; c < BP * H; c += L) {
                        if (BP > 1 && c == H && !all) break;
                        float* now = v[(c / L) & 1];
                        tc_wait_ld();
                        tc_ld16_done(now);
                        const int next = c + L;
                        if (next < BP * H && (next != H || all)) {
                            tc_ld16_start(at_ + next / H * W + next % H, v[(next / L) & 1]);
                        } else {
                            tc_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(t_free + t * 8);
                            // (the next step's products: the answer comes while the last sums are made)
                            if (PEEK) there = phase_done(&done[half][s], phase);
                        }
                        const float fg = !CROSS || c < split ? f[j + c / H] : g[j];
#pragma unroll
                        for (int e = 0; e < L; e += 2) {
                            float* to = acc + c % H + e;
                            f2_unpack(f2_fma(f2_pack(now[e], now[e + 1]), f2_pack(fg, fg), f2_pack(to[0], to[1])), to[0], to[1]);
                        }
                    }
                    if (PEEK) there = __all_sync(0xffffffffu, there);
                    if (++t == buffers) t = 0;
                }
            }
            if (!ok) {                                     // a result that is not valid shows
#pragma unroll
                for (int c = 0; c < C::COLS; ++c) acc[c] = CUDART_NAN_F;
            }
            if (MODE == kMmCluster) break;
            if (MODE == kMmTickets && end - at < blocks) {
                const MmParts parts(plan, tile);
                const int n = parts.p1 - parts.p0 + 1, w = (int)rank * C::EW + warp - 4;
                unsigned long long* ticket = reinterpret_cast<unsigned long long*>(a.ws + kMmTicketAt) + parts.p0 * 16 + w;
                auto part_of = [&](int p) {
                    return reinterpret_cast<float4*>(parts.part(plan, a.ws, p)) + (size_t)w * (C::PART / 4) + lane;
                };
                auto add = [&](int p) {
                    const float4* q = part_of(p);
                    constexpr int B = H < 32 ? H / 4 : 8, NBATCH = H / (4 * B);     // loads of a batch; one ahead
                    float4 x[2][B];
#pragma unroll
                    for (int c = 0; c < B; ++c) x[0][c] = __ldcg(q + 4 * c * 8);
#pragma unroll
                    for (int k = 0; k < NBATCH; ++k) {
                        if (k + 1 < NBATCH) {
#pragma unroll
                            for (int c = 0; c < B; ++c) x[(k + 1) & 1][c] = __ldcg(q + ((k + 1) * B + c) * 4 * 8);
                        }
#pragma unroll
                        for (int c = 0; c < B; ++c) {
                            float* to = acc + (k * B + c) * 4;
                            const float4 y = x[k & 1][c];
                            to[0] += y.x;
                            to[1] += y.y;
                            to[2] += y.z;
                            to[3] += y.w;
                        }
                    }
                };
                // (of two parts, the second to be ready need not be written: their order does not matter)
                bool second = false;
                if (n == 2) {
                    second = __any_sync(0xffffffffu, lane == 0 && tickets_taken(*reinterpret_cast<volatile unsigned long long*>(ticket), plan.tag) == 1);
                }
                if (!second) {
                    float4* mine = part_of(pair);
#pragma unroll
                    for (int c = 0; c < H; c += 4) __stcg(mine + c * 8, make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]));
                }
                if (!last_ticket(ticket, plan.tag, n, lane)) continue;
                if (n > 2) {
#pragma unroll
                    for (int c = 0; c < C::COLS; ++c) acc[c] = 0.f;
                }
#pragma unroll 1
                for (int p = parts.p0; p <= parts.p1; ++p)
                    if (n > 2 || p != pair) add(p);
            }
            output(tile, 0, H);
        }
        if (MODE == kMmCluster) {
            // The sums of the cluster's pairs (or CTAs) over distributed shared memory, in their order: each finishes
            // its share of the tile's columns, of 32 at least.  (They lie in the ring, which is free once the last
            // products are complete; where a wait ran out, copies may still arrive there.)
            static_assert(MODE != kMmCluster || !TWO, "a warp has seen all products complete");
            float* sums = reinterpret_cast<float*>(smem + (warp - 4) * H * 128) + lane;       // [column][row]
#pragma unroll
            for (int c = 0; c < H; ++c) sums[c * 32] = acc[c];
            if (!ok && lane == 0) fail();
            cluster_sync();
            const int share = max(1, W / 32 / plan.split) * 32, at = (int)place / CTAS * share, lo = at - part * H;
            if (at < W && lo >= 0 && lo < H) {
#pragma unroll
                for (int c = 0; c < H; ++c) acc[c] = 0.f;
#pragma unroll 1
                for (int p = 0; p < plan.split; ++p) {
                    const uint32_t from_ = cluster_addr(smem_addr(sums), CTAS * p + rank);
#pragma unroll
                    for (int c0 = 0; c0 < H; c0 += 32) {
                        if (c0 < lo || c0 >= lo + share) continue;
                        float x[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c) x[c] = ld_cluster(from_ + (c0 + c) * 128);
#pragma unroll
                        for (int c = 0; c < 32; ++c) acc[c0 + c] += x[c];
                    }
                    if (__float_as_int(ld_cluster(cluster_addr(smem_addr(&failed), CTAS * p + rank))) != 0) ok = false;
                }
                if (!ok) {
#pragma unroll
                    for (int c = 0; c < H; ++c) acc[c] = CUDART_NAN_F;
                }
                output(first_tile, lo, lo + share);
            }
        }
        if (lane == 0) tma_store_wait<0>();
        __syncwarp();
        if (!ok && lane == 0) fail();
    }
    tc_before();
    __syncthreads();
    if (failed) cluster_sync();                            // (arrivals that nobody has waited for)
    else cluster_meet();
    tc_after();
    if (warp == 1) {
        if (PAIR) pair_dealloc(tmem, 512);
        else tc_dealloc(tmem, 512);
    }
}

// ---- launches -----------------------------------------------------------------------
static bool map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* base, int64_t inner, int64_t rows, int64_t stride_bytes, int box_inner,
                   int box_rows, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return encoder() && encoder()(m, type, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename... KArgs, typename... Args>
static cudaError_t launch_clusters(void (*kfn)(KArgs...), int grid, int cluster, int threads, int smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kfn, args...);
}

static uint32_t wait_limit() { return ring_wait_limit() < kTcWaitLimit ? ring_wait_limit() : kTcWaitLimit; }

// How many clusters of n CTAs run at once (they stay within groups of SMs).
template <typename... KArgs>
static cudaError_t clusters_at_once(int* count, void (*kfn)(KArgs...), int n, int threads, int smem) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(8 * n));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(count, kfn, &cfg);
}

static bool rows_aligned(const MatmulArgs& a) { return is_aligned(a.out, 16) && a.old * (a.f32 ? 4 : 2) % 16 == 0; }

// What a device answers once: for each place of most, how many clusters run at once.  (Threads that ask
// at the same time write the same answers; one look-up a call, as asking for the device takes the host
// 30 ns.)
template <int N>
struct Clusters {
    std::atomic<int> ready[kMaxDevices] = {}, most[kMaxDevices][N] = {};
    template <typename F>
    cudaError_t get(int (&out)[N], F ask) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const bool kept = dev >= 0 && dev < kMaxDevices;
        if (kept && ready[dev].load(std::memory_order_acquire)) {
            for (int i = 0; i < N; ++i) out[i] = most[dev][i].load(std::memory_order_relaxed);
            return cudaSuccess;
        }
        for (int i = 0; i < N; ++i) {
            e = ask(i, &out[i]);
            if (e != cudaSuccess) return e;
            if (kept) most[dev][i].store(out[i], std::memory_order_relaxed);
        }
        if (kept) ready[dev].store(1, std::memory_order_release);
        return cudaSuccess;
    }
};

// Clusters of 1 to 8 CTAs.  The occupancy query takes a kernel that allocates tensor memory for one that
// wants an SM to itself: it is two, as shared memory and tensor memory are divided here.
template <int T>
static cudaError_t few_clusters(int (&most)[8]) {
    using C = FewCfg<T>;
    static Clusters<8> table;
    return table.get(most, [](int i, int* o) {
        cudaError_t e = cudaFuncSetAttribute(matmul_few_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e == cudaSuccess) e = clusters_at_once(o, matmul_few_kernel<T>, i + 1, C::THREADS, C::SMEM);
        *o *= C::CTAS;
        return e;
    });
}

template <int T, bool ANY = false>
static cudaError_t launch_few_t(const MatmulArgs& a, cudaStream_t st) {
    using C = FewCfg<T>;
    const auto kfn = matmul_few_kernel<T, ANY>;
    int most[8];
    cudaError_t e = few_clusters<T>(most);
    if (ANY && e == cudaSuccess) {
        static DeviceSlots slots = {};
        int unused = 0;
        e = device_once(slots, &unused, [&](int, int* o) {
            *o = 1;
            return cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        });
    }
    if (e != cudaSuccess) return e;
    const int tiles = (a.N - 1) / kMmTile + 1, blocks = scale_blocks(a.K);
    // Of the clusters of which all run at once, those that take the least: a CTA's blocks one after the other,
    // and the join (measured at N = 1024, K = 512 to 4096; more tiles only wait for memory).  One row, N =
    // 6144, K = 4096, 48 tiles: 6.3 us in clusters of five, of which 56 fit; 7.5 in four, 9.6 in six, of
    // which 46 do.  (Before a kernel's end lost its release: five take 5.9 now.)
    constexpr double kStep = T <= 16 ? 0.17 : T <= 32 ? 0.22 : 0.28;
    constexpr double kJoin[9] = {0, 0, 1.2, 0.9, 0.8, 1.0, 1.1, 1.3, 1.5};
    int S = 1;
    double best = 1e300;
    for (int i = 1; i <= 8 && i <= blocks; ++i) {
        if (i > 1 && tiles > most[i - 1]) continue;
        const int own = (blocks + i * C::BP - 1) / (i * C::BP) * C::BP;
        const double us = own * kStep + (i == 1 ? 0.0 : T <= 16 ? 1.3 : kJoin[i]);
        if (us <= best) {
            best = us;
            S = i;
        }
    }
    CUtensorMap xm, wm, sm = {};
    if (!map_2d(&xm, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x, a.K, a.M, a.xld, kMmTile, T, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !map_2d(&wm, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, a.K, a.N, a.wld, kMmTile, kMmTile, CU_TENSOR_MAP_SWIZZLE_128B) ||
        (!ANY && !map_2d(&sm, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.xscale, a.M, blocks, a.xs_stride * 4, T, C::BP, CU_TENSOR_MAP_SWIZZLE_NONE)))
        return cudaErrorInvalidValue;
    return launch_clusters(kfn, tiles * S, S, C::THREADS, C::SMEM, st, a, wait_limit(), blocks, S, rows_aligned(a), xm, wm, sm);
}

// What a block of a tile W columns wide takes, and a tile's end (us, measured at 512 rows, as many tiles
// as pairs, or as single CTAs, fit at once, and K = 1024 to 8192).  They know no memory: where the weights'
// bytes bound a call, at 65 to 256 rows, it takes longer than they say (128 x 24576 x 4096: 22.3 us for 14.5, 128 x
// 4096 x 12288: 16.6 for 10.8).
struct MmWidth {
    int W;
    double step, end;
};
constexpr MmWidth kMmPairs[4] = {{64, 0.16, 0.8}, {128, 0.245, 1.3}, {192, 0.345, 1.7}, {256, 0.405, 1.9}};
constexpr MmWidth kMmSingles[4] = {{64, 0.19, 0.8}, {128, 0.28, 1.3}, {192, 0.4, 1.7}, {256, 0.44, 1.9}};
// Joining a cluster's sums: of two, four and eight.
constexpr double kMmJoin[3] = {0.9, 2.2, 3.6};

// Whole tiles in the width whose rounds of all pairs or CTAs take the least, or equal shares, whose parts
// cost their writing and reading, where that is less: few tiles with long contractions, or
// little more than whole rounds.
static MmPlan plan_many(int M, int N, int K, int sms, const int (&clusters)[3]) {
    MmPlan p = {};
    p.blocks = scale_blocks(K);
    const long long pairs_most = sms / 2 < kMmMaxPairs ? sms / 2 : kMmMaxPairs;
    double best = 1e300;
    for (int single = 0; single < 2; ++single) {
        const int tiles_m = single ? (M - 1) / 128 + 1 : (M - 1) / 256 + 1;
        const long long most = single ? sms : pairs_most;
        for (const MmWidth& w : single ? kMmSingles : kMmPairs) {
            const long long tiles = (long long)tiles_m * ((N - 1) / w.W + 1), total = tiles * p.blocks;
            const auto take = [&](double us, long long pairs, int whole, int split) {
                if (us >= best) return;
                best = us;
                p.W = w.W;
                p.pair = !single;
                p.tiles_m = tiles_m;
                p.whole = whole;
                p.tiles = tiles;
                p.total = total;
                p.pairs = (int)pairs;
                p.split = split;
            };
            take((double)((tiles + most - 1) / most) * (p.blocks * w.step + w.end), tiles < most ? tiles : most, 1, 1);
            // Clusters, of up to eight CTAs.  (Of the wider tiles, two pairs only were the fastest anywhere:
            // 256 rows, 4096 x 12288: 19.1 us for 20.8 with whole tiles of 64.)
            for (int i = 0; i < (w.W == 64 ? (single ? 3 : 2) : w.W == 128 && !single ? 1 : 0); ++i) {
                const int split = 2 << i;
                if (tiles <= clusters[single ? i : i + 1] && split <= p.blocks)
                    take((p.blocks + split - 1) / split * w.step + w.end + kMmJoin[i], tiles * split, 1, split);
            }
            // Shares.  (Of tiles of 64 beside clusters with tiles of 128, which came later: 221 x 1175 x 32304 27.8 us for 35.0, 195 x
            // 4992 x 15872 34.3 for 36.7, but eight other sizes of ten that take them 0 to 30 % slower, 501 x 2616 x 15952
            // 41.6 for 31.6: their cost is set too low.)
            if (single || (w.W != 64 && w.W != 256)) continue;
            for (int n = 2; n <= 8; ++n) {
                // (n: parts of a tile)
                const long long pairs = tiles * n < most ? tiles * n : most;
                if (tiles * (n - 1) >= most && n > 2) break;
                if (total < 4 * pairs) break;
                const long long steps = (total + pairs - 1) / pairs;
                take(1.1 * steps * w.step + ((double)steps / p.blocks + 1) * w.end + (w.W == 64 ? 3.5 + 2.0 * (n - 1) : 4.0 + 3.0 * (n - 1)), pairs, 0, 1);
            }
        }
    }
    return p;
}

template <int W, MmMode MODE, bool PAIR>
static cudaError_t launch_many_t(const MatmulArgs& a, const MmPlan& p, cudaStream_t st) {
    using C = ManyCfg;
    auto kfn = matmul_many_kernel<W, MODE, PAIR>;
    constexpr int CTAS = PAIR ? 2 : 1;
    static DeviceSlots slots = {};
    int unused = 0;
    cudaError_t e = device_once(slots, &unused, [&](int, int* o) {
        *o = 1;
        return cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    const int elt = a.f32 ? 4 : 2;
    // (a TMA store writes whole 16 bytes, also where its tensor ends inside them)
    const bool by_tma = rows_aligned(a) && (int64_t)a.N * elt % 16 == 0 && a.old * elt < (1LL << 40);
    // else the widest pieces that every row's begin and end allow
    const uint64_t align = reinterpret_cast<uintptr_t>(a.out) | (uint64_t)a.old * elt | (uint64_t)a.N * elt;
    const int vec = align % 8 == 0 ? 8 : align % 4 == 0 ? 4 : 2;
    CUtensorMap xm, wm, om = {};
    if (!map_2d(&xm, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x, a.K, a.M, a.xld, kMmTile, kMmTile, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !map_2d(&wm, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, a.K, a.N, a.wld, kMmTile, PAIR && two_halves(W) ? W / 4 : W / CTAS, CU_TENSOR_MAP_SWIZZLE_128B) ||
        (by_tma && !map_2d(&om, a.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.out, a.N, a.M, a.old * elt,
                           64 / elt, 32, CU_TENSOR_MAP_SWIZZLE_64B)))
        return cudaErrorInvalidValue;
    return launch_clusters(kfn, p.pairs * CTAS, MODE == kMmCluster ? CTAS * p.split : CTAS, C::THREADS, C::SMEM, st, a, wait_limit(), p, xm, wm, om, by_tma, vec);
}

// Clusters of two, four and eight CTAs.
static cudaError_t many_clusters(int (&most)[3]) {
    using C = ManyCfg;
    static Clusters<3> table;
    return table.get(most, [](int i, int* o) {
        const auto kfn = matmul_many_kernel<64, kMmCluster, false>;
        const cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        return e != cudaSuccess ? e : clusters_at_once(o, kfn, 2 << i, C::THREADS, C::SMEM);
    });
}

template <bool PAIR>
static cudaError_t launch_whole(const MatmulArgs& a, const MmPlan& p, cudaStream_t st) {
    if (PAIR && p.split > 1 && p.W == 128) return launch_many_t<128, kMmCluster, true>(a, p, st);
    if (p.split > 1) return launch_many_t<64, kMmCluster, PAIR>(a, p, st);
    switch (p.W) {
        case 64: return launch_many_t<64, kMmWhole, PAIR>(a, p, st);
        case 128: return launch_many_t<128, kMmWhole, PAIR>(a, p, st);
        case 192: return launch_many_t<192, kMmWhole, PAIR>(a, p, st);
        default: return launch_many_t<256, kMmWhole, PAIR>(a, p, st);
    }
}

static bool tiles_fit(int M, int N) { return (long long)((M - 1) / 128 + 1) * ((N - 1) / 64 + 1) < (1LL << 31); }

static cudaError_t launch_many(const MatmulArgs& a, int sms, cudaStream_t st) {
    if (!tiles_fit(a.M, a.N)) return cudaErrorInvalidValue;
    int clusters[3];
    const cudaError_t e = many_clusters(clusters);
    if (e != cudaSuccess) return e;
    MmPlan p = plan_many(a.M, a.N, a.K, sms, clusters);
    // (times an odd number: one tag a launch as before, but none that small numbers left in a workspace could be)
    p.tag = next_launch_tag() * 0x9e3779b97bull & ((1ull << 40) - 1);
    if (!p.whole) return p.W == 64 ? launch_many_t<64, kMmTickets, true>(a, p, st) : launch_many_t<256, kMmTickets, true>(a, p, st);
    return p.pair ? launch_whole<true>(a, p, st) : launch_whole<false>(a, p, st);
}

// (Which calls of more rows share tiles depends on the device too, which is not asked here: all have room for parts, 42 MB.)
size_t matmul_workspace_size(int M, int, int) { return M <= kMmFew ? kMmTicketAt : kMmPartAt + 2 * kMmMaxPairs * kMmPartBytes; }

cudaError_t matmul_plan(int M, int N, int K, int sms, const int* clusters, int (&out)[5]) {
    if (M <= kMmFew) {
        out[0] = SPEC_MATMUL_FEW, out[1] = kMmTile, out[2] = 1, out[3] = 0, out[4] = 0;
        return cudaSuccess;
    }
    if (!tiles_fit(M, N)) return cudaErrorInvalidValue;
    int most[3];
    if (sms > 0) {
        for (int i = 0; i < 3; ++i) most[i] = clusters[i];
    } else {
        DeviceInfo di;
        cudaError_t e = device_info(&di);
        if (e == cudaSuccess) e = many_clusters(most);
        if (e != cudaSuccess) return e;
        sms = di.sm_count;
    }
    const MmPlan p = plan_many(M, N, K, sms, most);
    out[0] = !p.whole ? SPEC_MATMUL_SHARES : p.split > 1 ? SPEC_MATMUL_CLUSTERS : SPEC_MATMUL_WHOLE;
    out[1] = p.W;
    out[2] = p.pair ? 2 : 1;
    out[3] = p.pairs;
    out[4] = p.split;
    if (!p.whole) {
        for (long long t = 0; t < p.tiles; ++t) {
            const int n = p.of((t + 1) * p.blocks - 1) - p.of(t * p.blocks) + 1;
            if (n > out[4]) out[4] = n;
        }
    }
    return cudaSuccess;
}

cudaError_t launch_matmul(const MatmulArgs& a, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    if (a.M > kMmFew) return launch_many(a, di.sm_count, st);
    if (a.M == 1 && !(is_aligned(a.xscale, 16) && a.xs_stride % 4 == 0)) return launch_few_t<16, true>(a, st);
    return a.M <= 16 ? launch_few_t<16>(a, st) : a.M <= 32 ? launch_few_t<32>(a, st) : launch_few_t<64>(a, st);
}

}  // namespace sv
