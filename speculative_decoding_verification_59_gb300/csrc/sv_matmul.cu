// Products of 8-bit matrices with a scale for each block of 128, on the
// fifth-generation tensor cores:
//   out[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{k in block b} x[m, k] w[n, k].
// The scales change with every 128 elements of the contraction, so an
// accumulator in tensor memory holds one block's products only.  The inner sums
// are exact to fp32; the warps that read them add them, times the two scales, to
// running sums in registers, while the next blocks' products run into the other
// accumulators.
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
// A scale.  (Not a read-only load, which could move ahead of the wait for the kernel before.)
__device__ __forceinline__ float ld_scale(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// wait_bounded for a barrier that the other CTA of the pair arrives on.
__device__ __forceinline__ bool wait_bounded_cluster(uint64_t* bar, uint32_t parity, uint32_t limit) {
    for (uint32_t i = 0; i < limit; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
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
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
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
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_addr(bar)),
                 "h"((unsigned short)3)
                 : "memory");
}
// 32 columns of the warp's 32 lanes; nothing may use v before tc_wait_ld and ld32_done.
__device__ __forceinline__ void tc_ld32_start(uint32_t at, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
          "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
          "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
          "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(at));
}
__device__ __forceinline__ void tc_ld32_done(float* v) {
    tc_ld16_done(v);
    tc_ld16_done(v + 16);
}

// ---- few rows ----------------------------------------------------------------------
// Up to 128 rows of x: the product is taken transposed, so that 128 weight rows are the
// rows that the instruction wants and the few rows of x its free dimension T.  The weights are
// read once, which bounds these calls.  A tile of 128 weight rows is shared by a cluster of S
// CTAs, each with its part of the contraction; they add their sums over distributed shared
// memory, in the order of their ranks, each a part of the columns.
//   warp 0     loads: both operands and the rows' scales of a step into a ring, by TMA
//   warp 1     issues the products
//   warps 2-5  running sums: a thread owns a weight row, the rows' scales are read from shared
//              memory, the weights' scale is the tile's
template <int T>
struct FewCfg {
    static constexpr int SCALE = T * 4 < 128 ? 128 : T * 4;
    static constexpr int STAGES = T <= 32 ? 5 : T <= 64 ? 4 : 3;
    static constexpr int NB = T <= 64 ? 4 : 2;            // accumulators
    static constexpr int TMEM = NB * T;                   // columns: 64, 128, 256, 256
    static constexpr int X_AT = kMmBytes, STAGE = kMmBytes + T * kMmTile;
    static constexpr int SCALE_AT = STAGES * STAGE;
    static constexpr int SMEM = SCALE_AT + STAGES * SCALE + 1024;        // and room to align
    static constexpr int THREADS = 192;
    static_assert(2 * (SMEM + 2048) <= 228 * 1024, "two CTAs an SM");
    static_assert(T * 512 <= SCALE_AT, "the sums of a CTA fit the ring");
};

template <int T>
__global__ void __launch_bounds__(FewCfg<T>::THREADS, 2) matmul_few_kernel(const MatmulArgs a, uint32_t limit,
                                                                          const __grid_constant__ CUtensorMap xmap,
                                                                          const __grid_constant__ CUtensorMap wmap,
                                                                          const __grid_constant__ CUtensorMap smap, int S) {
    using C = FewCfg<T>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[C::STAGES], empty[C::STAGES], t_full[C::NB], t_empty[C::NB], drained;
    __shared__ uint32_t tmem_at;
    __shared__ int failed;
    unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tile = blockIdx.x / S, rank = blockIdx.x - tile * S;     // (a cluster: S consecutive CTAs)
    const int blocks = (a.K + kMmTile - 1) / kMmTile;
    const int b0 = (int)((long long)blocks * rank / S), n = (int)((long long)blocks * (rank + 1) / S) - b0;
    const int n0 = tile * kMmTile;

    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1 + 4);                   // the products, and four warps that read scales
        }
        for (int i = 0; i < C::NB; ++i) {
            mbar_init(&t_full[i], 1);
            mbar_init(&t_empty[i], 4);
        }
        mbar_init(&drained, 1);
        mbar_init_fence();
        failed = 0;
        // the first weights on their way into L2 while the kernel before ends
        for (int i = 0; i < C::STAGES && i < n; ++i) tma_prefetch_2d(&wmap, (b0 + i) * kMmTile, n0);
        map_prefetch(&xmap);
        map_prefetch(&smap);
    }
    if (warp == 1) tc_alloc(&tmem_at, C::TMEM);
    pdl_trigger();
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tmem_at;
    pdl_wait();

    f32x2 acc[T / 2];
    if (warp == 0) {
        if (lane == 0) {
            int i = 0;
            for (; i < n; ++i) {
                const int s = i % C::STAGES;
                if (i >= C::STAGES && !wait_bounded(&empty[s], (i / C::STAGES - 1) & 1, limit)) break;
                const uint32_t at = smem_addr(smem + s * C::STAGE);
                mbar_arrive_expect_tx(&full[s], C::STAGE + T * 4);
                tma_2d(at, &wmap, (b0 + i) * kMmTile, n0, &full[s]);
                tma_2d(at + C::X_AT, &xmap, (b0 + i) * kMmTile, 0, &full[s]);
                tma_2d(smem_addr(smem + C::SCALE_AT + s * C::SCALE), &smap, 0, b0 + i, &full[s]);
            }
            if (i < n) failed = 1;
            // every copy has landed and every commit has arrived before the CTA ends
            for (int j = max(0, i - C::STAGES); j < i; ++j) {
                const int s = j % C::STAGES;
                const uint32_t parity = (j / C::STAGES) & 1;
                if (!wait_bounded(&full[s], parity, kTcWaitLimit) || !wait_bounded(&empty[s], parity, limit)) failed = 1;
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t id = tc_idesc(true, false, false, T);
            bool ok = true;
            int i = 0;
            for (; i < n; ++i) {
                const int s = i % C::STAGES, t = i % C::NB;
                ok = wait_bounded(&full[s], (i / C::STAGES) & 1, limit) &&
                     (i < C::NB || wait_bounded(&t_empty[t], (i / C::NB - 1) & 1, limit));
                if (!ok) break;
                tc_after();
                const uint32_t at = smem_addr(smem + s * C::STAGE);
                const uint64_t wd = tc_desc(at, 16, 1024), xd = tc_desc(at + C::X_AT, 16, 1024);
#pragma unroll
                for (int k = 0; k < 4; ++k) tc_mma<true>(tmem + t * T, wd + 2 * k, xd + 2 * k, id, k > 0);
                tc_commit(&empty[s]);
                tc_commit(&t_full[t]);
            }
            if (!ok) {
                failed = 1;
                if (i > 0) {
                    tc_commit(&drained);
                    wait_bounded(&drained, 0, kTcWaitLimit);
                }
            }
        }
    } else {
        const int quad = warp & 3;
        const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16);
#pragma unroll
        for (int c = 0; c < T / 2; ++c) acc[c] = 0;
        const float* wsc = a.wscale + (int64_t)tile * a.ws_stride + b0;
        float wnext = ld_scale(wsc);
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int s = i % C::STAGES, t = i % C::NB;
            const f32x2 w2 = f2_pack(wnext, wnext);
            if (i + 1 < n) wnext = ld_scale(wsc + i + 1);
            ok = wait_bounded(&t_full[t], (i / C::NB) & 1, limit);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_after();
            const float4* xs = reinterpret_cast<const float4*>(smem + C::SCALE_AT + s * C::SCALE);
            float v[2][16];
            tc_ld16_start(from + t * T, v[0]);
#pragma unroll
            for (int c = 0; c < T; c += 16) {
                float* now = v[(c >> 4) & 1];
                tc_wait_ld();
                tc_ld16_done(now);
                if (c + 16 < T) tc_ld16_start(from + t * T + c + 16, v[((c >> 4) + 1) & 1]);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 f = xs[(c + e) >> 2];
                    f32x2& p = acc[(c + e) >> 1];
                    f32x2& q = acc[((c + e) >> 1) + 1];
                    p = f2_fma(f2_pack(now[e], now[e + 1]), f2_mul(f2_pack(f.x, f.y), w2), p);
                    q = f2_fma(f2_pack(now[e + 2], now[e + 3]), f2_mul(f2_pack(f.z, f.w), w2), q);
                }
            }
            tc_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&t_empty[t]);
                mbar_arrive(&empty[s]);
            }
        }
        if (!ok && lane == 0) failed = 1;
    }
    tc_before();
    __syncthreads();                                       // every product is done, the ring is free
    tc_after();
    const int row = (warp & 3) * 32 + lane;                // of the tile (warps 2 to 5)
    const float bad = failed ? CUDART_NAN_F : 0.f;         // a result that is not valid shows
    if (failed && tid == 0) raise_error(reinterpret_cast<int32_t*>(a.ws), SPEC_DEVERR_TIMEOUT);
    auto put = [&](int m, float v) {
        const int64_t at = (int64_t)m * a.old + n0 + row;
        if (a.f32) reinterpret_cast<float*>(a.out)[at] = v;
        else reinterpret_cast<unsigned short*>(a.out)[at] = (unsigned short)(pack_bf16(v, 0.f) & 0xffffu);
    };
    if (S == 1) {
        if (warp >= 2 && n0 + row < a.N) {
#pragma unroll
            for (int c = 0; c < T; c += 2) {
                float lo, hi;
                f2_unpack(acc[c >> 1], lo, hi);
                if (c < a.M) put(c, lo + bad);
                if (c + 1 < a.M) put(c + 1, hi + bad);
            }
        }
    } else {
        float* sums = reinterpret_cast<float*>(smem);      // [column][weight row]
        if (warp >= 2) {
#pragma unroll
            for (int c = 0; c < T; c += 2) {
                float lo, hi;
                f2_unpack(acc[c >> 1], lo, hi);
                if (c < a.M) sums[c * kMmTile + row] = lo + bad;
                if (c + 1 < a.M) sums[(c + 1) * kMmTile + row] = hi + bad;
            }
        }
        cluster_sync();
        if (warp >= 2 && n0 + row < a.N) {
            const uint32_t mine = smem_addr(sums) + row * 4;
            for (int c = rank; c < a.M; c += S) {
                float v = 0.f;
                for (int r = 0; r < S; ++r) v += ld_cluster(cluster_addr(mine + c * kMmTile * 4, r));
                put(c, v);
            }
        }
        cluster_sync();                                    // no CTA ends while another reads its sums
    }
    if (warp == 1) tc_dealloc(tmem, C::TMEM);
}

// ---- many rows ---------------------------------------------------------------------
// A pair of CTAs takes 256 rows of x times T weight rows (cta_group::2: each loads its 128
// rows of x and half of the weight rows, and holds its 128 rows' sums), and goes on to
// further tiles.  A thread of the sums owns a row of x and half of a tile's columns, which lie in one
// 128-block of the weights: the two scales of a step are one factor.
//   warp 0      loads, warp 1 issues the products (the pair's first CTA, for both)
//   warps 4-11  running sums, then the tile's output
template <int T>
struct ManyCfg {
    static constexpr int NB = 512 / T > 4 ? 4 : 512 / T;  // accumulators
    static constexpr int TMEM = NB * T;
    static constexpr int X_BYTES = kMmBytes, W_BYTES = T / 2 * kMmTile, STAGE = X_BYTES + W_BYTES;
    static constexpr int STAGES = 192 * 1024 / STAGE > 8 ? 8 : 192 * 1024 / STAGE;
    static constexpr int OUT_AT = STAGES * STAGE;         // 4 KB of a warp's output
    static constexpr int SMEM = OUT_AT + 8 * 4096 + 1024;
    static constexpr int HALF = T / 2;
    static constexpr int THREADS = 384;
    static_assert(SMEM <= 227 * 1024, "dynamic shared memory");
};

template <int T>
__global__ void __launch_bounds__(ManyCfg<T>::THREADS, 1) matmul_many_kernel(const MatmulArgs a, uint32_t limit, int tiles_m, int tiles,
                                                                            const __grid_constant__ CUtensorMap xmap,
                                                                            const __grid_constant__ CUtensorMap wmap) {
    using C = ManyCfg<T>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[C::STAGES], empty[C::STAGES], t_full[C::NB], t_empty[C::NB], drained;
    __shared__ uint32_t tmem_at;
    unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int blocks = (a.K + kMmTile - 1) / kMmTile;
    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::NB; ++i) {
            mbar_init(&t_full[i], 1);
            mbar_init(&t_empty[i], 2 * 8);                 // both CTAs' warps
        }
        mbar_init(&drained, 1);
        mbar_init_fence();
        map_prefetch(&xmap);
        map_prefetch(&wmap);
    }
    if (warp == 1) pair_alloc(&tmem_at, C::TMEM);
    pdl_trigger();
    tc_before();
    cluster_sync();
    tc_after();
    const uint32_t tmem = tmem_at;
    pdl_wait();
    int32_t* error = reinterpret_cast<int32_t*>(a.ws);

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0 && lane == 0) {
            unsigned it = 0;
            bool ok = true;
            for (int tile = pair; ok && tile < tiles; tile += pairs) {
                const int tn = tile / tiles_m, m0 = (tile - tn * tiles_m) * 256 + (int)rank * 128, n0 = tn * T + (int)rank * C::HALF;
                for (int b = 0; b < blocks; ++b, ++it) {
                    const unsigned s = it % C::STAGES;
                    if (it >= C::STAGES && !wait_bounded(&empty[s], (it / C::STAGES - 1) & 1, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = smem_addr(smem + s * C::STAGE), bar = cluster_addr(smem_addr(&full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE);
                    tma_2d_pair(at, &xmap, b * kMmTile, m0, bar);
                    tma_2d_pair(at + C::X_BYTES, &wmap, b * kMmTile, n0, bar);
                }
            }
            // every copy has landed and every commit has arrived before the CTA ends
            for (unsigned j = it > C::STAGES ? it - C::STAGES : 0; j < it; ++j) {
                const unsigned s = j % C::STAGES, parity = (j / C::STAGES) & 1;
                if (rank == 0 && !wait_bounded(&full[s], parity, kTcWaitLimit)) ok = false;
                if (!wait_bounded(&empty[s], parity, limit)) ok = false;
            }
            if (!ok) raise_error(error, SPEC_DEVERR_TIMEOUT);
        } else if (warp == 1 && rank == 0 && lane == 0) {
            const uint32_t id = tc_idesc(true, false, false, T, 256);
            unsigned it = 0;
            bool ok = true;
            for (int tile = pair; ok && tile < tiles; tile += pairs) {
                for (int b = 0; b < blocks; ++b, ++it) {
                    const unsigned s = it % C::STAGES, t = it % C::NB;
                    ok = wait_bounded_cluster(&full[s], (it / C::STAGES) & 1, limit) &&
                         (it < C::NB || wait_bounded_cluster(&t_empty[t], (it / C::NB - 1) & 1, limit));
                    if (!ok) break;
                    tc_after();
                    const uint32_t at = smem_addr(smem + s * C::STAGE);
                    const uint64_t xd = tc_desc(at, 16, 1024), wd = tc_desc(at + C::X_BYTES, 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k) pair_mma(tmem + t * T, xd + 2 * k, wd + 2 * k, id, k > 0);
                    pair_commit(&empty[s]);
                    pair_commit(&t_full[t]);
                }
            }
            if (!ok) {
                raise_error(error, SPEC_DEVERR_TIMEOUT);
                if (it > 0) {
                    pair_commit(&drained);
                    wait_bounded(&drained, 0, kTcWaitLimit);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int part = (warp - 4) >> 2, quad = warp & 3;
        const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + part * C::HALF;
        unsigned char* stage = smem + C::OUT_AT + (warp - 4) * 4096;
        unsigned it = 0;
        bool ok = true;
        for (int tile = pair; tile < tiles; tile += pairs) {
            const int tn = tile / tiles_m, m0 = (tile - tn * tiles_m) * 256 + (int)rank * 128 + quad * 32;
            const int n0 = tn * T + part * C::HALF, m = m0 + lane;
            f32x2 acc[C::HALF / 2];
#pragma unroll
            for (int c = 0; c < C::HALF / 2; ++c) acc[c] = 0;
            const float* xsc = a.xscale + m;
            const float* wsc = a.wscale + (int64_t)min(n0 / kScaleBlock, (a.N - 1) / kScaleBlock) * a.ws_stride;
            // factors of four steps ahead
            float f[4], g[4];
            auto load = [&](int b, int j) {
                const bool have = b < blocks && m < a.M;
                f[j] = have ? ld_scale(xsc + (int64_t)b * a.xs_stride) : 0.f;
                g[j] = b < blocks ? ld_scale(wsc + b) : 0.f;
            };
#pragma unroll
            for (int j = 0; j < 4; ++j) load(j, j);
            for (int b4 = 0; ok && b4 < blocks; b4 += 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!ok || b4 + j >= blocks) continue;
                    const unsigned t = it % C::NB;
                    const float fg = f[j] * g[j];
                    const f32x2 f2 = f2_pack(fg, fg);
                    load(b4 + j + 4, j);
                    ok = wait_bounded(&t_full[t], (it / C::NB) & 1, limit);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) continue;
                    tc_after();
                    float v[2][32];
                    tc_ld32_start(from + t * T, v[0]);
#pragma unroll
                    for (int c = 0; c < C::HALF; c += 32) {
                        float* now = v[(c >> 5) & 1];
                        tc_wait_ld();
                        tc_ld32_done(now);
                        if (c + 32 < C::HALF) {
                            tc_ld32_start(from + t * T + c + 32, v[((c >> 5) + 1) & 1]);
                        } else {
                            tc_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_addr(&t_empty[t]), 0));
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            acc[(c + e) >> 1] = f2_fma(f2_pack(now[e], now[e + 1]), f2, acc[(c + e) >> 1]);
                    }
                    ++it;
                }
            }
            // ---- the tile's output, 128 bytes (or a narrow tile's 64) of the warp's 32 rows at a time
            const float bad = ok ? 0.f : CUDART_NAN_F;
            const int elt = a.f32 ? 4 : 2;
            const bool wide = a.old * elt % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
            constexpr int G = C::HALF < 64 ? C::HALF : 64;  // columns at a time
#pragma unroll
            for (int c0 = 0; c0 < C::HALF; c0 += G) {
                if (n0 + c0 >= a.N) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {              // (fp32: 32 columns at a time)
                    if (h == 1 && (!a.f32 || G < 64)) break;
                    const int cols = a.f32 ? 32 : G, first = c0 + h * 32;
                    const int chunks = cols * elt / 16;    // 16-byte pieces of a row: 8, or 4
                    auto place = [&](int r, int c) {
                        return stage + (chunks == 8 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ (r >> 1 & 3)) << 4));
                    };
                    __syncwarp();
                    if (a.f32) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            float x0, x1, x2, x3;
                            f2_unpack(acc[(c0 + (h * 32) % G + 4 * c) >> 1], x0, x1);
                            f2_unpack(acc[((c0 + (h * 32) % G + 4 * c) >> 1) + 1], x2, x3);
                            *reinterpret_cast<float4*>(place(lane, c)) = make_float4(x0 + bad, x1 + bad, x2 + bad, x3 + bad);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < G / 8; ++c) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float lo, hi;
                                f2_unpack(acc[((c0 + 8 * c) >> 1) + e], lo, hi);
                                w[e] = pack_bf16(lo + bad, hi + bad);
                            }
                            *reinterpret_cast<uint4*>(place(lane, c)) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    __syncwarp();
                    const int per = 16 / elt;              // elements of a piece
                    for (int i = lane; i < 32 * chunks; i += 32) {
                        const int r = i / chunks, c = i - r * chunks, n = n0 + first + c * per;
                        if (m0 + r >= a.M || n >= a.N) continue;
                        char* to = a.out + ((int64_t)(m0 + r) * a.old + n) * elt;
                        const uint4 w = *reinterpret_cast<const uint4*>(place(r, c));
                        if (wide && n + per <= a.N) {
                            *reinterpret_cast<uint4*>(to) = w;
                        } else if (a.f32) {
                            for (int e = 0; e < 4 && n + e < a.N; ++e) reinterpret_cast<uint32_t*>(to)[e] = u4_get(w, e);
                        } else {
                            for (int e = 0; e < 8 && n + e < a.N; ++e)
                                reinterpret_cast<unsigned short*>(to)[e] = (unsigned short)(u4_get(w, e >> 1) >> 16 * (e & 1));
                        }
                    }
                }
            }
        }
        if (!ok && lane == 0) raise_error(error, SPEC_DEVERR_TIMEOUT);
    }
    tc_before();
    __syncthreads();
    cluster_sync();
    tc_after();
    if (warp == 1) pair_dealloc(tmem, C::TMEM);
}

// ---- launches -----------------------------------------------------------------------
static bool map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* base, int64_t inner, int64_t rows, int64_t stride_bytes, int box_inner,
                   int box_rows, bool swizzle) {
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride_bytes};
    const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return encoder() && encoder()(m, type, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

template <int T>
static cudaError_t launch_few_t(const MatmulArgs& a, int sms, cudaStream_t st) {
    using C = FewCfg<T>;
    auto kfn = matmul_few_kernel<T>;
    static DeviceSlots slots = {};
    int unused = 0;
    cudaError_t e = device_once(slots, &unused, [&](int, int* o) {
        *o = 1;
        return cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    const int tiles = (a.N - 1) / kMmTile + 1, blocks = scale_blocks(a.K);
    int S = 1;
    while (S < 8 && tiles * S * 2 <= 2 * sms && S * 2 <= blocks) S *= 2;
    CUtensorMap xm, wm, sm;
    if (!map_2d(&xm, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x, a.K, a.M, a.xld, kMmTile, T, true) ||
        !map_2d(&wm, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, a.K, a.N, a.wld, kMmTile, kMmTile, true) ||
        !map_2d(&sm, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.xscale, a.M, blocks, a.xs_stride * 4, T, 1, false))
        return cudaErrorInvalidValue;
    return launch_clusters(kfn, tiles * S, S, C::THREADS, C::SMEM, st, a, wait_limit(), xm, wm, sm, S);
}

template <int T>
static cudaError_t launch_many_t(const MatmulArgs& a, int sms, cudaStream_t st) {
    using C = ManyCfg<T>;
    auto kfn = matmul_many_kernel<T>;
    static DeviceSlots slots = {};
    int unused = 0;
    cudaError_t e = device_once(slots, &unused, [&](int, int* o) {
        *o = 1;
        return cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    const int tiles_m = (a.M - 1) / 256 + 1;
    const long long tiles = (long long)tiles_m * ((a.N - 1) / T + 1);
    if (tiles >= (1LL << 31)) return cudaErrorInvalidValue;
    const long long pairs = tiles < sms / 2 ? tiles : sms / 2;
    CUtensorMap xm, wm;
    if (!map_2d(&xm, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x, a.K, a.M, a.xld, kMmTile, kMmTile, true) ||
        !map_2d(&wm, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, a.K, a.N, a.wld, kMmTile, C::HALF, true))
        return cudaErrorInvalidValue;
    return launch_clusters(kfn, (int)pairs * 2, 2, C::THREADS, C::SMEM, st, a, wait_limit(), tiles_m, (int)tiles, xm, wm);
}

size_t matmul_workspace_size(int M, int N, int K) { return 256; }

cudaError_t launch_matmul(const MatmulArgs& a, cudaStream_t st) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    const int sms = di.sm_count;
    if (a.M <= 16) return launch_few_t<16>(a, sms, st);
    if (a.M <= 32) return launch_few_t<32>(a, sms, st);
    if (a.M <= 64) return launch_few_t<64>(a, sms, st);
    if (a.M <= 128) return launch_few_t<128>(a, sms, st);
    // the tile's width by the number of waves that it takes
    const long long tm = (a.M - 1) / 256 + 1, pairs = sms / 2;
    auto cost = [&](int T) { return (tm * ((a.N - 1) / T + 1) + pairs - 1) / pairs * (T + 32); };
    if (cost(256) <= cost(128) && cost(256) <= cost(64)) return launch_many_t<256>(a, sms, st);
    return cost(128) <= cost(64) ? launch_many_t<128>(a, sms, st) : launch_many_t<64>(a, sms, st);
}

}  // namespace sv
