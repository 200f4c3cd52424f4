// Log-probabilities of given tokens, with the entropy of their rows'
// distributions and the top alternatives, in one pass over the logits.
//
// With p = softmax(z / T), s = log2(e) / T, M = max z, a_j = (z_j - M) s:
//   Z = sum 2^a_j,  W = sum a_j 2^a_j,
//   ln p(x) = (z_x - M) / T - ln Z,   H = -sum p ln p = ln Z - ln 2 W / Z.
// Each 4 KB warp chunk of a row leaves its own maximum m with Z and W taken
// relative to it, and the elements that can still be among the row's top K;
// one CTA per row then brings the chunks to the common maximum and orders
// the candidates.
//
// The stream is a ring of bulk copies (one producer warp, kWarps consumer
// warps, 32 KB stages).  Rows may begin at any element: a row's chunks are cut
// from its 16-byte aligned span, and the neighbours' elements that share
// its first and last vectors are overwritten with -inf in shared memory.
// Every CTA takes a fixed contiguous range of chunks, so a call keeps nothing
// on the device and can be captured and replayed.
#include "sv_kv.h"
#include "sv_stream.cuh"

namespace sv {

constexpr int kMergeThreads = 128;
constexpr int kMergePool = 32;
constexpr float kArgFloor = -256.f;           // 2^-256 is zero in fp32, and -256 times it too
constexpr float kLn2f = 0.6931471805599453f;

struct LogprobArgs {
    const char* z;
    const int32_t* tok;
    float T, s;
    int rows, V, K, nseg;
    long long chunks;
    float4* stats;             // per warp chunk: m, Z, W (relative to m)
    float2* cand;              // per warp chunk: 2 KC candidates
    int* err;
    float *lp, *ent;
    int32_t* ti;
    float* tl;
    uint32_t wait_limit;
};

// A row's aligned span: its first byte, and the elements before the row in it.
__device__ __forceinline__ void row_span(const LogprobArgs& a, int elt, int r, long long* begin, int* lead, long long* bytes) {
    const long long at = (long long)r * a.V * elt;
    *begin = at & ~15LL;
    *lead = (int)(at - *begin) / elt;
    *bytes = (long long)*lead * elt + (long long)a.V * elt;
}

// (Z, W) of a warp chunk relative to its maximum m > -inf, over the warp.
// While m s is moderate the arguments are one FMA each, z s - fl(m s): off
// by the rounding r = m s - fl(m s), which the sums take back at the end
// (2^(a + r): Z = 2^-r Z', W = 2^-r W' - r Z).  Masked logits (-inf) would
// give 0 x inf in W; kArgFloor keeps their argument finite.
template <int ELT>
__device__ __forceinline__ void chunk_sums(const uint4 (&v)[kVecPerLane], float m, float s, float* Z, float* W) {
    const float ms = m * s;
    const bool direct = !(fabsf(ms) < kFmaArgLimit);
    const f32x2 s2 = f2_pack(s, s), off = direct ? f2_pack(0.f, 0.f) : f2_pack(-ms, -ms);
    const f32x2 sub = direct ? f2_pack(m, m) : f2_pack(0.f, 0.f);
    f32x2 z2 = f2_pack(0.f, 0.f), w2 = z2;
#pragma unroll
    for (int t = 0; t < kVecPerLane; ++t)
#pragma unroll
        for (int c = 0; c < 4; c += (ELT == 2 ? 1 : 2)) {
            f32x2 x;
            if constexpr (ELT == 2) {
                const uint32_t w = u4_get(v[t], c);
                x = f2_pack(bf16_lo(w), bf16_hi(w));
            } else {
                x = f2_pack(__uint_as_float(u4_get(v[t], c)), __uint_as_float(u4_get(v[t], c + 1)));
            }
            if (direct) x = f2_sub(x, sub);                    // uniform; tiny temperatures only
            float p, q;
            f2_unpack(f2_fma(x, s2, off), p, q);
            p = fmaxf(p, kArgFloor);
            q = fmaxf(q, kArgFloor);
            const f32x2 e = f2_pack(ex2_approx(p), ex2_approx(q));
            z2 = f2_add(z2, e);
            w2 = f2_fma(e, f2_pack(p, q), w2);
        }
    float z0, z1, w0, w1;
    f2_unpack(z2, z0, z1);
    f2_unpack(w2, w0, w1);
    const float zs = warp_sum(z0 + z1), ws = warp_sum(w0 + w1);
    const float r = direct ? 0.f : fmaf(m, s, -ms);
    const float f = direct ? 1.f : exp2f(-r);
    *Z = zs * f;
    *W = ws * f - r * (zs * f);
}

// The chunk's candidates for the row's top KC: as warp_topk_chunk
// (sv_stream.cuh), with elements outside the row (index below 0 or from V on)
// left out.  thr is a lower bound of the row's KC-th largest logit.
template <int ELT, int KC>
__device__ __forceinline__ void chunk_candidates(const uint4 (&v)[kVecPerLane], const unsigned char* chunk, int base,
                                                 int V, float2* out, float& thr, bool have_thr) {
    const int lane = threadIdx.x & 31;
    constexpr int PV = 16 / ELT;
    constexpr int KS = topk_slots(KC);
    if (!have_thr) {                                           // warp-uniform
        float x = lane_max<ELT>(v);
        thr = kNegInf;
#pragma unroll
        for (int r = 0; r < KC; ++r) {
            thr = warp_max(x);
            const unsigned own = __ballot_sync(0xffffffffu, x == thr);
            if (lane == __ffs(own) - 1) x = kNegInf;
        }
    }
    unsigned long long mask = 0ull;
    if constexpr (ELT == 2) {
        const uint32_t tb = __float_as_uint(thr) >> 16;        // a logit of the row or -inf: exact in bf16
        const uint32_t t2 = tb | (tb << 16);
        uint32_t lo = 0u, hi = 0u;
#pragma unroll
        for (int t = 0; t < kVecPerLane; ++t) {
            const uint32_t b = vec_ge_bits_bf16(v[t], t2);
            if (t < 4) lo |= b << (8 * t);
            else hi |= b << (8 * (t - 4));
        }
        mask = (unsigned long long)hi << 32 | lo;
    } else {
#pragma unroll
        for (int t = 0; t < kVecPerLane; ++t)
            if (vec_max_value<ELT>(vec_max_bits<ELT>(v[t])) >= thr) {
                unsigned bits = 0u;
#pragma unroll
                for (int e = 0; e < PV; ++e) bits |= (__uint_as_float(u4_get(v[t], e)) >= thr ? 1u : 0u) << e;
                mask |= (unsigned long long)bits << (8 * t);
            }
    }
    if (base < 0 || base + 32 * kLaneBytes / ELT > V) {        // warp-uniform: elements that are not the row's
#pragma unroll 1
        for (unsigned long long left = mask; left; left &= left - 1ull) {
            const int bit = __ffsll((long long)left) - 1;
            const int j = base + (lane + 32 * (bit >> 3)) * PV + (bit & 7);
            if (j < 0 || j >= V) mask &= ~(1ull << bit);
        }
    }
    const int n = __popcll(mask);
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    auto element = [&](int bit, float* y, int* j) {
        const int t = bit >> 3, e = bit & 7;
        const int off = (lane + 32 * t) * 16 + e * ELT;
        if constexpr (ELT == 4) *y = *reinterpret_cast<const float*>(chunk + off);
        else *y = __uint_as_float((uint32_t)*reinterpret_cast<const unsigned short*>(chunk + off) << 16);
        *y += 0.0f;                                            // -0.0 counts as +0.0
        *j = base + (lane + 32 * t) * PV + e;
    };
    if (total <= KS) {                                         // warp-uniform, nearly always
        int slot = incl - n;
#pragma unroll 1
        for (; mask; mask &= mask - 1ull) {
            float y;
            int j;
            element(__ffsll((long long)mask) - 1, &y, &j);
            out[slot++] = make_float2(y, __int_as_float(j));
        }
        if (lane >= total && lane < KS) out[lane] = make_float2(kNegInf, __int_as_float(0x7fffffff));
        return;
    }
    TopList<KC> L;
    L.init();
#pragma unroll 1
    for (; mask; mask &= mask - 1ull) {
        float y;
        int j;
        element(__ffsll((long long)mask) - 1, &y, &j);
        L.insert(y, j);
    }
    float ov[KC];
    int oi[KC];
    warp_merge_topk<KC>(L, ov, oi);
    if (lane == 0)
#pragma unroll
        for (int r = 0; r < KC; ++r) out[r] = make_float2(ov[r], __int_as_float(oi[r]));
    if (lane >= KC && lane < KS) out[lane] = make_float2(kNegInf, __int_as_float(0x7fffffff));
    thr = fmaxf(thr, ov[KC - 1]);
}

template <int ELT, int KC>
__global__ void __launch_bounds__(kRingThreads, 2) logprob_stream_kernel(const LogprobArgs a) {
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        mbar_init_fence();
    }
    __syncthreads();
    unsigned c0, c1;
    cta_range((unsigned)a.chunks, blockIdx.x, gridDim.x, &c0, &c1);
    pdl_trigger();
    pdl_wait();
    const long long tensor_bytes = (long long)a.rows * a.V * ELT;
    // bytes of chunk (r, seg): those that the span still has, and the whole
    // vectors of them that lie inside the tensor
    auto extent = [&](int r, int seg, long long* begin, int* lead, int* span, int* copied) {
        long long bytes;
        row_span(a, ELT, r, begin, lead, &bytes);
        const long long off = (long long)seg * kStageBytes;
        *span = (int)max(0LL, min((long long)kStageBytes, bytes - off));
        *begin += off;
        const long long whole = (tensor_bytes & ~15LL) - *begin;       // whole vectors left in the tensor
        *copied = (int)max(0LL, min((long long)((*span + 15) & ~15), whole));
    };

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t policy = l2_evict_first_policy();
            bool ok = true;
            unsigned c = c0;
            for (; c < c1; ++c) {
                const unsigned it = c - c0;
                const int st = (int)(it % kStages);
                if (it >= kStages && !wait_bounded(&empty[st], (it / kStages - 1) & 1u, a.wait_limit)) { ok = false; break; }
                long long begin;
                int lead, span, copied;
                extent((int)(c / (unsigned)a.nseg), (int)(c % (unsigned)a.nseg), &begin, &lead, &span, &copied);
                mbar_arrive_expect_tx(&full[st], (uint32_t)copied);
                if (copied > 0) bulk_g2s(ring + (size_t)st * kStageBytes, a.z + begin, (uint32_t)copied, &full[st], policy);
            }
            if (!ok) atomicOr(a.err, SPEC_DEVERR_TIMEOUT);
            // not before the copies in flight have landed
            const unsigned issued = c - c0;
            for (unsigned i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
                if (!wait_bounded(&full[i % kStages], (i / kStages) & 1u)) {
                    atomicOr(a.err, SPEC_DEVERR_TIMEOUT);
                    break;
                }
        }
        return;
    }
    const int cw = warp - 1;
    unsigned tk_row = 0xffffffffu;
    float tk_thr = kNegInf;
    bool ok = true;
    for (unsigned c = c0; c < c1; ++c) {
        const unsigned it = c - c0;
        const int st = (int)(it % kStages);
        if (!wait_bounded(&full[st], (it / kStages) & 1u, a.wait_limit)) ok = false;
        if (!__all_sync(0xffffffffu, ok)) break;
        const unsigned r = c / (unsigned)a.nseg;
        const int seg = (int)(c - r * (unsigned)a.nseg);
        long long begin;
        int lead, span, copied;
        extent((int)r, seg, &begin, &lead, &span, &copied);
        const int wb = span - cw * (32 * kLaneBytes);          // the warp chunk's bytes
        const size_t pi = ((size_t)r * a.nseg + seg) * kWarps + cw;
        float m = kNegInf, Z = 0.f, W = 0.f;
        if (wb > 0) {
            unsigned char* chunk = ring + (size_t)st * kStageBytes + cw * (32 * kLaneBytes);
            const int base = (seg * kStageBytes + cw * (32 * kLaneBytes)) / ELT - lead;
            if (base < 0 || base + 32 * kLaneBytes / ELT > a.V) {
                // the tensor's last, partial vector; then the neighbours' elements
                const int have = copied - cw * (32 * kLaneBytes);
                const int e0 = max(0, have) / ELT, e1 = min(wb, 32 * kLaneBytes) / ELT;
                for (int e = e0 + lane; e < e1; e += 32) {
                    if constexpr (ELT == 4) reinterpret_cast<float*>(chunk)[e] = load_logit<4>(a.z + begin + cw * (32 * kLaneBytes), e);
                    else reinterpret_cast<unsigned short*>(chunk)[e] =
                            __ldg(reinterpret_cast<const unsigned short*>(a.z + begin + cw * (32 * kLaneBytes)) + e);
                }
                constexpr int PV = 16 / ELT;
                if (lane < PV) {
                    const int f = lane;                        // before the row
                    const int g = a.V - base + lane;           // after it
                    if constexpr (ELT == 4) {
                        if (base + f < 0) reinterpret_cast<float*>(chunk)[f] = kNegInf;
                        if (g < ((wb + 15) & ~15) / ELT && g < 32 * kLaneBytes / ELT) reinterpret_cast<float*>(chunk)[g] = kNegInf;
                    } else {
                        if (base + f < 0) reinterpret_cast<unsigned short*>(chunk)[f] = 0xff80;
                        if (g < ((wb + 15) & ~15) / ELT && g < 32 * kLaneBytes / ELT) reinterpret_cast<unsigned short*>(chunk)[g] = 0xff80;
                    }
                }
                // the next copy into this stage follows these writes
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            uint4 v[kVecPerLane];
            lane_words<ELT>(chunk, wb, v);
            m = warp_max(lane_max<ELT>(v));
            if (m != kNegInf) chunk_sums<ELT>(v, m, a.s, &Z, &W);
            if constexpr (KC > 0) {
                chunk_candidates<ELT, KC>(v, chunk, base, a.V, a.cand + pi * topk_slots(KC), tk_thr, tk_row == r);
                tk_row = r;
            }
        } else if constexpr (KC > 0) {
            if (lane < topk_slots(KC)) a.cand[pi * topk_slots(KC) + lane] = make_float2(kNegInf, __int_as_float(0x7fffffff));
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&empty[st]);
            a.stats[pi] = make_float4(m, Z, W, 0.f);
        }
    }
    if (!ok && lane == 0) atomicOr(a.err, SPEC_DEVERR_TIMEOUT);
}

// One CTA per row.
template <int ELT, int KC>
__global__ void __launch_bounds__(kMergeThreads) logprob_merge_kernel(const LogprobArgs a) {
    constexpr int NW = kMergeThreads / 32;
    __shared__ float red[3][NW];
    __shared__ float2 pool[kMergePool];
    __shared__ int pool_n;
    __shared__ float best_v[NW];
    __shared__ int best_i[NW];
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.x;
    if (threadIdx.x == 0) pool_n = 0;
    pdl_wait();
    const int P = a.nseg * kWarps;
    const int tok = __ldg(a.tok + r);
    const bool tok_ok = (unsigned)tok < (unsigned)a.V;
    float zx = kNegInf;
    if (threadIdx.x == 0 && tok_ok) zx = load_logit<ELT>(a.z + (size_t)r * a.V * ELT, tok);

    const float4* st = a.stats + (size_t)r * P;
    float M = kNegInf;
    for (int i = threadIdx.x; i < P; i += kMergeThreads) M = fmaxf(M, __ldcg(st + i).x);
    M = warp_max(M);
    if (lane == 0) red[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, red[0][w]);
    const bool empty = M == kNegInf;
    float Z = 0.f, W = 0.f;
    for (int i = threadIdx.x; i < P; i += kMergeThreads) {
        const float4 q = __ldcg(st + i);
        if (q.x == kNegInf) continue;
        const float d = fmaxf((q.x - M) * a.s, kArgFloor);
        const float f = ex2_approx(d);
        Z = fmaf(f, q.y, Z);
        W = fmaf(f, fmaf(d, q.y, q.z), W);
    }
    Z = warp_sum(Z);
    W = warp_sum(W);
    if (lane == 0) { red[1][warp] = Z; red[2][warp] = W; }
    __syncthreads();
    Z = W = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) { Z += red[1][w]; W += red[2][w]; }
    const float lnz = logf(Z);
    if (threadIdx.x == 0) {
        a.lp[r] = empty || !tok_ok ? CUDART_NAN_F : (zx - M) / a.T - lnz;
        if (a.ent) a.ent[r] = empty ? CUDART_NAN_F : fmaxf(0.f, lnz - kLn2f * (W / Z));
        if (empty) atomicOr(a.err, SPEC_DEVERR_EMPTY_ROW);
        if (!tok_ok) atomicOr(a.err, SPEC_DEVERR_TOKEN_RANGE);
    }
    if constexpr (KC > 0) {
        // A lower bound of the KC-th largest: the KC-th largest thread maximum
        // of any one warp.
        const int n = P * topk_slots(KC);
        const float2* ca = a.cand + (size_t)r * n;
        float x = kNegInf;
        for (int i = threadIdx.x; i < n; i += kMergeThreads) x = fmaxf(x, __ldcg(ca + i).x);
        int k = ord_key(x), t = kNoKey;
#pragma unroll
        for (int q = 0; q < KC; ++q) {
            t = __reduce_max_sync(0xffffffffu, k);
            const unsigned own = __ballot_sync(0xffffffffu, k == t);
            if (lane == __ffs(own) - 1) k = kNoKey;
        }
        if (lane == 0) best_v[warp] = key_value(t);
        __syncthreads();
        float thr = best_v[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) thr = fmaxf(thr, best_v[w]);
        for (int i = threadIdx.x; i < n; i += kMergeThreads) {
            const float2 e = __ldcg(ca + i);
            if (e.x >= thr && __float_as_int(e.y) != 0x7fffffff) {
                const int at = atomicAdd(&pool_n, 1);
                if (at < kMergePool) pool[at] = e;
            }
        }
        __syncthreads();
        const int total = pool_n;
        auto put = [&](int q, float v, int j) {
            const bool none = j == 0x7fffffff || empty;
            a.ti[(size_t)r * a.K + q] = none ? -1 : j;
            a.tl[(size_t)r * a.K + q] = empty ? CUDART_NAN_F : none ? kNegInf : (v - M) / a.T - lnz;
        };
        if (total <= kMergePool) {
            if (warp == 0) {
                const float2 e = lane < total ? pool[lane] : make_float2(kNegInf, 0.f);
                int ck = lane < total ? ord_key(e.x) : kNoKey;
                const unsigned ci = lane < total ? (unsigned)__float_as_int(e.y) : 0x7fffffffu;
#pragma unroll
                for (int q = 0; q < KC; ++q) {
                    const int kk = __reduce_max_sync(0xffffffffu, ck);
                    const unsigned j = kk == kNoKey ? 0x7fffffffu : __reduce_min_sync(0xffffffffu, ck == kk ? ci : 0x7fffffffu);
                    if (lane == 0 && q < a.K) put(q, key_value(kk), (int)j);
                    if (ck == kk && ci == j) ck = kNoKey;
                }
            }
            return;
        }
        // many equal logits: K rounds over all candidates, each taking the best
        // one after the last
        float lv = 0.f;
        int li = -1;
        for (int q = 0; q < a.K; ++q) {
            float bv = kNegInf;
            int bi = 0x7fffffff;
            for (int i = threadIdx.x; i < n; i += kMergeThreads) {
                const float2 e = __ldcg(ca + i);
                const int j = __float_as_int(e.y);
                if (j != 0x7fffffff && (li < 0 || am_better(lv, li, e.x, j)) && am_better(e.x, j, bv, bi)) { bv = e.x; bi = j; }
            }
            warp_argmax(bv, bi);
            __syncthreads();
            if (lane == 0) { best_v[warp] = bv; best_i[warp] = bi; }
            __syncthreads();
#pragma unroll
            for (int w = 0; w < NW; ++w)
                if (am_better(best_v[w], best_i[w], bv, bi)) { bv = best_v[w]; bi = best_i[w]; }
            if (threadIdx.x == 0) put(q, bv, bi);
            lv = bv;
            li = bi;
            if (bi == 0x7fffffff) li = 0x7ffffffe;             // none left
        }
    }
}

static int list_len(int K) { return K <= 0 ? 0 : topk_list_len(K); }

static int logprob_nseg(int V, int elt) {
    return (int)(((long long)V * elt + (16 - elt) + kStageBytes - 1) / kStageBytes);
}

size_t logprobs_workspace_size(int rows, int V, int K) {
    // error word, then for every warp chunk (fp32 has the most) its sums and candidates
    const size_t chunks = (size_t)rows * (size_t)logprob_nseg(V, 4) * kWarps;
    return 256 + align256(chunks * sizeof(float4)) + align256(chunks * topk_slots(list_len(K)) * sizeof(float2));
}

template <int ELT, int KC>
static cudaError_t launch_logprobs_t(const LogprobArgs& a, const DeviceInfo& di, cudaStream_t st) {
    auto kfn = logprob_stream_kernel<ELT, KC>;
    const int smem = kStages * kStageBytes;
    static DeviceSlots slots = {};
    int occ = 0;
    cudaError_t e = device_once(slots, &occ, [&](int, int* o) {
        cudaError_t r = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (r != cudaSuccess) return r;
        r = cudaFuncSetAttribute(kfn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (r != cudaSuccess) return r;
        r = cudaFuncSetAttribute(logprob_merge_kernel<ELT, KC>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared);
        if (r != cudaSuccess) return r;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(o, kfn, kRingThreads, smem);
    });
    if (e != cudaSuccess) return e;
    long long g = (long long)di.sm_count * occ;
    if (a.chunks < g) g = a.chunks;
    e = launch_pdl(kfn, dim3((unsigned)g), kRingThreads, smem, st, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(logprob_merge_kernel<ELT, KC>, dim3((unsigned)a.rows), kMergeThreads, 0, st, a);
}

template <int ELT>
static cudaError_t launch_logprobs_e(const LogprobArgs& a, const DeviceInfo& di, cudaStream_t st) {
    switch (list_len(a.K)) {
        case 0: return launch_logprobs_t<ELT, 0>(a, di, st);
        case 2: return launch_logprobs_t<ELT, 2>(a, di, st);
        case 4: return launch_logprobs_t<ELT, 4>(a, di, st);
        default: return launch_logprobs_t<ELT, 8>(a, di, st);
    }
}

cudaError_t launch_logprobs(const void* z, spec_dtype_t dt, const int32_t* tok, float T, int rows, int V, int K,
                            float* lp, float* ent, int32_t* ti, float* tl, void* ws, cudaStream_t st) {
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    const int elt = elt_size(dt);
    char* w = static_cast<char*>(ws);
    LogprobArgs a = {};
    a.z = static_cast<const char*>(z);
    a.tok = tok;
    a.T = T;
    a.s = (float)(1.4426950408889634 / (double)T);
    a.rows = rows;
    a.V = V;
    a.K = K;
    a.nseg = logprob_nseg(V, elt);
    a.chunks = (long long)rows * a.nseg;
    a.err = reinterpret_cast<int*>(w);
    a.stats = reinterpret_cast<float4*>(w + 256);
    a.cand = reinterpret_cast<float2*>(w + 256 + align256((size_t)a.chunks * kWarps * sizeof(float4)));
    a.lp = lp;
    a.ent = ent;
    a.ti = ti;
    a.tl = tl;
    a.wait_limit = ring_wait_limit();
    return elt == 2 ? launch_logprobs_e<2>(a, di, st) : launch_logprobs_e<4>(a, di, st);
}

}  // namespace sv
