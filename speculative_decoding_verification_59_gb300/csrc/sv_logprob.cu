// Log-probabilities of given tokens, with the entropy of their rows'
// distributions and the top alternatives, in one pass over the logits.
//
// With p = softmax(z / T), s = log2(e) / T, M = max z, a_j = (z_j - M) s:
//   Z = sum 2^a_j,  W = sum a_j 2^a_j,
//   ln p(x) = (z_x - M) / T - ln Z,   H = -sum p ln p = ln Z - ln 2 W / Z.
// Each 4 KB warp chunk of a row leaves its own maximum m with Z and W taken
// relative to it; one CTA per row then brings the chunks to the common maximum.
// The K alternatives cost the stream nothing: the K-th largest chunk maximum is
// a lower bound of the row's K-th largest logit, so that CTA reads again only the
// chunks whose maximum reaches it -- K of them, unless maxima are equal -- and
// orders their logits that do.  (Collecting candidates while streaming took 61 us
// for 512 rows of 151936 bf16 logits and K = 5, against 35 without lists.)
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
constexpr int kMaxAlternatives = 8;
constexpr float kArgFloor = -256.f;           // 2^-256 is zero in fp32, and -256 times it too
constexpr float kLn2f = 0.6931471805599453f;

struct LogprobArgs {
    const char* z;
    const int32_t* tok;
    float T, s, inv_s;
    int rows, V, K, nseg;
    long long chunks;
    float4* stats;             // per warp chunk: m, Z, W (relative to m)
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
// The arguments are one FMA each, z s - fl(m s): off by the rounding r = m s -
// fl(m s), which the sums take back at the end (2^(a + r): Z = 2^-r Z', W =
// 2^-r W' - r Z).  Masked logits (-inf) would give 0 x inf in W: logits are
// first raised to one whose power is zero, bf16 ones two an instruction.  Where
// no such logit is near (tiny temperatures, where one step of a bf16 logit
// already counts; chunks of the type's lowest value; temperatures past 1e36, 256
// powers of two below the maximum being past fp32's range) the arguments (z - m) s
// are clamped instead.
template <int ELT>
__device__ __forceinline__ void chunk_sums(const uint4 (&v)[kVecPerLane], float m, float s, float inv_s, float* Z, float* W) {
    f32x2 z2 = f2_pack(0.f, 0.f), w2 = z2;
    float r = 0.f;
    const float below = kArgFloor * inv_s;                     // 256 powers of two below the maximum
    if (!(m + below > -3.3e38f) || !(below <= -fabsf(m) * 0.015625f)) {   // warp-uniform
#pragma unroll
        for (int t = 0; t < kVecPerLane; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t w = u4_get(v[t], c);
                const float p = fmaxf(((ELT == 2 ? bf16_lo(w) : __uint_as_float(w)) - m) * s, kArgFloor);
                const float q = ELT == 2 ? fmaxf((bf16_hi(w) - m) * s, kArgFloor) : kArgFloor;
                const f32x2 e = f2_pack(ex2_approx(p), ex2_approx(q));
                z2 = f2_add(z2, e);
                w2 = f2_fma(e, f2_pack(p, q), w2);
            }
    } else {
        const float ms = m * s;
        r = fmaf(m, s, -ms);
        const f32x2 s2 = f2_pack(s, s), off = f2_pack(-ms, -ms);
        const float low = m + below;                           // finite, and its bf16 rounding too
        uint32_t low2;
        asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(low2) : "f"(low));
#pragma unroll
        for (int t = 0; t < kVecPerLane; ++t)
#pragma unroll
            for (int c = 0; c < 4; c += (ELT == 2 ? 1 : 2)) {
                f32x2 x;
                if constexpr (ELT == 2) {
                    uint32_t w = u4_get(v[t], c);
                    asm("max.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(low2));
                    x = f2_pack(bf16_lo(w), bf16_hi(w));
                } else {
                    x = f2_pack(fmaxf(__uint_as_float(u4_get(v[t], c)), low), fmaxf(__uint_as_float(u4_get(v[t], c + 1)), low));
                }
                const f32x2 arg = f2_fma(x, s2, off);
                float p, q;
                f2_unpack(arg, p, q);
                const f32x2 e = f2_pack(ex2_approx(p), ex2_approx(q));
                z2 = f2_add(z2, e);
                w2 = f2_fma(e, arg, w2);
            }
    }
    float z0, z1, w0, w1;
    f2_unpack(z2, z0, z1);
    f2_unpack(w2, w0, w1);
    const float f = r == 0.f ? 1.f : exp2f(-r);
    const float zs = warp_sum(z0 + z1) * f;
    *Z = zs;
    *W = warp_sum(w0 + w1) * f - r * zs;
}

template <int ELT>
__global__ void __launch_bounds__(kRingThreads, 2) logprob_stream_kernel(const LogprobArgs a) {
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages];
    __shared__ int4 stage_info[kStages];                       // row, segment, lead, span a stage holds
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned c0, c1;
    cta_range((unsigned)a.chunks, blockIdx.x, gridDim.x, &c0, &c1);
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
    if (threadIdx.x == 0) {
        // the first chunks into L2 while the kernel before ends (as in sv_stream.cuh)
        if (a.chunks >= kPrefetchMinChunks)
            for (unsigned c = c0; c < c1 && c < c0 + kPrefetchChunks; ++c) {
                long long begin;
                int lead, span, copied;
                extent((int)(c / (unsigned)a.nseg), (int)(c % (unsigned)a.nseg), &begin, &lead, &span, &copied);
                if (copied > 0) bulk_prefetch_l2(a.z + begin, (uint32_t)copied);
            }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        mbar_init_fence();
    }
    __syncthreads();
    pdl_trigger();
    pdl_wait();

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
                const int r = (int)(c / (unsigned)a.nseg), seg = (int)(c - (unsigned)r * (unsigned)a.nseg);
                extent(r, seg, &begin, &lead, &span, &copied);
                stage_info[st] = make_int4(r, seg, lead, span);
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
    bool ok = true;
    unsigned c = c0;
    for (; c < c1; ++c) {
        const unsigned it = c - c0;
        const int st = (int)(it % kStages);
        if (!wait_bounded(&full[st], (it / kStages) & 1u, a.wait_limit)) ok = false;
        if (!__all_sync(0xffffffffu, ok)) break;
        const int4 info = stage_info[st];
        const int r = info.x, seg = info.y, lead = info.z, span = info.w;
        const int wb = span - cw * (32 * kLaneBytes);          // the warp chunk's bytes
        const size_t pi = ((size_t)r * a.nseg + seg) * kWarps + cw;
        float m = kNegInf, Z = 0.f, W = 0.f;
        if (wb > 0) {
            unsigned char* chunk = ring + (size_t)st * kStageBytes + cw * (32 * kLaneBytes);
            const int base = (seg * kStageBytes + cw * (32 * kLaneBytes)) / ELT - lead;
            if (base < 0 || base + 32 * kLaneBytes / ELT > a.V) {
                // the tensor's last, partial vector; then the neighbours' elements
                long long begin;
                int l_, s_, copied;
                extent(r, seg, &begin, &l_, &s_, &copied);
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
            if (m != kNegInf) chunk_sums<ELT>(v, m, a.s, a.inv_s, &Z, &W);
        }
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&empty[st]);
            a.stats[pi] = make_float4(m, Z, W, 0.f);
        }
    }
    if (c == c1) return;
    // a wait ran out: the sums of the chunks not seen are no numbers, and so are their rows' results
    for (c += lane; c < c1; c += 32) a.stats[(size_t)c * kWarps + cw] = make_float4(0.f, CUDART_NAN_F, CUDART_NAN_F, 0.f);
    if (lane == 0) atomicOr(a.err, SPEC_DEVERR_TIMEOUT);
}

// The first K of warp_merge_topk (sv_stream.cuh); the other entries say none.
template <int KC>
__device__ __forceinline__ void merge_lists(TopList<KC>& L, int K, float (&ov)[KC], int (&oi)[KC]) {
#pragma unroll
    for (int r = 0; r < KC; ++r) {
        float hv = kNegInf;
        int hi = 0x7fffffff;
        if (r < K) {                                           // uniform
            hv = L.v[0];
            hi = L.i[0];
            warp_argmax(hv, hi);
            if (L.i[0] == hi && hi != 0x7fffffff) {
#pragma unroll
                for (int k = 0; k < KC - 1; ++k) { L.v[k] = L.v[k + 1]; L.i[k] = L.i[k + 1]; }
                L.v[KC - 1] = kNegInf;
                L.i[KC - 1] = 0x7fffffff;
            }
        }
        ov[r] = hv;
        oi[r] = hi;
    }
}

// Element e of a vector as a float.
template <int ELT>
__device__ __forceinline__ float vec_value(const uint4& q, int e) {
    if constexpr (ELT == 4) return __uint_as_float(u4_get(q, e));
    else return (e & 1) ? bf16_hi(u4_get(q, e >> 1)) : bf16_lo(u4_get(q, e >> 1));
}

// A warp's chunk of row r straight from memory, at byte `at` of the row's
// span: what is not the row's reads as -inf.  row: the lane's elements of the row,
// as bits 8 t + e.  Returns the row index of the chunk's first element.
template <int ELT>
__device__ __forceinline__ int load_chunk(const LogprobArgs& a, int r, long long at, uint4 (&v)[kVecPerLane],
                                          unsigned long long& row) {
    constexpr int PV = 16 / ELT;
    const int lane = threadIdx.x & 31;
    long long begin, bytes;
    int lead;
    row_span(a, ELT, r, &begin, &lead, &bytes);
    const long long tensor_bytes = (long long)a.rows * a.V * ELT;
    const int base = (int)(at / ELT) - lead;
    const uint32_t ninf = ELT == 4 ? 0xff800000u : 0xff80ff80u;
#pragma unroll
    for (int t = 0; t < kVecPerLane; ++t) {
        const long long o = begin + at + (lane + 32 * t) * 16;
        v[t] = o + 16 <= tensor_bytes && o < begin + bytes ? ld_stream16(a.z + o) : make_uint4(ninf, ninf, ninf, ninf);
    }
    row = ~0ull;
    if (ELT == 4) row = 0x0f0f0f0f0f0f0f0full;
    if (base < 0 || base + 32 * kLaneBytes / ELT > a.V) {      // warp-uniform: the row's first or last chunk
        row = 0ull;
#pragma unroll
        for (int t = 0; t < kVecPerLane; ++t) {
            const int j = base + (lane + 32 * t) * PV;         // the vector's elements are j .. j + PV - 1
            if (j >= a.V || j <= -PV) {
                v[t] = make_uint4(ninf, ninf, ninf, ninf);
                continue;
            }
            unsigned bits = (1u << PV) - 1u;
            if (j < 0) bits &= bits << -j;
            if (j + PV > a.V) bits &= (1u << (a.V - j)) - 1u;
            row |= (unsigned long long)bits << (8 * t);
            const bool whole = begin + at + (lane + 32 * t) * 16 + 16 <= tensor_bytes;
            if (bits == (1u << PV) - 1u && whole) continue;    // (most lanes' by far)
            uint32_t w[4] = {v[t].x, v[t].y, v[t].z, v[t].w};
#pragma unroll
            for (int e = 0; e < PV; ++e) {
                // (a vector that the tensor ends in is read by element)
                uint32_t x = ELT == 4 ? 0xff800000u : 0xff80u;
                if ((bits >> e) & 1u) {
                    if (whole) {
                        x = ELT == 4 ? w[e] : (w[e >> 1] >> (16 * (e & 1))) & 0xffffu;
                    } else {
                        const float f = load_logit<ELT>(a.z + (size_t)r * a.V * ELT, j + e);
                        x = ELT == 4 ? __float_as_uint(f) : __float_as_uint(f) >> 16;
                    }
                }
                if constexpr (ELT == 4) w[e] = x;
                else w[e >> 1] = (w[e >> 1] & (0xffff0000u >> (16 * (e & 1)))) | x << (16 * (e & 1));
            }
            v[t] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    return base;
}

// The lane's logits of a chunk that reach a bound, as bits 8 t + e.
template <int ELT>
__device__ __forceinline__ unsigned long long reach(const uint4 (&v)[kVecPerLane], unsigned long long row, float bound) {
    unsigned long long mask = 0ull;
#pragma unroll
    for (int t = 0; t < kVecPerLane; ++t) {
        if (vec_max_value<ELT>(vec_max_bits<ELT>(v[t])) >= bound) {
#pragma unroll
            for (int e = 0; e < 16 / ELT; ++e)
                if (vec_value<ELT>(v[t], e) >= bound) mask |= 1ull << (8 * t + e);
        }
    }
    return mask & row;
}

// Calls take(value, row index) for the lane's marked logits.  room: 4 KB of
// shared memory of the warp's own, where each lane reads back what it wrote.
template <int ELT, typename F>
__device__ __forceinline__ void each_marked(const uint4 (&v)[kVecPerLane], unsigned long long mask, int base, unsigned char* room, F take) {
    constexpr int PV = 16 / ELT;
    const int lane = threadIdx.x & 31;
    if (mask == 0ull) return;
#pragma unroll
    for (int t = 0; t < kVecPerLane; ++t) *reinterpret_cast<uint4*>(room + (lane + 32 * t) * 16) = v[t];
#pragma unroll 1
    for (; mask; mask &= mask - 1ull) {
        const int bit = __ffsll((long long)mask) - 1;
        const unsigned char* p = room + (lane + 32 * (bit >> 3)) * 16 + (bit & 7) * ELT;
        float x;
        if constexpr (ELT == 4) x = *reinterpret_cast<const float*>(p);
        else x = __uint_as_float((uint32_t)*reinterpret_cast<const unsigned short*>(p) << 16);
        take(x + 0.0f, base + (lane + 32 * (bit >> 3)) * PV + (bit & 7));      // -0.0 counts as +0.0
    }
}

// The logits of a row that reach a lower bound of its K-th largest: K of them
// and a few more as a rule, so that a lane each holds them all.
constexpr int kPool = 32;
struct Pool {
    float v[kPool];
    int i[kPool];
    int n;
};
template <int ELT>
__device__ __forceinline__ void pool_chunk(const uint4 (&v)[kVecPerLane], unsigned long long row, int base, float thr,
                                           unsigned char* room, Pool& p) {
    each_marked<ELT>(v, reach<ELT>(v, row, thr), base, room, [&](float x, int j) {
        const int at = atomicAdd(&p.n, 1);
        if (at < kPool) {
            p.v[at] = x;
            p.i[at] = j;
        }
    });
}
// The pool's first K in order (a warp; n <= kPool entries).
__device__ __forceinline__ void pool_lists(const Pool& p, int n, int K, float (&ov)[kMaxAlternatives], int (&oi)[kMaxAlternatives]) {
    const int lane = threadIdx.x & 31;
    int ck = lane < n ? ord_key(p.v[lane]) : kNoKey;
    const unsigned ci = lane < n ? (unsigned)p.i[lane] : 0x7fffffffu;
#pragma unroll
    for (int q = 0; q < kMaxAlternatives; ++q) {
        ov[q] = kNegInf;
        oi[q] = 0x7fffffff;
        if (q < K) {                                           // uniform
            const int t = __reduce_max_sync(0xffffffffu, ck);
            const unsigned j = __reduce_min_sync(0xffffffffu, ck == t ? ci : 0x7fffffffu);
            if (t != kNoKey) {
                ov[q] = key_value(t);
                oi[q] = (int)j;
            }
            if (ck == t && ci == j) ck = kNoKey;
        }
    }
}

// Where more reach it than a pool holds (many equal logits, one chunk above
// all others): adds the chunk's logits that can be among the K largest to the
// lane's list.  thr is raised when many reach it (the K-th largest of the lanes'
// maxima is a bound too).
template <int ELT>
__device__ __forceinline__ void pick_chunk(const uint4 (&v)[kVecPerLane], unsigned long long row, int base, int K, float& thr,
                                           unsigned char* room, TopList<kMaxAlternatives>& L) {
    const int lane = threadIdx.x & 31;
    unsigned long long mask = reach<ELT>(v, row, thr);
    if (__reduce_add_sync(0xffffffffu, (unsigned)__popcll(mask)) > 24u) {
        int k = mask ? ord_key(lane_max<ELT>(v)) : kNoKey, t = kNoKey;
#pragma unroll
        for (int q = 0; q < kMaxAlternatives; ++q) {
            if (q >= K) break;
            t = __reduce_max_sync(0xffffffffu, k);
            const unsigned own = __ballot_sync(0xffffffffu, k == t);
            if (lane == __ffs(own) - 1) k = kNoKey;
        }
        if (t != kNoKey) thr = fmaxf(thr, key_value(t));
        mask = reach<ELT>(v, row, thr);
    }
    each_marked<ELT>(v, mask, base, room, [&](float x, int j) { L.insert(x, j); });
}

// The row's results, by its CTA's first thread.
__device__ __forceinline__ void put_row(const LogprobArgs& a, int r, bool empty, bool tok_ok, float zx, float M, float lnz,
                                        float inner) {
    a.lp[r] = empty || !tok_ok ? CUDART_NAN_F : (zx - M) / a.T - lnz;
    const float ent = lnz - kLn2f * inner;
    if (a.ent) a.ent[r] = empty ? CUDART_NAN_F : ent < 0.f ? 0.f : ent;       // (a row without sums: NaN)
    if (empty) atomicOr(a.err, SPEC_DEVERR_EMPTY_ROW);
    if (!tok_ok) atomicOr(a.err, SPEC_DEVERR_TOKEN_RANGE);
}
__device__ __forceinline__ void put_list(const LogprobArgs& a, int r, bool empty, float M, float lnz,
                                         const float (&ov)[kMaxAlternatives], const int (&oi)[kMaxAlternatives]) {
#pragma unroll
    for (int q = 0; q < kMaxAlternatives; ++q)
        if (q < a.K) {
            const bool none = oi[q] == 0x7fffffff || empty;
            a.ti[(size_t)r * a.K + q] = none ? -1 : oi[q];
            a.tl[(size_t)r * a.K + q] = empty ? CUDART_NAN_F : none ? kNegInf : (ov[q] - M) / a.T - lnz;
        }
}

// Short rows (up to kRowChunks warp chunks): one CTA does all of a row, its
// chunks straight from memory, in one launch.  Through the ring a 32 KB stage
// carries one short row, and the lists of many rows cost a second kernel more than
// here.  bf16, us here / through the ring: 33.5 / 538 for 14714 rows of 1400 with 5
// alternatives, 29.7 / 36.3 for 2048 of 16000, 45.4 / 45.4 of 32000; without lists
// 17.8 / 57.1 and 17.1 / 19.4 for 4000 of 8000, 2.9 / 4.1 for 64 of 16000, but
// 17.7 / 13.9 for 2048 of 16000 (a CTA a row does not keep the memory busy): there the
// ring takes the rows of more than kFewChunks.  With lists three CTAs an SM (80
// registers) are worth the spills: 29.7 for 56.3.
constexpr int kRowChunks = 16, kFewChunks = 4;
constexpr int kRowWarps = 8;
template <int ELT, bool LISTS>
__global__ void __launch_bounds__(kRowWarps * 32, LISTS ? 3 : 1) logprob_row_kernel(const LogprobArgs a, int chunks) {
    constexpr int KC = kMaxAlternatives;
    __shared__ float part[kRowWarps][3], lmax[kRowChunks][32]; // the lanes' maxima of every chunk
    __shared__ Pool pool;
    __shared__ float list_v[kRowWarps][KC];
    __shared__ int list_i[kRowWarps][KC];
    extern __shared__ __align__(16) unsigned char rooms[];
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5, r = blockIdx.x;
    if (threadIdx.x == 0) pool.n = 0;
    pdl_wait();
    const int tok = __ldg(a.tok + r);
    const bool tok_ok = (unsigned)tok < (unsigned)a.V;
    float zx = kNegInf;
    if (threadIdx.x == 0 && tok_ok) zx = load_logit<ELT>(a.z + (size_t)r * a.V * ELT, tok);
    uint4 v[kVecPerLane];
    unsigned long long row = 0ull;
    int base = 0;
    float M = kNegInf, Z = 0.f, W = 0.f;                       // the warp's
    for (int c = warp; c < chunks; c += nw) {
        base = load_chunk<ELT>(a, r, (long long)c * (32 * kLaneBytes), v, row);
        const float lm = lane_max<ELT>(v), m = warp_max(lm);
        if constexpr (LISTS) lmax[c][lane] = lm;
        if (m == kNegInf) continue;                            // warp-uniform
        float z, w;
        chunk_sums<ELT>(v, m, a.s, a.inv_s, &z, &w);
        // both at the larger maximum
        const float top = fmaxf(M, m);
        const float d0 = M == kNegInf ? kArgFloor : fmaxf((M - top) * a.s, kArgFloor), d1 = fmaxf((m - top) * a.s, kArgFloor);
        const float f0 = ex2_approx(d0), f1 = ex2_approx(d1);
        W = f0 * fmaf(d0, Z, W) + f1 * fmaf(d1, z, w);
        Z = f0 * Z + f1 * z;
        M = top;
    }
    if (lane == 0) { part[warp][0] = M; part[warp][1] = Z; part[warp][2] = W; }
    __syncthreads();
    // every warp brings the warps' sums together: a lane each
    const float pm = lane < nw ? part[lane][0] : kNegInf;
    M = warp_max(pm);
    const bool empty = M == kNegInf;
    const float d = pm == kNegInf ? kArgFloor : fmaxf((pm - M) * a.s, kArgFloor), f = ex2_approx(d);
    Z = warp_sum(lane < nw ? f * part[lane][1] : 0.f);
    W = warp_sum(lane < nw ? f * fmaf(d, part[lane][1], part[lane][2]) : 0.f);
    const float lnz = logf(Z);
    if (threadIdx.x == 0) put_row(a, r, empty, tok_ok, zx, M, lnz, W / Z);
    if constexpr (LISTS) {
        // The K-th largest of the lanes' maxima over all chunks (distinct logits, near
        // the K-th largest of all) is the bound; every warp finds it.
        float x = kNegInf;
        for (int c = 0; c < chunks; ++c) x = fmaxf(x, lmax[c][lane]);
        int k = ord_key(x), t = kNoKey;
#pragma unroll
        for (int q = 0; q < KC; ++q) {
            if (q >= a.K) break;
            t = __reduce_max_sync(0xffffffffu, k);
            const unsigned own = __ballot_sync(0xffffffffu, k == t);
            if (lane == __ffs(own) - 1) k = kNoKey;
        }
        float thr = key_value(t);                              // -inf when so many lanes hold nothing finite
        const int last = warp + (chunks - 1 - warp) / nw * nw;   // the chunk that v still holds
        unsigned char* room = rooms + warp * (32 * kLaneBytes);
        for (int c = last; c >= 0 && !empty; c -= nw) {
            if (!__any_sync(0xffffffffu, lmax[c][lane] >= thr)) continue;
            if (c != last) base = load_chunk<ELT>(a, r, (long long)c * (32 * kLaneBytes), v, row);
            pool_chunk<ELT>(v, row, base, thr, room, pool);
        }
        __syncthreads();
        float ov[KC];
        int oi[KC];
        const int n = pool.n;
        if (n <= kPool) {                                      // uniform
            if (warp == 0) {
                pool_lists(pool, n, a.K, ov, oi);
                if (lane == 0) put_list(a, r, empty, M, lnz, ov, oi);
            }
            return;
        }
        TopList<KC> L;
        L.init();
        for (int c = warp; c < chunks; c += nw) {
            if (!__any_sync(0xffffffffu, lmax[c][lane] >= thr)) continue;
            base = load_chunk<ELT>(a, r, (long long)c * (32 * kLaneBytes), v, row);
            pick_chunk<ELT>(v, row, base, a.K, thr, room, L);
        }
        merge_lists<KC>(L, a.K, ov, oi);
        if (nw > 1) {                                          // uniform
            if (lane == 0) {
#pragma unroll
                for (int q = 0; q < KC; ++q) { list_v[warp][q] = ov[q]; list_i[warp][q] = oi[q]; }
            }
            __syncthreads();
            if (warp > 0) return;
            L.init();
            for (int i = lane; i < nw * KC; i += 32) L.insert(list_v[i / KC][i & (KC - 1)], list_i[i / KC][i & (KC - 1)]);
            merge_lists<KC>(L, a.K, ov, oi);
        }
        if (lane == 0) put_list(a, r, empty, M, lnz, ov, oi);
    }
}

// Long rows: one CTA per row, after the stream.
template <int ELT, bool LISTS>
__global__ void __launch_bounds__(kMergeThreads) logprob_merge_kernel(const LogprobArgs a) {
    constexpr int NW = kMergeThreads / 32, KC = kMaxAlternatives;
    __shared__ float red[3][NW];
    __shared__ int keys[NW][KC];
    __shared__ float list_v[NW][KC];
    __shared__ int list_i[NW][KC];
    __shared__ int thr_key, n_sel;
    __shared__ Pool pool;
    __shared__ __align__(16) unsigned char chunks[LISTS ? NW : 1][32 * kLaneBytes];    // a warp's chunk
    extern __shared__ unsigned short sel[];                    // chunks that reach the bound
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.x;
    if (threadIdx.x == 0) n_sel = pool.n = 0;
    pdl_wait();
    const int P = a.nseg * kWarps;
    const int tok = __ldg(a.tok + r);
    const bool tok_ok = (unsigned)tok < (unsigned)a.V;
    float zx = kNegInf;
    if (threadIdx.x == 0 && tok_ok) zx = load_logit<ELT>(a.z + (size_t)r * a.V * ELT, tok);

    // ---- the chunks' sums at the row's maximum
    const float4* st = a.stats + (size_t)r * P;
    float4 first = make_float4(kNegInf, 0.f, 0.f, 0.f);        // the thread's first chunk stays at hand
    if ((int)threadIdx.x < P) first = __ldcg(st + threadIdx.x);
    float M = first.x;
    for (int i = threadIdx.x + kMergeThreads; i < P; i += kMergeThreads) M = fmaxf(M, __ldcg(st + i).x);
    const float mine = M;
    M = warp_max(M);
    if (lane == 0) red[0][warp] = M;
    if constexpr (LISTS) {
        // each warp's K largest thread maxima
        int k = ord_key(mine);
#pragma unroll
        for (int q = 0; q < KC; ++q) {
            if (q >= a.K) break;
            const int top = __reduce_max_sync(0xffffffffu, k);
            const unsigned own = __ballot_sync(0xffffffffu, k == top);
            if (lane == __ffs(own) - 1) k = kNoKey;
            if (lane == 0) keys[warp][q] = top;
        }
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, red[0][w]);
    const bool empty = M == kNegInf;
    float Z = 0.f, W = 0.f;
    for (int i = threadIdx.x; i < P; i += kMergeThreads) {
        const float4 q = i == (int)threadIdx.x ? first : __ldcg(st + i);
        if (q.x == kNegInf) continue;
        const float d = fmaxf((q.x - M) * a.s, kArgFloor);
        const float f = ex2_approx(d);
        Z = fmaf(f, q.y, Z);
        W = fmaf(f, fmaf(d, q.y, q.z), W);
    }
    Z = warp_sum(Z);
    W = warp_sum(W);
    if (lane == 0) { red[1][warp] = Z; red[2][warp] = W; }
    if constexpr (LISTS) {
        if (warp == 0) {
            // the K-th largest of the warps' lists, an entry a lane
            static_assert(NW * KC == 32, "an entry a lane");
            int k = (lane & (KC - 1)) < a.K ? keys[lane / KC][lane & (KC - 1)] : kNoKey, t = kNoKey;
#pragma unroll
            for (int q = 0; q < KC; ++q) {
                if (q >= a.K) break;
                t = __reduce_max_sync(0xffffffffu, k);
                const unsigned own = __ballot_sync(0xffffffffu, k == t);
                if (lane == __ffs(own) - 1) k = kNoKey;
            }
            if (lane == 0) thr_key = t;
        }
    }
    __syncthreads();
    Z = W = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) { Z += red[1][w]; W += red[2][w]; }
    const float lnz = logf(Z);
    if (threadIdx.x == 0) put_row(a, r, empty, tok_ok, zx, M, lnz, W / Z);
    if constexpr (LISTS) {
        // ---- the chunks that reach the bound, a warp each; every lane keeps the
        // best of its logits
        float thr = thr_key == kNoKey ? kNegInf : key_value(thr_key);
        const bool none = empty || Z != Z;                     // (a wait of the stream ran out)
        for (int i = threadIdx.x; i < P; i += kMergeThreads) {
            const float m = i == (int)threadIdx.x ? first.x : __ldcg(st + i).x;
            if (m >= thr && !none) sel[atomicAdd(&n_sel, 1)] = (unsigned short)i;
        }
        __syncthreads();
        const int n = none ? 0 : n_sel;
        for (int c = warp; c < n; c += NW) {
            uint4 v[kVecPerLane];
            unsigned long long row;
            const int base = load_chunk<ELT>(a, r, (long long)sel[c] * (32 * kLaneBytes), v, row);
            pool_chunk<ELT>(v, row, base, thr, chunks[warp], pool);
        }
        __syncthreads();
        float ov[KC];
        int oi[KC];
        const int got = pool.n;
        if (got <= kPool) {                                    // uniform
            if (warp == 0) {
                pool_lists(pool, got, a.K, ov, oi);
                if (lane == 0) put_list(a, r, none, M, lnz, ov, oi);
            }
            return;
        }
        TopList<KC> L;
        L.init();
        for (int c = warp; c < n; c += NW) {
            uint4 v[kVecPerLane];
            unsigned long long row;
            const int base = load_chunk<ELT>(a, r, (long long)sel[c] * (32 * kLaneBytes), v, row);
            pick_chunk<ELT>(v, row, base, a.K, thr, chunks[warp], L);
        }
        merge_lists<KC>(L, a.K, ov, oi);
        if (lane == 0) {
#pragma unroll
            for (int q = 0; q < KC; ++q) { list_v[warp][q] = ov[q]; list_i[warp][q] = oi[q]; }
        }
        __syncthreads();
        if (warp == 0) {
            L.init();
            L.insert(list_v[lane / KC][lane & (KC - 1)], list_i[lane / KC][lane & (KC - 1)]);
            merge_lists<KC>(L, a.K, ov, oi);
            if (lane == 0) put_list(a, r, none, M, lnz, ov, oi);
        }
    }
}

static int logprob_nseg(int V, int elt) {
    return (int)(((long long)V * elt + (16 - elt) + kStageBytes - 1) / kStageBytes);
}

size_t logprobs_workspace_size(int rows, int V, int K) {
    // error word, then the sums of every warp chunk (fp32 has the most)
    return 256 + align256((size_t)rows * (size_t)logprob_nseg(V, 4) * kWarps * sizeof(float4));
}

template <int ELT>
static cudaError_t launch_logprobs_e(const LogprobArgs& a, const DeviceInfo& di, cudaStream_t st) {
    const int span = (int)(((long long)a.V * ELT + (16 - ELT) + 32 * kLaneBytes - 1) / (32 * kLaneBytes));     // warp chunks of a row
    if (span <= kRowChunks && (a.K > 0 || span <= kFewChunks || (long long)a.rows * span <= kRowChunks * di.sm_count)) {
        const int turns = (span + kRowWarps - 1) / kRowWarps, warps = (span + turns - 1) / turns;
        const dim3 grid((unsigned)a.rows);
        if (a.K == 0) return launch_pdl(logprob_row_kernel<ELT, false>, grid, warps * 32, 0, st, a, span);
        return launch_pdl(logprob_row_kernel<ELT, true>, grid, warps * 32, (size_t)warps * 32 * kLaneBytes, st, a, span);
    }
    auto kfn = logprob_stream_kernel<ELT>;
    auto merge = a.K > 0 ? logprob_merge_kernel<ELT, true> : logprob_merge_kernel<ELT, false>;
    const int smem = kStages * kStageBytes;
    static DeviceSlots slots = {};
    int occ = 0;
    cudaError_t e = device_once(slots, &occ, [&](int, int* o) {
        cudaError_t r = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (r != cudaSuccess) return r;
        // the whole carveout as shared memory for all of them, so that an SM can
        // hold the merge's CTAs beside the stream's
        for (const void* f : {(const void*)kfn, (const void*)logprob_merge_kernel<ELT, true>, (const void*)logprob_merge_kernel<ELT, false>}) {
            r = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
            if (r != cudaSuccess) return r;
        }
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(o, kfn, kRingThreads, smem);
    });
    if (e != cudaSuccess) return e;
    long long g = (long long)di.sm_count * occ;
    if (a.chunks < g) g = a.chunks;
    e = launch_pdl(kfn, dim3((unsigned)g), kRingThreads, smem, st, a);
    if (e != cudaSuccess) return e;
    const size_t sel = a.K > 0 ? (size_t)a.nseg * kWarps * sizeof(unsigned short) : 0;
    return launch_pdl(merge, dim3((unsigned)a.rows), kMergeThreads, sel, st, a);
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
    a.inv_s = (float)((double)T / 1.4426950408889634);
    a.rows = rows;
    a.V = V;
    a.K = K;
    a.nseg = logprob_nseg(V, elt);
    a.chunks = (long long)rows * a.nseg;
    a.err = reinterpret_cast<int*>(w);
    a.stats = reinterpret_cast<float4*>(w + 256);
    a.lp = lp;
    a.ent = ent;
    a.ti = ti;
    a.tl = tl;
    a.wait_limit = ring_wait_limit();
    return elt == 2 ? launch_logprobs_e<2>(a, di, st) : launch_logprobs_e<4>(a, di, st);
}

}  // namespace sv
