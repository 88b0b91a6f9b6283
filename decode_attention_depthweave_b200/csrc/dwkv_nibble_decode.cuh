// dwkv_nibble_decode.cuh -- attention over the 4-bit cache for few rows a request: up to 32
// rows (query rows x query heads of a kv-head), the decode and draft-verify steps.
//
// o = sum_t w_t v_t over t, in one pass with a running maximum and sum.  Each byte of the cache
// (144 a token and kv-head at d = 128) is read once, but latency bounds it: 3.7 warps a scheduler, each in one
// chain of unpacking, score products, exponentials and value products, use 56 % of the issue slots and 47 %
// of the ALU pipe (every pair of codes passes a LOP3 and an HFMA2 on its way to the tensor cores; a 16-token
// block takes a warp some 335 instructions).  Measured (bf16, d 128, 8 kv-heads, G = 4): 300 tokens 12 to 13 us,
// 65536 tokens of one request 29 us (2.6 TB/s), 8 requests of 16384 to 32768 61.5 us (3.8 TB/s, 59 % of a copy's
// rate); 160 of 4096 at d 64, fp16, 29 us.
//
//  - Units of 16 kWarps tokens of a (request, kv-head), in one flat order, are cut into equal
//    contiguous ranges, one a CTA: any mix of lengths loads the SMs evenly, and no host code
//    has to know a length.  A (request, kv-head) cut by a range end leaves records that the last
//    CTA to finish merges (an atomic ticket, no wait).
//  - A consumer warp takes two 16-token blocks of each unit and keeps its own maximum, sum and
//    accumulator: consumers meet only where a (request, kv-head) ends.  A producer warp keeps a ring
//    of blocks in flight for each of them (bulk copies on mbarriers, across request borders), a
//    lane a block, and refills a warp's stage when that warp has read it: with stages shared by all
//    warps, the slowest held up the copies of the others (75 -> 109 us at two stages of 36 KB).
//  - S^T = K Q^T: tokens are the 16 MMA rows, query rows the 8 columns; a lane reads 16 bytes of
//    two tokens' codes and unpacks them to fp16 (exact) in registers.  O^T = V^T P^T: channels are
//    the MMA rows, ldmatrix.trans pairs two tokens' units, P is transposed by movmatrix.
//  - P is rounded to fp16 (11 bits) for the value product: finer than a bf16 output.  An fp16
//    output of up to 4 rows gets P's remainder too: the columns 4-7 hold the same queries again,
//    and in the value product what the rounding left, so P is good to 22 bits.
//  - P carries 2^7: with the maximum allowed to lag 2^8 behind, it stays below 2^15, and weights
//    down to 2^-31 keep a bit.
//  - Weights are 2^(s fac + (7 - m)) by one fma, with the rounded m = s_max fac.  From |m| = 2^21 on that rounding,
//    the same for all of a row, could carry P out of fp16: such rows' scores are multiplied and rounded as m is, which
//    leaves the largest weight at 2^0 to 2^8, and no lag is allowed.  That stands where the maximum moves, so that
//    the other rows' loop does not know of it.
#pragma once
#include "dwkv_nibble.cuh"

namespace dwkv {

// Seven consumers and the producer are 8 warps: two CTAs an SM leave a thread 128 registers, and the
// loop's accumulators, scores and fragments fit (with eight consumers, 96: it spilled, 75 -> 110 us at
// 8 requests of 16384 to 32768).
constexpr int kNdWarps = 7;
constexpr int kNdThreads = 32 * kNdWarps;               // consumers; one more warp produces
constexpr int kNdSub = 2;                                // blocks that a warp takes at a time
constexpr int kNdBlocks = kNdSub * kNdWarps;             // blocks of a unit
constexpr int kNdUnit = kNibBlock * kNdBlocks;           // tokens of a unit
constexpr float kNdNone = -3.402823466e38f;              // maximum of nothing
constexpr float kNdLag = 8.f, kNdBias = 7.f;             // log2
constexpr float kNdFar = 2097152.f;                      // log2

template <int D, int R>
struct NdLayout {
    static constexpr int kMr = R < 8 ? R : 8;            // rows merged at a time
    static constexpr int kCtas = R <= 8 ? 2 : 1;         // an SM
    static constexpr int kStages = (D == 128 ? 1 : 2) * (R <= 4 ? 3 : R <= 8 ? 2 : 4);
    static constexpr uint32_t kBlock = 18u * D;
    static constexpr uint32_t kStage = kNdSub * kBlock;  // of one warp
    static constexpr int kPitch = D + 4;                 // floats of a merge row: 16-byte accesses of a warp fall in distinct banks
    static constexpr uint32_t kMerge = (uint32_t)kNdWarps * kStages * kStage;       // [warps][kMr][kPitch] fp32
    static constexpr int kCols = R < 16 ? 16 : R;        // of the maxima and sums
    static constexpr uint32_t kMl = kMerge + (uint32_t)kNdWarps * kMr * kPitch * 4; // m [warps][kCols], l [warps][kCols]
    static constexpr uint32_t kQ = kMl + (uint32_t)kNdWarps * kCols * 8;               // the queries' fragments [tiles][D/32][lane] 16 bytes
    static constexpr uint32_t kBars = kQ + (R + 7u) / 8u * (D / 32) * 512;        // full [warps][stages], empty [warps][stages]
    static constexpr uint32_t kFlags = kBars + 2u * kNdWarps * kStages * 8;         // [warps][stages][2] bytes: bit 0 not there, bit 1 seen in part
    static constexpr uint32_t kScan = (kFlags + 2u * kNdWarps * kStages + 15u) & ~15u;         // scan scratch, 128 bytes
    static constexpr uint32_t kBytes = kScan + 128;
};

// Two units (unit u of two rows side by side in a word, 4 codes each) -> 4 fp16 pairs c * s / 32.
// r: the scales as fp16, b0 = -8.25 r, b1 = -0.75 r.  Code j of a unit sits at bits 2-5 (j = 0, 2)
// or 6-9 (j = 1, 3) of the half word or of its byte swap: as the mantissa of 8 and of 1/2 it is
// 8 + u/32 and 1/2 + u/32 for u = c + 8, and r times that plus b is r c / 32, exactly.
__device__ __forceinline__ uint32_t lop_and_or(uint32_t a, uint32_t m, uint32_t o) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(m), "r"(o));
    return r;
}
__device__ __forceinline__ uint32_t hfma2_(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t hmul2_(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// e8, eh: 8 and 1/2 as fp16 pairs, in registers (a LOP3 takes one immediate; of two, the compiler
// makes two instructions).
__device__ __forceinline__ uint32_t reg_const(uint32_t v) {
    uint32_t r;
    asm volatile("mov.u32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void nib_unpack(uint32_t u, uint32_t r, uint32_t b0, uint32_t b1, uint32_t e8, uint32_t eh, uint32_t (&o)[4]) {
    const uint32_t w = __byte_perm(u, 0, 0x2301);
    o[0] = hfma2_(lop_and_or(u, 0x003c003cu, e8), r, b0);
    o[1] = hfma2_(lop_and_or(u, 0x03c003c0u, eh), r, b1);
    o[2] = hfma2_(lop_and_or(w, 0x003c003cu, e8), r, b0);
    o[3] = hfma2_(lop_and_or(w, 0x03c003c0u, eh), r, b1);
}
// D (16x8 f32) = A (16x16 f16, row) * B (16x8 f16, col)
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.f));
}
constexpr uint32_t kNibB0 = 0xc820c820u, kNibB1 = 0xba00ba00u;      // -8.25, -0.75 as fp16 pairs
// One poll of an mbarrier's phase that may sleep for a fraction of a microsecond.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(200u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint32_t movm_t(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float half_lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))); }
__device__ __forceinline__ float half_hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }

// Queries enter the products as fp16, each row times the power of two that brings its largest magnitude a
// to [2^15, 2^16).  That is exact for fp16 rows (they only grow) and for bf16 ones down to 2^-32 of a; what is
// smaller errs by at most 2^-40 a.  Returns the factor; fac: from a score of such rows and of values in units of 32
// to log2 units, never 0, since a masked score is -inf times it.
__device__ __forceinline__ float nib_query_scale(const NibGeom& G, float a, float& fac) {
    const uint32_t e = min(max(__float_as_uint(a) >> 23, 15u), 254u);
    fac = fmaxf(G.tau * 1.4426950408889634f * 0x1p-10f * __uint_as_float(e << 23), 1.17549435e-38f);
    // an infinite query has no softmax, even where all its scores are -inf: NaN from here on
    return a < INFINITY ? __uint_as_float((269u - e) << 23) : __uint_as_float(0x7fc00000u);
}

// A row's maximum is so large that its scores are rounded, as it is, before it is taken from them.
__device__ __forceinline__ bool nib_far(float m) { return fabsf(m) >= kNdFar && m > kNdNone; }

// Empty units counted behind each (request, kv-head): what its end costs a CTA (merging the warps,
// writing, the next one's queries) in units, so that ranges with an end in them carry less.
constexpr int kNdBorder = 1;

// Where a request's tokens start and how many units they are (none where it has no rows).
struct NdSpan {
    int len, nq, base, units;                            // units: of one kv-head, kNdBorder of them empty
};
__device__ __forceinline__ NdSpan nd_span(const NibGeom& G, const NibAttend& A, int b) {
    NdSpan s{0, 0, 0, 0};
    if (b >= A.n) return s;
    if (!nib_request(G, A, b, s.len, s.nq) || s.nq == 0 || s.nq * G.g > A.rows_hi) { s.nq = 0; return s; }
    s.base = nib_first_seen(G, s.len - s.nq) & ~15;
    s.units = max(1, (s.len - s.base + kNdUnit - 1) / kNdUnit) + kNdBorder;
    return s;
}

// A warp's walk over the segments of its CTA's range: parts of (request, kv-head)s, in order.
// 32 requests' spans at a time sit in the lanes.
struct NdWalk {
    int b, h, unit, left;                // segment: request, kv-head, its first unit; units of the range from there on
    int from;                            // request in lane 0
    NdSpan mine;                         // this lane's
    int len, nq, base, units;            // the segment's request

    __device__ __forceinline__ void fetch(const NibGeom& G, const NibAttend& A, int lane) { mine = nd_span(G, A, from + lane); }
    __device__ __forceinline__ void take() {
        const int l = b - from;
        len = __shfl_sync(~0u, mine.len, l);
        nq = __shfl_sync(~0u, mine.nq, l);
        base = __shfl_sync(~0u, mine.base, l);
        units = __shfl_sync(~0u, mine.units, l);
    }
    __device__ __forceinline__ int real() const { return units - kNdBorder; }
    __device__ __forceinline__ int count() const { return min(left, real() - unit); }   // units of this segment
    // To the next segment; false at the end of the range.
    __device__ __forceinline__ bool next(const NibGeom& G, const NibAttend& A, int lane) {
        left -= min(left, units - unit);
        if (left <= 0) return false;
        unit = 0;
        if (++h < G.hkv) return true;
        h = 0;
        ++b;
        for (;;) {
            const uint32_t some = __ballot_sync(~0u, mine.units > 0);
            const uint32_t rest = b - from < 32 ? some >> (b - from) << (b - from) : 0u;
            if (rest) { b = from + __ffs(rest) - 1; break; }
            from += 32;
            b = from;
            if (from >= A.n) { left = 0; return false; }      // cannot be: left counts units that exist
            fetch(G, A, lane);
        }
        take();
        return true;
    }
};

// A record of a cut (request, kv-head): [R] m, [R] l, [R][D] unnormalised o.

template <int D, int R, bool SPLIT, bool FP16>
__global__ void __launch_bounds__(kNdThreads + 32, NdLayout<D, R>::kCtas) nib_decode_kernel(const NibGeom G, const NibAttend A) {
    using L = NdLayout<D, R>;
    constexpr int NT = (R + 7) / 8;                      // MMA column tiles
    constexpr int kWords = D / 32, kChunks = D / 32;
    static_assert(!SPLIT || R <= 4, "the remainders take columns 4-7");
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ int s_last[3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, i = lane & 3;
    const uint32_t sbase = smem_addr(sm);
    constexpr uint32_t kToEmpty = 8u * kNdWarps * L::kStages;        // from a stage's full barrier to its empty one
    const uint32_t bars = sbase + L::kBars;
    if (tid < kNdWarps * L::kStages) {
        mbar_init(bars + 8u * tid, kNdSub);
        mbar_init(bars + kToEmpty + 8u * tid, 1u);
        fence_mbar_init();
    }

    // ---- this CTA's range of units, floor(total c / n) of them before CTA c
    NdWalk w;
    int each, extra, at0, ctas;                          // total = ctas each + extra; at0: the range's first unit
    {
        int* red = reinterpret_cast<int*>(sm + L::kScan);   // [warps], start [3]
        long long total = 0, before = 0, mine = 0;
        w.from = 0;
        if (A.n <= 32) {                                 // a warp sees all requests: no block-wide scan
            w.fetch(G, A, lane);
            mine = (long long)w.mine.units * G.hkv;
        } else {
            const int per = (A.n + kNdThreads - 1) / kNdThreads;
            const int b0 = min(A.n, tid * per), b1 = min(A.n, b0 + per);   // none for the producer warp
            for (int b = b0; b < b1; ++b) mine += (long long)nd_span(G, A, b).units * G.hkv;
        }
        before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(~0u, before, o);
            if (lane >= o) before += x;
        }
        total = __shfl_sync(~0u, before, 31);
        before -= mine;
        long long* sums = reinterpret_cast<long long*>(red);
        if (A.n > 32) {
            if (lane == 0 && warp < kNdWarps) sums[warp] = total;
            __syncthreads();
            total = 0;
#pragma unroll
            for (int k = 0; k < kNdWarps; ++k) {
                if (k == warp) before += total;
                total += sums[k];
            }
        }
        if (total >= (1ll << 31)) {                      // more than this kernel counts
            if (blockIdx.x == 0 && tid == 0) nib_error(G, 10u /*DWKV_DEV_BAD_LENGTH*/, 0xffffffffu, (uint32_t)(total >> 31));
            return;
        }
        const int n = min((int)gridDim.x, (int)total);   // CTAs with work
        if ((int)blockIdx.x >= n) return;
        each = (int)total / n;
        extra = (int)total - each * n;
        ctas = n;
        at0 = each * (int)blockIdx.x + extra * (int)blockIdx.x / n;
        w.left = each * (int)(blockIdx.x + 1) + extra * (int)(blockIdx.x + 1) / n - at0;
        const bool here = at0 >= before && at0 < before + mine;
        if (A.n <= 32) {
            const uint32_t who = __ballot_sync(~0u, here);
            w.b = __ffs(who) - 1;
            w.take();
            const int at = at0 - (int)__shfl_sync(~0u, before, w.b);
            w.h = at / w.units;
            w.unit = at - w.h * w.units;
        } else {
            int* start = red + 2 * kNdWarps;
            if (here) {
                int at = at0 - (int)before;
                const int per = (A.n + kNdThreads - 1) / kNdThreads;
                for (int b = tid * per; b < A.n; ++b) {
                    const NdSpan s = nd_span(G, A, b);
                    if (at < s.units * G.hkv) {
                        start[0] = b;
                        start[1] = at / s.units;
                        start[2] = at % s.units;
                        break;
                    }
                    at -= s.units * G.hkv;
                }
            }
            __syncthreads();
            w.b = start[0];
            w.h = start[1];
            w.unit = start[2];
            w.from = w.b & ~31;
            w.fetch(G, A, lane);
            w.take();
        }
    }
    __syncthreads();                                     // the mbarriers are ready
    // The CTA that has unit u.
    auto cta_of = [&](int u) {
        return (int)((((long long)u + 1) * ctas - 1) / ((long long)each * ctas + extra));
    };

    int at = at0;                                        // the unit at which the walk stands
    if (w.unit >= w.real()) {                            // the range starts in the empty units behind a kv-head
        at += min(w.left, w.units - w.unit);
        if (!w.next(G, A, lane)) return;
    }

    // ---- producer: lane 2 w + k keeps block k of warp w's stages filled
    if (warp == kNdWarps) {
        const int cw = min(lane / kNdSub, kNdWarps - 1), sub = lane % kNdSub;
        const uint32_t ring = bars + 8u * cw * L::kStages;
        int stage = 0, rounds = 0;
        bool ok = true;
        for (bool some = true; ok && some; some = w.next(G, A, lane)) {
            const int cnt = lane < kNdBlocks ? w.count() : 0;
            const int end = min(w.len, w.base + (w.unit + w.count()) * kNdUnit);
            const int inner_hi = w.len - w.nq;           // tokens up to here are seen by every row,
            const int inner_lo = G.window > 0 ? w.len - G.window : 0;   // and from here on
            const int32_t* row = A.table + (size_t)w.b * G.max_blocks;
            int t = w.base + w.unit * kNdUnit + 16 * lane, u = 0;
            int id = cnt > 0 && t < end ? __ldg(row + (t >> G.page_shift)) : -1;
            uint32_t idle = 0;
            uint64_t since = 0;
            while (__any_sync(~0u, u < cnt)) {
                // a full turn of polls without a copy is timed
                const bool go = u < cnt && (rounds == 0 || mbar_poll(ring + kToEmpty + 8u * stage, (uint32_t)(rounds - 1) & 1u));
                if (__any_sync(~0u, go)) {
                    idle = 0;
                } else if ((++idle & 63u) == 0u) {
                    if (idle == 64u) since = global_ns();
                    if (__any_sync(~0u, global_ns() - since > kWaitLimitNs)) {
                        ok = false;
                        break;
                    }
                }
                if (go) {
                    const bool there = t < end, good = there && (unsigned)id < (unsigned)G.num_pages;
                    if (there && !good) nib_error(G, 11u /*DWKV_DEV_BAD_PAGE*/, (uint32_t)w.b, (uint32_t)id);
                    sm[L::kFlags + (cw * L::kStages + stage) * kNdSub + sub] = (uint8_t)((good ? 0 : 1) | (t + 15 > inner_hi || t < inner_lo ? 2 : 0));
                    if (good) {
                        mbar_arrive_expect_tx(ring + 8u * stage, L::kBlock);
                        bulk_g2s(sbase + (uint32_t)((cw * L::kStages + stage) * kNdSub + sub) * L::kBlock,
                                 A.pool + nib_block_at(G, id, w.h, t & (G.page - 1)), L::kBlock, ring + 8u * stage);
                    } else {
                        mbar_arrive(ring + 8u * stage);
                    }
                    if (++stage == L::kStages) {
                        stage = 0;
                        ++rounds;
                    }
                    t += kNdUnit;
                    ++u;
                    if (u < cnt && t < end) id = __ldg(row + (t >> G.page_shift));
                }
            }
        }
        if (!ok) {                                       // the copies in flight end first, each wait with a limit
            if (lane == 0) nib_error(G, 6u /*DWKV_DEV_TIMEOUT*/, 0x6e70u, (uint32_t)w.b);
            for (int k = 0; k < L::kStages; ++k)
                if (rounds > 0 || k < stage) mbar_wait_for(ring + 8u * k, (uint32_t)(rounds - (k >= stage)) & 1u, 10000000ull);
        }
        return;
    }

    // ---- consumer side
    const uint32_t c_ring = bars + 8u * warp * L::kStages;
    uint32_t c_stage = 0, c_phase = 0;
    const uint32_t e8 = reg_const(0x48004800u), eh = reg_const(0x38003800u);
    bool dead = false;                                   // a wait ran out: what is left is left out
    // ldmatrix row of this lane: token vrow, 16-byte chunk 0 or 1; chunks 2 and 3 are 32 bytes away, by xor
    const int vrow = (lane & 7) + ((lane >> 3) & 1) * 8;
    const uint32_t vaddr = 9u * D + (uint32_t)vrow * (D / 2) + (uint32_t)nib_vchunk(D, vrow, lane >> 4) * 16u;
    for (bool more = true; more; more = w.next(G, A, lane)) {
        const int cnt = w.count(), rows = w.nq * G.g;
        const int row0 = A.cu[w.b];
        // queries as B fragments, each row as nib_query_scale says
        uint4* qs = reinterpret_cast<uint4*>(sm + L::kQ) + lane;
        float fac[NT][2];                                // unscaled score -> log2 units, for the lane's columns; 1 for far rows
        // ... and as it was, where the warp's maxima go at the segment's end
        float* units_of = reinterpret_cast<float*>(sm + L::kMl) + warp * L::kCols + 2 * i;
        int pos[NT][2];                                  // position of the lane's columns' rows
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = SPLIT ? (g & 3) : nt * 8 + g;
            uint32_t raw[kWords][4];
            float a = 0.f;
            const bool have = r < rows;
            const int j = have ? r / G.g : 0;
            const uint16_t* qp = A.q + (size_t)(row0 + j) * A.q_stride + (size_t)(w.h * G.g + (have ? r - j * G.g : 0)) * D + i * (D / 4);
#pragma unroll
            for (int x = 0; x < kWords; ++x) {
                const uint4 v = have ? *reinterpret_cast<const uint4*>(qp + 8 * x) : make_uint4(0, 0, 0, 0);
                raw[x][0] = v.x; raw[x][1] = v.y; raw[x][2] = v.z; raw[x][3] = v.w;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    a = fmaxf(a, fabsf(FP16 ? half_lo(raw[x][y]) : bf16lo(raw[x][y])));
                    a = fmaxf(a, fabsf(FP16 ? half_hi(raw[x][y]) : bf16hi(raw[x][y])));
                }
            }
            a = fmaxf(a, __shfl_xor_sync(~0u, a, 1));
            a = fmaxf(a, __shfl_xor_sync(~0u, a, 2));
            float mult;
            const float sc = nib_query_scale(G, a, mult);
#pragma unroll
            for (int x = 0; x < kWords; ++x) {
                float f[8];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    f[2 * y] = (FP16 ? half_lo(raw[x][y]) : bf16lo(raw[x][y])) * sc;
                    f[2 * y + 1] = (FP16 ? half_hi(raw[x][y]) : bf16hi(raw[x][y])) * sc;
                }
                if (warp == 0)                           // every warp has the same; one writes
                    qs[(nt * kWords + x) * 32] = make_uint4(pack_half2(f[0], f[4]), pack_half2(f[1], f[5]),
                                                            pack_half2(f[2], f[6]), pack_half2(f[3], f[7]));
            }
            fac[nt][0] = __shfl_sync(~0u, mult, 8 * i);
            fac[nt][1] = __shfl_sync(~0u, mult, 8 * i + 4);
            if (g == 0) *reinterpret_cast<float2*>(units_of + nt * 8) = make_float2(fac[nt][0], fac[nt][1]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = SPLIT ? ((2 * i + c) & 3) : nt * 8 + 2 * i + c;
                pos[nt][c] = w.len - w.nq + min(col, rows - 1) / G.g;
            }
        }
        float m[NT][2], thr[NT][2], l[NT][2], o[NT][2 * kChunks][4];   // thr: the unscaled score that moves m
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = kNdNone;
            thr[nt][0] = thr[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int x = 0; x < 2 * kChunks; ++x) o[nt][x][0] = o[nt][x][1] = o[nt][x][2] = o[nt][x][3] = 0.f;
        }
        named_barrier(1, kNdThreads);
        int t0 = w.base + w.unit * kNdUnit + kNdSub * 16 * warp;
        for (int u = 0; u < cnt; ++u, t0 += kNdUnit) {
            const uint32_t at_s = warp * L::kStages + c_stage, c_off = at_s * L::kStage;
            if (!dead && !mbar_wait(c_ring + 8u * c_stage, c_phase)) {
                dead = true;
                if (lane == 0) nib_error(G, 6u /*DWKV_DEV_TIMEOUT*/, 0x6e64u, (uint32_t)w.b);
            }
            const uint32_t flag = *reinterpret_cast<const uint16_t*>(sm + L::kFlags + kNdSub * at_s);
            if (!dead && (flag & 0x101u) != 0x101u) {
                const bool edge = flag;                  // a block not there, or not seen whole by every row
                // ---- scores of 32 tokens
                float s[kNdSub][NT][4];
#pragma unroll
                for (int k = 0; k < kNdSub; ++k) {
                    const uint8_t* blk = sm + c_off + k * L::kBlock;
                    uint32_t kw[2][kWords];
                    if (D == 128) {
                        const uint4 a = *reinterpret_cast<const uint4*>(blk + g * 64 + i * 16);
                        const uint4 b = *reinterpret_cast<const uint4*>(blk + (g + 8) * 64 + i * 16);
                        kw[0][0] = a.x; kw[0][1] = a.y; kw[0][kWords - 2] = a.z; kw[0][kWords - 1] = a.w;
                        kw[1][0] = b.x; kw[1][1] = b.y; kw[1][kWords - 2] = b.z; kw[1][kWords - 1] = b.w;
                    } else {
                        const uint2 a = *reinterpret_cast<const uint2*>(blk + g * 32 + i * 8);
                        const uint2 b = *reinterpret_cast<const uint2*>(blk + (g + 8) * 32 + i * 8);
                        kw[0][0] = a.x; kw[0][1] = a.y;
                        kw[1][0] = b.x; kw[1][1] = b.y;
                    }
                    float s2[NT][4];
#pragma unroll
                    for (int grp = 0; grp < kWords / 2; ++grp) {     // 16 channels of the lane share a scale
                        uint32_t r[2], b0[2], b1[2];
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            // the scale byte << 7 in both halves
                            r[z] = 0x00800080u * blk[8 * D + (g + 8 * z) * (D / 16) + i * (D / 64) + grp];
                            b0[z] = hmul2_(r[z], kNibB0);
                            b1[z] = hmul2_(r[z], kNibB1);
                        }
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int x = 2 * grp + y;
                            uint32_t u0[4], u1[4];
                            nib_unpack(kw[0][x], r[0], b0[0], b1[0], e8, eh, u0);
                            nib_unpack(kw[1][x], r[1], b0[1], b1[1], e8, eh, u1);
                            const uint32_t a0[4] = {u0[0], u1[0], u0[1], u1[1]}, a1[4] = {u0[2], u1[2], u0[3], u1[3]};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint4 q = qs[(nt * kWords + x) * 32];
                                const uint32_t q0[2] = {q.x, q.y}, q1[2] = {q.z, q.w};
                                if (x == 0) {
                                    mma_f16_first(s[k][nt], a0, q0);
                                    mma_f16_first(s2[nt], a1, q1);
                                } else {
                                    mma_f16(s[k][nt], a0, q0);
                                    mma_f16(s2[nt], a1, q1);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[k][nt][x] += s2[nt][x];
                }
                if (edge) {                              // the volatile keeps this a branch: few blocks take it
                    asm volatile("" ::: "memory");
#pragma unroll
                    for (int k = 0; k < kNdSub; ++k)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const int t = t0 + 16 * k + g + 8 * (x >> 1), hi = pos[nt][x & 1];
                                if ((flag >> 8 * k & 1u) || t > hi || (G.window > 0 && t <= hi - G.window)) s[k][nt][x] = -INFINITY;
                            }
                }
                bool jump = false;
#pragma unroll
                for (int k = 0; k < kNdSub; ++k)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) jump |= s[k][nt][x] > thr[nt][x & 1];
                if (__any_sync(~0u, jump)) {             // the maximum moves: all rows take the new one
                    bool far = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float x = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
                            for (int k = 1; k < kNdSub; ++k) x = fmaxf(x, fmaxf(s[k][nt][c], s[k][nt][c + 2]));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                            const float unit = units_of[nt * 8 + c];
                            x = fmaxf(m[nt][c], unit * fmaxf(x, __shfl_xor_sync(~0u, x, 16)));
                            const float f = ex2(m[nt][c] - x);
                            m[nt][c] = x;
                            thr[nt][c] = x > kNdNone && !nib_far(x) ? (x + kNdLag) / unit : -INFINITY;
                            fac[nt][c] = nib_far(x) ? 1.f : unit;
                            far |= nib_far(x);
                            l[nt][c] *= f;
#pragma unroll
                            for (int y = 0; y < 2 * kChunks; ++y) {
                                o[nt][y][c] *= f;
                                o[nt][y][c + 2] *= f;
                            }
                        }
                    if (__any_sync(~0u, far)) {          // rounded scores in place of far rows' ones
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const float by = nib_far(m[nt][c]) ? units_of[nt * 8 + c] : 1.f;
#pragma unroll
                                for (int k = 0; k < kNdSub; ++k) {
                                    s[k][nt][c] *= by;
                                    s[k][nt][c + 2] *= by;
                                }
                            }
                    }
                }
#pragma unroll
                for (int k = 0; k < kNdSub; ++k) {
                    uint32_t pf[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float pr[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            pr[x] = ex2(fmaf(s[k][nt][x], fac[nt][x & 1], kNdBias - m[nt][x & 1]));
                            l[nt][x & 1] += pr[x];
                        }
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            uint32_t h = pack_half2(pr[2 * z], pr[2 * z + 1]);
                            if (SPLIT) {                 // columns 4-7: what the rounding left
                                const uint32_t rest = pack_half2(pr[2 * z] - half_lo(h), pr[2 * z + 1] - half_hi(h));
                                h = i >= 2 ? rest : h;
                            }
                            pf[nt][z] = movm_t(h);
                        }
                    }
                    // ---- values: O^T += V^T P^T
                    const uint8_t* blk = sm + c_off + k * L::kBlock;
                    uint32_t vs[kChunks];
                    if (D == 128) {
                        const uint4 v = *reinterpret_cast<const uint4*>(blk + 17 * D + ((g >> 2) * 4 + i) * 16);
                        vs[0] = v.x; vs[1] = v.y; vs[kChunks - 2] = v.z; vs[kChunks - 1] = v.w;
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(blk + 17 * D + ((g >> 2) * 4 + i) * 8);
                        vs[0] = v.x; vs[1] = v.y;
                    }
                    if (edge) {                          // bytes behind the last token are not to be believed
                        asm volatile("" ::: "memory");
                        const int t = t0 + 16 * k + 2 * i, len = flag >> 8 * k & 1u ? 0 : w.len;
                        uint32_t keep = 0;
                        if (t < len) keep |= 0xffu;
                        if (t + 1 < len) keep |= 0xff00u;
                        if (t + 8 < len) keep |= 0xff0000u;
                        if (t + 9 < len) keep |= 0xff000000u;
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) vs[c] &= keep;
                    }
#pragma unroll
                    for (int c2 = 0; c2 < kChunks; c2 += 2) {
                        uint32_t v[4];
                        ldsm_x4_t(sbase + c_off + k * L::kBlock + (vaddr ^ (uint32_t)(c2 * 16)), v);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int c = c2 + y;
                            uint32_t u[2][4];
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const uint32_t r = __byte_perm(vs[c], 0, z ? 0x3424 : 0x1404) >> 1;
                                nib_unpack(v[2 * y + z], r, hmul2_(r, kNibB0), hmul2_(r, kNibB1), e8, eh, u[z]);
                            }
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t a[4] = {u[0][2 * e], u[0][2 * e + 1], u[1][2 * e], u[1][2 * e + 1]};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][2 * c + e], a, pf[nt]);
                            }
                        }
                    }
                }
            }
            __syncwarp();                                // the blocks are read: their stage takes another unit
            if (lane == 0 && !dead) mbar_arrive(c_ring + kToEmpty + 8u * c_stage);
            if (++c_stage == L::kStages) {
                c_stage = 0;
                c_phase ^= 1u;
            }
        }

        // ---- the segment ends: merge the warps
        float* ml = reinterpret_cast<float*>(sm + L::kMl);
        float* mo = reinterpret_cast<float*>(sm + L::kMerge);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = l[nt][c];
                x += __shfl_xor_sync(~0u, x, 4);
                x += __shfl_xor_sync(~0u, x, 8);
                x += __shfl_xor_sync(~0u, x, 16);
                if (g == 0) {
                    ml[warp * L::kCols + nt * 8 + 2 * i + c] = m[nt][c];
                    ml[(kNdWarps + warp) * L::kCols + nt * 8 + 2 * i + c] = x;
                }
            }
        const bool whole = w.unit == 0 && cnt == w.real();
        const int first = at - w.unit;                   // unit 0 of this (request, kv-head)
        // Sums the warps' rows of a column tile against their common maximum: put(row, channel, m, l, o).
        auto merge = [&](int nt, auto put) {
            const int r_hi = min(rows - 8 * nt, L::kMr);
            for (int e = tid; e < r_hi * (D / 4); e += kNdThreads) {
                const int r = e / (D / 4), ch = e % (D / 4) * 4;
                float mm = kNdNone;
#pragma unroll
                for (int k = 0; k < kNdWarps; ++k) mm = fmaxf(mm, ml[k * L::kCols + nt * 8 + r]);
                float ll = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kNdWarps; ++k) {
                    const float f = ex2(ml[k * L::kCols + nt * 8 + r] - mm);
                    const float4 v = *reinterpret_cast<const float4*>(mo + (size_t)(k * L::kMr + r) * L::kPitch + ch);
                    ll = fmaf(f, ml[(kNdWarps + k) * L::kCols + nt * 8 + r], ll);
                    acc.x = fmaf(f, v.x, acc.x);
                    acc.y = fmaf(f, v.y, acc.y);
                    acc.z = fmaf(f, v.z, acc.z);
                    acc.w = fmaf(f, v.w, acc.w);
                }
                put(nt * 8 + r, ch, mm, ll, acc);
            }
        };
        float* rec = A.records + (size_t)(2 * blockIdx.x + (at == at0 ? 0 : 1)) * (R * (D + 2));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt) named_barrier(1, kNdThreads);        // the merge rows are free again
            if (SPLIT) {                                 // the remainders' products join their rows
#pragma unroll
                for (int y = 0; y < 2 * kChunks; ++y)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[nt][y][x] += __shfl_xor_sync(~0u, o[nt][y][x], 2);
            }
            if (R > 4 || i < 2) {
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        *reinterpret_cast<float4*>(mo + (size_t)(warp * L::kMr + 2 * i + y) * L::kPitch + 32 * c + 4 * g) =
                            make_float4(o[nt][2 * c][y], o[nt][2 * c][y + 2], o[nt][2 * c + 1][y], o[nt][2 * c + 1][y + 2]);
            }
            named_barrier(1, kNdThreads);
            merge(nt, [&](int r, int ch, float m_, float l_, float4 o_) {
                if (whole) {
                    nib_put<FP16>(G, A, row0, w.h, r, D, ch, m_, l_, o_);
                } else {
                    if (ch == 0) { rec[r] = m_; rec[R + r] = l_; }
                    *reinterpret_cast<float4*>(rec + 2 * R + (size_t)r * D + ch) = o_;
                }
            });
        }
        if (!whole) {                                    // the last CTA of this (request, kv-head) merges the records
            named_barrier(1, kNdThreads);
            if (tid == 0) {                              // the barrier, then one fence: the whole CTA's record is out
                __threadfence();
                const int c0 = cta_of(first), c1 = cta_of(first + w.real() - 1);
                const int k = atomicAdd(A.tickets + c0, 1);
                s_last[0] = k == c1 - c0;
                s_last[1] = c0;
                s_last[2] = c1;
                if (k == c1 - c0) A.tickets[c0] = 0;
                __threadfence();
            }
            named_barrier(1, kNdThreads);
            if (s_last[0]) {
                // A warp takes every kNdWarps-th record, a lane four channels of each row; the warps'
                // sums then meet as those of the segment did.
                constexpr int kRec = R * (D + 2), kLanes = D / 4;
                const int c0 = s_last[1], c1 = s_last[2];
                const int slot0 = first == each * c0 + extra * c0 / ctas ? 0 : 1;   // the first CTA's record; the others' are at 0
                const int ch = lane % kLanes * 4, half = lane / kLanes;             // d 64: the half warps take a record each
                constexpr int kHalves = 32 / kLanes;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (nt) named_barrier(1, kNdThreads);
                    float mm[L::kMr], ll[L::kMr];
                    float4 acc[L::kMr];
#pragma unroll
                    for (int r = 0; r < L::kMr; ++r) {
                        mm[r] = kNdNone;
                        ll[r] = 0.f;
                        acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                    constexpr int kAhead = L::kMr <= 4 ? 3 : 1;                     // records in flight
                    for (int c = c0 + warp * kHalves + half; c - half <= c1; c += kNdWarps * kHalves * kAhead) {
                        float m1[kAhead][L::kMr], l1[kAhead][L::kMr];
                        float4 v[kAhead][L::kMr];
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            const int ck = c + k * kNdWarps * kHalves;
                            const float* x = A.records + (size_t)(2 * ck + (ck == c0 ? slot0 : 0)) * kRec + 8 * nt;
#pragma unroll
                            for (int r = 0; r < L::kMr; ++r) {
                                const bool in = ck <= c1 && 8 * nt + r < rows;
                                m1[k][r] = in ? __ldcg(x + r) : kNdNone;
                                l1[k][r] = in ? __ldcg(x + R + r) : 0.f;
                                v[k][r] = in ? __ldcg(reinterpret_cast<const float4*>(x - 8 * nt + 2 * R + (size_t)(8 * nt + r) * D + ch))
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
                            }
                        }
#pragma unroll
                        for (int k = 0; k < kAhead; ++k)
#pragma unroll
                            for (int r = 0; r < L::kMr; ++r) {
                                const float mn = fmaxf(mm[r], m1[k][r]), f0 = ex2(mm[r] - mn), f1 = ex2(m1[k][r] - mn);
                                mm[r] = mn;
                                ll[r] = fmaf(f1, l1[k][r], ll[r] * f0);
                                acc[r].x = fmaf(f1, v[k][r].x, acc[r].x * f0);
                                acc[r].y = fmaf(f1, v[k][r].y, acc[r].y * f0);
                                acc[r].z = fmaf(f1, v[k][r].z, acc[r].z * f0);
                                acc[r].w = fmaf(f1, v[k][r].w, acc[r].w * f0);
                            }
                    }
                    if (kHalves == 2) {                  // the half warps' sums join
#pragma unroll
                        for (int r = 0; r < L::kMr; ++r) {
                            const float mo_ = __shfl_xor_sync(~0u, mm[r], 16), mn = fmaxf(mm[r], mo_);
                            const float f0 = ex2(mm[r] - mn);
                            mm[r] = mn;
                            ll[r] *= f0;
                            acc[r].x *= f0; acc[r].y *= f0; acc[r].z *= f0; acc[r].w *= f0;
                            ll[r] += __shfl_xor_sync(~0u, ll[r], 16);
                            acc[r].x += __shfl_xor_sync(~0u, acc[r].x, 16);
                            acc[r].y += __shfl_xor_sync(~0u, acc[r].y, 16);
                            acc[r].z += __shfl_xor_sync(~0u, acc[r].z, 16);
                            acc[r].w += __shfl_xor_sync(~0u, acc[r].w, 16);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < L::kMr; ++r) {
                        if (half == 0) *reinterpret_cast<float4*>(mo + (size_t)(warp * L::kMr + r) * L::kPitch + ch) = acc[r];
                        if (lane == 0) {
                            ml[warp * L::kCols + nt * 8 + r] = mm[r];
                            ml[(kNdWarps + warp) * L::kCols + nt * 8 + r] = ll[r];
                        }
                    }
                    named_barrier(1, kNdThreads);
                    merge(nt, [&](int r, int c, float m_, float l_, float4 o_) { nib_put<FP16>(G, A, row0, w.h, r, D, c, m_, l_, o_); });
                }
            }
        }
        named_barrier(1, kNdThreads);                    // the merge rows are free for the next segment
        at += min(w.left, w.units - w.unit);
    }
}

}  // namespace dwkv
