// dwkv_nibble_decode.cuh -- attention over the 4-bit cache for few rows a request: up to 8 NT
// rows (query rows x query heads of a kv-head), the decode and draft-verify steps.
//
// o = sum_t w_t v_t over t, in one pass with a running maximum and sum.  The bytes of the cache
// bound it (144 a token and kv-head at d = 128, each read once), the integer pipe comes next:
// every code passes one LOP3 and half an HFMA2 on its way to the tensor cores.
//
//  - Units of 16 kWarps tokens of a (request, kv-head), in one flat order, are cut into equal
//    contiguous ranges, one a CTA: any mix of lengths loads the SMs evenly, and no host code
//    has to know a length.  A (request, kv-head) cut by a range end leaves records that the last
//    CTA to finish merges (an atomic ticket, no wait).
//  - A warp takes the 16-token blocks w, w + kWarps, ... of a range.  It keeps its own ring of
//    blocks in flight (bulk copies on mbarriers, across request borders), its own maximum, sum and
//    accumulator: warps meet only where a (request, kv-head) ends.
//  - S^T = K Q^T: tokens are the 16 MMA rows, query rows the 8 columns; a lane reads 16 bytes of
//    two tokens' codes and unpacks them to fp16 (exact) in registers.  O^T = V^T P^T: channels are
//    the MMA rows, ldmatrix.trans pairs two tokens' units, P is transposed by movmatrix.
//  - Up to 4 rows, the columns 4-7 hold the same queries again, and P's rounding remainder in the
//    value product: P is then good to 22 bits at no cost.  Beyond, P is fp16 (11 bits), like the
//    output's own rounding or finer.
//  - P carries 2^7: with the maximum allowed to lag 2^8 behind, it stays below 2^15, and weights
//    down to 2^-31 keep a bit.
#pragma once
#include "dwkv_nibble.cuh"

namespace dwkv {

constexpr int kNdWarps = 8;
constexpr int kNdThreads = 32 * kNdWarps;
constexpr int kNdUnit = kNibBlock * kNdWarps;            // tokens of a unit
constexpr float kNdNone = -1e30f;                        // maximum of nothing
constexpr float kNdLag = 8.f, kNdBias = 7.f;             // log2

template <int D, int NT>
struct NdLayout {
    static constexpr int kStages = D == 128 ? (NT == 1 ? 4 : 6) : (NT == 1 ? 8 : 12);
    static constexpr int kCtas = NT == 1 ? 2 : 1;        // an SM
    static constexpr uint32_t kBlock = 18u * D;
    static constexpr int kPitch = D + 4;                 // floats of a merge row: 16-byte accesses of a warp fall in distinct banks
    static constexpr uint32_t kRing = (uint32_t)kNdWarps * kStages * kBlock;
    static constexpr uint32_t kMerge = kRing;                                    // [warps][8][kPitch] fp32
    static constexpr uint32_t kMl = kMerge + (uint32_t)kNdWarps * 8 * kPitch * 4;   // m [warps][8 NT], l [warps][8 NT]
    static constexpr uint32_t kBars = kMl + (uint32_t)kNdWarps * 8 * NT * 8;
    static constexpr uint32_t kScan = kBars + (uint32_t)kNdWarps * kStages * 8;     // scan scratch, 128 bytes
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
__device__ __forceinline__ void nib_unpack(uint32_t u, uint32_t r, uint32_t b0, uint32_t b1, uint32_t (&o)[4]) {
    const uint32_t w = __byte_perm(u, 0, 0x2301);
    o[0] = hfma2_(lop_and_or(u, 0x003c003cu, 0x48004800u), r, b0);
    o[1] = hfma2_(lop_and_or(u, 0x03c003c0u, 0x38003800u), r, b1);
    o[2] = hfma2_(lop_and_or(w, 0x003c003cu, 0x48004800u), r, b0);
    o[3] = hfma2_(lop_and_or(w, 0x03c003c0u, 0x38003800u), r, b1);
}
constexpr uint32_t kNibB0 = 0xc820c820u, kNibB1 = 0xba00ba00u;      // -8.25, -0.75 as fp16 pairs
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

// Where a request's tokens start and how many units they are (none where it has no rows).
struct NdSpan {
    int len, nq, base, units;
};
__device__ __forceinline__ NdSpan nd_span(const NibGeom& G, const NibAttend& A, int b) {
    NdSpan s{0, 0, 0, 0};
    if (b >= A.n) return s;
    if (!nib_request(G, A, b, s.len, s.nq) || s.nq == 0 || s.nq * G.g > A.rows_hi) { s.nq = 0; return s; }
    s.base = G.window > 0 ? max(0, s.len - s.nq - G.window + 1) & ~15 : 0;
    s.units = max(1, (s.len - s.base + kNdUnit - 1) / kNdUnit);
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
    __device__ __forceinline__ int count() const { return min(left, units - unit); }   // units of this segment
    // To the next segment; false at the end of the range.
    __device__ __forceinline__ bool next(const NibGeom& G, const NibAttend& A, int lane) {
        left -= count();
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

// One record of a cut (request, kv-head): [rows] m, [rows] l, [rows][D] unnormalised o.
template <int D>
__host__ __device__ constexpr int nd_record_floats(int rows) { return rows * (D + 2); }

template <int D, int NT, bool SPLIT, bool FP16>
__global__ void __launch_bounds__(kNdThreads, NdLayout<D, NT>::kCtas) nib_decode_kernel(const NibGeom G, const NibAttend A) {
    using L = NdLayout<D, NT>;
    constexpr int R = SPLIT ? 4 : 8 * NT;                // rows of a request at most
    constexpr int kKs = D / 16, kWords = D / 32, kChunks = D / 32;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, i = lane & 3;
    const uint32_t sbase = smem_addr(sm);
    const uint32_t ring = sbase + (uint32_t)warp * L::kStages * L::kBlock;
    const uint32_t bars = sbase + L::kBars + (uint32_t)warp * L::kStages * 8;
    if (lane < L::kStages) mbar_init(bars + 8u * lane, 1u);
    fence_mbar_init();
    __syncwarp();

    // ---- this CTA's range of units
    NdWalk w;
    long long total, at0;                                // units of the call; the range's first
    {
        long long* red = reinterpret_cast<long long*>(sm + L::kScan);
        const int per = (A.n + kNdThreads - 1) / kNdThreads;
        const int b0 = tid * per, b1 = min(A.n, b0 + per);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += (long long)nd_span(G, A, b).units * G.hkv;
        long long pre = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(~0u, pre, o);
            if (lane >= o) pre += x;
        }
        if (lane == 31) red[warp] = pre;
        __syncthreads();
        total = 0;
        long long before = 0;
#pragma unroll
        for (int k = 0; k < kNdWarps; ++k) {
            if (k == warp) before = total;
            total += red[k];
        }
        if (total == 0) return;                          // nothing to do, for every CTA
        const long long n = min((long long)gridDim.x, total);
        if (blockIdx.x >= n) return;
        at0 = total * blockIdx.x / n;
        w.left = (int)(total * (blockIdx.x + 1) / n - at0);
        pre += before - mine;                            // exclusive
        int* start = reinterpret_cast<int*>(red + kNdWarps);
        if (at0 >= pre && at0 < pre + mine) {
            long long at = at0 - pre;
            for (int b = b0; b < b1; ++b) {
                const NdSpan s = nd_span(G, A, b);
                const long long u = (long long)s.units * G.hkv;
                if (at < u) {
                    start[0] = b;
                    start[1] = (int)(at / s.units);
                    start[2] = (int)(at % s.units);
                    break;
                }
                at -= u;
            }
        }
        __syncthreads();
        w.b = start[0];
        w.h = start[1];
        w.unit = start[2];
    }
    w.from = w.b & ~31;
    w.fetch(G, A, lane);
    w.take();
    const long long ctas = min((long long)gridDim.x, total);

    // ---- producer side: the next block to fetch
    NdWalk p = w;
    int p_tok, p_end;                                    // this warp's next block of the segment; its end
    bool p_more = true;
    auto p_open = [&]() {
        p_tok = p.base + p.unit * kNdUnit + 16 * warp;
        p_end = min(p.len, p.base + (p.unit + p.count()) * kNdUnit);
    };
    auto p_find = [&]() {                                // to the first segment with a block left for this warp
        while (p_more && p_tok >= p_end) {
            p_more = p.next(G, A, lane);
            if (p_more) p_open();
        }
    };
    p_open();
    p_find();
    int p_id = 0;                                        // page of the block at p_tok
    auto p_look = [&]() {
        if (p_more) p_id = __ldg(A.table + (size_t)p.b * G.max_blocks + p_tok / G.page);
    };
    p_look();
    int p_stage = 0;
    uint32_t holes = 0;                                  // stages whose block lies in no page
    auto p_issue = [&]() {
        if (!p_more) return;
        const uint32_t bar = bars + 8u * p_stage;
        if ((unsigned)p_id < (unsigned)G.num_pages) {
            holes &= ~(1u << p_stage);
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, L::kBlock);
                bulk_g2s(ring + (uint32_t)p_stage * L::kBlock, A.pool + nib_block_at(G, p_id, p.h, p_tok % G.page), L::kBlock, bar);
            }
        } else {
            holes |= 1u << p_stage;
            if (lane == 0) {
                mbar_arrive(bar);
                nib_error(G, 11u /*DWKV_DEV_BAD_PAGE*/, (uint32_t)p.b, (uint32_t)p_id);
            }
        }
        p_stage = p_stage + 1 == L::kStages ? 0 : p_stage + 1;
        p_tok += kNdUnit;
        p_find();
        p_look();
    };
    for (int s = 0; s < L::kStages; ++s) p_issue();

    // ---- consumer side
    int c_stage = 0;
    uint32_t c_phase = 0;
    bool dead = false;                                   // a wait ran out: leave out what is left
    long long at = at0;
    const uint32_t vrow = (uint32_t)(lane & 7) + (uint32_t)((lane >> 3) & 1) * 8u;
    for (bool more = true; more; more = w.next(G, A, lane)) {
        const int cnt = w.count(), rows = w.nq * G.g;
        const int row0 = A.cu[w.b];
        // queries as B fragments, each row scaled by a power of two to below 2 (exact in fp16)
        uint32_t qf[NT][kKs][2];
        float fac[NT][2];                                // score -> log2 units, for the lane's columns
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
            const uint32_t e = min(max(__float_as_uint(a) >> 23, 1u), 253u);
            const float sc = __uint_as_float((254u - e) << 23);
#pragma unroll
            for (int x = 0; x < kWords; ++x) {
                float f[8];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    f[2 * y] = (FP16 ? half_lo(raw[x][y]) : bf16lo(raw[x][y])) * sc;
                    f[2 * y + 1] = (FP16 ? half_hi(raw[x][y]) : bf16hi(raw[x][y])) * sc;
                }
                qf[nt][2 * x][0] = pack_half2(f[0], f[4]);
                qf[nt][2 * x][1] = pack_half2(f[1], f[5]);
                qf[nt][2 * x + 1][0] = pack_half2(f[2], f[6]);
                qf[nt][2 * x + 1][1] = pack_half2(f[3], f[7]);
            }
            const float mult = G.tau * 1.4426950408889634f * 32.f * __uint_as_float(e << 23);
            fac[nt][0] = __shfl_sync(~0u, mult, 8 * i);
            fac[nt][1] = __shfl_sync(~0u, mult, 8 * i + 4);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = SPLIT ? ((2 * i + c) & 3) : nt * 8 + 2 * i + c;
                pos[nt][c] = w.len - w.nq + min(col, rows - 1) / G.g;
            }
        }
        float m[NT][2], l[NT][2], o[NT][2 * kChunks][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = kNdNone;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int x = 0; x < 2 * kChunks; ++x) o[nt][x][0] = o[nt][x][1] = o[nt][x][2] = o[nt][x][3] = 0.f;
        }
        const int end = min(w.len, w.base + (w.unit + cnt) * kNdUnit);
        const int inner_hi = w.len - w.nq;               // tokens up to here are seen by every row
        const int inner_lo = G.window > 0 ? w.len - G.window : 0;
        for (int t0 = w.base + w.unit * kNdUnit + 16 * warp; t0 < end; t0 += kNdUnit) {
            if (!dead && !mbar_wait(bars + 8u * c_stage, c_phase)) {
                dead = true;
                if (lane == 0) nib_error(G, 6u /*DWKV_DEV_TIMEOUT*/, 0x6e64u, (uint32_t)w.b);
                for (int k = 1; k < L::kStages; ++k) {   // the other copies in flight, each with a limit
                    const int st = (c_stage + k) % L::kStages;
                    mbar_wait_for(bars + 8u * st, c_phase ^ (uint32_t)(c_stage + k >= L::kStages), 10000000ull);
                }
            }
            const uint8_t* blk = sm + (size_t)(warp * L::kStages + c_stage) * L::kBlock;
            const uint32_t blk_s = ring + (uint32_t)c_stage * L::kBlock;
            if (!dead && !((holes >> c_stage) & 1u)) {
                const bool edge = t0 + 15 > inner_hi || t0 < inner_lo;
                // ---- scores of 16 tokens
                uint32_t kw[2][kWords];
                uint32_t ksc[2];
                if (D == 128) {
                    const uint4 a = *reinterpret_cast<const uint4*>(blk + g * 64 + i * 16);
                    const uint4 b = *reinterpret_cast<const uint4*>(blk + (g + 8) * 64 + i * 16);
                    kw[0][0] = a.x; kw[0][1] = a.y; kw[0][kWords - 2] = a.z; kw[0][kWords - 1] = a.w;
                    kw[1][0] = b.x; kw[1][1] = b.y; kw[1][kWords - 2] = b.z; kw[1][kWords - 1] = b.w;
                    ksc[0] = *reinterpret_cast<const uint16_t*>(blk + 8 * D + g * 8 + 2 * i);
                    ksc[1] = *reinterpret_cast<const uint16_t*>(blk + 8 * D + (g + 8) * 8 + 2 * i);
                } else {
                    const uint2 a = *reinterpret_cast<const uint2*>(blk + g * 32 + i * 8);
                    const uint2 b = *reinterpret_cast<const uint2*>(blk + (g + 8) * 32 + i * 8);
                    kw[0][0] = a.x; kw[0][1] = a.y;
                    kw[1][0] = b.x; kw[1][1] = b.y;
                    ksc[0] = blk[8 * D + g * 4 + i];
                    ksc[1] = blk[8 * D + (g + 8) * 4 + i];
                }
                float s[NT][4], s2[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[nt][x] = s2[nt][x] = 0.f;
#pragma unroll
                for (int grp = 0; grp < kWords / 2; ++grp) {     // 16 channels of the lane share a scale
                    uint32_t r[2], b0[2], b1[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        r[z] = __byte_perm(ksc[z], 0, grp ? 0x1414 : 0x0404) >> 1;
                        b0[z] = hmul2_(r[z], kNibB0);
                        b1[z] = hmul2_(r[z], kNibB1);
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int x = 2 * grp + y;
                        uint32_t u0[4], u1[4];
                        nib_unpack(kw[0][x], r[0], b0[0], b1[0], u0);
                        nib_unpack(kw[1][x], r[1], b0[1], b1[1], u1);
                        const uint32_t a0[4] = {u0[0], u1[0], u0[1], u1[1]}, a1[4] = {u0[2], u1[2], u0[3], u1[3]};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(s[nt], a0, qf[nt][2 * x]);
                            mma_f16(s2[nt], a1, qf[nt][2 * x + 1]);
                        }
                    }
                }
                bool jump = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        s[nt][x] = (s[nt][x] + s2[nt][x]) * fac[nt][x & 1];
                        if (edge) {
                            const int t = t0 + g + 8 * (x >> 1), hi = pos[nt][x & 1];
                            if (t > hi || (G.window > 0 && t <= hi - G.window)) s[nt][x] = -INFINITY;
                        }
                        jump |= s[nt][x] > m[nt][x & 1] + kNdLag;
                    }
                }
                if (__any_sync(~0u, jump)) {             // the maximum moves: all rows take the new one
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float x = fmaxf(m[nt][c], fmaxf(s[nt][c], s[nt][c + 2]));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                            const float f = ex2(m[nt][c] - x);
                            m[nt][c] = x;
                            l[nt][c] *= f;
#pragma unroll
                            for (int y = 0; y < 2 * kChunks; ++y) {
                                o[nt][y][c] *= f;
                                o[nt][y][c + 2] *= f;
                            }
                        }
                }
                uint32_t pf[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float pr[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        pr[x] = ex2(s[nt][x] - (m[nt][x & 1] - kNdBias));
                        l[nt][x & 1] += pr[x];
                    }
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        uint32_t h = pack_half2(pr[2 * z], pr[2 * z + 1]);
                        if (SPLIT) {                     // columns 4-7: what the rounding left
                            const uint32_t rest = pack_half2(pr[2 * z] - half_lo(h), pr[2 * z + 1] - half_hi(h));
                            h = i >= 2 ? rest : h;
                        }
                        pf[nt][z] = movm_t(h);
                    }
                }
                // ---- values: O^T += V^T P^T
                uint32_t vs[kChunks];
                if (D == 128) {
                    const uint4 v = *reinterpret_cast<const uint4*>(blk + 17 * D + ((g >> 2) * 4 + i) * 16);
                    vs[0] = v.x; vs[1] = v.y; vs[kChunks - 2] = v.z; vs[kChunks - 1] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2*>(blk + 17 * D + ((g >> 2) * 4 + i) * 8);
                    vs[0] = v.x; vs[1] = v.y;
                }
                if (t0 + 16 > w.len) {                   // bytes behind the last token are not to be believed
                    const int t = t0 + 2 * i;
                    uint32_t keep = 0;
                    if (t < w.len) keep |= 0xffu;
                    if (t + 1 < w.len) keep |= 0xff00u;
                    if (t + 8 < w.len) keep |= 0xff0000u;
                    if (t + 9 < w.len) keep |= 0xff000000u;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) vs[c] &= keep;
                }
#pragma unroll
                for (int c2 = 0; c2 < kChunks; c2 += 2) {
                    uint32_t v[4];
                    const int chunk = nib_vchunk(D, (int)vrow, c2 + (lane >> 4));
                    ldsm_x4_t(blk_s + 9u * D + vrow * (D / 2) + (uint32_t)chunk * 16u, v);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int c = c2 + y;
                        uint32_t u[2][4];
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const uint32_t r = __byte_perm(vs[c], 0, z ? 0x3424 : 0x1404) >> 1;
                            nib_unpack(v[2 * y + z], r, hmul2_(r, kNibB0), hmul2_(r, kNibB1), u[z]);
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
            __syncwarp();                                // the block is read: its stage takes the next one
            c_stage = c_stage + 1 == L::kStages ? 0 : c_stage + 1;
            if (c_stage == 0) c_phase ^= 1u;
            if (!dead) p_issue();
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
                    ml[warp * 8 * NT + nt * 8 + 2 * i + c] = m[nt][c];
                    ml[(kNdWarps + warp) * 8 * NT + nt * 8 + 2 * i + c] = x;
                }
            }
        const bool whole = w.unit == 0 && cnt == w.units;
        const long long first = at - w.unit;             // unit 0 of this (request, kv-head)
        const int c0 = (int)(((first + 1) * ctas - 1) / total), c1 = (int)(((first + w.units) * ctas - 1) / total);
        float* rec = A.records + (size_t)(2 * blockIdx.x + (at == at0 ? 0 : 1)) * nd_record_floats<D>(R);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt) __syncthreads();                     // the merge rows are free again
            if (SPLIT) {                                 // the remainders' products join their rows
#pragma unroll
                for (int y = 0; y < 2 * kChunks; ++y)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[nt][y][x] += __shfl_xor_sync(~0u, o[nt][y][x], 2);
            }
            if (!SPLIT || i < 2) {
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        *reinterpret_cast<float4*>(mo + (size_t)(warp * 8 + 2 * i + y) * L::kPitch + 32 * c + 4 * g) =
                            make_float4(o[nt][2 * c][y], o[nt][2 * c][y + 2], o[nt][2 * c + 1][y], o[nt][2 * c + 1][y + 2]);
            }
            __syncthreads();
            const int r_hi = min(rows - 8 * nt, SPLIT ? 4 : 8);
            for (int e = tid; e < r_hi * (D / 4); e += kNdThreads) {
                const int r = e / (D / 4), ch = e % (D / 4) * 4;
                float mm = kNdNone;
#pragma unroll
                for (int k = 0; k < kNdWarps; ++k) mm = fmaxf(mm, ml[k * 8 * NT + nt * 8 + r]);
                float ll = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kNdWarps; ++k) {
                    const float f = ex2(ml[k * 8 * NT + nt * 8 + r] - mm);
                    const float4 v = *reinterpret_cast<const float4*>(mo + (size_t)(k * 8 + r) * L::kPitch + ch);
                    ll = fmaf(f, ml[(kNdWarps + k) * 8 * NT + nt * 8 + r], ll);
                    acc.x = fmaf(f, v.x, acc.x);
                    acc.y = fmaf(f, v.y, acc.y);
                    acc.z = fmaf(f, v.z, acc.z);
                    acc.w = fmaf(f, v.w, acc.w);
                }
                if (whole) {
                    nib_put<FP16>(G, A, row0, w.h, nt * 8 + r, D, ch, mm, ll, acc);
                } else {
                    const int rr = nt * 8 + r;
                    if (ch == 0) { rec[rr] = mm; rec[R + rr] = ll; }
                    *reinterpret_cast<float4*>(rec + 2 * R + (size_t)rr * D + ch) = acc;
                }
            }
        }
        if (!whole) {                                    // the last CTA of this (request, kv-head) merges the records
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int n = c1 - c0 + 1;
                const int k = atomicAdd(A.tickets + c0, 1);
                s_last = k == n - 1;
                if (s_last) {
                    A.tickets[c0] = 0;
                    __threadfence();
                }
            }
            __syncthreads();
            if (s_last) {
                const int first_slot = first == total * c0 / ctas ? 0 : 1;
                for (int e = tid; e < rows * (D / 4); e += kNdThreads) {
                    const int r = e / (D / 4), ch = e % (D / 4) * 4;
                    float mm = kNdNone;
                    for (int c = c0; c <= c1; ++c)
                        mm = fmaxf(mm, __ldcg(A.records + (size_t)(2 * c + (c == c0 ? first_slot : 0)) * nd_record_floats<D>(R) + r));
                    float ll = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int c = c0; c <= c1; ++c) {
                        const float* x = A.records + (size_t)(2 * c + (c == c0 ? first_slot : 0)) * nd_record_floats<D>(R);
                        const float f = ex2(__ldcg(x + r) - mm);
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(x + 2 * R + (size_t)r * D + ch));
                        ll = fmaf(f, __ldcg(x + R + r), ll);
                        acc.x = fmaf(f, v.x, acc.x);
                        acc.y = fmaf(f, v.y, acc.y);
                        acc.z = fmaf(f, v.z, acc.z);
                        acc.w = fmaf(f, v.w, acc.w);
                    }
                    nib_put<FP16>(G, A, row0, w.h, r, D, ch, mm, ll, acc);
                }
            }
        }
        __syncthreads();                                 // the merge rows are free for the next segment
        at += cnt;
    }
}

}  // namespace dwkv
