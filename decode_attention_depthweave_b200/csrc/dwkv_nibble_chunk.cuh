// dwkv_nibble_chunk.cuh -- attention over the 4-bit cache for many rows a request (prompt chunks):
// above kNdRows rows (query rows x query heads of a kv-head), on the 5th-generation tensor cores.
//
// A (256 rows x 128 tokens) unit at d = 128 is 2048 cycles of tcgen05.mma and as many of exponentials; it
// takes 4800, bounded by the latencies and the issue slots of the softmax and unpacking warps (52 % of the
// issue slots are used; at 96 registers 132 bytes are spilled, at d = 64 84).  A chunk of 2048 rows of 32 heads,
// 8 kv-heads, at 32768 tokens: 1.13 to 1.15 ms, 925 to 940 TFLOP/s (57 to 58 % of a large library matrix
// product's rate).  A CTA's warps:
//   0   MMA: S = Q K^T (from shared memory), O += P V (P from tensor memory).  The warp walks and waits
//       together, one lane issues
//   1   loader: bulk copies of the keys' and the values' half of each 16-token block
//   2   on: softmax, 2 tiles x 8 warps, two threads a row (64 tokens each): maximum, exponentials, sum; P back
//       to tensor memory over S.  While their products run, the warps turn the next units' codes into fp16
//       keys (tile 0's warps, two units ahead) and values (tile 1's, one ahead: the furthest that two
//       buffers of each allow), exact, written as swizzled operand tiles: half a block a warp
// With a thread a row (eight softmax warps) a unit took 5800 cycles: two warps a scheduler, each in its own
// chain of latencies; warps of their own for the unpacking made it no shorter, nor did a warp for the values'
// copies or prefetches into L2.  For items of one tile, both tiles taking turns on its units were faster over
// long contexts and slower over short ones (82 against 59 us at one request of 16384).
//
// Two row tiles of 128 share each unpacked K / V tile and take turns on the tensor cores: while one is in
// its softmax, the other's products run.  (Scores in two pieces of 64 tokens, so that a tile's own products
// run beside its softmax, were slower: with 64 columns a score product took 190 cycles, with 128 70.)
// Tensor memory: S0 S1 O0 O1, all 512 columns at d = 128.
// The maximum may lag 2^8 behind (P carries 2^7, as in the decode kernel): O is rescaled only when
// a row's maximum moves by more.
//
// K and V tiles have one layout, [token][64 channels] rows of 128 bytes, 16-byte chunks xored with
// token % 8: the K-major swizzled layout for K (tokens are N, channels K) and the MN-major one for V
// (channels are N, tokens K).  A word of codes unpacks to channels 0 4 1 5 2 6 3 7 of its eight: the
// queries are stored in that order too, and the outputs are read back from it.
//
// Units of 128 tokens of a (request, kv-head, 256 rows), in flat order, are cut into equal ranges,
// one a CTA, as in the decode kernel; cut items leave records that their last CTA merges.
#pragma once
#include <type_traits>

#include "dwkv_nibble_decode.cuh"

namespace dwkv {

constexpr int kNcRows = 128;                             // of a tile
constexpr int kNcTokens = 128;                           // of a unit
constexpr int kNcBorder = 3;                             // what an item's end costs, in units (queries, epilogue)
constexpr int kNcSoftmax = 512;                          // threads
constexpr int kNcTile = 256;                             // of a tile
constexpr int kNcThreads = kNcSoftmax + 64;
constexpr int kNcBlocks = kNcTokens / kNibBlock;         // of a unit: its keys or values one a warp of a tile
static_assert(kNcBlocks * 32 == kNcTile, "a block a warp");

template <int D>
struct NcLayout {
    static constexpr uint32_t kTile = (uint32_t)kNcTokens * D * 2;                 // a fp16 tile of 128 rows
    static constexpr uint32_t kHalf = (uint32_t)kNcTokens * 128;                   // its 64 channels
    static constexpr uint32_t kBlock = 18u * D;
    static constexpr uint32_t kQ = 0;                                              // [2] tiles
    static constexpr uint32_t kK = 2 * kTile;                                      // [2] stages
    static constexpr uint32_t kV = 4 * kTile;                                      // [2]
    static constexpr uint32_t kRaw = 6 * kTile;                                    // keys' half blocks, values'
    static constexpr uint32_t kBars = kRaw + kNcBlocks * kBlock;
    static constexpr uint32_t kEx = kBars + 512;                                   // [2][2 tiles][2][128] maxima, sums
    static constexpr uint32_t kBytes = kEx + 4096 + 1024;                         // barriers and words; slack to align the tiles
    static constexpr int kRec = 2 * kNcRows * (D + 2);                             // floats of a record
};

// A request's tokens, query rows and 256-row items.
struct NcSpan {
    int len, nq, items;
};
// Item x of a request: first token and units.
__device__ __forceinline__ void nc_item(const NibGeom& G, int len, int nq, int x, int& base, int& units) {
    const int rows = nq * G.g, r0 = 2 * kNcRows * x, r1 = min(rows, r0 + 2 * kNcRows);
    const int hi = len - nq + (r1 - 1) / G.g;
    base = nib_first_seen(G, len - nq + r0 / G.g) & ~15;
    units = max(1, (hi + 1 - base + kNcTokens - 1) / kNcTokens) + kNcBorder;
}
__device__ __forceinline__ NcSpan nc_span(const NibGeom& G, const NibAttend& A, int b) {
    NcSpan s{0, 0, 0};
    if (!nib_request(G, A, b, s.len, s.nq) || s.nq == 0 || s.nq * G.g <= A.rows_lo) { s.nq = 0; return s; }
    s.items = (s.nq * G.g + 2 * kNcRows - 1) / (2 * kNcRows);
    return s;
}
// Units of one kv-head of a request; the warp's lanes share its items.
__device__ __forceinline__ long long nc_units(const NibGeom& G, const NcSpan& s, int lane) {
    long long sum = 0;
    for (int x = lane; x < s.items; x += 32) {
        int base, units;
        nc_item(G, s.len, s.nq, x, base, units);
        sum += units;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    return sum;
}

// The walk over the segments (parts of items) of a CTA's range.
struct NcWalk {
    int b, h, x, unit;
    long long left;
    NcSpan s;
    int base, units;                                     // of the item
    __device__ __forceinline__ int real() const { return units - kNcBorder; }
    __device__ __forceinline__ int count() const { return (int)min(left, (long long)(real() - unit)); }
    __device__ __forceinline__ int step() const { return (int)min(left, (long long)(units - unit)); }
    __device__ __forceinline__ bool next(const NibGeom& G, const NibAttend& A) {
        left -= step();
        if (left <= 0) return false;
        unit = 0;
        if (++x == s.items) {
            x = 0;
            if (++h == G.hkv) {
                h = 0;
                do {
                    if (++b >= A.n) { left = 0; return false; }
                    s = nc_span(G, A, b);
                } while (s.items == 0);
            }
        }
        nc_item(G, s.len, s.nq, x, base, units);
        return true;
    }
};

// Shared-memory matrix descriptor, 128-byte swizzle: its low word holds the address and the leading byte offset
// (each >> 4), its high word the stride between 8-row atoms, version 1 and the layout type 2.
constexpr uint32_t kNcDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t nc_desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr >> 4) & 0x3fffu) | (lbo >> 4) << 16; }
__device__ __forceinline__ uint64_t nc_desc(uint32_t lo) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kNcDescHi));
    return d;
}
__device__ __forceinline__ bool nc_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void nc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void nc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void nc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 32 columns of this lane's row; the values are there after nc_ld_wait().
__device__ __forceinline__ void nc_ld32_issue(uint32_t addr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr));
}
// Ties the values to the wait, so that no use moves before it.
__device__ __forceinline__ void nc_ld_wait(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14])
                 :: "memory");
    asm volatile(""
                 : "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                   "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]),
                   "+f"(v[31])
                 :: "memory");
}
__device__ __forceinline__ void nc_ld32(uint32_t addr, float (&v)[32]) {
    nc_ld32_issue(addr, v);
    nc_ld_wait(v);
}
// a * b + c and a + b on two floats at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ void nc_st32(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
        "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <int D, bool FP16>
__global__ void __launch_bounds__(kNcThreads, 1) nib_chunk_kernel(const NibGeom G, const NibAttend A) {
    using L = NcLayout<D>;
    constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kNcTokens >> 3) << 17) | ((uint32_t)(kNcRows >> 4) << 24);
    constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kNcRows >> 4) << 24);
    constexpr uint32_t kTmS = 0, kTmO = 256;             // columns: S tiles at 0 and 128, O tiles behind
    extern __shared__ uint8_t raw_sm[];
    __shared__ int s_last[2][3];
    __shared__ long long s_sum[kNcThreads / 32];
    __shared__ int s_start[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t sbase = (smem_addr(raw_sm) + 1023u) & ~1023u;
    uint8_t* sm = raw_sm + (sbase - smem_addr(raw_sm));
    // barriers
    const uint32_t bars = sbase + L::kBars;
    auto k_empty = [&](int s) { return bars + 16u + 8u * s; };
    auto v_full = [&](int s) { return bars + 32u + 8u * s; };
    auto v_empty = [&](int s) { return bars + 48u + 8u * s; };
    auto s_full = [&](int t) { return bars + 64u + 8u * t; };
    auto p_ready = [&](int t) { return bars + 80u + 8u * t; };
    auto o_full = [&](int t) { return bars + 96u + 8u * t; };
    auto raw_full = [&](int z) { return bars + 112u + 8u * z; };     // 0 keys, 1 values
    auto raw_empty = [&](int z) { return bars + 128u + 8u * z; };
    const uint32_t q_ready = bars + 144u;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::kBars + 152);
    volatile int* dead = reinterpret_cast<volatile int*>(sm + L::kBars + 156);
    uint8_t* raw_left = sm + L::kBars + 160;             // [2][blocks] tokens of a raw block that exist
    uint8_t* lost_at = sm + L::kBars + 176;              // [8] units: [blocks] 1: not there
    // Bounded wait; once one ran out, every role winds down.
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = global_ns();
        for (uint32_t it = 1;; ++it) {
            if (mbar_try_wait(bar, parity)) return true;
            if ((it & 63u) == 0u && (*dead || global_ns() - t0 > kWaitLimitNs)) {
                if (!*dead) nib_error(G, 6u /*DWKV_DEV_TIMEOUT*/, 0x6e63u, bar - bars);
                *dead = 1;
                return false;
            }
        }
    };
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(k_empty(s), 1u);
            mbar_init(v_full(s), kNcBlocks);
            mbar_init(v_empty(s), 1u);
            mbar_init(s_full(s), 1u);
            mbar_init(p_ready(s), kNcTile / 32);             // an arrival a warp: 256 on one address take their turns
            mbar_init(o_full(s), 1u);
            mbar_init(raw_full(s), kNcBlocks);
            mbar_init(raw_empty(s), kNcBlocks);
        }
        mbar_init(q_ready, kNcSoftmax / 32);
        *dead = 0;
        fence_mbar_init();
    }

    // ---- this CTA's range of units: floor(total c / n) of them before CTA c
    NcWalk w;
    long long total, at;
    int ctas;
    {
        // a warp a run of requests
        constexpr int kWarps = kNcThreads / 32;
        const int per = (A.n + kWarps - 1) / kWarps, b0 = min(A.n, warp * per), b1 = min(A.n, b0 + per);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += nc_units(G, nc_span(G, A, b), lane) * G.hkv;
        if (lane == 0) s_sum[warp] = mine;
        __syncthreads();
        long long before = 0;
        total = 0;
        for (int k = 0; k < kWarps; ++k) {
            if (k == warp) before = total;
            total += s_sum[k];
        }
        if (total == 0) return;
        ctas = (int)min((long long)gridDim.x, total);
        if ((int)blockIdx.x >= ctas) return;
        at = total * blockIdx.x / ctas;
        w.left = total * (blockIdx.x + 1) / ctas - at;
        if (at >= before && at < before + mine) {
            long long u = at - before;
            for (int b = b0; b < b1; ++b) {
                const NcSpan s = nc_span(G, A, b);
                const long long units = nc_units(G, s, lane);
                if (u >= units * G.hkv) {
                    u -= units * G.hkv;
                    continue;
                }
                const int h = (int)(u / units);
                u -= h * units;
                for (int x0 = 0;; x0 += 32) {            // 32 items at a time
                    int base, n = 0;
                    if (x0 + lane < s.items) nc_item(G, s.len, s.nq, x0 + lane, base, n);
                    int pre = n;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int y = __shfl_up_sync(~0u, pre, o);
                        if (lane >= o) pre += y;
                    }
                    const int all = __shfl_sync(~0u, pre, 31);
                    if (u >= all) {
                        u -= all;
                        continue;
                    }
                    if (u >= pre - n && u < pre) {
                        s_start[0] = b;
                        s_start[1] = h;
                        s_start[2] = x0 + lane;
                        s_start[3] = (int)u - (pre - n);
                    }
                    break;
                }
                break;
            }
        }
        __syncthreads();
        w.b = s_start[0];
        w.h = s_start[1];
        w.x = s_start[2];
        w.unit = s_start[3];
        w.s = nc_span(G, A, w.b);
        nc_item(G, w.s.len, w.s.nq, w.x, w.base, w.units);
    }
    const long long at0 = at;
    if (w.unit >= w.real()) {                            // the range starts in the empty units behind an item
        at += w.step();
        if (!w.next(G, A)) return;
    }
    auto cta_of = [&](long long u) { return (int)(((u + 1) * ctas - 1) / total); };
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tmem_slot;

    // units of the range, over all its segments
    int all_units = 0;
    {
        NcWalk c = w;
        do all_units += c.count(); while (c.next(G, A));
    }

    if (warp == 1) {
        // ================= loader: lane x copies the keys' half of block x of a unit, lane 8 + x the values' half, each
        // with a walk of its own
        if (lane < 2 * kNcBlocks) {
            const int z = lane / kNcBlocks, x = lane % kNcBlocks;
            const uint32_t full = raw_full(z), dst = sbase + L::kRaw + (uint32_t)lane * (L::kBlock / 2);
            bool ok = true;
            int t, left_units, end, id = -1;
            const uint8_t* from;                         // of the kv-head in page 0
            auto open = [&]() {
                left_units = w.count();
                t = w.base + w.unit * kNcTokens + kNibBlock * x;
                end = min(w.s.len, w.base + (w.unit + left_units) * kNcTokens);
                from = A.pool + (size_t)w.h * G.per * L::kBlock + z * (L::kBlock / 2);
            };
            auto look = [&]() {
                if (t < end) id = __ldg(A.table + (size_t)w.b * G.max_blocks + (t >> G.page_shift));
            };
            open();
            look();
            for (int n = 0; n < all_units; ++n) {
                if (n > 0 && !wait(raw_empty(z), (uint32_t)(n - 1) & 1u)) { ok = false; break; }
                const bool there = t < end, good = there && (unsigned)id < (unsigned)G.num_pages;
                raw_left[lane] = (uint8_t)(good ? min(kNibBlock, end - t) : 0);
                if (z == 0) lost_at[(n & 7) * kNcBlocks + x] = good ? 0 : 1;
                if (good) {
                    mbar_arrive_expect_tx(full, L::kBlock / 2);
                    bulk_g2s(dst, from + (size_t)id * G.page_bytes + (size_t)((t & (G.page - 1)) >> 4) * L::kBlock, L::kBlock / 2, full);
                } else {
                    mbar_arrive(full);
                    if (there) nib_error(G, 11u /*DWKV_DEV_BAD_PAGE*/, (uint32_t)w.b, (uint32_t)id);
                }
                t += kNcTokens;
                if (--left_units == 0 && w.next(G, A)) open();
                look();
            }
            if (!ok) mbar_wait_for(full, 0u, 10000000ull), mbar_wait_for(full, 1u, 10000000ull);   // what is in flight, within a limit
        }
        __syncwarp();
    } else if (warp == 0) {
        // ================= MMA: the warp walks and waits together, one elected lane issues, so that addresses
        // and descriptors stay in uniform registers
        bool ok = true, any = false;
        uint32_t j = 0, items = 0, done0 = 0, done1 = 0;  // units; segments; units of each tile
        uint32_t q_lo[2], k_lo[2], v_lo[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            q_lo[x] = nc_desc_lo(sbase + L::kQ + x * L::kTile, 16u);
            k_lo[x] = nc_desc_lo(sbase + L::kK + x * L::kTile, 16u);
            v_lo[x] = nc_desc_lo(sbase + L::kV + x * L::kTile, L::kHalf);
        }
        // S of unit jj; O += P V of it (start: O starts)
        auto qk = [&](int t, uint32_t jj) {
            const uint32_t a = t ? q_lo[1] : q_lo[0], b = jj & 1 ? k_lo[1] : k_lo[0], d = tmem + kTmS + t * 128, bar = s_full(t);
            if (nc_elect()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * L::kHalf + (k & 3) * 32u) >> 4;
                    nc_mma_ss(d, nc_desc(a + off), nc_desc(b + off), kIdescS, k ? 1u : 0u);
                }
                nc_commit(bar);
            }
            __syncwarp();
            any = true;
        };
        auto pv = [&](int t, uint32_t jj, bool start) {
            const uint32_t b = jj & 1 ? v_lo[1] : v_lo[0], d = tmem + kTmO + t * D, p = tmem + kTmS + t * 128;
            if (nc_elect()) {
#pragma unroll
                for (int k = 0; k < kNcTokens / 16; ++k)
                    nc_mma_ts(d, p + (k >> 2) * 64 + 8 * (k & 3), nc_desc(b + k * (2048u >> 4)), kIdescO, start && k == 0 ? 0u : 1u);
            }
            __syncwarp();
        };
        auto commit = [&](uint32_t bar) {
            if (nc_elect()) nc_commit(bar);
            __syncwarp();
        };
        auto after = [&](bool got) {
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            return got;
        };
        for (bool some = true; ok && some; some = w.next(G, A), ++items) {
            const int cnt = w.count(), tiles = w.s.nq * G.g - 2 * kNcRows * w.x > kNcRows ? 2 : 1;
            ok = __all_sync(~0u, wait(q_ready, items & 1u));   // tile 0's warps wrote the first unit's keys before
            if (!after(ok)) break;
            qk(0, j);
            if (tiles > 1) qk(1, j);
            commit(k_empty(j & 1));
            for (int u = 0; ok && u < cnt; ++u, ++j) {
                // a tile's weights are there: its values' product, and the next unit's scores
                auto turn = [&](int t, uint32_t& done) {
                    if (t == 0) ok = wait(v_full(j & 1), (j >> 1) & 1u);
                    ok = __all_sync(~0u, ok && wait(p_ready(t), done & 1u));
                    ++done;
                    if (!after(ok)) return;
                    pv(t, j, u == 0);
                    if (u + 1 == cnt) {
                        commit(o_full(t));
                    } else {
                        qk(t, j + 1);                    // its keys are there: tile 0's warps wrote them before these weights
                    }
                };
                turn(0, done0);
                if (ok && tiles > 1) turn(1, done1);
                if (!ok) break;
                commit(v_empty(j & 1));
                if (u + 1 < cnt) commit(k_empty((j + 1) & 1));
            }
        }
        if (!ok && any) {                                // the products in flight end first, within a limit
            commit(s_full(0));
            mbar_wait_for(s_full(0), j & 1u, 10000000ull);
        }
        __syncwarp();
    } else {
        // ================= softmax: two threads a row of tile t
        // A wait that ran out leaves ok false: the loops run to their end without waiting or issuing, so
        // that every thread meets the others at the barriers.
        const int sw = warp - 2, t = sw >> 3, hc = (sw >> 2) & 1;    // tile, its tokens' (and O's channels') half
        const int r = (warp & 3) * 32 + lane;                        // row: a warp reaches the tensor-memory lanes of its number mod 4
        const bool leader = (sw & 7) == 0 && lane == 0;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;           // this warp's tensor-memory lanes (32 of 128, bits 16 up)
        const uint32_t s_at = tmem + lanes + kTmS + t * 128 + hc * 64, o_at = tmem + lanes + kTmO + t * D + hc * (D / 2);
        float* ex = reinterpret_cast<float*>(sm + L::kEx) + t * 2 * kNcRows;       // [2][2 tiles][2 halves][rows]
        uint32_t j = 0, items = 0, units = 0, segs = 0;  // units and segments of this tile, of the CTA
        bool ok = true;
        const uint32_t e8 = reg_const(0x48004800u), eh = reg_const(0x38003800u);
        // This warp's block of unit n, keys (z = 0) or values, into its rows of the operand tile; bytes behind the last
        // token are not to be believed.  Eight lanes take one 32-channel chunk of eight tokens: all stores, and the
        // loads of values, fall in distinct banks.  All loads come before the first store, which the compiler could
        // not know to be elsewhere.
        const int blk_of = sw & (kNcBlocks - 1);
        auto unpack_as = [&](auto zz, uint32_t n) {
            constexpr int z = decltype(zz)::value;
            if (n >= (uint32_t)all_units) return;
            // the products that read this buffer two units ago are done, and the bytes are there
            if (ok && n >= 2) ok = wait(z ? v_empty(n & 1) : k_empty(n & 1), ((n >> 1) - 1) & 1u);
            if (ok) ok = wait(raw_full(z), n & 1u);
            constexpr int kIts = D / 64;
            const uint8_t* blk = sm + L::kRaw + (z * kNcBlocks + blk_of) * (L::kBlock / 2) - z * (L::kBlock / 2);   // as if the whole block were there
            const int left = raw_left[z * kNcBlocks + blk_of];
            uint4 cw[kIts];
            uint32_t s0[kIts], s1[kIts];
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
                const int q = it * 4 + (lane >> 3), tk = (lane & 7) + 8 * (q & 1), c = q >> 1;   // (token half, chunk)
                cw[it] = make_uint4(0, 0, 0, 0);
                s0[it] = s1[it] = 0;
                if (tk < left) {
                    cw[it] = *reinterpret_cast<const uint4*>(blk + (z ? nib_v_off(D, tk, 16 * c) : nib_k_off(D, tk) + 16 * c));
                    s0[it] = blk[z ? nib_vscale_off(D, tk, 2 * c) : nib_kscale_off(D, tk, 2 * c)];
                    s1[it] = blk[z ? nib_vscale_off(D, tk, 2 * c + 1) : nib_kscale_off(D, tk, 2 * c + 1)];
                }
            }
#pragma unroll
            for (int it = 0; it < kIts; ++it) {
                const int q = it * 4 + (lane >> 3), tk = (lane & 7) + 8 * (q & 1), c = q >> 1;
                const uint32_t words[4] = {cw[it].x, cw[it].y, cw[it].z, cw[it].w};
                const uint32_t r0 = 0x00800080u * s0[it], r1 = 0x00800080u * s1[it];
                const uint32_t b00 = hmul2_(r0, kNibB0), b01 = hmul2_(r0, kNibB1), b10 = hmul2_(r1, kNibB0), b11 = hmul2_(r1, kNibB1);
                uint8_t* dst = sm + (z ? L::kV : L::kK) + (n & 1) * L::kTile + (c >> 1) * L::kHalf + (kNibBlock * blk_of + tk) * 128;
                uint32_t o[4][4];
#pragma unroll
                for (int y = 0; y < 4; ++y) nib_unpack(words[y], y < 2 ? r0 : r1, y < 2 ? b00 : b10, y < 2 ? b01 : b11, e8, eh, o[y]);
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    *reinterpret_cast<uint4*>(dst + ((((c & 1) * 4 + y) ^ (tk & 7)) << 4)) = make_uint4(o[y][0], o[y][1], o[y][2], o[y][3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0 && ok) {
                mbar_arrive(raw_empty(z));
                if (z) mbar_arrive(v_full(n & 1));       // keys: the weights or queries that follow say it
            }
        };
        // what the tile's warps prepare after unit n: keys two units ahead, or values one
        auto unpack = [&](uint32_t n) {
            if (t == 0) unpack_as(std::integral_constant<int, 0>{}, n + 2);
            else unpack_as(std::integral_constant<int, 1>{}, n + 1);
        };
        if (t == 0) unpack_as(std::integral_constant<int, 0>{}, 0);
        unpack(0u - 1u);
        for (bool some = true; some; some = w.next(G, A)) {
            const int cnt = w.count(), rows = w.s.nq * G.g, row = 2 * kNcRows * w.x + kNcRows * t + r;
            const int tiles = rows - 2 * kNcRows * w.x > kNcRows ? 2 : 1;
            if (t >= tiles) {                            // no such tile; the queries' barrier counts all the same
                if (lane == 0) mbar_arrive(q_ready);
                for (int u = 0; u < cnt; ++u, ++units) {
                    unpack(units);
                }
                at += w.step();
                // the next arrival belongs to the next segment: not before this one has begun
                if (ok) ok = wait(q_ready, segs & 1u);
                ++segs;
                continue;
            }
            const int row0 = A.cu[w.b];
            const bool have = row < rows;
            const int jq = have ? row / G.g : 0, hg = have ? row - jq * G.g : 0;
            // ---- the query row, as nib_query_scale says; half a row a thread
            float fac;
            {
                const uint16_t* qp = A.q + (size_t)(row0 + jq) * A.q_stride + (size_t)(w.h * G.g + hg) * D + hc * (D / 2);
                uint4 v[D / 16];
                float a = 0.f;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) v[c] = have ? *reinterpret_cast<const uint4*>(qp + 8 * c) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    const uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        a = fmaxf(a, fabsf(FP16 ? half_lo(x[y]) : bf16lo(x[y])));
                        a = fmaxf(a, fabsf(FP16 ? half_hi(x[y]) : bf16hi(x[y])));
                    }
                }
                float* place = ex + (~units & 1u) * 4 * kNcRows;         // not where the last segment left its sums
                place[hc * kNcRows + r] = a;
                named_barrier(1 + t, kNcTile);
                a = fmaxf(a, place[(hc ^ 1) * kNcRows + r]);
                const float sc = nib_query_scale(G, a, fac);
                uint8_t* dst = sm + L::kQ + t * L::kTile + r * 128;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    const uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
                    const int c8 = hc * (D / 16) + c;
                    float f[8];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        f[2 * y] = (FP16 ? half_lo(x[y]) : bf16lo(x[y])) * sc;
                        f[2 * y + 1] = (FP16 ? half_hi(x[y]) : bf16hi(x[y])) * sc;
                    }
                    *reinterpret_cast<uint4*>(dst + (c8 >> 3) * L::kHalf + (((c8 & 7) ^ (r & 7)) << 4)) =
                        make_uint4(pack_half2(f[0], f[4]), pack_half2(f[1], f[5]), pack_half2(f[2], f[6]), pack_half2(f[3], f[7]));
                }
                fence_async_smem();
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready);         // the tile's queries are there, its O is read
            ++segs;
            const int hi = have ? w.s.len - w.s.nq + jq : -1;        // last token the row sees
            // the tile's rows see all of a unit within [all_lo, all_hi]
            const int tr0 = 2 * kNcRows * w.x + kNcRows * t, tr1 = min(rows, tr0 + kNcRows) - 1;
            const int all_hi = w.s.len - w.s.nq + tr0 / G.g;
            const int all_lo = G.window > 0 ? w.s.len - w.s.nq + max(tr1, 0) / G.g - G.window + 1 : 0;
            // a bit for each of the 32 tokens from t on: seen by this row and there (gone: a bit a block that is not)
            auto seen_of = [&](int tok, uint32_t gone) {
                const int n = hi - tok;                              // the last one seen
                uint32_t bits = n >= 31 ? ~0u : n < 0 ? 0u : (2u << n) - 1u;
                if (G.window > 0) {
                    const int f = n - G.window + 1;                  // the first one seen
                    bits &= f <= 0 ? ~0u : f > 31 ? 0u : ~0u << f;
                }
                return bits & ~((gone & 1u ? 0xffffu : 0u) | (gone & 2u ? 0xffff0000u : 0u));
            };
            float m = kNdNone, l = 0.f;
            for (int u = 0; u < cnt; ++u, ++j, ++units) {
                if (ok) ok = wait(s_full(t), j & 1u);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const int t0 = w.base + (w.unit + u) * kNcTokens;
                const uint2 lost = *reinterpret_cast<const uint2*>(lost_at + (units & 7u) * kNcBlocks);   // a byte a block
                const bool part = t0 + kNcTokens - 1 > all_hi || t0 < all_lo || (lost.x | lost.y);
                // the half's tokens that this row sees
                uint32_t seen[2] = {~0u, ~0u};
                if (part) {
                    const uint32_t gone = hc ? lost.y : lost.x;
#pragma unroll
                    for (int c = 0; c < 2; ++c) seen[c] = seen_of(t0 + 64 * hc + 32 * c, (gone >> (16 * c) & 1u) | (gone >> (16 * c + 8) & 1u) << 1);
                }
                auto mask = [&](float (&x)[32], int c) {
                    if (part) {
                        asm volatile("" ::: "memory");
#pragma unroll
                        for (int y = 0; y < 32; ++y) x[y] = (seen[c] >> y) & 1u ? x[y] : -INFINITY;
                    }
                };
                uint32_t pk[32];
                float sum, top;
                float zf = fac, zc = kNdBias - m;        // a weight's logarithm is zf s + zc
                for (bool again = false;;) {             // a second time when the maximum moves
                    const float2 c0 = make_float2(zc, zc), f2 = make_float2(zf, zf);
                    float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float x[32];
                        nc_ld32(s_at + 32 * c, x);
                        mask(x, c);
                        float tops[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int y = 0; y < 32; y += 2) {
                            tops[(y >> 1) & 1] = fmaxf(tops[(y >> 1) & 1], fmaxf(x[y], x[y + 1]));
                            const float2 z = fma2(make_float2(x[y], x[y + 1]), f2, c0);
                            const float2 p = make_float2(ex2(z.x), ex2(z.y));
                            sums[(y >> 1) & 1] = add2(sums[(y >> 1) & 1], p);
                            pk[16 * c + y / 2] = pack_half2(p.x, p.y);
                        }
                        top = fmaxf(top, fmaxf(tops[0], tops[1]));
                    }
                    const float2 sa = add2(sums[0], sums[1]);
                    sum = sa.x + sa.y;
                    if (again) break;
                    // the row's maximum over both halves; two places in turn, so that one barrier a unit will do
                    float* place = ex + (units & 1u) * 4 * kNcRows;
                    place[hc * kNcRows + r] = top;
                    named_barrier(1 + t, kNcTile);
                    top = fmaxf(top, place[(hc ^ 1) * kNcRows + r]);
                    const float mx = top > -INFINITY ? top * fac : kNdNone;
                    if (!__any_sync(~0u, mx > m + kNdLag || nib_far(m))) break;
                    again = true;
                    const float mn = fmaxf(m, mx), f = ex2(m - mn);
                    m = mn;
                    l *= f;
                    zc = kNdBias - m;
                    if (__any_sync(~0u, nib_far(m))) {   // rounded scores in place of far rows' ones
                        const float by = nib_far(m) ? fac : 1.f;
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            float x[32];
                            nc_ld32(s_at + 32 * c, x);
                            uint32_t xu[32];
#pragma unroll
                            for (int y = 0; y < 32; ++y) xu[y] = __float_as_uint(x[y] * by);
                            nc_st32(s_at + 32 * c, xu);
                        }
                        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                        if (nib_far(m)) zf = 1.f;
                    }
                    if (u > 0) {                         // O holds the units before: these scores came after their products
#pragma unroll 1
                        for (int c = 0; c < D / 64; ++c) {
                            float o[32];
                            nc_ld32(o_at + 32 * c, o);
                            uint32_t ou[32];
#pragma unroll
                            for (int y = 0; y < 32; ++y) ou[y] = __float_as_uint(o[y] * f);
                            nc_st32(o_at + 32 * c, ou);
                        }
                    }
                }
                l += sum;
                nc_st32(s_at, pk);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready(t));
                unpack(units);
            }
            // ---- the segment ends
            if (ok) ok = wait(o_full(t), items & 1u);
            ++items;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            // the row's sum, over both halves (the places that the last unit's maxima did not use)
            {
                float* place = ex + (units & 1u) * 4 * kNcRows;
                place[hc * kNcRows + r] = l;
                named_barrier(1 + t, kNcTile);
                l += place[(hc ^ 1) * kNcRows + r];
            }
            const bool whole = w.unit == 0 && cnt == w.real();
            const long long first = at - w.unit;
            const size_t out_at = (size_t)(row0 + jq) * G.hq + (size_t)(w.h * G.g + hg);
            // eight channels from their stored order, normalised
            auto put8 = [&](int c8, const float* v, float inv) {
                uint32_t x[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    // channel 2 y, 2 y + 1 of the eight: stored at 2 (c % 4) + c / 4
                    const float a = v[(2 * y & 3) * 2 + (2 * y >> 2)] * inv, b = v[((2 * y + 1) & 3) * 2 + ((2 * y + 1) >> 2)] * inv;
                    if (FP16) {
                        x[y] = pack_half2(a, b);
                    } else {
                        const __nv_bfloat162 z = __floats2bfloat162_rn(a, b);
                        x[y] = *reinterpret_cast<const uint32_t*>(&z);
                    }
                }
                *reinterpret_cast<uint4*>(A.out + out_at * D + 8 * c8) = make_uint4(x[0], x[1], x[2], x[3]);
            };
            auto put_lse = [&](float m_, float l_) {
                if (A.lse) A.lse[out_at] = l_ == 0.f ? -INFINITY : (m_ - kNdBias + log2f(l_)) * 0.6931471805599453f;
            };
            {
                float* rec = A.records + (size_t)(2 * blockIdx.x + (at == at0 ? 0 : 1)) * L::kRec + (size_t)t * kNcRows * (D + 2);
                const float inv = l == 0.f ? 0.f : 32.f / l;
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    const int c32 = hc * (D / 64) + c;   // 32 channels
                    float v[32];
                    nc_ld32(o_at + 32 * c, v);
                    if (whole) {
                        if (have) {
#pragma unroll
                            for (int y = 0; y < 4; ++y) put8(4 * c32 + y, v + 8 * y, inv);
                        }
                    } else {                             // [m][l][D / 4] of 128 rows each: rows side by side
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            *reinterpret_cast<float4*>(rec + 2 * kNcRows + (size_t)((8 * c32 + y) * kNcRows + r) * 4) =
                                make_float4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
                    }
                }
                if (hc == 0) {
                    if (whole) {
                        if (have) put_lse(m, l);
                    } else {
                        rec[r] = m;
                        rec[kNcRows + r] = l;
                    }
                }
            }
            if (!whole) {                                // the last CTA of this item merges the records
                named_barrier(1 + t, kNcTile);
                if (leader) {                            // the barrier, then one fence: the whole tile's record is out
                    __threadfence();
                    const int c0 = cta_of(first), c1 = cta_of(first + w.real() - 1);
                    const int k = atomicAdd(A.tickets + 2 * c0 + t, 1);
                    s_last[t][0] = k == c1 - c0;
                    s_last[t][1] = c0;
                    s_last[t][2] = c1;
                    if (k == c1 - c0) A.tickets[2 * c0 + t] = 0;
                    __threadfence();
                }
                named_barrier(1 + t, kNcTile);
                if (s_last[t][0] && have) {
                    const int c0 = s_last[t][1], c1 = s_last[t][2];
                    const int slot0 = first == total * c0 / ctas ? 0 : 1;
                    auto record = [&](int c) {
                        return A.records + (size_t)(2 * c + (c == c0 ? slot0 : 0)) * L::kRec + (size_t)t * kNcRows * (D + 2);
                    };
                    float mm = kNdNone, ll = 0.f;
                    for (int c = c0; c <= c1; ++c) mm = fmaxf(mm, __ldcg(record(c) + r));
                    for (int c = c0; c <= c1; ++c) ll = fmaf(ex2(__ldcg(record(c) + r) - mm), __ldcg(record(c) + kNcRows + r), ll);
                    const float inv = ll == 0.f ? 0.f : 32.f / ll;
#pragma unroll 1
                    for (int q = hc * (D / 32); q < (hc + 1) * (D / 32); ++q) {
                        float v[16];
#pragma unroll
                        for (int y = 0; y < 16; ++y) v[y] = 0.f;
#pragma unroll 2
                        for (int c = c0; c <= c1; ++c) {
                            const float* x = record(c);
                            const float f = ex2(__ldcg(x + r) - mm);
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float4 z = __ldcg(reinterpret_cast<const float4*>(x + 2 * kNcRows + (size_t)((4 * q + y) * kNcRows + r) * 4));
                                v[4 * y] = fmaf(f, z.x, v[4 * y]);
                                v[4 * y + 1] = fmaf(f, z.y, v[4 * y + 1]);
                                v[4 * y + 2] = fmaf(f, z.z, v[4 * y + 2]);
                                v[4 * y + 3] = fmaf(f, z.w, v[4 * y + 3]);
                            }
                        }
                        put8(2 * q, v, inv);
                        put8(2 * q + 1, v + 8, inv);
                    }
                    if (hc == 0) put_lse(mm, ll);
                }
                named_barrier(1 + t, kNcTile);           // s_last is read
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            at += w.step();
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 0) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace dwkv
