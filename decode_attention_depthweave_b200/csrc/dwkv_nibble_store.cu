// dwkv_nibble_store.cu -- the 4-bit cache's tables (which pages a request holds, where its new
// rows go), append (quantise rows into their slots) and read (the stored values).
#include "dwkv_nibble.cuh"

namespace dwkv {

// ------------------------------------------------------------------------------------
// Tables of a step.  Per slot b: held_b = ceil(len_b / P) pages; a released slot gives its pages
// back (pushed on the free stack in slot order, then block order) and starts from length 0; then
// need_b = ceil((len_b + new_b) / P) - ceil(len_b / P) pages come from the top of the stack, in
// slot order, while the running total of the needs fits.  Row i of slot b gets position
// len_b + i and slot page * P + position % P; rows of a refused request and rows behind the last
// one get -1.
//
// One cluster does it all.  Every CTA makes the three prefix sums (pages given back, pages
// needed, rows) in its own shared memory; pushes, pops and rows are then spread flat over the
// cluster's threads, each finding its request by bisection of a prefix sum, so one long prompt
// costs no more than many short ones.  The only dependency is pops and in-place updates after
// pushes and reads: one cluster barrier.  Bound by latency, a dozen loads and barriers in a row: 9 us
// for 8 requests of a row each, 15 us for 1024 requests.
// ------------------------------------------------------------------------------------
constexpr int kTabThreads = 1024;                 // at most
constexpr int kTabRows = 4;                       // rows in flight a thread
constexpr int kRowCap = 1 << 30;                 // the prefix sums saturate here

// Both operands are in [0, 2^30]: their sum needs 32 bits unsigned.
__device__ __forceinline__ int sat_add(int a, int b) { return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)kRowCap); }

// Largest i in [0, n) with pre[i] <= x (pre ascending, pre[0] <= x).
__device__ __forceinline__ int find_in(const int* pre, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

static size_t nib_tables_smem(int n) { return (size_t)(5 * (n + 1) + 3 * 32) * 4; }

__global__ void __launch_bounds__(kTabThreads) nib_tables_kernel(const NibGeom G, const NibTables T) {
    extern __shared__ int tsm[];
    const int n = T.n, P = G.page, sh = G.page_shift, threads = blockDim.x;
    int* back = tsm;                             // [n + 1] exclusive prefix sums
    int* need = back + n + 1;
    int* rows = need + n + 1;
    int* now = rows + n + 1;                     // [n] length before the new rows
    int* ok = now + n + 1;                       // [n] bit 0 served, bit 1 released
    int* red = ok + n + 1;                       // [3][32] warp sums
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t rank, ncta;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
    const long long most = (long long)G.max_blocks * P;
    const int per = (n + threads - 1) / threads;
    const int b0 = min(n, tid * per), b1 = min(n, b0 + per);
    int sb = 0, sn = 0, sr = 0;
    for (int b = b0; b < b1; ++b) {
        int len = T.len_in[b], nw = T.n_new[b];
        const bool bad = len < 0 || len > most || nw < 0;
        const bool rel = !bad && T.release && T.release[b] != 0;
        int f = rel ? 2 : 0, nd = 0, bk = 0;
        if (bad) {
            nw = 0;
            if (rank == 0) nib_error(G, 10u /*DWKV_DEV_BAD_LENGTH*/, (uint32_t)b, (uint32_t)len);
        } else {
            if (rel) { bk = (len + P - 1) >> sh; len = 0; }
            if ((long long)len + nw > most) {
                f |= 4;                          // longer than a table row: refused, its rows still count
                if (rank == 0) nib_error(G, 10u, (uint32_t)b, (uint32_t)nw);
            } else {
                nd = ((len + nw + P - 1) >> sh) - ((len + P - 1) >> sh);
            }
        }
        now[b] = len;
        ok[b] = f;
        back[b] = bk;
        need[b] = nd;
        rows[b] = nw;
        sb = sat_add(sb, bk);
        sn = sat_add(sn, nd);
        sr = sat_add(sr, min(nw, kRowCap));
    }
    // block-wide exclusive prefixes of (sb, sn, sr)
    int pb = sb, pn = sn, pr = sr;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(~0u, pb, o), y = __shfl_up_sync(~0u, pn, o), z = __shfl_up_sync(~0u, pr, o);
        if (lane >= o) { pb = sat_add(pb, x); pn = sat_add(pn, y); pr = sat_add(pr, z); }
    }
    if (lane == 31) { red[warp] = pb; red[32 + warp] = pn; red[64 + warp] = pr; }
    __syncthreads();
    if (warp == 0) {
        const bool in = lane < threads / 32;
        int x = in ? red[lane] : 0, y = in ? red[32 + lane] : 0, z = in ? red[64 + lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(~0u, x, o), v = __shfl_up_sync(~0u, y, o), w = __shfl_up_sync(~0u, z, o);
            if (lane >= o) { x = sat_add(x, u); y = sat_add(y, v); z = sat_add(z, w); }
        }
        red[lane] = x; red[32 + lane] = y; red[64 + lane] = z;
    }
    __syncthreads();
    {
        // exclusive: what the warps and lanes before this thread hold
        int xb = __shfl_up_sync(~0u, pb, 1), xn = __shfl_up_sync(~0u, pn, 1), xr = __shfl_up_sync(~0u, pr, 1);
        if (lane == 0) xb = xn = xr = 0;
        if (warp) { xb = sat_add(xb, red[warp - 1]); xn = sat_add(xn, red[32 + warp - 1]); xr = sat_add(xr, red[64 + warp - 1]); }
        for (int b = b0; b < b1; ++b) {
            const int vb = back[b], vn = need[b], vr = rows[b];
            back[b] = xb; need[b] = xn; rows[b] = xr;
            xb = sat_add(xb, vb); xn = sat_add(xn, vn); xr = sat_add(xr, min(vr, kRowCap));
        }
        if (tid == 0) { back[n] = red[31]; need[n] = red[63]; rows[n] = red[95]; }
    }
    __syncthreads();
    int count = *T.count_in;
    if (count < 0 || count > G.num_pages) {
        if (rank == 0 && tid == 0) nib_error(G, 10u, 0xffffffffu, (uint32_t)count);
        count = max(0, min(count, G.num_pages));
    }
    const int all_back = back[n];
    const int top = min(count + all_back, G.num_pages);
    if (rank == 0 && tid == 0 && count + all_back > G.num_pages) nib_error(G, 7u /*DWKV_DEV_FREE_LIST*/, (uint32_t)count, (uint32_t)all_back);
    // served: its pages fit and its rows have a place
    for (int b = tid; b < n; b += threads) {
        const int nd = need[b + 1] - need[b];
        int f = ok[b];
        if (!(f & 4)) {
            if (nd > 0 && need[b + 1] > top) {
                if (rank == 0) nib_error(G, 1u /*DWKV_DEV_POOL_EXHAUSTED*/, (uint32_t)b, (uint32_t)nd);
            } else if (rows[b + 1] > T.max_rows) {
                if (rank == 0) nib_error(G, 13u /*DWKV_DEV_BAD_ROWS*/, (uint32_t)b, (uint32_t)rows[b + 1]);
            } else {
                f |= 1;
            }
        }
        ok[b] = f;
    }
    const int gt = (int)rank * threads + tid, gn = (int)ncta * threads;
    // push
    for (int i = gt; i < all_back && count + i < G.num_pages; i += gn) {
        const int b = find_in(back, n, i);
        T.free_list[count + i] = T.table[(size_t)b * G.max_blocks + (i - back[b])];
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    // pop: page j of the running total is free_list[top - 1 - j]
    const int all_need = min(need[n], top);
    for (int i = gt; i < all_need; i += gn) {
        const int b = find_in(need, n, i);
        if (ok[b] & 1) T.table[(size_t)b * G.max_blocks + ((now[b] + P - 1) >> sh) + (i - need[b])] = T.free_list[top - 1 - i];
    }
    // rows, kTabRows in flight a thread: their requests, then their pages, then the stores
    const int all_rows = min(rows[n], T.max_rows);
    for (int r0 = gt; r0 < T.max_rows; r0 += gn * kTabRows) {
        int pos[kTabRows], id[kTabRows];
#pragma unroll
        for (int k = 0; k < kTabRows; ++k) {
            const int r = r0 + k * gn;
            pos[k] = id[k] = -1;
            if (r < all_rows) {
                const int b = find_in(rows, n, r);
                if (ok[b] & 1) {
                    const int at = now[b] + r - rows[b], had = (now[b] + P - 1) >> sh, j = at >> sh;
                    pos[k] = at;
                    id[k] = j < had ? T.table[(size_t)b * G.max_blocks + j] : T.free_list[top - 1 - (need[b] + j - had)];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kTabRows; ++k) {
            const int r = r0 + k * gn;
            if (r >= T.max_rows) break;
            const bool good = (unsigned)id[k] < (unsigned)G.num_pages;
            if (pos[k] >= 0 && !good) nib_error(G, 11u /*DWKV_DEV_BAD_PAGE*/, (uint32_t)r, (uint32_t)id[k]);
            T.slots[r] = good ? (id[k] << sh) + (pos[k] & (P - 1)) : -1;
            if (T.positions) T.positions[r] = pos[k];
        }
    }
    if (rank == 0) {
        int taken = 0;
        for (int b = b0; b < b1; ++b) {
            const int nw = rows[b + 1] - rows[b];
            if (ok[b] & 1) taken += need[b + 1] - need[b];
            // an invalid length is left as it was
            const int before = T.len_in[b];
            const bool bad = before < 0 || before > most;
            T.len_out[b] = bad ? before : now[b] + ((ok[b] & 1) ? nw : 0);
            T.cu_rows[b] = rows[b];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) taken += __shfl_xor_sync(~0u, taken, o);
        if (lane == 0) red[warp] = taken;
        __syncthreads();
        if (tid == 0) {
            int s = 0;
            for (int w = 0; w < threads / 32; ++w) s += red[w];
            *T.count_out = top - s;
            T.cu_rows[n] = rows[n];
        }
    }
}

// ------------------------------------------------------------------------------------
// Append and read: a warp a row of keys or of values, a lane 8 channels of a head (one 16-byte load or
// store), two lanes a block of 16; kAhead heads' loads are issued before the first is used.  16384 rows of 8
// kv-heads, d 128: append 29 us (3 TB/s), bound by issuing the quantiser's instructions (78 % of the slots while
// it runs; both lanes of a block make its scale); read 19 us (4.5 TB/s), by the ALU pipe (79 %) that takes the codes
// apart.  8 rows are a launch's latency, 5 and 4 us.
// ------------------------------------------------------------------------------------
constexpr int kRowWarps = 8;
constexpr int kAhead = 4;

// e5m3 byte of y >= 0 (finite): RNE of y to 4 significant bits (to multiples of 2^-17 below 2^-14).
__device__ __forceinline__ uint32_t e5m3_of(float y) {
    y = fminf(y, kNibScaleMax);
    if (y < 6.103515625e-05f) return (uint32_t)__float2int_rn(y * 131072.f);   // 2^-14; the carry to 8 is 2^-14 itself
    uint32_t u = __float_as_uint(y);
    u = (u + 0x7ffffu + ((u >> 20) & 1u)) >> 20;                              // 8 exponent bits, 3 mantissa bits
    return u - ((127u - 15u) << 3);
}

// The row and slot of a warp; false where there is nothing to do (slot -1: `skip`).
struct NibRow {
    int row, z, slot, tok;
    uint8_t* base;                               // of the slot's block of head 0
};
__device__ __forceinline__ bool nib_row(const NibGeom& G, const NibRows& R, NibRow& x) {
    const long long w = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    x.row = (int)(w >> 1);
    x.z = (int)(w & 1);
    x.slot = -1;
    x.tok = 0;
    x.base = R.pool;
    if (x.row >= R.n) return false;
    x.slot = __ldg(R.slots + x.row);
    if ((unsigned)x.slot >= (unsigned)G.num_pages * (unsigned)G.page) {
        if (x.slot != -1 && (threadIdx.x & 31) == 0) nib_error(G, 12u /*DWKV_DEV_BAD_SLOT*/, (uint32_t)x.row, (uint32_t)x.slot);
        x.slot = -1;
        return true;
    }
    x.tok = x.slot & (G.page - 1);
    x.base = R.pool + nib_block_at(G, x.slot >> G.page_shift, 0, x.tok);
    return true;
}

template <bool FP16>
__device__ __forceinline__ float lo16(uint32_t w) {
    return FP16 ? __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))) : bf16lo(w);
}
template <bool FP16>
__device__ __forceinline__ float hi16(uint32_t w) { return FP16 ? __half2float(__ushort_as_half((unsigned short)(w >> 16))) : bf16hi(w); }
template <bool FP16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if (FP16) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int D, bool FP16>
__global__ void __launch_bounds__(32 * kRowWarps) nib_append_kernel(const NibGeom G, const NibRows R) {
    constexpr int LV = D / 8, HS = 32 / LV;                       // lanes of a vector, heads side by side
    NibRow x;
    if (!nib_row(G, R, x) || x.slot < 0) return;
    const int lane = threadIdx.x & 31, part = lane % LV, t = x.tok & 15;
    const uint16_t* src = (x.z ? R.v + x.row * R.v_stride : R.k + x.row * R.k_stride) + part * 8;
    const uint32_t at = x.z ? nib_v_off(D, t, 4 * part) : nib_k_off(D, t) + 4 * part;
    const uint32_t at_s = x.z ? nib_vscale_off(D, t, part >> 1) : nib_kscale_off(D, t, part >> 1);
    const size_t head_bytes = (size_t)G.per * G.blk;
    for (int h0 = lane / LV; h0 < G.hkv; h0 += HS * kAhead) {
        uint4 in[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            in[k] = h0 + k * HS < G.hkv ? __ldg(reinterpret_cast<const uint4*>(src + (size_t)(h0 + k * HS) * D)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int h = h0 + k * HS;
            const uint32_t ws[4] = {in[k].x, in[k].y, in[k].z, in[k].w};
            // the largest magnitude, two 16-bit values at a time; a NaN makes it NaN
            const uint32_t top2 = max2<FP16>(max2<FP16>(ws[0] & 0x7fff7fffu, ws[1] & 0x7fff7fffu),
                                             max2<FP16>(ws[2] & 0x7fff7fffu, ws[3] & 0x7fff7fffu));
            float f[8], a = fmaxf(lo16<FP16>(top2), hi16<FP16>(top2));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = lo16<FP16>(ws[j]);
                f[2 * j + 1] = hi16<FP16>(ws[j]);
            }
            // NaN, infinite or beyond the largest value (rare): NaN to 0, the rest clamped.  (fmaxf leaves a NaN
            // out: one in either half shows in the other test.)
            if (!(lo16<FP16>(top2) <= 7.f * kNibScaleMax) || !(hi16<FP16>(top2) <= 7.f * kNibScaleMax)) {
                a = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    f[j] = f[j] != f[j] ? 0.f : fminf(fmaxf(f[j], -7.f * kNibScaleMax), 7.f * kNibScaleMax);
                    a = fmaxf(a, fabsf(f[j]));
                }
                nib_error(G, 9u /*DWKV_DEV_RANGE*/, (uint32_t)x.row, (uint32_t)(2 * h + x.z));
            }
            // the two lanes of a block are neighbours, of one head: both are here
            a = fmaxf(a, __shfl_xor_sync(3u << (lane & 30), a, 1));
            if (h >= G.hkv) continue;
            const uint32_t sb = e5m3_of(__fdiv_rn(a, 7.f));
            const float s = nib_scale((uint8_t)sb), r = sb ? __frcp_rn(s) : 0.f;
            // q = f / s rounded once: a product with 1/s and one step by its exact remainder.  At a tie of the codes q
            // is exact, and elsewhere far from one, so that the sum with 1.5 2^23 rounds it as the definition does
            // (ties to even).  All on the floating-point pipe: the integer one bound this kernel (40 us at 16384 rows).
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float q = f[j] * r;
                q = fmaf(fmaf(-q, s, f[j]), r, q);
                f[j] = (q + 12582912.f) - 12582912.f;
            }
            if (sb < 8) {                                         // below 2^-14 s is coarse and the codes may pass 7
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = fminf(fmaxf(f[j], -7.f), 7.f);
            }
            // a unit is a whole number below 2^16: the mantissa of its sum with 2^23
            const float u0 = fmaf(f[3], 4096.f, fmaf(f[2], 256.f, fmaf(f[1], 16.f, f[0] + (8388608.f + 34952.f))));
            const float u1 = fmaf(f[7], 4096.f, fmaf(f[6], 256.f, fmaf(f[5], 16.f, f[4] + (8388608.f + 34952.f))));
            uint32_t u = __byte_perm(__float_as_uint(u0), __float_as_uint(u1), 0x5410);
            // each 16-bit unit rotated left by 2
            u = ((u << 2) & 0xfffcfffcu) | ((u >> 14) & 0x00030003u);
            uint8_t* blk = x.base + h * head_bytes;
            *reinterpret_cast<uint32_t*>(blk + at) = u;
            if (!(part & 1)) blk[at_s] = (uint8_t)sb;
        }
    }
}

// The stored values of the given slots (zeros for -1), in the caller's 16-bit type: exact.
template <int D, bool FP16>
__global__ void __launch_bounds__(32 * kRowWarps) nib_read_kernel(const NibGeom G, const NibRows R) {
    constexpr int LV = D / 8, HS = 32 / LV;
    NibRow x;
    if (!nib_row(G, R, x)) return;
    const int lane = threadIdx.x & 31, part = lane % LV, t = x.tok & 15;
    uint16_t* dst = (x.z ? R.v_out : R.k_out) + (size_t)x.row * G.hkv * D + part * 8;
    const uint32_t at = x.z ? nib_v_off(D, t, 4 * part) : nib_k_off(D, t) + 4 * part;
    const uint32_t at_s = x.z ? nib_vscale_off(D, t, part >> 1) : nib_kscale_off(D, t, part >> 1);
    const size_t head_bytes = (size_t)G.per * G.blk;
    for (int h0 = lane / LV; h0 < G.hkv; h0 += HS * kAhead) {
        uint32_t u[kAhead], sb[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const bool in = x.slot >= 0 && h0 + k * HS < G.hkv;
            const uint8_t* blk = x.base + (h0 + k * HS) * head_bytes;
            u[k] = in ? *reinterpret_cast<const uint32_t*>(blk + at) : 0x22222222u;      // codes 0
            sb[k] = in ? blk[at_s] : 0u;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (h0 + k * HS >= G.hkv) break;
            const float s = nib_scale((uint8_t)sb[k]);
            const uint32_t v = ((u[k] >> 2) & 0x3fff3fffu) | ((u[k] & 0x00030003u) << 14);
            uint32_t o[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float f = x.slot >= 0 ? (float)((int)((v >> (4 * j)) & 15u) - 8) * s : 0.f;
                const uint32_t b = FP16 ? (uint32_t)__half_as_ushort(__float2half_rn(f)) : __float_as_uint(f) >> 16;
                o[j >> 1] |= b << (16 * (j & 1));
            }
            *reinterpret_cast<uint4*>(dst + (size_t)(h0 + k * HS) * D) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

cudaError_t nib_prepare_store() {
    return cudaFuncSetAttribute(nib_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)nib_tables_smem(kNibMaxSeqs));
}

cudaError_t nib_tables(const NibGeom& G, const NibTables& T, cudaStream_t s) {
    cudaLaunchConfig_t c{};
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    // a small step is bound by barriers and loads in a row: few warps; a large one by its rows and pages: 8 CTAs
    const bool large = T.n > 1024 || T.max_rows > 4096;
    const int threads = T.n <= 128 && T.max_rows <= 1024 ? 128 : kTabThreads;
    a.val.clusterDim.x = large ? 8 : 1;
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    c.gridDim = dim3(a.val.clusterDim.x);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = nib_tables_smem(T.n);
    c.stream = s;
    c.attrs = &a;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, nib_tables_kernel, G, T);
}

static unsigned row_grid(const NibRows& R) { return (unsigned)((2ll * R.n + kRowWarps - 1) / kRowWarps); }

cudaError_t nib_append(const NibGeom& G, const NibRows& R, cudaStream_t s) {
    auto k = G.d == 128 ? (G.fp16 ? nib_append_kernel<128, true> : nib_append_kernel<128, false>)
                        : (G.fp16 ? nib_append_kernel<64, true> : nib_append_kernel<64, false>);
    k<<<row_grid(R), 32 * kRowWarps, 0, s>>>(G, R);
    return cudaGetLastError();
}

cudaError_t nib_read(const NibGeom& G, const NibRows& R, cudaStream_t s) {
    auto k = G.d == 128 ? (G.fp16 ? nib_read_kernel<128, true> : nib_read_kernel<128, false>)
                        : (G.fp16 ? nib_read_kernel<64, true> : nib_read_kernel<64, false>);
    k<<<row_grid(R), 32 * kRowWarps, 0, s>>>(G, R);
    return cudaGetLastError();
}

}  // namespace dwkv
