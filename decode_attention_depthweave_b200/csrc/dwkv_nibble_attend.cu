// dwkv_nibble_attend.cu -- attention over the 4-bit cache.
#include <algorithm>

#include "dwkv_nibble_decode.cuh"

namespace dwkv {

// One warp a (row, query head): the tokens one by one, each lane d / 32 channels.
template <int D, bool FP16>
__global__ void __launch_bounds__(128) nib_attend_simple_kernel(const NibGeom G, const NibAttend A) {
    constexpr int C = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (w >= (long long)A.n_rows * G.hq) return;
    const int row = (int)(w / G.hq), head = (int)(w % G.hq), h = head / G.g;
    int lo = 0, hi = A.n;                                     // the slot with cu[b] <= row < cu[b + 1]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (A.cu[mid + 1] > row) hi = mid; else lo = mid + 1;
    }
    if (lo >= A.n) return;                                    // behind the last row
    int len, nq;
    if (!nib_request(G, A, lo, len, nq) || nq * G.g <= A.rows_hi) return;
    const int pos = len - nq + (row - A.cu[lo]);
    const int first = G.window > 0 ? max(0, pos - G.window + 1) : 0;
    float q[C], o[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const uint16_t b = A.q[(size_t)row * A.q_stride + head * D + lane * C + j];
        q[j] = FP16 ? __half2float(__ushort_as_half(b)) : __uint_as_float((uint32_t)b << 16);
        o[j] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int t = first; t <= pos; ++t) {
        const int id = A.table[(size_t)lo * G.max_blocks + t / G.page];
        if ((unsigned)id >= (unsigned)G.num_pages) {
            if (lane == 0) nib_error(G, 11u, (uint32_t)lo, (uint32_t)id);
            continue;
        }
        const int r = t & 15;
        const uint8_t* blk = A.pool + nib_block_at(G, id, h, t % G.page);
        const int unit = lane * C / 4, sh = (lane * C & 3) * 4;
        float kk[C], vv[C], s = 0.f;
        uint32_t u = *reinterpret_cast<const uint16_t*>(blk + nib_k_off(D, r) + 2 * unit);
        u = (u >> 2) | (u << 14);
        float sc = nib_scale(blk[nib_kscale_off(D, r, unit / 4)]);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            kk[j] = (float)((int)((u >> (sh + 4 * j)) & 15u) - 8) * sc;
            s = fmaf(q[j], kk[j], s);
        }
        u = *reinterpret_cast<const uint16_t*>(blk + nib_v_off(D, r, 2 * unit));
        u = (u >> 2) | (u << 14);
        sc = nib_scale(blk[nib_vscale_off(D, r, unit / 4)]);
#pragma unroll
        for (int j = 0; j < C; ++j) vv[j] = (float)((int)((u >> (sh + 4 * j)) & 15u) - 8) * sc;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
        s *= G.tau;
        const float mn = fmaxf(m, s);
        const float f = m == -INFINITY ? 0.f : __expf(m - mn), p = __expf(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int j = 0; j < C; ++j) o[j] = fmaf(p, vv[j], o[j] * f);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const float v = o[j] * inv;
        A.out[((size_t)row * G.hq + head) * D + lane * C + j] =
            FP16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
    if (A.lse && lane == 0) A.lse[(size_t)row * G.hq + head] = l > 0.f ? m + logf(l) : -INFINITY;
}

// ------------------------------------------------------------------------------ launches
constexpr int kNdRows = 16;                                   // rows x heads that the decode kernels take
constexpr int kMaxSms = 160;

static constexpr size_t kTicketBytes = (size_t)2 * kMaxSms * 4;

size_t nib_attend_bytes(int d) { return kTicketBytes + (size_t)2 * kMaxSms * 16 * (d + 2) * 4; }

template <int D, int R, bool FP16>
static cudaError_t decode_launch(const NibGeom& G, const NibAttend& A, int sms, cudaStream_t s, bool prepare) {
    using L = NdLayout<D, R>;
    auto k = nib_decode_kernel<D, R, R == 4 && FP16, FP16>;
    if (prepare) return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kBytes);
    k<<<std::min(sms, kMaxSms) * L::kCtas, kNdThreads + 32, L::kBytes, s>>>(G, A);
    return cudaGetLastError();
}

// The instantiation for up to `rows` rows x heads a request.
static cudaError_t decode_rows(const NibGeom& G, const NibAttend& A, int rows, int sms, cudaStream_t s, bool prepare) {
#define NIB_PICK(D, F)                                                                          \
    return rows <= 4 ? decode_launch<D, 4, F>(G, A, sms, s, prepare)                      \
         : rows <= 8 ? decode_launch<D, 8, F>(G, A, sms, s, prepare)                     \
                     : decode_launch<D, 16, F>(G, A, sms, s, prepare)
    if (G.d == 128) {
        if (G.fp16) NIB_PICK(128, true);
        NIB_PICK(128, false);
    }
    if (G.fp16) NIB_PICK(64, true);
    NIB_PICK(64, false);
#undef NIB_PICK
}

cudaError_t nib_prepare_attend(const NibGeom& G) {
    cudaError_t e = cudaSuccess;
    for (int rows : {4, 8, 16})
        if (e == cudaSuccess) e = decode_rows(G, NibAttend{}, rows, 0, nullptr, true);
    return e;
}

cudaError_t nib_attend(const NibGeom& G, NibAttend A, int sms, uint8_t* arena, cudaStream_t s) {
    A.tickets = reinterpret_cast<int*>(arena + 256);
    A.records = reinterpret_cast<float*>(arena + 256 + kTicketBytes);
    const long long most = (long long)A.max_q * G.g;          // rows x heads of a request at most
    A.rows_hi = (int)std::min<long long>(most, kNdRows);
    cudaError_t e = decode_rows(G, A, A.rows_hi, sms, s, false);
    if (e != cudaSuccess || most <= kNdRows) return e;
    const unsigned grid = (unsigned)(((long long)A.n_rows * G.hq + 3) / 4);
    if (G.d == 128) {
        if (G.fp16) nib_attend_simple_kernel<128, true><<<grid, 128, 0, s>>>(G, A);
        else nib_attend_simple_kernel<128, false><<<grid, 128, 0, s>>>(G, A);
    } else {
        if (G.fp16) nib_attend_simple_kernel<64, true><<<grid, 128, 0, s>>>(G, A);
        else nib_attend_simple_kernel<64, false><<<grid, 128, 0, s>>>(G, A);
    }
    return cudaGetLastError();
}

}  // namespace dwkv
