// dwkv_nibble_attend.cu -- attention over the 4-bit cache.
#include <algorithm>

#include "dwkv_nibble_chunk.cuh"
#include "dwkv_nibble_decode.cuh"

namespace dwkv {

// ------------------------------------------------------------------------------ launches
// Rows x heads a request that the decode kernels take.  24 requests of 12000 tokens, d 128, 8 kv-heads:
// 4 and 8 rows 90 us, 16 rows 127, 17 to 32 rows 247 to 257; the chunk kernel, which does 128 rows' work for
// one, takes 297 to 308 up to 128 rows, and 353 for 256.  One request of 16384: 32 rows 52 us, in the chunk kernel 58.
constexpr int kNdRows = 32;
// The chunk kernel's records, two of 256 rows a CTA, are the larger ones (43 MB at d 128, 22 MB at 64; the
// decode kernels' take 1.3 to 4.9 MB); the launches of a call run one after the other and share them.
size_t nib_attend_bytes(int d) { return (size_t)2 * kNibMaxSms * 2 * kNcRows * (d + 2) * 4; }

template <int D, int R, bool FP16>
static cudaError_t decode_launch(const NibGeom& G, const NibAttend& A, int sms, cudaStream_t s, bool prepare) {
    using L = NdLayout<D, R>;
    auto k = nib_decode_kernel<D, R, R == 4 && FP16, FP16>;
    if (prepare) return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kBytes);
    k<<<std::min(sms, kNibMaxSms) * L::kCtas, kNdThreads + 32, L::kBytes, s>>>(G, A);
    return cudaGetLastError();
}

// The instantiation for up to `rows` rows x heads a request.
static cudaError_t decode_rows(const NibGeom& G, const NibAttend& A, int rows, int sms, cudaStream_t s, bool prepare) {
#define NIB_PICK(D, F)                                                                          \
    return rows <= 4 ? decode_launch<D, 4, F>(G, A, sms, s, prepare)                      \
         : rows <= 8 ? decode_launch<D, 8, F>(G, A, sms, s, prepare)                     \
         : rows <= 16 ? decode_launch<D, 16, F>(G, A, sms, s, prepare)                   \
                      : decode_launch<D, 32, F>(G, A, sms, s, prepare)
    if (G.d == 128) {
        if (G.fp16) NIB_PICK(128, true);
        NIB_PICK(128, false);
    }
    if (G.fp16) NIB_PICK(64, true);
    NIB_PICK(64, false);
#undef NIB_PICK
}

template <int D, bool FP16>
static cudaError_t chunk_launch(const NibGeom& G, const NibAttend& A, int sms, cudaStream_t s, bool prepare) {
    using L = NcLayout<D>;
    auto k = nib_chunk_kernel<D, FP16>;
    if (prepare) return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::kBytes);
    k<<<std::min(sms, kNibMaxSms), kNcThreads, L::kBytes, s>>>(G, A);
    return cudaGetLastError();
}

static cudaError_t chunk_rows(const NibGeom& G, const NibAttend& A, int sms, cudaStream_t s, bool prepare) {
    if (G.d == 128) return G.fp16 ? chunk_launch<128, true>(G, A, sms, s, prepare) : chunk_launch<128, false>(G, A, sms, s, prepare);
    return G.fp16 ? chunk_launch<64, true>(G, A, sms, s, prepare) : chunk_launch<64, false>(G, A, sms, s, prepare);
}

cudaError_t nib_prepare_attend(const NibGeom& G) {
    cudaError_t e = chunk_rows(G, NibAttend{}, 0, nullptr, true);
    for (int rows : {4, 8, 16, 32})
        if (e == cudaSuccess) e = decode_rows(G, NibAttend{}, rows, 0, nullptr, true);
    return e;
}

cudaError_t nib_attend(const NibGeom& G, NibAttend A, int sms, uint8_t* arena, cudaStream_t s) {
    A.tickets = reinterpret_cast<int*>(arena + kNibTickets);
    A.records = reinterpret_cast<float*>(arena + kNibRecords);
    const long long most = (long long)A.max_q * G.g;          // rows x heads of a request at most
    A.rows_hi = (int)std::min<long long>(most, kNdRows);
    if (most <= kNdRows) return decode_rows(G, A, A.rows_hi, sms, s, false);
    // Of a batch with longer requests, those of one query row (and what else fits that instantiation) go to the
    // decode kernel, the others to the chunk kernel; a request alone needs one launch only.
    cudaError_t e = cudaSuccess;
    if (A.n > 1 && G.g <= kNdRows) {
        A.rows_lo = A.rows_hi = G.g <= 4 ? 4 : G.g <= 8 ? 8 : G.g <= 16 ? 16 : kNdRows;
        e = decode_rows(G, A, A.rows_hi, sms, s, false);
    }
    return e != cudaSuccess ? e : chunk_rows(G, A, sms, s, false);
}

}  // namespace dwkv
