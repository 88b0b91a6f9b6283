// dwkv_nibble.cuh -- layout and device helpers of the 4-bit key/value cache (dwkv_nibble_*):
// every channel of every key and value kept, in 4 bits with an 8-bit scale per 16 channels.
//
// Codec, per block of 16 channels x of one vector: s = e5m3(max |x| / 7) (fp16's exponent, 3
// mantissa bits, unsigned: the byte b stands for the fp16 number of bits b << 7), codes
// c = clamp(rint(x / s), -7, 7).  c * s has at most 3 + 4 significant bits, so it is exact in
// fp16 and in bf16: the tensor cores multiply the cache's values themselves, nothing is rounded
// between the stored bytes and the products.
//
// Storage: 16 tokens of one (page, kv-head) are a block of 18 d bytes,
//   key units   [16][d/4]  u16   unit = 4 consecutive channels, (c_j + 8) << 4 j, rotated left by 2
//   key scales  [16][d/16] u8
//   value units [16][d/4]  u16   16-byte chunks of a row permuted (vchunk), so that the 8 rows an
//                                ldmatrix reads fall in distinct banks
//   value scales [2][4][d/32][4] u8   what one lane of an MMA fragment needs, side by side (vscale_off)
// A page of P tokens is [kv-head][P / 16] such blocks: one kv-head's tokens are contiguous.  The
// rotation puts codes 0 and 1 of a unit at bits 2-5 and 6-9 and, after a byte swap, codes 2 and 3
// there: one mask turns them into the mantissa of an fp16 number (unpack_unit2).
#pragma once
#include "dwkv_common.cuh"

namespace dwkv {

constexpr int kNibBlock = 16;                    // tokens of a block
constexpr int kNibMaxSeqs = 8192;                // sequence slots (the table kernel's shared memory)
constexpr float kNibScaleMax = 7680.f;           // largest scale; 7 * 7680 = 53760 the largest value

struct NibGeom {
    int hq, hkv, g, d, page, page_shift, per, num_pages, max_seqs, max_blocks, window, fp16;
    float tau;
    uint32_t blk;                                // bytes of a block
    size_t page_bytes;
    uint32_t* err;
};

__host__ __device__ inline uint32_t nib_block_bytes(int d) { return 18u * (uint32_t)d; }
// Byte offsets within a block.
__host__ __device__ inline uint32_t nib_k_off(int d, int t) { return (uint32_t)t * (uint32_t)(d / 2); }
__host__ __device__ inline uint32_t nib_kscale_off(int d, int t, int grp) {
    return 8u * (uint32_t)d + (uint32_t)t * (uint32_t)(d / 16) + (uint32_t)grp;
}
__host__ __device__ inline int nib_vchunk(int d, int t, int chunk) { return chunk ^ (d == 128 ? (t >> 1) & 3 : (t >> 2) & 1); }
__host__ __device__ inline uint32_t nib_v_off(int d, int t, int byte) {
    return 9u * (uint32_t)d + (uint32_t)t * (uint32_t)(d / 2) + (uint32_t)nib_vchunk(d, t, byte >> 4) * 16u + (uint32_t)(byte & 15);
}
__host__ __device__ inline uint32_t nib_vscale_off(int d, int t, int grp) {
    return 17u * (uint32_t)d +
           (uint32_t)((((grp & 1) * 4 + ((t & 7) >> 1)) * (d / 32) + (grp >> 1)) * 4 + (t & 1) + 2 * (t >> 3));
}

// Where a slot's block starts in the pool, and the slot's row in it.
__host__ __device__ inline size_t nib_block_at(const NibGeom& G, int page, int head, int tok) {
    return (size_t)page * G.page_bytes + ((size_t)head * G.per + (tok >> 4)) * G.blk;
}

// ------------------------------------------------------------------------------ calls
// Tables of a step (dwkv_nibble_tables).
struct NibTables {
    int n, max_rows;
    const int32_t* n_new;
    const int32_t* release;                      // nullable
    const int32_t* len_in;
    int32_t* table;
    int32_t* free_list;
    const int32_t* count_in;
    int32_t* len_out;
    int32_t* count_out;
    int32_t* cu_rows;
    int32_t* positions;                          // nullable
    int32_t* slots;
};

// Rows of keys and values and the slots they go to or come from (append, read).
struct NibRows {
    int n;
    long long k_stride, v_stride;                // elements between rows
    const uint16_t* k;
    const uint16_t* v;
    const int32_t* slots;
    uint8_t* pool;
    uint16_t* k_out;                             // read: [n][hkv][d]
    uint16_t* v_out;
};

// Attention of a step's query rows.
struct NibAttend {
    int n, n_rows, max_q;
    long long q_stride;                          // elements between rows of q
    const uint16_t* q;                           // [n_rows][hq][d]
    const int32_t* cu;                           // [n + 1]
    const int32_t* len;                          // [n]
    const int32_t* table;                        // [n][max_blocks]
    const uint8_t* pool;
    uint16_t* out;                               // [n_rows][hq][d]
    float* lse;                                  // nullable [n_rows][hq]
    int rows_lo, rows_hi;                        // a launch takes requests of rows_lo < rows x heads <= rows_hi
    int* tickets;                                // [CTAs] zero between launches
    float* records;                              // [2 CTAs] parts of requests cut between CTAs
};

cudaError_t nib_prepare_store();
cudaError_t nib_tables(const NibGeom& G, const NibTables& T, cudaStream_t s);
cudaError_t nib_append(const NibGeom& G, const NibRows& R, cudaStream_t s);
cudaError_t nib_read(const NibGeom& G, const NibRows& R, cudaStream_t s);
// The handle's arena: 256 bytes (the error word), the tickets, the records.  kNibMaxSms: CTAs of a launch
// at two an SM need a ticket each, the chunk kernel's one an SM two.
constexpr int kNibMaxSms = 160;
constexpr size_t kNibTickets = 256, kNibRecords = kNibTickets + (size_t)2 * kNibMaxSms * 4;
// Bytes of the records.
size_t nib_attend_bytes(int d);
cudaError_t nib_prepare_attend(const NibGeom& G);
cudaError_t nib_attend(const NibGeom& G, NibAttend A, int sms, uint8_t* arena, cudaStream_t s);

#ifdef __CUDACC__
__device__ __forceinline__ void nib_error(const NibGeom& G, uint32_t code, uint32_t a, uint32_t b) {
    if (atomicCAS(G.err, 0u, code) == 0u) {
        G.err[1] = a;
        G.err[2] = b;
    }
}

// The first token that a row at position p (below 0 where a request has more rows than tokens) sees.
__device__ __forceinline__ int nib_first_seen(const NibGeom& G, int p) {
    return G.window > 0 ? (int)max(0ll, (long long)p - G.window + 1) : 0;
}

// Length and query rows of slot b; false (and the device error word) where they cannot be.
__device__ __forceinline__ bool nib_request(const NibGeom& G, const NibAttend& A, int b, int& len, int& nq) {
    const int c0 = A.cu[b], c1 = A.cu[b + 1];
    len = A.len[b];
    nq = 0;
    if (c0 == c1) return true;                                // idle: nothing to look at
    if (c0 < 0 || c1 < c0 || c1 > A.n_rows || c1 - c0 > A.max_q) {
        nib_error(G, 13u /*DWKV_DEV_BAD_ROWS*/, (uint32_t)b, (uint32_t)c1);
        return false;
    }
    if (len < 0 || len > (long long)G.max_blocks * G.page) {
        nib_error(G, 10u /*DWKV_DEV_BAD_LENGTH*/, (uint32_t)b, (uint32_t)len);
        return false;
    }
    nq = c1 - c0;
    return true;
}

// Four channels of row r (of a kv-head's rows x heads) of a request whose rows start at row0: the
// output (o in units of 1/32, unnormalised against the maximum mm - 7 in log2 units and the sum ll).
template <bool FP16>
__device__ __forceinline__ void nib_put(const NibGeom& G, const NibAttend& A, int row0, int h, int r, int d, int ch, float mm,
                                        float ll, float4 o) {
    const int j = r / G.g;
    const size_t at = (size_t)(row0 + j) * G.hq + (size_t)(h * G.g + r - j * G.g);
    const float inv = ll == 0.f ? 0.f : 32.f / ll;            // a NaN (of the queries) stays one
    uint32_t lo, hi;
    if (FP16) {
        const __half2 a = __floats2half2_rn(o.x * inv, o.y * inv), b = __floats2half2_rn(o.z * inv, o.w * inv);
        lo = *reinterpret_cast<const uint32_t*>(&a);
        hi = *reinterpret_cast<const uint32_t*>(&b);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        lo = *reinterpret_cast<const uint32_t*>(&a);
        hi = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint2*>(A.out + at * d + ch) = make_uint2(lo, hi);
    if (A.lse && ch == 0) A.lse[at] = ll == 0.f ? -INFINITY : (mm - 7.f + log2f(ll)) * 0.6931471805599453f;
}

__device__ __forceinline__ float nib_scale(uint8_t b) { return __half2float(__ushort_as_half((unsigned short)(b << 7))); }
#endif

}  // namespace dwkv
