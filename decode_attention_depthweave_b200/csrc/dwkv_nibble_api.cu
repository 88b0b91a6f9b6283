// dwkv_nibble_api.cu -- host side of the 4-bit key/value cache: argument checks, the handle,
// launches.  Every entry point is documented in include/dwkv.h.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "dwkv.h"
#include "dwkv_nibble.cuh"

namespace dwkv {
void set_last_error(const char* msg);            // dwkv_api.cu: the message dwkv_last_error() returns
}

using namespace dwkv;

struct dwkv_nibble_ctx {
    dwkv_nibble_config cfg;
    NibGeom geom;
    uint8_t* arena;
    int device, num_sms;
};

namespace {

dwkv_status fail(dwkv_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return st;
}

dwkv_status cuda_fail(cudaError_t e, const char* what) {
    return fail(DWKV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

dwkv_status check_cfg(const dwkv_nibble_config* c) {
    if (!c) return fail(DWKV_ERR_INVALID_ARG, "config is NULL");
    if (c->num_kv_heads <= 0 || c->num_q_heads <= 0 || c->num_q_heads % c->num_kv_heads)
        return fail(DWKV_ERR_INVALID_ARG, "num_q_heads (%d) must be a positive multiple of num_kv_heads (%d)",
                    c->num_q_heads, c->num_kv_heads);
    if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
        return fail(DWKV_ERR_INVALID_ARG, "page_tokens must be 16, 32, 64 or 128 (got %d)", c->page_tokens);
    if (c->num_pages <= 0 || (long long)c->num_pages * c->page_tokens >= (1ll << 31))
        return fail(DWKV_ERR_INVALID_ARG, "num_pages (%d) must be positive and hold fewer than 2^31 tokens", c->num_pages);
    if (c->max_seqs <= 0 || c->max_seqs > kNibMaxSeqs)
        return fail(DWKV_ERR_INVALID_ARG, "max_seqs %d out of [1, %d]", c->max_seqs, kNibMaxSeqs);
    if (c->max_blocks <= 0 || (long long)c->max_blocks * c->page_tokens >= (1ll << 30))
        return fail(DWKV_ERR_INVALID_ARG, "max_blocks (%d) must be positive and hold fewer than 2^30 tokens", c->max_blocks);
    if (c->dtype != DWKV_BF16 && c->dtype != DWKV_FP16)
        return fail(DWKV_ERR_INVALID_ARG, "dtype must be DWKV_BF16 or DWKV_FP16 (got %d)", c->dtype);
    if (c->window < 0) return fail(DWKV_ERR_INVALID_ARG, "window %d is negative", c->window);
    if (!std::isfinite(c->softmax_scale)) return fail(DWKV_ERR_INVALID_ARG, "softmax_scale must be finite");
    if (c->head_dim <= 0 || c->head_dim > 256) return fail(DWKV_ERR_INVALID_ARG, "head_dim %d out of range", c->head_dim);
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(DWKV_ERR_UNSUPPORTED, "this build has kernels for head_dim 64 and 128");
    if (c->num_q_heads / c->num_kv_heads > 64)
        return fail(DWKV_ERR_UNSUPPORTED, "this build has kernels for up to 64 query heads per kv head");
    if (c->num_kv_heads > 1024) return fail(DWKV_ERR_UNSUPPORTED, "this build has kernels for up to 1024 kv heads");
    return DWKV_OK;
}

NibGeom make_geom(const dwkv_nibble_config* c) {
    NibGeom G{};
    G.hq = c->num_q_heads;
    G.hkv = c->num_kv_heads;
    G.g = c->num_q_heads / c->num_kv_heads;
    G.d = c->head_dim;
    G.page = c->page_tokens;
    while ((1 << G.page_shift) < c->page_tokens) ++G.page_shift;
    G.per = c->page_tokens / kNibBlock;
    G.num_pages = c->num_pages;
    G.max_seqs = c->max_seqs;
    G.max_blocks = c->max_blocks;
    // A window that holds the longest request hides nothing.  What is left is below 2^30, as lengths are: positions minus
    // a window stay in 32 bits.
    G.window = c->window < (long long)c->max_blocks * c->page_tokens ? c->window : 0;
    G.fp16 = c->dtype == DWKV_FP16;
    G.tau = c->softmax_scale > 0.f ? c->softmax_scale : 1.0f / std::sqrt((float)c->head_dim);
    G.blk = nib_block_bytes(c->head_dim);
    G.page_bytes = (size_t)G.hkv * G.per * G.blk;
    return G;
}

// The handle's device for the length of a call.
struct OnDevice {
    int prev = -1;
    cudaError_t err;
    explicit OnDevice(int dev) {
        err = cudaGetDevice(&prev);
        if (err == cudaSuccess && prev != dev) err = cudaSetDevice(dev);
        else prev = -1;
    }
    ~OnDevice() {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

#define NIB_DEVICE(h)                                                       \
    OnDevice on_((h)->device);                                              \
    if (on_.err != cudaSuccess) return cuda_fail(on_.err, "select the handle's device")

dwkv_status check_handle(dwkv_nibble_handle h) {
    if (!h) return fail(DWKV_ERR_INVALID_ARG, "handle is NULL");
    return DWKV_OK;
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

dwkv_status check_pool(const void* pool) {
    if (!pool) return fail(DWKV_ERR_INVALID_ARG, "pool is NULL");
    if (misaligned(pool, 128)) return fail(DWKV_ERR_INVALID_ARG, "pool must be 128-byte aligned");
    return DWKV_OK;
}

dwkv_status check_rows(const NibGeom& G, int32_t n, const void* k, int64_t ks, const void* v, int64_t vs,
                       const int32_t* slots) {
    if (n < 0) return fail(DWKV_ERR_INVALID_ARG, "n_rows %d is negative", n);
    if (n == 0) return DWKV_OK;
    if (!k || !v || !slots) return fail(DWKV_ERR_INVALID_ARG, "k, v and slots must be non-NULL");
    if (misaligned(k, 16) || misaligned(v, 16)) return fail(DWKV_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
    const int64_t w = (int64_t)G.hkv * G.d;
    if (ks < w || vs < w || ks % 8 || vs % 8)
        return fail(DWKV_ERR_INVALID_ARG, "row strides (%lld, %lld elements) must be multiples of 8 and at least %lld",
                    (long long)ks, (long long)vs, (long long)w);
    return DWKV_OK;
}

size_t arena_need(const dwkv_nibble_config* c) { return kNibRecords + nib_attend_bytes(c->head_dim); }

}  // namespace

extern "C" {

dwkv_status dwkv_nibble_config_check(const dwkv_nibble_config* cfg) { return check_cfg(cfg); }

size_t dwkv_nibble_page_bytes(const dwkv_nibble_config* cfg) {
    if (check_cfg(cfg) != DWKV_OK) return 0;
    return make_geom(cfg).page_bytes;
}

size_t dwkv_nibble_pool_bytes(const dwkv_nibble_config* cfg) {
    if (check_cfg(cfg) != DWKV_OK) return 0;
    return make_geom(cfg).page_bytes * (size_t)cfg->num_pages;
}

size_t dwkv_nibble_arena_bytes(const dwkv_nibble_config* cfg) {
    if (check_cfg(cfg) != DWKV_OK) return 0;
    return arena_need(cfg);
}

dwkv_status dwkv_nibble_create(const dwkv_nibble_config* cfg, void* arena, size_t arena_bytes, void* stream,
                               dwkv_nibble_handle* out) {
    dwkv_status st;
    if (!out) return fail(DWKV_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if ((st = check_cfg(cfg)) != DWKV_OK) return st;
    if (!arena || misaligned(arena, 256)) return fail(DWKV_ERR_INVALID_ARG, "arena must be non-NULL and 256-byte aligned");
    if (arena_bytes < arena_need(cfg))
        return fail(DWKV_ERR_CAPACITY, "arena of %zu bytes is below the %zu needed", arena_bytes, arena_need(cfg));
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    cudaPointerAttributes pa{};
    e = cudaPointerGetAttributes(&pa, arena);
    if (e != cudaSuccess) return cuda_fail(e, "cudaPointerGetAttributes(arena)");
    if (pa.type != cudaMemoryTypeDevice || pa.device != dev)
        return fail(DWKV_ERR_INVALID_ARG, "arena must be device memory of the current device %d", dev);
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = nib_prepare_store();
    if (e == cudaSuccess) e = nib_prepare_attend(make_geom(cfg));
    if (e == cudaSuccess) e = cudaMemsetAsync(arena, 0, arena_need(cfg), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dwkv_nibble_create");
    auto* h = new (std::nothrow) dwkv_nibble_ctx();
    if (!h) return fail(DWKV_ERR_CAPACITY, "out of host memory");
    h->cfg = *cfg;
    h->geom = make_geom(cfg);
    h->arena = static_cast<uint8_t*>(arena);
    h->geom.err = reinterpret_cast<uint32_t*>(h->arena);
    h->device = dev;
    h->num_sms = std::max(1, sms);
    *out = h;
    return DWKV_OK;
}

dwkv_status dwkv_nibble_destroy(dwkv_nibble_handle h) {
    if (!h) return fail(DWKV_ERR_INVALID_ARG, "handle is NULL");
    delete h;
    return DWKV_OK;
}

dwkv_status dwkv_nibble_tables(dwkv_nibble_handle h, int32_t n_seqs, const int32_t* n_new, const int32_t* release,
                               const int32_t* seq_lens, int32_t* block_tables, int32_t* free_list,
                               const int32_t* free_count, int32_t* seq_lens_out, int32_t* free_count_out,
                               int32_t max_rows, int32_t* cu_rows, int32_t* positions, int32_t* slots, void* stream) {
    dwkv_status st;
    if ((st = check_handle(h)) != DWKV_OK) return st;
    if (n_seqs < 0 || n_seqs > h->geom.max_seqs)
        return fail(DWKV_ERR_INVALID_ARG, "n_seqs %d out of [0, %d]", n_seqs, h->geom.max_seqs);
    if (max_rows < 0 || max_rows >= (1 << 30)) return fail(DWKV_ERR_INVALID_ARG, "max_rows %d out of [0, 2^30)", max_rows);
    if (!free_list || !free_count || !free_count_out || !cu_rows)
        return fail(DWKV_ERR_INVALID_ARG, "free_list, free_count, free_count_out and cu_rows must be non-NULL");
    if (n_seqs && (!n_new || !seq_lens || !block_tables || !seq_lens_out))
        return fail(DWKV_ERR_INVALID_ARG, "n_new, seq_lens, block_tables and seq_lens_out must be non-NULL");
    if (max_rows && !slots) return fail(DWKV_ERR_INVALID_ARG, "slots must be non-NULL");
    NIB_DEVICE(h);
    const NibTables T{n_seqs, max_rows, n_new, release, seq_lens, block_tables, free_list, free_count,
                      seq_lens_out, free_count_out, cu_rows, positions, slots};
    const cudaError_t e = nib_tables(h->geom, T, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dwkv_nibble_tables launch");
    return DWKV_OK;
}

dwkv_status dwkv_nibble_append(dwkv_nibble_handle h, int32_t n_rows, const void* k, int64_t k_stride, const void* v,
                               int64_t v_stride, const int32_t* slots, void* pool, void* stream) {
    dwkv_status st;
    if ((st = check_handle(h)) != DWKV_OK) return st;
    if ((st = check_rows(h->geom, n_rows, k, k_stride, v, v_stride, slots)) != DWKV_OK) return st;
    if (n_rows == 0) return DWKV_OK;
    if ((st = check_pool(pool)) != DWKV_OK) return st;
    NIB_DEVICE(h);
    const NibRows R{n_rows, k_stride, v_stride, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), slots,
                    static_cast<uint8_t*>(pool), nullptr, nullptr};
    const cudaError_t e = nib_append(h->geom, R, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dwkv_nibble_append launch");
    return DWKV_OK;
}

dwkv_status dwkv_nibble_read(dwkv_nibble_handle h, int32_t n_rows, const int32_t* slots, const void* pool, void* k_out,
                             void* v_out, void* stream) {
    dwkv_status st;
    if ((st = check_handle(h)) != DWKV_OK) return st;
    const int64_t w = (int64_t)h->geom.hkv * h->geom.d;
    if ((st = check_rows(h->geom, n_rows, k_out, w, v_out, w, slots)) != DWKV_OK) return st;
    if (n_rows == 0) return DWKV_OK;
    if ((st = check_pool(pool)) != DWKV_OK) return st;
    NIB_DEVICE(h);
    const NibRows R{n_rows, w, w, nullptr, nullptr, slots, static_cast<uint8_t*>(const_cast<void*>(pool)),
                    static_cast<uint16_t*>(k_out), static_cast<uint16_t*>(v_out)};
    const cudaError_t e = nib_read(h->geom, R, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dwkv_nibble_read launch");
    return DWKV_OK;
}

dwkv_status dwkv_nibble_attention(dwkv_nibble_handle h, int32_t n_seqs, int32_t n_rows, int32_t max_q, const void* q,
                                  int64_t q_stride, const int32_t* cu_rows, const int32_t* seq_lens,
                                  const int32_t* block_tables, const void* pool, void* out, float* lse, void* stream) {
    dwkv_status st;
    if ((st = check_handle(h)) != DWKV_OK) return st;
    const NibGeom& G = h->geom;
    if (n_seqs < 0 || n_seqs > G.max_seqs)
        return fail(DWKV_ERR_INVALID_ARG, "n_seqs %d out of [0, %d]", n_seqs, G.max_seqs);
    if (n_rows < 0 || max_q < 0) return fail(DWKV_ERR_INVALID_ARG, "n_rows %d or max_q %d is negative", n_rows, max_q);
    if (n_seqs == 0 || n_rows == 0) return DWKV_OK;      // with max_q 0, requests that have rows are still recorded
    if (!q || !cu_rows || !seq_lens || !block_tables || !out)
        return fail(DWKV_ERR_INVALID_ARG, "q, cu_rows, seq_lens, block_tables and out must be non-NULL");
    if (misaligned(q, 16) || misaligned(out, 16)) return fail(DWKV_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
    if (q_stride < (int64_t)G.hq * G.d || q_stride % 8)
        return fail(DWKV_ERR_INVALID_ARG, "q's row stride (%lld elements) must be a multiple of 8 and at least %lld",
                    (long long)q_stride, (long long)G.hq * G.d);
    if ((long long)n_rows * G.hq >= (1ll << 31)) return fail(DWKV_ERR_INVALID_ARG, "n_rows x num_q_heads must be below 2^31");
    if ((st = check_pool(pool)) != DWKV_OK) return st;
    NIB_DEVICE(h);
    const NibAttend A{n_seqs, n_rows, std::min(max_q, n_rows), q_stride, static_cast<const uint16_t*>(q), cu_rows, seq_lens,
                      block_tables, static_cast<const uint8_t*>(pool), static_cast<uint16_t*>(out), lse, 0, 0, nullptr, nullptr};
    const cudaError_t e = nib_attend(G, A, h->num_sms, h->arena, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "dwkv_nibble_attention launch");
    return DWKV_OK;
}

dwkv_status dwkv_nibble_sync_status(dwkv_nibble_handle h, void* stream) {
    dwkv_status st;
    if ((st = check_handle(h)) != DWKV_OK) return st;
    NIB_DEVICE(h);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t w[3] = {0, 0, 0};
    cudaError_t e = cudaMemcpyAsync(w, h->geom.err, sizeof(w), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "read device error word");
    if (w[0] == 0) return DWKV_OK;
    e = cudaMemsetAsync(h->arena, 0, kNibRecords, s);              // the tickets too: a wait that ran out leaves some taken
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "clear device error word");
    const char* nm = "unknown";
    switch (w[0]) {
        case DWKV_DEV_POOL_EXHAUSTED: nm = "no free page left for a request"; break;
        case DWKV_DEV_TIMEOUT: nm = "bounded wait timed out"; break;
        case DWKV_DEV_FREE_LIST: nm = "more pages given back than the pool has"; break;
        case DWKV_DEV_RANGE: nm = "a key or value is NaN, infinite or beyond 53760"; break;
        case DWKV_DEV_BAD_LENGTH: nm = "a length or count is out of range"; break;
        case DWKV_DEV_BAD_PAGE: nm = "a block table names a page outside the pool"; break;
        case DWKV_DEV_BAD_SLOT: nm = "a slot is outside the pool"; break;
        case DWKV_DEV_BAD_ROWS: nm = "a request's rows do not fit the call"; break;
        default: break;
    }
    return fail(DWKV_ERR_DEVICE_CHECK, "device check failed: %s (code %u, info %u, %u)", nm, w[0], w[1], w[2]);
}

}  // extern "C"
