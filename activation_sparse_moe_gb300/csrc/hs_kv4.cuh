// Geometry of the 4-bit key/value cache (see hs_kv4_cache in hs.h), shared by
// its kernels: plan, append, read, attention.  sm_103a.
#pragma once

#include "hs_common.cuh"
#include "hs_host.h"

namespace hs {

constexpr int kKvMaxSeqs = 4096;
constexpr int kKvMaxTokens = 1 << 20;   // tokens of one append or read

struct KvGeom {
    uint8_t* pool;
    long long slots;     // n_pages * page_tokens
    int n_pages;
    int page_log2;
    int heads;
    int rec;             // bytes of one (page, kv head) record
};

// Bytes of a record of `tokens` tokens: K and V codes, K and V pairs.
__host__ __device__ constexpr int kv_record_bytes(int tokens, int dim) { return tokens * (dim + dim / 8); }

__device__ __forceinline__ uint8_t* kv_record(const KvGeom& g, int page, int head) {
    return g.pool + ((size_t)page * g.heads + head) * (size_t)g.rec;  // past 4 GB in a long cache: 64 bits
}

}  // namespace hs

namespace hs_host {

inline bool kv4_shape_ok(const hs_kv4_cache* c) {
    return c->n_pages >= 1 && (c->page_tokens == 16 || c->page_tokens == 32 || c->page_tokens == 64) &&
           c->n_kv_heads >= 1 && c->n_kv_heads <= 256 && (c->head_dim == 64 || c->head_dim == 128);
}

inline int kv4_check(const hs_kv4_cache* c) {
    if (!c || !c->pool) return HS_ERR_INVALID_ARG;
    if (!kv4_shape_ok(c)) return HS_ERR_UNSUPPORTED_SHAPE;
    return al16(c->pool) ? HS_OK : HS_ERR_MISALIGNED;
}

inline hs::KvGeom kv4_geom(const hs_kv4_cache* c) {
    hs::KvGeom g;
    g.pool = static_cast<uint8_t*>(c->pool);
    g.slots = (long long)c->n_pages * c->page_tokens;
    g.n_pages = c->n_pages;
    g.page_log2 = c->page_tokens == 16 ? 4 : c->page_tokens == 32 ? 5 : 6;
    g.heads = c->n_kv_heads;
    g.rec = hs::kv_record_bytes(c->page_tokens, c->head_dim);
    return g;
}

// SMs of the current device, asked once per device.
inline int sm_count() {
    static int n[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!n[dev] && cudaDeviceGetAttribute(&n[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) n[dev] = 0;
    return n[dev];
}

}  // namespace hs_host
