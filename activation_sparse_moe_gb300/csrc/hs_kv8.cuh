// Geometry and codes of the 8-bit key/value cache (see hs_kv8_cache in hs.h).
// sm_103a.
#pragma once

#include "hs_kv4.cuh"

namespace hs {

constexpr int kKv8Block = 16;      // tokens of a scale
constexpr int kKv8Low = -15, kKv8High = 7;   // a scale's exponents

// Bytes of a record of `tokens` tokens: K and V codes, 16 bytes of scales a block.
__host__ __device__ constexpr int kv8_record_bytes(int tokens, int dim) { return tokens * (2 * dim + 1); }

// The 16-byte chunk c of a token at offset o stands at place c ^ kv8_turn(o).
template <int D>
__device__ __forceinline__ int kv8_turn(int o) {
    return D == 128 ? ((o & 3) << 1) ^ (o & 4) : o & 2;
}

__device__ __forceinline__ float kv8_pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Two codes (the low byte first) as fp16, exact.
__device__ __forceinline__ uint32_t e4m3x2_half2(uint16_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
    return r;
}
// Two values of at most 448 as codes, to nearest, ties to even; NaN as 0x7f.
__device__ __forceinline__ uint16_t half_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace hs

namespace hs_host {

inline bool kv8_shape_ok(const hs_kv8_cache* c) {
    return c->n_pages >= 1 && (c->page_tokens == 16 || c->page_tokens == 32 || c->page_tokens == 64) &&
           c->n_kv_heads >= 1 && c->n_kv_heads <= 256 && (c->head_dim == 64 || c->head_dim == 128);
}

inline int kv8_check(const hs_kv8_cache* c) {
    if (!c || !c->pool) return HS_ERR_INVALID_ARG;
    if (!kv8_shape_ok(c)) return HS_ERR_UNSUPPORTED_SHAPE;
    return al16(c->pool) ? HS_OK : HS_ERR_MISALIGNED;
}

inline hs::KvGeom kv8_geom(const hs_kv8_cache* c) {
    hs::KvGeom g;
    g.pool = static_cast<uint8_t*>(c->pool);
    g.slots = (long long)c->n_pages * c->page_tokens;
    g.n_pages = c->n_pages;
    g.page_log2 = c->page_tokens == 16 ? 4 : c->page_tokens == 32 ? 5 : 6;
    g.heads = c->n_kv_heads;
    g.rec = hs::kv8_record_bytes(c->page_tokens, c->head_dim);
    return g;
}

}  // namespace hs_host
