// Geometry of the 4-bit key/value cache (see hs_kv4_cache in hs.h), shared by
// its kernels: plan, append, read, attention.  sm_103a.
#pragma once

#include "hs_common.cuh"
#include "hs_host.h"

namespace hs {

constexpr int kKvMaxSeqs = 4096;
constexpr int kKvMaxTokens = 1 << 20;   // tokens of one append or read
constexpr long long kKvMaxKeys = (1ll << 31) - (1 << 13);  // of a table's row: the loads look some 4000 keys ahead in 32 bits

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

// bulk_g2s with shared-memory addresses of the 32-bit window.
__device__ __forceinline__ void bulk_g2s_to(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// mbar_wait by a whole warp: it gives up as one, where its lanes would run out of
// patience one by one and come to its next vote or shuffle in parts.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    if (__all_sync(~0u, mbar_try_wait(bar, parity))) [[likely]] return true;
    const unsigned long long t0 = clock64();
    while (!__all_sync(~0u, mbar_try_wait(bar, parity))) {
        if (__any_sync(~0u, clock64() - t0 > kWaitLimitCycles)) {
            atomicOr(&g_status, 1u);
            return false;
        }
    }
    return true;
}

// True in one lane of the (converged) warp; the compiler then knows the branch
// to be taken by one thread, and keeps the operands in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(ok));
    return ok != 0;
}

// 32 lanes x 32 columns without the wait: the registers hold their values only
// after tmem_ld_wait over them.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        :
          "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}
// Completes this thread's tensor-memory loads; every use of v comes after it.
__device__ __forceinline__ void tmem_ld_wait(float (&v)[128]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        :
          "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
          "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
          "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
          "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]),
          "+f"(v[32]), "+f"(v[33]), "+f"(v[34]), "+f"(v[35]), "+f"(v[36]), "+f"(v[37]), "+f"(v[38]), "+f"(v[39]),
          "+f"(v[40]), "+f"(v[41]), "+f"(v[42]), "+f"(v[43]), "+f"(v[44]), "+f"(v[45]), "+f"(v[46]), "+f"(v[47]),
          "+f"(v[48]), "+f"(v[49]), "+f"(v[50]), "+f"(v[51]), "+f"(v[52]), "+f"(v[53]), "+f"(v[54]), "+f"(v[55]),
          "+f"(v[56]), "+f"(v[57]), "+f"(v[58]), "+f"(v[59]), "+f"(v[60]), "+f"(v[61]), "+f"(v[62]), "+f"(v[63]),
          "+f"(v[64]), "+f"(v[65]), "+f"(v[66]), "+f"(v[67]), "+f"(v[68]), "+f"(v[69]), "+f"(v[70]), "+f"(v[71]),
          "+f"(v[72]), "+f"(v[73]), "+f"(v[74]), "+f"(v[75]), "+f"(v[76]), "+f"(v[77]), "+f"(v[78]), "+f"(v[79]),
          "+f"(v[80]), "+f"(v[81]), "+f"(v[82]), "+f"(v[83]), "+f"(v[84]), "+f"(v[85]), "+f"(v[86]), "+f"(v[87]),
          "+f"(v[88]), "+f"(v[89]), "+f"(v[90]), "+f"(v[91]), "+f"(v[92]), "+f"(v[93]), "+f"(v[94]), "+f"(v[95]),
          "+f"(v[96]), "+f"(v[97]), "+f"(v[98]), "+f"(v[99]), "+f"(v[100]), "+f"(v[101]), "+f"(v[102]), "+f"(v[103]),
          "+f"(v[104]), "+f"(v[105]), "+f"(v[106]), "+f"(v[107]), "+f"(v[108]), "+f"(v[109]), "+f"(v[110]), "+f"(v[111]),
          "+f"(v[112]), "+f"(v[113]), "+f"(v[114]), "+f"(v[115]), "+f"(v[116]), "+f"(v[117]), "+f"(v[118]), "+f"(v[119]),
          "+f"(v[120]), "+f"(v[121]), "+f"(v[122]), "+f"(v[123]), "+f"(v[124]), "+f"(v[125]), "+f"(v[126]), "+f"(v[127])
        :
        : "memory");
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
