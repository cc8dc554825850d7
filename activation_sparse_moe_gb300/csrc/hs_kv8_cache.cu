// Rows of the 8-bit key/value cache: append and read, GB300 (sm_103a).  Format
// and contracts: hs.h.
#include "hs_kv8.cuh"

namespace hs {

struct Kv8AppendArgs {
    KvGeom g;
    const uint16_t* x[2];    // K, V
    long long st[2], sh[2];  // strides of tokens and heads, elements
    const long long* slot;
    int n, span;             // tokens; of a warp: the runs that begin among so many are its own
};

// A block's scale belongs to up to 16 tokens, so a run of tokens of one block is one
// warp's work (a head's K or V): it finds the largest magnitude, brings older codes to a scale that
// has grown (rarely), and rounds the new rows, which it keeps in registers: they are read
// once.  D / 8 lanes take a row, 16 bytes of it each.  What is past 57344 or NaN is found by
// comparing bf16 bits.
//
// Bound by latencies: the slots, then the rows (which a prefetch brings nearer meanwhile: 12.7 to
// 11.7 us); 830 instructions a warp.  8191 tokens of 8 kv heads of 128 channels, 2048 CTAs where 912
// are resident (2.25 waves): 11.1 us, where their 50 MB take 7.4.  Six CTAs an SM are what fits without a spill
// (five 11.7 us, seven with one 12.5).
constexpr uint32_t kLargest = 0x4760u;  // 57344 in bf16

template <int D>
__global__ void __launch_bounds__(128, 6) kv8_append_kernel(const Kv8AppendArgs a) {
    constexpr int kL = D / 8, kR = 32 / kL, kIts = kKv8Block / kR;  // lanes a row, rows at a time, turns for 16 rows
    const int lane = threadIdx.x & 31, sub = lane / kL, c8 = lane % kL;
    const int unit = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int per = 2 * a.g.heads, seg = unit / per, kv = unit % per / a.g.heads, head = unit % a.g.heads;
    pdl_wait();
    pdl_trigger();
    const int t0 = seg * a.span;
    if (t0 >= a.n) return;
    const uint16_t* x = (kv ? a.x[1] : a.x[0]) + (long long)head * (kv ? a.sh[1] : a.sh[0]);
    const long long st = kv ? a.st[1] : a.st[0];
    // The rows' addresses are known before the slots are: they come into L2 meanwhile.
    if (D == 128 ? lane < 2 * a.span : lane < a.span) {
        const int t = t0 + (D == 128 ? lane >> 1 : lane);
        if (t < a.n) prefetch_l2(x + t * st + (D == 128 ? (lane & 1) * 64 : 0));
    }
    auto block_at = [&](int t, long long& s) -> long long {
        s = t >= 0 && t < a.n ? a.slot[t] : -1;
        return s >= 0 && s < a.g.slots ? s >> 4 : -1;
    };
    long long slot, unused;
    const long long mine = block_at(t0 + lane, slot);
    long long before = __shfl_up_sync(~0u, mine, 1);
    if (lane == 0) before = block_at(t0 - 1, unused);
    unsigned runs = __ballot_sync(~0u, lane < a.span && mine >= 0 && mine != before);
    x += c8 * 8;
    const int P = 1 << a.g.page_log2;
    for (; runs; runs &= runs - 1) {
        const int l = __ffs(runs) - 1;
        const long long block = __shfl_sync(~0u, mine, l);
        const unsigned same = __ballot_sync(~0u, mine == block) >> l;
        const int count = min(~same ? __ffs(~same) - 1 : 32, kKv8Block);
        const int first = (int)warp_min_u32(lane >= l && lane < l + count ? (uint32_t)slot & 15u : 16u);
        uint4 v[kIts];  // the rows (absent ones as zeros)
#pragma unroll
        for (int i = 0; i < kIts; ++i) {
            const int j = i * kR + sub;
            v[i] = make_uint4(0, 0, 0, 0);
            if (j < count) v[i] = *reinterpret_cast<const uint4*>(x + (long long)(t0 + l + j) * st);
        }
        uint8_t* rec = kv_record(a.g, (int)((block << 4) >> a.g.page_log2), head);
        const int base = (int)(block << 4) & (P - 1);
        float* scale = reinterpret_cast<float*>(rec + 2 * P * D + base) + kv;
        int e_old = kKv8Low;
        if (first > 0) e_old = min(max((int)(__float_as_uint(*scale) >> 23) - 127, kKv8Low), kKv8High);
        // the largest magnitude of all rows; only if that cannot be held, group by group of 64
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < kIts; ++i)
            most = __vmaxu2(most, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu), __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
        uint32_t top = warp_max_u32(max(most & 0xffffu, most >> 16)), bad = 0;
        if (top > kLargest) {  // past 57344, or NaN
            top = 0;
#pragma unroll
            for (int i = 0; i < kIts; ++i) {
                uint32_t m = __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu), __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(~0u, m, o));
                m = max(m & 0xffffu, m >> 16);
                if (m > kLargest) bad |= 1u << i;
                else top = max(top, m);
            }
            top = warp_max_u32(top);
        }
        // the smallest e with top <= 448 * 2^e = 1.75 * 2^(e + 8)
        int e = max((int)(top >> 7) - 127 - 8 + ((top & 127u) > 96u ? 1 : 0), kKv8Low);
        e = max(e, e_old);
        uint8_t* codes = rec + kv * P * D + (c8 & 1) * 8;
        auto place = [&](int o) { return codes + (base + o) * D + (((c8 >> 1) ^ kv8_turn<D>(o)) << 4); };
        if (first > 0 && e > e_old) {
            const float down = kv8_pow2(e_old - e);
#pragma unroll 1
            for (int o = sub; o < first; o += kR) {
                uint2* at = reinterpret_cast<uint2*>(place(o));
                const uint2 w = *at;
                uint32_t r[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t u = h ? w.y : w.x;
                    const float2 p = half2_to_float2(e4m3x2_half2((uint16_t)u)), q = half2_to_float2(e4m3x2_half2((uint16_t)(u >> 16)));
                    r[h] = half_e4m3x2(p.x * down, p.y * down) | (uint32_t)half_e4m3x2(q.x * down, q.y * down) << 16;
                }
                *at = make_uint2(r[0], r[1]);
            }
        }
        const float up = kv8_pow2(-e);
#pragma unroll
        for (int i = 0; i < kIts; ++i) {
            if (i * kR >= count) break;
            const int j = i * kR + sub, o = (int)__shfl_sync(~0u, (uint32_t)slot & 15u, (l + j) & 31);
            if (j >= count) continue;
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t r[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t z = 0;
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    z |= (uint32_t)half_e4m3x2(__uint_as_float(w[2 * h + k] << 16) * up, __uint_as_float(w[2 * h + k] & 0xffff0000u) * up) << (16 * k);
                r[h] = (bad >> i) & 1u ? 0x7f7f7f7fu : z;
            }
            *reinterpret_cast<uint2*>(place(o)) = make_uint2(r[0], r[1]);
        }
        __syncwarp();  // (the old scale has been read)
        if (lane == 0) {
            *scale = kv8_pow2(e);
            if (!kv) *reinterpret_cast<uint2*>(scale + 2) = make_uint2(0, 0);
        }
    }
}

struct Kv8ReadArgs {
    KvGeom g;
    const long long* slot;
    int n, per;  // tokens; sets of eight channels of a token
    uint16_t* b16[2];
    float* f32[2];
};

// A thread takes eight channels of a key and those of its value.  (Sixteen write
// their 32 bytes in two halves, 16 bytes of every sector at a time: 14.8 us for 8191 tokens of
// 8 kv heads, two sets a thread 12.1, this 10.8, where their 50 MB take 7.4; what is left are two
// dependent reads in each of 4098 CTAs, of which 1216 are resident: 3.4 waves.)
template <int D>
__global__ void __launch_bounds__(256) kv8_read_kernel(const Kv8ReadArgs a) {
    constexpr int kL = D / 8;
    pdl_wait();
    pdl_trigger();
    const int P = 1 << a.g.page_log2;
    const long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (at >= (long long)a.n * a.per) return;
    const uint32_t t = (uint32_t)at / (uint32_t)a.per, rest = (uint32_t)at - t * (uint32_t)a.per, head = rest / kL, c8 = rest % kL;  // (below 2^32)
    uint2 w[2] = {make_uint2(0, 0), make_uint2(0, 0)};
    float2 s = make_float2(0.f, 0.f);
    const long long slot = a.slot[t];
    if (slot >= 0 && slot < a.g.slots) {
        const uint8_t* rec = kv_record(a.g, (int)(slot >> a.g.page_log2), (int)head);
        const int o = (int)slot & (P - 1);
        const uint8_t* code = rec + o * D + (((int)(c8 >> 1) ^ kv8_turn<D>(o)) << 4) + (c8 & 1) * 8;
        w[0] = *reinterpret_cast<const uint2*>(code);
        w[1] = *reinterpret_cast<const uint2*>(code + P * D);
        s = *reinterpret_cast<const float2*>(rec + 2 * P * D + (o & ~15));
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const __half2 scale = __float2half2_rn(kv ? s.y : s.x);  // (exact, and so are the products)
        float2 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t h = e4m3x2_half2((uint16_t)((k < 2 ? w[kv].x : w[kv].y) >> (16 * (k & 1))));
            x[k] = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&h), scale));
        }
        uint16_t* b16 = kv ? a.b16[1] : a.b16[0];
        float* f32 = kv ? a.f32[1] : a.f32[0];
        if (b16) {
            uint32_t z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 y = __float22bfloat162_rn(x[k]);
                z[k] = *reinterpret_cast<const uint32_t*>(&y);
            }
            *reinterpret_cast<uint4*>(b16 + at * 8) = make_uint4(z[0], z[1], z[2], z[3]);
        }
        if (f32) {
            *reinterpret_cast<float4*>(f32 + at * 8) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
            *reinterpret_cast<float4*>(f32 + at * 8 + 4) = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
        }
    }
}

}  // namespace hs

using namespace hs_host;

extern "C" size_t hs_kv8_pool_bytes(const hs_kv8_cache* c) {
    if (!c || !kv8_shape_ok(c)) return 0;
    return (size_t)c->n_pages * c->n_kv_heads * hs::kv8_record_bytes(c->page_tokens, c->head_dim);
}

extern "C" int hs_kv8_append(const hs_kv8_cache* cache, const uint16_t* k, long long k_st, long long k_sh, const uint16_t* v,
                             long long v_st, long long v_sh, const long long* slot, int n_tokens, hs_stream_t stream) {
    const int st = kv8_check(cache);
    if (st != HS_OK) return st;
    if (!k || !v || !slot || n_tokens < 0) return HS_ERR_INVALID_ARG;
    if (n_tokens > hs::kKvMaxTokens) return HS_ERR_UNSUPPORTED_SHAPE;
    if (!al16(k) || !al16(v) || ((uintptr_t)slot & 7u) || (k_st | k_sh | v_st | v_sh) & 7) return HS_ERR_MISALIGNED;
    if (!n_tokens) return HS_OK;
    const int sms = sm_count();
    if (!sms) return HS_ERR_CUDA;
    // A warp looks for runs among `span` tokens: one where that alone gives few warps, 16 where there
    // are many, whose runs are whole blocks if they are a prompt's.  If they are single tokens of many
    // requests a warp does its runs in turn: 256, 1024 and 4096 of 8 kv heads 4.6, 10.3 and 31 us.
    const long long rows = 2ll * cache->n_kv_heads;
    int span = 1;
    while (span < hs::kKv8Block && (n_tokens + 2 * span - 1) / (2 * span) * rows >= 16ll * sms) span *= 2;
    const long long warps = (n_tokens + span - 1) / span * rows;
    hs::Kv8AppendArgs a = {kv8_geom(cache), {k, v}, {k_st, v_st}, {k_sh, v_sh}, slot, n_tokens, span};
    auto kern = cache->head_dim == 64 ? hs::kv8_append_kernel<64> : hs::kv8_append_kernel<128>;
    if (launch_pdl(kern, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
        return HS_ERR_CUDA;
    return launch_err();
}

extern "C" int hs_kv8_read(const hs_kv8_cache* cache, const long long* slot, int n_tokens, uint16_t* k16, uint16_t* v16,
                           float* k32, float* v32, hs_stream_t stream) {
    const int st = kv8_check(cache);
    if (st != HS_OK) return st;
    if (!slot || n_tokens < 0 || !(k16 || v16 || k32 || v32)) return HS_ERR_INVALID_ARG;
    if (n_tokens > hs::kKvMaxTokens) return HS_ERR_UNSUPPORTED_SHAPE;
    if (((uintptr_t)slot & 7u) || !al16(k16) || !al16(v16) || !al16(k32) || !al16(v32)) return HS_ERR_MISALIGNED;
    if (!n_tokens) return HS_OK;
    const int per = cache->n_kv_heads * cache->head_dim / 8;
    hs::Kv8ReadArgs a = {kv8_geom(cache), slot, n_tokens, per, {k16, v16}, {k32, v32}};
    const long long threads = (long long)n_tokens * per;  // at most 2^32
    auto kern = cache->head_dim == 64 ? hs::kv8_read_kernel<64> : hs::kv8_read_kernel<128>;
    if (launch_pdl(kern, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
        return HS_ERR_CUDA;
    return launch_err();
}
