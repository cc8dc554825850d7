// The 4-bit key/value cache's bookkeeping and its rows: step plan, append and
// read, GB300 (sm_103a).  Formats and contracts: hs.h.
#include "hs_kv4.cuh"

namespace hs {

// ------------------------------------------------------------------ plan
struct PlanArgs {
    const int* cached;
    const int* fresh;
    int n, page_log2, n_pages, width;
    const int* table_in;
    int* ring;
    const long long* counters_in;
    int max_tokens;
    int* table_out;
    int* seq_len;
    int* q_start;
    long long* slot;
    int* position;
    long long* counters_out;
    int* short_out;
};

constexpr int kPlanThreads = 256;

// Every CTA scans all requests (three running sums over at most 4096 of them,
// held in shared memory) and then writes its share of the rows and tokens: the
// CTAs need nothing from one another, so one launch does the step.  Bound by
// the launch and two dependent reads for small steps, by the tables' bytes for
// large ones.
__global__ void __launch_bounds__(kPlanThreads) kv4_plan_kernel(const PlanArgs a) {
    extern __shared__ int plan_smem[];
    int* have = plan_smem;              // [n] cached pages, -1 - pages for an ended request
    int* start = plan_smem + a.n;       // [n + 1] new tokens before each request
    int* taken = start + a.n + 1;       // [n + 1] new pages before it
    int* given = taken + a.n + 1;       // [n] pages of ended requests before it
    __shared__ long long part[kPlanThreads / 32][4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = 1 << a.page_log2;

    pdl_wait();
    pdl_trigger();
    const long long head = a.counters_in[0], tail = a.counters_in[1];
    const int per = (a.n + kPlanThreads - 1) / kPlanThreads;
    const int i0 = min(tid * per, a.n), i1 = min(i0 + per, a.n);
    long long tok = 0, need = 0, back = 0, over = 0;
    for (int i = i0; i < i1; ++i) {
        const long long c = max(a.cached[i], 0), f = a.fresh[i];
        const long long held = (c + P - 1) >> a.page_log2, h = min(held, (long long)a.width);
        if (f < 0) {
            have[i] = (int)(-1 - h);
            back += h;
        } else {
            have[i] = (int)h;
            const long long want = (c + f + P - 1) >> a.page_log2;
            need += want - held;
            over += max(want - a.width, 0ll);
            tok += f;
        }
    }
    // exclusive sums over the threads' runs of requests
    long long s_tok = tok, s_need = need, s_back = back;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t0 = __shfl_up_sync(~0u, s_tok, o), t1 = __shfl_up_sync(~0u, s_need, o),
                        t2 = __shfl_up_sync(~0u, s_back, o);
        if (lane >= o) s_tok += t0, s_need += t1, s_back += t2;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) over += __shfl_xor_sync(~0u, over, o);
    if (lane == 31) part[warp][0] = s_tok, part[warp][1] = s_need, part[warp][2] = s_back, part[warp][3] = over;
    __syncthreads();
    long long all_tok = 0, all_need = 0, all_back = 0, all_over = 0, b_tok = 0, b_need = 0, b_back = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp) b_tok = all_tok, b_need = all_need, b_back = all_back;
        all_tok += part[w][0], all_need += part[w][1], all_back += part[w][2], all_over += part[w][3];
    }
    const long long missing = all_over + max(all_need - (tail - head), 0ll) + max(all_tok - a.max_tokens, 0ll);
    const bool ok = missing == 0;
    if (!ok) all_tok = all_need = 0;
    b_tok += s_tok - tok, b_need += s_need - need, b_back += s_back - back;
    for (int i = i0; i < i1; ++i) {
        const int h = have[i];
        start[i] = ok ? (int)b_tok : 0;
        taken[i] = ok ? (int)b_need : 0;
        given[i] = (int)b_back;
        if (h < 0) {
            b_back += -1 - h;
        } else {
            const long long c = max(a.cached[i], 0), f = a.fresh[i];
            b_need += ((c + f + P - 1) >> a.page_log2) - ((c + P - 1) >> a.page_log2);
            b_tok += f;
        }
    }
    if (tid == 0) start[a.n] = (int)all_tok, taken[a.n] = (int)all_need;
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int i = tid; i <= a.n; i += kPlanThreads) {
            a.q_start[i] = start[i];
            if (i < a.n)
                a.seq_len[i] = have[i] < 0 ? 0 : max(a.cached[i], 0) + (start[i + 1] - start[i]);
        }
        if (tid == 0) {
            a.counters_out[0] = head + all_need;
            a.counters_out[1] = tail + all_back;
            a.short_out[0] = (int)min(missing, (long long)INT32_MAX);
        }
    }
    const uint32_t np = (uint32_t)a.n_pages;
    const uint32_t head_m = (uint32_t)((head % a.n_pages + a.n_pages) % a.n_pages);
    const uint32_t tail_m = (uint32_t)((tail % a.n_pages + a.n_pages) % a.n_pages);

    // Table rows, a warp a row.
    const bool in_place = a.table_in == a.table_out;
    for (int i = blockIdx.x * (kPlanThreads / 32) + warp; i < a.n; i += gridDim.x * (kPlanThreads / 32)) {
        const int h = have[i];
        const int* src = a.table_in + (size_t)i * a.width;
        int* dst = a.table_out + (size_t)i * a.width;
        if (h < 0) {
            const int hh = -1 - h;
            const uint32_t at = (tail_m + (uint32_t)given[i]) % np;
            for (int c = lane; c < a.width; c += 32) {
                if (c < hh) a.ring[(at + (uint32_t)c) % np] = src[c];
                dst[c] = -1;
            }
        } else {
            const int want = h + taken[i + 1] - taken[i];
            const uint32_t at = (head_m + (uint32_t)taken[i]) % np;
            if (in_place) {
                for (int c = h + lane; c < want; c += 32) dst[c] = a.ring[(at + (uint32_t)(c - h)) % np];
            } else {
#pragma unroll 4
                for (int c = lane; c < a.width; c += 32)
                    dst[c] = c < h ? src[c] : c < want ? a.ring[(at + (uint32_t)(c - h)) % np] : -1;
            }
        }
    }
    // Tokens, a thread each; their pages come from the old table or the ring,
    // not from the rows that other CTAs are writing.
    for (int j = blockIdx.x * kPlanThreads + tid; j < a.max_tokens; j += gridDim.x * kPlanThreads) {
        long long s = -1;
        int pos = -1;
        if (j < (int)all_tok) {
            int lo = 0, hi = a.n;  // the last request with start <= j
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (start[mid] <= j) lo = mid;
                else hi = mid;
            }
            pos = max(a.cached[lo], 0) + (j - start[lo]);
            const int c = pos >> a.page_log2, h = have[lo];
            const int page = c < h ? a.table_in[(size_t)lo * a.width + c]
                                   : a.ring[((head_m + (uint32_t)taken[lo]) % np + (uint32_t)(c - h)) % np];
            if (page >= 0) s = ((long long)page << a.page_log2) + (pos & (P - 1));
        }
        a.slot[j] = s;
        if (a.position) a.position[j] = pos;
    }
}

// ------------------------------------------------------- append and read
// A unit is a group of 64 channels of one (token, K or V, kv head); eight lanes
// take one, eight channels each, and a CTA kUnits of them at a time, two a
// lane group with their loads in flight together.
constexpr int kUnits = 64;

struct KvRows {
    KvGeom g;
    const long long* slot;
    uint32_t units, per;  // tokens * per; groups of a token's K (and of its V)
    uint32_t inv;         // ceil(2^32 / per)
};

struct KvUnit {
    uint32_t t, kv, head, grp;
    bool in;
};

// Unit `off` of the run that starts at unit u0 = q0 * per + r0.
template <int NG>
__device__ __forceinline__ KvUnit kv_unit(const KvRows& a, uint32_t u0, uint32_t q0, uint32_t r0, uint32_t off) {
    KvUnit u;
    u.in = u0 + off < a.units;
    const uint32_t local = r0 + (u.in ? off : 0), q = __umulhi(local, a.inv);  // exact: local * per < 2^32
    const uint32_t row = q0 + (a.per > 1 ? q : local), rest = a.per > 1 ? local - q * a.per : 0;
    u.t = row >> 1, u.kv = row & 1;
    u.head = rest / NG, u.grp = rest % NG;
    return u;
}

struct KvPlace {
    uint8_t *codes, *pair;  // of the group
};
template <int D>
__device__ __forceinline__ KvPlace kv_place(const KvGeom& g, const KvUnit& u, long long slot) {
    constexpr int NG = D / 64;
    const int page = (int)(slot >> g.page_log2), off = (int)slot & ((1 << g.page_log2) - 1);
    uint8_t* rec = kv_record(g, page, (int)u.head);
    const int half_b = (D / 2) << g.page_log2, pairs = (NG * 4) << g.page_log2;
    return {rec + u.kv * half_b + off * (D / 2) + u.grp * 32, rec + 2 * half_b + u.kv * pairs + (off * NG + u.grp) * 4};
}

struct AppendArgs {
    KvRows r;
    const uint16_t* x[2];    // K, V
    long long st[2], sh[2];  // strides of tokens and heads, elements
};

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t v) { return *reinterpret_cast<__nv_bfloat162*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }

// Minimum and maximum in packed bf16 (exact), the codes in fp32.  The
// definition's code is rint of the rounded quotient (x - b) / s; (x - b) times
// the reciprocal is off by at most 2^-19 for quotients up to 16, so its rint is
// the same unless it lies within 2^-16 of a half, and only then (one group in
// some thousands) are the quotients taken.  Bound by bytes: 2 in and 0.56 out a
// value.
template <int D>
__global__ void __launch_bounds__(256) kv4_append_kernel(const AppendArgs a) {
    const int lane8 = threadIdx.x & 7;
    pdl_wait();
    pdl_trigger();
    for (uint32_t u0 = blockIdx.x * (uint32_t)kUnits; u0 < a.r.units; u0 += gridDim.x * (uint32_t)kUnits) {
        const uint32_t q0 = u0 / a.r.per, r0 = u0 - q0 * a.r.per;
        KvUnit un[2];
        uint4 v[2];
        long long slot[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            un[j] = kv_unit<D / 64>(a.r, u0, q0, r0, (threadIdx.x >> 3) + 32 * j);
            const KvUnit& u = un[j];
            const uint16_t* src = u.kv ? a.x[1] + (long long)u.t * a.st[1] + u.head * a.sh[1]
                                       : a.x[0] + (long long)u.t * a.st[0] + u.head * a.sh[0];
            v[j] = *reinterpret_cast<const uint4*>(src + u.grp * 64 + lane8 * 8);
            slot[j] = a.r.slot[u.t];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t w4[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            __nv_bfloat162 mn = __hmin2_nan(__hmin2_nan(as_bf2(w4[0]), as_bf2(w4[1])), __hmin2_nan(as_bf2(w4[2]), as_bf2(w4[3])));
            __nv_bfloat162 mx = __hmax2_nan(__hmax2_nan(as_bf2(w4[0]), as_bf2(w4[1])), __hmax2_nan(as_bf2(w4[2]), as_bf2(w4[3])));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                mn = __hmin2_nan(mn, as_bf2(__shfl_xor_sync(~0u, as_u32(mn), o)));
                mx = __hmax2_nan(mx, as_bf2(__shfl_xor_sync(~0u, as_u32(mx), o)));
            }
            const float lo = __bfloat162float(__hmin_nan(mn.x, mn.y)), hi = __bfloat162float(__hmax_nan(mx.x, mx.y));
            __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
            __half bh = __float2half_rn(lo);
            float s = __half2float(sh);
            const float b = __half2float(bh);
            if (!(fabsf(lo) < 65536.f && fabsf(hi) < 65536.f)) {  // the group reads back as NaN
                sh = __ushort_as_half(0);
                bh = __ushort_as_half(0x7e00);
                s = 0.f;
            }
            uint32_t word = 0;
            if (s > 0.f) {
                const float inv = __frcp_rn(s);
                float worst = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = __uint_as_float(i & 1 ? w4[i >> 1] & 0xffff0000u : w4[i >> 1] << 16);
                    const float q = fminf(fmaxf(__fsub_rn(x, b) * inv, 0.f), 15.f);
                    const float y = __fadd_rn(q, 12582912.f);  // 1.5 * 2^23: rint(q) in the low bits
                    worst = fmaxf(worst, fabsf(q - __fsub_rn(y, 12582912.f)));
                    word |= (__float_as_uint(y) & 15u) << (4 * i);
                }
                if (worst > 0.5f - 1.f / 65536.f) {
                    word = 0;
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t pair = i < 2 ? w4[0] : i < 4 ? w4[1] : i < 6 ? w4[2] : w4[3];
                        const float x = __uint_as_float(i & 1 ? pair & 0xffff0000u : pair << 16);
                        const float q = rintf(__fdiv_rn(__fsub_rn(x, b), s));
                        word |= (uint32_t)fminf(fmaxf(q, 0.f), 15.f) << (4 * i);
                    }
                }
            }
            if (!un[j].in || slot[j] < 0 || slot[j] >= a.r.g.slots) continue;
            const KvPlace p = kv_place<D>(a.r.g, un[j], slot[j]);
            reinterpret_cast<uint32_t*>(p.codes)[lane8] = word;
            if (lane8 == 0) *reinterpret_cast<uint32_t*>(p.pair) = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(bh) << 16);
        }
    }
}

struct ReadArgs {
    KvRows r;
    uint16_t* b16[2];
    float* f32[2];
};

// The append's mapping turned round.
template <int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(const ReadArgs a) {
    const int lane8 = threadIdx.x & 7;
    pdl_wait();
    pdl_trigger();
    for (uint32_t u0 = blockIdx.x * (uint32_t)kUnits; u0 < a.r.units; u0 += gridDim.x * (uint32_t)kUnits) {
        const uint32_t q0 = u0 / a.r.per, r0 = u0 - q0 * a.r.per;
        KvUnit un[2];
        uint32_t word[2], sb[2];
        long long slot[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            un[j] = kv_unit<D / 64>(a.r, u0, q0, r0, (threadIdx.x >> 3) + 32 * j);
            slot[j] = a.r.slot[un[j].t];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            word[j] = sb[j] = 0;
            if (slot[j] >= 0 && slot[j] < a.r.g.slots) {
                const KvPlace p = kv_place<D>(a.r.g, un[j], slot[j]);
                word[j] = reinterpret_cast<const uint32_t*>(p.codes)[lane8];
                sb[j] = *reinterpret_cast<const uint32_t*>(p.pair);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (!un[j].in) continue;
            const float2 p = half2_to_float2(sb[j]);
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(p.x, (float)((word[j] >> (4 * i)) & 15u), p.y);
            const size_t at = ((size_t)un[j].t * a.r.g.heads + un[j].head) * D + un[j].grp * 64 + lane8 * 8;
            if (uint16_t* o = un[j].kv ? a.b16[1] : a.b16[0]) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = as_u32(__floats2bfloat162_rn(x[2 * i], x[2 * i + 1]));
                *reinterpret_cast<uint4*>(o + at) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (float* o = un[j].kv ? a.f32[1] : a.f32[0]) {
                *reinterpret_cast<float4*>(o + at) = make_float4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<float4*>(o + at + 4) = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
    }
}

// Units of a call, its grid: 16 CTAs an SM at most.
inline KvRows kv_rows(const KvGeom& g, int dim, const long long* slot, int n_tokens) {
    const uint32_t per = (uint32_t)g.heads * (uint32_t)(dim / 64);
    return {g, slot, (uint32_t)n_tokens * 2u * per, per, (uint32_t)(((1ull << 32) + per - 1) / per)};
}
inline dim3 kv_rows_grid(const KvRows& r, int sms) {
    return dim3(std::min((r.units + (uint32_t)kUnits - 1u) / (uint32_t)kUnits, (uint32_t)sms * 16u));
}

}  // namespace hs

using namespace hs_host;

extern "C" size_t hs_kv4_pool_bytes(const hs_kv4_cache* c) {
    if (!c || !kv4_shape_ok(c)) return 0;
    return (size_t)c->n_pages * c->n_kv_heads * hs::kv_record_bytes(c->page_tokens, c->head_dim);
}

extern "C" int hs_kv4_plan(const int* cached, const int* fresh, int n_seqs, int page_tokens, int n_pages,
                           const int* table_in, int table_width, int* ring, const long long* counters_in,
                           int max_tokens, int* table_out, int* seq_len, int* q_start, long long* slot, int* position,
                           long long* counters_out, int* short_out, hs_stream_t stream) {
    if (!cached || !fresh || !table_in || !ring || !counters_in || !table_out || !seq_len || !q_start || !slot ||
        !counters_out || !short_out)
        return HS_ERR_INVALID_ARG;
    if (n_seqs < 1 || n_pages < 1 || table_width < 1 || max_tokens < 1 || counters_in == counters_out)
        return HS_ERR_INVALID_ARG;
    if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64) return HS_ERR_UNSUPPORTED_SHAPE;
    if (n_seqs > hs::kKvMaxSeqs || (long long)n_seqs * table_width >= (1 << 30) || max_tokens >= (1 << 30) ||
        n_pages >= (1 << 30) || (long long)table_width * page_tokens >= (1ll << 31))
        return HS_ERR_UNSUPPORTED_SHAPE;
    const void* p4[] = {cached, fresh, table_in, ring, table_out, seq_len, q_start, position, short_out};
    for (const void* p : p4)
        if (!al4(p)) return HS_ERR_MISALIGNED;
    const void* p8[] = {counters_in, counters_out, slot};
    for (const void* p : p8)
        if ((uintptr_t)p & 7u) return HS_ERR_MISALIGNED;
    const int smem = (4 * n_seqs + 2) * (int)sizeof(int);
    if (smem > 48 * 1024) {
        const int st = set_smem_attr((const void*)hs::kv4_plan_kernel, smem);
        if (st != HS_OK) return st;
    }
    hs::PlanArgs a = {cached, fresh,      n_seqs,    page_tokens == 16 ? 4 : page_tokens == 32 ? 5 : 6, n_pages, table_width,
                      table_in, ring,     counters_in, max_tokens, table_out, seq_len, q_start, slot, position,
                      counters_out, short_out};
    // A CTA takes eight table rows or 1024 tokens at a time, up to two CTAs an SM.
    const int sms = sm_count();
    if (!sms) return HS_ERR_CUDA;
    const int want = std::max((n_seqs + 7) / 8, (max_tokens + 1023) / 1024);
    if (launch_pdl(hs::kv4_plan_kernel, dim3(std::min(want, 2 * sms)), dim3(hs::kPlanThreads), smem,
                   reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
        return HS_ERR_CUDA;
    return launch_err();
}

extern "C" int hs_kv4_append(const hs_kv4_cache* cache, const uint16_t* k, long long k_st, long long k_sh,
                             const uint16_t* v, long long v_st, long long v_sh, const long long* slot, int n_tokens,
                             hs_stream_t stream) {
    const int st = kv4_check(cache);
    if (st != HS_OK) return st;
    if (!k || !v || !slot || n_tokens < 0) return HS_ERR_INVALID_ARG;
    if (n_tokens > hs::kKvMaxTokens) return HS_ERR_UNSUPPORTED_SHAPE;
    if (!al16(k) || !al16(v) || ((uintptr_t)slot & 7u) || (k_st | k_sh | v_st | v_sh) & 7) return HS_ERR_MISALIGNED;
    if (!n_tokens) return HS_OK;
    const int sms = sm_count();
    if (!sms) return HS_ERR_CUDA;
    hs::AppendArgs a = {hs::kv_rows(kv4_geom(cache), cache->head_dim, slot, n_tokens), {k, v}, {k_st, v_st}, {k_sh, v_sh}};
    auto kern = cache->head_dim == 64 ? hs::kv4_append_kernel<64> : hs::kv4_append_kernel<128>;
    if (launch_pdl(kern, hs::kv_rows_grid(a.r, sms), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
        return HS_ERR_CUDA;
    return launch_err();
}

extern "C" int hs_kv4_read(const hs_kv4_cache* cache, const long long* slot, int n_tokens, uint16_t* k16, uint16_t* v16,
                           float* k32, float* v32, hs_stream_t stream) {
    const int st = kv4_check(cache);
    if (st != HS_OK) return st;
    if (!slot || n_tokens < 0 || !(k16 || v16 || k32 || v32)) return HS_ERR_INVALID_ARG;
    if (n_tokens > hs::kKvMaxTokens) return HS_ERR_UNSUPPORTED_SHAPE;
    if (((uintptr_t)slot & 7u) || !al16(k16) || !al16(v16) || !al16(k32) || !al16(v32)) return HS_ERR_MISALIGNED;
    if (!n_tokens) return HS_OK;
    const int sms = sm_count();
    if (!sms) return HS_ERR_CUDA;
    hs::ReadArgs a = {hs::kv_rows(kv4_geom(cache), cache->head_dim, slot, n_tokens), {k16, v16}, {k32, v32}};
    auto kern = cache->head_dim == 64 ? hs::kv4_read_kernel<64> : hs::kv4_read_kernel<128>;
    if (launch_pdl(kern, hs::kv_rows_grid(a.r, sms), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
        return HS_ERR_CUDA;
    return launch_err();
}
