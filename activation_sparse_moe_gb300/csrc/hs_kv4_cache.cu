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
// the launch and two dependent reads for small steps (8 requests: 3.4 us), by the
// scan and the tables' bytes for large ones (1000 requests, 4.4 MB read and written:
// 6.2 us).
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
// Eight lanes take a group of 64 channels, eight channels each.  A warp's four
// lane groups walk along one row (a token's K or V over all its heads), or
// along two or four rows where a row has two groups or one: a row's addresses
// are worked out once, then only stepped (worked out group by group they took
// half of the instructions).  Four groups of a lane group are in flight at a time.
// Bound by instructions: 8191 tokens of 8 kv heads of 128 channels take 22.7 us for
// both calls, where their bytes take 12.7.
constexpr int kAhead = 4;        // groups a lane group has in flight
constexpr int kRowGroups = 64;   // groups of a row that one warp takes; more go to gridDim.y

struct KvRows {
    KvGeom g;
    const long long* slot;
    int rows, per;   // 2 * tokens; groups of a row
    int abreast;     // lane groups on one row: 1, 2 or 4
};

// The place of the calling lane group: its row and its first group there.
template <int D>
struct KvLane {
    static constexpr int NG = D / 64;
    int t, kv, group, end, head, grp;
    long long slot;
    uint8_t *codes, *pair;  // of its first group; the next one's are `step` bytes on
    size_t step;
    __device__ __forceinline__ KvLane(const KvRows& a) {
        const int lg = (threadIdx.x & 31) >> 3, warp = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
        const int row = a.abreast == 4 ? warp : a.abreast == 2 ? warp * 2 + (lg >> 1) : warp * 4 + lg;
        group = blockIdx.y * kRowGroups + (lg & (a.abreast - 1));
        end = row < a.rows ? min(a.per, (int)(blockIdx.y + 1) * kRowGroups) : 0;
        t = row < a.rows ? row >> 1 : 0;
        kv = row & 1;
        head = group / NG, grp = group % NG;
        slot = end ? a.slot[t] : -1;
        if (slot >= a.g.slots) slot = -1;
        const long long at = max(slot, 0ll);
        const int page = (int)(at >> a.g.page_log2), off = (int)at & ((1 << a.g.page_log2) - 1);
        uint8_t* rec = kv_record(a.g, page, head);
        const int half_b = (D / 2) << a.g.page_log2, pairs = (NG * 4) << a.g.page_log2;
        codes = rec + kv * half_b + off * (D / 2) + grp * 32;
        pair = rec + 2 * half_b + kv * pairs + (off * NG + grp) * 4;
        step = (size_t)(a.abreast > NG ? a.abreast / NG : 1) * (size_t)a.g.rec;
    }
};

struct AppendArgs {
    KvRows r;
    const uint16_t* x[2];    // K, V
    long long st[2], sh[2];  // strides of tokens and heads, elements
};

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t v) { return *reinterpret_cast<__nv_bfloat162*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }

// Minimum and maximum in packed bf16 (exact), the codes in fp32.  The
// definition's code is rint of the rounded quotient (x - b) / s, clamped.
// Here t = sat((x - b) * r), r an approximate 1 / (15 s): 15 t is within 2^-17
// of the clamped quotient, so its rint is the same unless it lies within 2^-16
// of a half, and only then (one group in some thousands) are the quotients
// taken.  The four codes of a half word are summed as a float, exactly.  The
// division of the range by 15 is one correction step of the product with the
// rounded 1 / 15, which rounds as the division does.  Ten instructions a value
// where the quotients took thirty: the instructions bounded this, not the bytes
// (2 in and 0.56 out a value).
template <int D>
__global__ void __launch_bounds__(128) kv4_append_kernel(const AppendArgs a) {
    const int lane8 = threadIdx.x & 7;
    pdl_wait();
    pdl_trigger();
    const KvLane<D> u(a.r);
    const uint16_t* src = (u.kv ? a.x[1] : a.x[0]) + (long long)u.t * (u.kv ? a.st[1] : a.st[0]) +
                          (long long)u.head * (u.kv ? a.sh[1] : a.sh[0]) + u.grp * 64 + lane8 * 8;
    const long long src_step = (u.kv ? a.sh[1] : a.sh[0]) * (a.r.abreast > D / 64 ? a.r.abreast / (D / 64) : 1);
    uint8_t *codes = u.codes, *pair = u.pair;
    // the same number of turns for all lanes of a warp: they shuffle
    for (int g0 = u.group; __any_sync(~0u, g0 < u.end); g0 += kAhead * a.r.abreast) {
        uint4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            v[j] = make_uint4(0, 0, 0, 0);
            if (g0 + j * a.r.abreast < u.end) v[j] = *reinterpret_cast<const uint4*>(src);
            src += src_step;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j, codes += u.step, pair += u.step) {
            if (!__any_sync(~0u, g0 + j * a.r.abreast < u.end)) break;
            const uint32_t w4[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            __nv_bfloat162 mn = __hmin2_nan(__hmin2_nan(as_bf2(w4[0]), as_bf2(w4[1])), __hmin2_nan(as_bf2(w4[2]), as_bf2(w4[3])));
            __nv_bfloat162 mx = __hmax2_nan(__hmax2_nan(as_bf2(w4[0]), as_bf2(w4[1])), __hmax2_nan(as_bf2(w4[2]), as_bf2(w4[3])));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                mn = __hmin2_nan(mn, as_bf2(__shfl_xor_sync(~0u, as_u32(mn), o)));
                mx = __hmax2_nan(mx, as_bf2(__shfl_xor_sync(~0u, as_u32(mx), o)));
            }
            const float lo = __bfloat162float(__hmin_nan(mn.x, mn.y)), hi = __bfloat162float(__hmax_nan(mx.x, mx.y));
            const float range = __fsub_rn(hi, lo), fifteenth = range * (1.f / 15.f);
            __half sh = __float2half_rn(__fmaf_rn(__fmaf_rn(-15.f, fifteenth, range), 1.f / 15.f, fifteenth));
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
                float inv, worst = 0.f;
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s * 15.f));
                uint32_t half[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float sum = 8388608.f;  // 2^23: the sum's integer stands in the low bits
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t w = w4[2 * h + (i >> 1)];
                        const float x = __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
                        const float t = __saturatef(__fsub_rn(x, b) * inv);
                        const float q = __fadd_rn(__fmaf_rn(t, 15.f, 12582912.f), -12582912.f);  // 1.5 * 2^23: rounds to an integer
                        worst = fmaxf(worst, fabsf(__fmaf_rn(t, 15.f, -q)));
                        sum = __fmaf_rn(q, (float)(1 << (4 * i)), sum);
                    }
                    half[h] = __float_as_uint(sum);
                }
                word = __byte_perm(half[0], half[1], 0x5410);
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
            if (g0 + j * a.r.abreast >= u.end || u.slot < 0) continue;
            // Two stores: of tokens with one slot the codes of one and the pair of the other may stay
            // (one owner a slot would take a search of the slots, or a lock a group).
            reinterpret_cast<uint32_t*>(codes)[lane8] = word;
            if (lane8 == 0) *reinterpret_cast<uint32_t*>(pair) = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(bh) << 16);
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
__global__ void __launch_bounds__(128) kv4_read_kernel(const ReadArgs a) {
    const int lane8 = threadIdx.x & 7;
    pdl_wait();
    pdl_trigger();
    const KvLane<D> u(a.r);
    const uint8_t *codes = u.codes, *pair = u.pair;
    uint16_t* b16 = u.kv ? a.b16[1] : a.b16[0];
    float* f32 = u.kv ? a.f32[1] : a.f32[0];
    size_t at = ((size_t)u.t * a.r.g.heads + u.head) * D + u.grp * 64 + lane8 * 8;
    const int at_step = a.r.abreast * 64;  // outputs are packed: groups follow one another
    for (int g0 = u.group; g0 < u.end; g0 += kAhead * a.r.abreast) {
        uint32_t word[kAhead], sb[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j, codes += u.step, pair += u.step) {
            word[j] = sb[j] = 0;
            if (u.slot >= 0 && g0 + j * a.r.abreast < u.end) {
                word[j] = reinterpret_cast<const uint32_t*>(codes)[lane8];
                sb[j] = *reinterpret_cast<const uint32_t*>(pair);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j, at += at_step) {
            if (g0 + j * a.r.abreast >= u.end) break;
            const float2 p = half2_to_float2(sb[j]);
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // channels i and i + 4: 1024 + code is exact in fp16
                uint32_t h = ((word[j] >> (4 * i)) & 0x000f000fu) | 0x64006400u;
                const float2 c = __half22float2(__hsub2(*reinterpret_cast<__half2*>(&h), __half2half2(__ushort_as_half(0x6400))));
                x[i] = fmaf(p.x, c.x, p.y);
                x[i + 4] = fmaf(p.x, c.y, p.y);
            }
            if (b16) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = as_u32(__floats2bfloat162_rn(x[2 * i], x[2 * i + 1]));
                *reinterpret_cast<uint4*>(b16 + at) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (f32) {
                *reinterpret_cast<float4*>(f32 + at) = make_float4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<float4*>(f32 + at + 4) = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
    }
}

constexpr int kRowThreads = 128;
inline KvRows kv_rows(const KvGeom& g, int dim, const long long* slot, int n_tokens) {
    const int per = g.heads * (dim / 64);
    return {g, slot, 2 * n_tokens, per, per >= 3 ? 4 : per};
}
inline dim3 kv_rows_grid(const KvRows& r) {
    const int rows = kRowThreads / 32 * (4 / r.abreast);  // of a CTA
    return dim3((r.rows + rows - 1) / rows, (r.per + kRowGroups - 1) / kRowGroups);
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
    // What the call writes overlaps nothing else: every CTA reads the lengths, the old
    // table and the ring while others write.  Only the table may be updated in place.
    const long long n = n_seqs, cells = n * table_width;
    struct Range {
        const void* p;
        long long bytes;
    } const ranges[] = {{table_out, cells * 4}, {ring, n_pages * 4ll}, {seq_len, n * 4}, {q_start, (n + 1) * 4}, {slot, max_tokens * 8ll},
                        {position, max_tokens * 4ll}, {counters_out, 16}, {short_out, 4},  // written up to here
                        {table_in, cells * 4}, {cached, n * 4}, {fresh, n * 4}, {counters_in, 16}};
    for (int i = 0; i < 8; ++i)
        for (int j = i + 1; j < 12; ++j) {
            const Range &x = ranges[i], &y = ranges[j];
            if (!x.p || !y.p || (i == 0 && j == 8 && x.p == y.p)) continue;
            const uintptr_t a = (uintptr_t)x.p, b = (uintptr_t)y.p;
            if (a < b + (uintptr_t)y.bytes && b < a + (uintptr_t)x.bytes) return HS_ERR_INVALID_ARG;
        }
    const int smem = (4 * n_seqs + 2) * (int)sizeof(int);
    if (smem > 48 * 1024) {
        const int st = set_smem_attr((const void*)hs::kv4_plan_kernel, (4 * hs::kKvMaxSeqs + 2) * (int)sizeof(int));
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
    hs::AppendArgs a = {hs::kv_rows(kv4_geom(cache), cache->head_dim, slot, n_tokens), {k, v}, {k_st, v_st}, {k_sh, v_sh}};
    auto kern = cache->head_dim == 64 ? hs::kv4_append_kernel<64> : hs::kv4_append_kernel<128>;
    if (launch_pdl(kern, hs::kv_rows_grid(a.r), dim3(hs::kRowThreads), 0, reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
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
    hs::ReadArgs a = {hs::kv_rows(kv4_geom(cache), cache->head_dim, slot, n_tokens), {k16, v16}, {k32, v32}};
    auto kern = cache->head_dim == 64 ? hs::kv4_read_kernel<64> : hs::kv4_read_kernel<128>;
    if (launch_pdl(kern, hs::kv_rows_grid(a.r), dim3(hs::kRowThreads), 0, reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
        return HS_ERR_CUDA;
    return launch_err();
}
