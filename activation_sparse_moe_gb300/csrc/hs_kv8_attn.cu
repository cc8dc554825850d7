// Attention of new tokens over the 8-bit key/value cache, GB300 (sm_103a): the
// kernel for few query rows (decode, verification of drafts).  Contract:
// hs_kv8_attention in hs.h; the division of the work: hs_kv4_sched.cuh.
//
// Mathematics.  With k_j = 2^e c_j, e the exponent of the key's block of 16,
//   q . k_j = 2^e (q . c_j),
// so the matrix product runs on the codes, and a block's scale acts on 16 rows of one
// product.  The values' scales fold into the probabilities, o = sum_j (p_j 2^e) c_j, which go to fp16 under
// a power of two of each row's own, that of the largest scale among the blocks that the row sees: what it does not
// see leaves its roundings alone.  (Powers a row cost 0.7 of 13.4 us in 16 x 3 windowed drafts, 2% in other short calls
// and nothing in long ones.)
// e4m3 is exact in fp16, by one conversion for two codes.  Each query row is scaled by the power
// of two that brings its largest channel to [2^8, 2^9), whatever stands in the others:
// bf16 values down to 2^-25 of it then lose nothing as fp16, smaller ones move a
// score by less than 2^-33 of the largest channel's part.
//
// Bounds.  64 decode requests of up to 8192 tokens (32 / 8 heads of 128 channels, 703 MB of
// rows): 108 us, 6.5 TB/s, 96% of the copy bandwidth.  One of 131,071 tokens (32 / 2
// heads): 24.9 us; the rows come in within 9 of them, the start takes 3 and two rounds of joins
// about 10.  A step of 32 keys is some 600 to 900 instructions in long chains of dependent
// products, conversions and exponentials, 0.6 to 1 us to a warp that has the scheduler nearly for itself: that
// bounds short items and those with more than 16 rows.
#include <type_traits>

#include "hs_kv8.cuh"
#include "hs_kv8_join.cuh"

namespace hs {

constexpr int kKvTile = 64;        // keys of a tile; pages of 16 to 64 tokens divide it
constexpr int kKvStep = 32;        // keys of a warp's step

// D += A * B, one 16 x 8 x 16 product of fp16 operands in fp32.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit numbers, lane 4 r + c holding columns 2c and 2c + 1
// of row r, transposed across the warp.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float bf16_f32(uint32_t w, int hi) { return __uint_as_float(hi ? w & 0xffff0000u : w << 16); }

// NQ: query rows of a warp, in eights; RT: warps along the rows; KW: warps along the keys.
template <int D, int NQ, int RT, int KW>
struct Decode8Cfg {
    static constexpr int kNg = D / 64;
    static constexpr int kCtas = RT * KW > 4 ? 1 : 2;  // resident on an SM
    static constexpr int kSlots = D == 128 ? 2 : 3;  // steps of a warp's ring
    static constexpr int kSlotBytes = kv8_record_bytes(kKvStep, D);
    static constexpr int kWarps = RT * KW;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRingBytes = kWarps * kSlots * kSlotBytes;
    static constexpr int kLine = D + 4;               // floats of a row of the warps' sums (padded against bank conflicts)
    static constexpr int kMergeBytes = kWarps * 8 * NQ * (kLine + 2) * 4;
    static constexpr int kRows = 8 * NQ * RT;
    static constexpr int kJoinSets = D == 128 && NQ == 2 ? 2 : 1;  // a warp's share of the rows in the joins
    static int smem(int n_seqs) { return kRingBytes + kMergeBytes + 256 + (n_seqs <= kKvFew ? 0 : n_seqs + 1) * 4; }
};

// Warp (rt, kw): rows 8 NQ rt and up of the item's row tile, the 32-key steps
// kw, kw + KW, ... of the CTA's piece of it.  Every warp keeps its own ring of
// steps full: a lane issues the bulk copies of K codes, V codes and scales as soon as the
// warp has used a slot up, across the ends of items.
//
// Both products have the cache on the left: scores (16 keys x 8 rows) = K q^T
// and outputs (channels x 8 rows) = V^T p^T, so that codes converted once serve all
// rows, and eight rows do not pay for sixteen.  The scores' fragment becomes the
// second product's right operand by one 8 x 8 transposition.  Row r (0..7) of a key
// block stands for key r / 2 + 4 (r % 2): the four lanes of a group then read
// neighbouring rows of V, which the turned chunks of a row bring to different banks,
// 16 channels (eight at 64) a lane; a lane's bytes of two keys are interleaved, and
// bytes 2i and 2i + 1 are rows g and g + 8 of the i-th product.
template <int D, int NQ, int RT, int KW>
__global__ void __launch_bounds__(32 * RT * KW, (Decode8Cfg<D, NQ, RT, KW>::kCtas)) kv8_decode_kernel(const KvAttnArgs a) {
    using C = Decode8Cfg<D, NQ, RT, KW>;
    constexpr int NG = C::kNg;
    extern __shared__ __align__(128) uint8_t smem[];
    float* merge = reinterpret_cast<float*>(smem + C::kRingBytes);  // [warp][row][kLine], then (maximum, sum) [warp][row]
    float2* merge_ml = reinterpret_cast<float2*>(merge + C::kWarps * 8 * NQ * C::kLine);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kRingBytes + C::kMergeBytes);
    uint32_t* cum = reinterpret_cast<uint32_t*>(bars + 32);
    const int *qs = a.q_start, *ls = a.seq_len;  // looked at once an item
    // Where a warp computes and where it loads, a copy a warp in shared memory
    // (every lane writes the same): looked at once an item, and registers are short.
    __shared__ KvWalk walks[C::kWarps], ahead[C::kWarps], comings[C::kWarps];
    __shared__ int join_last;
    static_assert(C::kWarps * C::kSlots < 32, "barriers");  // the last one is the joins'
    uint32_t joins = 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rt = warp / KW, kw = warp % KW, g = lane >> 2, t = lane & 3;  // fragment row or column, and pair

    if (tid < C::kWarps * C::kSlots) {
        mbar_init(bars + tid, 1);
        fence_mbar_init();
    }
    if (tid == 31) {
        mbar_init(bars + 31, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    KvWalk& w = walks[warp];
    uint32_t total;
    if (a.n_seqs <= kKvFew) {
        __syncthreads();  // the barriers are ready
        w = kv_begin_few<KvBound::kShortLine, true>(a, total);
    } else {
        kv_schedule(a, qs, ls, cum);
        w = kv_begin<KvBound::kShortLine>(a, qs, ls, cum);
        total = cum[a.n_seqs];
    }
    ahead[warp] = w;
    __syncwarp();
    const int P = 1 << a.g.page_log2;

    // ---- the warp's ring
    uint8_t* ring = smem + warp * C::kSlots * C::kSlotBytes;
    uint64_t* full = bars + warp * C::kSlots;
    const int parts_log2 = a.g.page_log2 == 4 ? 1 : 0;  // pages of a step: two of 16, or one
    const uint8_t* src = nullptr;  // the head's record in page 0
    uint32_t gone = 0;             // two bits a slot: blocks of 16 keys that are not there
    int key = 0, key_end = 0;      // the next step's first key, and the end of the piece that is being loaded
    int seen = 0, held = -1;       // its steps so far; lane: a table entry of the coming ones
    int in_slot = 0;
    auto piece_to_load = [&](const KvWalk& v) {
        key = (v.lo + v.tile) * kKvTile;
        key_end = key + kv_piece_tiles(v) * kKvTile;
        key += kw * kKvStep;
        seen = 0;
        src = kv_record(a.g, 0, v.head);
    };
    if (w.left > 0) piece_to_load(w);
    auto load = [&]() {
        if (key >= key_end) {  // to the next piece in which this warp has a step
            if (ahead[warp].left <= 0) return;
            do {
                KvWalk n = ahead[warp];
                kv_next_piece(a, qs, ls, n);
                if (n.left > 0) piece_to_load(n);
                __syncwarp();
                ahead[warp] = n;
                __syncwarp();
                if (n.left <= 0) return;
            } while (key >= key_end);
        }
        const int at = (seen++ << parts_log2) & 31;
        if (at == 0) {  // the table entries of the next 16 or 32 steps, one a lane
            const KvWalk& v = ahead[warp];
            const int k = key + (lane >> parts_log2) * KW * kKvStep + ((lane << 4) & (parts_log2 << 4));
            held = v.hi >= v.lo && k < v.len ? a.table[(size_t)v.seq * a.width + (k >> a.g.page_log2)] : -1;
        }
        // Two pages of 16 tokens, or (part of) one: K codes, V codes and scales by a copy
        // each, issued by one lane.
        const int page0 = __shfl_sync(~0u, held, at), page1 = __shfl_sync(~0u, held, at + parts_log2);
        const bool here0 = (uint32_t)page0 < (uint32_t)a.g.n_pages, here1 = (uint32_t)page1 < (uint32_t)a.g.n_pages;
        gone = (gone & ~(3u << (2 * in_slot))) | ((here0 ? 0u : 1u) | (here1 ? 0u : 2u)) << (2 * in_slot);
        if (elect_one()) {
            const uint32_t tokens = kKvStep >> parts_log2, bar = smem_u32(full + in_slot), dst = smem_u32(ring) + in_slot * C::kSlotBytes;
            mbar_arrive_expect_tx(full + in_slot, (here0 ? tokens : 0u) * (2 * D + 1) + (parts_log2 && here1 ? tokens : 0u) * (2 * D + 1));
            const uint64_t policy = policy_evict_first();
            auto copy_page = [&](int page, uint32_t to) {  // to: the step's token that its tokens start at
                const uint8_t* rec = src + (size_t)(uint32_t)page * (uint32_t)(a.g.heads * a.g.rec);
                const uint32_t from = key & (P - 1) & ~15u & (parts_log2 ? 0u : ~0u);
                bulk_g2s_to(dst + to * D, rec + from * D, tokens * D, bar, policy);
                bulk_g2s_to(dst + (kKvStep + to) * D, rec + (P + from) * D, tokens * D, bar, policy);
                bulk_g2s_to(dst + 2 * kKvStep * D + to, rec + 2 * P * D + from, tokens, bar, policy);  // 16 bytes a block of 16
            };
            if (here0) copy_page(page0, 0);
            if (parts_log2 && here1) copy_page(page1, 16);
        }
        __syncwarp();
        key += KW * kKvStep;
        in_slot = in_slot + 1 == C::kSlots ? 0 : in_slot + 1;
    };
    // The queries of an item (lane: row g, 16 channels of each group), read ahead: the
    // first ones before the ring's first pages are looked up, the next ones while
    // the warps' sums of an item are joined.
    uint4 v[NQ][NG][2];
    auto fetch_q = [&](const KvWalk& of) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int row = rt * 8 * NQ + n * 8 + g, in_tile = kv_row_token(a, row), tok = of.r * a.tq + in_tile;
            const bool valid = of.left > 0 && row < a.tq * a.group && tok < of.n;
            const uint16_t* src = a.q + (long long)(of.row0 + tok) * a.q_st + (long long)(of.head * a.group + row - in_tile * a.group) * a.q_sh;
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    v[n][i][h] = valid ? *reinterpret_cast<const uint4*>(src + i * 64 + t * 16 + h * 8) : make_uint4(0, 0, 0, 0);
        }
    };
    fetch_q(w);
    for (int i = 0; i < C::kSlots; ++i) load();

    // ---- the items
    int slot = 0;
    uint32_t phase = 0;  // bit 0: the ring's parity; bit 1: a wait has given up
    while (w.left > 0) {
        const int cnt = kv_piece_tiles(w);
        const int ctx = w.len - w.n;
        // the warp's rows see no key past max_lim or before back_min, and all of those from
        // back_max to min_lim
        const int row0 = rt * 8 * NQ, back_keys = a.back;
        const int tok0 = w.r * a.tq + kv_row_token(a, row0);
        const int tok1 = min(w.r * a.tq + kv_row_token(a, min(row0 + 8 * NQ - 1, a.tq * a.group - 1)), w.n - 1);
        const bool some = row0 < a.tq * a.group && tok0 < w.n;
        const int min_lim = ctx + tok0, max_lim = some ? ctx + tok1 : -1;
        const int back_min = max(min_lim, 0) - back_keys, back_max = max(max_lim, 0) - back_keys;  // (no position before 0: no overflow)

        // Query rows as the right operand of the first product (lane: row g, 16
        // channels of each group), each scaled by the power of two that brings its
        // largest channel to [2^8, 2^9).
        uint32_t Q[4 * NG][NQ][2];
        float sc[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    top = max(max(top, v[n][i][h].x & 0x7fff7fffu), max(v[n][i][h].y & 0x7fff7fffu, max(v[n][i][h].z & 0x7fff7fffu, v[n][i][h].w & 0x7fff7fffu)));
                    top = max(top, max(max((v[n][i][h].x << 16) & 0x7fffffffu, (v[n][i][h].y << 16) & 0x7fffffffu),
                                       max((v[n][i][h].z << 16) & 0x7fffffffu, (v[n][i][h].w << 16) & 0x7fffffffu)));
                }
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));  // of row g
            int e = (int)(top >> 23);
            const bool none = e >= kNoQuery;
            e = e == 0 || none ? 0 : max(-110, e - 127);  // a row of zeros keeps 2^8
            const float f = none ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 + 8 - e) << 23);
            const float to_score = kv_score_range(a.scale_log2 * __uint_as_float((uint32_t)(127 - 8 + e) << 23));
            sc[n][0] = __shfl_sync(~0u, to_score, 8 * t);  // of rows 2t and 2t + 1
            sc[n][1] = __shfl_sync(~0u, to_score, 8 * t + 4);
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t u[4] = {v[n][i][h].x, v[n][i][h].y, v[n][i][h].z, v[n][i][h].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        Q[(i * 2 + h) * 2 + (j >> 1)][n][j & 1] = pack_half2(bf16_f32(u[j], 0) * f, bf16_f32(u[j], 1) * f);
                }
        }

        // Lane: outputs of channels kV g + 2 u + (e / 2), rows 2t + e % 2.
        constexpr int kV = D / 8;  // channels of a lane
        float O[kV / 2][NQ][4];
        float m[NQ][2], l[NQ][2];
        // A row's largest value scale so far 2^e, of the blocks that it sees (others say nothing
        // about it): probability * scale * 2^(6 - e) is at most 2^14.  up: 2^(6 - e); low: the
        // smallest e of the lane's rows, as the field of 2^e in fp32.
        RowPowers<NQ> up(127 + 6 - kKv8Low);
        uint32_t low = 127 + kKv8Low;
        // Some row goes by another factor than its scores' own (kv_score_factor).  Those
        // then stand in the second words of merge_ml, which are the warp's until the piece ends.
        bool far = false;
        float2* own_sc = merge_ml + warp * 8 * NQ + 2 * t;  // of rows 2t and 2t + 1
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            m[n][0] = m[n][1] = kNoMax;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int u = 0; u < kV / 2; ++u) O[u][n][0] = O[u][n][1] = O[u][n][2] = O[u][n][3] = 0.f;
        }

        // One step of 32 keys at `rec`, key0 on.  MASKED: some row does not see some
        // of them, or a block of 16 is not there (bit h of none).
        auto step32 = [&](auto masked_tag, const uint8_t* rec, const int key0, const uint32_t none) {
            constexpr bool MASKED = decltype(masked_tag)::value;
            const int kr = (g >> 1) + 4 * (g & 1);  // the key of fragment row g
            const uint8_t *krow = rec + kr * D, *scales = rec + 2 * kKvStep * D;
            float s[2][2][NQ][2];  // [block][rows 0-7, 8-15][query row]
            float vs[2];
            bool grow = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float S[NQ][4];
#pragma unroll
                for (int n = 0; n < NQ; ++n) S[n][0] = S[n][1] = S[n][2] = S[n][3] = 0.f;
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    uint4 c[2];  // 16 channels of the keys of rows g and g + 8 (which turn alike)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        c[j] = *reinterpret_cast<const uint4*>(krow + (16 * h + 8 * j) * D + (((t + 4 * i) ^ kv8_turn<D>(kr)) << 4));
                    const uint32_t x[4] = {c[0].x, c[0].y, c[0].z, c[0].w}, y[4] = {c[1].x, c[1].y, c[1].z, c[1].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t A[4] = {e4m3x2_half2((uint16_t)x[k]), e4m3x2_half2((uint16_t)y[k]), e4m3x2_half2((uint16_t)(x[k] >> 16)),
                                               e4m3x2_half2((uint16_t)(y[k] >> 16))};
#pragma unroll
                        for (int n = 0; n < NQ; ++n) mma_16816(S[n], A, Q[i * 4 + k][n][0], Q[i * 4 + k][n][1]);
                    }
                }
                const float2 scale = *reinterpret_cast<const float2*>(scales + 16 * h);
                // what no row sees may be anything: behind the last key, before the window, in a page that is not there
                vs[h] = !MASKED || (key0 + 16 * h <= max_lim && key0 + 16 * h + 15 >= back_min && !((none >> h) & 1u)) ? scale.y : 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v = S[n][2 * j + e] * scale.x;
                            if (MASKED) {
                                const int row = row0 + n * 8 + 2 * t + e, lim = ctx + w.r * a.tq + kv_row_token(a, row);
                                const int key = key0 + 16 * h + 8 * j + kr;
                                if (key > lim || key < max(lim, 0) - back_keys || ((none >> h) & 1u)) v = -INFINITY;
                            }
                            s[h][j][n][e] = v;
                        }
            }
            auto largest = [&](int n, int e) { return fmaxf(fmaxf(s[0][0][n][e], s[0][1][n][e]), fmaxf(s[1][0][n][e], s[1][1][n][e])); };
            const uint32_t top = max(__float_as_uint(vs[0]), __float_as_uint(vs[1])) >> 23;
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) grow |= fmaf(largest(n, e), sc[n][e], -m[n][e]) > kLazy;
            if (__any_sync(~0u, grow || top > low)) {  // rare: a maximum passed the lag, or a scale a row's exponent
                bool over = far;
                low = 255;
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = largest(n, e);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
                        const float y = x * sc[n][e], nm = fmaxf(m[n][e], y), f = ex2(m[n][e] - nm);
                        m[n][e] = nm;
                        uint32_t see = top;  // of the blocks of which the row sees a key
                        if (MASKED) {
                            const int row = row0 + n * 8 + 2 * t + e, lim = ctx + w.r * a.tq + kv_row_token(a, row), from = max(lim, 0) - back_keys;
                            see = 0;
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (key0 + 16 * h <= lim && key0 + 16 * h + 15 >= from) see = max(see, __float_as_uint(vs[h]) >> 23);
                        }
                        const uint32_t was = up.field(n, e), now = min(was, 254u + 6u - min(see, 127u + kKv8High));
                        const float down = __uint_as_float((127u + now - was) << 23);
                        up.set(n, e, now);
                        low = min(low, 254u + 6u - now);
                        over |= fabsf(y) >= kFarScore && y > kNoMax;  // (-infinity: the row sees no key of these)
                        l[n][e] *= f;
#pragma unroll
                        for (int u = 0; u < kV / 2; ++u) O[u][n][e] *= f * down, O[u][n][2 + e] *= f * down;
                    }
                if (__any_sync(~0u, over)) [[unlikely]] {  // scores far from any use: see kv_score_factor
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = largest(n, e);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
                            if (!far) own_sc[n * 8 + e].y = sc[n][e];  // (the same from a row's eight lanes)
                            __syncwarp();
                            if (m[n][e] == x * sc[n][e]) {
                                sc[n][e] = kv_score_factor(x, own_sc[n * 8 + e].y);
                                m[n][e] = x * sc[n][e];
                            }
                        }
                    far = true;
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t B[NQ][2];
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const float ke[2] = {vs[h] * up(n, 0), vs[h] * up(n, 1)};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            x[e] = ex2(fmaf(s[h][j][n][e], sc[n][e], -m[n][e]));
                            l[n][e] += x[e];
                        }
                        B[n][j] = transpose_8x8(pack_half2(x[0] * ke[0], x[1] * ke[1]));
                    }
                }
                // the codes of keys t, t + 4, t + 8 and t + 12: kV channels from kV g on
                constexpr int kW = kV / 4;
                uint32_t c[4][kW];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int o = t + 4 * e, turn = kv8_turn<D>(o);
                    const uint8_t* pv = rec + (kKvStep + 16 * h + o) * D;
                    if (D == 128)
                        *reinterpret_cast<uint4*>(c[e]) = *reinterpret_cast<const uint4*>(pv + ((g ^ turn) << 4));
                    else
                        *reinterpret_cast<uint2*>(c[e]) = *reinterpret_cast<const uint2*>(pv + (((g >> 1) ^ turn) << 4) + (g & 1) * 8);
                }
                // Where some row does not see all of the keys, a code that is NaN (behind the last
                // token anything may stand) is taken out: its probability of 0 would make
                // NaN of a row that does not see it.
                uint32_t nan = 0;
                auto seen = [&](int o) {  // by some row
                    const int key = key0 + 16 * h + o;
                    return key <= max_lim && key >= back_min && !((none >> h) & 1u);
                };
                auto nan_bytes = [](uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
                if (MASKED) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int k = 0; k < kW; ++k) {
                            const uint32_t x = seen(t + 4 * e) ? c[e][k] : 0u, b = nan_bytes(x);
                            c[e][k] = x & ~((b >> 7) * 255u);
                            nan |= b;
                        }
                }
#pragma unroll
                for (int k = 0; k < kW; ++k)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t x = __byte_perm(c[0][k], c[1][k], q ? 0x7362 : 0x5140);
                        const uint32_t y = __byte_perm(c[2][k], c[3][k], q ? 0x7362 : 0x5140);
                        const uint32_t A[4] = {e4m3x2_half2((uint16_t)x), e4m3x2_half2((uint16_t)(x >> 16)), e4m3x2_half2((uint16_t)y),
                                               e4m3x2_half2((uint16_t)(y >> 16))};
#pragma unroll
                        for (int n = 0; n < NQ; ++n) mma_16816(O[2 * k + q][n], A, B[n][0], B[n][1]);
                    }
                // The rows that do see one get theirs from a product of the places that hold one
                // with the places that a row sees.
                if (MASKED && __any_sync(~0u, nan)) [[unlikely]] {
                    uint32_t see[NQ][2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
                            see[n][j] = transpose_8x8((s[h][j][n][0] != -INFINITY ? 0x3c00u : 0u) | (s[h][j][n][1] != -INFINITY ? 0x3c000000u : 0u));
                    auto ones = [](uint32_t two) { return (two & 0x80u ? 0x3c00u : 0u) | (two & 0x8000u ? 0x3c000000u : 0u); };
                    uint64_t hit = 0;  // four bits a product and set of eight rows
#pragma unroll 1
                    for (int k = 0; k < kW; ++k) {
                        uint32_t b[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int o = t + 4 * e, at = D == 128 ? g : g >> 1;
                            const uint8_t* pv = rec + (kKvStep + 16 * h + o) * D + ((at ^ kv8_turn<D>(o)) << 4) + (D == 128 ? 0 : (g & 1) * 8);
                            b[e] = seen(o) ? nan_bytes(reinterpret_cast<const uint32_t*>(pv)[k]) : 0u;
                        }
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint32_t x = __byte_perm(b[0], b[1], q ? 0x7362 : 0x5140), y = __byte_perm(b[2], b[3], q ? 0x7362 : 0x5140);
                            const uint32_t A[4] = {ones(x), ones(x >> 16), ones(y), ones(y >> 16)};
#pragma unroll
                            for (int n = 0; n < NQ; ++n) {
                                float count[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_16816(count, A, see[n][0], see[n][1]);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (count[e] > 0.f) hit |= 1ull << (((2 * k + q) * NQ + n) * 4 + e);
                            }
                        }
                    }
#pragma unroll
                    for (int u = 0; u < kV / 2; ++u)
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if ((hit >> ((u * NQ + n) * 4 + e)) & 1u) O[u][n][e] = __uint_as_float(0x7fc00000u);
                }
            }
        };

        const int end = (w.lo + w.tile + cnt) * kKvTile;
#pragma unroll 1
        for (int key0 = (w.lo + w.tile) * kKvTile + kw * kKvStep; key0 < end; key0 += KW * kKvStep) {
            const uint32_t none = (gone >> (2 * slot)) & 3u;
            // A wait that gives up (the error word is set) ends this warp's loads and
            // sums; it still meets the others where they wait for it.
            if (phase >= 2) break;
            if (!warp_wait(full + slot, phase)) {
                phase |= 2;
                break;
            }
            if (none != 3u && key0 <= max_lim && key0 + kKvStep > back_min) {
                const uint8_t* rec = ring + slot * C::kSlotBytes;
                if (none || key0 + kKvStep - 1 > min_lim || key0 < back_max)
                    step32(std::true_type(), rec, key0, none);
                else
                    step32(std::false_type(), rec, key0, none);
            }
            if (++slot == C::kSlots) slot = 0, phase ^= 1;
            __syncwarp();
            load();
        }

        // ---- the piece's sums: over the lanes of a row, then over the key warps
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(~0u, l[n][e], o);
        if (far) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) m[n][e] = kv_whole_max(m[n][e], sc[n][e], own_sc[n * 8 + e].y);
            __syncwarp();
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float back_to = __uint_as_float((254u << 23) - __float_as_uint(up(n, e)));  // 2^(e - 6)
#pragma unroll
                for (int u = 0; u < kV / 2; ++u) O[u][n][e] *= back_to, O[u][n][2 + e] *= back_to;
            }
        // The key warps' sums meet in shared memory; then a warp takes a row at a time,
        // adds them in the order of the warps and writes the row, as output or as a piece.
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int at = warp * 8 * NQ + n * 8 + 2 * t + e;
#pragma unroll
                for (int u = 0; u < kV / 2; u += 2)
                    *reinterpret_cast<float4*>(merge + at * C::kLine + g * kV + u * 2) =
                        make_float4(O[u][n][e], O[u][n][2 + e], O[u + 1][n][e], O[u + 1][n][2 + e]);
                if (g == 0) merge_ml[at] = make_float2(m[n][e], l[n][e]);
            }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kWarps) : "memory");
        KvWalk& coming = comings[warp];
        {
            KvWalk n = w;
            kv_next_piece(a, qs, ls, n);
            coming = n;
            __syncwarp();
            fetch_q(coming);
        }
        const bool whole = cnt == w.tiles;
        const int rows = min(a.tq, w.n - w.r * a.tq) * a.group;
        const size_t piece = (2 * (size_t)blockIdx.x + (w.tile == 0 ? 1 : 0)) * a.rows;
#pragma unroll 1
        for (int row = warp; row < rows; row += C::kWarps) {
            constexpr int V = D / 32;
            using Vec = typename std::conditional<V == 4, float4, float2>::type;
            const int from = (row / (8 * NQ)) * KW * 8 * NQ + row % (8 * NQ);
            float2 ml[KW];
            float top = kNoMax, sum = 0.f, acc[V];
#pragma unroll
            for (int i = 0; i < KW; ++i) {
                ml[i] = merge_ml[from + i * 8 * NQ];
                top = fmaxf(top, ml[i].x);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
            for (int i = 0; i < KW; ++i) {
                const float f = ex2(ml[i].x - top);
                const Vec y = reinterpret_cast<const Vec*>(merge + (from + i * 8 * NQ) * C::kLine)[lane];
                sum = fmaf(f, ml[i].y, sum);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = fmaf(f, reinterpret_cast<const float*>(&y)[e], acc[e]);
            }
            if (whole) {
                const int in_tile = kv_row_token(a, row);
                const float inv = sum != 0.f ? 1.f / sum : 0.f;
                uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + (long long)(w.row0 + w.r * a.tq + in_tile) * a.o_st +
                                                            (long long)(w.head * a.group + row - in_tile * a.group) * a.o_sh) + lane * (V / 2);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const __nv_bfloat162 z = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
                    dst[e] = *reinterpret_cast<const uint32_t*>(&z);
                }
            } else {
                Vec o;
#pragma unroll
                for (int e = 0; e < V; ++e) reinterpret_cast<float*>(&o)[e] = acc[e];
                reinterpret_cast<Vec*>(a.part_o + (piece + row) * D)[lane] = o;
                if (lane == 0) a.part_ml[piece + row] = make_float2(top, sum);
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kWarps) : "memory");
        if (!whole) {
            const KvPieces of = kv_pieces<KvBound::kShortLine>(a, w, total);
            auto meet = []() { asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kWarps) : "memory"); };
            join_pieces_in_runs(of, a.joined, tid == 0, &join_last, meet, [&](int first, int step, int count, bool final) {
                // (no copy is under way then, but where a wait gave up)
                if (coming.left == 0 && join_bytes<D>(count, rows) <= C::kRingBytes + C::kMergeBytes) {
                    add_pieces_at_end<D, 32 * C::kWarps>(a, w, smem, bars + 31, joins++ & 1, of.c, first, step, count, rows, final, meet);
                    return;
                }
                add_pieces<D, C::kJoinSets, 8 / C::kJoinSets>(a, w, warp, C::kWarps, 0, rows, of.c, first, step, count, final);
            });
        }
        __syncwarp();
        w = coming;
        __syncwarp();
    }
    // After a wait gave up no step was taken and no copy asked for: from `slot`, whose
    // copies that wait was for, to in_slot (all of the ring where they are the same) they
    // may still be under way, and the shared memory is the next CTA's.
    if (phase >= 2) {
        do {
            mbar_wait(full + slot, phase & 1);
            if (++slot == C::kSlots) slot = 0, phase ^= 1;
        } while (slot != in_slot);
    }
}

template <int D, int NQ, int RT, int KW>
int launch_decode8(KvAttnArgs& a, int sms, cudaStream_t s) {
    using C = Decode8Cfg<D, NQ, RT, KW>;
    const int smem = C::smem(a.n_seqs);
    const int st = hs_host::set_smem_attr((const void*)kv8_decode_kernel<D, NQ, RT, KW>, C::smem(kKvMaxSeqs));
    if (st != HS_OK) return st;
    a.rows = C::kRows;
    a.tq = C::kRows / a.group;
    a.min_units = 2;
    a.tile_log2 = 6;
    a.pad = RT == 1 ? 6 : 8;
    // Up to 16 pieces of an item are joined in one round, more in two, which costs as much as eight
    // warps take for some ten tiles: few and short items are cut in 12 (one request of 4096 tokens with
    // two kv heads 11.8 instead of 13.1 us, two of 8000 13.2 instead of 13.8).
    if (KW == 8) {
        const uint32_t items = (uint32_t)a.n_seqs * (uint32_t)a.g.heads;
        a.short_line = items * (uint32_t)(a.pad + 128);
        a.short_ctas = 12 * items;
    }
    // A CTA for itself takes an item of 8 tiles in 7.1 us where cutting and joining it takes 8.0, one of
    // 16 in 10.3 and 8.4; eight warps one of 16 in 10.0 and 10.7.
    a.whole_tiles = KW == 8 ? 17 : 10;
    const int ctas = std::min(152, sms) * C::kCtas;
    static_assert(2 * 152 * C::kCtas * C::kRows <= kKvWsRows && 152 * C::kCtas <= kKvMaxCtas, "workspace");
    static_assert(kKvTile + 31 * KW * kKvStep + 16 <= kKvAhead, "32 table entries of a warp's steps, from any key of a row's last tile");
    if (!kv_line_ok(a)) return HS_ERR_UNSUPPORTED_SHAPE;
    if (hs_host::launch_pdl(kv8_decode_kernel<D, NQ, RT, KW>, dim3(ctas), dim3(C::kThreads), smem, s, a) != cudaSuccess)
        return HS_ERR_CUDA;
    return HS_OK;
}

// Row tiles of 8, 16, 32 or 64: the smallest that holds a request's rows.  Up to sixteen
// rows of few or of short items are shared by eight warps along the keys, one CTA an SM in place of
// two: half as many pieces to join, room to join 16 of them in shared memory, and a short item done in half the
// steps.  us, against four (16 and 4 rows of a kv head): 2 items of 131,071 keys 24.6 and 27.3,
// of 8000 13.2 and 16.6 (4 rows 10.5 and 11.3), of 500 7.7 and 10.0 (6.0 and 7.1); 128 items of up to 1000 11.1 and
// 15.2 (9.2 and 12.2); but 32 items of up to 4000 17.4 and 16.6 (14.3 and 12.0), 128 of up to 2000 22.2
// and 19.4 (17.8 and 15.4), and up to 128 keys 5.8 and 5.6.  At 64 channels registers hold 32 rows
// a warp: 64 windowed items of 18 rows and 1000 keys 13.3 and 14.6 (of up to 4000 keys 21.5 and
// 20.5).  The host knows the tables' width and the window only, not the lengths.
template <int D>
int launch_rows8(KvAttnArgs& a, long long rows, int window, int sms, cudaStream_t s) {
    const int items = a.n_seqs * a.g.heads, width = a.width << a.g.page_log2, keys = window ? std::min(width, window) : width;
    const bool brief = items <= std::min(152, sms) && keys <= 1024;
    if (rows <= 16 && keys > 128 && (items <= 16 || brief))
        return rows <= 8 ? launch_decode8<D, 1, 1, 8>(a, sms, s) : launch_decode8<D, 2, 1, 8>(a, sms, s);
    if constexpr (D == 64)
        if (rows > 16 && rows <= 32 && brief) return launch_decode8<D, 4, 1, 8>(a, sms, s);
    if (rows <= 8) return launch_decode8<D, 1, 1, 4>(a, sms, s);
    if (rows <= 16) return launch_decode8<D, 2, 1, 4>(a, sms, s);
    if (rows <= 32) return launch_decode8<D, 2, 2, 4>(a, sms, s);
    return launch_decode8<D, 2, 4, 2>(a, sms, s);
}

}  // namespace hs

using namespace hs_host;

// Rows of a request (new tokens x query heads of a kv head) that the few-row kernel takes: 32, and 64
// of short or few items, whose start is shorter here.  us, this kernel and the chunk kernel, 40 to 64 rows of 128
// channels: 32 items of up to 300 keys 12.9 and 13.8, of 1000 18.5 and 22, of 2000 21.8 and 22.9, but of 4000 28 and 26.9;
// 48 items of 1000 19.9 and 22.1, but 64 of 700 20.8 and 18.7; 4 items of 16,000 33.2 and 35.5.  More than 32 requests, where the chunk kernel
// gives no item to a CTA whole: 128 items of 300 20 and 26, of 700 26 and 28.7, 512 items of 1000 77 and 72.
constexpr int kFewRows = 32, kFewRowsShort = 64;

// The tensor-core kernel for chunks (hs_kv8_prefill.cu), and its device error word.
int hs_kv8_prefill(hs::KvAttnArgs a, int dim, int sms, cudaStream_t stream);
unsigned hs_kv8_prefill_take_status();

// Counters of arrived pieces, (maximum, sum) pairs and partial sums of the widest launch.
static size_t kv8_ws_bytes(int dim) {
    const size_t rows = hs::kKvWsRows;
    return round_up(3 * hs::kKvMaxCtas * 4, 256) + round_up(rows * 8, 256) + rows * dim * 4;
}

extern "C" size_t hs_kv8_attention_workspace_size(const hs_kv8_cache* c, int n_seqs, int n_q_heads) {
    if (!c || !kv8_shape_ok(c) || n_seqs < 1 || n_seqs > hs::kKvMaxSeqs || n_q_heads < c->n_kv_heads ||
        n_q_heads % c->n_kv_heads || n_q_heads / c->n_kv_heads > 64)
        return 0;
    return kv8_ws_bytes(c->head_dim);
}

extern "C" int hs_kv8_attention(const hs_kv8_cache* cache, const uint16_t* q, long long q_st, long long q_sh,
                                const int* q_start, const int* seq_len, const int* table, int table_width, int n_seqs,
                                int n_tokens, int n_q_heads, int max_new, float scale, int window, uint16_t* out,
                                long long o_st, long long o_sh, void* ws, size_t ws_bytes, hs_stream_t stream) {
    const int st = kv8_check(cache);
    if (st != HS_OK) return st;
    if (!q || !q_start || !seq_len || !table || !out || table_width < 1 || n_seqs < 1 || n_tokens < 0 || max_new < 0 ||
        window < 0 || !(scale > 0.f) || scale > 1e30f)
        return HS_ERR_INVALID_ARG;
    if (n_q_heads < cache->n_kv_heads || n_q_heads % cache->n_kv_heads || n_q_heads / cache->n_kv_heads > 64 ||
        n_seqs > hs::kKvMaxSeqs || (long long)table_width * cache->page_tokens > hs::kKvMaxKeys)
        return HS_ERR_UNSUPPORTED_SHAPE;
    if (!al16(q) || !al16(out) || (q_st | q_sh | o_st | o_sh) & 7 || !al4(q_start) || !al4(seq_len) || !al4(table))
        return HS_ERR_MISALIGNED;
    if (!ws || ws_bytes < kv8_ws_bytes(cache->head_dim)) return HS_ERR_WORKSPACE;
    if (!al16(ws)) return HS_ERR_MISALIGNED;
    if (!n_tokens) return HS_OK;
    const int sms = sm_count();
    if (!sms) return HS_ERR_CUDA;
    const int dim = cache->head_dim;
    const size_t rows = hs::kKvWsRows;
    uint8_t* w = static_cast<uint8_t*>(ws);
    hs::KvAttnArgs a = {};
    a.g = kv8_geom(cache);
    a.q = q, a.q_st = q_st, a.q_sh = q_sh;
    a.out = out, a.o_st = o_st, a.o_sh = o_sh;
    a.q_start = q_start, a.seq_len = seq_len, a.table = table;
    a.width = table_width, a.n_seqs = n_seqs, a.n_tokens = n_tokens;
    a.group = n_q_heads / cache->n_kv_heads;
    a.group_inv = (65536u + (uint32_t)a.group - 1u) / (uint32_t)a.group;
    a.back = window ? window - 1 : INT32_MAX;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.joined = reinterpret_cast<int*>(w);
    w += round_up(3 * hs::kKvMaxCtas * 4, 256);
    a.part_ml = reinterpret_cast<float2*>(w);
    a.part_o = reinterpret_cast<float*>(w + round_up(rows * 8, 256));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const long long need = std::max((long long)max_new, 1ll) * a.group;
    const long long items = (long long)n_seqs * a.g.heads, width = (long long)a.width << a.g.page_log2;
    const long long keys = window ? std::min<long long>(width, window) : width;  // that a row may see
    const bool brief = keys <= (n_seqs > 32 ? 768 : 384) || (items <= 48 && keys <= 2048) || (items <= 16 && items * keys <= 1 << 17);
    if (need > (brief ? kFewRowsShort : kFewRows)) return hs_kv8_prefill(a, dim, sms, s);
    const int r = dim == 64 ? hs::launch_rows8<64>(a, need, window, sms, s) : hs::launch_rows8<128>(a, need, window, sms, s);
    return r != HS_OK ? r : launch_err();
}

// Reads and clears this translation unit's device error word.
unsigned hs_kv8_take_status() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, hs::g_status, sizeof(v)) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(hs::g_status, &zero, sizeof(zero));
    return v | hs_kv8_prefill_take_status();
}
