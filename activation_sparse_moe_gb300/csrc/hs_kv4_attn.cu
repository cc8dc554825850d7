// Attention of new tokens over the 4-bit key/value cache, GB300 (sm_103a):
// the kernel for few query rows (decode, verification of drafts).  Contract: hs_kv4_attention in hs.h.
//
// Mathematics.  With k_j = s_jg c_jd + b_jg (g the channel's group of 64),
//   q . k_j = sum_g s_jg (q . c_j)_g + b_jg (sum of q over g),
// so the matrix product runs on the codes themselves, and a key's scales act
// on one number per row.  The values' scales fold into the probabilities,
//   o_d = sum_j (p_j s_jg) c_jd + sum_j p_j b_jg,
// the first sum a matrix product on codes, the second one number per (row,
// group).  A code becomes an fp16 operand by masking alone: the four bits of
// nibble 0 (of each half of a word) are the subnormal c * 2^-24 and those of
// nibble 1 c * 2^-20, exact, five logic instructions for eight codes; the
// powers of two go into q (per channel) and the output.  Each query row is scaled
// by the power of two that brings its largest channel near 1, whatever stands in
// the others: bf16 values then lose nothing as fp16, unless they are 2^25 times
// smaller than that channel.
//
// Bounds.  Instructions of the steps: taking 32 keys' codes apart, the products'
// issue and the exponentials, about half the issue slots; the integer pipe is
// the busiest.  64 decode requests of up to 8192 tokens (32 / 8 heads of 128
// channels, 316 MB of rows): 68 us, 4.7 TB/s, 69% of the copy bandwidth.  One of
// 131,071 tokens (32 / 2 heads): 24.8 us, of which the steps take 9.5 and the
// joins of 152 pieces a head about 8.
#include <type_traits>

#include "hs_kv4_join.cuh"

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
struct DecodeCfg {
    static constexpr int kNg = D / 64;
    static constexpr int kCtas = RT > 1 ? 1 : NQ == 1 ? 3 : 2;  // resident on an SM
    static constexpr int kSlots = 3;  // steps of a warp's ring
    static constexpr int kSlotBytes = kv_record_bytes(kKvStep, D);
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
// steps full: a lane issues the bulk copies of K codes, V codes, K pairs and V
// pairs as soon as the warp has used a slot up, across the ends of items.  So the warps do not wait for one another until an
// item ends (a ring shared by the CTA's warps held them in step: 30% of the
// issue slots went into waiting).
//
// Both products have the cache on the left: scores (16 keys x 8 rows) = K q^T
// and outputs (channels x 8 rows) = V^T p^T, so that a word of codes taken
// apart once serves all rows, and eight rows do not pay for sixteen.  The
// scores' fragment becomes the second product's right operand by one 8 x 8
// transposition.  Row r (0..7) of a key block stands for key r / 2 + 4 (r % 2):
// the four lanes of a group then read neighbouring rows of V.  The k index of
// the first product runs over the channels in the order in which the nibbles
// of a word come apart.
template <int D, int NQ, int RT, int KW>
__global__ void __launch_bounds__(32 * RT * KW, (DecodeCfg<D, NQ, RT, KW>::kCtas)) kv4_decode_kernel(const KvAttnArgs a) {
    using C = DecodeCfg<D, NQ, RT, KW>;
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
    static_assert(C::kWarps * C::kSlots <= 32, "barriers");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rt = warp / KW, kw = warp % KW, g = lane >> 2, t = lane & 3;  // fragment row or column, and pair

    if (tid < C::kWarps * C::kSlots) {
        mbar_init(bars + tid, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    KvWalk& w = walks[warp];
    uint32_t total;
    if (a.n_seqs <= kKvFew) {
        __syncthreads();  // the barriers are ready
        w = kv_begin_few(a, total);
    } else {
        kv_schedule(a, qs, ls, cum);
        w = kv_begin(a, qs, ls, cum);
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
        // Two pages of 16 tokens, or (part of) one: K codes, V codes, K pairs and V pairs
        // by a copy each, issued by one lane.
        const int page0 = __shfl_sync(~0u, held, at), page1 = __shfl_sync(~0u, held, at + parts_log2);
        const bool here0 = (uint32_t)page0 < (uint32_t)a.g.n_pages, here1 = (uint32_t)page1 < (uint32_t)a.g.n_pages;
        gone = (gone & ~(3u << (2 * in_slot))) | ((here0 ? 0u : 1u) | (here1 ? 0u : 2u)) << (2 * in_slot);
        if (elect_one()) {
            const uint32_t tokens = kKvStep >> parts_log2, bar = smem_u32(full + in_slot), dst = smem_u32(ring) + in_slot * C::kSlotBytes;
            mbar_arrive_expect_tx(full + in_slot, (here0 ? tokens : 0u) * (D + D / 8) + (parts_log2 && here1 ? tokens : 0u) * (D + D / 8));
            const uint64_t policy = policy_evict_first();
            auto copy_page = [&](int page, uint32_t to) {  // to: the step's token that its tokens start at
                const uint8_t* rec = src + (size_t)(uint32_t)page * (uint32_t)(a.g.heads * a.g.rec);
                const uint32_t from = key & (P - 1) & ~15u & (parts_log2 ? 0u : ~0u);
                bulk_g2s_to(dst + to * (D / 2), rec + from * (D / 2), tokens * (D / 2), bar, policy);
                bulk_g2s_to(dst + (kKvStep + to) * (D / 2), rec + (P + from) * (D / 2), tokens * (D / 2), bar, policy);
                bulk_g2s_to(dst + kKvStep * D + to * (NG * 4), rec + P * D + from * (NG * 4), tokens * (NG * 4), bar, policy);
                bulk_g2s_to(dst + kKvStep * D + (kKvStep + to) * (NG * 4), rec + P * D + (P + from) * (NG * 4), tokens * (NG * 4), bar, policy);
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
        // channels of each group), each scaled by the power of two that brings
        // its largest channel near 1.  Channels of even nibbles come times 2^12, those
        // of odd nibbles times 2^8: bf16 values of those keep all bits down to 2^-25 of
        // the largest (even ones to 2^-29), and smaller ones move a score by less than
        // 2^-33 of the largest channel's part.
        uint32_t Q[4 * NG][NQ][2];
        float sq[NG][NQ][2], sc[NQ][2];
        {
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
                // f8 = 2^(12-e), 2^e <= largest < 2^(e+1); a row of zeros keeps 2^12.  The even
                // nibbles stand for c * 2^-24, the odd ones for c * 2^-20.
                int e = (int)(top >> 23);
                const bool none = e >= kNoQuery;
                e = e == 0 || none ? 0 : max(-110, e - 127);
                const float f8 = none ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(139 - e) << 23), f4 = f8 * 0.0625f;
                const float to_score = kv_score_range(a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23) * 4096.f);
                sc[n][0] = __shfl_sync(~0u, to_score, 8 * t);  // of rows 2t and 2t + 1
                sc[n][1] = __shfl_sync(~0u, to_score, 8 * t + 4);
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    float sum = 0.f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t u[4] = {v[n][i][h].x, v[n][i][h].y, v[n][i][h].z, v[n][i][h].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) sum = fmaf(bf16_f32(u[j], 0), f8, fmaf(bf16_f32(u[j], 1), f8, sum));
#pragma unroll
                        for (int j = 0; j < 2; ++j) {  // nibbles (2j, 2j + 4) and (2j + 1, 2j + 5)
                            Q[(i * 2 + h) * 2 + j][n][0] = pack_half2(bf16_f32(u[j], 0) * f8, bf16_f32(u[j + 2], 0) * f8);
                            Q[(i * 2 + h) * 2 + j][n][1] = pack_half2(bf16_f32(u[j], 1) * f4, bf16_f32(u[j + 2], 1) * f4);
                        }
                    }
                    sum += __shfl_xor_sync(~0u, sum, 1);
                    sum += __shfl_xor_sync(~0u, sum, 2);
                    sum *= 1.f / 16777216.f;
                    sq[i][n][0] = __shfl_sync(~0u, sum, 8 * t);
                    sq[i][n][1] = __shfl_sync(~0u, sum, 8 * t + 4);
                }
            }
        }

        // Lane: outputs of channels 64 i + 8 g + 2 u + (e / 2), rows 2t + e % 2.
        float O[NG][4][NQ][4];
        float m[NQ][2], l[NQ][2], bs[NG][NQ][2];
        // Exponent field of the largest value scale so far: probability * scale *
        // 2^(21 - eb) stays below 2^15.
        uint32_t eb = 0;
        // Some row goes by another factor than its scores' own (kv_score_factor).  Those
        // then stand in the second words of merge_ml, which are the warp's until the piece ends.
        bool far = false;
        float2* own_sc = merge_ml + warp * 8 * NQ + 2 * t;  // of rows 2t and 2t + 1
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            m[n][0] = m[n][1] = kNoMax;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                bs[i][n][0] = bs[i][n][1] = 0.f;
#pragma unroll
                for (int u = 0; u < 4; ++u) O[i][u][n][0] = O[i][u][n][1] = O[i][u][n][2] = O[i][u][n][3] = 0.f;
            }
        }

        // One step of 32 keys at `rec`, key0 on.  MASKED: some row does not see some
        // of them, or a block of 16 is not there (bit h of none).
        auto step32 = [&](auto masked_tag, const uint8_t* rec, const int key0, const uint32_t none) {
            constexpr bool MASKED = decltype(masked_tag)::value;
            constexpr int kV = kKvStep * D / 2, kKp = kKvStep * D, kVp = kKvStep * (D + NG * 4);
            const int kr = (g >> 1) + 4 * (g & 1);  // the key of fragment row g
            float S[2][NG][NQ][4];
            uint32_t kp[2][2][NG], vp[2][2][NG];  // the pairs of the keys of rows g and g + 8
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint2 kc[2][NG];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < NG; ++i)
                        kc[j][i] = *reinterpret_cast<const uint2*>(rec + (16 * h + 8 * j + kr) * (D / 2) + i * 32 + t * 8);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint8_t* pk = rec + (16 * h + 8 * j + kr) * (NG * 4);
                    // what lies behind the last key may be anything
                    const bool there = !MASKED || (key0 + 16 * h + 8 * j + kr < w.len && !((none >> h) & 1u));
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        kp[h][j][i] = there ? reinterpret_cast<const uint32_t*>(pk + kKp)[i] : 0;
                        vp[h][j][i] = there ? reinterpret_cast<const uint32_t*>(pk + kVp)[i] : 0;
                    }
                }
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int n = 0; n < NQ; ++n) S[h][i][n][0] = S[h][i][n][1] = S[h][i][n][2] = S[h][i][n][3] = 0.f;
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        uint32_t x = c ? kc[0][i].y : kc[0][i].x, y = c ? kc[1][i].y : kc[1][i].x;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t A[4] = {x & 0x000f000fu, y & 0x000f000fu, x & 0x00f000f0u, y & 0x00f000f0u};
#pragma unroll
                            for (int n = 0; n < NQ; ++n)
                                mma_16816(S[h][i][n], A, Q[(i * 2 + c) * 2 + j][n][0], Q[(i * 2 + c) * 2 + j][n][1]);
                            x >>= 8;
                            y >>= 8;
                        }
                    }
            }
            float s[2][2][NQ][2];  // [block][rows 0-7, 8-15][query row]
            bool grow = false;
            uint32_t top = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float2 p[NG];
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        p[i] = half2_to_float2(kp[h][j][i]);
                        top = max(top, vp[h][j][i] & 0x7c00u);
                    }
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v = p[0].y * sq[0][n][e];
#pragma unroll
                            for (int i = 1; i < NG; ++i) v = fmaf(p[i].y, sq[i][n][e], v);
#pragma unroll
                            for (int i = 0; i < NG; ++i) v = fmaf(p[i].x, S[h][i][n][2 * j + e], v);
                            if (MASKED) {
                                const int row = row0 + n * 8 + 2 * t + e, lim = ctx + w.r * a.tq + kv_row_token(a, row);
                                const int key = key0 + 16 * h + 8 * j + kr;
                                if (key > lim || key < max(lim, 0) - back_keys || ((none >> h) & 1u)) v = -INFINITY;
                            }
                            s[h][j][n][e] = v;
                        }
                }
            auto largest = [&](int n, int e) { return fmaxf(fmaxf(s[0][0][n][e], s[0][1][n][e]), fmaxf(s[1][0][n][e], s[1][1][n][e])); };
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) grow |= fmaf(largest(n, e), sc[n][e], -m[n][e]) > kLazy;
            if (__any_sync(~0u, grow || top > eb << 10)) {  // rare: a maximum passed the lag, or a scale the exponent
                const uint32_t neb = max(eb, warp_max_u32(top) >> 10);
                const float down = __uint_as_float((127u + eb - neb) << 23);
                eb = neb;
                bool over = far;
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = largest(n, e);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
                        const float y = x * sc[n][e], nm = fmaxf(m[n][e], y), f = ex2(m[n][e] - nm);
                        m[n][e] = nm;
                        over |= fabsf(y) >= kFarScore && y > kNoMax;  // (-infinity: the row sees no key of these)
                        l[n][e] *= f;
#pragma unroll
                        for (int i = 0; i < NG; ++i) {
                            bs[i][n][e] *= f;
#pragma unroll
                            for (int u = 0; u < 4; ++u) O[i][u][n][e] *= f * down, O[i][u][n][2 + e] *= f * down;
                        }
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
                const float ke = __uint_as_float((148u - eb) << 23);
                uint32_t B[NG][NQ][2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float2 p[NG];
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        p[i] = half2_to_float2(vp[h][j][i]);
                        p[i].x *= ke;
                    }
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        float x[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            x[e] = ex2(fmaf(s[h][j][n][e], sc[n][e], -m[n][e]));
                            l[n][e] += x[e];
                        }
#pragma unroll
                        for (int i = 0; i < NG; ++i) {
                            float y[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const bool hide = MASKED && s[h][j][n][e] == -INFINITY;  // a key that the row does not see may hold a NaN
                                bs[i][n][e] = hide ? bs[i][n][e] : fmaf(x[e], p[i].y, bs[i][n][e]);
                                y[e] = hide ? 0.f : x[e] * p[i].x;
                            }
                            B[i][n][j] = transpose_8x8(pack_half2(y[0], y[1]));
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    const uint8_t* pv = rec + kV + (16 * h + t) * (D / 2) + i * 32 + g * 4;
                    uint32_t c[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = *reinterpret_cast<const uint32_t*>(pv + 4 * e * (D / 2));
#pragma unroll
                    for (int hw = 0; hw < 2; ++hw) {
                        uint32_t x = __byte_perm(c[0], c[1], hw ? 0x7632 : 0x5410);
                        uint32_t y = __byte_perm(c[2], c[3], hw ? 0x7632 : 0x5410);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t A[4] = {x & 0x000f000fu, x & 0x00f000f0u, y & 0x000f000fu, y & 0x00f000f0u};
#pragma unroll
                            for (int n = 0; n < NQ; ++n) mma_16816(O[i][2 * hw + j][n], A, B[i][n][0], B[i][n][1]);
                            x >>= 8;
                            y >>= 8;
                        }
                    }
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
                for (int o = 4; o < 32; o <<= 1) {
                    l[n][e] += __shfl_xor_sync(~0u, l[n][e], o);
#pragma unroll
                    for (int i = 0; i < NG; ++i) bs[i][n][e] += __shfl_xor_sync(~0u, bs[i][n][e], o);
                }
        if (far) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) m[n][e] = kv_whole_max(m[n][e], sc[n][e], own_sc[n * 8 + e].y);
            __syncwarp();
        }
        const float even = __uint_as_float((uint32_t)(127 + 24 - 21 + (int)eb) << 23);  // 2^24 / 2^(21 - eb)
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        O[i][u][n][e] = fmaf(O[i][u][n][e], e < 2 ? even : even * 0.0625f, bs[i][n][e & 1]);
        // The key warps' sums meet in shared memory; then a warp takes a row at a time,
        // adds them in the order of the warps and writes the row, as output or as a piece.
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int at = warp * 8 * NQ + n * 8 + 2 * t + e;
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int u = 0; u < 4; u += 2)
                        *reinterpret_cast<float4*>(merge + at * C::kLine + i * 64 + g * 8 + u * 2) =
                            make_float4(O[i][u][n][e], O[i][u][n][2 + e], O[i][u + 1][n][e], O[i][u + 1][n][2 + e]);
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
            const KvPieces of = kv_pieces(a, w, total);
            auto meet = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kWarps) : "memory"); };
            join_pieces(of, a.joined, tid == 0, &join_last, meet, [&](int first, int step, int count, bool final) {
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
int launch_decode(KvAttnArgs& a, int sms, cudaStream_t s) {
    using C = DecodeCfg<D, NQ, RT, KW>;
    const int smem = C::smem(a.n_seqs);
    const int st = hs_host::set_smem_attr((const void*)kv4_decode_kernel<D, NQ, RT, KW>, C::smem(kKvMaxSeqs));
    if (st != HS_OK) return st;
    a.rows = C::kRows;
    a.tq = C::kRows / a.group;
    a.min_units = 2;
    a.tile_log2 = 6;
    // An item's own time in tiles, for 64 ragged decode requests and 33 windowed ones: 6, 8 and 10 take
    // 71.2, 71.6 and 73.3 us, 11.2, 11.4 and 11.4 us; none at all took 91.0 instead of 77.3 us, 17.7
    // instead of 13.7 us. Two row tiles' tiles take longer: 4 gave 29.7 us for 48 rows, 8 gave 30.9 us.
    a.pad = RT == 1 ? 6 : 4;
    const int ctas = std::min(152, sms) * C::kCtas;
    static_assert(2 * 152 * C::kCtas * C::kRows <= kKvWsRows && 152 * C::kCtas <= kKvMaxCtas, "workspace");
    if (!kv_line_ok(a)) return HS_ERR_UNSUPPORTED_SHAPE;
    if (hs_host::launch_pdl(kv4_decode_kernel<D, NQ, RT, KW>, dim3(ctas), dim3(C::kThreads), smem, s, a) != cudaSuccess)
        return HS_ERR_CUDA;
    return HS_OK;
}

// Row tiles of 8, 16, 32 or 64: the smallest that holds a request's rows.
template <int D>
int launch_rows(KvAttnArgs& a, long long rows, int sms, cudaStream_t s) {
    if (rows <= 8) return launch_decode<D, 1, 1, 4>(a, sms, s);
    if (rows <= 16) return launch_decode<D, 2, 1, 4>(a, sms, s);
    if (rows <= 32) return launch_decode<D, 2, 2, 4>(a, sms, s);
    return launch_decode<D, 2, 4, 2>(a, sms, s);
}

}  // namespace hs

using namespace hs_host;

// Rows of a request (new tokens x query heads of a kv head) from which the
// chunk kernel is used.  This kernel against that one, us: 32 rows, 16 requests
// (32 / 2 heads) 18.2 and 20.7, one 15.8 and 26.0, 64 (32 / 8 heads) 104 and 134; 24 rows 37 and
// 46.  With 48 rows, four row warps take the same codes apart, which costs where
// there is much to read (16 requests, 32 / 8 heads: 56 and 41; one of 131,000
// tokens 60 and 51) and does not where the start and the joins bound the call: one request of
// 4096 tokens (32 / 2 heads) 22.8 and 29.1, four 25.0 and 29.2, eight of 1000 tokens 17.1 and
// 19.2.  So up to 64 rows stay here if requests x kv heads are at most 16 and the
// tables hold no more than 2^17 keys of them.  The host knows the tables' width only, not
// the lengths: short requests in tables made for long contexts go to the chunk kernel.
constexpr int kPrefillRows = 33;

// Counters of arrived pieces, (maximum, sum) pairs and partial sums of the widest launch.
static size_t kv4_ws_bytes(int dim) {
    const size_t rows = hs::kKvWsRows;
    return round_up(3 * hs::kKvMaxCtas * 4, 256) + round_up(rows * 8, 256) + rows * dim * 4;
}

extern "C" size_t hs_kv4_attention_workspace_size(const hs_kv4_cache* c, int n_seqs, int n_q_heads) {
    if (!c || !kv4_shape_ok(c) || n_seqs < 1 || n_seqs > hs::kKvMaxSeqs || n_q_heads < c->n_kv_heads ||
        n_q_heads % c->n_kv_heads || n_q_heads / c->n_kv_heads > 64)
        return 0;
    return kv4_ws_bytes(c->head_dim);
}

extern "C" int hs_kv4_attention(const hs_kv4_cache* cache, const uint16_t* q, long long q_st, long long q_sh,
                                const int* q_start, const int* seq_len, const int* table, int table_width, int n_seqs,
                                int n_tokens, int n_q_heads, int max_new, float scale, int window, uint16_t* out,
                                long long o_st, long long o_sh, void* ws, size_t ws_bytes, hs_stream_t stream) {
    const int st = kv4_check(cache);
    if (st != HS_OK) return st;
    if (!q || !q_start || !seq_len || !table || !out || table_width < 1 || n_seqs < 1 || n_tokens < 0 || max_new < 0 ||
        window < 0 || !(scale > 0.f) || scale > 1e30f)
        return HS_ERR_INVALID_ARG;
    if (n_q_heads < cache->n_kv_heads || n_q_heads % cache->n_kv_heads || n_q_heads / cache->n_kv_heads > 64 ||
        n_seqs > hs::kKvMaxSeqs || (long long)table_width * cache->page_tokens > hs::kKvMaxKeys)
        return HS_ERR_UNSUPPORTED_SHAPE;
    if (!al16(q) || !al16(out) || (q_st | q_sh | o_st | o_sh) & 7 || !al4(q_start) || !al4(seq_len) || !al4(table))
        return HS_ERR_MISALIGNED;
    if (!ws || ws_bytes < kv4_ws_bytes(cache->head_dim)) return HS_ERR_WORKSPACE;
    if (!al16(ws)) return HS_ERR_MISALIGNED;
    if (!n_tokens) return HS_OK;
    const int sms = sm_count();
    if (!sms) return HS_ERR_CUDA;
    const int dim = cache->head_dim;
    const size_t rows = hs::kKvWsRows;
    uint8_t* w = static_cast<uint8_t*>(ws);
    hs::KvAttnArgs a = {};
    a.g = kv4_geom(cache);
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
    const long long items = (long long)n_seqs * a.g.heads, keys = items * ((long long)a.width << a.g.page_log2);
    if (need >= (items <= 16 && keys <= 1 << 17 ? 65 : kPrefillRows)) return hs_kv4_prefill(a, dim, sms, s);
    const int r = dim == 64 ? hs::launch_rows<64>(a, need, sms, s) : hs::launch_rows<128>(a, need, sms, s);
    return r != HS_OK ? r : launch_err();
}

// Reads and clears this translation unit's device error word.
unsigned hs_kv4_take_status() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, hs::g_status, sizeof(v)) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(hs::g_status, &zero, sizeof(zero));
    return v | hs_kv4_prefill_take_status();
}
