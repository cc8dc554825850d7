// Joining the pieces of an attention item that several CTAs worked on.
//
// Piece i of an item lies in slot 2 (c + i), the first one in slot 2 c + 1 of
// the CTA c in which the item began.  Up to kJoin pieces are added by the CTA
// that comes last.  More are added in runs of kJoin by the last CTA of each
// run, and the runs' sums by the CTA whose run comes last: the order is that of
// the keys either way, so the result does not depend on who comes last.  One
// launch does everything; a second kernel for the sums cost 5 to 10 us a call.
// A latency bounds this, not bytes: 152 pieces of 16 rows (1.2 MB) take about 8 us in
// two rounds; 256 rows of two pieces 20,000 cycles, which is why the chunk kernel
// adds a pair's second piece on its way out instead.
#pragma once

#include "hs_kv4_sched.cuh"

namespace hs {

constexpr int kJoin = 16;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ size_t piece_slot(int c, int i) { return i ? 2 * (size_t)(c + i) : 2 * (size_t)c + 1; }

// Of a row whose KL lanes know the (maximum, sum) of its pieces, lane i those of
// pieces i, i + KL, ...: the common maximum, the pieces' weights and the sum.
template <int KL, int KP>
__device__ __forceinline__ void weigh(float (&top)[KP], const float (&sum)[KP], int i, int count, float& m, float& l) {
#pragma unroll
    for (int o = KL / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    l = 0.f;
#pragma unroll
    for (int y = 0; y < KP; ++y) {
        top[y] = i + y * KL < count ? ex2(top[y] - m) : 0.f;
        l = fmaf(top[y], sum[y], l);
    }
#pragma unroll
    for (int o = KL / 2; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8], float scale) {
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        u[e] = (uint32_t)f32_to_bf16_bits(v[2 * e] * scale) | ((uint32_t)f32_to_bf16_bits(v[2 * e + 1] * scale) << 16);
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Adds pieces first, first + step, ... (count of them, at most 32) of the item
// that began in CTA c, their rows row0 <= row < row1: into out if `final`, else
// into piece `first`.  Called by
// whole warps, `warp` of `warps`.  D / 8 lanes take a row, eight channels each; a
// warp takes SETS sets of 32 / (D / 8) rows and BATCH pieces of each at a time,
// as many bytes in flight as its registers hold.  Lane i of a row knows the
// weight of pieces i, i + D / 8, ...
template <int D, int SETS, int BATCH>
__device__ __forceinline__ void add_pieces(const KvAttnArgs& a, const KvWalk& w, int warp, int warps, int row0, int row1, int c, int first,
                                           int step, int count, bool final) {
    constexpr int kL = D / 8, kR = 32 / kL, kP = 32 / kL;  // lanes a row, rows at a time, pieces a lane
    const int lane = threadIdx.x & 31, sub = lane / kL, i8 = lane % kL;
    // row `row` of piece i: fewer than 2^18 rows of the workspace (kKvWsRows)
    auto place = [&](int i, int row) { return (uint32_t)(piece_slot(c, first + min(i, count - 1) * step) * a.rows + row); };
    for (int s0 = warp; row0 + s0 * kR < row1; s0 += SETS * warps) {
        float wt[SETS][kP], part[SETS][kP], acc[SETS][8], m[SETS], l[SETS];
        float4 v[BATCH][SETS][2];
        int row[SETS];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
#pragma unroll
                for (int x = 0; x < SETS; ++x) {
                    const float4* src = reinterpret_cast<const float4*>(a.part_o + place(i0 + i, row[x]) * (uint32_t)D + i8 * 8);
                    v[i][x][0] = __ldcg(src);
                    v[i][x][1] = __ldcg(src + 1);
                }
        };
#pragma unroll
        for (int x = 0; x < SETS; ++x) {
            row[x] = min(row0 + (s0 + x * warps) * kR + sub, row1 - 1);
            m[x] = kNoMax;
#pragma unroll
            for (int y = 0; y < kP; ++y) {
                float2 ml = make_float2(kNoMax, 0.f);
                if (i8 + y * kL < count) ml = __ldcg(a.part_ml + place(i8 + y * kL, row[x]));
                wt[x][y] = ml.x, part[x][y] = ml.y;
                m[x] = fmaxf(m[x], ml.x);
            }
        }
        fetch(0);
#pragma unroll
        for (int x = 0; x < SETS; ++x) {
            weigh<kL, kP>(wt[x], part[x], i8, count, m[x], l[x]);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[x][e] = 0.f;
        }
        for (int i0 = 0; i0 < count; i0 += BATCH) {
            if (i0) fetch(i0);
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
#pragma unroll
                for (int x = 0; x < SETS; ++x) {
                    float mine = wt[x][0];
#pragma unroll
                    for (int y = 1; y < kP; ++y) mine = i0 + i >= y * kL ? wt[x][y] : mine;
                    float f = __shfl_sync(~0u, mine, (i0 + i) % kL, kL);
                    if (i0 + i >= count) f = 0.f;
                    const float* from = reinterpret_cast<const float*>(v[i][x]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[x][e] = fmaf(f, from[e], acc[x][e]);
                }
        }
#pragma unroll
        for (int x = 0; x < SETS; ++x) {
            if (row0 + (s0 + x * warps) * kR + sub >= row1) continue;
            if (final) {
                const float inv = l[x] != 0.f ? 1.f / l[x] : 0.f;
                const int tok = kv_row_token(a, row[x]);
                *reinterpret_cast<uint4*>(a.out + (long long)(w.row0 + w.r * a.tq + tok) * a.o_st +
                                          (long long)(w.head * a.group + row[x] - tok * a.group) * a.o_sh + i8 * 8) =
                    pack_bf16x8(acc[x], inv);
            } else {
                const uint32_t at = place(0, row[x]);
                float4* dst = reinterpret_cast<float4*>(a.part_o + at * (uint32_t)D + i8 * 8);
                dst[0] = make_float4(acc[x][0], acc[x][1], acc[x][2], acc[x][3]);
                dst[1] = make_float4(acc[x][4], acc[x][5], acc[x][6], acc[x][7]);
                if (i8 == 0) a.part_ml[at] = make_float2(m[x], l[x]);
            }
        }
    }
}

// The pieces of the item that a CTA's piece belongs to: the CTA of the first one, their number.
struct KvPieces {
    int c, count;
};
template <KvBound B = KvBound::kNone>
__device__ __forceinline__ KvPieces kv_pieces(const KvAttnArgs& a, const KvWalk& w, uint32_t total) {
    const KvCut cut = kv_cut<B>(a, total);
    // the unit with which this piece began: of the run's first item the run's, else
    // what the run has left lies before the run's end
    const uint32_t begin = w.first ? cut.at(blockIdx.x) - w.tile : cut.at(blockIdx.x + 1) - w.left, end = begin + (uint32_t)w.tiles;
    const int c = cut.cta_of(begin);
    return {c, cut.cta_of(end - 1) - c + 1};
}

// Called by the warps that have written a CTA's piece.  meet is a barrier of
// theirs, lead one thread of them, joined their counters (kKvMaxCtas apart),
// *last a word of shared memory; add(first, step, count, final) is add_pieces.
template <typename Meet, typename Add>
__device__ __forceinline__ void join_pieces(const KvPieces& of, int* joined, bool lead, int* last, Meet meet, Add add) {
    auto arrive = [&](int* counter, int wanted) -> bool {
        meet();  // the CTA's writes ...
        if (lead) {
            // ... are seen before its arrival, and the other CTAs' after the last one's
            int before;
            asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
            *last = before == wanted - 1;
            if (before == wanted - 1) *counter = 0;  // for the next call
        }
        meet();
        return *last != 0;
    };
    if (of.count <= kJoin) {
        if (arrive(joined + of.c, of.count)) add(0, 1, of.count, true);
        return;
    }
    const int run = ((int)blockIdx.x - of.c) / kJoin, size = min(kJoin, of.count - run * kJoin);
    // A run's counter is that of its first CTA; an item that begins in that CTA has another.
    if (!arrive(joined + kKvMaxCtas * (run ? 2 : 1) + of.c + run * kJoin, size)) return;
    add(run * kJoin, 1, size, false);
    const int runs = (of.count + kJoin - 1) / kJoin;
    if (arrive(joined + of.c, runs)) add(0, kJoin, runs, true);
}

}  // namespace hs
