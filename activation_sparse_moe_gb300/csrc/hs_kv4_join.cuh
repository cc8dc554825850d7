// Joining the pieces of an attention item that several CTAs worked on.
//
// Piece i of an item lies in slot 2 (c + i), the first one in slot 2 c + 1 of
// the CTA c in which the item began.  Up to kJoin pieces are added by the CTA
// that comes last.  More are added in runs of kJoin by the last CTA of each
// run, and the runs' sums by the CTA whose run comes last: the order is that of
// the keys either way, so the result does not depend on who comes last.  One
// launch does everything; a second kernel for the sums cost 5 to 10 us a call.
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

template <int N> struct FloatVec;
template <> struct FloatVec<2> { using T = float2; };
template <> struct FloatVec<4> { using T = float4; };

// Adds pieces first, first + step, ... (count of them, at most 64) of the item
// that began in CTA c: into out if `final`, else into piece `first`.  Called by
// whole warps, `warp` of WARPS; a warp takes ROWS rows of BATCH pieces at a
// time (it is latency that bounds this).
template <int D, int WARPS, int ROWS = 4, int BATCH = 4>
__device__ __forceinline__ void add_pieces(const KvAttnArgs& a, const KvWalk& w, int warp, int c, int first, int step, int count,
                                        bool final) {
    constexpr int V = D / 32;
    using Vec = typename FloatVec<V>::T;
    const int lane = threadIdx.x & 31;
    const int rows = min(a.tq, w.n - w.r * a.tq) * a.group;
    for (int r0 = warp; r0 < rows; r0 += ROWS * WARPS) {
        float m[ROWS], l[ROWS], acc[ROWS][V];
        int row[ROWS];
        if (count <= 2) {  // the commonest case: everything is read at once
            Vec v[2][ROWS];
            float2 ml[2][ROWS];
#pragma unroll
            for (int x = 0; x < ROWS; ++x) {
                row[x] = min(r0 + x * WARPS, rows - 1);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const size_t at = piece_slot(c, first + min(i, count - 1) * step) * a.rows + row[x];
                    v[i][x] = __ldcg(reinterpret_cast<const Vec*>(a.part_o + at * D) + lane);
                    ml[i][x] = __ldcg(a.part_ml + at);
                }
            }
#pragma unroll
            for (int x = 0; x < ROWS; ++x) {
                if (count == 1) ml[1][x] = make_float2(-1e30f, 0.f);
                m[x] = fmaxf(ml[0][x].x, ml[1][x].x);
                const float f0 = ex2(ml[0][x].x - m[x]), f1 = count == 1 ? 0.f : ex2(ml[1][x].x - m[x]);
                l[x] = f0 * ml[0][x].y + f1 * ml[1][x].y;
#pragma unroll
                for (int e = 0; e < V; ++e)
                    acc[x][e] = f0 * reinterpret_cast<const float*>(&v[0][x])[e] + f1 * reinterpret_cast<const float*>(&v[1][x])[e];
            }
        } else {
            // the first pieces' rows come along with all pieces' (maximum, sum)
            float wt[ROWS][2];
            Vec v[BATCH][ROWS];
            auto fetch = [&](int i0) {
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const size_t at = piece_slot(c, first + min(i0 + i, count - 1) * step) * a.rows;
#pragma unroll
                    for (int x = 0; x < ROWS; ++x) v[i][x] = __ldcg(reinterpret_cast<const Vec*>(a.part_o + (at + row[x]) * D) + lane);
                }
            };
#pragma unroll
            for (int x = 0; x < ROWS; ++x) {
                row[x] = min(r0 + x * WARPS, rows - 1);
                float2 ml[2];
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    ml[y] = lane + 32 * y < count ? __ldcg(a.part_ml + piece_slot(c, first + (lane + 32 * y) * step) * a.rows + row[x])
                                                  : make_float2(-1e30f, 0.f);
                m[x] = fmaxf(ml[0].x, ml[1].x);
                wt[x][0] = ml[0].x, wt[x][1] = ml[1].x;
                l[x] = ml[0].y, acc[x][0] = ml[1].y;
            }
            fetch(0);
#pragma unroll
            for (int x = 0; x < ROWS; ++x) {
#pragma unroll
                for (int o = 16; o; o >>= 1) m[x] = fmaxf(m[x], __shfl_xor_sync(~0u, m[x], o));
                wt[x][0] = ex2(wt[x][0] - m[x]);
                wt[x][1] = ex2(wt[x][1] - m[x]);
                l[x] = wt[x][0] * l[x] + wt[x][1] * acc[x][0];
#pragma unroll
                for (int o = 16; o; o >>= 1) l[x] += __shfl_xor_sync(~0u, l[x], o);
#pragma unroll
                for (int e = 0; e < V; ++e) acc[x][e] = 0.f;
            }
            for (int i0 = 0; i0 < count; i0 += BATCH) {
                if (i0) fetch(i0);
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
#pragma unroll
                    for (int x = 0; x < ROWS; ++x) {
                        float f = __shfl_sync(~0u, i0 + i < 32 ? wt[x][0] : wt[x][1], (i0 + i) & 31);
                        if (i0 + i >= count) f = 0.f;
#pragma unroll
                        for (int e = 0; e < V; ++e) acc[x][e] = fmaf(f, reinterpret_cast<const float*>(&v[i][x])[e], acc[x][e]);
                    }
            }
        }
#pragma unroll
        for (int x = 0; x < ROWS; ++x) {
            if (r0 + x * WARPS >= rows) continue;
            if (final) {
                const float inv = l[x] != 0.f ? 1.f / l[x] : 0.f;
                uint32_t u[V / 2];
#pragma unroll
                for (int e = 0; e < V / 2; ++e)
                    u[e] = (uint32_t)f32_to_bf16_bits(acc[x][2 * e] * inv) | ((uint32_t)f32_to_bf16_bits(acc[x][2 * e + 1] * inv) << 16);
                const int tok = kv_row_token(a, row[x]);
                uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + (long long)(w.row0 + w.r * a.tq + tok) * a.o_st +
                                                            (long long)(w.head * a.group + row[x] - tok * a.group) * a.o_sh) + lane * (V / 2);
                if (V == 4)
                    *reinterpret_cast<uint2*>(dst) = make_uint2(u[0], u[V / 2 - 1]);
                else
                    *dst = u[0];
            } else {
                const size_t at = piece_slot(c, first) * a.rows + row[x];
                Vec o;
#pragma unroll
                for (int e = 0; e < V; ++e) reinterpret_cast<float*>(&o)[e] = acc[x][e];
                reinterpret_cast<Vec*>(a.part_o + at * D)[lane] = o;
                if (lane == 0) a.part_ml[at] = make_float2(m[x], l[x]);
            }
        }
    }
}

// Called by WARPS warps (`warp` the calling one's index) of a CTA that has
// written its piece of w's item.  *last is a word of shared memory; the warps meet at named barrier BAR; add is
// add_pieces.
template <int WARPS, int BAR, typename Add>
__device__ __forceinline__ void join_pieces(const KvAttnArgs& a, const KvWalk& w, int warp, uint32_t total, int* last, Add add) {
    const KvCut cut = kv_cut(a, total);
    const int me = blockIdx.x;
    const bool lead = warp == 0 && (threadIdx.x & 31) == 0;
    // the unit with which this piece began: of the run's first item the run's, else
    // what the run has left lies before the run's end
    const uint32_t begin = w.first ? cut.at(me) - w.tile : cut.at(me + 1) - w.left, end = begin + (uint32_t)w.tiles;
    const int c = cut.cta_of(begin), pieces = cut.cta_of(end - 1) - c + 1;
    auto meet = [&]() { asm volatile("bar.sync %0, %1;" ::"n"(BAR), "n"(32 * WARPS) : "memory"); };
    auto arrive = [&](int* counter, int of) -> bool {
        meet();  // the CTA's writes ...
        if (lead) {
            // ... are seen before its arrival, and the other CTAs' after the last one's
            int before;
            asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
            *last = before == of - 1;
            if (before == of - 1) *counter = 0;  // for the next call
        }
        meet();
        return *last != 0;
    };
    if (pieces <= kJoin) {
        if (arrive(a.joined + c, pieces)) add(a, w, warp, c, 0, 1, pieces, true);
        return;
    }
    const int run = (me - c) / kJoin, size = min(kJoin, pieces - run * kJoin);
    // A run's counter is that of its first CTA; an item that begins in that CTA has another.
    if (!arrive(a.joined + kKvMaxCtas * (run ? 2 : 1) + c + run * kJoin, size)) return;
    add(a, w, warp, c, run * kJoin, 1, size, false);
    const int runs = (pieces + kJoin - 1) / kJoin;
    if (arrive(a.joined + c, runs)) add(a, w, warp, c, 0, kJoin, runs, true);
}

}  // namespace hs
