// Joining the pieces of an attention item in the few-row kernel over the 8-bit
// cache: as hs_kv4_join.cuh, whose pieces, counters and order these are, but by a
// CTA that has no work left in its shared memory.
//
// Adding pieces out of memory (add_pieces) is code that runs once or twice a call, so its
// instructions have to be fetched, and its loads come in four rounds: 16 pieces of
// 16 rows took 4 to 5 us, twice in a long decode call.  A CTA at its end has its rings
// free: there the pieces come in by bulk copies, all at once, and little loops add
// them.  The operations and their order are those of add_pieces, so that
// the result does not depend on which CTA comes last.
#pragma once

#include "hs_kv4_join.cuh"

namespace hs {

// Shared memory that adding `count` pieces of `rows` rows takes: the pieces, a weight
// for each row of each, and a row's sum.
template <int D>
__device__ __forceinline__ int join_bytes(int count, int rows) {
    return (count * D + count + 1) * rows * 4;
}

// add_pieces by the CTA's THREADS threads.  room: shared memory of join_bytes bytes, `bar`
// an mbarrier of one arrival whose next phase has this parity, meet a barrier of
// the CTA.  Called by a thread that sees what the pieces' CTAs have written.
template <int D, int THREADS, typename Meet>
__device__ __noinline__ void add_pieces_at_end(const KvAttnArgs& a, const KvWalk& w, uint8_t* room, uint64_t* bar, uint32_t parity, int c,
                                               int first, int step, int count, int rows, bool final, Meet meet) {
    constexpr int kL = D / 8, kR = 32 / kL, kP = 32 / kL;
    const int tid = threadIdx.x, lane = tid & 31, sub = lane / kL, i8 = lane % kL;
    const uint32_t bytes = (uint32_t)(rows * D * 4);
    float* weights = reinterpret_cast<float*>(room + count * bytes);  // [row][count]
    float* inv = weights + rows * count;                              // [row]: 1 / sum, or the sum
    auto slot = [&](int i) { return piece_slot(c, first + i * step) * a.rows; };
    // The last warp asks for the copies, a lane each, while the others begin with the weights.
    if (tid >= THREADS - 32) {
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes * (uint32_t)count);
        __syncwarp();
        if (lane < count) {
            asm volatile("fence.proxy.async;" ::: "memory");  // the other CTAs' writes, seen by the arrival before
            bulk_g2s(room + lane * bytes, a.part_o + slot(lane) * D, bytes, bar, policy_evict_first());
        }
        __syncwarp();
    }
#pragma unroll 1
    for (int r0 = (tid >> 5) * kR; r0 < rows; r0 += THREADS / 32 * kR) {
        float wt[kP], part[kP], m = kNoMax, l;
        const int row = min(r0 + sub, rows - 1);
#pragma unroll
        for (int y = 0; y < kP; ++y) {
            float2 ml = make_float2(kNoMax, 0.f);
            if (i8 + y * kL < count) ml = __ldcg(a.part_ml + slot(i8 + y * kL) + row);
            wt[y] = ml.x, part[y] = ml.y;
            m = fmaxf(m, ml.x);
        }
        weigh<kL, kP>(wt, part, i8, count, m, l);
        if (r0 + sub >= rows) continue;
#pragma unroll
        for (int y = 0; y < kP; ++y)
            if (i8 + y * kL < count) weights[row * count + i8 + y * kL] = wt[y];
        if (i8 == 0) {
            inv[row] = l != 0.f ? 1.f / l : 0.f;
            if (!final) a.part_ml[slot(0) + row] = make_float2(m, l);
        }
    }
    meet();
    if (!mbar_wait(bar, parity)) mbar_wait(bar, parity);  // once more: the copies under way write into this CTA's shared memory
#pragma unroll 1
    for (int at = tid; at < rows * kL; at += THREADS) {
        const int row = at / kL, d = at % kL * 8;
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        const uint8_t* src = room + (row * D + d) * 4;
#pragma unroll 4
        for (int i = 0; i < count; ++i) {
            const float f = weights[row * count + i];
            const float4 v0 = reinterpret_cast<const float4*>(src + i * bytes)[0], v1 = reinterpret_cast<const float4*>(src + i * bytes)[1];
            const float from[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(f, from[e], acc[e]);
        }
        if (final) {
            const int tok = kv_row_token(a, row);
            *reinterpret_cast<uint4*>(a.out + (long long)(w.row0 + w.r * a.tq + tok) * a.o_st +
                                      (long long)(w.head * a.group + row - tok * a.group) * a.o_sh + d) = pack_bf16x8(acc, inv[row]);
        } else {
            float4* dst = reinterpret_cast<float4*>(a.part_o + (slot(0) + row) * D + d);
            dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        }
    }
}

// join_pieces with runs of about the square root of the pieces, which two
// rounds of bulk copies bring in soonest: at most 18 of the at most 304 there are.
template <typename Meet, typename Add>
__device__ __forceinline__ void join_pieces_in_runs(const KvPieces& of, int* joined, bool lead, int* last, Meet meet, Add add) {
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
    int size = 5;
    while (size * size < of.count) ++size;
    const int run = ((int)blockIdx.x - of.c) / size, mine = min(size, of.count - run * size);
    // A run's counter is that of its first CTA; an item that begins in that CTA has another.
    if (!arrive(joined + kKvMaxCtas * (run ? 2 : 1) + of.c + run * size, mine)) return;
    add(run * size, 1, mine, false);
    const int runs = (of.count + size - 1) / size;
    if (arrive(joined + of.c, runs)) add(0, size, runs, true);
}

}  // namespace hs
