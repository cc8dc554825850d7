// Division of the attention's work among the CTAs of one launch, shared by
// the kernels of hs_kv4_attention.
//
// An item is (request, kv head, row tile): the row tile holds TQ of the
// request's new tokens for all G query heads of the kv head.  Its work is the
// run of key tiles (64 or 128 keys) that some row of it sees.  All items' tiles, in the
// order (request, kv head, row tile, key tile), form one line that is cut into
// equal pieces, one a CTA: long and short requests, prompts and single tokens
// load the SMs alike, and the host needs none of the lengths.  The pieces of an
// item that a cut divides are joined by the CTA that comes last.
#pragma once

#include "hs_kv4.cuh"

namespace hs {

constexpr float kLazy = 8.f;     // a row's maximum may lag by a factor 2^8 before the sums are rescaled
constexpr float kNoMax = -3e38f; // the maximum of a row that has seen no key
constexpr float kFarScore = 2097152.f;  // 2^21, see kv_score_factor
constexpr int kNoQuery = 255;    // exponent field of infinities and NaN: a query row that holds one gives NaN
constexpr int kKvMaxCtas = 456;  // three on each of 152 SMs
constexpr int kKvWsRows = 2 * 152 * 256;  // rows of partial sums of the widest launch

struct KvAttnArgs {
    KvGeom g;
    const uint16_t* q;
    long long q_st, q_sh;
    uint16_t* out;
    long long o_st, o_sh;
    const int* q_start;
    const int* seq_len;
    const int* table;
    int width, n_seqs, n_tokens, group, rows, tq, min_units, pad, tile_log2;
    int back;            // a row at position p >= 0 sees the keys from p - back on: window - 1, or all of int
    uint32_t group_inv;  // ceil(2^16 / group)
    float scale_log2;    // scale * log2(e)
    float* part_o;       // [2 * CTAs][rows][dim] partial sums
    float2* part_ml;     // [2 * CTAs][rows] (maximum, sum)
    int* joined;         // [3 * CTAs] arrivals of pieces, zero between calls
};

// Token of a row of a row tile: row / group, for the at most 256 rows there are.
__device__ __forceinline__ int kv_row_token(const KvAttnArgs& a, int row) { return (int)(((uint32_t)row * a.group_inv) >> 16); }

struct KvSpan {
    int lo, hi;  // first and last key tile of an item (hi < lo: no key, counted as one tile)
};

// Key tiles of row tile r of a request with n new tokens and length len.
__device__ __forceinline__ KvSpan kv_span(const KvAttnArgs& a, int n, int len, int r) {
    const int ctx = len - n, t0 = r * a.tq, t1 = min(n, t0 + a.tq) - 1;
    const int last = min(ctx + t1, len - 1);
    const int first = max(0, max(ctx + t0, 0) - a.back);
    KvSpan s;
    if (last < 0 || first > last) {
        s.lo = 0, s.hi = -1;
    } else {
        s.lo = first >> a.tile_log2, s.hi = last >> a.tile_log2;
    }
    return s;
}
__device__ __forceinline__ int kv_span_tiles(const KvSpan& s) { return max(1, s.hi - s.lo + 1); }
__device__ __forceinline__ int kv_span_units(const KvAttnArgs& a, const KvSpan& s) { return kv_span_tiles(s) + a.pad; }

// Where a CTA's run of units stands; it always stands on a tile.
struct KvWalk {
    uint32_t left;           // units of the CTA's run still to do (this one included)
    int seq, head, r, tile;  // tile: unit within the item
    int n, len, row0;        // of the request: new tokens, length, first row of q
    int units, tiles;        // of the item: with its pad, and without
    int lo, hi;
    bool first;              // the run began inside this item
};

// The lengths the schedule goes by: a length is cut to the table's width, and
// a count of new tokens that q_start does not ascend by is 0.
__device__ __forceinline__ int kv_start(const KvAttnArgs& a, const int* qs, int i) {
    return min(max(qs[i], 0), a.n_tokens);  // no row outside q, whatever the device holds
}
__device__ __forceinline__ void kv_request(const KvAttnArgs& a, const int* qs, const int* ls, int i, int& n, int& len) {
    n = max(kv_start(a, qs, i + 1) - kv_start(a, qs, i), 0);
    len = min(max(ls[i], 0), a.width << a.g.page_log2);  // (the host has checked that product)
}

// Key tiles of a request, over its row tiles (whole warps; every lane gets it).
__device__ __forceinline__ int kv_many_units(const KvAttnArgs& a, int n, int len) {
    const int tiles = (n + a.tq - 1) / a.tq;
    int s = 0;
    for (int r = threadIdx.x & 31; r < tiles; r += 32) s += kv_span_units(a, kv_span(a, n, len, r));
    return (int)warp_add_u32((uint32_t)s);
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// Fills cum[0..n_seqs] (units before each request) in shared memory, by all
// threads of the CTA.  qs and ls: the requests' starts and lengths.
__device__ __forceinline__ void kv_schedule(const KvAttnArgs& a, const int* qs, const int* ls, uint32_t* cum) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
    bool many = false;  // some request has more than one row tile
    for (int i = tid; i < a.n_seqs; i += nt) {
        int n, len;
        kv_request(a, qs, ls, i, n, len);
        if (n <= a.tq)
            cum[i + 1] = n ? (uint32_t)a.g.heads * (uint32_t)kv_span_units(a, kv_span(a, n, len, 0)) : 0;
        else
            many = true;
    }
    if (__syncthreads_or(many)) {
        for (int i = warp; i < a.n_seqs; i += nw) {
            int n, len;
            kv_request(a, qs, ls, i, n, len);
            if (n <= a.tq) continue;
            const int s = kv_many_units(a, n, len);
            if (lane == 0) cum[i + 1] = (uint32_t)a.g.heads * (uint32_t)s;
        }
        __syncthreads();
    }
    if (warp == 0) {
        uint32_t base = 0;
        for (int i0 = 0; i0 < a.n_seqs; i0 += 32) {
            const int i = i0 + lane;
            const uint32_t v = warp_scan(i < a.n_seqs ? cum[i + 1] : 0u);
            if (i < a.n_seqs) cum[i + 1] = base + v;
            base += __shfl_sync(~0u, v, 31);
        }
        if (lane == 0) cum[0] = 0;
    }
    __syncthreads();
}

__device__ __forceinline__ void kv_set_item(const KvAttnArgs& a, KvWalk& w) {
    const KvSpan s = kv_span(a, w.n, w.len, w.r);
    w.lo = s.lo, w.hi = s.hi, w.tiles = kv_span_tiles(s), w.units = w.tiles + a.pad;
}

// An exponent is one fused operation on a dot product, the scores' factor sc and
// the row's maximum, which is rounded: from 2^24 on the exponents would be off by
// whole units and the probabilities leave the fp16 range.  So a row whose
// maximum is the dot product x, 2^21 and more times sc, goes by a power of two
// that brings it to [2^20, 2^21): products and maximum are then exact, and what that levels
// out (2^-20 of the scores) is of the size of their own rounding in fp32.
__device__ __forceinline__ float kv_score_factor(float x, float sc) {
    const int fx = (int)((__float_as_uint(x) >> 23) & 255u), fs = (int)((__float_as_uint(sc) >> 23) & 255u);
    return fx + fs - 254 <= 20 ? sc : __uint_as_float((uint32_t)max(254 + 20 - fx, 1) << 23);
}
// Kept off 0 and infinity, which make NaN of a hidden key (0 times -infinity) or of a product that is 0.
__device__ __forceinline__ float kv_score_range(float sc) { return fminf(fmaxf(sc, 1.2e-38f), 1e38f); }
// A row's maximum as the joins take it: by the scores' own factor.
__device__ __forceinline__ float kv_whole_max(float m, float sc, float own_sc) { return fminf(fmaxf(m / sc * own_sc, kNoMax), -kNoMax); }

// The cut of the line: the first `more` of `active` CTAs take q + 1 units, the others q.
struct KvCut {
    uint32_t q, active, more;
    __device__ __forceinline__ uint32_t at(uint32_t c) const { return q * c + min(c, more); }
    __device__ __forceinline__ int cta_of(uint32_t unit) const {
        const uint32_t wide = (q + 1) * more;
        return (int)(unit < wide ? unit / (q + 1) : more + (unit - wide) / q);
    }
};
__device__ __forceinline__ KvCut kv_cut(const KvAttnArgs& a, uint32_t total) {
    KvCut c;
    c.active = max(1u, min(gridDim.x, total / (uint32_t)a.min_units));
    c.q = total / c.active;
    c.more = total - c.q * c.active;
    return c;
}

// To the next item (the current one's units are done).
__device__ __forceinline__ void kv_next_item(const KvAttnArgs& a, const int* qs, const int* ls, KvWalk& w) {
    w.first = false;
    w.tile = 0;
    if (++w.r * a.tq >= w.n) {
        w.r = 0;
        if (++w.head == a.g.heads) {
            w.head = 0;
            do {
                ++w.seq;
                kv_request(a, qs, ls, w.seq, w.n, w.len);
            } while (!w.n);
            w.row0 = kv_start(a, qs, w.seq);
        }
    }
    kv_set_item(a, w);
}

// The tiles of the run's current item that are its own, and the units they end with.
__device__ __forceinline__ int kv_piece_tiles(const KvWalk& w) { return (int)min(w.left, (uint32_t)(w.tiles - w.tile)); }
// Takes `units` units off the run, which end the current item or the run.
__device__ __forceinline__ void kv_skip(const KvAttnArgs& a, const int* qs, const int* ls, KvWalk& w, uint32_t units) {
    w.left -= min(w.left, units);
    if (w.left > 0) kv_next_item(a, qs, ls, w);
}
__device__ __forceinline__ void kv_next_piece(const KvAttnArgs& a, const int* qs, const int* ls, KvWalk& w) {
    kv_skip(a, qs, ls, w, w.units - w.tile);
}

// Puts w at this CTA's first unit, which lies in request lo, whose units run
// from `before` to `after` (called by whole warps).
__device__ __forceinline__ void kv_place_run(const KvAttnArgs& a, const int* qs, const int* ls, KvWalk& w, uint32_t cut_at, int lo,
                                             uint32_t before, uint32_t after) {
    w.seq = lo;
    kv_request(a, qs, ls, lo, w.n, w.len);
    w.row0 = kv_start(a, qs, lo);
    const uint32_t per_head = (after - before) / (uint32_t)a.g.heads;
    uint32_t rest = cut_at - before;
    w.head = (int)(rest / per_head);
    rest -= (uint32_t)w.head * per_head;
    const int tiles = (w.n + a.tq - 1) / a.tq;
    w.r = 0;
    if (tiles > 1) {
        const int lane = threadIdx.x & 31;
        for (int r0 = 0; r0 < tiles; r0 += 32) {
            const uint32_t mine = r0 + lane < tiles ? (uint32_t)kv_span_units(a, kv_span(a, w.n, w.len, r0 + lane)) : 0u;
            const uint32_t incl = warp_scan(mine);
            const unsigned past = __ballot_sync(~0u, mine && incl > rest);
            if (past) {
                const int l = __ffs(past) - 1;
                rest -= __shfl_sync(~0u, incl - mine, l);
                w.r = r0 + l;
                break;
            }
            rest -= __shfl_sync(~0u, incl, 31);
        }
    }
    w.tile = (int)rest;
    w.first = true;
    kv_set_item(a, w);
    if (w.tile >= w.tiles) kv_skip(a, qs, ls, w, w.units - w.tile);  // the run begins in a pad
}

// Start of this CTA's run (called by whole warps; every lane gets the same).
__device__ __forceinline__ KvWalk kv_begin(const KvAttnArgs& a, const int* qs, const int* ls, const uint32_t* cum) {
    KvWalk w;
    const uint32_t total = cum[a.n_seqs];
    const KvCut cut = kv_cut(a, total);
    w.left = 0;
    if (!total || blockIdx.x >= cut.active) return w;
    const uint32_t u0 = cut.at(blockIdx.x);
    w.left = cut.at(blockIdx.x + 1) - u0;
    int lo = 0, hi = a.n_seqs;
    while (hi - lo > 1) {  // the last request with cum <= u0: it has units
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= u0) lo = mid;
        else hi = mid;
    }
    kv_place_run(a, qs, ls, w, u0, lo, cum[lo], cum[lo + 1]);
    return w;
}

// The same by one warp alone, for at most 128 requests: four a lane at most,
// and neither the CTA's other warps nor shared memory are waited for.
__device__ __forceinline__ KvWalk kv_begin_few(const KvAttnArgs& a, uint32_t& total) {
    const int lane = threadIdx.x & 31, per = (a.n_seqs + 31) >> 5;
    uint32_t mine = 0, units[4];
    int start[5], len[4];
#pragma unroll
    for (int j = 0; j < 5; ++j) start[j] = j <= per && lane * per + j <= a.n_seqs ? a.q_start[lane * per + j] : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) len[j] = j < per && lane * per + j < a.n_seqs ? a.seq_len[lane * per + j] : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        units[j] = 0;
        if (j >= per) break;
        const bool in = lane * per + j < a.n_seqs;
        const int n = in ? max(min(max(start[j + 1], 0), a.n_tokens) - min(max(start[j], 0), a.n_tokens), 0) : 0;
        const int l = min(max(len[j], 0), a.width << a.g.page_log2);
        if (n && n <= a.tq) units[j] = (uint32_t)a.g.heads * (uint32_t)kv_span_units(a, kv_span(a, n, l, 0));
        for (unsigned many = __ballot_sync(~0u, n > a.tq); many; many &= many - 1) {
            const int x = __ffs(many) - 1;
            const uint32_t u = (uint32_t)a.g.heads * (uint32_t)kv_many_units(a, __shfl_sync(~0u, n, x), __shfl_sync(~0u, l, x));
            if (lane == x) units[j] = u;
        }
        mine += units[j];
    }
    const uint32_t incl = warp_scan(mine);
    total = __shfl_sync(~0u, incl, 31);
    KvWalk w;
    const KvCut cut = kv_cut(a, total);
    w.left = 0;
    if (!total || blockIdx.x >= cut.active) return w;
    const uint32_t u0 = cut.at(blockIdx.x);
    w.left = cut.at(blockIdx.x + 1) - u0;
    const int x = __ffs(__ballot_sync(~0u, incl > u0)) - 1;  // the lane whose requests the run begins in
    uint32_t before = __shfl_sync(~0u, incl - mine, x);
    int seq = x * per;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t u = __shfl_sync(~0u, units[j], x);
        if (j < per - 1 && before + u <= u0 && seq == x * per + j) before += u, ++seq;
        if (seq == x * per + j) mine = u;
    }
    kv_place_run(a, a.q_start, a.seq_len, w, u0, seq, before, before + mine);
    return w;
}

// Whether the line of a call with these row and key tiles stays below 2^32 units.
inline bool kv_line_ok(const KvAttnArgs& a) {
    const double row_tiles = (double)(a.n_tokens / a.tq) + a.n_seqs;
    const double units = (double)((((long long)a.width << a.g.page_log2) >> a.tile_log2) + 2 + a.pad);
    return row_tiles * units * a.g.heads < 4294967296.0;
}

constexpr int kKvFew = 128;  // requests that kv_begin_few takes

}  // namespace hs

// The tensor-core kernel for chunks (hs_kv4_prefill.cu).
int hs_kv4_prefill(hs::KvAttnArgs a, int dim, int sms, cudaStream_t stream);
// Reads and clears its device error word.
unsigned hs_kv4_prefill_take_status();
