// Pages of a paged key/value cache that several requests own, or that move:
// fork, copy, release, compact, GB300 (sm_103a).  Contracts: hs.h.  Nothing here
// depends on how many bits the cache holds a value in: a page is a number, and for
// the copies a run of bytes.
//
// A page's owners beyond the first are counted (`shared`), so that a page taken
// from the ring or given to it has the count 0 and the step plan needs no counts.
#include "hs_kv4.cuh"

namespace hs {

constexpr int kPageThreads = 256, kPageWarps = kPageThreads / 32;
constexpr int kMaxPools = 64;

// What release and compact keep between their steps.  The arrivals and the marks are
// zero between calls; the rest is written before it is read.
struct PageScratch {
    int* arrived;     // CTAs that are done with their rows
    int* totals;      // compact: used pages, those of them below that number, moves, refused
    uint8_t* mark;    // [n_pages] 1: release: to be given back; compact: used (bytes, for a store each; bits would take atomics)
    int* before;      // [words] compact: used pages before the first of 32
    int* move_of;     // [n_pages] compact: the move that takes a page away
    int* moved;       // [n_pages / 2] compact: a move's count of owners
};

__host__ __device__ inline int page_words(int n_pages) { return (n_pages + 31) >> 5; }

// The marks of 64 pages (four times 16 bytes, past the pool zeros) as two words of bits.
__device__ __forceinline__ void marks64(const uint8_t* mark, uint32_t (&word)[2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        word[k] = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 v = __ldcg(reinterpret_cast<const uint4*>(mark) + 2 * k + j);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) word[k] |= ((u[i] | u[i] >> 7 | u[i] >> 14 | u[i] >> 21) & 15u) << (16 * j + 4 * i);
        }
    }
}

struct PageRows {
    const int* cached;
    int n, page_log2, n_pages, width;
    const int* table_in;
    int* table_out;
    __device__ __forceinline__ int pages(int tokens) const {  // of a row that holds so many
        return (int)min(((long long)max(tokens, 0) + (1 << page_log2) - 1) >> page_log2, (long long)width);
    }
    __device__ __forceinline__ bool there(int page) const { return (uint32_t)page < (uint32_t)n_pages; }
};

__device__ __forceinline__ uint32_t ring_at(long long counter, int n_pages) {
    return (uint32_t)((counter % n_pages + n_pages) % n_pages);
}

// Sum over the threads before this one, and over all of them; called by whole CTAs.
__device__ __forceinline__ int block_scan(int v, int& all) {
    __shared__ int part[kPageWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += t;
    }
    __syncthreads();
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int base = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kPageWarps; ++w) {
        if (w == warp) base = all;
        all += part[w];
    }
    return base + incl - v;
}

// True in the CTA that comes last, which then sees what all the others have written.
__device__ __forceinline__ bool last_to_arrive(int* arrived) {
    __shared__ int last;
    __syncthreads();
    if (threadIdx.x == 0) {
        int before;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(arrived) : "memory");
        last = before == (int)gridDim.x - 1;
        if (last) *arrived = 0;  // for the next call
    }
    __syncthreads();
    return last != 0;
}

// ------------------------------------------------------------------ fork
struct ForkArgs {
    PageRows r;
    const int *parent, *child, *length;
    int forks;
    int* shared;
    const int* ring;
    const long long* counters_in;
    int* len_out;
    int *copy_src, *copy_dst;
    long long* counters_out;
    int* short_out;
};

// As the step plan: every CTA looks at all forks (whether they can be done, and the
// pages taken before each) and then writes its share of the rows.  Bound by the launch and
// three dependent reads: 3.4 us for 4 forks, 4.3 for 512 of rows of up to 32 pages.  A row is one
// warp's, whose turns of 32 pages follow one another: 4 forks of 131,071 tokens 18 us at 64 tokens a page, 63 at 16.
__global__ void __launch_bounds__(kPageThreads) kv_fork_kernel(const ForkArgs a) {
    extern __shared__ int fork_smem[];
    int* fork_of = fork_smem;           // [n] the row's fork with kFork on, or how many name it as their child
    int* taken = fork_smem + a.r.n;     // [forks] pages taken before it
    constexpr int kFork = 1 << 30;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = 1 << a.r.page_log2;
    for (int i = tid; i < a.r.n; i += kPageThreads) fork_of[i] = 0;
    pdl_wait();
    pdl_trigger();
    const long long head = a.counters_in[0], tail = a.counters_in[1];
    __syncthreads();
    const int per = (a.forks + kPageThreads - 1) / kPageThreads;
    const int i0 = min(tid * per, a.forks), i1 = min(i0 + per, a.forks);
    int bad = 0, need = 0;
    for (int i = i0; i < i1; ++i) {
        const int p = a.parent[i], c = a.child[i], len = a.length[i];
        bool ok = (uint32_t)p < (uint32_t)a.r.n && (uint32_t)c < (uint32_t)a.r.n && p != c && len >= 0;
        if (ok) ok = len <= max(a.r.cached[p], 0) && a.r.cached[c] <= 0 && ((long long)len + P - 1) >> a.r.page_log2 <= a.r.width;
        if ((uint32_t)c < (uint32_t)a.r.n) atomicAdd(fork_of + c, 1);
        bad += !ok;
        taken[i] = ok ? 0 : -1;
        need += (len & (P - 1)) != 0;
    }
    int all_need, all_bad;
    int at = block_scan(need, all_need);  // (its barriers: all children have been counted)
    for (int i = i0; i < i1; ++i) {
        const int c = a.child[i];
        if (taken[i] == 0 && fork_of[c] != 1) ++bad;
    }
    block_scan(bad, all_bad);
    const long long missing = all_bad + max((long long)all_need - (tail - head), 0ll);
    const bool ok = missing == 0;
    for (int i = i0; i < i1; ++i) {
        taken[i] = at;
        at += (a.length[i] & (P - 1)) != 0;
        if (ok) fork_of[a.child[i]] = kFork | i;
    }
    __syncthreads();
    const uint32_t np = (uint32_t)a.r.n_pages, head_m = ring_at(head, a.r.n_pages);
    if (blockIdx.x == 0 && tid == 0) {
        a.counters_out[0] = head + (ok ? all_need : 0);
        a.counters_out[1] = tail;
        a.short_out[0] = (int)min(missing, (long long)INT32_MAX);
    }
    for (int i = blockIdx.x * kPageThreads + tid; i < a.forks; i += gridDim.x * kPageThreads) {
        int src = -1, dst = -1;
        if (ok && (a.length[i] & (P - 1))) {
            src = a.r.table_in[(size_t)a.parent[i] * a.r.width + (a.length[i] >> a.r.page_log2)];
            dst = a.ring[(head_m + (uint32_t)taken[i]) % np];
        }
        a.copy_src[i] = src;
        a.copy_dst[i] = dst;
    }
    const bool in_place = a.r.table_in == a.r.table_out;
    for (int i = blockIdx.x * kPageWarps + warp; i < a.r.n; i += gridDim.x * kPageWarps) {
        const bool forked = ok && (fork_of[i] & kFork);
        const int f = fork_of[i] & (kFork - 1);
        if (lane == 0) a.len_out[i] = forked ? a.length[f] : max(a.r.cached[i], 0);
        if (!forked && in_place) continue;
        // (a parent that is a child itself holds nothing, and nothing is read of it)
        const int* src = a.r.table_in + (size_t)(forked ? a.parent[f] : i) * a.r.width;
        int* dst = a.r.table_out + (size_t)i * a.r.width;
        const int whole = forked ? a.length[f] >> a.r.page_log2 : a.r.width;
        const int own = forked && (a.length[f] & (P - 1)) ? a.ring[(head_m + (uint32_t)taken[f]) % np] : -1;
#pragma unroll 4
        for (int c = lane; c < a.r.width; c += 32) {
            const int page = c < whole ? src[c] : c == whole ? own : -1;
            dst[c] = page;
            if (forked && c < whole && a.r.there(page)) atomicAdd(a.shared + page, 1);
        }
    }
}

// ---------------------------------------------------------------- copies
struct CopyArgs {
    uint8_t* pool[kMaxPools];
    int pools, n_pages, n, segments;
    uint32_t page_bytes, segment;  // of a page; that a CTA copies of it
    const int *src, *dst;
};

constexpr int kCopyThreads = 128, kCopyAhead = 5;
constexpr uint32_t kSegment = kCopyThreads * kCopyAhead * 16;  // bytes that a CTA copies at a time, at most

// A CTA takes one segment of the pages of one pool, and every gridDim.x-th pair: it
// reads 128 of its pairs at a time and keeps those that are ones, so that a long list
// with few copies costs a read a CTA.  Bound by memory: 6,200 pages of 8 KB in two pools
// (204 MB read and written) 32 us, 93% of the copy bandwidth; four CTAs for each that an SM holds even out
// the pairs (one for each: 37.6).
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const CopyArgs a) {
    __shared__ int2 todo[kCopyThreads];
    __shared__ int first[kCopyThreads / 32 + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    for (long long base = blockIdx.x; base < a.n; base += (long long)gridDim.x * kCopyThreads) {
        const long long i = base + (long long)tid * gridDim.x;
        int2 p = make_int2(-1, -1);
        if (i < a.n) p = make_int2(a.src[i], a.dst[i]);
        const bool some = (uint32_t)p.x < (uint32_t)a.n_pages && (uint32_t)p.y < (uint32_t)a.n_pages && p.x != p.y;
        const unsigned mask = __ballot_sync(~0u, some);
        if (lane == 0) first[warp] = __popc(mask);
        __syncthreads();
        int at = 0, count = 0;
        for (int w = 0; w < kCopyThreads / 32; ++w) {
            if (w == warp) at = count;
            count += first[w];
        }
        if (some) todo[at + __popc(mask & ((1u << lane) - 1))] = p;
        __syncthreads();
        for (int y = blockIdx.y; y < a.pools * a.segments; y += gridDim.y) {
            uint8_t* pool = a.pool[y / a.segments];
            const uint32_t first = (uint32_t)(y % a.segments) * a.segment, end = min(first + a.segment, a.page_bytes), from = first + (uint32_t)tid * 16;
            for (int j = 0; j < count; ++j) {
                const uint8_t* src = pool + (size_t)todo[j].x * a.page_bytes;
                uint8_t* dst = pool + (size_t)todo[j].y * a.page_bytes;
                uint4 v[kCopyAhead];
#pragma unroll
                for (int k = 0; k < kCopyAhead; ++k)
                    if (from + k * kCopyThreads * 16 < end)
                        v[k] = __ldcs(reinterpret_cast<const uint4*>(src + from + k * kCopyThreads * 16));
#pragma unroll
                for (int k = 0; k < kCopyAhead; ++k)
                    if (from + k * kCopyThreads * 16 < end)
                        __stcs(reinterpret_cast<uint4*>(dst + from + k * kCopyThreads * 16), v[k]);
            }
        }
        __syncthreads();
    }
}

// --------------------------------------------------------------- release
struct ReleaseArgs {
    PageRows r;
    const int* keep;
    int* shared;
    int* ring;
    const long long* counters_in;
    int* len_out;
    long long* counters_out;
    PageScratch s;
};

// A warp a row takes an owner off each page that the row gives up, and marks those
// that had one left; the CTA that comes last puts the marked pages into the ring, in
// the order of their numbers, whatever the order of the rows' atomics was.  Bound by the chain
// of lengths, table, atomics, arrivals and the last CTA's pass over the marks: 3.8 us for 5 rows, 5.0 for
// 576 of 2331 pages (13.2 while one warp wrote the ring word by word).  The marks are the whole pool's, whatever is
// given back: one short row 8.2 us in a pool of 30,000 pages, 24 in one of 300,000; and a row is one warp's: 4 rows of
// 131,071 tokens 41 us at 64 tokens a page, 153 at 16.
__global__ void __launch_bounds__(kPageThreads) kv_release_kernel(const ReleaseArgs a) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const bool in_place = a.r.table_in == a.r.table_out;
    for (int i = blockIdx.x * kPageWarps + warp; i < a.r.n; i += gridDim.x * kPageWarps) {
        const int have = max(a.r.cached[i], 0), keep = min(max(a.keep[i], 0), have);
        const int held = a.r.pages(have), stay = a.r.pages(keep);
        const int* src = a.r.table_in + (size_t)i * a.r.width;
        int* dst = a.r.table_out + (size_t)i * a.r.width;
        if (lane == 0) a.len_out[i] = keep;
#pragma unroll 4
        for (int c = (in_place ? stay & ~31 : 0) + lane; c < a.r.width; c += 32) {
            const int page = c < held ? src[c] : -1;
            if (!(in_place && c < stay)) dst[c] = c < stay ? page : -1;
            if (c >= stay && a.r.there(page) && atomicSub(a.shared + page, 1) <= 0) {
                atomicAdd(a.shared + page, 1);
                a.s.mark[page] = 1;
            }
        }
    }
    if (!last_to_arrive(a.s.arrived)) return;
    __shared__ uint2 found[kPageThreads * 2];  // of 32 pages: those to be given back, and how many come before them
    const long long tail = a.counters_in[1];
    const uint32_t tail_m = ring_at(tail, a.r.n_pages), np = (uint32_t)a.r.n_pages;
    const int words = page_words(a.r.n_pages);
    uint32_t done = 0;
    for (int w0 = 0; w0 < words; w0 += kPageThreads * 2) {  // a thread 64 pages that follow one another
        uint32_t v[2] = {0, 0};
        const int w = w0 + tid * 2;
        int all;
        if (w < words) {
            uint8_t* mark = a.s.mark + (size_t)w * 32;
            marks64(mark, v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (v[j >> 1]) reinterpret_cast<uint4*>(mark)[j] = make_uint4(0, 0, 0, 0);
        }
        const int at = block_scan(__popc(v[0]) + __popc(v[1]), all);
        if (!all) continue;
        found[tid * 2] = make_uint2(v[0], (uint32_t)at);
        found[tid * 2 + 1] = make_uint2(v[1], (uint32_t)(at + __popc(v[0])));
        __syncthreads();
        for (int x = warp; x < min(kPageThreads * 2, words - w0); x += kPageWarps) {  // a page a lane
            const uint2 y = found[x];
            uint32_t to = tail_m + done + y.y + (uint32_t)__popc(y.x & ((1u << lane) - 1));  // (at most n_pages on)
            if (to >= np) to -= np;
            if ((y.x >> lane) & 1u) a.ring[to] = (w0 + x) * 32 + lane;
        }
        done += (uint32_t)all;  // (`found` is written again behind the next scan's barriers)
    }
    if (tid == 0) {
        a.counters_out[0] = a.counters_in[0];
        a.counters_out[1] = tail + done;
    }
}

// --------------------------------------------------------------- compact
struct CompactArgs {
    PageRows r;
    const int* shared_in;
    int* shared_out;
    int* ring;
    const long long* counters_in;
    int max_copies;
    int *copy_src, *copy_dst;
    long long* counters_out;
    int* short_out;
    PageScratch s;
};

// First of three launches: the pages that the rows list are marked; the CTA that comes
// last counts them by thirty-two.  All three are bound by their launches and chains of
// reads: 6.5 us for 8 rows, 8.8 for 1000 rows and 25,000 pages.
__global__ void __launch_bounds__(kPageThreads) kv_compact_mark_kernel(const CompactArgs a) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    for (int i = blockIdx.x * kPageWarps + warp; i < a.r.n; i += gridDim.x * kPageWarps) {
        const int held = a.r.pages(a.r.cached[i]);
        const int* src = a.r.table_in + (size_t)i * a.r.width;
#pragma unroll 4
        for (int c = lane; c < held; c += 32) {
            const int page = src[c];
            if (a.r.there(page)) a.s.mark[page] = 1;
        }
    }
    if (!last_to_arrive(a.s.arrived)) return;
    const int words = page_words(a.r.n_pages);
    int used = 0;
    for (int w0 = 0; w0 < words; w0 += kPageThreads * 2) {
        uint32_t v[2] = {0, 0};
        const int w = w0 + tid * 2;
        int all;
        if (w < words) marks64(a.s.mark + (size_t)w * 32, v);
        const int at = used + block_scan(__popc(v[0]) + __popc(v[1]), all);
        if (w < words) a.s.before[w] = at;
        if (w + 1 < words) a.s.before[w + 1] = at + __popc(v[0]);
        used += all;
    }
    __syncthreads();
    if (tid == 0) {
        int below = used;  // used pages among the first `used` ones
        if (used < a.r.n_pages) {
            uint32_t v[2];
            marks64(a.s.mark + (size_t)(used >> 6) * 64, v);
            below = a.s.before[used >> 5] + __popc(v[used >> 5 & 1] & ((1u << (used & 31)) - 1));
        }
        const int moves = used - below, over = max(moves - a.max_copies, 0);
        a.s.totals[0] = used, a.s.totals[1] = below, a.s.totals[2] = over ? 0 : moves, a.s.totals[3] = over;
        a.counters_out[0] = over ? a.counters_in[0] : 0;
        a.counters_out[1] = over ? a.counters_in[1] : a.r.n_pages - used;
        a.short_out[0] = over;
    }
}

// Second: a warp 32 pages.  The k-th used page past the first `used` ones goes into the
// k-th free one among them.
__global__ void __launch_bounds__(kPageThreads) kv_compact_list_kernel(const CompactArgs a) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const int used = a.s.totals[0], below = a.s.totals[1], moves = a.s.totals[2];
    const bool ok = a.s.totals[3] == 0;
    const int words = page_words(a.r.n_pages);
    for (int w = blockIdx.x * kPageWarps + warp; w < words; w += gridDim.x * kPageWarps) {
        const int page = w * 32 + lane;
        const bool live = a.s.mark[page] != 0;  // (of whole words: past the pool 0)
        const int rank = a.s.before[w] + __popc(__ballot_sync(~0u, live) & ((1u << lane) - 1));
        if (page >= a.r.n_pages) continue;
        if (live) a.s.mark[page] = 0;  // for the next call
        const int owners = a.shared_in[page];
        if (!ok) {
            a.shared_out[page] = owners;
            continue;
        }
        if (page >= used) {
            a.ring[page - used] = page;
            if (live) {
                const int m = rank - below;
                a.copy_src[m] = page;
                a.s.moved[m] = owners;
                a.s.move_of[page] = m;
            }
            a.shared_out[page] = 0;
        } else if (live) {
            a.shared_out[page] = owners;
        } else {
            a.copy_dst[page - rank] = page;  // (its owners: with the third launch)
        }
    }
    for (int i = moves + blockIdx.x * kPageThreads + tid; i < a.max_copies; i += gridDim.x * kPageThreads)
        a.copy_src[i] = a.copy_dst[i] = -1;
}

// Third: the tables, and the owners of the pages that moved.
__global__ void __launch_bounds__(kPageThreads) kv_compact_rows_kernel(const CompactArgs a) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const int used = a.s.totals[0], moves = a.s.totals[2];
    const bool ok = a.s.totals[3] == 0;
    for (int i = blockIdx.x * kPageWarps + warp; i < a.r.n; i += gridDim.x * kPageWarps) {
        const int held = a.r.pages(a.r.cached[i]);
        const int* src = a.r.table_in + (size_t)i * a.r.width;
        int* dst = a.r.table_out + (size_t)i * a.r.width;
#pragma unroll 4
        for (int c = lane; c < a.r.width; c += 32) {
            int page = ok && c >= held ? -1 : src[c];
            if (ok && page >= used && a.r.there(page)) page = a.copy_dst[a.s.move_of[page]];
            dst[c] = page;
        }
    }
    for (int m = blockIdx.x * kPageThreads + tid; m < moves; m += gridDim.x * kPageThreads) a.shared_out[a.copy_dst[m]] = a.s.moved[m];
}

}  // namespace hs

using namespace hs_host;

namespace {

struct Range {
    const void* p;
    long long bytes;
};

// HS_OK if none of the first `written` ranges overlaps another one; ranges x and y
// (and u and v) may be one and the same buffer.
int apart(const Range* r, int n, int written, int x, int y, int u = -1, int v = -1) {
    for (int i = 0; i < written; ++i)
        for (int j = i + 1; j < n; ++j) {
            const bool pair = (i == x && j == y) || (i == u && j == v);
            if (pair && r[i].p == r[j].p) continue;
            const uintptr_t a = (uintptr_t)r[i].p, b = (uintptr_t)r[j].p;
            if (a < b + (uintptr_t)r[j].bytes && b < a + (uintptr_t)r[i].bytes) return HS_ERR_INVALID_ARG;
        }
    return HS_OK;
}

// Alignment of the ranges: 8 bytes for those whose bit is set, else 4.
int aligned(const Range* r, int n, unsigned wide) {
    for (int i = 0; i < n; ++i)
        if ((uintptr_t)r[i].p & ((wide >> i) & 1u ? 7u : 3u)) return HS_ERR_MISALIGNED;
    return HS_OK;
}

int rows_ok(int n_seqs, int page_tokens, int n_pages, int table_width) {
    if (n_seqs < 1 || n_pages < 1 || table_width < 1) return HS_ERR_INVALID_ARG;
    if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64) return HS_ERR_UNSUPPORTED_SHAPE;
    if (n_seqs > hs::kKvMaxSeqs || (long long)n_seqs * table_width >= (1 << 30) || n_pages >= (1 << 30) ||
        (long long)table_width * page_tokens >= (1ll << 31))
        return HS_ERR_UNSUPPORTED_SHAPE;
    return HS_OK;
}

hs::PageRows rows_of(const int* cached, int n, int page_tokens, int n_pages, int width, const int* in, int* out) {
    return {cached, n, page_tokens == 16 ? 4 : page_tokens == 32 ? 5 : 6, n_pages, width, in, out};
}

size_t scratch_bytes(int n_pages, uint8_t* base, hs::PageScratch* s) {
    const size_t marks = round_up((size_t)n_pages, 256), words = round_up((size_t)hs::page_words(n_pages) * 4, 256),
                 pages = round_up((size_t)n_pages * 4, 256);
    if (s) {
        s->arrived = reinterpret_cast<int*>(base);
        s->totals = s->arrived + 4;
        s->mark = base + 256;
        s->before = reinterpret_cast<int*>(base + 256 + marks);
        s->move_of = reinterpret_cast<int*>(base + 256 + marks + words);
        s->moved = reinterpret_cast<int*>(base + 256 + marks + words + pages);
    }
    return 256 + marks + words + 2 * pages;
}

// CTAs for rows a warp each, up to two on an SM.
int row_ctas(int n, int sms) { return std::min((n + hs::kPageWarps - 1) / hs::kPageWarps, 2 * sms); }

}  // namespace

extern "C" size_t hs_kv_pages_workspace_size(int n_pages) {
    return n_pages >= 1 && n_pages < (1 << 30) ? scratch_bytes(n_pages, nullptr, nullptr) : 0;
}

extern "C" int hs_kv_fork(const int* parent, const int* child, const int* length, int n_forks, const int* cached, int n_seqs,
                          int page_tokens, int n_pages, const int* table_in, int table_width, int* shared, const int* ring,
                          const long long* counters_in, int* table_out, int* len_out, int* copy_src, int* copy_dst,
                          long long* counters_out, int* short_out, hs_stream_t stream) {
    if (!parent || !child || !length || !cached || !table_in || !shared || !ring || !counters_in || !table_out || !len_out || !copy_src ||
        !copy_dst || !counters_out || !short_out || n_forks < 1)
        return HS_ERR_INVALID_ARG;
    int st = rows_ok(n_seqs, page_tokens, n_pages, table_width);
    if (st != HS_OK) return st;
    if (n_forks > hs::kKvMaxSeqs) return HS_ERR_UNSUPPORTED_SHAPE;
    const long long f = n_forks * 4ll, n = n_seqs * 4ll, cells = n * table_width;
    const Range r[] = {{table_out, cells}, {len_out, n}, {copy_src, f}, {copy_dst, f}, {counters_out, 16}, {short_out, 4}, {shared, n_pages * 4ll},
                       {parent, f}, {child, f}, {length, f}, {cached, n}, {table_in, cells}, {ring, n_pages * 4ll}, {counters_in, 16}};
    st = aligned(r, 14, 1u << 4 | 1u << 13);
    if (st == HS_OK) st = apart(r, 14, 7, 0, 11);
    if (st != HS_OK) return st;
    const int sms = sm_count();
    if (!sms) return HS_ERR_CUDA;
    hs::ForkArgs a = {rows_of(cached, n_seqs, page_tokens, n_pages, table_width, table_in, table_out), parent, child, length, n_forks, shared,
                      ring, counters_in, len_out, copy_src, copy_dst, counters_out, short_out};
    if (launch_pdl(hs::kv_fork_kernel, dim3(row_ctas(n_seqs, sms)), dim3(hs::kPageThreads), (size_t)(n_seqs + n_forks) * sizeof(int),
                   reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
        return HS_ERR_CUDA;
    return launch_err();
}

extern "C" int hs_kv_copy_pages(void* const* pools, int n_pools, long long page_bytes, int n_pages, const int* src, const int* dst,
                                int n_copies, hs_stream_t stream) {
    if (!pools || !src || !dst || n_pools < 1 || n_pages < 1 || n_copies < 0 || page_bytes < 1) return HS_ERR_INVALID_ARG;
    if (n_pools > hs::kMaxPools || page_bytes > (1ll << 30) || n_copies >= (1 << 30)) return HS_ERR_UNSUPPORTED_SHAPE;
    if (page_bytes & 15 || !al4(src) || !al4(dst)) return HS_ERR_MISALIGNED;
    hs::CopyArgs a = {};
    for (int i = 0; i < n_pools; ++i) {
        if (!pools[i]) return HS_ERR_INVALID_ARG;
        if (!al16(pools[i])) return HS_ERR_MISALIGNED;
        a.pool[i] = static_cast<uint8_t*>(pools[i]);
    }
    if (!n_copies) return HS_OK;
    const int sms = sm_count();
    if (!sms) return HS_ERR_CUDA;
    a.pools = n_pools, a.n_pages = n_pages, a.n = n_copies, a.src = src, a.dst = dst;
    a.page_bytes = (uint32_t)page_bytes;
    a.segments = (int)((page_bytes + hs::kSegment - 1) / hs::kSegment);
    a.segment = (uint32_t)round_up((size_t)(page_bytes + a.segments - 1) / a.segments, 16);
    const int y = (int)std::min((long long)n_pools * a.segments, 65535ll);
    const int x = std::max(1, std::min(n_copies, sms * 64 / y));
    if (launch_pdl(hs::kv_copy_kernel, dim3(x, y), dim3(hs::kCopyThreads), 0, reinterpret_cast<cudaStream_t>(stream), a) != cudaSuccess)
        return HS_ERR_CUDA;
    return launch_err();
}

extern "C" int hs_kv_release(const int* cached, const int* keep, int n_seqs, int page_tokens, int n_pages, const int* table_in,
                             int table_width, int* shared, int* ring, const long long* counters_in, int* table_out, int* len_out,
                             long long* counters_out, void* ws, size_t ws_bytes, hs_stream_t stream) {
    if (!cached || !keep || !table_in || !shared || !ring || !counters_in || !table_out || !len_out || !counters_out) return HS_ERR_INVALID_ARG;
    int st = rows_ok(n_seqs, page_tokens, n_pages, table_width);
    if (st != HS_OK) return st;
    const long long n = n_seqs * 4ll, cells = n * table_width, pages = n_pages * 4ll;
    const size_t need = scratch_bytes(n_pages, nullptr, nullptr);
    if (!ws || ws_bytes < need) return HS_ERR_WORKSPACE;
    if (!al16(ws)) return HS_ERR_MISALIGNED;
    const Range r[] = {{table_out, cells}, {len_out, n}, {counters_out, 16}, {shared, pages}, {ring, pages}, {ws, (long long)need},
                       {cached, n}, {keep, n}, {table_in, cells}, {counters_in, 16}};
    st = aligned(r, 10, 1u << 2 | 1u << 9);
    if (st == HS_OK) st = apart(r, 10, 6, 0, 8);
    if (st != HS_OK) return st;
    const int sms = sm_count();
    if (!sms) return HS_ERR_CUDA;
    hs::ReleaseArgs a = {rows_of(cached, n_seqs, page_tokens, n_pages, table_width, table_in, table_out), keep, shared, ring, counters_in, len_out,
                         counters_out, {}};
    scratch_bytes(n_pages, static_cast<uint8_t*>(ws), &a.s);
    if (launch_pdl(hs::kv_release_kernel, dim3(row_ctas(n_seqs, sms)), dim3(hs::kPageThreads), 0, reinterpret_cast<cudaStream_t>(stream), a) !=
        cudaSuccess)
        return HS_ERR_CUDA;
    return launch_err();
}

extern "C" int hs_kv_compact(const int* cached, int n_seqs, int page_tokens, int n_pages, const int* table_in, int table_width,
                             const int* shared_in, int* ring, const long long* counters_in, int max_copies, int* table_out,
                             int* shared_out, int* copy_src, int* copy_dst, long long* counters_out, int* short_out, void* ws,
                             size_t ws_bytes, hs_stream_t stream) {
    if (!cached || !table_in || !shared_in || !ring || !counters_in || !table_out || !shared_out || !copy_src || !copy_dst || !counters_out ||
        !short_out || max_copies < 1)
        return HS_ERR_INVALID_ARG;
    int st = rows_ok(n_seqs, page_tokens, n_pages, table_width);
    if (st != HS_OK) return st;
    if (max_copies >= (1 << 30)) return HS_ERR_UNSUPPORTED_SHAPE;
    const long long n = n_seqs * 4ll, cells = n * table_width, pages = n_pages * 4ll, c = max_copies * 4ll;
    const size_t need = scratch_bytes(n_pages, nullptr, nullptr);
    if (!ws || ws_bytes < need) return HS_ERR_WORKSPACE;
    if (!al16(ws)) return HS_ERR_MISALIGNED;
    const Range r[] = {{table_out, cells}, {shared_out, pages}, {copy_src, c}, {copy_dst, c}, {counters_out, 16}, {short_out, 4}, {ring, pages},
                       {ws, (long long)need}, {cached, n}, {table_in, cells}, {shared_in, pages}, {counters_in, 16}};
    st = aligned(r, 12, 1u << 4 | 1u << 11);
    if (st == HS_OK) st = apart(r, 12, 8, 0, 9, 1, 10);
    if (st != HS_OK) return st;
    const int sms = sm_count();
    if (!sms) return HS_ERR_CUDA;
    hs::CompactArgs a = {rows_of(cached, n_seqs, page_tokens, n_pages, table_width, table_in, table_out), shared_in, shared_out, ring, counters_in,
                         max_copies, copy_src, copy_dst, counters_out, short_out, {}};
    scratch_bytes(n_pages, static_cast<uint8_t*>(ws), &a.s);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 rows(row_ctas(n_seqs, sms)), words(std::min((hs::page_words(n_pages) + hs::kPageWarps - 1) / hs::kPageWarps, 4 * sms));
    if (launch_pdl(hs::kv_compact_mark_kernel, rows, dim3(hs::kPageThreads), 0, s, a) != cudaSuccess ||
        launch_pdl(hs::kv_compact_list_kernel, words, dim3(hs::kPageThreads), 0, s, a) != cudaSuccess ||
        launch_pdl(hs::kv_compact_rows_kernel, rows, dim3(hs::kPageThreads), 0, s, a) != cudaSuccess)
        return HS_ERR_CUDA;
    return launch_err();
}
