// Attention of chunks of new tokens over the 4-bit key/value cache on the
// tensor cores, GB300 (sm_103a).  Contract: hs_kv4_attention in hs.h; the
// division of the work: hs_kv4_sched.cuh.
//
// A CTA takes 256 query rows (tokens x the query heads of one kv head) against
// tiles of 128 keys: two row tiles of 128, each S = Q K^T (tcgen05, fp16
// operands, fp32 in tensor memory), its softmax, and O += P V with P read from
// tensor memory where S stood.  Roles, one CTA an SM:
//   warps 0-3, 4-7   a row tile each, a thread a row: queries in, softmax, output
//   warp 12          copies packed codes and pairs, page by page
//   warp 13          issues the matrix products
//   warps 8-11, 14, 15   take the codes apart: K and V tiles of 128 keys in fp16
// The two row tiles take turns: one's softmax runs under the other's products,
// and both use a K and V tile that was taken apart once.  Keys and values are
// scale * code + bias rounded once to fp16; channels stand in both operands in
// the order in which a word's nibbles come apart ([0 4 1 5 2 6 3 7] of each
// eight), which the output undoes.
//
// Bounds, for 256 rows x 128 keys at head_dim 128 on one SM: the products 2048
// cycles at the dense fp16 rate, the exponentials 1024 to 2048, the softmax's
// other arithmetic about 1000 issue cycles, taking codes apart about 500.  A
// row tile's scores, softmax and output follow one another (tensor memory holds
// no second set of scores beside 2 x 128 columns of scores and outputs at head_dim 128), so
// that a tile takes 3500 cycles for both; an item costs some 12,000 more: filling,
// draining, writing.  A prompt of 4096 tokens (32 / 8 heads of 128 channels):
// 148 us, 926 TFLOP/s, 48% of the measured bf16 peak; within long items 1340 TFLOP/s.
#include "hs_kv4_join.cuh"
#include "hs_tc.cuh"

namespace hs {

constexpr int kPfKeys = 128, kPfRows = 256, kPfPacked = 3, kPfSlots = 3, kPfInfo = 8;
constexpr int kPfThreads = 16 * 32;
constexpr int kPfApart = 6;  // warps that take codes apart
constexpr int kPfMaxSmem = 227 * 1024 - 2048;  // dynamic; the rest is the static part
constexpr float kPfUp = 6.f;  // probabilities are held times 2^6: at most 2^14 in fp16, and small ones keep their bits

template <int D>
struct PrefillCfg {
    static constexpr int kNg = D / 64;
    static constexpr int kQBytes = 128 * D * 2;          // of a row tile
    static constexpr int kTileBytes = kPfKeys * D * 2;   // a K or V tile
    static constexpr int kPackedBytes = kPfKeys * (D / 2 + 4 * kNg);
    static constexpr int kPiecesRoom = 2 * kQBytes + kPfSlots * kTileBytes + kPfPacked * kPackedBytes;  // all before the output buffers
    static constexpr int kFixed = kPiecesRoom + 8 * 2048;
    static constexpr int smem(int n_seqs) { return 1024 + kFixed + 1024 + (n_seqs + 1) * 4; }
};

struct PfShared {
    uint64_t packed_full[kPfPacked], packed_empty[kPfPacked], kv_full[kPfSlots], kv_empty[kPfSlots];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    uint32_t gone[kPfInfo];            // per key tile: blocks of 16 keys that are not there
    uint32_t nan_any[kPfInfo];         // some value of the tile is NaN
    uint32_t nan_keys[kPfInfo][2][4];  // by group of channels: the keys whose values are
    uint32_t tmem;
    // (Behind what every tile reads: before it, with those words elsewhere, chunks took 1% more.)
    uint64_t pieces_full, products_done;
    int join_last[2];   // by row tile
    int direct[2][2];   // by end of the run (0: its first piece) and row tile: the item's other piece is there
};

// Shared-memory descriptor of a tile whose rows run along K (keys) and whose
// 128-byte swizzled lines hold 64 elements along N: `lead` bytes to the next 64
// along N, 1024 to the next 8 rows.
__device__ __forceinline__ uint64_t umma_desc_sw128_mn(uint32_t smem_addr, uint32_t lead) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(lead >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }

__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)), "l"(reinterpret_cast<uint64_t&>(z)));
    return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(x)), "l"(reinterpret_cast<uint64_t&>(y)));
    return r;
}
// (x & mask) | bits, one instruction (the constants in registers).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
    return r;
}

// Eight codes of a word as scale * code + bias in fp16: 1024 + c is exact in
// fp16, so is c after the subtraction, and the product is rounded once.
__device__ __forceinline__ uint4 take_apart(uint32_t w, __half2 s, __half2 b) {
    const __half2 k = as_h2(0x64006400u);
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = as_u32(__hfma2(__hsub2(as_h2(and_or(w >> (4 * i), 0x000f000fu, 0x64006400u)), k), s, b));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// A call of its own: its registers are not the softmax's.
template <int D>
__device__ __noinline__ void add_pieces_apart(const KvAttnArgs& a, const KvWalk& w, int warp, int warps, int row0, int row1, int c, int first,
                                              int step, int count, bool final) {
    add_pieces<D, 4, 2>(a, w, warp, warps, row0, row1, c, first, step, count, final);
}

// The same by the 256 softmax threads of a CTA that has no work left: its
// shared memory is free, and the pieces (at most kJoin of them) come in whole by
// bulk copies.  A few loops of little code: that of add_pieces runs once a call, and
// costs fetching it besides the rounds of loads (48 rows of five pieces: 9,400
// cycles, here 5,800; 16 requests of three drafts gained 1.6 of 25.2 us).  The
// operations and their order are those of add_pieces.
template <int D>
__device__ __noinline__ void add_pieces_at_end(const KvAttnArgs& a, const KvWalk& w, int c, int count, int rows) {
    constexpr int kL = D / 8, kR = 32 / kL, kP = kJoin / kL, kAtOnce = 4;
    const int tid = threadIdx.x, lane = tid & 31, sub = lane / kL, i8 = lane % kL;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* room = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* buffers = room + PrefillCfg<D>::kPiecesRoom;
    float* weights = reinterpret_cast<float*>(buffers);  // [row][kJoin]
    uint64_t* bar = &reinterpret_cast<PfShared*>(buffers + 8 * 2048)->pieces_full;
    const uint32_t bytes = (uint32_t)(rows * D * 4);
    float* inv = weights + 128 * kJoin;
    if (tid == 224) {  // (of the idle row tile)
        asm volatile("fence.proxy.async;" ::: "memory");  // the other CTAs' writes, seen by the arrival before
        mbar_arrive_expect_tx(bar, bytes * (uint32_t)count);
        for (int i = 0; i < count; ++i)
            bulk_g2s(room + i * bytes, a.part_o + piece_slot(c, i) * a.rows * D, bytes, bar, policy_evict_first());
    }
    __syncwarp();
#pragma unroll 1
    for (int r0 = (tid >> 5) * kR; r0 < rows; r0 += kAtOnce * 8 * kR) {
        float wt[kAtOnce][kP], part[kAtOnce][kP], m[kAtOnce], l;
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
            const int row = min(r0 + x * 8 * kR + sub, rows - 1);
            m[x] = kNoMax;
#pragma unroll
            for (int y = 0; y < kP; ++y) {
                float2 ml = make_float2(kNoMax, 0.f);
                if (i8 + y * kL < count) ml = __ldcg(a.part_ml + (uint32_t)(piece_slot(c, i8 + y * kL) * a.rows + row));
                wt[x][y] = ml.x, part[x][y] = ml.y;
                m[x] = fmaxf(m[x], ml.x);
            }
        }
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
            const int row = r0 + x * 8 * kR + sub;
            if (r0 + x * 8 * kR >= rows) break;
            weigh<kL, kP>(wt[x], part[x], i8, count, m[x], l);
            if (row >= rows) continue;
#pragma unroll
            for (int y = 0; y < kP; ++y) weights[row * kJoin + i8 + y * kL] = wt[x][y];
            if (i8 == 0) inv[row] = l != 0.f ? 1.f / l : 0.f;
        }
    }
    asm volatile("bar.sync 3, 256;" ::: "memory");
    if (!mbar_wait(bar, 0)) {
        mbar_wait(bar, 0);  // once more: the copies under way write into this CTA's shared memory
        return;
    }
#pragma unroll 1
    for (int at = tid; at < rows * kL; at += 256) {
        const int row = at / kL, d = at % kL * 8, tok = kv_row_token(a, row);
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll 4
        for (int i = 0; i < count; ++i) {
            const float f = weights[row * kJoin + i];
            const float4* v = reinterpret_cast<const float4*>(room + i * bytes + (row * D + d) * 4);
            const float4 v0 = v[0], v1 = v[1];
            const float from[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(f, from[e], acc[e]);
        }
        *reinterpret_cast<uint4*>(a.out + (long long)(w.row0 + w.r * a.tq + tok) * a.o_st +
                                  (long long)(w.head * a.group + row - tok * a.group) * a.o_sh + d) = pack_bf16x8(acc, inv[row]);
    }
}

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1) kv4_prefill_kernel(const KvAttnArgs a) {
    using C = PrefillCfg<D>;
    constexpr int NG = C::kNg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* q_s = smem;                                    // [2] row tiles
    uint8_t* kv_s = smem + 2 * C::kQBytes;                  // [kPfSlots] K and V tiles in turn
    uint8_t* packed_s = kv_s + kPfSlots * C::kTileBytes;    // [kPfPacked] codes, pairs
    uint8_t* out_s = packed_s + kPfPacked * C::kPackedBytes;  // [8] warps' buffers of 32 rows of 64 bytes
    PfShared& sh = *reinterpret_cast<PfShared*>(out_s + 8 * 2048);
    static_assert(sizeof(PfShared) <= 1024, "barriers");
    uint32_t* cum = reinterpret_cast<uint32_t*>(out_s + 8 * 2048 + 1024);
    const int *qs = a.q_start, *ls = a.seq_len;  // looked at once an item: no room here for 4096 requests' copies
    // (Reductions of values that all lanes share: they come out in uniform registers,
    // which the tensor-core instructions' operands have to be in.)
    const int tid = threadIdx.x, lane = tid & 31, warp = (int)warp_max_u32(threadIdx.x >> 5);

    if (tid == 0) {
        for (int i = 0; i < kPfPacked; ++i) mbar_init(sh.packed_full + i, 1), mbar_init(sh.packed_empty + i, kPfApart);
        for (int i = 0; i < kPfSlots; ++i) mbar_init(sh.kv_full + i, kPfApart), mbar_init(sh.kv_empty + i, 1);
        for (int i = 0; i < 2; ++i)
            mbar_init(sh.q_full + i, 4), mbar_init(sh.s_full + i, 1), mbar_init(sh.p_full + i, 4), mbar_init(sh.o_full + i, 1);
        mbar_init(&sh.pieces_full, 1);
        mbar_init(&sh.products_done, 1);
        fence_mbar_init();
    }
    if (tid < kPfInfo) {
        sh.nan_any[tid] = 0;
        for (int i = 0; i < 8; ++i) sh.nan_keys[tid][i >> 2][i & 3] = 0;
    }
    if (warp == 13) tmem_alloc(&sh.tmem, 512);
    pdl_wait();
    pdl_trigger();
    tc_fence_before();
    kv_schedule(a, qs, ls, cum);
    tc_fence_after();
    const uint32_t tmem = warp_max_u32(sh.tmem);  // S and P of the row tiles at columns 0 and 128, O at 256 and 384
    // A warp's place in the line, in shared memory: looked at once an item.
    __shared__ KvWalk walks[kPfThreads / 32], coming[8];
    KvWalk& w = walks[warp];
    if (warp == 0) walks[0] = kv_begin(a, qs, ls, cum);
    __syncthreads();
    if (warp) w = walks[0];
    __syncthreads();
    auto next_piece = [&]() {
        KvWalk n = w;
        kv_next_piece(a, qs, ls, n);
        __syncwarp();
        w = n;
        __syncwarp();
    };
    // 128 registers a thread at launch: 184 for the softmax, 72 for the others (2 * 184 + 2 * 72 = 4 * 128).
    auto rows_of = [&](const KvWalk& v) { return min(a.tq, v.n - v.r * a.tq) * a.group; };

    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 12) {
        // ---- packed codes and pairs: K then V of each tile, two copies a page
        const int per_tile = kPfKeys >> a.g.page_log2, codes = (D / 2) << a.g.page_log2, pairs = (NG * 4) << a.g.page_log2;
        const int pg = lane >> 1, what = lane & 1;  // lane: codes or pairs of page pg of a tile
        uint32_t f = 0, tiles = 0;
        bool dead = false;
        for (; w.left > 0 && !dead; next_piece()) {
            const int cnt = kv_piece_tiles(w);
            int base = -1, held = -1;
            for (int k = 0; k < cnt && !dead; ++k, ++tiles) {
                const int p0 = (w.lo + w.tile + k) * per_tile;
                if (base < 0 || p0 - base >= 32) {  // the next 32 table entries, one a lane
                    base = p0;
                    const bool in = w.hi >= w.lo && (long long)(base + lane) << a.g.page_log2 < w.len;
                    held = in ? a.table[(size_t)w.seq * a.width + base + lane] : -1;
                }
                const int page = __shfl_sync(~0u, held, (p0 - base + pg) & 31);
                const bool here = pg < per_tile && (uint32_t)page < (uint32_t)a.g.n_pages;
                const unsigned mask = __ballot_sync(~0u, here);
                for (int v = 0; v < 2; ++v, ++f) {
                    const int st = f % kPfPacked;
                    if (f >= kPfPacked && !warp_wait(sh.packed_empty + st, (f / kPfPacked + 1) & 1)) {
                        dead = true;
                        break;
                    }
                    if (lane == 0) {
                        if (v == 0) {
                            uint32_t gone = 0;
                            for (int i = 0; i < 8; ++i)
                                if (!((mask >> (2 * (i * 16 >> a.g.page_log2))) & 1u)) gone |= 1u << i;
                            sh.gone[tiles % kPfInfo] = gone;
                        }
                        mbar_arrive_expect_tx(sh.packed_full + st, (uint32_t)(__popc(mask) >> 1) * (uint32_t)(codes + pairs));
                    }
                    __syncwarp();
                    if (here) {
                        const uint8_t* src = kv_record(a.g, page, w.head) + (what ? 2 * codes + v * pairs : v * codes);
                        uint8_t* dst = packed_s + st * C::kPackedBytes + (what ? kPfKeys * (D / 2) + pg * pairs : pg * codes);
                        bulk_g2s(dst, src, (uint32_t)(what ? pairs : codes), sh.packed_full + st, policy_evict_last());
                    }
                }
            }
        }
        // Where a wait gave up, here or in the warps that use the copies, the last ones may
        // still be under way; the CTA stays until they have come.
        for (uint32_t i = f > kPfPacked ? f - kPfPacked : 0; i < f; ++i) mbar_wait(sh.packed_full + i % kPfPacked, (i / kPfPacked) & 1);
    } else if (warp == 13) {
        // ---- matrix products, issued by one lane
        constexpr uint32_t idesc_s = umma_idesc_f16_f32(128, kPfKeys);
        constexpr uint32_t idesc_o = umma_idesc_f16_f32(128, D) | (1u << 16);  // V: rows along K
        const uint32_t q_at = smem_u32(q_s), kv_at = smem_u32(kv_s);
        uint32_t slot = 0, phase = 0, p_phase[2] = {0, 0}, q_phase[2] = {0, 0};  // slot: of the next K tile
        bool dead = false;
        auto wait = [&](uint64_t* bar, uint32_t parity) { dead |= !warp_wait(bar, parity); };
        while (w.left > 0 && !dead) {
            const int cnt = (int)warp_max_u32((uint32_t)kv_piece_tiles(w));
            const bool two = warp_max_u32((uint32_t)rows_of(w)) > 128u;
            uint32_t v_slot = 0, v_phase = 0;  // of the V tile before
            for (int k = 0; k <= cnt && !dead; ++k) {
                // tile k's scores and tile k - 1's outputs, a row tile at a time
                if (k) wait(sh.kv_full + v_slot, v_phase);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if ((x && !two) || dead) continue;
                    if (k) {
                        wait(sh.p_full + x, p_phase[x]);
                        p_phase[x] ^= 1;
                    } else {
                        wait(sh.q_full + x, q_phase[x]);
                        q_phase[x] ^= 1;
                    }
                    if (dead) continue;
                    const bool last = x || !two;
                    if (k) {  // O += P V
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t vd = umma_desc_sw128_mn(kv_at + v_slot * C::kTileBytes, kPfKeys * 128);
#pragma unroll
                            for (int kk = 0; kk < kPfKeys / 16; ++kk)
                                umma_f16_tmem_a(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, vd + kk * (2048 >> 4), idesc_o, kk ? 1 : k > 1);
                            if (k == cnt) umma_commit(sh.o_full + x);
                            if (last) umma_commit(sh.kv_empty + v_slot);
                        }
                        __syncwarp();
                    }
                    if (k < cnt) {  // S = Q K^T; the tile of K has had the outputs' time to come
                        if (!x) wait(sh.kv_full + slot, phase);
                        if (dead) continue;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t qd = umma_desc_sw128(q_at + x * C::kQBytes), kd = umma_desc_sw128(kv_at + slot * C::kTileBytes);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t at = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
                                umma_f16(tmem + x * 128, qd + at, kd + at, idesc_s, kk != 0);
                            }
                            umma_commit(sh.s_full + x);
                            if (last) umma_commit(sh.kv_empty + slot);
                        }
                    }
                    __syncwarp();
                }
                if (k < cnt) {  // K k, V k, K k + 1 follow one another round the ring
                    v_slot = slot + 1 == kPfSlots ? 0 : slot + 1;
                    v_phase = slot + 1 == kPfSlots ? phase ^ 1 : phase;
                    const uint32_t next = v_slot + 1 == kPfSlots ? 0 : v_slot + 1;
                    phase = v_slot + 1 == kPfSlots ? v_phase ^ 1 : v_phase;
                    slot = next;
                }
            }
            next_piece();
        }
        // The products read shared memory and write tensor memory, which is given back below.
        if (elect_one()) umma_commit(&sh.products_done);
        __syncwarp();
        mbar_wait(&sh.products_done, 0);
    } else {
        // ---- codes taken apart into swizzled fp16 tiles
        const int idx = (warp < 12 ? warp - 8 : warp - 10) * 32 + lane;  // of 192
        uint32_t f = 0, tiles = 0;
        bool dead = false;
        for (; w.left > 0 && !dead; next_piece()) {
            const int cnt = kv_piece_tiles(w);
            for (int k = 0; k < cnt && !dead; ++k, ++tiles) {
                const int key0 = (w.lo + w.tile + k) * kPfKeys, info = tiles % kPfInfo;
                for (int v = 0; v < 2; ++v, ++f) {
                    const int st = f % kPfPacked, slot = f % kPfSlots;
                    if (!warp_wait(sh.packed_full + st, (f / kPfPacked) & 1)) {
                        dead = true;
                        break;
                    }
                    // 32 channels of a key at a time, into registers while the tile's place may
                    // still be in use; eight lanes that store together hold four keys and both
                    // halves of a 128-byte line: no two in one bank.
                    constexpr int kItems = kPfKeys * 2 * NG, kMine = (kItems + 32 * kPfApart - 1) / (32 * kPfApart);
                    const uint32_t gone = sh.gone[info];
                    const uint8_t* from = packed_s + st * C::kPackedBytes;
                    uint4 q[kMine];
                    uint32_t sb[kMine];
                    bool nan = false;
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        const int id = idx + i * 32 * kPfApart;
                        const int key = NG == 1 ? id >> 1 : (id >> 1 & 3) | (id >> 4) << 2, c = NG == 1 ? id & 1 : (id & 1) | (id >> 2 & 2);
                        if (kItems % (32 * kPfApart) == 0 || id < kItems) {
                            q[i] = *reinterpret_cast<const uint4*>(from + key * (D / 2) + c * 16);
                            sb[i] = *reinterpret_cast<const uint32_t*>(from + kPfKeys * (D / 2) + (key * NG + (c >> 1)) * 4);
                            if (key0 + key >= w.len || (gone >> (key >> 4)) & 1u) sb[i] = 0;
                            nan |= (sb[i] & 0x7c000000u) == 0x7c000000u;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sh.packed_empty + st);
                    if (v == 0 && idx < 9) {  // for four tiles on: no warp here is two ahead of another
                        const int on = (tiles + 4) % kPfInfo;
                        if (idx == 8) sh.nan_any[on] = 0;
                        else sh.nan_keys[on][idx >> 2][idx & 3] = 0;
                    }
                    if (v && nan) {  // a NaN value must not meet the zero probability of a row that does not see it
#pragma unroll
                        for (int i = 0; i < kMine; ++i) {
                            const int id = idx + i * 32 * kPfApart;
                            const int key = NG == 1 ? id >> 1 : (id >> 1 & 3) | (id >> 4) << 2, c = NG == 1 ? id & 1 : (id & 1) | (id >> 2 & 2);
                            if (id < kItems && (sb[i] & 0x7c000000u) == 0x7c000000u) {
                                atomicOr(&sh.nan_keys[info][c >> 1][key >> 5], 1u << (key & 31));
                                sh.nan_any[info] = 1;
                                sb[i] = 0;
                            }
                        }
                    }
                    if (f >= kPfSlots && !warp_wait(sh.kv_empty + slot, (f / kPfSlots + 1) & 1)) {
                        dead = true;
                        break;
                    }
                    uint8_t* to = kv_s + slot * C::kTileBytes;
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        const int id = idx + i * 32 * kPfApart;
                        const int key = NG == 1 ? id >> 1 : (id >> 1 & 3) | (id >> 4) << 2, c = NG == 1 ? id & 1 : (id & 1) | (id >> 2 & 2);
                        if (kItems % (32 * kPfApart) == 0 || id < kItems) {
                            const __half2 p = as_h2(sb[i]), s = __low2half2(p), b = __high2half2(p);
                            uint8_t* line = to + (c >> 1) * (kPfKeys * 128) + key * 128;
                            const uint32_t words[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                *reinterpret_cast<uint4*>(line + ((((c & 1) * 4 + x) ^ (key & 7)) << 4)) = take_apart(words[x], s, b);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sh.kv_full + slot);
                }
            }
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ---- a row tile's queries, softmax and output, a thread a row
        const int x = warp >> 2, row = tid & 127, r = x * 128 + row;
        const uint32_t tl = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
        const int back_keys = a.back;  // taken off no position before 0: no overflow
        uint32_t tiles = 0, s_count = 0, o_count = 0;
        bool dead = false;
        // The warp's 32 rows of a piece's queries, a row by D / 8 lanes: fetched as they are
        // into the lines of the tile that they will fill (16-byte chunk c of a row at place c
        // of its line), ...
        constexpr int kL = D / 8, kAt = 32 / kL, kB = 32 / kAt;  // lanes a row, rows at a time
        const int sub = lane / kL, c = lane % kL;
        uint8_t* q_lines = q_s + x * C::kQBytes + (c >> 3) * (128 * 128) + ((warp & 3) * 32 + sub) * 128;
        auto fetch_q = [&](const KvWalk& v) {
            const int nr = rows_of(v);
#pragma unroll 4
            for (int i = 0; i < kB; ++i) {
                const int qr = x * 128 + (warp & 3) * 32 + i * kAt + sub, qt = kv_row_token(a, qr);
                uint8_t* dst = q_lines + i * kAt * 128 + (c & 7) * 16;
                if (qr < nr)
                    cp_async16_hint(dst, a.q + (long long)(v.row0 + v.r * a.tq + qt) * a.q_st +
                                             (long long)(v.head * a.group + qr - qt * a.group) * a.q_sh + c * 8, policy_evict_first());
                else
                    *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
            }
        };
        // ... then put into fp16 in place, each row scaled by the power of two that brings its
        // largest channel to [2^8, 2^9), whatever stands in the others: bf16 values down to 2^-25
        // of it stay exact, smaller ones move a score by less than 2^-33 of the largest channel's
        // part.  A lane looks at its own row (eight lanes at eight places of the lines: no
        // two in one bank).  Returns that row's factor of the scores.
        auto convert_q = [&]() -> float {
            cp_async_wait_all();
            __syncwarp();
            const uint8_t* own = q_s + x * C::kQBytes + ((warp & 3) * 32 + lane) * 128;
            uint32_t top = 0;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(own + (i >> 3) * (128 * 128) + (((i ^ lane) & 7) << 4));
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) top = max(top, max(u[j] & 0x7fff0000u, (u[j] << 16) & 0x7fff0000u));
            }
            int e = (int)(top >> 23);
            const bool none = e >= kNoQuery;
            e = e == 0 || none ? 0 : max(-110, e - 127);  // a row of zeros keeps 2^8
            const float row_f = none ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 + 8 - e) << 23);
#pragma unroll 4
            for (int i = 0; i < kB; ++i) {
                const float f = __shfl_sync(~0u, row_f, i * kAt + sub);
                uint8_t* line = q_lines + i * kAt * 128;
                const uint4 v = *reinterpret_cast<const uint4*>(line + (c & 7) * 16);
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // channels j and j + 4
                    const uint32_t lo = u[j >> 1], hi = u[2 + (j >> 1)];
                    h[j] = as_u32(__floats2half2_rn(__uint_as_float(j & 1 ? lo & 0xffff0000u : lo << 16) * f,
                                                    __uint_as_float(j & 1 ? hi & 0xffff0000u : hi << 16) * f));
                }
                __syncwarp();  // the line has been read
                *reinterpret_cast<uint4*>(line + (((c & 7) ^ ((i * kAt + sub) & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(sh.q_full + x);
            return kv_score_range(a.scale_log2 * __uint_as_float((uint32_t)(127 - 8 + e) << 23));
        };
        float sc = 0.f;
        if (w.left > 0 && x * 128 < rows_of(w)) {
            fetch_q(w);
            sc = convert_q();
        }
        while (w.left > 0) {
            const int cnt = kv_piece_tiles(w), nrows = rows_of(w), ctx = w.len - w.n;
            const bool whole = cnt == w.tiles, two = nrows > 128;
            // An item's pieces are joined by row tile, by the warps of the row tile (the counters
            // of the second lie 228 further on); by all eight where there is one row tile.
            auto joined = [&]() { return a.joined + (two ? x * (kKvMaxCtas / 2) : 0); };
            auto lead = [&]() { return lane == 0 && (two ? (warp & 3) == 0 : warp == 0); };
            auto meet = [&]() {
                if (!two)
                    asm volatile("bar.sync 3, 256;" ::: "memory");
                else if (x)
                    asm volatile("bar.sync 2, 128;" ::: "memory");
                else
                    asm volatile("bar.sync 1, 128;" ::: "memory");
            };
            KvPieces of{0, 1};
            // Of an item's two pieces the second comes at the start of a run, the first at the end
            // of one, when the other's sums have long been in memory: they are added on the way
            // out, and this piece is never written (and read again, with both row tiles waiting).
            auto other_is_there = [&]() { return of.count == 2 && (meet(), *(volatile int*)&sh.direct[w.tile == 0][two ? x : 0] != 0); };
            KvWalk& nx = coming[warp];  // the piece after this one
            {
                KvWalk n = w;
                kv_next_piece(a, qs, ls, n);
                __syncwarp();
                nx = n;
                __syncwarp();
            }
            const bool more = nx.left > 0 && x * 128 < rows_of(nx);
            if (x * 128 >= nrows && more) {  // this row tile has been idle
                fetch_q(nx);
                sc = convert_q();
            }
            bool direct = false;
            if (x * 128 < nrows) {
                const bool valid = r < nrows;
                const int lim = ctx + w.r * a.tq + kv_row_token(a, r);
                const int low = max(lim, 0) - back_keys;  // the row's first key
                const int min_lim = -warp_max_s32(valid ? -lim : -0x7fffffff), max_lim = warp_max_s32(valid ? lim : -1);

                float m = kNoMax, l = 0.f;
                const float own_sc = sc;  // (kv_score_factor)
                uint32_t nan = 0;  // by group: the row sees a value that is NaN
                auto see_nan = [&](int k) {  // of tile k of the piece
                    const int info = (tiles + k) % kPfInfo, key0 = (w.lo + w.tile + k) * kPfKeys;
                    if (!*(volatile uint32_t*)&sh.nan_any[info]) return;
                    for (int i = 0; i < NG * 4; ++i)
                        for (uint32_t b = sh.nan_keys[info][i >> 2][i & 3]; b; b &= b - 1) {
                            const int key = key0 + (i & 3) * 32 + __ffs(b) - 1;
                            if (key <= lim && key >= max(lim, 0) - back_keys) nan |= 1u << (i >> 2);
                        }
                };
                for (int k = 0; k < cnt && !dead; ++k) {
                    const int key0 = (w.lo + w.tile + k) * kPfKeys;
                    if (!warp_wait(sh.s_full + x, s_count++ & 1)) {
                        dead = true;
                        break;
                    }
                    tc_fence_after();
                    if (k == cnt - 1 && more) fetch_q(nx);  // the last scores are there: the queries' place is free
                    if (k) see_nan(k - 1);  // its values have been taken apart: its product is done
                    const uint32_t gone = sh.gone[(tiles + k) % kPfInfo];
                    const bool masked = gone || key0 + kPfKeys - 1 > min_lim || key0 < max(max_lim, 0) - back_keys;
                    float v[kPfKeys];
#pragma unroll
                    for (int c = 0; c < kPfKeys / 32; ++c) tmem_ld32_async(tl + x * 128 + c * 32, v + c * 32);
                    tmem_ld_wait(v);
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < kPfKeys; ++i) {
                            const int key = key0 + i;
                            if (key > lim || key < low || ((gone >> (i >> 4)) & 1u)) v[i] = -INFINITY;
                        }
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < kPfKeys; i += 2) m4[(i >> 1) & 3] = fmaxf(m4[(i >> 1) & 3], fmaxf(v[i], v[i + 1]));
                    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    if (__any_sync(~0u, fmaf(mx, sc, -m) > kLazy)) {  // rare: raise the maximum and bring the sums to it
                        const float y = mx * sc, nm = fmaxf(m, y), f = ex2(m - nm);
                        if (y > m && (sc != own_sc || fabsf(y) >= kFarScore)) {
                            sc = kv_score_factor(mx, own_sc);
                            m = mx * sc;
                        } else {
                            m = nm;
                        }
                        l *= f;
                        if (k) {
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                float o[16];
                                uint32_t u[16];
                                tmem_ld16(tl + 256 + x * 128 + c * 16, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i] * f);
                                tmem_st16(tl + 256 + x * 128 + c * 16, u);
                                tmem_st_wait();
                            }
                        }
                    }
                    const float2 sc2 = make_float2(sc, sc), mo2 = make_float2(kPfUp - m, kPfUp - m);
                    float2 l2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int h = 0; h < kPfKeys / 32; ++h) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 e = fma2(make_float2(v[h * 32 + 2 * i], v[h * 32 + 2 * i + 1]), sc2, mo2);
                            e.x = ex2(e.x), e.y = ex2(e.y);
                            l2[i & 3] = add2(l2[i & 3], e);
                            p[i] = as_u32(__floats2half2_rn(e.x, e.y));
                        }
                        tmem_st16(tl + x * 128 + h * 16, p);  // over the scores
                    }
                    tmem_st_wait();
                    l2[0] = add2(add2(l2[0], l2[1]), add2(l2[2], l2[3]));
                    l += l2[0].x + l2[0].y;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sh.p_full + x);
                }
                if (sc != own_sc) m = kv_whole_max(m, sc, own_sc);
                if (!whole) {
                    of = kv_pieces(a, w, cum[a.n_seqs]);
                    if (of.count == 2 && lead()) {
                        int there;
                        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(there) : "l"(joined() + of.c) : "memory");
                        sh.direct[w.tile == 0][two ? x : 0] = there;
                        if (there) joined()[of.c] = 0;  // for the next call
                    }
                }
                // The next piece's first scores are worked out while this one is written.
                const float next_sc = more ? convert_q() : 0.f;
                if (!dead && !warp_wait(sh.o_full + x, o_count++ & 1)) dead = true;
                direct = other_is_there();
                if (!dead) {
                    tc_fence_after();
                    see_nan(cnt - 1);
                    const uint32_t at = (2 * blockIdx.x + (w.tile == 0 ? 1 : 0)) * (uint32_t)a.rows + r;
                    // The other piece's row, and the weights of both: the operations of add_pieces,
                    // so that the result is the same whoever comes last.
                    const uint32_t other = (w.tile == 0 ? 2 * blockIdx.x + 2 : 2 * blockIdx.x - 1) * (uint32_t)a.rows;
                    float mine = 1.f, its = 0.f;
                    if (direct) {
                        const float2 ml = valid ? __ldcg(a.part_ml + other + r) : make_float2(kNoMax, 0.f);
                        const float top = fmaxf(m, ml.x);
                        mine = ex2(m - top), its = ex2(ml.x - top);
                        l = __fadd_rn(__fmul_rn(mine, l), __fmul_rn(its, ml.y));
                    }
                    const float inv = l != 0.f ? 1.f / l : 0.f;
                    // 64 bytes of each of the warp's rows at a time, by way of a buffer (chunk j of
                    // row i at j ^ (i / 2 % 4): no two in one bank), so that four lanes write a row's
                    // 64 bytes together: a thread writing its own row took the load-store unit 4000
                    // cycles a piece.
                    int ln = lane, wq = warp & 3;
                    asm volatile("" : "+r"(ln), "+r"(wq));  // (what follows from them is not kept through the loop above)
                    uint8_t* buf = out_s + warp * 2048;
                    auto write64 = [&](const uint4 (&u)[4], uint8_t* base, bool part, int d) {
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(buf + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) = u[j];
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int orow = i * 8 + (lane >> 2), qr = x * 128 + (warp & 3) * 32 + orow, qt = kv_row_token(a, qr);
                            const uint4 z = *reinterpret_cast<const uint4*>(buf + orow * 64 + (((lane & 3) ^ (orow >> 1 & 3)) << 4));
                            if (qr >= nrows) continue;
                            uint8_t* dst = part ? base + ((at - r + qr) * (uint32_t)D + d) * (size_t)4
                                                : base + ((long long)qt * a.o_st + (long long)(qr - qt * a.group) * a.o_sh + d) * 2;
                            *reinterpret_cast<uint4*>(dst + (lane & 3) * 16) = z;
                        }
                    };
                    // The same with the other piece's sums, four channels a lane.
                    float4 its_rows[4];  // the next 16 channels of the other piece
                    auto fetch_its = [&](int d) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int qr = min(x * 128 + wq * 32 + i * 8 + (ln >> 2), nrows - 1);
                            its_rows[i] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (other + qr) * (uint32_t)D + d) + (ln & 3));
                        }
                    };
                    auto add64 = [&](const uint4 (&u)[4], uint8_t* base, int d) {
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(buf + ln * 64 + ((j ^ (ln >> 1 & 3)) << 4)) = u[j];
                        float4 y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = its_rows[i];
                        if (d + 16 < D) fetch_its(d + 16);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int orow = i * 8 + (ln >> 2), qr = x * 128 + wq * 32 + orow, qt = kv_row_token(a, qr);
                            const float4 z = *reinterpret_cast<const float4*>(buf + orow * 64 + (((ln & 3) ^ (orow >> 1 & 3)) << 4));
                            const float f = __shfl_sync(~0u, mine, orow), g = __shfl_sync(~0u, its, orow), n = __shfl_sync(~0u, inv, orow);
                            const bool ahead = w.tile == 0;  // this piece's keys come first
                            const float f0 = ahead ? f : g, f1 = ahead ? g : f;
                            auto sum = [&](float u, float v) { return __fmaf_rn(f1, ahead ? v : u, __fmaf_rn(f0, ahead ? u : v, 0.f)) * n; };
                            const __nv_bfloat162 lo = __floats2bfloat162_rn(sum(z.x, y[i].x), sum(z.y, y[i].y)),
                                                 hi = __floats2bfloat162_rn(sum(z.z, y[i].z), sum(z.w, y[i].w));
                            if (qr >= nrows) continue;
                            uint8_t* dst = base + ((long long)qt * a.o_st + (long long)(qr - qt * a.group) * a.o_sh + d) * 2;
                            *reinterpret_cast<uint2*>(dst + (ln & 3) * 8) =
                                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                        }
                    };
                    uint8_t* out0 = reinterpret_cast<uint8_t*>(a.out + (long long)(w.row0 + w.r * a.tq) * a.o_st + (long long)w.head * a.group * a.o_sh);
                    if (whole) {
#pragma unroll 1
                        for (int d = 0; d < D; d += 32) {
                            float v[32];
                            tmem_ld32(tl + 256 + x * 128 + d, v);
                            if ((nan >> (d >> 6)) & 1u) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(0x7fc00000u);
                            }
                            uint4 u[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t z[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int from = 8 * j + (i & 1) * 4 + (i >> 1);  // channels 2i and 2i + 1 of eight
                                    const __nv_bfloat162 y = __floats2bfloat162_rn(v[from] * inv, v[from + 2] * inv);
                                    z[i] = *reinterpret_cast<const uint32_t*>(&y);
                                }
                                u[j] = make_uint4(z[0], z[1], z[2], z[3]);
                            }
                            write64(u, out0, false, d);
                        }
                    } else if (direct) {
                        fetch_its(0);
#pragma unroll 1
                        for (int d = 0; d < D; d += 16) {
                            float v[16];
                            tmem_ld16(tl + 256 + x * 128 + d, v);
                            if ((nan >> (d >> 6)) & 1u) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(0x7fc00000u);
                            }
                            uint4 u[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int from = 8 * (j >> 1) + (j & 1);  // channels 0-3 or 4-7 of eight
                                u[j] = make_uint4(__float_as_uint(v[from]), __float_as_uint(v[from + 2]), __float_as_uint(v[from + 4]),
                                                  __float_as_uint(v[from + 6]));
                            }
                            add64(u, out0, d);
                        }
                    } else {
#pragma unroll 1
                        for (int d = 0; d < D; d += 16) {
                            float v[16];
                            tmem_ld16(tl + 256 + x * 128 + d, v);
                            if ((nan >> (d >> 6)) & 1u) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(0x7fc00000u);
                            }
                            uint4 u[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int from = 8 * (j >> 1) + (j & 1);  // channels 0-3 or 4-7 of eight
                                u[j] = make_uint4(__float_as_uint(v[from]), __float_as_uint(v[from + 2]), __float_as_uint(v[from + 4]),
                                                  __float_as_uint(v[from + 6]));
                            }
                            write64(u, reinterpret_cast<uint8_t*>(a.part_o), true, d);
                        }
                    }
                    if (valid && !whole && !direct) a.part_ml[at] = make_float2(m, l);
                    tc_fence_before();
                }
                sc = next_sc;
            } else if (!whole) {
                of = kv_pieces(a, w, cum[a.n_seqs]);
                direct = other_is_there();
            }
            tiles += cnt;
            if (!whole && !direct) {
                join_pieces(of, joined(), lead(), &sh.join_last[two ? x : 0], meet, [&](int first, int step, int count, bool final) {
                    const bool at_end = !two && nx.left == 0 && of.count <= kJoin;  // (no copy or product is under way then)
                    if (at_end && count * rows_of(w) * D * 4 <= C::kPiecesRoom) {
                        add_pieces_at_end<D>(a, w, of.c, count, rows_of(w));
                        return;
                    }
                    add_pieces_apart<D>(a, w, two ? warp & 3 : warp, two ? 4 : 8, two ? x * 128 : 0, two && !x ? 128 : nrows, of.c, first, step,
                                        count, final);
                });
            }
            __syncwarp();
            w = nx;
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) tmem_dealloc(tmem, 512);
}

template <int D>
int launch_prefill(KvAttnArgs& a, int sms, cudaStream_t s) {
    const int st = hs_host::set_smem_attr((const void*)kv4_prefill_kernel<D>, kPfMaxSmem);
    if (st != HS_OK) return st;
    a.rows = kPfRows;
    a.tq = kPfRows / a.group;
    a.tile_log2 = 7;
    a.min_units = 1;
    a.pad = 4;
    static_assert(2 * 152 * kPfRows <= kKvWsRows, "workspace");
    static_assert(PrefillCfg<D>::smem(kKvMaxSeqs) <= kPfMaxSmem, "shared memory");
    if (!kv_line_ok(a)) return HS_ERR_UNSUPPORTED_SHAPE;
    if (hs_host::launch_pdl(kv4_prefill_kernel<D>, dim3(std::min(152, sms)), dim3(kPfThreads), PrefillCfg<D>::smem(a.n_seqs), s, a) !=
        cudaSuccess)
        return HS_ERR_CUDA;
    return hs_host::launch_err();
}

}  // namespace hs

int hs_kv4_prefill(hs::KvAttnArgs a, int dim, int sms, cudaStream_t s) {
    return dim == 64 ? hs::launch_prefill<64>(a, sms, s) : hs::launch_prefill<128>(a, sms, s);
}

unsigned hs_kv4_prefill_take_status() {
    unsigned v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, hs::g_status, sizeof(v)) != cudaSuccess) return 0;
    cudaMemcpyToSymbol(hs::g_status, &zero, sizeof(zero));
    return v;
}
