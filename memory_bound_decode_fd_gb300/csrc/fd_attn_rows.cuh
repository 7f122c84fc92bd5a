// fd_attn_rows.cuh - attention of few query rows per key head over a paged cache: decoding, and
// short chunks. Compiled by fd_attn_rows.cu for a bf16 cache, by fd_attn_rows_kv8.cu for one in 8 bits.
//
// For a (sequence, key head) the rows are its new tokens times the query heads that share the
// key head; up to 16 of them are one pass over the keys. Bound by memory: with 16 rows there are
// 16 multiply-adds per byte of the cache, far below what the tensor cores do, so what matters is
// that every SM streams pages all the time.
//
//   * The keys of all (sequence, block of 16 rows, key head) items, in tiles of 32 keys a warp,
//     form one long list, and CTA c of G takes tiles [T c / G, T (c + 1) / G) of it: every SM gets
//     the same number of tiles whatever the lengths of the sequences, with nothing planned on the
//     host (the lengths are device memory, a captured graph sees new ones). An item that several
//     CTAs share is joined by the CTA that finishes last: each writes its rows' (maximum, sum,
//     accumulator) to its own slot, takes a ticket, and the holder of the last ticket adds the
//     slots in the order of the CTAs, so results do not depend on who is last. Where whole items
//     are dealt out evenly enough, no item is shared (kJoinTiles): 128 sequences of up to 1000 at
//     head_dim 64 take 36 us in whole items, 47 in shared ones, 64 of up to 8192 at 128 take 239
//     and 186.
//   * Each of the warps that compute has a warp that copies for it: its 32 keys and values of a
//     tile, by tensor-map copies (64 elements of the tokens of a page, 128-byte swizzle) into a
//     ring of their own in shared memory, across the ends of items; page numbers are read kAhead
//     tiles early. Four copying warps, because one thread issues such a copy in about 60 ns: one
//     warp for all kept 16-token pages (2 KB a copy) at 4.9 TB/s where 64-token pages ran at
//     6.7. Plain 16-byte asynchronous copies stayed at 5.9 TB/s for every page size.
//   * Each warp keeps its own running maximum, sum and fp32 accumulator in registers (online
//     softmax, one pass over the data) and the warps meet only at the end of an item.
//   * Scores are Q K^T with the rows as the M = 16 of mma.sync m16n8k16, so that the
//     probabilities come out in the layout that P V takes as its A operand; rounded to bf16 there
//     (V is bf16, both operands have one type), each by 2^-8 relative at most, while the sum is
//     that of the unrounded ones. These legacy instructions are used on purpose: they hide under
//     the copies, and tcgen05 would pad the rows to 128.
//
// Over a cache in 8 bits (KV8) half of the bytes are to be read, and making operands of the codes costs as much
// as the copies hide: 64 sequences of up to 8192, 4 heads a key head, take 103 us, 89 % of the copy bandwidth, 2 of
// 131072 88 to 92 us (88 to 91 %), one of 4097 10.4 to 10.8. A warp's tile of 32 keys at head_dim 128 is 1750 cycles of work, 500 of
// waiting.
//   * s(i, j) = 2^ek <q_i, code_j>, and sum_j p_j v_j = sum_j (p_j 2^ev) code_j: the codes go into the MMAs as f16,
//     exactly and without a scale, the keys' scales are put on the scores and the values' on the probabilities.
//   * The products are computed transposed: 16 keys (or elements) are the M of m16n8k16 and the rows its N = 8 or 16.
//     Of codes it is the operands that cost, so the side that is made of them is the one read once for all rows, and
//     single tokens of up to 8 heads a key head pad to 8 rows, not 16 (64 of up to 8192, before items were counted with what they cost: 111 us, 129 with the rows as M).
//   * What beginning an item costs is counted in the list (kItemTiles): CTAs with many short items get fewer tiles.
//   * Queries in f16, a row scaled by a power of two to its largest element. Probabilities in f16 against a maximum of
//     their own, that of scores with the values' scales: whatever those are, what is rounded is at most 2^15.
//   * Each warp that computes has 200 registers and its copying warp 56. The lanes of a copying warp hold a block of
//     16 keys or values each, its page and scale, several tiles ahead. 4 bytes that the scale's byte lies in are
//     copied (never across a 4-byte boundary, so never past an allocation).
#pragma once

#include <atomic>
#include <type_traits>

#include "fd_attn.h"
#include "fd_kv8.cuh"
#include "fd_tc.cuh"

namespace fd {
namespace {

// What joining the parts of an item costs, in tiles: a partial result written, a ticket, the
// other parts read.
constexpr int kJoinTiles = 6;
// Over codes, what beginning an item costs, in tiles: its queries as operands, the warps' meeting at its end. Counted
// where there are at least as many items as CTAs: 64 sequences of up to 8192 take 103 us (113 uncounted), 16 of up to
// 6000 and 2 to 8 new tokens 51 (76); but 2 of 131072, parts of which every CTA has, 88 uncounted and 93 counted.
constexpr int kItemTiles = 3;

// KV8: the keys and values are codes of one byte, a row is one column of D bytes.
template <int D, bool KV8, int ROWS>
struct RowsShape {
    static constexpr int kRows = ROWS;                      // of one pass over the keys
    static constexpr int kWarps = KV8 ? 8 : rows_warps(D);
    static constexpr int kKeys = KV8 && D == 64 ? 64 : 32;  // of a tile, a warp's
    static constexpr int kBlocks = kKeys / 16;
    static constexpr int kConsumers = kWarps * 32;
    static constexpr int kThreads = 2 * kConsumers;      // each computing warp, its copying warp
    static constexpr int kTile = kWarps * kKeys;         // keys of a tile
    static constexpr int kHalves = KV8 ? 1 : D / 64;     // columns of a row
    static constexpr int kRow = KV8 ? D : 128;           // bytes of a row of a column
    static constexpr int kColumn = kKeys * kRow;         // bytes of one of a warp's keys
    static constexpr int kPart = kHalves * kColumn;      // a warp's keys (or values) of a tile
    static constexpr int kStages = 2;                    // 128 KB of shared memory in all
    // Registers: 512 threads launch with 128 each; of codes, whose rows need more, the copying warps leave the others
    // some of theirs (0: none do).
    static constexpr int kWorkRegs = KV8 ? 200 : 0, kCopyRegs = 56, kLaunchRegs = 128;
    static_assert(kConsumers * kWorkRegs + (kThreads - kConsumers) * kCopyRegs <= kThreads * kLaunchRegs || !KV8, "registers");
    // arrivals that fill a stage: its rows' copies as one; of codes also a scale for each block of keys and of values
    static constexpr int kArrivals = KV8 ? 1 + 2 * kBlocks : 1;
    static constexpr int kRing = kStages * 2 * kPart;    // of one warp
    static constexpr int kPitch = D + 8;                 // floats; conflict-free accumulator rows
    static constexpr int kMergeBytes = kWarps * kRows * kPitch * 4;
    static constexpr int kMlBytes = kWarps * kRows * 8;
    static_assert(kRows <= kRowsM && kMergeBytes >= kAttnMaxCtas * kRows * 8, "the parts' maxima and sums fit the buffer");
};

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// An 8 x 8 matrix of 16-bit words, two of a row in each lane, transposed.
__device__ __forceinline__ uint32_t turn_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// 4 bytes to shared memory, asynchronously.
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A tile that a copying warp is to copy: its warp's first key, key head (-1: none is left), and
// the pages of the first and second 16 keys (bit i of `read`: the page is needed).
struct TileCopy {
    int tok, hk, read, page[2];
};
constexpr int kAhead = 3;

// The scales of a warp's keys and values: of the keys' blocks, then of the values'; the 4 bytes that each
// lies in, and which of them it is.
template <int BLOCKS>
struct __align__(16) TileScales {  // (the words are read as vectors)
    uint32_t word[2 * BLOCKS];
    uint8_t at[2 * BLOCKS];
};
// The arrival at `bar` of what this thread has copied so far (one of those that the barrier counts).
__device__ __forceinline__ void copy_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One run of tiles of one item.
struct Segment {
    SeqInfo s;
    int b, item;        // item: block of rows * kv_heads + key head
    int rb, hk;
    int i0, i1;         // first and last new token of the block's rows
    int rows;           // rows of the block
    int sink_tiles, shift;  // tile t of the item is tile t, or t + shift from sink_tiles on
    int from, to;       // the segment's tiles, counted in the item
    int nt;             // tiles of the item; 0: nothing to do
    int steps;          // what it counts for in the list: its tiles, and what beginning it costs
    bool whole;         // the segment is the item
    long long item0;    // the item's first step in the list
    long long next;     // what comes after the segment
};

// Tiles that the keys of sequence s take (at least one, so that every row is written). The same for
// all of the sequence's items.
template <int TILE, bool SINKS>
__device__ __forceinline__ KeyTiles seq_tiles(const SeqInfo &s, const AttnArgs &a) {
    if (s.rows <= 0) return {0, 0, 0};
    KeyTiles t = key_tiles<TILE>(key_lo(s, 0, a.window), key_hi(s, s.rows - 1, a.causal), SINKS ? a.sinks : 0);
    t.count = max(t.count, 1);
    return t;
}

// How the list of tiles is dealt out.
struct Deal {
    // Steps of one key head of each sequence before b: of the blocks of rows that the sequence has (`ragged`), or of
    // one block, and every sequence counts as having as many as the longest.
    const unsigned *prefix;
    bool ragged;
    int per;                  // what a sequence's steps are to be multiplied by: its key heads, or its items
    int items;                // of a sequence, at most
    int cost;                 // steps that an item counts for beside its tiles (0 or kItemTiles)
    long long total;          // steps
    int G;                    // CTAs that work
    bool whole;               // items c, c + G, ... instead of steps [begin, end)
    long long begin, end;     // steps, or items
};

// The segment at x (a step of the list, or an item); `b` is a sequence at or before x's.
template <int TILE, bool SINKS, int ROWS, bool KV8>
__device__ __forceinline__ Segment segment_at(const AttnArgs &a, const Deal &d, long long x, int b) {
    Segment g;
    const unsigned *prefix = d.prefix;
    const int per = d.per;
    if (d.whole)
        b = (int)((unsigned)x / (unsigned)d.items);
    else {
        // the first b with prefix[b + 1] * per > x: this sequence, the next, or by bisection
        if ((long long)prefix[b + 1] * per <= x && (long long)prefix[++b + 1] * per <= x) {
            int up = a.m.batch - 1;
            for (++b; b < up;) {
                const int mid = (b + up) >> 1;
                if ((long long)prefix[mid + 1] * per > x)
                    up = mid;
                else
                    b = mid + 1;
            }
        }
    }
    g.s = load_seq(a.m, b);
    const KeyTiles t = seq_tiles<TILE, SINKS>(g.s, a);
    g.nt = KV8 ? t.count : (int)(prefix[b + 1] - prefix[b]);
    g.steps = g.nt + (KV8 ? d.cost : 0);
    if (d.whole) {
        g.item = (int)x - b * d.items;
        if (KV8 && d.ragged && g.item / a.kv_heads * ROWS >= g.s.rows * a.group) g.nt = 0;
        g.from = 0, g.to = g.nt;
        g.whole = true;
        g.item0 = 0;
        g.next = x + d.G;
    } else {
        const long long in_seq = x - (long long)prefix[b] * per;
        // 32 bits where they do: a 64-bit division is a hundred instructions
        g.item = in_seq >> 32 ? (int)(in_seq / g.steps) : (int)((unsigned)in_seq / (unsigned)g.steps);
        g.from = (int)(in_seq - (long long)g.item * g.steps);
        g.item0 = x - g.from;
        g.to = (int)min((long long)g.steps, d.end - g.item0);
        g.next = g.item0 + g.to;
        g.whole = g.from == 0 && g.to == g.steps;
        // the tiles of its steps (none, perhaps: then a part of nothing)
        if (KV8) {
            auto tiles = [&](int v) { return v - (d.cost * v + g.steps - 1) / g.steps; };
            g.from = tiles(g.from), g.to = tiles(g.to);
        }
    }
    g.b = b;
    g.rb = g.item / a.kv_heads;
    g.hk = g.item - g.rb * a.kv_heads;
    g.sink_tiles = t.sinks, g.shift = t.shift;
    const int all = g.s.rows * a.group;
    g.rows = min(ROWS, all - g.rb * ROWS);  // <= 0: no such block in this sequence
    g.i0 = g.rb * ROWS / a.group;
    g.i1 = min(g.s.rows, (g.rb * ROWS + ROWS - 1) / a.group + 1) - 1;
    return g;
}

// CAPPED: the scores go through the tanh (apart, so that its code costs the others nothing: in one
// kernel, 128 sequences of 500 at head_dim 64 took 29.9 us without a cap, 28.9 apart). SINKS: a window
// leaves the first tokens visible (in one kernel, one token of 4097 keys took 11.6 us without, 11.2 apart).
// TYPE: 0, or the codes of a cache in 8 bits.
template <int D, bool CAPPED, bool SINKS, int TYPE, int ROWS>
__global__ void __launch_bounds__(RowsShape<D, TYPE != 0, ROWS>::kThreads, 1)
    attn_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const AttnArgs a, int row_blocks) {
    constexpr bool KV8 = TYPE != 0;
    using S = RowsShape<D, KV8, ROWS>;
    const int sinks = SINKS ? a.sinks : 0;
    constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kTile = S::kTile, kKeys = S::kKeys;
    using Scales = TileScales<S::kBlocks>;
    static_assert(sizeof(Scales) % 16 == 0, "every entry of an array on 16 bytes");
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    __shared__ int last_s, abort_flag;
    __shared__ __align__(8) uint64_t full[kWarps][S::kStages], empty[kWarps][S::kStages];
    __shared__ TileCopy next_tiles[KV8 ? 1 : kWarps][kAhead];
    __shared__ Scales scales[KV8 ? kWarps : 1][S::kStages];
    __shared__ unsigned warp_sum[kThreads / 32], warp_max[kThreads / 32];
    float *merge = reinterpret_cast<float *>(smem + kWarps * S::kRing);
    float2 *ml = reinterpret_cast<float2 *>(smem + kWarps * S::kRing + S::kMergeBytes);
    unsigned *prefix = reinterpret_cast<unsigned *>(smem + kWarps * S::kRing + S::kMergeBytes + S::kMlBytes);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = tid / 32 % kWarps;  // of its kind
    if (tid == 0) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < S::kStages; ++i) {
                mbar_init(&full[w][i], S::kArrivals);
                mbar_init(&empty[w][i], 1);
            }
        abort_flag = 0;
        fence_mbar_init();
    }
    grid_dep_wait();
    grid_dep_launch();

    // ------------------------------------------------------------------- the list
    Deal deal;
    {
        const int per = (a.m.batch + kThreads - 1) / kThreads;
        const int b0 = min(tid * per, a.m.batch), b1 = min(b0 + per, a.m.batch);
        // 16 sequences of 2 to 8 new tokens, 4 heads a key head, up to 6000 keys: 52 us, and 60 where each counts as two
        // blocks of 16 rows; where all have two, 64 of 1000 keys, 77 and 76. For up to 8 blocks, so that the tiles' count
        // stays far from 2^32.
        deal.ragged = KV8 && row_blocks > 1 && row_blocks <= 8;
        deal.items = row_blocks * a.kv_heads;
        const int G = gridDim.x;
        const long long n = (long long)a.m.batch * deal.items;
        deal.cost = KV8 && n >= G ? kItemTiles : 0;
        auto blocks_of = [&](const SeqInfo &s) { return deal.ragged ? (s.rows * a.group + S::kRows - 1) / S::kRows : 1; };
        unsigned sum = 0, most = 0;
        for (int b = b0; b < b1; ++b) {
            const SeqInfo s = load_seq(a.m, b);
            unsigned n = (unsigned)seq_tiles<kTile, SINKS>(s, a).count;
            if (KV8 && n > 0) n += deal.cost;
            prefix[b] = sum;  // of this thread's sequences
            sum += KV8 ? n * (unsigned)blocks_of(s) : n;
            most = max(most, n);
        }
        unsigned inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += up;
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        if (lane == 31) warp_sum[tid >> 5] = inc, warp_max[tid >> 5] = most;
        __syncthreads();
        unsigned before = inc - sum, all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < (tid >> 5)) before += warp_sum[w];
            all += warp_sum[w];
            most = max(most, warp_max[w]);
        }
        for (int b = b0; b < b1; ++b) prefix[b] += before;
        if (tid == 0) prefix[a.m.batch] = all;
        __syncthreads();
        deal.prefix = prefix;
        deal.per = deal.ragged ? a.kv_heads : deal.items;
        deal.total = (long long)all * deal.per;
        const int c = blockIdx.x;
        // Whole items one after the other, or equal runs of tiles joined where they meet: what a CTA
        // gets of the first at most, counted, or estimated where that would take long.
        long long share = most;
        if (n > 16 * G) {
            share = deal.total / G + 3 * ((long long)most - min((int)most, deal.cost));
        } else if (n > G) {
            unsigned *const of = reinterpret_cast<unsigned *>(merge);  // not in use yet
            for (int i = tid; i < kAttnMaxCtas; i += kThreads) of[i] = 0;
            __syncthreads();
            for (int i = tid; i < (int)n; i += kThreads) {
                const int b = i / deal.items;
                unsigned n = prefix[b + 1] - prefix[b];
                if (deal.ragged) {
                    const int blocks = blocks_of(load_seq(a.m, b));
                    n = (i - b * deal.items) / a.kv_heads < blocks ? n / (unsigned)max(blocks, 1) : 0u;
                }
                atomicAdd(&of[i % G], n);
            }
            __syncthreads();
            unsigned m = 0;
            for (int i = lane; i < kAttnMaxCtas; i += 32) m = max(m, of[i]);
            share = __reduce_max_sync(0xFFFFFFFFu, m);
            __syncthreads();
        }
        deal.whole = n < (1ll << 31) && share * G <= deal.total + (long long)kJoinTiles * G;
        if (deal.whole) {
            deal.G = gridDim.x;
            deal.begin = c, deal.end = n;
        } else {
            // no more CTAs than tiles: each CTA between an item's first and last has a part of it
            deal.G = (int)min((long long)gridDim.x, deal.total);
            if (c >= deal.G) return;
            deal.begin = deal.total * c / deal.G, deal.end = deal.total * (c + 1) / deal.G;
        }
    }

    const uint32_t ring = smem_u32(smem) + warp * S::kRing;
    // The item's tiles in the order of the list: where the k-th begins.
    auto first_key = [](const Segment &g, int k) { return (k + (SINKS && k < g.sink_tiles ? 0 : g.shift)) * kTile; };
    const long long wait_limit = a.test_timeout ? kTestWaitLimitCycles : kWaitLimitCycles;
    auto wait_for = [&](uint64_t *bar, uint32_t parity) {
        if constexpr (S::kWorkRegs > 0)
            return mbar_wait_inline(bar, parity, &abort_flag, wait_limit);
        else
            return mbar_wait_bounded(bar, parity, &abort_flag, wait_limit);
    };
    if (tid >= S::kConsumers) {
        // ---------------------------------------------------------------------- copies
        if constexpr (S::kWorkRegs > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kCopyRegs));
        if constexpr (KV8) {
            // A lane has one block of 16 of the tile's keys, or its values: it copies them and their scale. The lanes
            // of a tile are a group; the groups take turns, so that each has looked up its pages (and they have arrived)
            // kGroups tiles before it copies.
            constexpr int kLanes = 2 * S::kBlocks, kGroups = 32 / kLanes;
            const int w = warp, grp = lane / kLanes, blk = lane % S::kBlocks, v = lane / S::kBlocks & 1;
            const Kv8Plane &plane = v ? a.kv8.v : a.kv8.k;
            const MapOrder ord = v ? a.ov : a.ok;
            const CUtensorMap *const map = v ? &map_v : &map_k;
            const int page_mask = (1 << a.m.page_shift) - 1, box = min(page_mask + 1, kRowsBox);
            const uint64_t policy = policy_evict_first();
            unsigned char *const to = smem + w * S::kRing + v * S::kPart + blk * 16 * S::kRow;
            constexpr int kNone = -1 << 30;
            Segment g;
            g.to = 0;
            int tile = 0, lo = 0, hi = 0, b_at = 0;
            long long x = deal.begin;
            bool more = true;
            int off = 0, hk = -1, page = kNone;  // of the lane's block: its place in its page, key head (-1: none is left)
            auto describe = [&](int n) {  // the next tile, for group n
                while (more && ++tile >= g.to) {
                    if (x >= deal.end) {
                        more = false;
                        break;
                    }
                    g = segment_at<kTile, SINKS, S::kRows, KV8>(a, deal, x, b_at);
                    b_at = g.b;
                    x = g.next;
                    tile = g.from - 1;
                    lo = key_lo(g.s, 0, a.window), hi = key_hi(g.s, g.s.rows - 1, a.causal);
                }
                if (grp == n) {
                    const int tok = first_key(g, tile) + w * kKeys + 16 * blk, first = tok & ~(box - 1);
                    off = tok & page_mask, hk = more ? g.hk : -1, page = kNone;
                    if (more && first < hi && (first + box > lo || first < sinks))
                        page = a.m.table[(long long)g.b * a.m.table_stride + (tok >> a.m.page_shift)];
                }
            };
#pragma unroll 1
            for (int i = 0; i < kGroups; ++i) describe(i);
            uint32_t issued = 0, phase = 1;
            int slot = 0, turn = 0;
            bool ok = true;
            while (__shfl_sync(0xFFFFFFFFu, hk, turn * kLanes) >= 0) {
                ok = __all_sync(0xFFFFFFFFu, wait_for(&empty[w][slot], phase));
                if (!ok) break;
                const bool mine = grp == turn && !(a.test_timeout && w == 0 && issued == 0);
                if (mine) {
                    uint64_t *const bar = &full[w][slot];
                    const bool none = (unsigned)page >= (unsigned)a.m.num_pages;
                    const int pg = none ? a.m.num_pages : page;  // a copy from behind the last page fills zeros
                    if (none && page != kNone) atomicOr(&g_wait_status, (unsigned)FD_DEVICE_STATUS_BAD_PAGE);
                    Scales &s = scales[w][slot];
                    const int i = v * S::kBlocks + blk;
                    if (!none) {
                        const uintptr_t at = reinterpret_cast<uintptr_t>(plane.scale + pg * plane.scale_page +
                                                                         off / kKv8Block * plane.scale_block + hk * plane.scale_head);
                        s.at[i] = (uint8_t)(at & 3);
                        copy4(smem_u32(&s.word[i]), reinterpret_cast<const void *>(at & ~(uintptr_t)3));
                        copy_arrive(bar);
                    } else {  // of a block that is not read, 1
                        s.at[i] = 0;
                        s.word[i] = 127;
                    }
                }
                __syncwarp();
                if (mine) {
                    uint64_t *const bar = &full[w][slot];
                    const bool none = (unsigned)page >= (unsigned)a.m.num_pages;
                    const int pg = none ? a.m.num_pages : page;
                    if (blk == 0 && v == 0) mbar_arrive_expect_tx(bar, 2 * S::kPart);  // (behind the lanes' stores)
                    if (box == 16 || !(blk & 1)) {
                        const int y1 = ord.tok == 1 ? off : ord.head == 1 ? hk : pg;
                        const int y2 = ord.tok == 2 ? off : ord.head == 2 ? hk : pg;
                        const int y3 = ord.tok == 3 ? off : ord.head == 3 ? hk : pg;
                        tma_load_4d(to + slot * 2 * S::kPart, map, 0, y1, y2, y3, bar, policy);
                    }
                    if (none) mbar_arrive(bar);
                }
                ++issued;
                describe(turn);
                if (++slot == S::kStages) slot = 0, phase ^= 1u;
                if (++turn == kGroups) turn = 0;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (!ok && lane == 0) {  // wait (bounded) for the copies in flight before the CTA ends
                const uint32_t n = issued < (uint32_t)S::kStages ? issued : (uint32_t)S::kStages;
                for (uint32_t i = issued - n; i < issued; ++i) {
                    const long long t0 = clock64();
                    while (!mbar_try_parity(&full[w][i % S::kStages], (i / S::kStages) & 1u) &&
                           clock64() - t0 < wait_limit) {
                    }
                }
            }
            return;
        }
        const uint64_t policy = policy_evict_first();
        const int page_mask = (1 << a.m.page_shift) - 1;
        // What is to be copied, kAhead tiles before its turn: by then its page number has arrived,
        // copied to the description asynchronously (a load would hold this warp up in order).
        volatile TileCopy *ahead = next_tiles[warp];
        Segment g;
        g.to = 0;
        int tile = 0, lo = 0, hi = 0, b_at = 0;
        long long x = deal.begin;
        bool more = true;
        auto describe = [&](int entry) {
            while (more && ++tile >= g.to) {
                if (x >= deal.end) {
                    more = false;
                    break;
                }
                g = segment_at<kTile, SINKS, S::kRows, KV8>(a, deal, x, b_at);
                b_at = g.b;
                x = g.next;
                tile = g.from - 1;
                lo = key_lo(g.s, 0, a.window), hi = key_hi(g.s, g.s.rows - 1, a.causal);
            }
            if (lane == 0) {
                volatile TileCopy &t = ahead[entry];
                const int tok = first_key(g, tile) + warp * kKeys;
                const int *row = a.m.table + (long long)g.b * a.m.table_stride;
                int read = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int first = tok + 16 * i;
                    if (more && first < hi && (first + 16 > lo || first < sinks)) {
                        copy4(smem_u32(const_cast<int *>(&t.page[i])), row + (first >> a.m.page_shift));
                        read |= 1 << i;
                    }
                }
                t.tok = tok, t.hk = more ? g.hk : -1, t.read = read;
            }
        };
#pragma unroll 1
        for (int i = 0; i < kAhead; ++i) {
            describe(i);
            copy_commit();
        }
        int entry = 0, slot = 0;
        uint32_t phase = 1, issued = 0;
        bool ok = true;
        while (true) {
            copy_wait<kAhead - 1>();  // the description's pages
            __syncwarp();
            const int hk = ahead[entry].hk, tok = ahead[entry].tok, read = ahead[entry].read;
            int page[2] = {ahead[entry].page[0], ahead[entry].page[1]};
            if (hk < 0) break;
            __syncwarp();
            describe(entry);
            ok = __all_sync(0xFFFFFFFFu, wait_for(&empty[warp][slot], phase));
            if (!ok) break;
            if (lane == 0 && !(a.test_timeout && warp == 0 && issued == 0)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if ((read >> i & 1) && (unsigned)page[i] >= (unsigned)a.m.num_pages)
                        atomicOr(&g_wait_status, (unsigned)FD_DEVICE_STATUS_BAD_PAGE);
                    // a copy from behind the last page fills zeros
                    if (!(read >> i & 1) || (unsigned)page[i] >= (unsigned)a.m.num_pages) page[i] = a.m.num_pages;
                }
                uint64_t *const bar = &full[warp][slot];
                mbar_arrive_expect_tx(bar, 2 * S::kPart);
                unsigned char *const dst = smem + warp * S::kRing + slot * 2 * S::kPart;
                auto copy = [&](int first, int pg) {  // the box of tokens that begins with key `first`
                    const int at = (tok + first) & page_mask;
                    const int k1 = a.ok.tok == 1 ? at : a.ok.head == 1 ? hk : pg;
                    const int k2 = a.ok.tok == 2 ? at : a.ok.head == 2 ? hk : pg;
                    const int k3 = a.ok.tok == 3 ? at : a.ok.head == 3 ? hk : pg;
                    const int v1 = a.ov.tok == 1 ? at : a.ov.head == 1 ? hk : pg;
                    const int v2 = a.ov.tok == 2 ? at : a.ov.head == 2 ? hk : pg;
                    const int v3 = a.ov.tok == 3 ? at : a.ov.head == 3 ? hk : pg;
#pragma unroll
                    for (int h = 0; h < S::kHalves; ++h) {
                        unsigned char *const to = dst + h * S::kColumn + first * S::kRow;
                        tma_load_4d(to, &map_k, 64 * h, k1, k2, k3, bar, policy);
                        tma_load_4d(to + S::kPart, &map_v, 64 * h, v1, v2, v3, bar, policy);
                    }
                };
                // boxes of 16 tokens, or of 32 (one page, whichever half of it is needed)
                copy(0, a.m.page_shift == 4 || (read & 1) ? page[0] : page[1]);
                if (a.m.page_shift == 4) copy(16, page[1]);
            }
            __syncwarp();
            ++issued;
            copy_commit();
            if (++slot == S::kStages) slot = 0, phase ^= 1u;
            if (++entry == kAhead) entry = 0;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!ok && lane == 0) {  // wait (bounded) for the copies in flight before the CTA ends
            const uint32_t n = issued < (uint32_t)S::kStages ? issued : (uint32_t)S::kStages;
            for (uint32_t i = issued - n; i < issued; ++i) {
                const long long t0 = clock64();
                while (!mbar_try_parity(&full[warp][i % S::kStages], (i / S::kStages) & 1u) &&
                       clock64() - t0 < wait_limit) {
                }
            }
        }
        return;
    }

    // ------------------------------------------------------------------------- the work
    if constexpr (S::kWorkRegs > 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kWorkRegs));
    const int g8 = lane >> 2, c2 = (lane & 3) * 2;  // accumulator row and column of this lane
    const float to_log2 = a.scale * kLog2e;
    const float cap_in = CAPPED ? a.scale / a.softcap : 0.f, cap_out = a.softcap * kLog2e;
    // ldmatrix rows: keys (lane & 7) + 8 * (lane >> 4), chunk bit (lane >> 3) & 1
    const int k_row = (lane & 7) + ((lane >> 4) << 3), k_bit = (lane >> 3) & 1;
    // values, transposed: keys (lane & 15), chunk bit lane >> 4
    const int v_row = lane & 15, v_bit = lane >> 4;
    int stage = 0, b_at = 0;
    uint32_t phase = 0;
    bool dead = false;
    for (long long x = deal.begin; x < deal.end;) {
        const Segment g = segment_at<kTile, SINKS, S::kRows, KV8>(a, deal, x, b_at);
        b_at = g.b;
        x = g.next;
        if (g.nt == 0) continue;
        // Of codes, scores and results are computed transposed, 16 keys (or elements) by 8 rows: a key head's rows, 4 or
        // 8 of them mostly, are the narrow side of the MMAs (16 x 8 x 16), and what it takes to make operands of codes is
        // done once for all of them. A lane has the rows 8 r + c2 and 8 r + c2 + 1.
        if constexpr (KV8) {
            constexpr int RB = S::kRows / 8, kC = D / 16, kB = S::kBlocks;
            uint32_t qf[RB][kC][2];
            float q_mul[RB][2];  // what a score of the queries in f16 is to be multiplied by
            int hi[RB][2], lo[RB][2];
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                // Row 8 r + g8, elements 2 c2 .. + 3 of each 16, as a lane gets them of the keys. In f16, the row's largest
                // between 2^14 and 2^15: exact for all that are no smaller than 2^-31 of it, the others off by half of fp16's smallest
                // step, 2^-25, or 2^-39 of it. (Below 2^-100 nothing is lost: bf16's own smallest step is 2^-19 there.)
                const int all = g.rb * S::kRows + 8 * r + g8, i = all / a.group;
                const bool live = 8 * r + g8 < g.rows;
                const uint16_t *q = a.q.p + (g.s.q0 + i) * a.q.ts + (g.hk * a.group + all - i * a.group) * a.q.hs + 2 * c2;
                uint32_t top = 0;
#pragma unroll
                for (int ks = 0; ks < kC; ++ks) {
                    const uint2 x = live ? *reinterpret_cast<const uint2 *>(q + ks * 16) : make_uint2(0u, 0u);
                    qf[r][ks][0] = x.x, qf[r][ks][1] = x.y;
                    top = max(top, max(max(x.x << 16 & 0x7FFFFFFFu, x.x & 0x7FFF0000u), max(x.y << 16 & 0x7FFFFFFFu, x.y & 0x7FFF0000u)));
                }
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                const int k = max((int)(top >> 23) - 127, -100) - 14;
                const float f = two_to(-k), mul = (CAPPED ? 1.f : to_log2) * two_to(k);
#pragma unroll
                for (int ks = 0; ks < kC; ++ks)
#pragma unroll
                    for (int n = 0; n < 2; ++n) qf[r][ks][n] = pack_f16x2(bf16lo(qf[r][ks][n]) * f, bf16hi(qf[r][ks][n]) * f);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    q_mul[r][e] = __shfl_sync(0xFFFFFFFFu, mul, (c2 + e) * 4);
                    const int row = 8 * r + c2 + e, tok = (g.rb * S::kRows + row) / a.group;
                    hi[r][e] = row < g.rows ? key_hi(g.s, tok, a.causal) : 0;
                    lo[r][e] = row < g.rows ? key_lo(g.s, tok, a.window) : 0;
                }
            }
            const int in_lo = key_lo(g.s, g.i1, a.window), in_hi = key_hi(g.s, g.i0, a.causal);
            const int any_lo = key_lo(g.s, g.i0, a.window), any_hi = key_hi(g.s, g.i1, a.causal);
            float o[RB][kC][4];
            float m[RB][2], l[RB][2];
            // The sum of p v is kept in units of its own, 2^(w - kUp): w is the running maximum of the scores with the
            // scales of their values, so that what is rounded to f16 is at most 2^kUp, whatever the scales.
            float w[RB][2];
            constexpr float kUp = 15.f;
#pragma unroll
            for (int r = 0; r < RB; ++r) {
#pragma unroll
                for (int n = 0; n < kC; ++n) o[r][n][0] = o[r][n][1] = o[r][n][2] = o[r][n][3] = 0.f;
                m[r][0] = m[r][1] = w[r][0] = w[r][1] = -INFINITY, l[r][0] = l[r][1] = 0.f;
            }
#pragma unroll 1
            for (int t = g.from; t < g.to; ++t) {
                if (!dead) dead = !__all_sync(0xFFFFFFFFu, wait_for(&full[warp][stage], phase));
                if (dead) break;
                const uint32_t kb = ring + stage * 2 * S::kPart, vb = kb + S::kPart;
                uint64_t *const done = &empty[warp][stage];
                const Scales &ts = scales[warp][stage];
                if (++stage == S::kStages) stage = 0, phase ^= 1u;
                const int tok = first_key(g, t) + warp * kKeys;  // the warp's first key
                if (g.rows <= 0 || tok >= any_hi || (tok + kKeys <= any_lo && tok >= sinks)) {
                    if (lane == 0) mbar_arrive(done);
                    continue;
                }
                float s[RB][kB][4];
#pragma unroll
                for (int r = 0; r < RB; ++r)
#pragma unroll
                    for (int b = 0; b < kB; ++b) s[r][b][0] = s[r][b][1] = s[r][b][2] = s[r][b][3] = 0.f;
                const int swizzle = D == 128 ? lane & 7 : lane >> 1 & 3;
#pragma unroll
                for (int ks = 0; ks < kC; ++ks)
#pragma unroll
                    for (int b = 0; b < kB; b += 2) {
                        uint32_t kf[4];  // 8 keys each
                        ldsm_x4(kf, kb + (16 * b + lane) * D + ((ks ^ swizzle) << 4));
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            uint32_t op[4];
                            kv8_halves<TYPE>(kf[2 * n], false, op[0], op[2]);
                            kv8_halves<TYPE>(kf[2 * n + 1], false, op[1], op[3]);
#pragma unroll
                            for (int r = 0; r < RB; ++r) mma_f16(s[r][b + n], op, qf[r][ks][0], qf[r][ks][1]);
                        }
                    }
                // the scales of the blocks, and of the queries
                float ek[kB], ev[kB];  // of keys, of values (the exponents)
#pragma unroll
                for (int i = 0; i < 2 * kB; i += 4) {
                    const uint4 x = lds_v4(smem_u32(ts.word + i));
                    const uint32_t at = *reinterpret_cast<const volatile uint32_t *>(ts.at + i);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t byte = __byte_perm(k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w, 0, 0x4440u | (at >> 8 * k & 3));
                        if (i + k < kB)
                            ek[(i + k) % kB] = __uint_as_float(byte << 23);
                        else
                            ev[(i + k) % kB] = (float)((int)byte - 127);
                    }
                }
#pragma unroll
                for (int r = 0; r < RB; ++r)
#pragma unroll
                    for (int b = 0; b < kB; ++b) {
                        const float f0 = q_mul[r][0] * ek[b], f1 = q_mul[r][1] * ek[b];
                        s[r][b][0] *= f0, s[r][b][1] *= f1, s[r][b][2] *= f0, s[r][b][3] *= f1;
                    }
                const bool inside = (tok >= in_lo || tok + kKeys <= sinks) && tok + kKeys <= in_hi;
                if constexpr (CAPPED) {
                    // all of the warp's scores below half the cap, as most are: the shorter form
                    float size = 0.f;
#pragma unroll
                    for (int r = 0; r < RB; ++r)
#pragma unroll
                        for (int b = 0; b < kB; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i) size = fmaxf(size, fabsf(s[r][b][i]));
                    auto cap = [&](auto near) {
#pragma unroll
                        for (int r = 0; r < RB; ++r)
#pragma unroll
                            for (int b = 0; b < kB; ++b)
#pragma unroll
                                for (int i = 0; i < 4; i += 2) {
                                    const float2 y = capped_log2<decltype(near)::value>(make_float2(s[r][b][i], s[r][b][i + 1]), to_log2,
                                                                                        cap_in, cap_out);
                                    s[r][b][i] = y.x, s[r][b][i + 1] = y.y;
                                }
                    };
                    if (__all_sync(0xFFFFFFFFu, size * fabsf(cap_in) <= 0.5f))
                        cap(std::true_type{});
                    else
                        cap(std::false_type{});
                }
                if (!inside) {
#pragma unroll
                    for (int b = 0; b < kB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = tok + 16 * b + g8 + 8 * (i >> 1);
#pragma unroll
                            for (int r = 0; r < RB; ++r)
                                if ((key < lo[r][i & 1] && key >= sinks) || key >= hi[r][i & 1]) s[r][b][i] = -INFINITY;
                        }
                }
                bool same = true;  // no maximum has grown
                uint32_t p[RB][kB][2];
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    float up[2], off[2], off_w[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = -INFINITY, wx = -INFINITY;
#pragma unroll
                        for (int b = 0; b < kB; ++b) {
                            const float part = fmaxf(s[r][b][e], s[r][b][e + 2]);
                            mx = fmaxf(mx, part), wx = fmaxf(wx, part + ev[b]);
                        }
                        auto raise = [](float x, float &held) {  // x over the row's lanes and what was there; 0 from the first on
#pragma unroll
                            for (int k = 4; k < 32; k *= 2) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, k));
                            x = fmaxf(x, held);
                            const float f = x > held ? ex2(held - x) : 1.f;
                            held = x;
                            return f;
                        };
                        l[r][e] *= raise(mx, m[r][e]);
                        up[e] = raise(wx, w[r][e]);
                        off[e] = m[r][e] == -INFINITY ? 0.f : m[r][e];
                        off_w[e] = w[r][e] == -INFINITY ? 0.f : kUp - w[r][e];
                    }
                    same = up[0] == 1.f && up[1] == 1.f;
                    if (__any_sync(0xFFFFFFFFu, !same)) {
#pragma unroll
                        for (int n = 0; n < kC; ++n)
                            o[r][n][0] *= up[0], o[r][n][1] *= up[1], o[r][n][2] *= up[0], o[r][n][3] *= up[1];
                    }
#pragma unroll
                    for (int b = 0; b < kB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const float y0 = s[r][b][i], y1 = s[r][b][i + 1];
                            l[r][0] += ex2(y0 - off[0]), l[r][1] += ex2(y1 - off[1]);
                            // both rows of a key; turned so that a lane has two keys of a row
                            const uint32_t x = pack_f16x2(ex2(y0 + (ev[b] + off_w[0])), ex2(y1 + (ev[b] + off_w[1])));
                            p[r][b][i >> 1] = turn_8x8(x);
                        }
                }
                // Values that no row sees are cleared before their conversion, a lane's register holding two elements
                // of keys c2 and c2 + 1 (or + 8): 0 x NaN would reach the sum otherwise.
                auto values = [&](auto masked) {
#pragma unroll
                    for (int b = 0; b < kB; ++b) {
                        uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
                        if constexpr (decltype(masked)::value) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int key = tok + 16 * b + 8 * e + c2;
                                auto any_sees = [&](int x) { return (x >= any_lo || x < sinks) && x < any_hi; };
                                keep[e] = (any_sees(key) ? 0xFFFFu : 0u) | (any_sees(key + 1) ? 0xFFFF0000u : 0u);
                            }
                        }
#pragma unroll
                        for (int n = 0; n < kC; n += 2) {
                            uint32_t vf[4];
                            ldsm_x4_t(vf, vb + (16 * b + v_row) * D + (((n + v_bit) ^ (D == 128 ? v_row & 7 : v_row >> 1 & 3)) << 4));
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                uint32_t op[4];  // even elements, odd ones; of 8 keys, of 8 more
                                if constexpr (decltype(masked)::value) vf[2 * j] &= keep[0], vf[2 * j + 1] &= keep[1];
                                kv8_halves<TYPE>(vf[2 * j], true, op[0], op[1]);
                                kv8_halves<TYPE>(vf[2 * j + 1], true, op[2], op[3]);
#pragma unroll
                                for (int r = 0; r < RB; ++r) mma_f16(o[r][n + j], op, p[r][b][0], p[r][b][1]);
                            }
                        }
                    }
                };
                if (inside)
                    values(std::false_type{});
                else
                    values(std::true_type{});
                __syncwarp();
                if (lane == 0) mbar_arrive(done);
            }

            // -------------------------------------------- the warps of this segment meet
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int k = 4; k < 32; k *= 2) l[r][e] += __shfl_xor_sync(0xFFFFFFFFu, l[r][e], k);
                    if (dead) m[r][e] = 0.f, l[r][e] = NAN;
                    const int row = warp * S::kRows + 8 * r + c2 + e;
                    if (g8 == 0) ml[row] = make_float2(m[r][e], l[r][e]);
                    // in units of the maximum, as the sum
                    const float f = m[r][e] == -INFINITY ? 0.f : ex2(w[r][e] - kUp - m[r][e]);
#pragma unroll
                    for (int n = 0; n < kC; ++n)
                        *reinterpret_cast<float2 *>(merge + row * S::kPitch + 16 * n + 2 * g8) =
                            make_float2(o[r][n][e] * f, o[r][n][e + 2] * f);
                }
        } else {
        // the rows of this lane: tokens, heads and visible keys
        uint32_t qf[D / 16][4];
        int hi[2], lo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = g8 + 8 * e, all = g.rb * S::kRows + row;
            const int i = all / a.group;
            const bool live = row < g.rows;
            hi[e] = live ? key_hi(g.s, i, a.causal) : 0;
            lo[e] = live ? key_lo(g.s, i, a.window) : 0;
            const uint16_t *q = a.q.p + (g.s.q0 + i) * a.q.ts + (g.hk * a.group + all - i * a.group) * a.q.hs + c2;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                qf[ks][e] = live ? *reinterpret_cast<const uint32_t *>(q + ks * 16) : 0u;
                qf[ks][e + 2] = live ? *reinterpret_cast<const uint32_t *>(q + ks * 16 + 8) : 0u;
            }
        }
        // the range all live rows see: no masks inside it
        const int in_lo = key_lo(g.s, g.i1, a.window), in_hi = key_hi(g.s, g.i0, a.causal);
        const int any_lo = key_lo(g.s, g.i0, a.window), any_hi = key_hi(g.s, g.i1, a.causal);
        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

#pragma unroll 1
        for (int t = g.from; t < g.to; ++t) {
            if (!dead) dead = !__all_sync(0xFFFFFFFFu, wait_for(&full[warp][stage], phase));
            if (dead) break;
            const uint32_t kb = ring + stage * 2 * S::kPart, vb = kb + S::kPart;
            uint64_t *const done = &empty[warp][stage];
            if (++stage == S::kStages) stage = 0, phase ^= 1u;
            const int tok = first_key(g, t) + warp * kKeys;  // the warp's first key
            // a warp's keys outside every row's range (the ends of a window) add nothing
            if (g.rows <= 0 || tok >= any_hi || (tok + kKeys <= any_lo && tok >= sinks)) {
                if (lane == 0) mbar_arrive(done);
                continue;
            }
            constexpr int kN = kKeys / 8;  // blocks of 8 keys
            float s[kN][4];
#pragma unroll
            for (int n = 0; n < kN; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
                for (int n = 0; n < kN; n += 2) {
                    uint32_t kf[4];
                    ldsm_x4(kf, kb + (ks >> 2) * S::kColumn + (n * 8 + k_row) * 128 +
                                    ((((ks & 3) * 2 + k_bit) ^ (k_row & 7)) << 4));
                    mma_bf16(s[n], qf[ks], kf[0], kf[1]);
                    mma_bf16(s[n + 1], qf[ks], kf[2], kf[3]);
                }
            }
            const bool inside = (tok >= in_lo || tok + kKeys <= sinks) && tok + kKeys <= in_hi;
            if constexpr (CAPPED) {
                // all of the warp's scores below half the cap, as most are: the shorter form
                float size = 0.f;
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) size = fmaxf(size, fabsf(s[n][i]));
                auto cap = [&](auto near) {
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const float2 y = capped_log2<decltype(near)::value>(make_float2(s[n][i], s[n][i + 1]),
                                                                                to_log2, cap_in, cap_out);
                            s[n][i] = y.x, s[n][i + 1] = y.y;
                        }
                };
                if (__all_sync(0xFFFFFFFFu, size * fabsf(cap_in) <= 0.5f))
                    cap(std::true_type{});
                else
                    cap(std::false_type{});
            } else {
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[n][i] *= to_log2;
            }
            if (!inside) {
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = tok + n * 8 + c2 + (i & 1);
                        if ((key < lo[i >> 1] && key >= sinks) || key >= hi[i >> 1]) s[n][i] = -INFINITY;
                    }
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) mx[e] = fmaxf(fmaxf(mx[e], s[n][2 * e]), s[n][2 * e + 1]);
            float up[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 1));
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 2));
                mx[e] = fmaxf(mx[e], m[e]);
                up[e] = mx[e] > m[e] ? ex2(m[e] - mx[e]) : 1.f;  // 0 from the first maximum on
                m[e] = mx[e];
            }
            if (__any_sync(0xFFFFFFFFu, up[0] != 1.f || up[1] != 1.f)) {
                l[0] *= up[0], l[1] *= up[1];
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][0] *= up[0], o[n][1] *= up[0];
                    o[n][2] *= up[1], o[n][3] *= up[1];
                }
            }
            const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
            for (int h = 0; h < kKeys / 16; ++h) {
                uint32_t p[4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = ex2(s[2 * h + n][0] - m0), p1 = ex2(s[2 * h + n][1] - m0);
                    const float p2 = ex2(s[2 * h + n][2] - m1), p3 = ex2(s[2 * h + n][3] - m1);
                    l[0] += p0 + p1, l[1] += p2 + p3;
                    p[2 * n] = pack_bf16x2(p0, p1);
                    p[2 * n + 1] = pack_bf16x2(p2, p3);
                }
                // values that no row sees are cleared in the operand registers, which hold keys c2,
                // c2 + 1 and c2 + 8, c2 + 9: 0 x NaN would reach the sum otherwise
                uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
                if (!inside) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = tok + 16 * h + 8 * e + c2;
                        auto any_sees = [&](int x) { return (x >= any_lo || x < sinks) && x < any_hi; };
                        keep[e] = (any_sees(key) ? 0xFFFFu : 0u) | (any_sees(key + 1) ? 0xFFFF0000u : 0u);
                    }
                }
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t vf[4];
                    ldsm_x4_t(vf, vb + (n >> 2) * S::kColumn + (16 * h + v_row) * 128 +
                                      ((((n & 3) * 2 + v_bit) ^ (v_row & 7)) << 4));
                    mma_bf16(o[2 * n], p, vf[0] & keep[0], vf[1] & keep[1]);
                    mma_bf16(o[2 * n + 1], p, vf[2] & keep[0], vf[3] & keep[1]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(done);
        }

        // ------------------------------------------------ the warps of this segment meet
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
            l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
            if (dead) m[e] = 0.f, l[e] = NAN;
            if ((lane & 3) == 0) ml[warp * S::kRows + g8 + 8 * e] = make_float2(m[e], l[e]);
        }
        float *mine = merge + (warp * S::kRows + g8) * S::kPitch + c2;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            *reinterpret_cast<float2 *>(mine + n * 8) = make_float2(o[n][0], o[n][1]);
            *reinterpret_cast<float2 *>(mine + 8 * S::kPitch + n * 8) = make_float2(o[n][2], o[n][3]);
        }
        }
        named_bar_sync(1, S::kConsumers);
        // CTAs that share the item, in the order of their tiles
        const bool whole = g.whole;
        constexpr int kSlot = rows_slot_words(D);
        const int n4 = max(g.rows, 0) * (D / 4);
        auto finish = [&](int row, int d4, float M, float L, float4 acc) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const int all = g.rb * S::kRows + row, i = all / a.group, h = g.hk * a.group + all - i * a.group;
            const long long tok = g.s.q0 + i;
            uint2 w = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            *reinterpret_cast<uint2 *>(a.out.p + tok * a.out.ts + h * a.out.hs + 4 * d4) = w;
            if (d4 == 0 && a.lse) a.lse[tok * a.q_heads + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
        };
        int first = 0, last = 0;
        float *slot_out = a.partials;
        if (!whole) {
            first = (int)(((g.item0 + 1) * deal.G - 1) / deal.total);
            last = (int)(((g.item0 + g.steps) * deal.G - 1) / deal.total);
            slot_out += (size_t)(2 * blockIdx.x + ((int)blockIdx.x == first ? 1 : 0)) * kSlot;
        }
        for (int idx = tid; idx < n4; idx += S::kConsumers) {
            const int row = idx / (D / 4), d4 = idx - row * (D / 4);
            float2 s[kWarps];
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s[w] = ml[w * S::kRows + row], M = fmaxf(M, s[w].x);
            const float base = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(s[w].x - base);
                const float4 v = *reinterpret_cast<const float4 *>(merge + (w * S::kRows + row) * S::kPitch + 4 * d4);
                L = fmaf(s[w].y, f, L);
                acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
                acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
            }
            if (whole) {
                finish(row, d4, M, L, acc);
            } else {
                __stcg(reinterpret_cast<float4 *>(slot_out + row * D + 4 * d4), acc);
                if (d4 == 0) __stcg(reinterpret_cast<float2 *>(slot_out + S::kRows * D + 2 * row), make_float2(M, L));
            }
        }
        if (!whole) __threadfence();
        named_bar_sync(1, S::kConsumers);  // also: the buffers are free for the next segment
        if (whole) continue;
        if (tid == 0) {
            const unsigned ticket = atomicAdd(&a.counters[first], 1u);
            last_s = ticket == (unsigned)(last - first);
            if (last_s) a.counters[first] = 0;
            __threadfence();
        }
        named_bar_sync(1, S::kConsumers);
        if (last_s) {
            // all parts' maxima and sums at once, then every part's rows with their weights
            float2 *parts = reinterpret_cast<float2 *>(merge);
            const int n = last - first + 1;
            for (int i = tid; i < n * S::kRows; i += S::kConsumers) {
                const int k = first + i / S::kRows;
                if ((i % S::kRows) < g.rows)
                    parts[i] = __ldcg(reinterpret_cast<const float2 *>(
                        a.partials + (size_t)(2 * k + (k == first ? 1 : 0)) * kSlot + S::kRows * D + 2 * (i % S::kRows)));
            }
            named_bar_sync(1, S::kConsumers);
            for (int idx = tid; idx < n4; idx += S::kConsumers) {
                const int row = idx / (D / 4), d4 = idx - row * (D / 4);
                float M = -INFINITY, L = 0.f;
                for (int k = 0; k < n; ++k) M = fmaxf(M, parts[k * S::kRows + row].x);
                const float base = M == -INFINITY ? 0.f : M;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int k = 0; k < n; ++k) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(
                        a.partials + (size_t)(2 * (first + k) + (k == 0 ? 1 : 0)) * kSlot + row * D + 4 * d4));
                    const float2 s = parts[k * S::kRows + row];
                    const float f = ex2(s.x - base);
                    L = fmaf(s.y, f, L);
                    acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
                    acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
                }
                finish(row, d4, M, L, acc);
            }
        }
        named_bar_sync(1, S::kConsumers);  // the buffers and last_s are read before the next segment writes them
    }
}

template <int D, bool CAPPED, bool SINKS, int TYPE, int ROWS>
cudaError_t launch_d(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t stream) {
    using S = RowsShape<D, TYPE != 0, ROWS>;
    static std::atomic<uint64_t> attr_done{0};
    DeviceInfo di;
    cudaError_t err = device_info(&di);
    if (err != cudaSuccess) return err;
    int dev = 0;
    err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    constexpr size_t kFixed = 1024 + S::kWarps * S::kRing + S::kMergeBytes + S::kMlBytes;
    static_assert(kFixed + 4 * (FD_MAX_BATCH + 1) + 1024 <= 227 * 1024, "shared memory");
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 64 || !(attr_done.load(std::memory_order_acquire) & bit)) {
        if (S::kWorkRegs > 0) {  // the warps' register shares wait for one another if the launch brings fewer
            cudaFuncAttributes fa;
            err = cudaFuncGetAttributes(&fa, attn_rows_kernel<D, CAPPED, SINKS, TYPE, ROWS>);
            if (err != cudaSuccess) return err;
            if (fa.numRegs < S::kLaunchRegs) return cudaErrorInvalidConfiguration;
        }
        err = cudaFuncSetAttribute(attn_rows_kernel<D, CAPPED, SINKS, TYPE, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)(kFixed + 4 * (FD_MAX_BATCH + 1)));
        if (err != cudaSuccess) return err;
        if (dev < 64) attr_done.fetch_or(bit, std::memory_order_acq_rel);
    }
    const long long row_blocks = ((long long)a.m.max_q * a.group + S::kRows - 1) / S::kRows;
    const long long tiles = (a.m.capacity + S::kTile - 1) / S::kTile;
    const long long most = (long long)a.m.batch * row_blocks * a.kv_heads * (tiles > 0 ? tiles : 1);
    long long grid = di.sm_count < kAttnMaxCtas ? di.sm_count : kAttnMaxCtas;
    if (grid > most) grid = most;
    // nothing is read before the wait: one token of 4097 keys 11.1 us a call, 12.3 without
    err = launch_kernel_as(true, attn_rows_kernel<D, CAPPED, SINKS, TYPE, ROWS>, dim3((unsigned)grid), dim3(S::kThreads),
                        kFixed + 4 * (size_t)(a.m.batch + 1), stream, 1, mk, mv, a, (int)row_blocks);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

// The kernel that a call takes, of those over one kind of cache.
template <int TYPE, int ROWS>
cudaError_t launch_as(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t stream) {
    auto launch = [&](auto capped, auto sinks) {
        constexpr bool kCapped = decltype(capped)::value, kSinks = decltype(sinks)::value;
        return a.head_dim == 128 ? launch_d<128, kCapped, kSinks, TYPE, ROWS>(a, mk, mv, stream)
                                 : launch_d<64, kCapped, kSinks, TYPE, ROWS>(a, mk, mv, stream);
    };
    auto with_cap = [&](auto sinks) {
        return a.softcap > 0.f ? launch(std::true_type{}, sinks) : launch(std::false_type{}, sinks);
    };
    return a.sinks > 0 ? with_cap(std::true_type{}) : with_cap(std::false_type{});
}

}  // namespace
}  // namespace fd
