// fd_attn_rows.cu - attention of few query rows per key head over a paged cache: decoding, and
// short chunks.
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
#include <atomic>
#include <type_traits>

#include "fd_attn.h"
#include "fd_tc.cuh"

namespace fd {
namespace {

// What joining the parts of an item costs, in tiles: a partial result written, a ticket, the
// other parts read.
constexpr int kJoinTiles = 6;

constexpr int kKeys = 32;  // of a tile, a warp's

template <int D>
struct RowsShape {
    static constexpr int kWarps = rows_warps(D);
    static constexpr int kConsumers = kWarps * 32;
    static constexpr int kThreads = 2 * kConsumers;      // each computing warp, its copying warp
    static constexpr int kTile = kWarps * kKeys;         // keys of a tile
    static constexpr int kHalves = D / 64;               // 128-byte columns of a row
    static constexpr int kColumn = kKeys * 128;          // bytes of one of a warp's keys
    static constexpr int kPart = kHalves * kColumn;      // a warp's keys (or values) of a tile
    static constexpr int kStages = 2;                    // 128 KB of shared memory in all
    static constexpr int kRing = kStages * 2 * kPart;    // of one warp
    static constexpr int kPitch = D + 8;                 // floats; conflict-free accumulator rows
    static constexpr int kMergeBytes = kWarps * kRowsM * kPitch * 4;
    static constexpr int kMlBytes = kWarps * kRowsM * 8;
    static_assert(kMergeBytes >= kAttnMaxCtas * kRowsM * 8, "the parts' maxima and sums fit the buffer");
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

// One run of tiles of one item.
struct Segment {
    SeqInfo s;
    int b, item;        // item: block of rows * kv_heads + key head
    int rb, hk;
    int i0, i1;         // first and last new token of the block's rows
    int rows;           // rows of the block
    int tile0;          // number of the first tile of the item's keys
    int from, to;       // the segment's tiles, counted in the item
    int nt;             // tiles of the item; 0: nothing to do
    long long item0;    // the item's first tile in the list
    long long next;     // what comes after the segment
};

// Tiles that the keys of sequence s take (at least one, so that every row is written), and the
// first of them. The same for all of the sequence's items.
template <int TILE>
__device__ __forceinline__ int seq_tiles(const SeqInfo &s, const AttnArgs &a, int *first) {
    *first = 0;
    if (s.rows <= 0) return 0;
    const int lo = key_lo(s, 0, a.window), hi = key_hi(s, s.rows - 1, a.causal);
    if (hi <= lo) return 1;
    *first = lo / TILE;
    return (hi + TILE - 1) / TILE - *first;
}

// How the list of tiles is dealt out.
struct Deal {
    const unsigned *prefix;   // tiles of one item of each sequence before b
    int items;                // of a sequence
    long long total;          // tiles
    int G;                    // CTAs that work
    bool whole;               // items c, c + G, ... instead of tiles [begin, end)
    long long begin, end;     // tiles, or items
};

// The segment at x (a tile of the list, or an item); `b` is a sequence at or before x's.
template <int TILE>
__device__ __forceinline__ Segment segment_at(const AttnArgs &a, const Deal &d, long long x, int b) {
    Segment g;
    const unsigned *prefix = d.prefix;
    const int items = d.items;
    if (d.whole) {
        b = (int)((unsigned)x / (unsigned)items);
        g.item = (int)x - b * items;
        g.nt = (int)(prefix[b + 1] - prefix[b]);
        g.from = 0, g.to = g.nt;
        g.item0 = 0;
        g.next = x + d.G;
    } else {
        // the first b with prefix[b + 1] * items > x: this sequence, the next, or by bisection
        if ((long long)prefix[b + 1] * items <= x && (long long)prefix[++b + 1] * items <= x) {
            int up = a.m.batch - 1;
            for (++b; b < up;) {
                const int mid = (b + up) >> 1;
                if ((long long)prefix[mid + 1] * items > x)
                    up = mid;
                else
                    b = mid + 1;
            }
        }
        g.nt = (int)(prefix[b + 1] - prefix[b]);
        const long long in_seq = x - (long long)prefix[b] * items;
        // 32 bits where they do: a 64-bit division is a hundred instructions
        g.item = in_seq >> 32 ? (int)(in_seq / g.nt) : (int)((unsigned)in_seq / (unsigned)g.nt);
        g.from = (int)(in_seq - (long long)g.item * g.nt);
        g.item0 = x - g.from;
        g.to = (int)min((long long)g.nt, d.end - g.item0);
        g.next = g.item0 + g.to;
    }
    g.b = b;
    g.s = load_seq(a.m, b);
    g.rb = g.item / a.kv_heads;
    g.hk = g.item - g.rb * a.kv_heads;
    seq_tiles<TILE>(g.s, a, &g.tile0);
    const int all = g.s.rows * a.group;
    g.rows = min(kRowsM, all - g.rb * kRowsM);  // <= 0: no such block in this sequence
    g.i0 = g.rb * kRowsM / a.group;
    g.i1 = min(g.s.rows, (g.rb * kRowsM + kRowsM - 1) / a.group + 1) - 1;
    return g;
}

// CAPPED: the scores go through the tanh (apart, so that its code costs the others nothing: in one
// kernel, 128 sequences of 500 at head_dim 64 took 29.9 us without a cap, 28.9 apart).
template <int D, bool CAPPED>
__global__ void __launch_bounds__(RowsShape<D>::kThreads, 1)
    attn_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const AttnArgs a, int row_blocks) {
    using S = RowsShape<D>;
    constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kTile = S::kTile;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    __shared__ int last_s, abort_flag;
    __shared__ __align__(8) uint64_t full[kWarps][S::kStages], empty[kWarps][S::kStages];
    __shared__ TileCopy next_tiles[kWarps][kAhead];
    __shared__ unsigned warp_sum[2 * kWarps], warp_max[2 * kWarps];
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
                mbar_init(&full[w][i], 1);
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
        unsigned sum = 0, most = 0;
        int first;
        for (int b = b0; b < b1; ++b) {
            const unsigned n = (unsigned)seq_tiles<kTile>(load_seq(a.m, b), a, &first);
            prefix[b] = sum;  // of this thread's sequences
            sum += n;
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
        for (int w = 0; w < 2 * kWarps; ++w) {
            if (w < (tid >> 5)) before += warp_sum[w];
            all += warp_sum[w];
            most = max(most, warp_max[w]);
        }
        for (int b = b0; b < b1; ++b) prefix[b] += before;
        if (tid == 0) prefix[a.m.batch] = all;
        __syncthreads();
        deal.prefix = prefix;
        deal.items = row_blocks * a.kv_heads;
        deal.total = (long long)all * deal.items;
        const long long n = (long long)a.m.batch * deal.items;
        const int c = blockIdx.x;
        // Whole items one after the other, or equal runs of tiles joined where they meet: what a CTA
        // gets of the first at most, counted, or estimated where that would take long.
        const int G = gridDim.x;
        long long share = most;
        if (n > 16 * G) {
            share = deal.total / G + 3 * most;
        } else if (n > G) {
            unsigned *const of = reinterpret_cast<unsigned *>(merge);  // not in use yet
            for (int i = tid; i < kAttnMaxCtas; i += kThreads) of[i] = 0;
            __syncthreads();
            for (int i = tid; i < (int)n; i += kThreads) {
                const int b = i / deal.items;
                atomicAdd(&of[i % G], prefix[b + 1] - prefix[b]);
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
    const long long wait_limit = a.test_timeout ? kTestWaitLimitCycles : kWaitLimitCycles;
    if (tid >= S::kConsumers) {
        // ---------------------------------------------------------------------- copies
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
                g = segment_at<kTile>(a, deal, x, b_at);
                b_at = g.b;
                x = g.next;
                tile = g.from - 1;
                lo = key_lo(g.s, 0, a.window), hi = key_hi(g.s, g.s.rows - 1, a.causal);
            }
            if (lane == 0) {
                volatile TileCopy &t = ahead[entry];
                const int tok = (g.tile0 + tile) * kTile + warp * kKeys;
                const int *row = a.m.table + (long long)g.b * a.m.table_stride;
                int read = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int first = tok + 16 * i;
                    if (more && first < hi && first + 16 > lo) {
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
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&empty[warp][slot], phase, &abort_flag, wait_limit));
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
                        unsigned char *const to = dst + h * S::kColumn + first * 128;
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
        const Segment g = segment_at<kTile>(a, deal, x, b_at);
        b_at = g.b;
        x = g.next;
        if (g.nt == 0) continue;
        // the rows of this lane: tokens, heads and visible keys
        uint32_t qf[D / 16][4];
        int hi[2], lo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = g8 + 8 * e, all = g.rb * kRowsM + row;
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
            if (!dead) dead = !__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[warp][stage], phase, &abort_flag, wait_limit));
            if (dead) break;
            const uint32_t kb = ring + stage * 2 * S::kPart, vb = kb + S::kPart;
            uint64_t *const done = &empty[warp][stage];
            if (++stage == S::kStages) stage = 0, phase ^= 1u;
            const int tok = (g.tile0 + t) * kTile + warp * kKeys;  // the warp's first key
            // a warp's keys outside every row's range (the ends of a window) add nothing
            if (g.rows <= 0 || tok >= any_hi || tok + kKeys <= any_lo) {
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
            const bool inside = tok >= in_lo && tok + kKeys <= in_hi;
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
                        if (key < lo[i >> 1] || key >= hi[i >> 1]) s[n][i] = -INFINITY;
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
                        keep[e] = (key >= any_lo && key < any_hi ? 0xFFFFu : 0u) |
                                  (key + 1 >= any_lo && key + 1 < any_hi ? 0xFFFF0000u : 0u);
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
            if ((lane & 3) == 0) ml[warp * kRowsM + g8 + 8 * e] = make_float2(m[e], l[e]);
        }
        float *mine = merge + (warp * kRowsM + g8) * S::kPitch + c2;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            *reinterpret_cast<float2 *>(mine + n * 8) = make_float2(o[n][0], o[n][1]);
            *reinterpret_cast<float2 *>(mine + 8 * S::kPitch + n * 8) = make_float2(o[n][2], o[n][3]);
        }
        named_bar_sync(1, S::kConsumers);
        // CTAs that share the item, in the order of their tiles
        const bool whole = g.from == 0 && g.to == g.nt;
        constexpr int kSlot = rows_slot_words(D);
        const int n4 = max(g.rows, 0) * (D / 4);
        auto finish = [&](int row, int d4, float M, float L, float4 acc) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const int all = g.rb * kRowsM + row, i = all / a.group, h = g.hk * a.group + all - i * a.group;
            const long long tok = g.s.q0 + i;
            uint2 w = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            *reinterpret_cast<uint2 *>(a.out.p + tok * a.out.ts + h * a.out.hs + 4 * d4) = w;
            if (d4 == 0 && a.lse) a.lse[tok * a.q_heads + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
        };
        int first = 0, last = 0;
        float *slot_out = a.partials;
        if (!whole) {
            first = (int)(((g.item0 + 1) * deal.G - 1) / deal.total);
            last = (int)(((g.item0 + g.nt) * deal.G - 1) / deal.total);
            slot_out += (size_t)(2 * blockIdx.x + ((int)blockIdx.x == first ? 1 : 0)) * kSlot;
        }
        for (int idx = tid; idx < n4; idx += S::kConsumers) {
            const int row = idx / (D / 4), d4 = idx - row * (D / 4);
            float2 s[kWarps];
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s[w] = ml[w * kRowsM + row], M = fmaxf(M, s[w].x);
            const float base = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(s[w].x - base);
                const float4 v = *reinterpret_cast<const float4 *>(merge + (w * kRowsM + row) * S::kPitch + 4 * d4);
                L = fmaf(s[w].y, f, L);
                acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
                acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
            }
            if (whole) {
                finish(row, d4, M, L, acc);
            } else {
                __stcg(reinterpret_cast<float4 *>(slot_out + row * D + 4 * d4), acc);
                if (d4 == 0) __stcg(reinterpret_cast<float2 *>(slot_out + kRowsM * D + 2 * row), make_float2(M, L));
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
            for (int i = tid; i < n * kRowsM; i += S::kConsumers) {
                const int k = first + (i >> 4);
                if ((i & 15) < g.rows)
                    parts[i] = __ldcg(reinterpret_cast<const float2 *>(
                        a.partials + (size_t)(2 * k + (k == first ? 1 : 0)) * kSlot + kRowsM * D + 2 * (i & 15)));
            }
            named_bar_sync(1, S::kConsumers);
            for (int idx = tid; idx < n4; idx += S::kConsumers) {
                const int row = idx / (D / 4), d4 = idx - row * (D / 4);
                float M = -INFINITY, L = 0.f;
                for (int k = 0; k < n; ++k) M = fmaxf(M, parts[k * kRowsM + row].x);
                const float base = M == -INFINITY ? 0.f : M;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int k = 0; k < n; ++k) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(
                        a.partials + (size_t)(2 * (first + k) + (k == 0 ? 1 : 0)) * kSlot + row * D + 4 * d4));
                    const float2 s = parts[k * kRowsM + row];
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

template <int D, bool CAPPED>
cudaError_t launch_d(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t stream) {
    using S = RowsShape<D>;
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
        err = cudaFuncSetAttribute(attn_rows_kernel<D, CAPPED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)(kFixed + 4 * (FD_MAX_BATCH + 1)));
        if (err != cudaSuccess) return err;
        if (dev < 64) attr_done.fetch_or(bit, std::memory_order_acq_rel);
    }
    const long long row_blocks = ((long long)a.m.max_q * a.group + kRowsM - 1) / kRowsM;
    const long long tiles = (a.m.capacity + S::kTile - 1) / S::kTile;
    const long long most = (long long)a.m.batch * row_blocks * a.kv_heads * (tiles > 0 ? tiles : 1);
    long long grid = di.sm_count < kAttnMaxCtas ? di.sm_count : kAttnMaxCtas;
    if (grid > most) grid = most;
    // nothing is read before the wait: one token of 4097 keys 11.1 us a call, 12.3 without
    err = launch_kernel_as(true, attn_rows_kernel<D, CAPPED>, dim3((unsigned)grid), dim3(S::kThreads),
                        kFixed + 4 * (size_t)(a.m.batch + 1), stream, 1, mk, mv, a, (int)row_blocks);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                             cudaStream_t stream) {
    if (a.softcap > 0.f)
        return a.head_dim == 128 ? launch_d<128, true>(a, mk, mv, stream) : launch_d<64, true>(a, mk, mv, stream);
    return a.head_dim == 128 ? launch_d<128, false>(a, mk, mv, stream) : launch_d<64, false>(a, mk, mv, stream);
}

FD_DEFINE_STATUS_ACCESSOR(status_attn_rows)

}  // namespace fd
