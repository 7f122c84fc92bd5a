// fd_attn_tc.cu - attention of chunks of new tokens over a paged cache on the fifth-generation
// tensor cores.
//
// The rows of a key head are (new token, query head of its group) pairs, token by token; a CTA
// takes 2 x 128 of them (two halves of floor(128 / group) tokens), so that each tile of keys and
// values, copied once, serves all the heads that share it. Per tile of 128 keys and half:
//     S = Q K^T (128 x 128 in tensor memory),  P = exp(S - m),  O = O + P V (in tensor memory).
// Bound by the tensor cores: 4 * 128 * 128 * D flops a tile and half. A prompt of 8192 (32 heads on
// 8, D 128) takes 361 us: 1520 TFLOP/s, 79 % of what a large matrix product reaches, while the SM clock
// is 2070 MHz. Run on end for longer than some 50 ms, singly or in a graph, it takes 382 (1440 TFLOP/s,
// 85 % of the product's rate under the power limit): the clock is then 1960 MHz. 512 tokens behind 16000
// take 118 us, 1150 TFLOP/s. A CTA spends 3500 cycles on a tile of both halves: the 32
// MMAs take 70 each, 2250 in all (64 at the tensor cores' full rate), and for the rest the tensor
// cores wait for probabilities, a half's softmax (1600 cycles, latencies more than issue slots) being
// longer than the other half's MMAs (1130). At D = 64 the MMAs are shorter and the softmax is not:
// 700 TFLOP/s. Tiles of 64 keys, whose scores can be ready before they are wanted, need more and
// shorter MMAs: 500 us for that prompt.
//
//   * One warp copies key and value tiles (tensor-map copies of a page's 64-element columns) into a
//     ring, one warp issues the MMAs, one deals out the work, and two groups of eight warps do the
//     softmax of one half each, two threads a row. While one half is in the softmax the tensor cores
//     run the other's P V and next S: per tile the MMA warp issues, for each half in turn, P V of
//     this tile and then S of the next, and never waits for its own results.
//   * Registers: at 104 a softmax thread the kernels spill 8 to 14 words a thread, with large caps 17.
//   * S, P and O stay in tensor memory: P (bf16, two a column) takes the first half of S's
//     columns and is the A operand of the second product from there. MMAs run in the order of
//     issue, so the next S may overwrite P without a wait. Q and both operands of S are
//     128-byte-swizzled K-major tiles; V is read as it lies, N-major.
//   * The running maximum that P is taken against is only raised when a row's maximum has grown by
//     more than 2^8 (then O is rescaled in tensor memory); up to there the sums hold the larger
//     values exactly as well, fp32 and bf16 being floating point. P is rounded to bf16 (2^-8
//     relative at most), the row's sum is that of the unrounded values, in fp32.
//   * Work: up to kMaxListed pairs of halves and the grid is one CTA an SM, which deals itself
//     items (a pair and a key head), or, where whole items do not come out even, equal runs of the
//     tiles of all items; what several CTAs share is joined by a second kernel (512 tokens behind
//     16000: 118 us, 241 in whole items). More pairs than that are whole items in any case (a prompt
//     of 8192, with a list long enough and without: 380 and 376 us). With more sequences than a CTA lists, each CTA takes one item, the
//     longest first (100 chunks of 40 behind 1000: 105 us, 94 by the list).
//   * Values of the first and last tile that no row of the item sees are cleared in shared memory
//     before their MMA (0 x NaN): pages hold anything past the last token.
//   * Every wait is bounded; a CTA that gives up writes NaN, drains its copies and MMAs and frees
//     its tensor memory.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fd_attn.h"
#include "fd_tc.cuh"

namespace fd {
namespace {

constexpr int kTile = 128;           // keys of a tile, rows of a half
constexpr int kSoftmax = 512;        // softmax threads: two for each row, half of its columns each
constexpr int kHalf = kSoftmax / 2;  // of one half
constexpr int kMmaWarp = 16, kCopyWarp = 17, kDealWarp = 18;
constexpr int kThreads = 640;        // the last four warps: MMA, copies, dealing, one idle
// Registers: 640 threads launch with 96 each (61440 in all); 512 x 104 + 128 x 64 = 61440.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 104, kOtherRegs = 64;
static_assert(kSoftmax * kSoftmaxRegs + (kThreads - kSoftmax) * kOtherRegs <= kThreads * kLaunchRegs, "registers");
constexpr int kMaxListed = kAttnTcListed;  // pairs, and sequences, of one list
// How the work is dealt out (launch_d).
enum { kOneItem, kListed, kPersistent };
// The kernels for capped scores. Where a warp has scores past the cap, all of its scores in that tile
// are c (1 - 2 / (e^(2 y) + 1)), off by 6 2^-24 of the cap; of a cap of kLargeCap 4 10^-4, a tenth of a
// probability's rounding. Past that, those below the cap go by the polynomial there too (two prompts of
// 2048 in 28 heads of 64 capped at 3: 114 us, 157 so).
enum { kUncapped, kUsualCaps, kLargeCaps };
constexpr float kLargeCap = 1024.f;
// How a tile's scores are capped: not at all, all of a warp's below half the cap or below the cap, any.
enum { kNoCap, kNearCap, kBelowCap, kAnyCap };
constexpr float kRaise = 8.f;        // log2 units
// In tiles: what beginning an item costs (its queries loaded, the last result written), and what
// joining the parts of one costs, at all and for each part of 256 rows (128 KB written and read
// again).
constexpr int kItemTiles = 2, kJoinTiles = 4;
constexpr float kPartTiles = 0.3f;

template <int D>
struct TcShape {
    static constexpr int kHalves = D / 64;
    static constexpr int kQ = kTile * D * 2;       // bytes of one half's queries
    static constexpr int kStage = kTile * D * 2;   // a tile of keys or of values
    static constexpr int kStages = 4;
    static constexpr int kSmem = 1024 + 2 * kQ + kStages * kStage;
    // tensor memory columns: S (and P in its first half) and O of both halves
    static constexpr uint32_t kS0 = 0, kO0 = 2 * kTile;
};

// Makes the registers of a tensor-memory load depend on the wait that came before.
template <int N>
__device__ __forceinline__ void pin(uint32_t *r) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ long long wait_limit(int test) { return test ? kTestWaitLimitCycles : kWaitLimitCycles; }

// Bounded wait that ignores the abort flag (copies landing, MMAs completing).
__device__ __forceinline__ void wait_hw(uint64_t *bar, uint32_t parity, int test) {
    const long long t0 = clock64();
    while (!mbar_try_parity(bar, parity) && clock64() - t0 < wait_limit(test)) {
    }
}

// mbar_wait_bounded with the slow path in line: a call would bind this kernel's registers to the
// calling convention, which a kernel that moves registers between its warps has none left for.
__device__ __forceinline__ bool wait_bounded(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int test) {
    if (mbar_try_parity(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_parity(bar, parity)) {
        if (*abort_flag) return false;
        if (clock64() - t0 > wait_limit(test)) {
            *abort_flag = 1;
            record_wait_timeout();
            return false;
        }
    }
    return true;
}

// Sum over the lanes up to this one.
__device__ __forceinline__ unsigned warp_sum_to(unsigned v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned up = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += up;
    }
    return v;
}

// Tiles of 128 keys [a, b) that new tokens i0 .. i1 see together (a >= b: none).
struct TileRange {
    int a, b;
};
__device__ __forceinline__ TileRange tiles_of(const SeqInfo &s, const AttnArgs &p, int i0, int i1) {
    const int lo = key_lo(s, i0, p.window), hi = key_hi(s, i1, p.causal);
    if (i1 < i0 || hi <= lo) return {0, 0};
    return {lo / kTile, (hi + kTile - 1) / kTile};
}

// What a CTA does.
struct Deal {
    int begin, end;   // of the list, or rounds of whole items
    int run;          // 0: whole items; else the list is dealt out in runs of this length
    int n_pairs;
};

// One run of tiles of one item (pair of halves, key head).
struct Segment {
    SeqInfo s;
    int b, hk;
    int i0;            // first new token of the pair
    int ja, jb;        // tiles of the run
    TileRange h[2];    // of it, what each half sees
    int lo, hi;        // keys that some row of the pair sees
    int first, last;   // CTAs that share the item
    int next;          // what comes behind the run
    int valid;         // 0: there are no more runs
};

__device__ __forceinline__ void clip_halves(Segment &g, const AttnArgs &a, int tokens, int from, int to) {
    g.lo = key_lo(g.s, g.i0, a.window);
    g.hi = key_hi(g.s, min(g.s.rows, g.i0 + 2 * tokens) - 1, a.causal);
    g.ja = 1 << 30, g.jb = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i0 = g.i0 + e * tokens;
        TileRange r = tiles_of(g.s, a, i0, min(g.s.rows, i0 + tokens) - 1);
        r.a = max(r.a, from), r.b = min(r.b, to);
        if (r.b <= r.a) r = {0, 0};
        g.h[e] = r;
        if (r.b > r.a) g.ja = min(g.ja, r.a), g.jb = max(g.jb, r.b);
    }
    if (g.jb == 0) g.ja = 0;
}

// Tiles of the pair that begins at token i0 (at least one, so that every row is written).
__device__ __forceinline__ TileRange pair_tiles(const SeqInfo &s, const AttnArgs &a, int i0, int tokens) {
    TileRange r = tiles_of(s, a, i0, min(s.rows, i0 + 2 * tokens) - 1);
    if (r.b <= r.a) r = {0, 1};
    return r;
}

// The k-th whole item of CTA c: there and back again.
__device__ __forceinline__ int item_of(int k, int c, int G) { return k * G + (k & 1 ? G - 1 - c : c); }

constexpr int kRuns = 4;  // runs known ahead

// Barrier over `threads` threads that also tells all of them whether `any` held in one.
__device__ __forceinline__ bool bar_or(int id, int threads, bool any) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %3, 0;\n\t"
        "barrier.cta.red.or.pred p, %1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"((uint32_t)any)
        : "memory");
    return r != 0;
}

// CAP: whether the scores go through the tanh (apart, so that its code costs the others no registers).
template <int D, int CAP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const AttnArgs a, int tokens /* of a half */, int mode) {
    using T = TcShape<D>;
    constexpr bool CAPPED = CAP != kUncapped;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2];
    __shared__ __align__(8) uint64_t full[T::kStages], empty[T::kStages], done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ unsigned scan_s[kThreads / 32];
    __shared__ unsigned prefix[kMaxListed + 1];       // tiles of one key head before each pair
    __shared__ unsigned pairs_before[kMaxListed];     // of each sequence
    __shared__ Segment runs[kRuns];
    __shared__ __align__(8) uint64_t run_full[kRuns], run_empty[kRuns];
    __shared__ int pick_b, pick_t;                    // the one item of a CTA without a list
    unsigned char *smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    const uint32_t q_base = smem_u32(smem), ring = q_base + 2 * T::kQ;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        for (int e = 0; e < 2; ++e) {
            mbar_init(&q_full[e], 8);
            mbar_init(&s_full[e], 1);
            mbar_init(&p_full[e][0], 8);
            mbar_init(&p_full[e][1], 8);
            mbar_init(&o_full[e], 1);
        }
        for (int i = 0; i < T::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&done, 1);
        for (int i = 0; i < kRuns; ++i) {
            mbar_init(&run_full[i], 1);
            mbar_init(&run_empty[i], kMmaWarp + 2);  // every warp that works on it
        }
        abort_flag = 0;
        pick_b = -1;
        fence_mbar_init();
    }
    grid_dep_wait();
    // Between the two: a kernel that holds tensor memory never waits for one that wants some.
    if (warp == kMmaWarp) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }

    auto pairs_of = [&](int b) { return (unsigned)((load_seq(a.m, b).rows + 2 * tokens - 1) / (2 * tokens)); };
    if (mode == kOneItem) {
        // the last pairs of a sequence see the most keys, so they come first
        const int per = (a.m.batch + kThreads - 1) / kThreads;
        const int b0 = min(tid * per, a.m.batch), b1 = min(b0 + per, a.m.batch);
        unsigned mine = 0, total = 0;
        for (int b = b0; b < b1; ++b) mine += pairs_of(b);
        unsigned at = warp_sum_to(mine, lane);  // up to this thread's, in its warp
        if (lane == 31) scan_s[warp] = at;
        __syncthreads();
        at -= mine;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) at += scan_s[w];
            total += scan_s[w];
        }
        const unsigned back = blockIdx.x / a.kv_heads, want = total - 1 - back;
        if (back < total && at <= want && want < at + mine) {
            unsigned left = want - at;
            int b = b0;
            for (unsigned n; left >= (n = pairs_of(b)); ++b) left -= n;
            pick_b = b, pick_t = (int)left;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    grid_dep_launch();

    // The n-th run, as the dealing warp has written it down (its own waits are the shorter ones, so
    // this one ends), and that this warp is done with it.
    auto take = [&](int n) -> const volatile Segment & {
        const long long t0 = clock64();
        while (!mbar_try_parity(&run_full[n % kRuns], (uint32_t)(n / kRuns) & 1u) &&
               clock64() - t0 < 8 * kWaitLimitCycles) {
        }
        return runs[n % kRuns];
    };
    auto release = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&run_empty[n % kRuns]);
    };

    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kCopyWarp) {
        // ------------------------------------------------------------------ copies
        const int box = min(1 << a.m.page_shift, kTile);
        const int boxes = kTile / box;
        const int ops = boxes * T::kHalves;  // at most 16
        const int my_box = lane / T::kHalves, my_half = lane - my_box * T::kHalves;
        const uint32_t dst0 = my_half * (kTile * 128) + my_box * box * 128;
        const uint64_t policy = policy_evict_last();  // the other pairs of the sequence read them too
        int stage = 0;
        uint32_t phase = 0, issued = 0;
        bool ok = true;
        for (int n = 0;; ++n) {
            const volatile Segment &g = take(n);
            if (!g.valid) break;
            const int hk = g.hk, ja = g.ja, jb = g.jb, lo = g.lo, hi = g.hi;
            const int *const row = a.m.table + (long long)g.b * a.m.table_stride;
            release(n);
            if (!ok) continue;
            auto page_of = [&](int j) {
                const int tok = j * kTile + my_box * box;
                int page = a.m.num_pages;  // reads as zeros
                if (j < jb && lane < ops && tok < hi && tok + box > lo) {
                    const int id = row[tok >> a.m.page_shift];
                    if (id >= 0 && id < a.m.num_pages)
                        page = id;
                    else
                        atomicOr(&g_wait_status, (unsigned)FD_DEVICE_STATUS_BAD_PAGE);
                }
                return page;
            };
            int next_page = page_of(ja);
            for (int j = ja; j < jb && ok; ++j) {
                const int page = next_page;
                next_page = page_of(j + 1);
                const int off = (j * kTile + my_box * box) & ((1 << a.m.page_shift) - 1);
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    ok = __all_sync(0xFFFFFFFFu, wait_bounded(&empty[stage], phase ^ 1u, &abort_flag, a.test_timeout));
                    if (!ok) break;
                    const bool copy = !(a.test_timeout && issued == 0);
                    if (copy && lane == 0) mbar_arrive_expect_tx(&full[stage], T::kStage);
                    __syncwarp();
                    if (copy && lane < ops) {
                        const MapOrder ord = v ? a.ov : a.ok;
                        const int y1 = ord.tok == 1 ? off : ord.head == 1 ? hk : page;
                        const int y2 = ord.tok == 2 ? off : ord.head == 2 ? hk : page;
                        const int y3 = ord.tok == 3 ? off : ord.head == 3 ? hk : page;
                        tma_load_4d(smem + 2 * T::kQ + stage * T::kStage + dst0, v ? &map_v : &map_k, my_half * 64,
                                    y1, y2, y3, &full[stage], policy);
                    }
                    ++issued;
                    if (++stage == T::kStages) stage = 0, phase ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) {  // wait (bounded) for the copies in flight before the CTA ends
            const uint32_t n = issued < (uint32_t)T::kStages ? issued : (uint32_t)T::kStages;
            for (uint32_t i = issued - n; i < issued; ++i)
                wait_hw(&full[i % T::kStages], (i / T::kStages) & 1u, a.test_timeout);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------------------------- MMAs
        constexpr uint32_t idesc_s = idesc_bf16_f32(kTile, kTile);
        constexpr uint32_t idesc_o = idesc_bf16_f32(kTile, D) | (1u << 16);  // B is N-major
        // What the tensor-core instructions take is kept the same in all lanes, and broadcast, so
        // that it lies in uniform registers: issued from others, one MMA took 110 cycles. Broadcast
        // where it is used, or all of the loop's descriptors are kept in registers, and spill.
        auto same = [](uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
        const uint32_t tm = same(tmem), q_desc = same(desc_sw128_low(q_base)), k_desc = same(desc_sw128_low(ring));
        const uint32_t v_desc = same(desc_sw128_mn_low(ring, kTile * 128));
        int stage = 0;
        uint32_t phase = 0, q_ph[2] = {0, 0}, p_ph[2] = {0, 0};
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (!__all_sync(0xFFFFFFFFu, mbar_try_parity(bar, parity)))
                ok = ok && __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, &abort_flag, a.test_timeout));
            return ok;
        };
        auto scores = [&](int e, int st) {  // S_e = Q_e K^T
            const uint32_t qd = same(q_desc + e * (T::kQ >> 4)), kd = same(k_desc + st * (T::kStage >> 4));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4;
                    tc_mma_f16(tm + T::kS0 + e * kTile, desc_of(qd + off), desc_of(kd + off), idesc_s, k > 0);
                }
                tc_commit(&s_full[e]);
            }
            __syncwarp();
        };
        auto commit = [&](uint64_t *bar) { tc_commit_if(elect_one(), bar); };
        for (int n = 0;; ++n) {
            const volatile Segment &g = take(n);
            if (!same(g.valid)) break;
            const int ja = same(g.ja), jb = same(g.jb), lo = same(g.lo), hi = same(g.hi);
            const int ha[2] = {(int)same(g.h[0].a), (int)same(g.h[1].a)}, hb[2] = {(int)same(g.h[0].b), (int)same(g.h[1].b)};
            release(n);
            if (!ok) continue;
            if (jb <= ja) continue;
            if (!wait(&full[stage], phase)) continue;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (hb[e] > ha[e]) {
                    if (!wait(&q_full[e], q_ph[e])) break;
                    q_ph[e] ^= 1u;
                    tc_fence_after();
                    if (ja >= ha[e]) scores(e, stage);
                }
            if (!ok) continue;
            commit(&empty[stage]);
            if (++stage == T::kStages) stage = 0, phase ^= 1u;
            for (int j = ja; j < jb && ok; ++j) {
                const int vs = stage;
                const uint32_t vp = phase;
                if (++stage == T::kStages) stage = 0, phase ^= 1u;
                const int ks = stage;
                const uint32_t kp = phase;
                const bool more = j + 1 < jb;
                if (!wait(&full[vs], vp)) break;
                const int t0 = j * kTile;
                if (t0 < lo || t0 + kTile > hi) {
                    // rows of the tile that no row sees
                    const int n0 = max(lo - t0, 0), n1 = min(hi - t0, kTile);
                    for (int i = lane; i < kTile * T::kHalves * 8; i += 32) {
                        const int row = (i >> 3) & (kTile - 1);
                        if (row < n0 || row >= n1)
                            sts_v4(ring + vs * T::kStage + i * 16, make_uint4(0, 0, 0, 0));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                const uint32_t vd = same(v_desc + vs * (T::kStage >> 4));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (j >= ha[e] && j < hb[e]) {
                        // The first 32 keys of both 64s as soon as their probabilities are there, then
                        // the other ones.
                        // Predicated, not in a branch on the elected lane like the scores (a prompt of
                        // 8192: 367 us, 380 with both in branches, 370 with both predicated).
                        const bool issue = elect_one();
                        auto values = [&](int k, uint32_t accumulate) {  // keys 16 k ..
                            tc_mma_f16_ts_if(issue, tm + T::kO0 + e * kTile,
                                             tm + T::kS0 + e * kTile + (k >> 2) * 64 + (k & 3) * 8,
                                             desc_of(vd + k * (2048 >> 4)), idesc_o, accumulate);
                        };
                        if (!wait(&p_full[e][0], p_ph[e])) break;
                        tc_fence_after();
                        values(0, j > ha[e]);
                        values(1, 1), values(4, 1), values(5, 1);
                        if (!wait(&p_full[e][1], p_ph[e])) break;
                        p_ph[e] ^= 1u;
                        tc_fence_after();
                        values(2, 1), values(3, 1), values(6, 1), values(7, 1);
                        if (j + 1 == hb[e]) tc_commit_if(issue, &o_full[e]);
                    }
                    if (e == 1) commit(&empty[vs]);
                    if (more) {
                        if (e == 0) {
                            if (!wait(&full[ks], kp)) break;
                            tc_fence_after();
                        }
                        if (j + 1 >= ha[e] && j + 1 < hb[e]) scores(e, ks);
                        if (e == 1) commit(&empty[ks]);
                    }
                }
                if (more && ++stage == T::kStages) stage = 0, phase ^= 1u;
            }
        }
        if (elect_one()) {  // nothing may be in flight when the memory is given back
            tc_commit(&done);
            wait_hw(&done, 0, a.test_timeout);
        }
        __syncwarp();
    } else if (warp == kDealWarp) {
        // ----------------------------------------------------- what this CTA does, run by run
        const int G = gridDim.x, c = blockIdx.x;
        // the sequence of pair p
        auto seq_of = [&](unsigned p) {
            int b = 0;
            for (int up = a.m.batch - 1; b < up;) {  // the last one with no more than p pairs before it
                const int mid = (b + up + 1) >> 1;
                if (pairs_before[mid] <= p)
                    b = mid;
                else
                    up = mid - 1;
            }
            return b;
        };
        Deal deal{0, 0, 0, 0};
        if (mode == kOneItem) {
            deal.end = pick_b >= 0;
        } else {
            unsigned n_pairs = 0;
#pragma unroll 1
            for (int b0 = 0; b0 < a.m.batch; b0 += 32) {
                const int b = b0 + lane;
                const unsigned n = b < a.m.batch ? pairs_of(b) : 0, upto = warp_sum_to(n, lane);
                if (b < a.m.batch) pairs_before[b] = n_pairs + upto - n;
                n_pairs += __shfl_sync(0xFFFFFFFFu, upto, 31);
            }
            __syncwarp();
            unsigned all = 0, most = 0;  // the list's length for one key head; the longest item
            if (mode == kListed) {
                n_pairs = min(n_pairs, (unsigned)kMaxListed);  // more only where sequences share rows
                // one list: key head by key head, pair by pair, tile by tile
#pragma unroll 1
                for (unsigned p0 = 0; p0 < n_pairs; p0 += 32) {
                    const unsigned p = p0 + lane;
                    unsigned cost = 0;
                    if (p < n_pairs) {
                        const int b = seq_of(p);
                        const TileRange r = pair_tiles(load_seq(a.m, b), a, (p - pairs_before[b]) * 2 * tokens, tokens);
                        cost = r.b - r.a + kItemTiles;
                    }
                    const unsigned upto = warp_sum_to(cost, lane);
                    if (p < n_pairs) prefix[p] = all + upto - cost;
                    all += __shfl_sync(0xFFFFFFFFu, upto, 31);
                    most = max(most, cost);
                }
                if (lane == 0) prefix[n_pairs] = all;
                __syncwarp();
            }
            // Whole items, the last pairs of a sequence (which see the most keys) first and the order of
            // the CTAs turned round every time; or, where the longest share of that is too long, equal
            // runs of the list, joined where they meet. A run is long enough that joining an item's
            // parts takes no longer than one: C / run parts of f each cost as much as the run at
            // run = sqrt(f C).
            most = __reduce_max_sync(0xFFFFFFFFu, most);
            const float part = kPartTiles / 256.f * (float)min((long long)a.m.max_q * a.group, 256ll);
            const long long total = (long long)all * a.kv_heads;
            const long long run = max((total + G - 1) / G, (long long)ceilf(sqrtf(part * (float)most)));
            const float joined = (float)run + kJoinTiles + part * ceilf((float)most / (float)max(run, 1ll));
            const int n_items = (int)n_pairs * a.kv_heads;
            if (mode == kListed && n_items > G) {
                unsigned share[kAttnMaxCtas / 32] = {};
                const unsigned magic = 0xFFFFFFFFu / (unsigned)a.kv_heads + 1u;  // i / kv_heads, i < 2^18
#pragma unroll 1
                for (int k = 0; k * G < n_items; ++k) {
#pragma unroll
                    for (int q = 0; q < kAttnMaxCtas / 32; ++q) {
                        const int cta = lane + 32 * q, i = item_of(k, cta, G);
                        if (cta < G && i < n_items) {
                            const int p = (int)n_pairs - 1 -
                                          (a.kv_heads == 1 ? i : (int)__umulhi((unsigned)i, magic));
                            share[q] += prefix[p + 1] - prefix[p];
                        }
                    }
                }
                most = 0;
#pragma unroll
                for (int q = 0; q < kAttnMaxCtas / 32; ++q) most = max(most, share[q]);
            }
            most = __reduce_max_sync(0xFFFFFFFFu, most);  // of the shares, or of the items where they are that
            deal.n_pairs = (int)n_pairs;
            if (mode == kPersistent || total >= (1ll << 31) || (float)most <= joined) {
                deal.end = n_items / G;
                if (deal.end * G < n_items && item_of(deal.end, c, G) < n_items) ++deal.end;
            } else {
                deal.run = (int)run;
                const long long begin = run * c;
                if (begin < total) deal.begin = (int)begin, deal.end = (int)min(total, begin + run);
            }
        }
        int x = deal.begin;
        for (int n = 0;; ++n) {
            Segment g{};
            if (x < deal.end) {
                g.valid = 1;
                int from = 0, to = 1 << 30, t;
                g.next = x + 1;
                if (mode == kOneItem) {
                    g.b = pick_b, g.hk = c % a.kv_heads, t = pick_t;
                } else if (deal.run == 0) {
                    const int i = item_of(x, c, G), p = i / a.kv_heads;
                    const unsigned pair = deal.n_pairs - 1 - p;
                    g.hk = i - p * a.kv_heads, g.b = seq_of(pair), t = (int)(pair - pairs_before[g.b]);
                } else {
                    const int head = prefix[deal.n_pairs];
                    g.hk = x / head;
                    const unsigned in_head = (unsigned)(x - g.hk * head);
                    int p = 0;
                    for (int up = deal.n_pairs - 1; p < up;) {  // the last pair with prefix[p] <= in_head
                        const int mid = (p + up + 1) >> 1;
                        if (prefix[mid] <= in_head)
                            p = mid;
                        else
                            up = mid - 1;
                    }
                    g.b = seq_of(p), t = (int)(p - pairs_before[g.b]);
                    const int item0 = g.hk * head + prefix[p], item1 = g.hk * head + prefix[p + 1];
                    g.next = min(item1, deal.end);
                    // the run's share of the item's tiles: of v steps, kItemTiles in each
                    // (item1 - item0) are what beginning the item costs
                    const int cost = item1 - item0;
                    auto share = [&](int v) { return v - (kItemTiles * v + cost - 1) / cost; };
                    from = share(x - item0), to = share(g.next - item0);
                    g.first = item0 / deal.run;
                    g.last = (item1 - 1) / deal.run;
                }
                g.s = load_seq(a.m, g.b);
                g.i0 = t * 2 * tokens;
                const int base = deal.run == 0 ? 0 : pair_tiles(g.s, a, g.i0, tokens).a;
                clip_halves(g, a, tokens, base + from, base + to);
                x = g.next;
            }
            // room for it (bounded: those who hold a run give up on their own waits)
            const long long t0 = clock64();
            while (!mbar_try_parity(&run_empty[n % kRuns], ((uint32_t)(n / kRuns) & 1u) ^ 1u) &&
                   clock64() - t0 < 4 * kWaitLimitCycles) {
            }
            if (lane == 0) {
                runs[n % kRuns] = g;
                mbar_arrive(&run_full[n % kRuns]);
            }
            __syncwarp();
            if (!g.valid) break;
        }
    }
    } else {
        // ----------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // Thread (half e, columns 64 c .. 64 c + 63, row r). The two threads of a row keep the same
        // maximum; P takes the first 32 columns of each one's scores, O is shared out by columns too.
        const int e = warp >> 3, cg = warp >> 2 & 1;
        const int r = (warp & 3) * 32 + lane;        // row of the half, TMEM lane
        const int bar = 2 + e;                       // of the half's threads
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_addr = lane_base + T::kS0 + e * kTile + cg * 64;
        const uint32_t o_addr = lane_base + T::kO0 + e * kTile + cg * (D / 2);
        // The scale is positive (attn_uses_tc), so that what follows is monotone in S: the maximum of a
        // row is taken before scale and cap.
        const float cap_in = CAPPED ? a.scale / a.softcap : 0.f, cap_out = a.softcap * kLog2e;
        const float mul = CAPPED ? cap_in * (2.f * kLog2e) : a.scale * kLog2e, lin = a.scale * kLog2e;
        // a score in log2 units; c tanh(y) = c (1 - 2 / (e^(2 y) + 1))
        auto log2_score = [&](float v) {
            return CAPPED ? cap_out - __fdividef(2.f * cap_out, ex2(v * mul) + 1.f) : v * mul;
        };
        uint32_t s_ph = 0, o_ph = 0;
        bool dead = false;
        constexpr int kSlot = tc_slot_words(D);
        int ja = 0, jb = 0, lo = 0, hi = 0, in_lo = 0, in_hi = 0;
        constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes;  // of a row of Q in 16-byte loads
        constexpr int kLoads = 16 / kRowsAtOnce;                  // 16 rows a warp
        int head0 = 0, row0 = 0, rows = 0;  // of the run's Q: first head and row, tokens of the half
        // Takes up the n-th run: its tiles and visible keys for this row, and 16 rows of Q. False: there
        // is none.
        auto enter = [&](int n) {
            const volatile Segment &g = take(n);
            if (!g.valid) return false;
            const SeqInfo seq{g.s.q0, g.s.rows, g.s.kv, g.s.base};
            const int i_first = g.i0 + e * tokens, i_last = min(seq.rows, i_first + tokens) - 1;
            const int tl = r / a.group, i = i_first + tl;
            const bool live = tl < tokens && i < seq.rows;
            ja = e ? g.h[1].a : g.h[0].a, jb = e ? g.h[1].b : g.h[0].b;
            hi = live ? key_hi(seq, i, a.causal) : 0, lo = live ? key_lo(seq, i, a.window) : 0;
            in_hi = key_hi(seq, i_first, a.causal), in_lo = key_lo(seq, i_last, a.window);
            head0 = g.hk * a.group, row0 = seq.q0 + i_first, rows = min(tokens, seq.rows - i_first);
            return true;
        };
        // 16 rows of Q into the swizzled tile, asynchronously (rows without a token: zeros), and their
        // arrival. A loop, not unrolled: this is the first code of a launch, read from far.
        auto fetch_q = [&]() {
#pragma unroll 1
            for (int n = 0; n < kLoads; ++n) {
                const int row = (warp & 7) * 16 + n * kRowsAtOnce + lane / kLanes, c = lane % kLanes;
                const int t = row / a.group;
                const uint16_t *from = a.q.p + (long long)(row0 + t) * a.q.ts + (head0 + row - t * a.group) * a.q.hs + c * 8;
                const bool there = t < rows;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 q_base + e * T::kQ + row * 128 + (c >> 3) * (kTile * 128) + (((c & 7) ^ (row & 7)) << 4)),
                             "l"(there ? from : a.q.p), "r"(there ? 16 : 0)
                             : "memory");
            }
        };
        auto give_q = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[e]);
        };
        AttnPart part{0, 0, 0, 0, -1};
        bool more = enter(0);
        if (more && jb > ja) {
            fetch_q();
            give_q();
        }
        for (int run = 0; more; ++run) {
            float m = -INFINITY;      // what the exponentials are taken against, log2 units
            float m_seen = -INFINITY; // CAPPED: the score that it is, before scale and cap
            float2 l2 = make_float2(0.f, 0.f);
            const bool any = jb > ja && !dead;
            const int j0 = ja;
            for (int j = ja; j < jb && !dead; ++j) {
                const bool ok = __all_sync(0xFFFFFFFFu, wait_bounded(&s_full[e], s_ph, &abort_flag, a.test_timeout));
                s_ph ^= 1u;
                tc_fence_after();
                // Half of the scores are read twice, for their maximum and for the exponentials: tensor
                // memory is near, and all kept in registers they would leave too few for the rest
                // (what spills goes to L2, the shared memory has all of the L1).
                // Columns [c0, c1) of this thread's 64 are visible; all of them inside the range that
                // every row sees.
                const int t0 = j * kTile + cg * 64, c0 = lo - t0, c1 = hi - t0;
                const bool masked = t0 < in_lo || t0 + 64 > in_hi;
                uint32_t seen[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};  // a bit a column
                if (masked) {
                    auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; };
                    seen[0] = below(c1) & ~below(c0), seen[1] = below(c1 - 32) & ~below(c0 - 32);
                }
                float top, size = 0.f;
                uint32_t last_score, v0[16], v1[16];
                {
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    uint32_t u[32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tmem_ld_x32(s_addr + 32 * c, u);
                        tmem_ld_wait();
                        pin<32>(u);
                        if (masked) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                const bool see = seen[c] >> k & 1;
                                // how far from 0 the lowest one is
                                if (CAPPED && see) size = fmaxf(size, -__uint_as_float(u[k]));
                                if (!see) u[k] = 0xFF800000u;  // -infinity
                            }
                        } else if (CAPPED) {
#pragma unroll
                            for (int k = 0; k < 32; k += 2)
                                size = fmaxf(fmaxf(size, -__uint_as_float(u[k])), -__uint_as_float(u[k + 1]));
                        }
#pragma unroll
                        for (int k = 0; k < 32; k += 2)
                            mx[k >> 1 & 3] = fmaxf(fmaxf(mx[k >> 1 & 3], __uint_as_float(u[k])), __uint_as_float(u[k + 1]));
                        if (c == 1) last_score = u[31];
                    }
                    const float raw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    top = CAPPED || raw == -INFINITY ? raw : raw * mul;
                    size = fmaxf(size, raw);
                }
                // Raise the maximum: at the first keys, and when a row has grown by 2^kRaise (before the cap,
                // which makes growth smaller; what it makes of the maximum is computed here alone). All of
                // the half do it together, or none (and a wait that gave up ends the loop for all).
                const float over = CAPPED ? (top - m_seen) * lin : top - m;  // NaN where both are -infinity
                if (bar_or(bar, kHalf, !ok || over > kRaise)) {
                    if (bar_or(bar, kHalf, !ok)) {
                        dead = true;
                        break;
                    }
                    // the row's other maximum, by way of this thread's last column
                    tmem_st_x1(s_addr + 63, __float_as_uint(top));
                    tmem_st_wait();
                    tc_fence_before();
                    named_bar_sync(bar, kHalf);
                    tc_fence_after();
                    uint32_t other;
                    tmem_ld_x1((s_addr ^ 64u) + 63, &other);
                    tmem_ld_wait();
                    pin<1>(&other);
                    tc_fence_before();
                    named_bar_sync(bar, kHalf);
                    tc_fence_after();
                    tmem_st_x1(s_addr + 63, last_score);
                    tmem_st_wait();
                    float up = fmaxf(fmaxf(top, __uint_as_float(other)), CAPPED ? m_seen : m);
                    if (CAPPED) {
                        m_seen = up;
                        if (up != -INFINITY) up = capped_log2<false>(make_float2(up, up), lin, cap_in, cap_out).x;
                    }
                    const float f = m == -INFINITY ? 0.f : ex2(m - up);
                    m = up;
                    l2.x *= f, l2.y *= f;
                    if (j > j0) {
#pragma unroll 1
                        for (int c = 0; c < D / 2; c += 16) {
                            uint32_t o[16];
                            tmem_ld_x16(o_addr + c, o);
                            tmem_ld_wait();
                            pin<16>(o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st_x16(o_addr + c, o);
                        }
                    }
                }
                const float off = m == -INFINITY ? 0.f : -m;
                float2 la = make_float2(0.f, 0.f), lb = la;
                // Groups of 16 columns, one behind the other: the exponentials of a group are issued
                // between the sums and roundings of the one before, whose results have arrived by
                // then. Left together the compiler waits for each of them.
                auto step = [&](auto cap, auto hidden, uint32_t *su, const uint32_t *done, int n) {
                    float *y = reinterpret_cast<float *>(su);
                    const float *v = reinterpret_cast<const float *>(done);
                    constexpr int kCap = decltype(cap)::value;
                    uint32_t p[8];
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        if (n < 4) {
                            float2 f = make_float2(y[k], y[k + 1]);
                            if constexpr (kCap == kNoCap) {
                                f = ffma2(f, make_float2(mul, mul), make_float2(off, off));
                            } else if constexpr (kCap == kAnyCap) {
                                if constexpr (CAP == kLargeCaps)
                                    f = fadd2(capped_log2<false>(f, lin, cap_in, cap_out), make_float2(off, off));
                                else
                                    f.x = log2_score(f.x) + off, f.y = log2_score(f.y) + off;
                            } else {
                                // (s tanh(y) / y, as in capped_log2: y may be 0 where s is not)
                                const float2 zero = make_float2(0.f, 0.f);
                                const float2 z = ffma2(f, make_float2(cap_in, cap_in), zero);
                                const float2 t = tanh_over<kCap == kNearCap>(ffma2(z, z, zero));
                                f = ffma2(ffma2(f, make_float2(lin, lin), zero), t, make_float2(off, off));
                            }
                            if constexpr (decltype(hidden)::value) {
                                const uint32_t see = seen[(16 * n + k) >> 5] >> ((16 * n + k) & 31);
                                f.x = see & 1 ? f.x : -INFINITY;
                                f.y = see & 2 ? f.y : -INFINITY;
                            }
                            y[k] = ex2(f.x), y[k + 1] = ex2(f.y);
                        }
                        if (n > 0) {
                            p[k / 2] = pack_bf16x2(v[k], v[k + 1]);
                            if (k & 2)
                                lb = fadd2(lb, make_float2(v[k], v[k + 1]));
                            else
                                la = fadd2(la, make_float2(v[k], v[k + 1]));
                        }
                    }
                    if (n > 0) tmem_st_x8(s_addr + 8 * (n - 1), p);
                };
                tmem_ld_x16(s_addr, v0);
                tmem_ld_x16(s_addr + 16, v1);
                tmem_ld_wait();
                pin<16>(v0), pin<16>(v1);
                auto hand_over = [&](int part) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[e][part]);
                };
                auto steps = [&](auto cap, auto hidden) {
                    step(cap, hidden, v0, v0, 0);
                    step(cap, hidden, v1, v0, 1);
                    tmem_ld_x16(s_addr + 32, v0);
                    tmem_ld_wait();
                    pin<16>(v0);
                    step(cap, hidden, v0, v1, 2);
                    tmem_ld_x16(s_addr + 48, v1);
                    hand_over(0);
                    tmem_ld_wait();
                    pin<16>(v1);
                    step(cap, hidden, v1, v0, 3);
                    step(cap, hidden, v1, v1, 4);
                };
                // Each case by itself, without a branch from its first load to its last store; the cap
                // by a polynomial where all of the warp's scores are below it, a shorter one where they
                // are below half of it, else by an exponential and a quotient (three prompts of up to 2500
                // tokens, capped, in a window of 512: 80 us; 98 with the longer polynomial alone, 141 with
                // neither).
                auto with_cap = [&](auto cap) {
                    if (masked)
                        steps(cap, std::true_type{});
                    else
                        steps(cap, std::false_type{});
                };
                if constexpr (!CAPPED)
                    with_cap(std::integral_constant<int, kNoCap>{});
                else if (__all_sync(0xFFFFFFFFu, size * cap_in <= 0.5f))
                    with_cap(std::integral_constant<int, kNearCap>{});
                else if (__all_sync(0xFFFFFFFFu, size * cap_in <= 1.f))
                    with_cap(std::integral_constant<int, kBelowCap>{});
                else
                    steps(std::integral_constant<int, kAnyCap>{}, std::true_type{});
                hand_over(1);
                l2 = fadd2(l2, fadd2(la, lb));
            }
            // ------------------------------------------------------- the run's result
            more = enter(run + 1);
            float l = l2.x + l2.y;
            if (any) {
                // the other half of the row's sum, by way of the scores' first columns, now free
                const bool ok = !dead && __all_sync(0xFFFFFFFFu, wait_bounded(&o_full[e], o_ph, &abort_flag, a.test_timeout));
                o_ph ^= 1u;
                tc_fence_after();
                tmem_st_x1(s_addr, __float_as_uint(l));
                tmem_st_wait();
                tc_fence_before();
                dead = bar_or(bar, kHalf, !ok);
                tc_fence_after();
                uint32_t other;
                tmem_ld_x1(s_addr ^ 64u, &other);
                tmem_ld_wait();
                pin<1>(&other);
                // the same order of the two in both threads
                l = cg ? __uint_as_float(other) + l : l + __uint_as_float(other);
                tc_fence_before();
            }
            const bool next_q = more && jb > ja;  // Q's tile is free: nothing of this run reads it any more
            if (next_q) fetch_q();
            float m2 = m;
            if (dead) l = NAN, m2 = 0.f;
            const int tl = r / a.group;
            const volatile Segment &g = runs[run % kRuns];
            const int first = g.first, last = g.last, n_tokens = g.s.rows - g.i0;
            const bool whole = first == last, live = tl < tokens && e * tokens + tl < n_tokens;
            const int hk = g.hk, h = hk * a.group + r - tl * a.group;
            const long long tok0 = g.s.q0 + g.i0, tok = tok0 + e * tokens + tl;
            release(run);
            const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            // whole: a row of the result; else of this CTA's slot, [D / 4][256 rows] of 4 floats, then
            // (maximum, sum) of each row
            uint16_t *const out = a.out.p + tok * a.out.ts + h * a.out.hs + cg * (D / 2);
            float *const slot = a.partials + (size_t)(2 * blockIdx.x + ((int)blockIdx.x == first ? 1 : 0)) * kSlot;
            const int row = e * kTile + r;
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 16) {
                uint32_t o[16];
                if (any && !dead) {
                    tmem_ld_x16(o_addr + c, o);
                    tmem_ld_wait();
                    pin<16>(o);
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float y = any && !dead && l != 0.f ? __uint_as_float(o[k]) * inv : dead ? NAN : 0.f;
                    o[k] = __float_as_uint(y);
                }
                if (live && whole) {
#pragma unroll
                    for (int k = 0; k < 16; k += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int n = 0; n < 4; ++n)
                            w[n] = pack_bf16x2(__uint_as_float(o[k + 2 * n]), __uint_as_float(o[k + 2 * n + 1]));
                        *reinterpret_cast<uint4 *>(out + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else if (live) {
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        __stcg(reinterpret_cast<float4 *>(slot) + (cg * (D / 2) + c + k) / 4 * (2 * kTile) + row,
                               make_float4(__uint_as_float(o[k]), __uint_as_float(o[k + 1]),
                                           __uint_as_float(o[k + 2]), __uint_as_float(o[k + 3])));
                }
                if (c == 0 && next_q) give_q();  // read meanwhile; the next scores need not wait for the rest
            }
            if (live && cg == 0) {
                if (!whole)
                    __stcg(reinterpret_cast<float2 *>(slot + 2 * kTile * D) + row, make_float2(m2, l));
                else if (a.lse)
                    a.lse[tok * a.q_heads + h] = l == 0.f ? -INFINITY : (m2 + log2f(l)) * kLn2;
            }
            if (tid == 0 && !whole && (int)blockIdx.x == first) part = AttnPart{tok0, n_tokens, hk, first, last};
            tc_fence_before();  // the loads of O, before the next run's MMAs
        }
        // the item that begins in this CTA and ends in another, if there is one
        if (mode == kListed && tid == 0) a.parts[blockIdx.x] = part;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the items that several CTAs of a list had a part of, in the order of the CTAs: block (c, y)
// the rows 32 y .. of the item that begins in CTA c. By itself and over the whole GPU: a part is
// up to 128 KB, and joined by the last CTA to finish, six of them took 14 us. The programmatic launch
// hides the launch alone: an attention CTA holds 61440 of its SM's 65536 registers, so a block of this
// kernel starts where one of those has ended.
constexpr int kJoinRows = 32, kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_tc_join_kernel(const AttnArgs a, int tokens) {
    grid_dep_wait();
    grid_dep_launch();
    const AttnPart p = a.parts[blockIdx.x];
    if (p.last < 0) return;
    constexpr int kSlot = tc_slot_words(D), kEach = D / 4 / (kJoinThreads / kJoinRows);
    const int row = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows, e = row / kTile, r = row % kTile;
    const int tl = r / a.group;
    if (tl >= tokens || e * tokens + tl >= p.rows) return;
    auto slot_of = [&](int k) { return a.partials + (size_t)(2 * k + (k == p.first ? 1 : 0)) * kSlot; };
    float M = -INFINITY, L = 0.f;
#pragma unroll 4
    for (int k = p.first; k <= p.last; ++k) M = fmaxf(M, __ldcg(slot_of(k) + 2 * kTile * D + 2 * row));
    const float base = M == -INFINITY ? 0.f : M;
    const int d0 = threadIdx.x / kJoinRows * kEach;
    float4 acc[kEach];
#pragma unroll
    for (int q = 0; q < kEach; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k = p.first; k <= p.last; ++k) {
        const float *sl = slot_of(k);
        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(sl + 2 * kTile * D) + row);
        const float f = ex2(ml.x - base);
        L = fmaf(ml.y, f, L);
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(sl) + (d0 + q) * (2 * kTile) + row);
            acc[q].x = fmaf(v.x, f, acc[q].x), acc[q].y = fmaf(v.y, f, acc[q].y);
            acc[q].z = fmaf(v.z, f, acc[q].z), acc[q].w = fmaf(v.w, f, acc[q].w);
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int h = p.hk * a.group + r - tl * a.group;
    const long long tok = p.row0 + e * tokens + tl;
    uint16_t *out = a.out.p + tok * a.out.ts + h * a.out.hs + 4 * d0;
#pragma unroll
    for (int q = 0; q < kEach; q += 2)
        *reinterpret_cast<uint4 *>(out + 4 * q) =
            make_uint4(pack_bf16x2(acc[q].x * inv, acc[q].y * inv), pack_bf16x2(acc[q].z * inv, acc[q].w * inv),
                       pack_bf16x2(acc[q + 1].x * inv, acc[q + 1].y * inv),
                       pack_bf16x2(acc[q + 1].z * inv, acc[q + 1].w * inv));
    if (d0 == 0 && a.lse) a.lse[tok * a.q_heads + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <int D, int CAP>
cudaError_t launch_d(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t stream) {
    static std::atomic<uint64_t> attr_done{0};
    DeviceInfo di;
    cudaError_t err = device_info(&di);
    if (err != cudaSuccess) return err;
    int dev = 0;
    err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 64 || !(attr_done.load(std::memory_order_acquire) & bit)) {
        // the warps' register shares wait for one another if the launch brings fewer
        cudaFuncAttributes fa;
        err = cudaFuncGetAttributes(&fa, attn_tc_kernel<D, CAP>);
        if (err != cudaSuccess) return err;
        if (fa.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
        err = cudaFuncSetAttribute(attn_tc_kernel<D, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   TcShape<D>::kSmem);
        if (err != cudaSuccess) return err;
        if (dev < 64) attr_done.fetch_or(bit, std::memory_order_acq_rel);
    }
    // most pairs of halves that the batch can have (its lengths are device memory)
    const int tokens = kTile / a.group;
    const long long by_rows = a.m.total_q / (2 * tokens) + (long long)a.m.batch;
    const long long by_seq = (long long)a.m.batch * ((a.m.max_q + 2 * tokens - 1) / (2 * tokens));
    const long long pairs = by_rows < by_seq ? by_rows : by_seq;
    const int sms = di.sm_count < kAttnMaxCtas ? di.sm_count : kAttnMaxCtas;
    // Few sequences: one CTA an SM, and a list by which the tiles come out even where the pairs are
    // few too. Many: an item a CTA, in the order in which the hardware finds room.
    const int mode = a.m.batch > kMaxListed ? kOneItem : pairs > kMaxListed ? kPersistent : kListed;
    const long long tiles = (a.m.capacity + kTile - 1) / kTile;
    long long grid = pairs * a.kv_heads;
    if (mode == kListed) grid *= tiles > 0 ? tiles : 1;
    if (mode != kOneItem && grid > sms) grid = sms;
    // Nothing is read before the wait, so programmatic launches are always right: 35 tokens in each of 3
    // sequences 10.2 us a call, 12.3 without. Not of long calls by themselves: their CTAs then find
    // their SMs in the order in which these become free (three capped prompts 84.6 us, 82.0 without).
    const bool programmatic = mode != kPersistent || (launch_flags() & FD_LAUNCH_PDL) != 0;
    err = launch_kernel_as(programmatic, attn_tc_kernel<D, CAP>, dim3((unsigned)grid), dim3(kThreads),
                           (size_t)TcShape<D>::kSmem, stream, 1, mk, mv, a, tokens, mode);
    if (err != cudaSuccess) return err;
    err = cudaGetLastError();
    if (err != cudaSuccess || mode != kListed || grid < 2) return err;
    const int rows = (int)std::min((long long)a.m.max_q * a.group, 2ll * kTile);
    // rows of a pair are spread over its two halves
    const int blocks = rows > tokens * a.group ? 2 * kTile / kJoinRows : (rows + kJoinRows - 1) / kJoinRows;
    err = launch_kernel_as(true, attn_tc_join_kernel<D>, dim3((unsigned)grid, (unsigned)blocks), dim3(kJoinThreads), 0,
                           stream, 1, a, tokens);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                           cudaStream_t stream) {
    auto launch = [&](auto cap) {
        constexpr int kCap = decltype(cap)::value;
        return a.head_dim == 128 ? launch_d<128, kCap>(a, mk, mv, stream) : launch_d<64, kCap>(a, mk, mv, stream);
    };
    if (a.softcap > kLargeCap) return launch(std::integral_constant<int, kLargeCaps>{});
    if (a.softcap > 0.f) return launch(std::integral_constant<int, kUsualCaps>{});
    return launch(std::integral_constant<int, kUncapped>{});
}

FD_DEFINE_STATUS_ACCESSOR(status_attn_tc)

}  // namespace fd
