// fd_attn_rows.cu - attention of few query rows per key head over a paged cache: decoding, and
// short chunks.
//
// For a (sequence, key head) the rows are its new tokens times the query heads that share the
// key head; up to 16 of them are one pass over the keys. Bound by memory: with 16 rows there are
// 16 multiply-adds per byte of the cache, far below what the tensor cores do, so what matters is
// that every SM streams pages all the time.
//
//   * The keys of all (sequence, block of 16 rows, key head) items, in tiles of 64, form one long
//     list, and CTA c of G takes tiles [T c / G, T (c + 1) / G) of it: every SM gets the same
//     number of tiles whatever the lengths of the sequences, with nothing planned on the host (the
//     lengths are device memory, a captured graph sees new ones). An item that several CTAs share
//     is joined by the CTA that finishes last: each writes its rows' (maximum, sum, accumulator)
//     to its own slot, takes a ticket, and the holder of the last ticket adds the slots in the
//     order of the CTAs, so results do not depend on who is last.
//   * One producer warp copies tiles (tensor-map copies of one page's 64-element columns each, all
//     lanes issuing, page numbers read one tile ahead) into a ring of shared memory; four consumer
//     warps take 16 keys of each tile. Each keeps its own running maximum, sum and fp32
//     accumulator in registers (online softmax, one pass over the data) and they meet only at
//     the end of an item, in shared memory.
//   * Scores are Q K^T with the rows as the M = 16 of mma.sync m16n8k16, so that the
//     probabilities come out in the layout that P V takes as its A operand; rounded to bf16 there
//     (V is bf16, both operands have one type), each by 2^-8 relative at most, while the sum is
//     that of the unrounded ones. These legacy instructions are used on purpose: 128 of them a
//     tile hide under its copy, and tcgen05 would pad the rows to 128.
//   * Values outside the visible range are cleared in the operand registers: 0 x NaN would reach
//     the sum otherwise, and pages hold anything past the last token.
#include <atomic>

#include "fd_attn.h"
#include "fd_tc.cuh"

namespace fd {
namespace {

constexpr int kWarps = 4;                       // consumers
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;

template <int D>
struct RowsShape {
    static constexpr int kHalves = D / 64;             // 128-byte columns of a row
    static constexpr int kTensor = kRowsTile * D * 2;  // bytes of a tile's keys (or values)
    static constexpr int kStage = 2 * kTensor;
    static constexpr int kStages = D == 128 ? 5 : 10;  // 160 KB in flight
    static constexpr int kPitch = D + 8;               // floats; conflict-free accumulator rows
    static constexpr int kMergeBytes = kWarps * kRowsM * kPitch * 4;
    static constexpr int kMlBytes = kWarps * kRowsM * 8;
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
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One run of tiles of one item.
struct Segment {
    SeqInfo s;
    int b, item;        // item: block of rows * kv_heads + key head
    int rb, hk;
    int i0, i1;         // first and last new token of the block's rows
    int rows;           // rows of the block
    int tile0;          // number of the first tile of the item's keys
    int from, to;       // the segment's tiles, counted in the item
    int nt;             // tiles of the item
    long long item0;    // the item's first tile in the list
};

// Tiles that the keys of sequence s take (at least one, so that every row is written), and the
// first of them. The same for all of the sequence's items.
__device__ __forceinline__ int seq_tiles(const SeqInfo &s, const AttnArgs &a, int *first) {
    *first = 0;
    if (s.rows <= 0) return 0;
    const int lo = key_lo(s, 0, a.window), hi = key_hi(s, s.rows - 1, a.causal);
    if (hi <= lo) return 1;
    *first = lo / kRowsTile;
    return (hi + kRowsTile - 1) / kRowsTile - *first;
}

// The segment that begins at tile x of the list and ends at `end` or with its item; `b` is a
// sequence at or before x's.
__device__ __forceinline__ Segment segment_at(const AttnArgs &a, const unsigned *prefix, int items,
                                              long long x, long long end, int b) {
    Segment g;
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
    g.b = b;
    g.s = load_seq(a.m, b);
    g.nt = (int)(prefix[b + 1] - prefix[b]);
    const long long in_seq = x - (long long)prefix[b] * items;
    g.item = (int)(in_seq / g.nt);
    g.from = (int)(in_seq - (long long)g.item * g.nt);
    g.item0 = x - g.from;
    g.to = (int)min((long long)g.nt, end - g.item0);
    g.rb = g.item / a.kv_heads;
    g.hk = g.item - g.rb * a.kv_heads;
    seq_tiles(g.s, a, &g.tile0);
    const int all = g.s.rows * a.group;
    g.rows = min(kRowsM, all - g.rb * kRowsM);  // <= 0: no such block in this sequence
    g.i0 = g.rb * kRowsM / a.group;
    g.i1 = min(g.s.rows, (g.rb * kRowsM + kRowsM - 1) / a.group + 1) - 1;
    return g;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const AttnArgs a, int row_blocks) {
    using S = RowsShape<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages];
    __shared__ int abort_flag;
    __shared__ int last_s;
    __shared__ unsigned warp_sum[kThreads / 32];
    unsigned char *smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
    float *merge = reinterpret_cast<float *>(smem + S::kStages * S::kStage);
    float2 *ml = reinterpret_cast<float2 *>(smem + S::kStages * S::kStage + S::kMergeBytes);
    unsigned *prefix = reinterpret_cast<unsigned *>(smem + S::kStages * S::kStage + S::kMergeBytes + S::kMlBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWarps);
        }
        abort_flag = 0;
        fence_mbar_init();
    }
    grid_dep_wait();
    grid_dep_launch();

    // The list: prefix[b] = tiles of one item of each sequence before b.
    {
        const int per = (a.m.batch + kThreads - 1) / kThreads;
        const int b0 = min(tid * per, a.m.batch), b1 = min(b0 + per, a.m.batch);
        unsigned sum = 0;
        int first;
        for (int b = b0; b < b1; ++b) sum += (unsigned)seq_tiles(load_seq(a.m, b), a, &first);
        unsigned inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += up;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        unsigned at = inc - sum;
        for (int w = 0; w < warp; ++w) at += warp_sum[w];
        for (int b = b0; b < b1; ++b) {
            prefix[b] = at;
            at += (unsigned)seq_tiles(load_seq(a.m, b), a, &first);
        }
        if (tid == kThreads - 1) prefix[a.m.batch] = at;
    }
    __syncthreads();
    const int items = row_blocks * a.kv_heads;
    const long long total = (long long)prefix[a.m.batch] * items;
    // no more CTAs than tiles: each of the CTAs between an item's first and last has a part of it
    const int G = (int)min((long long)gridDim.x, total), c = blockIdx.x;
    if (c >= G) return;
    const long long begin = total * c / G, end = total * (c + 1) / G;

    if (warp == kWarps) {
        // ------------------------------------------------------------------ producer
        const int box = min(1 << a.m.page_shift, kRowsTile);  // tokens of one copy
        const int boxes = kRowsTile / box;
        const int per_tensor = boxes * S::kHalves;
        const int ops = 2 * per_tensor;  // at most 16
        const bool is_v = lane >= per_tensor;
        const int r = lane - (is_v ? per_tensor : 0);
        const int my_box = r / S::kHalves, my_half = r - my_box * S::kHalves;
        const uint32_t dst0 = (is_v ? S::kTensor : 0) + my_half * (kRowsTile * 128) + my_box * box * 128;
        const CUtensorMap *map = is_v ? &map_v : &map_k;
        const MapOrder ord = is_v ? a.ov : a.ok;
        const uint64_t policy = policy_evict_first();
        Segment g = segment_at(a, prefix, items, begin, end, 0);
        int tile = g.from;
        long long x = begin;
        // this lane's page for the tile at hand; num_pages (reads as zeros) where none is needed
        auto page_of = [&](const Segment &sg, int t) {
            const int tok = (sg.tile0 + t) * kRowsTile + my_box * box;
            const int lo = key_lo(sg.s, 0, a.window), hi = key_hi(sg.s, sg.s.rows - 1, a.causal);
            int page = a.m.num_pages;
            if (lane < ops && tok < hi && tok + box > lo) {
                const int id = a.m.table[(long long)sg.b * a.m.table_stride + (tok >> a.m.page_shift)];
                if (id >= 0 && id < a.m.num_pages)
                    page = id;
                else
                    atomicOr(&g_wait_status, (unsigned)FD_DEVICE_STATUS_BAD_PAGE);
            }
            return page;
        };
        int page = page_of(g, tile);
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        long long issued = 0;
        while (true) {
            const int tok = (g.tile0 + tile) * kRowsTile + my_box * box;
            const int off = tok & ((1 << a.m.page_shift) - 1);
            const int hk = g.hk, this_page = page;
            // read the next tile's page numbers before this one waits for room
            ++x;
            const bool more = x < end;
            if (more) {
                if (++tile == g.to) {
                    g = segment_at(a, prefix, items, x, end, g.b);
                    tile = g.from;
                }
                page = page_of(g, tile);
            }
            ok = mbar_wait_bounded(&empty[stage], phase ^ 1u, &abort_flag);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[stage], S::kStage);
            __syncwarp();
            if (lane < ops) {
                const int y1 = ord.tok == 1 ? off : ord.head == 1 ? hk : this_page;
                const int y2 = ord.tok == 2 ? off : ord.head == 2 ? hk : this_page;
                const int y3 = ord.tok == 3 ? off : ord.head == 3 ? hk : this_page;
                tma_load_4d(smem + stage * S::kStage + dst0, map, my_half * 64, y1, y2, y3, &full[stage], policy);
            }
            ++issued;
            if (++stage == S::kStages) stage = 0, phase ^= 1u;
            if (!more) break;
        }
        if (!ok && lane == 0) {
            // a consumer gave up: wait (bounded) for the copies in flight before the CTA ends
            const long long n = issued < S::kStages ? issued : S::kStages;
            for (long long i = issued - n; i < issued; ++i) {
                const long long t0 = clock64();
                while (!mbar_try_parity(&full[i % S::kStages], (uint32_t)((i / S::kStages) & 1)) &&
                       clock64() - t0 < kWaitLimitCycles) {
                }
            }
        }
        return;
    }

    // ---------------------------------------------------------------------- consumers
    const int g8 = lane >> 2, c2 = (lane & 3) * 2;  // accumulator row and column of this lane
    const float to_log2 = a.scale * kLog2e;
    const float cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f, cap_out = a.softcap * kLog2e;
    // ldmatrix rows: keys (lane & 7) + 8 * (lane >> 4) of the warp's 16, chunk bit (lane >> 3) & 1
    const int k_row = warp * 16 + (lane & 7) + ((lane >> 4) << 3), k_bit = (lane >> 3) & 1;
    // values, transposed: keys (lane & 15), chunk bit lane >> 4
    const int v_row = warp * 16 + (lane & 15), v_bit = lane >> 4;
    const uint32_t ring = smem_u32(smem);
    int stage = 0;
    uint32_t phase = 0;
    bool dead = false;
    int b_at = 0;
    for (long long x = begin; x < end;) {
        const Segment g = segment_at(a, prefix, items, x, end, b_at);
        b_at = g.b;
        x = g.item0 + g.to;
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

        for (int t = g.from; t < g.to; ++t) {
            if (!dead) dead = !__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[stage], phase, &abort_flag));
            if (dead) break;
            const uint32_t kb = ring + stage * S::kStage, vb = kb + S::kTensor;
            const int tok = (g.tile0 + t) * kRowsTile + warp * 16;  // the warp's first key
            // a warp's 16 keys outside every row's range (the ends of a window) add nothing
            if (g.rows > 0 && tok < any_hi && tok + 16 > any_lo) {
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    uint32_t kf[4];
                    const int chunk = (ks & 3) * 2 + k_bit;
                    ldsm_x4(kf, kb + (ks >> 2) * (kRowsTile * 128) + k_row * 128 + ((chunk ^ (k_row & 7)) << 4));
                    mma_bf16(s[0], qf[ks], kf[0], kf[1]);
                    mma_bf16(s[1], qf[ks], kf[2], kf[3]);
                }
                const bool inside = tok >= in_lo && tok + 16 <= in_hi;
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v = s[n][i];
                        if (a.softcap > 0.f)  // c tanh(y) = c (1 - 2 / (e^(2 y) + 1))
                            v = cap_out * (1.f - __fdividef(2.f, ex2(v * cap_in * (2.f * kLog2e)) + 1.f));
                        else
                            v *= to_log2;
                        const int key = tok + n * 8 + c2 + (i & 1);
                        if (!inside && (key < lo[i >> 1] || key >= hi[i >> 1])) v = -INFINITY;
                        s[n][i] = v;
                        mx[i >> 1] = fmaxf(mx[i >> 1], v);
                    }
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
                uint32_t p[4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float p0 = ex2(s[n][0] - m0), p1 = ex2(s[n][1] - m0);
                    const float p2 = ex2(s[n][2] - m1), p3 = ex2(s[n][3] - m1);
                    l[0] += p0 + p1, l[1] += p2 + p3;
                    p[2 * n] = pack_bf16x2(p0, p1);
                    p[2 * n + 1] = pack_bf16x2(p2, p3);
                }
                // values of this lane's operand registers: keys c2, c2 + 1 and c2 + 8, c2 + 9
                uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
                if (!inside) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = tok + 8 * e + c2;
                        keep[e] = (key >= any_lo && key < any_hi ? 0xFFFFu : 0u) |
                                  (key + 1 >= any_lo && key + 1 < any_hi ? 0xFFFF0000u : 0u);
                    }
                }
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t vf[4];
                    const int chunk = (n & 3) * 2 + v_bit;
                    ldsm_x4_t(vf, vb + (n >> 2) * (kRowsTile * 128) + v_row * 128 + ((chunk ^ (v_row & 7)) << 4));
                    mma_bf16(o[2 * n], p, vf[0] & keep[0], vf[1] & keep[1]);
                    mma_bf16(o[2 * n + 1], p, vf[2] & keep[0], vf[3] & keep[1]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
            if (++stage == S::kStages) stage = 0, phase ^= 1u;
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
        named_bar_sync(1, kConsumers);
        // CTAs that share the item, in the order of their tiles
        const int first = (int)(((g.item0 + 1) * G - 1) / total);
        const int last = (int)(((g.item0 + g.nt) * G - 1) / total);
        const bool whole = first == last;
        float *slots = a.partials;
        constexpr int kSlot = rows_slot_words(D);
        float *slot = slots + (size_t)(2 * c + (c == first ? 1 : 0)) * kSlot;
        const int n4 = max(g.rows, 0) * (D / 4);
        auto finish = [&](int row, int d4, float M, float L, float4 acc) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const int all = g.rb * kRowsM + row, i = all / a.group, h = g.hk * a.group + all - i * a.group;
            const long long tok = g.s.q0 + i;
            uint2 w = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            *reinterpret_cast<uint2 *>(a.out.p + tok * a.out.ts + h * a.out.hs + 4 * d4) = w;
            if (d4 == 0 && a.lse) a.lse[tok * a.q_heads + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
        };
        for (int idx = tid; idx < n4; idx += kConsumers) {
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
                __stcg(reinterpret_cast<float4 *>(slot + row * D + 4 * d4), acc);
                if (d4 == 0) __stcg(reinterpret_cast<float2 *>(slot + kRowsM * D + 2 * row), make_float2(M, L));
            }
        }
        if (!whole) __threadfence();
        named_bar_sync(1, kConsumers);  // also: the buffers are free for the next segment
        if (whole) continue;
        if (tid == 0) {
            const unsigned ticket = atomicAdd(&a.counters[first], 1u);
            last_s = ticket == (unsigned)(last - first);
            if (last_s) a.counters[first] = 0;
            __threadfence();
        }
        named_bar_sync(1, kConsumers);
        if (last_s) {
            for (int idx = tid; idx < n4; idx += kConsumers) {
                const int row = idx / (D / 4), d4 = idx - row * (D / 4);
                float M = -INFINITY, L = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int k = first; k <= last; ++k) {
                    const float *sl = slots + (size_t)(2 * k + (k == first ? 1 : 0)) * kSlot;
                    const float2 s = __ldcg(reinterpret_cast<const float2 *>(sl + kRowsM * D + 2 * row));
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(sl + row * D + 4 * d4));
                    const float top = fmaxf(M, s.x), base = top == -INFINITY ? 0.f : top;
                    const float f0 = ex2(M - base), f1 = ex2(s.x - base);
                    M = top;
                    L = L * f0 + s.y * f1;
                    acc.x = acc.x * f0 + v.x * f1, acc.y = acc.y * f0 + v.y * f1;
                    acc.z = acc.z * f0 + v.z * f1, acc.w = acc.w * f0 + v.w * f1;
                }
                finish(row, d4, M, L, acc);
            }
        }
        named_bar_sync(1, kConsumers);  // last_s is read before the next segment writes it
    }
}

template <int D>
cudaError_t launch_d(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t stream) {
    using S = RowsShape<D>;
    static std::atomic<uint64_t> attr_done{0};
    DeviceInfo di;
    cudaError_t err = device_info(&di);
    if (err != cudaSuccess) return err;
    int dev = 0;
    err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    constexpr size_t kFixed = 1024 + S::kStages * S::kStage + S::kMergeBytes + S::kMlBytes;
    static_assert(kFixed + 4 * (FD_MAX_BATCH + 1) + 1024 <= 227 * 1024, "shared memory");
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 64 || !(attr_done.load(std::memory_order_acquire) & bit)) {
        err = cudaFuncSetAttribute(attn_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)(kFixed + 4 * (FD_MAX_BATCH + 1)));
        if (err != cudaSuccess) return err;
        if (dev < 64) attr_done.fetch_or(bit, std::memory_order_acq_rel);
    }
    const long long row_blocks = ((long long)a.m.max_q * a.group + kRowsM - 1) / kRowsM;
    const long long most = (long long)a.m.batch * row_blocks * a.kv_heads * ((a.m.capacity + kRowsTile - 1) / kRowsTile);
    long long grid = di.sm_count < kAttnMaxCtas ? di.sm_count : kAttnMaxCtas;
    if (grid > most) grid = most;
    err = launch_kernel(attn_rows_kernel<D>, dim3((unsigned)grid), dim3(kThreads),
                        kFixed + 4 * (size_t)(a.m.batch + 1), stream, 1, mk, mv, a, (int)row_blocks);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                             cudaStream_t stream) {
    return a.head_dim == 128 ? launch_d<128>(a, mk, mv, stream) : launch_d<64>(a, mk, mv, stream);
}

FD_DEFINE_STATUS_ACCESSOR(status_attn_rows)

}  // namespace fd
