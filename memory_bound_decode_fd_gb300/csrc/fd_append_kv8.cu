// fd_append_kv8.cu - a batch's new tokens rotated, their keys and values written to a paged cache in 8 bits.
//
//   e(block, head)  = max(e before, smallest e >= -100 with max |x| <= M 2^e over the block's new tokens)
//   code            = round(x 2^-e);  of the block's earlier tokens, where e grew: round(code 2^(e before - e))
//
// The scale of a block of 16 tokens and head is needed before its first code can be written, so the unit
// of work is a block's new tokens (up to 16) of a head: a warp holds them in registers, as 32-bit values
// that are rounded once, takes their maximum and writes them; nothing is read or written twice but the
// codes of a block that an earlier call began and whose exponent grows. No two warps share a scale, so there are no atomics.
// The scales are powers of two, so that lowering the earlier codes is exact but for what falls below
// their last place, and what attention reads is exact in bf16.
//
// Bound by memory for prompts (8195 tokens of 32 heads on 8 of 128: 36 us, 3.9 TB/s, 58 % of the copy; the queries, three
// quarters of the bytes, are in bf16 as they come) and by latency for single tokens (one: 4.5 to 5 us, 64: 5.5, the
// launch and three dependent loads). In the prompts every unit waits for its block's angles and its rows, and the
// rotation is done twice, for the maximum and for the codes: rows held in 32 bits between the two took 42 us, with
// twice the registers and half the warps. Angles are those of fd_rope, their cosines and sines in 32 bits (off by a few
// 2^-24): an element next to the border of two codes may so take either, and a maximum next to that of two scales too. A CTA takes the blocks that begin in a
// run of `run` tokens (a block begins at a sequence's first new token or at a multiple of 16): its threads look
// up all tokens of the run, make the cosines and sines of a block's tokens in shared memory, then its
// warps take heads of keys and values, and its threads units of 16 elements of the queries.
#include <atomic>

#include "fd_attn.h"
#include "fd_kv8.cuh"
#include "fd_rope.cuh"

namespace fd {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMostRun = 16;  // tokens of a run
constexpr int kUnit = 16;     // elements that a lane handles at a time
constexpr int kAtOnce = 4;    // units of queries that a thread has on their way

__device__ unsigned int g_page_status;

// The new tokens of a block: the first of them, how many, the first one's number in the cache, and the
// page (-1: they have no place).
struct Tokens {
    int t, n, at, page;
};

// Half (8 elements each) of a unit, rotated or as it is, in 32 bits. f: the unit's cosines and sines,
// `pitch` apart (fd_rope.cu).
__device__ __forceinline__ void turn_unit(const uint4 &x, const uint4 &y, bool rotate, bool halves, const float4 *f, int pitch,
                                          float (&o)[kUnit]) {
    if (!rotate) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o[2 * k] = bf16lo(word(x, k)), o[2 * k + 1] = bf16hi(word(x, k));
            o[8 + 2 * k] = bf16lo(word(y, k)), o[9 + 2 * k] = bf16hi(word(y, k));
        }
    } else if (halves) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 g = f[k * pitch];
            const float2 co = make_float2(g.x, g.y), si = make_float2(g.z, g.w), no = make_float2(-g.z, -g.w);
            const float2 p = make_float2(bf16lo(word(x, k)), bf16hi(word(x, k)));
            const float2 q = make_float2(bf16lo(word(y, k)), bf16hi(word(y, k)));
            const float2 zero = make_float2(0.f, 0.f);
            const float2 xr = ffma2(p, co, ffma2(q, no, zero)), yr = ffma2(p, si, ffma2(q, co, zero));
            o[2 * k] = xr.x, o[2 * k + 1] = xr.y, o[8 + 2 * k] = yr.x, o[9 + 2 * k] = yr.y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float4 g = f[(k >> 1) * pitch];
            const uint32_t p = k < 4 ? word(x, k) : word(y, k - 4);
            const float a = bf16lo(p), b = bf16hi(p), c = k & 1 ? g.y : g.x, s = k & 1 ? g.w : g.z;
            o[2 * k] = a * c - b * s, o[2 * k + 1] = a * s + b * c;
        }
    }
}

// VEC: rot_dim is a multiple of 16 (a unit of 16 elements is rotated or not, and each of its halves
// lies on 16 bytes); otherwise pair by pair. q_magic: ceil(2^32 / units of a token's queries), exact for the at most
// 2^17 units of a block with at most 2^13 a token.
template <int D, int TYPE, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) append_kv8_kernel(const RopeArgs a, const Kv8Cache c, int run, unsigned q_magic) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int half = a.rot_dim >> 1, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned long long *const step = reinterpret_cast<unsigned long long *>(smem);  // [half] of a turn
    float *const cs = reinterpret_cast<float *>(step + half + (half & 1));          // [16][rot_dim], as in fd_rope.cu
    __shared__ Tokens begun[kMostRun];
    __shared__ int seq_s, n_begun;
    const int s0 = blockIdx.x * run, n_run = min(run, a.tokens - s0);
    grid_dep_wait();
    grid_dep_launch();

    // the sequence of the run's first token: how many sequences end at or before it
    if (tid == 0) seq_s = 0;
    __syncthreads();
    int before = 0;
    for (int b = tid; b < a.m.batch; b += kThreads) before += a.m.q_start[b + 1] <= s0;
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    if (lane == 0 && before) atomicAdd(&seq_s, before);
    for (int i = tid; i < half; i += kThreads) step[i] = turns_64(a.inv_freq[i]);
    __syncthreads();
    if (warp == 0) {
        Tokens k{0, 0, 0, -1};
        if (lane < n_run) {
            const int t = s0 + lane;
            int b = seq_s;
            while (b < a.m.batch && a.m.q_start[b + 1] <= t) ++b;
            if (b < a.m.batch && a.m.q_start[b] <= t) {
                const int len = a.m.kv_len[b], kv = min(max(len, 0), a.m.capacity);
                const int end = a.m.q_start[b + 1], at = kv - (end - t), off = at & (kKv8Block - 1);
                if (off == 0 || t == max(a.m.q_start[b], 0)) {
                    k = Tokens{t, min(min(end, a.tokens) - t, kKv8Block - off), at, -1};
                    if (len > a.m.capacity) {  // its tokens would go over others'
                        atomicOr(&g_page_status, (unsigned)FD_DEVICE_STATUS_BAD_PAGE);
                    } else if (at >= 0) {
                        const int page = a.m.table[(long long)b * a.m.table_stride + (at >> a.m.page_shift)];
                        if (page >= 0 && page < a.m.num_pages)
                            k.page = page;
                        else
                            atomicOr(&g_page_status, (unsigned)FD_DEVICE_STATUS_BAD_PAGE);
                    }
                }
            }
        }
        const unsigned some = __ballot_sync(0xFFFFFFFFu, k.n > 0);
        if (k.n > 0) begun[__popc(some & ((1u << lane) - 1))] = k;
        if (lane == 0) n_begun = __popc(some);
    }
    __syncthreads();

    // this CTA's share of the heads of keys and values, and of the queries' units
    const int parts = gridDim.y, part = blockIdx.y;
    const int kv0 = 2 * a.k_heads * part / parts, kv1 = 2 * a.k_heads * (part + 1) / parts;
    for (int u = 0; u < n_begun; ++u) {
        const Tokens k = begun[u];
        if (u > 0) __syncthreads();  // the angles of the last block are read
        for (int i = tid; i < k.n * half; i += kThreads) {
            const int t = i / half, p = i - t * half;
            const int pos = a.positions ? a.positions[k.t + t] : k.at + t;
            const long long frac = (long long)((unsigned long long)(long long)pos * step[p]);
            float sn, co;
            sincospif((float)frac * 1.0842021724855044e-19f, &sn, &co);  // 2^-63: half turns
            float *const to = cs + t * a.rot_dim + (VEC ? (((p >> 1 & 3) * (half >> 3) + (p >> 3)) << 2) + (p & 1) : p);
            to[0] = co * a.scale;
            to[VEC ? 2 : half] = sn * a.scale;
        }
        __syncthreads();

        // ------------------------------------------------------------ keys and values
        if (k.page >= 0) {
            const int off = k.at & ((1 << a.m.page_shift) - 1), first = off & (kKv8Block - 1);
            for (int j = kv0 + warp; j < kv1; j += kWarps) {
                const bool keys = j < a.k_heads;
                const int h = keys ? j : j - a.k_heads;
                const HeadsView in = keys ? a.k : a.v;
                const uint16_t *const from = in.p + k.t * in.ts + h * in.hs;
                const Kv8Plane to = keys ? c.k : c.v;
                uint8_t *const codes = to.codes + k.page * to.page + off * to.token + h * to.head;
                uint8_t *const scale = to.scale + k.page * to.scale_page + (off / kKv8Block) * to.scale_block + h * to.scale_head;
                const int e_old = first ? (int)*scale - 127 : kKv8Lowest;
                // Lane l: VEC: 16 elements (unit l % (D / 16)) of every (512 / D)th token; else 1 or 2
                // pairs of each.
                constexpr int kLanes = VEC ? D / kUnit : 32, kStep = 32 / kLanes;
                constexpr int kPasses = kKv8Block / kStep, kEach = VEC ? kUnit : D / 32;
                const int unit = lane % kLanes, row = lane / kLanes;
                // VEC: the rows as they are read, rotated once for the maximum and once more for the codes: in 32 bits
                // they would take twice the registers, and half as many warps find room.
                uint4 lo[VEC ? kPasses : 1], hi[VEC ? kPasses : 1];
                float x[VEC ? 1 : kPasses][kEach];
                const bool rotate = keys && unit * kUnit < a.rot_dim, halves = rotate && !a.interleaved;
                const int j0 = halves ? unit * 8 : unit * kUnit, j1 = halves ? unit * 8 + half : unit * kUnit + 8;
                // elements of pair p
                auto pair = [&](int p, int *e0, int *e1) {
                    const bool apart = keys && p < half && !a.interleaved;
                    *e0 = apart ? p : 2 * p, *e1 = apart ? p + half : 2 * p + 1;
                };
                auto turned = [&](int i, float (&y)[kUnit]) {
                    turn_unit(lo[i], hi[i], rotate, halves,
                              reinterpret_cast<const float4 *>(cs + min(i * kStep + row, k.n - 1) * a.rot_dim) + unit, half >> 3, y);
                };
                if constexpr (VEC) {
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
                        lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
                        if (i * kStep + row < k.n) {
                            lo[i] = __ldcs(reinterpret_cast<const uint4 *>(from + (i * kStep + row) * in.ts + j0));
                            hi[i] = __ldcs(reinterpret_cast<const uint4 *>(from + (i * kStep + row) * in.ts + j1));
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
#pragma unroll
                        for (int r = 0; r < kEach / 2; ++r) {
                            x[i][2 * r] = x[i][2 * r + 1] = 0.f;
                            if (i >= k.n) continue;
                            const int p = lane + 32 * r;
                            int e0, e1;
                            pair(p, &e0, &e1);
                            const float v0 = bf16lo(from[i * in.ts + e0]), v1 = bf16lo(from[i * in.ts + e1]);
                            const bool turn = keys && p < half;
                            const float co = turn ? cs[i * a.rot_dim + p] : 1.f, sn = turn ? cs[i * a.rot_dim + half + p] : 0.f;
                            x[i][2 * r] = turn ? v0 * co - v1 * sn : v0;
                            x[i][2 * r + 1] = turn ? v0 * sn + v1 * co : v1;
                        }
                    }
                }
                auto largest = [&](auto size) {  // of the elements that count, as bits
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
                        if (i * kStep >= k.n) continue;  // (rows behind the last token within a pass are zeros)
                        if constexpr (VEC) {
                            float y[kUnit];
                            turned(i, y);
#pragma unroll
                            for (int n = 0; n < kUnit; ++n) m = fmaxf(m, size(y[n]));
                        } else {
#pragma unroll
                            for (int n = 0; n < kEach; ++n) m = fmaxf(m, size(x[i][n]));
                        }
                    }
                    return __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
                };
                uint32_t top = largest([](float y) { return fabsf(y); });  // (a NaN is no maximum)
                if (top >= 0x7F800000u) top = largest([](float y) { return fabsf(y) < INFINITY ? fabsf(y) : 0.f; });
                const int e = max(kv8_exponent<TYPE>(top), e_old);
                if (first && e > e_old) {
                    // the block's earlier tokens, 16 codes a lane
                    constexpr int kAcross = D / 16;
                    for (int i = lane / kAcross; i < first; i += 32 / kAcross) {
                        uint4 *const at = reinterpret_cast<uint4 *>(codes + (i - first) * to.token + lane % kAcross * 16);
                        uint4 w = *at;
                        w.x = kv8_lower<TYPE>(w.x, e - e_old), w.y = kv8_lower<TYPE>(w.y, e - e_old);
                        w.z = kv8_lower<TYPE>(w.z, e - e_old), w.w = kv8_lower<TYPE>(w.w, e - e_old);
                        *at = w;
                    }
                }
                const float f = e > 126 ? 0.f : two_to(-e);
                if constexpr (VEC) {
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
                        if (i * kStep >= k.n) continue;
                        float y[kUnit];
                        turned(i, y);
                        if (i * kStep + row >= k.n) continue;
                        uint32_t w[4];
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const float2 u = __fmul2_rn(make_float2(y[4 * n], y[4 * n + 1]), make_float2(f, f));
                            const float2 v = __fmul2_rn(make_float2(y[4 * n + 2], y[4 * n + 3]), make_float2(f, f));
                            w[n] = kv8_encode<TYPE>(u.x, u.y, v.x, v.y);
                        }
                        uint8_t *const at = codes + (i * kStep + row) * to.token;
                        *reinterpret_cast<uint2 *>(at + j0) = make_uint2(w[0], w[1]);
                        *reinterpret_cast<uint2 *>(at + j1) = make_uint2(w[2], w[3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
                        if (i >= k.n) continue;
#pragma unroll
                        for (int r = 0; r < kEach / 2; ++r) {
                            int e0, e1;
                            pair(lane + 32 * r, &e0, &e1);
                            const uint32_t w = kv8_encode<TYPE>(x[i][2 * r] * f, x[i][2 * r + 1] * f, 0.f, 0.f);
                            codes[i * to.token + e0] = (uint8_t)w;
                            codes[i * to.token + e1] = (uint8_t)(w >> 8);
                        }
                    }
                }
                __syncwarp();  // every lane has read the earlier scale
                if (lane == 0) *scale = (uint8_t)(e + 127);
            }
        }

        // --------------------------------------------------------------------- queries
        if constexpr (VEC) {
            constexpr int kPerHead = D / kUnit;
            const int all = a.q_heads * kPerHead;
            const int i1 = k.n * all * (part + 1) / parts;
            struct {
                uint4 x, y;
            } unit[kAtOnce];
            auto place = [&](int i, int *t, int *h, int *e, int *j0, int *j1) {
                *t = all == 1 ? i : (int)__umulhi((unsigned)i, q_magic);
                const int q = i - *t * all;
                *h = q / kPerHead, *e = (q % kPerHead) * kUnit;
                const bool halves = *e < a.rot_dim && !a.interleaved;
                *j0 = halves ? *e >> 1 : *e, *j1 = halves ? (*e >> 1) + half : *e + 8;
            };
            for (int i0 = k.n * all * part / parts + tid; i0 < i1; i0 += kAtOnce * kThreads) {
#pragma unroll
                for (int m = 0; m < kAtOnce; ++m) {
                    const int i = i0 + m * kThreads;
                    if (i >= i1) break;
                    int t, h, e, j0, j1;
                    place(i, &t, &h, &e, &j0, &j1);
                    const uint16_t *const from = a.q.p + (k.t + t) * a.q.ts + h * a.q.hs;
                    unit[m].x = __ldcs(reinterpret_cast<const uint4 *>(from + j0));
                    unit[m].y = __ldcs(reinterpret_cast<const uint4 *>(from + j1));
                }
#pragma unroll
                for (int m = 0; m < kAtOnce; ++m) {
                    const int i = i0 + m * kThreads;
                    if (i >= i1) break;
                    int t, h, e, j0, j1;
                    place(i, &t, &h, &e, &j0, &j1);
                    uint16_t *const to = a.q_out.p + (k.t + t) * a.q_out.ts + h * a.q_out.hs;
                    uint4 x = unit[m].x, y = unit[m].y;
                    if (e < a.rot_dim) {
                        float o[kUnit];
                        turn_unit(x, y, true, !a.interleaved, reinterpret_cast<const float4 *>(cs + t * a.rot_dim) + (e >> 4),
                                  half >> 3, o);
                        x = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
                        y = make_uint4(pack_bf16x2(o[8], o[9]), pack_bf16x2(o[10], o[11]), pack_bf16x2(o[12], o[13]), pack_bf16x2(o[14], o[15]));
                    }
                    *reinterpret_cast<uint4 *>(to + j0) = x;
                    *reinterpret_cast<uint4 *>(to + j1) = y;
                }
            }
        } else {
            constexpr int kPairs = D / 2;
            const int all = a.q_heads * kPairs, u0 = all * part / parts, mine = all * (part + 1) / parts - u0;
            for (int i = tid; i < k.n * mine; i += kThreads) {
                const int t = i / mine, q = u0 + i - t * mine, h = q / kPairs, p = q % kPairs;
                const bool rotate = p < half, halves = rotate && !a.interleaved;
                const int j0 = halves ? p : 2 * p, j1 = halves ? p + half : 2 * p + 1;
                const uint16_t *const from = a.q.p + (k.t + t) * a.q.ts + h * a.q.hs;
                uint16_t *const to = a.q_out.p + (k.t + t) * a.q_out.ts + h * a.q_out.hs;
                uint32_t x = (uint32_t)from[j0] | ((uint32_t)from[j1] << 16);
                if (rotate) x = rotate_pair(x, cs[t * a.rot_dim + p], cs[t * a.rot_dim + half + p]);
                to[j0] = (uint16_t)x;
                to[j1] = (uint16_t)(x >> 16);
            }
        }
    }
}

template <int D, int TYPE>
cudaError_t launch_d(const RopeArgs &a, const Kv8Cache &c, cudaStream_t stream) {
    DeviceInfo di;
    cudaError_t err = device_info(&di);
    if (err != cudaSuccess) return err;
    const bool vec = a.rot_dim % kUnit == 0;
    // Up to four tokens an SM: one a CTA, and up to one an SM its heads over several CTAs. Of a sequence's tokens
    // only the first of each block then finds work, so that this suits single tokens (64: 5.1 us, 16 a CTA 40; 608: 14
    // and 43) and not chunks (one of 512: 15.4 us, 16 a CTA 8.0). Above, CTAs of 16 tokens suit chunks (one of 1200: 8.4 us,
    // one a CTA 18) and not single tokens, up to 16 blocks one after the other in a CTA (1024: 43 us, one a CTA 23).
    const bool few = a.tokens <= 4 * di.sm_count;
    const int run = few ? 1 : kMostRun;
    const int jobs = 2 * a.k_heads + (a.q_heads * D + 511) / 512;
    int parts = few && a.tokens <= di.sm_count ? (jobs + kWarps - 1) / kWarps : few ? 1 : 2;
    if (parts > 2 * a.k_heads) parts = 2 * a.k_heads;
    const dim3 grid((unsigned)((a.tokens + run - 1) / run), (unsigned)parts);
    const size_t smem = (size_t)(a.rot_dim / 2 + 1) * sizeof(unsigned long long) + (size_t)a.rot_dim * kKv8Block * sizeof(float);
    const unsigned units = (unsigned)(a.q_heads * (D / kUnit)), magic = (unsigned)(((1ull << 32) + units - 1) / units);
    void (*kern)(const RopeArgs, const Kv8Cache, int, unsigned) = vec ? append_kv8_kernel<D, TYPE, true> : append_kv8_kernel<D, TYPE, false>;
    err = launch_kernel_as(true, kern, grid, dim3(kThreads), smem, stream, 1, a, c, run, magic);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_kv8(const RopeArgs &a, const Kv8Cache &c, int type, cudaStream_t stream) {
    if (type == FD_KV8_E4M3)
        return a.head_dim == 128 ? launch_d<128, FD_KV8_E4M3>(a, c, stream) : launch_d<64, FD_KV8_E4M3>(a, c, stream);
    return a.head_dim == 128 ? launch_d<128, FD_KV8_INT8>(a, c, stream) : launch_d<64, FD_KV8_INT8>(a, c, stream);
}

cudaError_t status_append_kv8(cudaStream_t stream, unsigned *out, bool clear) {
    cudaError_t err = cudaMemcpyFromSymbolAsync(out, g_page_status, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, stream);
    if (err != cudaSuccess || !clear) return err;
    void *p = nullptr;
    err = cudaGetSymbolAddress(&p, g_page_status);
    if (err != cudaSuccess) return err;
    return cudaMemsetAsync(p, 0, sizeof(unsigned), stream);
}

}  // namespace fd
