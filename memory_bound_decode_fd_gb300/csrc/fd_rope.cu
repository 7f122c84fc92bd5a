// fd_rope.cu - rotary positions, and the same with the keys and values written to the pages of a
// cache.
//
//   (y0, y1) = scale * (x0 cos a - x1 sin a, x0 sin a + x1 cos a),   a = position * inv_freq[i]
//
// Bound by memory for long inputs (each element read and written once) and by latency for single
// tokens. Each CTA of a grid that fills the GPU takes an equal run of the tokens, four at a time: its
// threads make the cosines and sines of the next four in shared memory, one (token, pair) each, so
// that they are computed once for all the heads that share them, and rotate the present four, in
// units of 16 elements of a head: two 16-byte loads and two 16-byte stores (the unit's two vectors
// are the partners of each other: adjacent ones for interleaved pairs, rot_dim / 2 apart for halves).
// Few tokens: one a CTA, its heads over several, so that a single token's 40 or 48 heads are not
// one CTA's work (one token: 2.6 us against 2.9; the appends of 64: 3.6 against 4.0; with as many
// parts for 600 tokens 5.8 against 4.3, the angles being made in every part; all of these without
// programmatic launches).
//
// 8191 tokens of 40 heads of 128, half of each rotated, take 29.7 us, 83 % of the copy bandwidth;
// five prompts of up to 1639 appended 29.0, 78 %. Each thread has two units on their way; other
// depths, pass sizes and CTAs an SM took 29.5 to 46 us.
//
// Angle: position * inv_freq grows to 1e6 radians and more, where 32 bits leave nothing of the
// fraction. The fraction of inv_freq / (2 pi) is made a 64-bit fixed-point number u of turns, from
// inv_freq's 53 bits and 128 of 1 / (2 pi) in integer arithmetic, so that it is off by less than 2^-64
// of a turn whatever inv_freq is (a product in 64-bit floating point is off by up to 2^-53 of itself,
// 2^-22 of a turn and more at position 2^31). position * u wraps, which is the reduction to one turn,
// exactly and for negative positions too. The remaining fraction goes to sincospif in 32 bits (error
// 2^-24 of a half turn at most).
#include <atomic>

#include "fd_attn.h"

namespace fd {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;     // tokens of a pass
constexpr int kRopeAhead = 32;     // tokens whose places are looked up together
constexpr int kUnit = 16;          // elements a thread handles at a time
constexpr int kRopeCtas = 4;       // CTAs of an SM

__device__ unsigned int g_page_status;

// Rotates the pair in the two halves of x.
__device__ __forceinline__ uint32_t rotate_pair(uint32_t x, float c, float s) {
    const float a = bf16lo(x), b = bf16hi(x);
    return pack_bf16x2(a * c - b * s, a * s + b * c);
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// The fraction of f / (2 pi), |f| < 2^53, as a 64-bit fixed-point number, rounded towards 0: of the
// product of f's mantissa m and the first 128 bits of 1 / (2 pi) the bits that belong there.
__device__ __forceinline__ unsigned long long turns_64(double f) {
    constexpr unsigned long long kHigh = 0x28BE60DB9391054Aull, kLow = 0x7F09D5F47D4D3770ull;
    const unsigned long long bits = (unsigned long long)__double_as_longlong(f), one = 1ull << 52;
    const int e = (int)(bits >> 52) & 0x7FF, s = max(1075 - max(e, 1), 0);  // |f| = m 2^-s
    const unsigned long long m = (bits & (one - 1)) | (e ? one : 0);
    const unsigned long long carry = __umul64hi(m, kLow), w1 = carry + m * kHigh;  // bits 64 .. 127
    const unsigned long long w2 = __umul64hi(m, kHigh) + (w1 < carry ? 1 : 0);     // 128 ..
    const unsigned long long u = s == 0   ? w1
                                 : s < 64 ? w1 >> s | w2 << (64 - s)
                                          : s < 128 ? w2 >> (s - 64) : 0;
    return bits >> 63 ? 0 - u : u;
}

// A token: element offsets of its queries, keys and values, and of where they go.
struct Token {
    long long q, k, v, q_to, k_to, v_to;
    int pos;
    int state;   // 0: it belongs to no sequence, 1: it has no place in the cache, 2: both
};

// One unit: where it comes from and goes to.
struct Unit {
    const uint16_t *from;
    uint16_t *to;
    int e;         // its place in the head; -1: nothing to do
    bool rotate;
    int t;         // token of the pass
    uint4 x, y;
};

// VEC: head_dim and rot_dim are multiples of 16, so that units of 16 elements never straddle the
// end of the rotated part and every half begins on 16 bytes. Otherwise pairs one by one.
// head_magic: ceil(2^32 / units of a head), exact for the at most 3 * 1024 * 16 units of a token.
template <bool APPEND, bool VEC>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    rope_kernel(const RopeArgs a, int units_cta, unsigned head_magic) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int half = a.rot_dim >> 1;
    unsigned long long *const step = reinterpret_cast<unsigned long long *>(smem);  // [half] of a turn
    // Cosines and sines times scale, 2 x [kRopeTokens][rot_dim]. VEC: as (cos, cos, sin, sin) of two
    // pairs, the first two pairs of all units, then the second two ..: neighbouring threads read
    // neighbouring 16 bytes. Otherwise all cosines, then all sines.
    float *const cs0 = reinterpret_cast<float *>(step + half + (half & 1));
    __shared__ Token tokens[kRopeAhead];
    __shared__ int seq_s;
    const int tid = threadIdx.x;
    const int t_begin = (int)((long long)a.tokens * blockIdx.x / gridDim.x);
    const int t_end = (int)((long long)a.tokens * (blockIdx.x + 1) / gridDim.x);
    grid_dep_wait();
    grid_dep_launch();

    for (int i = tid; i < half; i += kRopeThreads) step[i] = turns_64(a.inv_freq[i]);
    // Those of the tokens [first, first + n) of the ones looked up.
    auto angles = [&](int first, int n, float *cs) {
        for (int i = tid; i < n * half; i += kRopeThreads) {
            const int t = i / half, p = i - t * half;
            const long long frac = (long long)((unsigned long long)(long long)tokens[first + t].pos * step[p]);
            float s, c;
            sincospif((float)frac * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
            float *const to = cs + t * a.rot_dim +
                              (VEC ? (((p >> 1 & 3) * (half >> 3) + (p >> 3)) << 2) + (p & 1) : p);
            to[0] = c * a.scale;
            to[VEC ? 2 : half] = s * a.scale;
        }
    };
    // Source and destination of head h (queries, keys, values) of a token.
    auto locate = [&](const Token &t, int h, const uint16_t **from, uint16_t **to, bool *rotate) {
        *rotate = true;
        if (h < a.q_heads) {
            *from = a.q.p + t.q + h * a.q.hs;
            *to = a.q_out.p + t.q_to + h * a.q_out.hs;
            return !APPEND || t.state != 0;
        }
        h -= a.q_heads;
        if (h < a.k_heads) {
            *from = a.k.p + t.k + h * a.k.hs;
            *to = a.k_out.p + t.k_to + h * a.k_out.hs;
            return !APPEND || t.state == 2;
        }
        h -= a.k_heads;
        *rotate = false;
        *from = a.v.p + t.v + h * a.v.hs;
        *to = a.v_out.p + t.v_to + h * a.v_out.hs;
        return t.state == 2;
    };
    const int heads = a.q_heads + (APPEND ? 2 : 1) * a.k_heads;

    for (int s0 = t_begin; s0 < t_end; s0 += kRopeAhead) {
        const int n_ahead = min(kRopeAhead, t_end - s0);
        __syncthreads();
        if (APPEND) {
            // the sequence of the first token: how many sequences end at or before it
            if (tid == 0) seq_s = 0;
            __syncthreads();
            int before = 0;
            for (int b = tid; b < a.m.batch; b += kRopeThreads) before += a.m.q_start[b + 1] <= s0;
            before = __reduce_add_sync(0xFFFFFFFFu, before);
            if ((tid & 31) == 0 && before) atomicAdd(&seq_s, before);
            __syncthreads();
            if (tid < n_ahead) {
                const long long t = s0 + tid;
                int b = seq_s;
                while (b < a.m.batch && a.m.q_start[b + 1] <= t) ++b;
                Token k{t * a.q.ts, t * a.k.ts, t * a.v.ts, t * a.q_out.ts, 0, 0, 0, 0};
                if (b < a.m.batch && a.m.q_start[b] <= t) {
                    const int kv = min(max(a.m.kv_len[b], 0), a.m.capacity);
                    const int first = a.m.q_start[b];
                    const int at = kv - (a.m.q_start[b + 1] - first) + ((int)t - first);
                    k.pos = at;
                    k.state = 1;
                    if (a.m.kv_len[b] > a.m.capacity) {  // its tokens would go over others'
                        atomicOr(&g_page_status, (unsigned)FD_DEVICE_STATUS_BAD_PAGE);
                    } else if (at >= 0) {
                        const int page = a.m.table[(long long)b * a.m.table_stride + (at >> a.m.page_shift)];
                        if (page >= 0 && page < a.m.num_pages) {
                            const int off = at & ((1 << a.m.page_shift) - 1);
                            k.k_to = page * a.k_page + off * a.k_out.ts;
                            k.v_to = page * a.v_page + off * a.v_out.ts;
                            k.state = 2;
                        } else {
                            atomicOr(&g_page_status, (unsigned)FD_DEVICE_STATUS_BAD_PAGE);
                        }
                    }
                }
                if (a.positions) k.pos = a.positions[t];
                tokens[tid] = k;
            }
        } else if (tid < n_ahead) {
            const long long t = s0 + tid;
            tokens[tid] = Token{t * a.q.ts, t * a.k.ts, 0, t * a.q_out.ts, t * a.k_out.ts, 0, a.positions[t], 0};
        }
        __syncthreads();
        angles(0, min(kRopeTokens, n_ahead), cs0);
        __syncthreads();

        for (int c = 0; c < n_ahead; c += kRopeTokens) {
            const int n = min(kRopeTokens, n_ahead - c);
            const float *const cs = cs0 + (c / kRopeTokens & 1) * kRopeTokens * a.rot_dim;
            float *const cs_next = cs0 + ((c / kRopeTokens & 1) ^ 1) * kRopeTokens * a.rot_dim;
            const int n_next = min(kRopeTokens, n_ahead - c - kRopeTokens);  // <= 0: no more
            if (VEC) {
                const int per_head = a.head_dim / kUnit;
                const int u0 = blockIdx.y * units_cta;
                const int nu = min(units_cta, heads * per_head - u0);
                auto load = [&](int i, Unit &w) {
                    w.e = -1;
                    if (i >= n * nu) return;
                    w.t = (i >= nu) + (i >= 2 * nu) + (i >= 3 * nu);
                    const unsigned u = u0 + i - w.t * nu;
                    const int h = per_head == 1 ? (int)u : (int)__umulhi(u, head_magic);
                    const int e = (int)u - h * per_head;
                    if (!locate(tokens[c + w.t], h, &w.from, &w.to, &w.rotate)) return;
                    w.e = e * kUnit;
                    w.rotate = w.rotate && w.e < a.rot_dim;
                    // halves: elements e/2 .. e/2 + 7 of each half; else 16 adjacent ones
                    const bool halves = w.rotate && !a.interleaved;
                    const int j0 = halves ? w.e >> 1 : w.e, j1 = halves ? (w.e >> 1) + half : w.e + 8;
                    w.x = __ldcs(reinterpret_cast<const uint4 *>(w.from + j0));
                    w.y = __ldcs(reinterpret_cast<const uint4 *>(w.from + j1));
                };
                auto store = [&](const Unit &w) {
                    if (w.e < 0) return;
                    uint4 x = w.x, y = w.y;
                    const bool halves = w.rotate && !a.interleaved;
                    const int j0 = halves ? w.e >> 1 : w.e, j1 = halves ? (w.e >> 1) + half : w.e + 8;
                    if (w.rotate) {
                        const float4 *f = reinterpret_cast<const float4 *>(cs + w.t * a.rot_dim) + (w.e >> 4);
                        uint32_t xo[4], yo[4];
                        if (halves) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float4 g = f[k * (half >> 3)];
                                const float2 co = make_float2(g.x, g.y), si = make_float2(g.z, g.w);
                                const float2 no = make_float2(-g.z, -g.w);
                                const float2 p = make_float2(bf16lo(word(x, k)), bf16hi(word(x, k)));
                                const float2 q = make_float2(bf16lo(word(y, k)), bf16hi(word(y, k)));
                                const float2 zero = make_float2(0.f, 0.f);
                                const float2 xr = ffma2(p, co, ffma2(q, no, zero));
                                const float2 yr = ffma2(p, si, ffma2(q, co, zero));
                                xo[k] = pack_bf16x2(xr.x, xr.y);
                                yo[k] = pack_bf16x2(yr.x, yr.y);
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float4 g = f[k * (half >> 3)];
                                const uint32_t p0 = k < 2 ? word(x, 2 * k) : word(y, 2 * k - 4);
                                const uint32_t p1 = k < 2 ? word(x, 2 * k + 1) : word(y, 2 * k - 3);
                                const uint32_t r0 = rotate_pair(p0, g.x, g.z), r1 = rotate_pair(p1, g.y, g.w);
                                if (k < 2)
                                    xo[2 * k] = r0, xo[2 * k + 1] = r1;
                                else
                                    yo[2 * k - 4] = r0, yo[2 * k - 3] = r1;
                            }
                        }
                        x = make_uint4(xo[0], xo[1], xo[2], xo[3]);
                        y = make_uint4(yo[0], yo[1], yo[2], yo[3]);
                    }
                    *reinterpret_cast<uint4 *>(w.to + j0) = x;
                    *reinterpret_cast<uint4 *>(w.to + j1) = y;
                };
                Unit w0, w1;
                load(tid, w0);
                load(tid + kRopeThreads, w1);
                if (n_next > 0) angles(c + kRopeTokens, n_next, cs_next);  // while the loads are on their way
                for (int i = tid; i < n * nu; i += 2 * kRopeThreads) {
                    store(w0);
                    store(w1);
                    load(i + 2 * kRopeThreads, w0);
                    load(i + 3 * kRopeThreads, w1);
                }
            } else {
                if (n_next > 0) angles(c + kRopeTokens, n_next, cs_next);
                // pairs one by one: head_dim / 2 of them, the rotated ones first
                const int per_head = a.head_dim / 2;
                for (int i = tid; i < n * heads * per_head; i += kRopeThreads) {
                    const int t = i / (heads * per_head), r = i - t * heads * per_head;
                    const int h = r / per_head, p = r - h * per_head;
                    const uint16_t *from;
                    uint16_t *to;
                    bool rotate;
                    if (!locate(tokens[c + t], h, &from, &to, &rotate)) continue;
                    rotate = rotate && p < half;
                    const bool halves = rotate && !a.interleaved;
                    const int j0 = halves ? p : 2 * p, j1 = halves ? p + half : 2 * p + 1;
                    uint32_t x = (uint32_t)from[j0] | ((uint32_t)from[j1] << 16);
                    if (rotate) x = rotate_pair(x, cs[t * a.rot_dim + p], cs[t * a.rot_dim + half + p]);
                    to[j0] = (uint16_t)x;
                    to[j1] = (uint16_t)(x >> 16);
                }
            }
            __syncthreads();
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, bool append, cudaStream_t stream) {
    DeviceInfo di;
    cudaError_t err = device_info(&di);
    if (err != cudaSuccess) return err;
    const bool vec = a.head_dim % kUnit == 0 && a.rot_dim % kUnit == 0;
    const int heads = a.q_heads + (append ? 2 : 1) * a.k_heads;
    const int per_head = vec ? a.head_dim / kUnit : 1;
    const int units = heads * per_head;
    void (*kern)(const RopeArgs, int, unsigned) =
        append ? (vec ? rope_kernel<true, true> : rope_kernel<true, false>)
               : (vec ? rope_kernel<false, true> : rope_kernel<false, false>);
    // a run of tokens for each CTA that the GPU holds at a time; few tokens: one a CTA, its units
    // over several
    const int most = kRopeCtas * di.sm_count;
    const int split = vec && a.tokens < 2 * di.sm_count ? (units + kRopeThreads - 1) / kRopeThreads : 1;
    const int units_cta = (units + split - 1) / split;
    const dim3 grid((unsigned)(a.tokens < most ? a.tokens : most), (unsigned)split);
    const size_t smem = (size_t)(a.rot_dim / 2 + 1) * sizeof(unsigned long long) +
                        (size_t)a.rot_dim * 2 * kRopeTokens * sizeof(float);
    const unsigned magic = (unsigned)(((1ull << 32) + per_head - 1) / per_head);
    // nothing is read before the wait: 8191 tokens one call behind the other 30.1 us, 32.9 without
    err = launch_kernel_as(true, kern, grid, dim3(kRopeThreads), smem, stream, 1, a, units_cta, magic);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

cudaError_t status_rope(cudaStream_t stream, unsigned *out, bool clear) {
    cudaError_t err = cudaMemcpyFromSymbolAsync(out, g_page_status, sizeof(unsigned), 0,
                                                cudaMemcpyDeviceToHost, stream);
    if (err != cudaSuccess || !clear) return err;
    void *p = nullptr;
    err = cudaGetSymbolAddress(&p, g_page_status);
    if (err != cudaSuccess) return err;
    return cudaMemsetAsync(p, 0, sizeof(unsigned), stream);
}

}  // namespace fd
