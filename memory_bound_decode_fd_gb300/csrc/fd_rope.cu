// fd_rope.cu - rotary positions, and the same with the keys and values written to the pages of a
// cache.
//
//   (y0, y1) = scale * (x0 cos a - x1 sin a, x0 sin a + x1 cos a),   a = position * inv_freq[i]
//
// Bound by memory for long inputs (each element read and written once) and by latency for single
// tokens. A CTA takes kRopeTokens tokens (one when tokens are few, and then only a part of the
// heads): its threads first make the cosines and sines of those tokens in shared memory, one
// (token, pair) each, so that they are computed once for all the heads that share them; then each
// thread takes units of 16 elements of a head, two 16-byte loads and two 16-byte stores (the unit's
// two vectors are the partners of each other: adjacent ones for interleaved pairs, rot_dim / 2
// apart for halves).
//
// Angle: position * inv_freq grows to 1e6 radians and more, where 32 bits leave nothing of the
// fraction. inv_freq / (2 pi) is taken in 64-bit floating point, its fraction made a 64-bit
// fixed-point number u of turns, and position * u wraps in 64-bit integer arithmetic, which is the
// reduction to one turn, exactly and for negative positions too. The remaining fraction goes to
// sincospif in 32 bits (error 2^-24 of a half turn at most).
#include <atomic>

#include "fd_attn.h"

namespace fd {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;     // tokens of a CTA's pass when there are many
constexpr int kUnit = 16;          // elements a thread handles at a time

__device__ unsigned int g_page_status;

// Rotates packed pairs: word w of x holds (x0, x1) of pair w.
__device__ __forceinline__ uint32_t rotate_pair(uint32_t x, float2 cs) {
    const float a = bf16lo(x), b = bf16hi(x);
    return pack_bf16x2(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// What a token's rows go to.
struct Place {
    long long k, v;   // element offsets of the token in the cache
    int state;        // 0: the token belongs to no sequence, 1: no place in the cache, 2: both
};

// VEC: head_dim and rot_dim are multiples of 16, so that units of 16 elements never straddle the
// end of the rotated part and every half begins on 16 bytes. Otherwise pairs one by one.
template <bool APPEND, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int tile, int units_cta) {
    extern __shared__ float2 cs[];  // [tile][rot_dim / 2] of (cos, sin) * scale
    __shared__ Place place[kRopeTokens];
    __shared__ int pos_s[kRopeTokens];
    __shared__ int seq_s;
    const int tid = threadIdx.x;
    const int half = a.rot_dim >> 1;
    const int t0 = blockIdx.x * tile;
    const int n = min(tile, a.tokens - t0);
    grid_dep_wait();
    grid_dep_launch();

    if (APPEND) {
        // the sequence of the first token: how many sequences end at or before it
        if (tid == 0) seq_s = 0;
        __syncthreads();
        int before = 0;
        for (int b = tid; b < a.m.batch; b += kRopeThreads) before += a.m.q_start[b + 1] <= t0;
        before = __reduce_add_sync(0xFFFFFFFFu, before);
        if ((tid & 31) == 0 && before) atomicAdd(&seq_s, before);
        __syncthreads();
        if (tid < n) {
            const int t = t0 + tid;
            int b = seq_s;
            while (b < a.m.batch && a.m.q_start[b + 1] <= t) ++b;
            Place p{0, 0, 0};
            int pos = 0;
            if (b < a.m.batch && a.m.q_start[b] <= t) {
                const int kv = min(max(a.m.kv_len[b], 0), a.m.capacity);
                const int first = a.m.q_start[b];
                const int at = kv - (a.m.q_start[b + 1] - first) + (t - first);
                pos = at;
                p.state = 1;
                if (at >= 0 && at < a.m.capacity) {
                    const int page = a.m.table[(long long)b * a.m.table_stride + (at >> a.m.page_shift)];
                    if (page >= 0 && page < a.m.num_pages) {
                        const int off = at & ((1 << a.m.page_shift) - 1);
                        p.k = page * a.k_page + off * a.k_out.ts;
                        p.v = page * a.v_page + off * a.v_out.ts;
                        p.state = 2;
                    } else {
                        atomicOr(&g_page_status, (unsigned)FD_DEVICE_STATUS_BAD_PAGE);
                    }
                }
            }
            if (a.positions) pos = a.positions[t];
            place[tid] = p;
            pos_s[tid] = pos;
        }
    } else if (tid < n) {
        pos_s[tid] = a.positions[t0 + tid];
    }
    __syncthreads();

    for (int i = tid; i < n * half; i += kRopeThreads) {
        const int t = i / half, p = i - t * half;
        double turns = a.inv_freq[p] * 0.15915494309189533577;  // 1 / (2 pi)
        turns -= floor(turns);
        const unsigned long long step = (unsigned long long)(turns * 18446744073709551616.0);
        const long long frac = (long long)((unsigned long long)(long long)pos_s[t] * step);
        float s, c;
        sincospif((float)frac * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
        cs[i] = make_float2(c * a.scale, s * a.scale);
    }
    __syncthreads();

    const int heads = a.q_heads + (APPEND ? 2 : 1) * a.k_heads;
    if (VEC) {
        const int per_head = a.head_dim / kUnit;
        const int u0 = blockIdx.y * units_cta;
        const int nu = min(units_cta, heads * per_head - u0);
#pragma unroll 2
        for (int i = tid; i < n * nu; i += kRopeThreads) {
            const int t = i / nu, u = u0 + i - t * nu;
            int h = u / per_head;
            const int e = (u - h * per_head) * kUnit;  // the unit's place in the head
            const bool rotate = e < a.rot_dim && h < a.q_heads + a.k_heads;
            const HeadsView *src, *dst;
            long long to;
            if (h < a.q_heads) {
                src = &a.q, dst = &a.q_out;
                to = (t0 + t) * dst->ts;
                if (APPEND && place[t].state == 0) continue;
            } else if (h < a.q_heads + a.k_heads) {
                h -= a.q_heads;
                src = &a.k, dst = &a.k_out;
                if (APPEND && place[t].state != 2) continue;
                to = APPEND ? place[t].k : (t0 + t) * dst->ts;
            } else {
                h -= a.q_heads + a.k_heads;
                src = &a.v, dst = &a.v_out;
                if (place[t].state != 2) continue;
                to = place[t].v;
            }
            const uint16_t *from = src->p + (t0 + t) * src->ts + h * src->hs;
            uint16_t *out = dst->p + to + h * dst->hs;
            // halves: elements e/2 .. e/2 + 7 of each half; else 16 adjacent ones
            const bool halves = rotate && !a.interleaved;
            const int j0 = halves ? e >> 1 : e, j1 = halves ? (e >> 1) + half : e + 8;
            uint4 x = *reinterpret_cast<const uint4 *>(from + j0);
            uint4 y = *reinterpret_cast<const uint4 *>(from + j1);
            if (rotate) {
                const float2 *f = cs + t * half + (e >> 1);
                uint32_t xo[4], yo[4];
                if (halves) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t xw = word(x, w), yw = word(y, w);
                        const float2 f0 = f[2 * w], f1 = f[2 * w + 1];
                        const float a0 = bf16lo(xw), b0 = bf16lo(yw), a1 = bf16hi(xw), b1 = bf16hi(yw);
                        xo[w] = pack_bf16x2(a0 * f0.x - b0 * f0.y, a1 * f1.x - b1 * f1.y);
                        yo[w] = pack_bf16x2(a0 * f0.y + b0 * f0.x, a1 * f1.y + b1 * f1.x);
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        xo[w] = rotate_pair(word(x, w), f[w]);
                        yo[w] = rotate_pair(word(y, w), f[w + 4]);
                    }
                }
                x = make_uint4(xo[0], xo[1], xo[2], xo[3]);
                y = make_uint4(yo[0], yo[1], yo[2], yo[3]);
            }
            *reinterpret_cast<uint4 *>(out + j0) = x;
            *reinterpret_cast<uint4 *>(out + j1) = y;
        }
    } else {
        // pairs one by one: head_dim / 2 of them, the rotated ones first
        const int per_head = a.head_dim / 2;
        for (int i = tid; i < n * heads * per_head; i += kRopeThreads) {
            const int t = i / (heads * per_head), r = i - t * heads * per_head;
            int h = r / per_head;
            const int p = r - h * per_head;
            const bool rotate = p < half && h < a.q_heads + a.k_heads;
            const HeadsView *src, *dst;
            long long to;
            if (h < a.q_heads) {
                src = &a.q, dst = &a.q_out;
                to = (t0 + t) * dst->ts;
                if (APPEND && place[t].state == 0) continue;
            } else if (h < a.q_heads + a.k_heads) {
                h -= a.q_heads;
                src = &a.k, dst = &a.k_out;
                if (APPEND && place[t].state != 2) continue;
                to = APPEND ? place[t].k : (t0 + t) * dst->ts;
            } else {
                h -= a.q_heads + a.k_heads;
                src = &a.v, dst = &a.v_out;
                if (place[t].state != 2) continue;
                to = place[t].v;
            }
            const uint16_t *from = src->p + (t0 + t) * src->ts + h * src->hs;
            uint16_t *out = dst->p + to + h * dst->hs;
            const bool halves = rotate && !a.interleaved;
            const int j0 = halves ? p : 2 * p, j1 = halves ? p + half : 2 * p + 1;
            uint32_t x = (uint32_t)from[j0] | ((uint32_t)from[j1] << 16);
            if (rotate) x = rotate_pair(x, cs[t * half + p]);
            out[j0] = (uint16_t)x;
            out[j1] = (uint16_t)(x >> 16);
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
    // Few tokens: one a CTA, and its units over several CTAs, so that a single token's 40 or 48
    // heads are not one CTA's work. Many: kRopeTokens a CTA, so that each thread has several
    // loads in flight and the angles of four tokens keep 256 threads busy.
    const bool few = a.tokens < 4 * di.sm_count;
    const int tile = few ? 1 : kRopeTokens;
    const int units = heads * (a.head_dim / kUnit);
    int units_cta = units;
    if (few && vec && units > kRopeThreads) units_cta = kRopeThreads;
    const int split = vec ? (units + units_cta - 1) / units_cta : 1;
    const dim3 grid((unsigned)((a.tokens + tile - 1) / tile), (unsigned)split);
    const size_t smem = (size_t)tile * (a.rot_dim / 2) * sizeof(float2);
    void (*kern)(const RopeArgs, int, int) =
        append ? (vec ? rope_kernel<true, true> : rope_kernel<true, false>)
               : (vec ? rope_kernel<false, true> : rope_kernel<false, false>);
    err = launch_kernel(kern, grid, dim3(kRopeThreads), smem, stream, 1, a, tile, units_cta);
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
