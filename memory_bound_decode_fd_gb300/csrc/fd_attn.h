// fd_attn.h - what the rotary, cache and attention sources share: the device view of a paged
// batch, the visible range of a row, and the launchers (see include/fd.h for the operators).
#pragma once

#include <cuda.h>  // CUtensorMap (type only)

#include "fd_internal.h"

namespace fd {

// A bf16 [tokens, heads, head_dim] view: strides in elements.
struct HeadsView {
    uint16_t *p;
    long long ts, hs;
};

// The paged batch as a kernel reads it.
struct PagedMeta {
    const int *q_start;
    const int *kv_len;
    const int *table;
    int table_stride;
    int batch;
    int total_q;
    int max_q;
    int capacity;    // max_pages * page_size
    int num_pages;
    int page_shift;  // log2(page_size)
};

struct SeqInfo {
    int q0;    // first activation row
    int rows;  // new tokens that are computed
    int kv;    // tokens in the cache
    int base;  // number of new token 0 (negative where it has no place)
};

// Reads sequence b's entries. Whatever the arrays hold, the rows lie in [0, total_q) and the
// tokens in [0, capacity].
__device__ __forceinline__ SeqInfo load_seq(const PagedMeta &m, int b) {
    int q0 = m.q_start[b], q1 = m.q_start[b + 1], kv = m.kv_len[b];
    q0 = min(max(q0, 0), m.total_q);
    q1 = min(max(q1, q0), m.total_q);
    kv = min(max(kv, 0), m.capacity);
    return {q0, min(q1 - q0, m.max_q), kv, kv - (q1 - q0)};
}

// Keys [lo, hi) that new token i sees; lo >= hi: none.
__device__ __forceinline__ int key_hi(const SeqInfo &s, int i, int causal) {
    return causal ? min(s.kv, s.base + i + 1) : s.kv;
}
__device__ __forceinline__ int key_lo(const SeqInfo &s, int i, int window) {
    return window > 0 ? max(0, s.base + i - window + 1) : 0;
}

// How the keys of a call are cut into tiles: those that the rows with the visible keys [lo, hi) need, in
// order, are the `sinks` tiles of the first tokens that lie before lo's, then all from lo's on. Tile t of
// the `count` is tile t, or t + shift from t = sinks on.
struct KeyTiles {
    int count, sinks, shift;
};
template <int TILE>
__device__ __forceinline__ KeyTiles key_tiles(int lo, int hi, int sinks) {
    if (hi <= lo) return {0, 0, 0};
    const int first = lo / TILE, n = min((int)((min(sinks, hi) + TILE - 1) / TILE), first);
    return {(hi + TILE - 1) / TILE - first + n, n, first - n};
}

// Where a dimension of the cache lies in its tensor map (1 .. 3, dimension 0 is head_dim).
struct MapOrder {
    int tok, head, page;
};

// The keys or the values of a cache in 8 bits: strides in bytes.
struct Kv8Plane {
    uint8_t *codes, *scale;
    long long page, token, head, scale_page, scale_block, scale_head;
};
struct Kv8Cache {
    Kv8Plane k, v;
};

struct AttnArgs {
    PagedMeta m;
    HeadsView q, out;
    float *lse;       // [total_q, q_heads] or null
    MapOrder ok, ov;  // of the cache's tensor maps
    int q_heads, kv_heads, group, head_dim;
    int causal, window;
    int sinks;        // the first tokens that a window leaves visible (0 without one)
    float scale;      // multiplies q.k
    float softcap;    // 0: none
    int kv_type;      // 0: a bf16 cache; else FD_KV8_*, and its scales are those of kv8
    Kv8Cache kv8;
    unsigned *counters;  // one per CTA, zero between calls
    float *partials;     // one slot for the first and one for the last item of each CTA
    struct AttnPart *parts;  // of fd_attn_tc.cu: one for each CTA
    // FD_LAUNCH_TEST_WAIT_TIMEOUT: short waits, and the first copy of every CTA is left out.
    int test_timeout;
};
// An item that begins in one CTA and ends in another (last < 0: there is none).
struct AttnPart {
    long long row0;  // activation row of the first token
    int rows, hk;    // tokens from there on, key head
    int first, last; // the CTAs that share it
};

constexpr int kAttnMaxCtas = 256;             // largest grid (counters in the scratch)
constexpr int kAttnCounterBytes = 4 * 4096;   // the scratch begins with them
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---- scores in log2 units
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// tanh(y) / y as a polynomial in z = y^2: the minimax ones (found by exchange on a fine grid) for
// |y| <= 1/2, degree 4, and |y| <= 1, degree 7; with the rounding of its steps off by at most
// 1.3 2^-24 of itself.
template <bool NEAR>
__device__ __forceinline__ float2 tanh_over(float2 z) {
    constexpr int kDegree = NEAR ? 4 : 7;
    const float near[8] = {1.0f, -0.3333306909f, 0.1332477927f, -0.0529860742f, 0.0171350073f};
    const float below[8] = {1.0f, -0.3333328366f, 0.1333224028f, -0.0538756959f,
                            0.0214784257f, -0.0079373326f, 0.0022966541f, -0.0003574573f};
    auto c = [&](int i) { return NEAR ? make_float2(near[i], near[i]) : make_float2(below[i], below[i]); };
    float2 p = c(kDegree);
#pragma unroll
    for (int i = kDegree - 1; i >= 0; --i) p = ffma2(p, z, c(i));
    return p;
}

// Two scores s = scale v capped, c tanh(y) with y = s / c, in log2 units (lin = scale log2(e),
// cap_in = scale / c, cap_out = c log2(e)). Below the cap it is s times tanh(y) / y: the error is one of
// the score, where that of c (1 - 2 / (e^(2 y) + 1)) would be one of the cap (0.9 at c = 10^7, and of
// scores of a few from c = 10^9 on nothing would be left). Above, tanh is no smaller than 0.76 and the
// quotient is as good. NEAR: both are known to be below half the cap.
template <bool NEAR>
__device__ __forceinline__ float2 capped_log2(float2 v, float lin, float cap_in, float cap_out) {
    const float2 zero = make_float2(0.f, 0.f);
    const float2 y = ffma2(v, make_float2(cap_in, cap_in), zero);
    float2 s = ffma2(ffma2(v, make_float2(lin, lin), zero), tanh_over<NEAR>(ffma2(y, y, zero)), zero);
    if (NEAR) return s;
    auto far = [&](float u) { return cap_out * (1.f - __fdividef(2.f, ex2(u * (2.f * kLog2e)) + 1.f)); };
    if (fabsf(y.x) > 1.f) s.x = far(y.x);
    if (fabsf(y.y) > 1.f) s.y = far(y.y);
    return s;
}

// ---- attention of few rows per key head (fd_attn_rows.cu)
constexpr int kRowsM = 16;      // query rows of one pass over the keys
constexpr int kRowsBox = 32;    // tokens of a copy (16 where a page has no more)
__host__ __device__ constexpr int rows_warps(int d) { return d == 128 ? 4 : 8; }
// fp32 words of a partial result: 16 rows of head_dim, then (maximum, sum) of each
__host__ __device__ constexpr int rows_slot_words(int d) { return kRowsM * (d + 2); }
cudaError_t launch_attn_rows(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                             cudaStream_t stream);
cudaError_t launch_attn_rows_kv8(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                                 cudaStream_t stream);
cudaError_t status_attn_rows(cudaStream_t stream, unsigned *out, bool clear);
cudaError_t status_attn_rows_kv8(cudaStream_t stream, unsigned *out, bool clear);

// ---- attention of chunks (fd_attn_tc.cu)
constexpr int kAttnTcTile = 128;    // keys of a tile
constexpr int kAttnTcListed = 152;  // pairs of halves, and sequences, that a CTA can list
// fp32 words of a partial result: 256 rows of head_dim, then (maximum, sum) of each
__host__ __device__ constexpr int tc_slot_words(int d) { return 2 * 128 * (d + 2); }
cudaError_t launch_attn_tc(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                           cudaStream_t stream);
cudaError_t launch_attn_tc_kv8(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                               cudaStream_t stream);
cudaError_t status_attn_tc(cudaStream_t stream, unsigned *out, bool clear);
cudaError_t status_attn_tc_kv8(cudaStream_t stream, unsigned *out, bool clear);

// Which of the two: up to 16 rows a key head are one pass of the first (16 sequences of up to 6000,
// 4 heads a key head: 4 new tokens, 16 rows, 51 us in the first and 65 in the second; 8, 32 rows, 78
// in two passes of the first and 51 in the second); a group of more than 128 query heads does not
// fit the second's tile, and it wants a positive scale. The batch's longest chunk decides for all of it:
// 32 tokens and a chunk of 512, 8192 keys each, take 235 us in one call, 162 and 61 in two. 64 single tokens
// of 4096 keys take 38 us with 32 heads on one (the second kernel), 33 with 16 on one.
// Over a cache in 8 bits two passes of the first kernel are the shorter ones too (16 sequences of 3000, 20 to 32 rows:
// 49 us in the first and 65 in the second, 31 and 49 at head_dim 64; of up to 6000 and 8 to 32 rows 52 and 76). Three are
// at head_dim 64 alone (40 to 48 rows: 45 and 49; at 128 74 and 65), four are not (59 and 49, 94 and 65).
inline bool attn_uses_tc(int max_q, int group, float scale, bool kv8 = false) {
    return (long long)max_q * group > (kv8 ? 2 : 1) * kRowsM && group <= kAttnTcTile && scale > 0.f;
}

// ---- rotary positions (fd_rope.cu)
struct RopeArgs {
    HeadsView q, k, v, q_out, k_out, v_out;  // k_out / v_out: the cache with its token and head strides
    long long k_page, v_page;                // page strides of the cache
    const int *positions;
    const double *inv_freq;
    PagedMeta m;                             // the batch (append only)
    int tokens, q_heads, k_heads, head_dim, rot_dim, interleaved;
    float scale;
};
cudaError_t launch_rope(const RopeArgs &a, bool append, cudaStream_t stream);
cudaError_t status_rope(cudaStream_t stream, unsigned *out, bool clear);
// The append to a cache in 8 bits (fd_append_kv8.cu); of `a` k_out, v_out, k_page and v_page are not used.
cudaError_t launch_append_kv8(const RopeArgs &a, const Kv8Cache &c, int type, cudaStream_t stream);
cudaError_t status_append_kv8(cudaStream_t stream, unsigned *out, bool clear);

}  // namespace fd
