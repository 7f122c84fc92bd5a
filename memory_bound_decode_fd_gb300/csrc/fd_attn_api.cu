// fd_attn_api.cu - entry points of rotary positions, the cache append and paged attention:
// argument checks (all on the host, before any CUDA call), tensor maps and kernel choice.
#include <atomic>
#include <cmath>
#include <cstdint>

#include <cudaTypedefs.h>

#include "fd_attn.h"

namespace fd {
namespace {

constexpr long long kMaxStride = 1ll << 36;  // elements; a tensor map's strides end at 2^40 bytes
constexpr int kMaxTokens = 1 << 28;
constexpr float kMaxScale = 1e30f;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The memory of an activation.
struct Span {
    uintptr_t at;
    long long bytes;  // from the first element to behind the last
    long long period; // bytes between tokens
    long long inner;  // bytes from a token's first element to behind its last
};

Span span_of(const fd_heads &h, int tokens, int head_dim) {
    const long long inner = ((long long)(h.heads - 1) * h.head_stride + head_dim) * 2;
    return {reinterpret_cast<uintptr_t>(h.data), (long long)(tokens - 1) * h.token_stride * 2 + inner,
            h.token_stride * 2, inner};
}

// Whether two activations may share an element: their spans meet, and where both have the same
// distance between tokens (views of one wider row) also their parts of a row do.
bool spans_meet(const Span &a, const Span &b) {
    if (a.at >= b.at + b.bytes || b.at >= a.at + a.bytes) return false;
    if (a.period != b.period || a.period <= 0 || a.inner > a.period || b.inner > a.period) return true;
    const long long delta =
        (long long)(((b.at % a.period) + a.period - (a.at % a.period)) % a.period);  // b behind a, in a row
    return delta < a.inner || delta + b.inner > a.period;
}
bool span_meets(const Span &a, const void *p, long long bytes) {
    const uintptr_t q = reinterpret_cast<uintptr_t>(p);
    return a.at < q + bytes && q < a.at + a.bytes;
}

int check_heads(const fd_heads &h, int tokens, int head_dim, bool output) {
    if (h.heads <= 0) return FD_ERR_SHAPE;
    if (h.heads > FD_MAX_HEADS) return FD_ERR_UNSUPPORTED;
    if (!h.data) return FD_ERR_NULL;
    if (h.token_stride < 0 || h.head_stride < 0 || h.token_stride % 8 != 0 || h.head_stride % 8 != 0)
        return FD_ERR_SHAPE;
    if (h.token_stride > kMaxStride || h.head_stride > kMaxStride) return FD_ERR_UNSUPPORTED;
    if (!aligned(h.data, 16)) return FD_ERR_ALIGN;
    if (output) {
        const bool heads_ok = h.heads == 1 || h.head_stride >= head_dim;
        const bool tokens_ok = tokens <= 1 || h.token_stride >= head_dim;
        const bool nested = h.heads == 1 || tokens <= 1 ||
                            h.token_stride >= (long long)(h.heads - 1) * h.head_stride + head_dim ||
                            h.head_stride >= (long long)(tokens - 1) * h.token_stride + head_dim;
        if (!heads_ok || !tokens_ok || !nested) return FD_ERR_OVERLAP;
    }
    return FD_OK;
}

// A dimension of the cache.
struct Dim {
    long long extent, stride;
    int kind;  // 0 token, 1 head, 2 page
};

// The three outer dimensions by ascending stride, those of one entry last (their stride is that
// of the largest). FD_ERR_SHAPE for strides that are not positive multiples of 8, or of the
// next smaller one.
int order_dims(const fd_paged_cache &c, bool keys, Dim (&d)[3]) {
    d[0] = {c.page_size, keys ? c.k_token_stride : c.v_token_stride, 0};
    d[1] = {c.kv_heads, keys ? c.k_head_stride : c.v_head_stride, 1};
    d[2] = {c.num_pages, keys ? c.k_page_stride : c.v_page_stride, 2};
    for (const Dim &x : d) {
        if (x.extent == 1) continue;
        if (x.stride <= 0 || x.stride % 8 != 0) return FD_ERR_SHAPE;
        if (x.stride > kMaxStride) return FD_ERR_UNSUPPORTED;
    }
    const auto before = [](const Dim &x, const Dim &y) {
        if ((x.extent == 1) != (y.extent == 1)) return y.extent == 1;
        return x.extent != 1 && x.stride < y.stride;
    };
    for (int i = 1; i < 3; ++i)
        for (int j = i; j > 0 && before(d[j], d[j - 1]); --j) {
            const Dim t = d[j];
            d[j] = d[j - 1], d[j - 1] = t;
        }
    long long largest = 8;
    for (Dim &x : d) {
        if (x.extent == 1)
            x.stride = largest;
        else if (x.stride % largest != 0)
            return FD_ERR_SHAPE;
        largest = x.stride;
    }
    return FD_OK;
}

// Bytes from a cache tensor's first element to behind its last; its dimensions may not overlap.
int cache_bytes(const Dim (&d)[3], int head_dim, long long *bytes) {
    long long span = head_dim;
    for (const Dim &x : d) {
        if (x.extent > 1 && x.stride < span) return FD_ERR_OVERLAP;
        span += (x.extent - 1) * (x.extent > 1 ? x.stride : 0);
    }
    *bytes = span * 2;
    return FD_OK;
}

int check_cache(const fd_paged_cache &c, Dim (&dk)[3], Dim (&dv)[3], long long *kb, long long *vb) {
    if (c.num_pages <= 0 || c.kv_heads <= 0 || c.page_size < 16 ||
        (c.page_size & (c.page_size - 1)) != 0)
        return FD_ERR_SHAPE;
    if (c.page_size > FD_MAX_PAGE_SIZE || c.kv_heads > FD_MAX_HEADS ||
        (c.head_dim != 64 && c.head_dim != 128))
        return FD_ERR_UNSUPPORTED;
    if (!c.k || !c.v) return FD_ERR_NULL;
    int st = order_dims(c, true, dk);
    if (st == FD_OK) st = order_dims(c, false, dv);
    if (st != FD_OK) return st;
    if (!aligned(c.k, 16) || !aligned(c.v, 16)) return FD_ERR_ALIGN;
    st = cache_bytes(dk, c.head_dim, kb);
    return st != FD_OK ? st : cache_bytes(dv, c.head_dim, vb);
}

// Whether no element of the keys is one of the values: their spans are apart, or both are views
// of one buffer with the same strides, the values in the gaps of one dimension of the keys.
bool keys_apart(const fd_paged_cache &c, const Dim (&dk)[3], const Dim (&dv)[3], long long kb, long long vb) {
    const uintptr_t k = reinterpret_cast<uintptr_t>(c.k), v = reinterpret_cast<uintptr_t>(c.v);
    if (k >= v + vb || v >= k + kb) return true;
    for (int i = 0; i < 3; ++i)
        if (dk[i].kind != dv[i].kind || (dk[i].extent > 1 && dk[i].stride != dv[i].stride)) return false;
    const long long delta = (long long)(k < v ? v - k : k - v);
    long long inner = 2ll * c.head_dim;  // bytes of the dimensions inside
    for (int i = 0; i < 3 && dk[i].extent > 1; ++i) {
        if (delta >= inner && delta + inner <= dk[i].stride * 2) return true;
        inner += (dk[i].extent - 1) * dk[i].stride * 2;
    }
    return false;
}

int check_batch(const fd_paged_batch &b, int page_size) {
    if (b.batch < 0 || b.total_q < 0 || b.max_q < 0 || b.max_pages < 0 || b.table_stride < b.max_pages)
        return FD_ERR_SHAPE;
    if (b.batch > FD_MAX_BATCH || b.total_q > kMaxTokens ||
        (long long)b.max_pages * page_size > FD_MAX_SEQ)
        return FD_ERR_UNSUPPORTED;
    if (!b.q_start || !b.kv_len || (b.max_pages > 0 && !b.block_table)) return FD_ERR_NULL;
    if (!aligned(b.q_start, 4) || !aligned(b.kv_len, 4) || !aligned(b.block_table, 4)) return FD_ERR_ALIGN;
    return FD_OK;
}

// Whether memory that a call writes is part of the batch's index arrays.
bool meets_index(const Span &out, const fd_paged_batch &b) {
    return span_meets(out, b.q_start, 4ll * (b.batch + 1)) || span_meets(out, b.kv_len, 4ll * b.batch) ||
           (b.max_pages > 0 && span_meets(out, b.block_table, 4ll * ((long long)(b.batch - 1) * b.table_stride + b.max_pages)));
}

HeadsView view(const fd_heads &h) {
    return {static_cast<uint16_t *>(h.data), h.token_stride, h.head_stride};
}

PagedMeta meta(const fd_paged_batch &b, const fd_paged_cache &c) {
    int shift = 0;
    while ((1 << shift) < c.page_size) ++shift;
    return {b.q_start, b.kv_len, b.block_table, b.table_stride, b.batch, b.total_q,
            b.max_q < b.total_q ? b.max_q : b.total_q, b.max_pages * c.page_size, c.num_pages, shift};
}

bool in_place(const fd_heads &a, const fd_heads &b) {
    return a.data == b.data && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

using EncodeTiled = PFN_cuTensorMapEncodeTiled_v12000;

EncodeTiled encode_fn() {
    static std::atomic<void *> fn{nullptr};
    void *f = fn.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !f)
            return nullptr;
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// The cache tensor as a 4D map (head_dim, then the dimensions of `d`), with boxes of 64 elements
// of `tokens` tokens in the 128-byte swizzle. Copies outside the tensor read zeros.
bool encode_cache(CUtensorMap *map, const void *base, const Dim (&d)[3], int head_dim, int tokens,
                  MapOrder *order) {
    EncodeTiled enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)head_dim};
    cuuint64_t strides[3];
    cuuint32_t box[4] = {64, 1, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    int place[3];
    for (int i = 0; i < 3; ++i) {
        dims[i + 1] = (cuuint64_t)d[i].extent;
        strides[i] = (cuuint64_t)d[i].stride * 2;
        if (d[i].kind == 0) box[i + 1] = (cuuint32_t)tokens;
        place[d[i].kind] = i + 1;
    }
    *order = {place[0], place[1], place[2]};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace fd

using namespace fd;

extern "C" {

int fd_rope(const fd_heads *q, const fd_heads *k, const fd_heads *q_out, const fd_heads *k_out,
            const int *positions, const double *inv_freq, int tokens, int head_dim, int rot_dim,
            int interleaved, float scale, fd_stream_t stream) {
    if (tokens < 0 || head_dim <= 0 || head_dim % 8 != 0 || rot_dim < 2 || rot_dim % 2 != 0 ||
        rot_dim > head_dim || !std::isfinite(scale))
        return FD_ERR_SHAPE;
    if (head_dim > FD_MAX_ROPE_DIM || tokens > kMaxTokens) return FD_ERR_UNSUPPORTED;
    if (tokens == 0) return FD_OK;  // empty: nothing read or written
    if (!q || !q_out || !k != !k_out || !positions || !inv_freq) return FD_ERR_NULL;
    const fd_heads *in[2] = {q, k}, *out[2] = {q_out, k_out};
    const int n = k ? 2 : 1;
    for (int i = 0; i < n; ++i) {
        int st = check_heads(*in[i], tokens, head_dim, false);
        if (st == FD_OK) st = check_heads(*out[i], tokens, head_dim, true);
        if (st != FD_OK) return st;
        if (in[i]->heads != out[i]->heads) return FD_ERR_SHAPE;
    }
    if (!aligned(positions, 4) || !aligned(inv_freq, 8)) return FD_ERR_ALIGN;
    for (int i = 0; i < n; ++i) {
        const Span o = span_of(*out[i], tokens, head_dim);
        for (int j = 0; j < n; ++j) {
            if (!(i == j && in_place(*in[i], *out[i])) && spans_meet(o, span_of(*in[j], tokens, head_dim)))
                return FD_ERR_OVERLAP;
            if (j > i && spans_meet(o, span_of(*out[j], tokens, head_dim))) return FD_ERR_OVERLAP;
        }
        if (span_meets(o, positions, 4ll * tokens) || span_meets(o, inv_freq, 4ll * rot_dim))
            return FD_ERR_OVERLAP;
    }
    if (api_launch_fails()) return api_status(cudaErrorLaunchOutOfResources);
    RopeArgs a{};
    a.q = view(*q), a.q_out = view(*q_out);
    if (k) a.k = view(*k), a.k_out = view(*k_out);
    a.positions = positions, a.inv_freq = inv_freq;
    a.tokens = tokens, a.q_heads = q->heads, a.k_heads = k ? k->heads : 0;
    a.head_dim = head_dim, a.rot_dim = rot_dim, a.interleaved = interleaved != 0, a.scale = scale;
    return api_status(launch_rope(a, false, reinterpret_cast<cudaStream_t>(stream)));
}

int fd_rope_append(const fd_heads *q, const fd_heads *k, const fd_heads *v, const fd_heads *q_out,
                   const fd_paged_cache *cache, const fd_paged_batch *batch, const int *positions,
                   const double *inv_freq, int rot_dim, int interleaved, float scale,
                   fd_stream_t stream) {
    if (!cache || !batch) return FD_ERR_NULL;
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > cache->head_dim || !std::isfinite(scale))
        return FD_ERR_SHAPE;
    if (batch->total_q == 0 || batch->batch == 0) return FD_OK;  // empty: nothing read or written
    if (!q || !k || !v || !q_out || !inv_freq) return FD_ERR_NULL;
    Dim dk[3], dv[3];
    long long kb = 0, vb = 0;
    int st = check_cache(*cache, dk, dv, &kb, &vb);
    if (st == FD_OK) st = check_batch(*batch, cache->page_size);
    const int n = batch->total_q, d = cache->head_dim;
    if (st == FD_OK) st = check_heads(*q, n, d, false);
    if (st == FD_OK) st = check_heads(*k, n, d, false);
    if (st == FD_OK) st = check_heads(*v, n, d, false);
    if (st == FD_OK) st = check_heads(*q_out, n, d, true);
    if (st != FD_OK) return st;
    if (q->heads != q_out->heads || k->heads != cache->kv_heads || v->heads != cache->kv_heads)
        return FD_ERR_SHAPE;
    if (!aligned(positions, 4) || !aligned(inv_freq, 8)) return FD_ERR_ALIGN;
    const Span o = span_of(*q_out, n, d);
    if (!in_place(*q, *q_out) && spans_meet(o, span_of(*q, n, d))) return FD_ERR_OVERLAP;
    for (const fd_heads *x : {q, k, v}) {
        const Span s = span_of(*x, n, d);
        if (x != q && spans_meet(o, s)) return FD_ERR_OVERLAP;
        if (span_meets(s, cache->k, kb) || span_meets(s, cache->v, vb)) return FD_ERR_OVERLAP;
    }
    if (span_meets(o, cache->k, kb) || span_meets(o, cache->v, vb)) return FD_ERR_OVERLAP;
    for (const Span &w : {o, Span{reinterpret_cast<uintptr_t>(cache->k), kb, 0, 0},
                          Span{reinterpret_cast<uintptr_t>(cache->v), vb, 0, 0}})
        if (meets_index(w, *batch) || span_meets(w, inv_freq, 4ll * rot_dim) ||
            (positions && span_meets(w, positions, 4ll * n)))
            return FD_ERR_OVERLAP;
    if (!keys_apart(*cache, dk, dv, kb, vb)) return FD_ERR_OVERLAP;
    if (api_launch_fails()) return api_status(cudaErrorLaunchOutOfResources);
    RopeArgs a{};
    a.q = view(*q), a.k = view(*k), a.v = view(*v), a.q_out = view(*q_out);
    a.k_out = {static_cast<uint16_t *>(cache->k), cache->k_token_stride, cache->k_head_stride};
    a.v_out = {static_cast<uint16_t *>(cache->v), cache->v_token_stride, cache->v_head_stride};
    a.k_page = cache->k_page_stride, a.v_page = cache->v_page_stride;
    a.positions = positions, a.inv_freq = inv_freq;
    a.m = meta(*batch, *cache);
    a.tokens = n, a.q_heads = q->heads, a.k_heads = cache->kv_heads;
    a.head_dim = d, a.rot_dim = rot_dim, a.interleaved = interleaved != 0, a.scale = scale;
    return api_status(launch_rope(a, true, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fd_paged_attention_scratch_bytes(int batch, int total_q, int q_heads, int kv_heads,
                                        int head_dim, int max_q) {
    if (batch < 0 || batch > FD_MAX_BATCH || total_q < 0 || total_q > kMaxTokens || max_q < 0 ||
        q_heads <= 0 || kv_heads <= 0 || q_heads > FD_MAX_HEADS || q_heads % kv_heads != 0 ||
        (head_dim != 64 && head_dim != 128))
        return 0;
    const size_t slots = 2 * kAttnMaxCtas * sizeof(float);
    if (attn_uses_tc(max_q, q_heads / kv_heads, 1.f))
        return kAttnCounterBytes + slots * tc_slot_words(head_dim) + kAttnMaxCtas * sizeof(AttnPart);
    return kAttnCounterBytes + slots * rows_slot_words(head_dim);
}

int fd_paged_attention(const fd_heads *q, const fd_paged_cache *cache, const fd_paged_batch *batch,
                       const fd_heads *out, float *lse, float scale, int causal, int window,
                       float softcap, void *scratch, size_t scratch_bytes, fd_stream_t stream) {
    if (!cache || !batch) return FD_ERR_NULL;
    if (!std::isfinite(scale) || window < 0 || !(softcap >= 0.f) || !std::isfinite(softcap))
        return FD_ERR_SHAPE;
    // what the kernels make of them stays finite
    if (std::fabs(scale) > kMaxScale || (softcap > 0.f && (softcap > kMaxScale || std::fabs(scale) / softcap > kMaxScale)))
        return FD_ERR_UNSUPPORTED;
    // empty: nothing read or written
    if (batch->total_q == 0 || batch->batch == 0 || batch->max_q == 0) return FD_OK;
    if (!q || !out || !scratch) return FD_ERR_NULL;
    Dim dk[3], dv[3];
    long long kb = 0, vb = 0;
    int st = check_cache(*cache, dk, dv, &kb, &vb);
    if (st == FD_OK) st = check_batch(*batch, cache->page_size);
    const int n = batch->total_q, d = cache->head_dim;
    if (st == FD_OK) st = check_heads(*q, n, d, false);
    if (st == FD_OK) st = check_heads(*out, n, d, true);
    if (st != FD_OK) return st;
    if (q->heads != out->heads || q->heads % cache->kv_heads != 0) return FD_ERR_SHAPE;
    if (!aligned(lse, 4) || !aligned(scratch, 16)) return FD_ERR_ALIGN;
    const size_t need = fd_paged_attention_scratch_bytes(batch->batch, n, q->heads, cache->kv_heads, d, batch->max_q);
    if (scratch_bytes < need) return FD_ERR_SHAPE;
    const Span o = span_of(*out, n, d), i = span_of(*q, n, d);
    const long long lse_bytes = 4ll * n * q->heads;
    if (spans_meet(o, i) || span_meets(o, cache->k, kb) || span_meets(o, cache->v, vb) ||
        span_meets(o, scratch, (long long)need) || span_meets(i, scratch, (long long)need))
        return FD_ERR_OVERLAP;
    const Span sc{reinterpret_cast<uintptr_t>(scratch), (long long)need, 0, 0};
    if (span_meets(sc, cache->k, kb) || span_meets(sc, cache->v, vb)) return FD_ERR_OVERLAP;
    if (meets_index(o, *batch) || meets_index(sc, *batch)) return FD_ERR_OVERLAP;
    if (lse) {
        const Span ls{reinterpret_cast<uintptr_t>(lse), lse_bytes, 0, 0};
        if (span_meets(o, lse, lse_bytes) || span_meets(i, lse, lse_bytes) || span_meets(sc, lse, lse_bytes) ||
            span_meets(ls, cache->k, kb) || span_meets(ls, cache->v, vb) || meets_index(ls, *batch))
            return FD_ERR_OVERLAP;
    }
    if (api_launch_fails()) return api_status(cudaErrorLaunchOutOfResources);
    AttnArgs a{};
    a.m = meta(*batch, *cache);
    a.q = view(*q), a.out = view(*out), a.lse = lse;
    a.q_heads = q->heads, a.kv_heads = cache->kv_heads, a.group = q->heads / cache->kv_heads;
    a.head_dim = d, a.causal = causal != 0;
    a.window = window > 2 * FD_MAX_SEQ ? 2 * FD_MAX_SEQ : window;
    a.scale = scale, a.softcap = softcap;
    a.test_timeout = (launch_flags() & FD_LAUNCH_TEST_WAIT_TIMEOUT) != 0;
    a.counters = static_cast<unsigned *>(scratch);
    a.partials = reinterpret_cast<float *>(static_cast<unsigned char *>(scratch) + kAttnCounterBytes);
    const bool tc = attn_uses_tc(a.m.max_q, a.group, scale);
    if (tc) a.parts = reinterpret_cast<AttnPart *>(a.partials + (size_t)2 * kAttnMaxCtas * tc_slot_words(d));
    const int most = tc ? kAttnTcTile : kRowsBox;
    const int box = cache->page_size < most ? cache->page_size : most;
    CUtensorMap mk, mv;
    if (!encode_cache(&mk, cache->k, dk, d, box, &a.ok) || !encode_cache(&mv, cache->v, dv, d, box, &a.ov))
        return api_status(cudaErrorInvalidValue);
    cudaStream_t st_ = reinterpret_cast<cudaStream_t>(stream);
    return api_status(tc ? launch_attn_tc(a, mk, mv, st_) : launch_attn_rows(a, mk, mv, st_));
}

}  // extern "C"
