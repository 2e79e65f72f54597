// C ABI of the serving operators (declared in include/softmax.h): argument
// checks and dispatch to their launchers.
#include "serving.h"

#include <cmath>
#include <cstdint>

namespace rwsm {
namespace {

constexpr int64_t kMaxCapacity = int64_t{1} << 30;
constexpr int64_t kMaxStride = int64_t{1} << 47;          // elements: products stay in int64
constexpr int64_t kMaxCount = int64_t{1} << 31;           // rows, heads, sequences: below
constexpr int64_t kMaxPacked = kMaxCount - 65536;         // packed rows: a tile past the last
                                                          // one still counts in 32 bits

struct Span {                                            // bytes [a, b)
    uintptr_t a, b;
};

bool meet(const Span& x, const Span& y) { return x.a < y.b && y.a < x.b; }

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride && s % 8 == 0; }

// A [rows][heads][d] tensor that a kernel may read.
bool heads_ok(const softmax_heads_t* t)
{
    return t && t->data && aligned16(t->data) && stride_ok(t->row_stride) &&
           stride_ok(t->head_stride);
}

// Two strided extents whose places (n1 of stride s1, n2 of stride s2, units
// of len elements) are all apart: one nests within the other's stride.
bool places_apart(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t len)
{
    const bool one = n1 <= 1 || (s1 >= len && (n2 <= 1 || s2 >= (n1 - 1) * s1 + len));
    const bool two = n2 <= 1 || (s2 >= len && (n1 <= 1 || s1 >= (n2 - 1) * s2 + len));
    return (n2 <= 1 || s2 >= len) && (n1 <= 1 || s1 >= len) && (one || two);
}

Span span_of(const softmax_heads_t& t, int64_t rows, int64_t heads, int64_t d)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(t.data);
    if (rows <= 0 || heads <= 0)
        return Span{a, a};
    const int64_t last = (rows - 1) * t.row_stride + (heads - 1) * t.head_stride + d;
    return Span{a, a + static_cast<uintptr_t>(last) * 2};
}

bool same(const softmax_heads_t& x, const softmax_heads_t& y)
{
    return x.data == y.data && x.row_stride == y.row_stride && x.head_stride == y.head_stride;
}

// May `out` be written while `in` is read?  Apart in memory, or parts of one
// row layout: the same row stride, and each row's bytes apart from the
// other's rows.
bool apart(const softmax_heads_t& out, int64_t out_rows, int64_t out_heads,
           const softmax_heads_t& in, int64_t in_rows, int64_t in_heads, int64_t d)
{
    const Span o = span_of(out, out_rows, out_heads, d), i = span_of(in, in_rows, in_heads, d);
    if (!meet(o, i))
        return true;
    if (out.row_stride != in.row_stride || out.row_stride == 0)
        return false;
    const int64_t pitch = out.row_stride * 2;
    const int64_t w_out = ((out_heads - 1) * out.head_stride + d) * 2;
    const int64_t w_in = ((in_heads - 1) * in.head_stride + d) * 2;
    // Where a row of `in` begins, past the nearest row of `out` before it.
    const int64_t diff = static_cast<int64_t>(i.a) - static_cast<int64_t>(o.a);
    const int64_t at = ((diff % pitch) + pitch) % pitch;
    return at >= w_out && at + w_in <= pitch;
}

int check_dtype(int dtype, int64_t head_dim)
{
    if (dtype != SOFTMAX_F32 && dtype != SOFTMAX_BF16 && dtype != SOFTMAX_F16)
        return SOFTMAX_ERR_INVALID_ARG;
    if (dtype == SOFTMAX_F32 || (head_dim != 64 && head_dim != 128))
        return SOFTMAX_ERR_UNSUPPORTED;
    return SOFTMAX_OK;
}

// Bytes a cache's k (or v) may touch.
Span cache_span(const void* base, int64_t page, int64_t row, int64_t head,
                const softmax_paged_cache_t& c)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(base);
    if (c.n_pages <= 0)
        return Span{a, a};
    const int64_t last = (c.n_pages - 1) * page + (c.page_size - 1) * row +
                         (c.n_kv_heads - 1) * head + c.head_dim;
    return Span{a, a + static_cast<uintptr_t>(last) * 2};
}

int check_cache(const softmax_paged_cache_t& c, PagedCache* out)
{
    if (c.n_pages < 0 || c.n_pages >= kMaxCount || c.page_size < 1 || c.n_kv_heads < 1 ||
        c.n_kv_heads >= kMaxCount || c.n_seqs < 0 || c.n_seqs >= kMaxCount || c.table_width < 0 ||
        c.table_stride < 0 || c.table_stride > kMaxStride)
        return SOFTMAX_ERR_INVALID_ARG;
    if (c.page_size > kMaxCapacity || c.table_width > kMaxCapacity / c.page_size)
        return SOFTMAX_ERR_INVALID_ARG;
    if (c.n_seqs > 1 && c.table_stride < c.table_width)
        return SOFTMAX_ERR_INVALID_ARG;
    for (int64_t s : {c.k_page_stride, c.k_row_stride, c.k_head_stride, c.v_page_stride,
                      c.v_row_stride, c.v_head_stride})
        if (!stride_ok(s))
            return SOFTMAX_ERR_INVALID_ARG;
    if (c.n_pages > 0 && (!c.k || !c.v || !aligned16(c.k) || !aligned16(c.v)))
        return SOFTMAX_ERR_INVALID_ARG;
    if (c.n_seqs > 0 && c.table_width > 0 &&
        (!c.page_table || reinterpret_cast<uintptr_t>(c.page_table) % 4))
        return SOFTMAX_ERR_INVALID_ARG;
    // Byte extents stay in int64.
    const int64_t lim = INT64_MAX / 8;
    for (int64_t s : {c.k_page_stride, c.v_page_stride})
        if (s > 0 && c.n_pages > lim / s)
            return SOFTMAX_ERR_INVALID_ARG;
    for (int64_t s : {c.k_row_stride, c.v_row_stride})
        if (s > 0 && c.page_size > lim / s)
            return SOFTMAX_ERR_INVALID_ARG;
    for (int64_t s : {c.k_head_stride, c.v_head_stride})
        if (s > 0 && c.n_kv_heads > lim / s)
            return SOFTMAX_ERR_INVALID_ARG;
    *out = PagedCache{c.k, c.v, c.page_table, c.k_page_stride, c.k_row_stride, c.k_head_stride,
                      c.v_page_stride, c.v_row_stride, c.v_head_stride, c.n_seqs, c.table_stride,
                      static_cast<int32_t>(c.n_pages), static_cast<int32_t>(c.table_width),
                      static_cast<int32_t>(c.n_kv_heads),
                      static_cast<int32_t>(c.table_width * c.page_size),
                      divisor_of(static_cast<uint32_t>(c.page_size)), false};
    out->near_rows = c.k_page_stride == c.v_page_stride && c.k_row_stride == c.v_row_stride &&
                     (c.n_pages - 1) * c.k_page_stride + (c.page_size - 1) * c.k_row_stride <
                         (int64_t{8} << 31);
    return SOFTMAX_OK;
}

Heads heads(const softmax_heads_t& t) { return Heads{t.data, t.row_stride, t.head_stride}; }

bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

int status_of(cudaError_t err)
{
    if (err == cudaSuccess)
        return SOFTMAX_OK;
    cudaGetLastError();
    return err == cudaErrorNotSupported ? SOFTMAX_ERR_UNSUPPORTED : SOFTMAX_ERR_CUDA;
}

}  // namespace
}  // namespace rwsm

using namespace rwsm;

extern "C" {

int softmax_kv_append(const softmax_paged_cache_t* cache, const softmax_heads_t* k,
                      const softmax_heads_t* v, const softmax_heads_t* q,
                      const softmax_heads_t* q_out, int64_t n_heads, const int32_t* positions,
                      const int32_t* seq_ids, int64_t n_tokens, const double* inv_freq,
                      int64_t rot_dim, int interleaved, int dtype, void* stream)
{
    if (!cache || n_tokens < 0 || n_tokens >= kMaxCount || rot_dim < 0 ||
        (interleaved != 0 && interleaved != 1) || (q == nullptr) != (q_out == nullptr))
        return SOFTMAX_ERR_INVALID_ARG;
    AppendProblem p = {};
    int st = check_cache(*cache, &p.cache);
    if (st != SOFTMAX_OK)
        return st;
    if (q && (n_heads < 1 || n_heads >= kMaxCount))
        return SOFTMAX_ERR_INVALID_ARG;
    st = check_dtype(dtype, cache->head_dim);
    if (st != SOFTMAX_OK)
        return st;
    const int64_t d = cache->head_dim, nk = cache->n_kv_heads;
    if (rot_dim > d || rot_dim % 16)
        return SOFTMAX_ERR_INVALID_ARG;
    if (n_tokens == 0)
        return SOFTMAX_OK;
    if (!heads_ok(k) || !heads_ok(v) || (q && (!heads_ok(q) || !heads_ok(q_out))))
        return SOFTMAX_ERR_INVALID_ARG;
    if (!positions || !aligned4(positions) || (seq_ids && !aligned4(seq_ids)) ||
        (rot_dim > 0 && (!inv_freq || reinterpret_cast<uintptr_t>(inv_freq) % 8)))
        return SOFTMAX_ERR_INVALID_ARG;
    // The (token, head) rows are counted in 32 bits per CTA of four tokens.
    if (((q ? n_heads : 0) + 2 * nk) * (d / 16) >= (int64_t{1} << 28))
        return SOFTMAX_ERR_UNSUPPORTED;
    // Places of the cache are apart, and nothing that is read is written.
    if (!places_apart(cache->page_size, cache->k_row_stride, nk, cache->k_head_stride, d) ||
        !places_apart(cache->page_size, cache->v_row_stride, nk, cache->v_head_stride, d))
        return SOFTMAX_ERR_INVALID_ARG;
    const Span ck = cache_span(cache->k, cache->k_page_stride, cache->k_row_stride,
                               cache->k_head_stride, *cache);
    const Span cv = cache_span(cache->v, cache->v_page_stride, cache->v_row_stride,
                               cache->v_head_stride, *cache);
    for (const softmax_heads_t* t : {k, v}) {
        const Span x = span_of(*t, n_tokens, nk, d);
        if (meet(x, ck) || meet(x, cv))
            return SOFTMAX_ERR_INVALID_ARG;
    }
    if (q) {
        for (const softmax_heads_t* t : {q, q_out}) {
            const Span x = span_of(*t, n_tokens, n_heads, d);
            if (meet(x, ck) || meet(x, cv))
                return SOFTMAX_ERR_INVALID_ARG;
        }
        if (!places_apart(n_tokens, q_out->row_stride, n_heads, q_out->head_stride, d) ||
            (!same(*q, *q_out) && !apart(*q_out, n_tokens, n_heads, *q, n_tokens, n_heads, d)) ||
            !apart(*q_out, n_tokens, n_heads, *k, n_tokens, nk, d) ||
            !apart(*q_out, n_tokens, n_heads, *v, n_tokens, nk, d))
            return SOFTMAX_ERR_INVALID_ARG;
    }
    if (!usable_device())
        return SOFTMAX_ERR_UNSUPPORTED;
    p.k = heads(*k);
    p.v = heads(*v);
    if (q) {
        p.q = heads(*q);
        p.q_out = heads(*q_out);
        p.n_heads = static_cast<int32_t>(n_heads);
    }
    p.positions = positions;
    p.seq_ids = seq_ids;
    p.inv_freq = inv_freq;
    p.n_tokens = n_tokens;
    p.head_dim = static_cast<int32_t>(d);
    p.rot_dim = static_cast<int32_t>(rot_dim);
    p.interleaved = interleaved;
    p.dtype = dtype;
    return status_of(launch_kv_append(p, static_cast<cudaStream_t>(stream)));
}

int64_t softmax_attention_decode_workspace(int64_t n_seqs, int64_t n_heads, int64_t n_kv_heads,
                                           int64_t head_dim, int64_t capacity)
{
    if (n_seqs < 0 || n_seqs >= kMaxCount || n_heads < 1 || n_heads >= kMaxCount ||
        n_kv_heads < 1 || n_heads % n_kv_heads || (head_dim != 64 && head_dim != 128) ||
        capacity < 0 || capacity > kMaxCapacity)
        return -1;
    if (n_seqs == 0)
        return 0;
    if (!usable_device())
        return -1;
    return static_cast<int64_t>(
        attention_decode_workspace(n_seqs, n_heads, n_kv_heads, head_dim, capacity));
}

int softmax_attention_decode(const softmax_paged_cache_t* cache, const softmax_heads_t* q,
                             const softmax_heads_t* o, float* lse, int64_t n_heads,
                             const int32_t* lengths, float scale, int dtype, void* workspace,
                             size_t workspace_bytes, void* stream)
{
    if (!cache || n_heads < 1 || n_heads >= kMaxCount || !(scale > 0.0f) || !(scale <= 0x1p127f))
        return SOFTMAX_ERR_INVALID_ARG;
    DecodeProblem p = {};
    int st = check_cache(*cache, &p.cache);
    if (st != SOFTMAX_OK)
        return st;
    st = check_dtype(dtype, cache->head_dim);
    if (st != SOFTMAX_OK)
        return st;
    if (n_heads % cache->n_kv_heads)
        return SOFTMAX_ERR_INVALID_ARG;
    if (cache->n_seqs == 0)
        return SOFTMAX_OK;
    const int64_t d = cache->head_dim, b = cache->n_seqs;
    if (!heads_ok(q) || !heads_ok(o) || !lengths || !aligned4(lengths) || (lse && !aligned4(lse)))
        return SOFTMAX_ERR_INVALID_ARG;
    if (!places_apart(b, o->row_stride, n_heads, o->head_stride, d) ||
        (!same(*q, *o) && !apart(*o, b, n_heads, *q, b, n_heads, d)))
        return SOFTMAX_ERR_INVALID_ARG;
    const Span ck = cache_span(cache->k, cache->k_page_stride, cache->k_row_stride,
                               cache->k_head_stride, *cache);
    const Span cv = cache_span(cache->v, cache->v_page_stride, cache->v_row_stride,
                               cache->v_head_stride, *cache);
    const Span so = span_of(*o, b, n_heads, d), sq = span_of(*q, b, n_heads, d);
    if (meet(so, ck) || meet(so, cv))
        return SOFTMAX_ERR_INVALID_ARG;
    const uintptr_t a_lse = reinterpret_cast<uintptr_t>(lse);
    const Span sl{a_lse, a_lse + (lse ? static_cast<uintptr_t>(b * n_heads) * 4 : 0)};
    if (lse) {
        if (meet(sl, so) || meet(sl, sq) || meet(sl, ck) || meet(sl, cv))
            return SOFTMAX_ERR_INVALID_ARG;
    }
    if (!usable_device())
        return SOFTMAX_ERR_UNSUPPORTED;
    const size_t need = attention_decode_workspace(b, n_heads, cache->n_kv_heads, d,
                                                   p.cache.capacity);
    if (need > 0) {
        if (!workspace || !aligned16(workspace) || workspace_bytes < need)
            return SOFTMAX_ERR_INVALID_ARG;
        const uintptr_t a = reinterpret_cast<uintptr_t>(workspace);
        const Span sw{a, a + need};
        if (meet(sw, so) || meet(sw, sq) || meet(sw, sl) || meet(sw, ck) || meet(sw, cv))
            return SOFTMAX_ERR_INVALID_ARG;
    }
    p.q = heads(*q);
    p.o = heads(*o);
    p.lse = lse;
    p.lengths = lengths;
    p.workspace = workspace;
    p.n_seqs = b;
    p.n_heads = static_cast<int32_t>(n_heads);
    p.head_dim = static_cast<int32_t>(d);
    p.dtype = dtype;
    p.scale = scale;
    return status_of(launch_attention_decode(p, static_cast<cudaStream_t>(stream)));
}

int64_t softmax_attention_packed_workspace(int64_t n_seqs, int64_t total_q, int64_t total_k,
                                           int64_t n_heads, int64_t n_kv_heads, int64_t head_dim)
{
    if (n_seqs < 0 || n_seqs >= kMaxCount || total_q < 0 || total_q > kMaxPacked || total_k < 0 ||
        total_k > kMaxPacked || n_heads < 1 || n_heads >= kMaxCount || n_kv_heads < 1 ||
        n_heads % n_kv_heads || (head_dim != 64 && head_dim != 128))
        return -1;
    if (n_seqs == 0 || total_q == 0)
        return 0;
    if (!usable_device())
        return -1;
    return static_cast<int64_t>(
        attention_packed_workspace(n_seqs, total_q, total_k, n_heads, n_kv_heads, head_dim));
}

int softmax_attention_packed(const softmax_heads_t* q, const softmax_heads_t* k,
                             const softmax_heads_t* v, const softmax_heads_t* o, float* lse,
                             const int32_t* cu_q, const int32_t* cu_k, int64_t n_seqs,
                             int64_t total_q, int64_t total_k, int64_t n_heads,
                             int64_t n_kv_heads, int64_t head_dim, float scale, int causal,
                             int dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    if (n_seqs < 0 || n_seqs >= kMaxCount || total_q < 0 || total_q > kMaxPacked || total_k < 0 ||
        total_k > kMaxPacked || n_heads < 1 || n_heads >= kMaxCount || n_kv_heads < 1 ||
        n_heads % n_kv_heads || !(scale > 0.0f) || !(scale <= 0x1p127f) ||
        (causal != 0 && causal != 1))
        return SOFTMAX_ERR_INVALID_ARG;
    const int st = check_dtype(dtype, head_dim);
    if (st != SOFTMAX_OK)
        return st;
    if (n_seqs == 0 || total_q == 0)
        return SOFTMAX_OK;
    const int64_t d = head_dim;
    if (!heads_ok(q) || !heads_ok(o) || (total_k > 0 && (!heads_ok(k) || !heads_ok(v))) ||
        !cu_q || !cu_k || !aligned4(cu_q) || !aligned4(cu_k) || (lse && !aligned4(lse)))
        return SOFTMAX_ERR_INVALID_ARG;
    if (!places_apart(total_q, o->row_stride, n_heads, o->head_stride, d) ||
        (!same(*q, *o) && !apart(*o, total_q, n_heads, *q, total_q, n_heads, d)) ||
        (total_k > 0 && (!apart(*o, total_q, n_heads, *k, total_k, n_kv_heads, d) ||
                         !apart(*o, total_q, n_heads, *v, total_k, n_kv_heads, d))))
        return SOFTMAX_ERR_INVALID_ARG;
    const uintptr_t a_lse = reinterpret_cast<uintptr_t>(lse);
    const Span sl{a_lse, a_lse + (lse ? static_cast<uintptr_t>(total_q * n_heads) * 4 : 0)};
    auto meets_operands = [&](const Span& x) {
        return meet(x, span_of(*o, total_q, n_heads, d)) ||
               meet(x, span_of(*q, total_q, n_heads, d)) ||
               (total_k > 0 && (meet(x, span_of(*k, total_k, n_kv_heads, d)) ||
                                meet(x, span_of(*v, total_k, n_kv_heads, d))));
    };
    if (lse && meets_operands(sl))
        return SOFTMAX_ERR_INVALID_ARG;
    if (!usable_device())
        return SOFTMAX_ERR_UNSUPPORTED;
    const size_t need =
        attention_packed_workspace(n_seqs, total_q, total_k, n_heads, n_kv_heads, d);
    if (need > 0) {
        if (!workspace || !aligned16(workspace) || workspace_bytes < need)
            return SOFTMAX_ERR_INVALID_ARG;
        const uintptr_t a = reinterpret_cast<uintptr_t>(workspace);
        const Span sw{a, a + need};
        if (meet(sw, sl) || meets_operands(sw))
            return SOFTMAX_ERR_INVALID_ARG;
    }
    const Heads none{nullptr, 0, 0};
    const PackedProblem p{heads(*q), total_k > 0 ? heads(*k) : none,
                          total_k > 0 ? heads(*v) : none, heads(*o), lse, cu_q, cu_k, n_seqs,
                          total_q, total_k, static_cast<int32_t>(n_heads),
                          static_cast<int32_t>(n_kv_heads), static_cast<int32_t>(d), causal,
                          dtype, scale, workspace};
    return status_of(launch_attention_packed(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
