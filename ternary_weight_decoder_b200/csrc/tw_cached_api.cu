// tw_cached_api.cu — the C entry points of the paged key-value cache, the
// residual norms and the decoder-layer chain that runs on them: argument
// checks and dispatch.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "tw_device.cuh"
#include "tw_internal.h"

static_assert(TW_KV_MAX_REQUESTS == tw::kAssignMaxRequests, "request limit");

namespace {

int fail(int code, const char *fmt, ...)
{
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return tw::record_error(code, msg);
}

int launched(cudaError_t e, const char *what)
{
    return e == cudaSuccess ? TW_OK : fail(TW_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Whether [a, a + an) and [b, b + bn) share a byte (null: no).
bool overlap(const void *a, int64_t an, const void *b, int64_t bn)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && an > 0 && bn > 0 && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// Whether n rows of aw bytes, al bytes apart, and n of bw, bl apart, share a byte
// (al >= aw, bl >= bw: rows of one buffer side by side do not).
bool rows_overlap(const void *a, int64_t al, int64_t aw, const void *b, int64_t bl, int64_t bw, int64_t n)
{
    if (!overlap(a, (n - 1) * al + aw, b, (n - 1) * bl + bw))
        return false;
    const int64_t to_b = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    // Row i of a and the first of b that ends behind its beginning: j * bl > i * al - to_b - bw
    auto hit = [&](int64_t i, int64_t first) {
        const int64_t after = i * al - to_b - bw;
        const int64_t q = after / bl, j = (after < 0 && after % bl ? q - 1 : q) + 1;   // (the quotient's floor, plus one)
        const int64_t row = j < first ? first : j;
        return row <= first + n - 1 && row * bl < i * al - to_b + aw;
    };
    if (al == bl)   // row 0 of a against every distance between two rows
        return hit(0, -(n - 1)) || hit(0, 0);
    for (int64_t i = 0; i < n; ++i)
        if (hit(i, 0))
            return true;
    return false;
}

int check_cache(const tw_kv_cache *c, const char *who)
{
    if (!c || !c->k || !c->v)
        return fail(TW_ERR_NULL, "%s: cache with key and value pools required", who);
    if (c->dtype != TW_KV_BF16 && c->dtype != TW_KV_F16 && c->dtype != TW_KV_I8)
        return fail(TW_ERR_UNSUPPORTED, "%s: cache type %lld", who, (long long)c->dtype);
    const bool i8 = c->dtype == TW_KV_I8;
    const int64_t unit = i8 ? 16 : 8;   // elements in 16 bytes
    if (c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->num_pages > INT32_MAX ||
        c->page_size > INT32_MAX || c->kv_heads > 65536 || c->num_pages * c->page_size > INT32_MAX)
        return fail(TW_ERR_SHAPE, "%s: %lld pages of %lld tokens, %lld KV heads: all must be >= 1, "
                    "slots below 2^31", who, (long long)c->num_pages, (long long)c->page_size,
                    (long long)c->kv_heads);
    if (c->head_dim < unit || c->head_dim > 256 || c->head_dim % unit)
        return fail(TW_ERR_SHAPE, "%s: head_dim %lld is not a multiple of %lld up to 256", who,
                    (long long)c->head_dim, (long long)unit);
    if (c->page_stride < c->head_dim || c->token_stride < c->head_dim || c->head_stride < c->head_dim)
        return fail(TW_ERR_SHAPE, "%s: cache strides below head_dim", who);
    if (c->page_stride % unit || c->token_stride % unit || c->head_stride % unit ||
        !aligned(c->k, 16) || !aligned(c->v, 16))
        return fail(TW_ERR_ALIGN, "%s: cache pools and strides must be multiples of 16 bytes", who);
    if (i8 && (!c->k_scale || !c->v_scale))
        return fail(TW_ERR_NULL, "%s: a cache of codes needs its scales", who);
    if (i8 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
        return fail(TW_ERR_ALIGN, "%s: scales must be 4-byte aligned", who);
    return TW_OK;
}

struct Bytes {
    const void *p;
    int64_t n;
    const char *name;
};

// An output beside n operands (null: none).
int apart(const Bytes &out, const Bytes *in, int n, const char *who)
{
    for (int i = 0; i < n; ++i)
        if (overlap(out.p, out.n, in[i].p, in[i].n))
            return fail(TW_ERR_SHAPE, "%s: %s overlaps %s", who, out.name, in[i].name);
    return TW_OK;
}

int apart_from_cache(const Bytes &out, const tw_kv_cache &c, const char *who)
{
    const __int128 last = (__int128)(c.num_pages - 1) * c.page_stride + (__int128)(c.page_size - 1) * c.token_stride +
                          (__int128)(c.kv_heads - 1) * c.head_stride + c.head_dim;
    const int64_t pool = (int64_t)(last < INT64_MAX / 4 ? last : INT64_MAX / 4) * (c.dtype == TW_KV_I8 ? 1 : 2);
    const int64_t scales = 4 * c.num_pages * c.page_size * c.kv_heads;
    const Bytes in[] = {{c.k, pool, "the key pool"}, {c.v, pool, "the value pool"},
                        {c.k_scale, scales, "the key scales"}, {c.v_scale, scales, "the value scales"}};
    return apart(out, in, 4, who);
}

int check_rows(const float *p, int64_t ld, int64_t width, const char *who, const char *name)
{
    if (!p)
        return fail(TW_ERR_NULL, "%s: %s required", who, name);
    if (ld < width)
        return fail(TW_ERR_SHAPE, "%s: row stride %lld of %s below its %lld columns", who,
                    (long long)ld, name, (long long)width);
    if (!aligned(p, 16) || ld % 4)
        return fail(TW_ERR_ALIGN, "%s: rows of %s must be 16-byte aligned", who, name);
    return TW_OK;
}

int check_append(const tw::RopeAppend &r, const char *who)
{
    const int64_t wide = (int64_t)r.kv_heads * r.head_dim, q = (int64_t)r.heads * r.head_dim;
    int rc;
    if ((rc = check_rows(r.q, r.ldq, q, who, "q")) || (rc = check_rows(r.k, r.ldk, wide, who, "k")) ||
        (rc = check_rows(r.v, r.ldv, wide, who, "v")) ||
        (rc = check_rows(r.q_out, r.ldqo, q, who, "q_out")))
        return rc;
    if (!r.positions || !r.slots || (r.rotary && !r.inv_freq))
        return fail(TW_ERR_NULL, "%s: positions, slots and inv_freq required", who);
    if (!aligned(r.positions, 4) || !aligned(r.slots, 4) || !aligned(r.inv_freq, 8))
        return fail(TW_ERR_ALIGN, "%s: positions, slots or inv_freq misaligned", who);
    if (r.rotary < 0 || r.rotary > r.head_dim || r.rotary % 8)
        return fail(TW_ERR_SHAPE, "%s: rotary %d is not a multiple of 8 up to head_dim", who, r.rotary);
    if (r.q_out == r.q && r.ldqo != r.ldq)
        return fail(TW_ERR_SHAPE, "%s: q_out is q with another row stride", who);
    // Rows are rotated in no order: what one writes none may read, but its own.
    const struct { const float *p; int64_t ld, width; const char *name; } in[] = {
        {r.q_out == r.q ? nullptr : r.q, r.ldq, q, "q"}, {r.k, r.ldk, wide, "k"}, {r.v, r.ldv, wide, "v"}};
    for (const auto &i : in)
        if (rows_overlap(r.q_out, 4 * r.ldqo, 4 * q, i.p, 4 * i.ld, 4 * i.width, r.rows))
            return fail(TW_ERR_SHAPE, "%s: q_out overlaps %s", who, i.name);
    const Bytes other[] = {{r.positions, 4 * r.rows, "positions"}, {r.slots, 4 * r.rows, "slots"},
                           {r.rotary ? r.inv_freq : nullptr, 4 * r.rotary, "inv_freq"}};
    const Bytes out{r.q_out, 4 * ((r.rows - 1) * r.ldqo + q), "q_out"};
    if (int rc = apart_from_cache(out, r.cache, who))
        return rc;
    return apart(out, other, 3, who);
}

int check_attention(const tw::PagedAttention &p, size_t ws_bytes, const char *who)
{
    const int64_t D = p.cache.head_dim;
    int rc;
    if ((rc = check_rows(p.q, p.ldq, p.heads * D, who, "q")) ||
        (rc = check_rows(p.out, p.ldo, p.heads * D, who, "out")))
        return rc;
    if (!p.block_table || !p.lengths)
        return fail(TW_ERR_NULL, "%s: block table and lengths required", who);
    if (!aligned(p.block_table, 4) || !aligned(p.lengths, 4) || !aligned(p.first, 4) || !aligned(p.lse, 4))
        return fail(TW_ERR_ALIGN, "%s: an int32 or fp32 array is not 4-byte aligned", who);
    if (p.max_pages < 1 || p.max_pages > INT32_MAX || p.table_stride < p.max_pages ||
        p.table_stride > INT32_MAX)
        return fail(TW_ERR_SHAPE, "%s: block table of %lld columns, row stride %lld", who,
                    (long long)p.max_pages, (long long)p.table_stride);
    if (!tw::paged_attention_fits(p.requests, p.heads, p.cache.kv_heads, p.max_pages, p.cache.page_size))
        return fail(TW_ERR_SHAPE, "%s: %lld requests with tables of %lld pages are too many for one call", who,
                    (long long)p.requests, (long long)p.max_pages);
    if (!std::isfinite(p.scale))
        return fail(TW_ERR_NONFINITE, "%s: scale is not finite", who);
    if (rows_overlap(p.out, 4 * p.ldo, 4 * p.heads * D, p.q, 4 * p.ldq, 4 * p.heads * D, p.requests))
        return fail(TW_ERR_SHAPE, "%s: out overlaps q", who);
    const size_t need = (size_t)tw::paged_attention_ws_bytes(D);
    if (!p.ws || ws_bytes < need)
        return fail(TW_ERR_BUFSIZE, "%s: workspace %zu < %zu bytes", who, ws_bytes, need);
    if (!aligned(p.ws, 16))
        return fail(TW_ERR_ALIGN, "%s: workspace must be 16-byte aligned", who);
    // what one block writes no other may read or write
    const int64_t n = 4 * p.requests, q = 4 * ((p.requests - 1) * p.ldq + p.heads * D);
    const Bytes in[] = {{p.block_table, 4 * ((p.requests - 1) * p.table_stride + p.max_pages), "the block table"},
                        {p.lengths, n, "lengths"}, {p.first, n, "first"}, {p.q, q, "q"}};
    const Bytes out[] = {{p.out, 4 * ((p.requests - 1) * p.ldo + p.heads * D), "out"}, {p.lse, n * p.heads, "lse"},
                         {p.ws, (int64_t)need, "the workspace"}};
    for (int i = 0; i < 3; ++i) {
        if ((rc = apart(out[i], in, i == 0 ? 3 : 4, who)) || (rc = apart(out[i], out + i + 1, 2 - i, who)) ||
            (rc = apart_from_cache(out[i], p.cache, who)))
            return rc;
    }
    return TW_OK;
}

// Up to 2^24 rows of up to 2^16 query heads, an equal number for each KV head.
int check_heads(int64_t rows, int64_t heads, int64_t kv_heads, const char *who)
{
    if (rows < 1 || rows > (1 << 24))
        return fail(TW_ERR_SHAPE, "%s: %lld rows outside 1..2^24", who, (long long)rows);
    if (heads < 1 || heads > 65536 || heads % kv_heads)
        return fail(TW_ERR_SHAPE, "%s: %lld query heads over %lld KV heads", who, (long long)heads,
                    (long long)kv_heads);
    return TW_OK;
}

}  // namespace

namespace tw {

int cached_layer_ops(const tw_chain_buffers &b, const tw_chain_cache &c, const tw_cached_layer &L,
                     RopeAppend *append, PagedAttention *attention)
{
    const char *who = "tw_decoder_chain_cached";
    if (int rc = check_cache(&L.cache, who))
        return rc;
    if (L.cache.head_dim != b.head_dim || L.cache.kv_heads * L.cache.head_dim != b.kv_dim)
        return fail(TW_ERR_SHAPE, "%s: cache of %lld heads of %lld, chain of %lld / %lld", who,
                    (long long)L.cache.kv_heads, (long long)L.cache.head_dim, (long long)b.kv_dim,
                    (long long)b.head_dim);
    if (!L.norm_in || !L.norm_mid || !c.norm_out)
        return fail(TW_ERR_NULL, "%s: norm gains required", who);
    if (!aligned(L.norm_in, 4) || !aligned(L.norm_mid, 4) || !aligned(c.norm_out, 4))
        return fail(TW_ERR_ALIGN, "%s: norm gains must be 4-byte aligned", who);
    if (!(c.eps >= 0.f) || !std::isfinite(c.eps))
        return fail(TW_ERR_NONFINITE, "%s: eps must be finite and >= 0", who);
    if (c.rotary < 0 || c.rotary > 256)
        return fail(TW_ERR_SHAPE, "%s: rotary %lld outside 0..256", who, (long long)c.rotary);
    const int heads = (int)(b.hidden / b.head_dim);
    if (int rc = check_heads(b.M, heads, L.cache.kv_heads, who))
        return rc;
    *append = RopeAppend{c.q, c.k, b.v, c.q, b.hidden, b.kv_dim, b.kv_dim, b.hidden, c.positions,
                         c.slots, c.inv_freq, b.M, heads, (int)L.cache.kv_heads,
                         (int)L.cache.head_dim, (int)c.rotary, c.interleaved != 0, L.cache};
    if (int rc = check_append(*append, who))
        return rc;
    *attention = PagedAttention{c.q, b.a, nullptr, b.hidden, b.hidden, c.block_table, c.lengths,
                                c.first, b.M, c.max_pages, c.table_stride, heads, c.scale, L.cache,
                                static_cast<uint8_t *>(c.attention_ws)};
    return check_attention(*attention, c.attention_ws_bytes, who);
}

}  // namespace tw

extern "C" {

int tw_kv_assign(const int32_t *lengths, const int32_t *delta, int64_t requests, int64_t page_size,
                 int32_t *block_table, int64_t max_pages, int64_t table_stride, int32_t *free_pages,
                 int64_t free_capacity, const int32_t *free_count, int32_t *lengths_out,
                 int32_t *free_count_out, int32_t *slots, int32_t *positions,
                 int32_t *request_of_row, int64_t rows, int32_t *row_start, tw_stream_t stream)
{
    tw::clear_error();
    const char *who = "tw_kv_assign";
    if (!lengths || !delta || !block_table || !free_pages || !free_count || !lengths_out ||
        !free_count_out || (rows > 0 && (!slots || !positions || !request_of_row)))
        return fail(TW_ERR_NULL, "%s: a required array is missing", who);
    if (requests < 1 || requests > TW_KV_MAX_REQUESTS)
        return fail(TW_ERR_SHAPE, "%s: %lld requests outside 1..%d", who, (long long)requests,
                    TW_KV_MAX_REQUESTS);
    if (page_size < 1 || page_size > INT32_MAX || max_pages < 1 || max_pages > INT32_MAX ||
        table_stride < max_pages || table_stride > INT32_MAX || free_capacity < 1 ||
        free_capacity > INT32_MAX || rows < 0 || rows > INT32_MAX)
        return fail(TW_ERR_SHAPE, "%s: page size %lld, %lld table columns (row stride %lld), free "
                    "list of %lld, %lld rows", who, (long long)page_size, (long long)max_pages,
                    (long long)table_stride, (long long)free_capacity, (long long)rows);
    const int64_t n = 4 * requests;
    const struct { const void *p; int64_t bytes; const char *name; } arr[] = {
        {delta, n, "delta"}, {block_table, 4 * ((requests - 1) * table_stride + max_pages), "block_table"},
        {free_pages, 4 * free_capacity, "free_pages"}, {lengths_out, n, "lengths_out"},
        {free_count_out, 4, "free_count_out"}, {slots, 4 * rows, "slots"},
        {positions, 4 * rows, "positions"}, {request_of_row, 4 * rows, "request_of_row"},
        {row_start, n + 4, "row_start"}, {lengths, n, "lengths"}, {free_count, 4, "free_count"}};
    constexpr int kArr = sizeof(arr) / sizeof(arr[0]);
    for (int i = 0; i < kArr; ++i) {
        if (!aligned(arr[i].p, 4))
            return fail(TW_ERR_ALIGN, "%s: %s is not 4-byte aligned", who, arr[i].name);
        for (int j = i + 1; j < kArr; ++j) {
            const bool same = arr[i].p == arr[j].p &&
                              ((arr[i].p == lengths_out && arr[j].p == lengths && j == 9 && i == 3) ||
                               (i == 4 && j == 10));
            if (!same && overlap(arr[i].p, arr[i].bytes, arr[j].p, arr[j].bytes))
                return fail(TW_ERR_SHAPE, "%s: %s overlaps %s", who, arr[i].name, arr[j].name);
        }
    }
    uint32_t *err = nullptr;
    if (int rc = tw::error_word(&err))
        return rc;
    const tw::KvAssign a{lengths, delta, block_table, free_pages, free_count, lengths_out,
                         free_count_out, slots, positions, request_of_row, row_start, requests,
                         page_size, max_pages, table_stride, free_capacity, rows};
    return launched(tw::launch_kv_assign(a, err, stream), "cache assignment launch");
}

int tw_rope_append(const float *q, int64_t ldq, const float *k, int64_t ldk, const float *v,
                   int64_t ldv, int64_t rows, int64_t heads, int64_t rotary, const double *inv_freq,
                   int interleaved, const int32_t *positions, const int32_t *slots,
                   const tw_kv_cache *cache, float *q_out, int64_t ldqo, tw_stream_t stream)
{
    tw::clear_error();
    const char *who = "tw_rope_append";
    if (int rc = check_cache(cache, who))
        return rc;
    if (int rc = check_heads(rows, heads, cache->kv_heads, who))
        return rc;
    if (rotary < 0 || rotary > 256)
        return fail(TW_ERR_SHAPE, "%s: rotary %lld outside 0..256", who, (long long)rotary);
    const tw::RopeAppend r{q, k, v, q_out, ldq, ldk, ldv, ldqo, positions, slots, inv_freq, rows,
                           (int)heads, (int)cache->kv_heads, (int)cache->head_dim, (int)rotary,
                           interleaved != 0, *cache};
    if (int rc = check_append(r, who))
        return rc;
    uint32_t *err = nullptr;
    if (int rc = tw::error_word(&err))
        return rc;
    return launched(tw::launch_rope_append(r, err, stream), "cache append launch");
}

size_t tw_paged_attention_workspace_bytes(int64_t requests, int64_t heads, int64_t kv_heads,
                                          int64_t head_dim)
{
    if (requests < 1 || requests > (1 << 24) || heads < 1 || heads > 65536 || kv_heads < 1 ||
        heads % kv_heads || head_dim < 8 || head_dim > 256)
        return 0;
    return (size_t)tw::paged_attention_ws_bytes(head_dim);
}

int tw_paged_attention(const float *q, int64_t ldq, int64_t requests, int64_t heads,
                       const tw_kv_cache *cache, const int32_t *block_table, int64_t max_pages,
                       int64_t table_stride, const int32_t *lengths, const int32_t *first,
                       float scale, float *out, int64_t ldo, float *lse, void *ws, size_t ws_bytes,
                       tw_stream_t stream)
{
    tw::clear_error();
    const char *who = "tw_paged_attention";
    if (int rc = check_cache(cache, who))
        return rc;
    if (int rc = check_heads(requests, heads, cache->kv_heads, who))
        return rc;
    const tw::PagedAttention p{q, out, lse, ldq, ldo, block_table, lengths, first, requests, max_pages,
                               table_stride, (int)heads, scale, *cache, static_cast<uint8_t *>(ws)};
    if (int rc = check_attention(p, ws_bytes, who))
        return rc;
    uint32_t *err = nullptr;
    if (int rc = tw::error_word(&err))
        return rc;
    return launched(tw::launch_paged_attention(p, err, stream), "paged attention launch");
}

int tw_residual_norm(const tw_residual_norm_args *g, tw_stream_t stream)
{
    tw::clear_error();
    const char *who = "tw_residual_norm";
    if (!g || !g->x)
        return fail(TW_ERR_NULL, "%s: x required", who);
    if (!g->h && !g->n && !g->xq)
        return fail(TW_ERR_NULL, "%s: one output at least required", who);
    if ((g->xq != nullptr) != (g->amax != nullptr) || (g->qsum && !g->xq))
        return fail(TW_ERR_NULL, "%s: xq and amax go together, qsum with them", who);
    if (g->M < 1 || g->M > (1 << 24) || g->K < 1 || g->K > tw::kNormMaxK)
        return fail(TW_ERR_SHAPE, "%s: M=%lld K=%lld outside 1..2^24, 1..%lld", who, (long long)g->M,
                    (long long)g->K, (long long)tw::kNormMaxK);
    const int32_t kinds[] = {g->post, g->pre};
    for (int32_t k : kinds)
        if (k != TW_NORM_NONE && k != TW_NORM_RMS && k != TW_NORM_LAYER)
            return fail(TW_ERR_UNSUPPORTED, "%s: norm %d", who, k);
    if ((g->post_bias && g->post != TW_NORM_LAYER) || (g->pre_bias && g->pre != TW_NORM_LAYER) ||
        (g->post_weight && g->post == TW_NORM_NONE) || (g->pre_weight && g->pre == TW_NORM_NONE))
        return fail(TW_ERR_SHAPE, "%s: a weight or bias without its norm", who);
    if (!g->y && (g->gate || g->post != TW_NORM_NONE))
        return fail(TW_ERR_NULL, "%s: gate and post norm need y", who);
    if (!std::isfinite(g->alpha) || !(g->eps >= 0.f) || !std::isfinite(g->eps))
        return fail(TW_ERR_NONFINITE, "%s: alpha must be finite, eps finite and >= 0", who);
    const int64_t K = g->K, M = g->M;
    if (g->ldx < K || (g->y && g->ldy < K) || (g->gate && g->ldgate != 0 && g->ldgate < K) ||
        (g->h && g->ldh < K) || (g->n && g->ldn < K))
        return fail(TW_ERR_SHAPE, "%s: a row stride is below K=%lld", who, (long long)K);
    const struct { const void *p; int64_t ld; const char *name; } in[] = {
        {g->x, g->ldx, "x"}, {g->y, g->ldy, "y"}, {g->gate, g->ldgate, "gate"},
        {g->post_weight, 0, "post_weight"}, {g->post_bias, 0, "post_bias"},
        {g->pre_weight, 0, "pre_weight"}, {g->pre_bias, 0, "pre_bias"}};
    const struct { const void *p; int64_t ld; int64_t bytes; const char *name; } out[] = {
        {g->h, g->ldh, 4 * ((M - 1) * g->ldh + K), "h"}, {g->n, g->ldn, 4 * ((M - 1) * g->ldn + K), "n"},
        {g->xq, K, M * K, "xq"}, {g->amax, 1, 4 * M, "amax"}, {g->qsum, 1, 4 * M, "qsum"}};
    for (const auto &i : in)
        if (!aligned(i.p, 4))
            return fail(TW_ERR_ALIGN, "%s: %s is not 4-byte aligned", who, i.name);
    for (int o = 0; o < 5; ++o) {
        if (o != 2 && !aligned(out[o].p, 4))
            return fail(TW_ERR_ALIGN, "%s: %s is not 4-byte aligned", who, out[o].name);
        for (int i = 0; i < 7; ++i) {
            // a row of x or y may be overwritten by that row of h or n
            const bool in_place = o < 2 && i < 2 && in[i].p == out[o].p && in[i].ld == out[o].ld;
            if (!in_place && overlap(in[i].p, 4 * ((M - 1) * in[i].ld + K), out[o].p, out[o].bytes))
                return fail(TW_ERR_SHAPE, "%s: %s overlaps %s", who, out[o].name, in[i].name);
        }
        for (int p = o + 1; p < 5; ++p)
            if (overlap(out[o].p, out[o].bytes, out[p].p, out[p].bytes))
                return fail(TW_ERR_SHAPE, "%s: %s overlaps %s", who, out[o].name, out[p].name);
    }
    uint32_t *err = nullptr;
    if (int rc = tw::error_word(&err))
        return rc;
    tw::ResidualNorm a{};
    a.x = g->x, a.y = g->y, a.post_w = g->post_weight, a.post_b = g->post_bias, a.gate = g->gate;
    a.pre_w = g->pre_weight, a.pre_b = g->pre_bias, a.h = g->h, a.n = g->n, a.xq = g->xq;
    a.amax = g->amax, a.qsum = g->qsum, a.M = M, a.K = K, a.ldx = g->ldx, a.ldy = g->y ? g->ldy : 0;
    a.ldg = g->gate ? g->ldgate : 0, a.ldh = g->h ? g->ldh : 0, a.ldn = g->n ? g->ldn : 0;
    a.post = g->y ? g->post : TW_NORM_NONE, a.pre = g->pre, a.alpha = g->alpha, a.eps = g->eps;
    return launched(tw::launch_residual_norm(a, stream), "residual norm launch");
}

}  // extern "C"
