// cache.hpp -- the 4-bit attention cache: its checks and addresses (include/gptq.h, gptq_cache).
#pragma once
#include "check.hpp"
#include "codes16.hpp"

namespace gptq {

// Pages, positions and rows stay below 2^31; a page's byte offset is 64 bits.
struct CacheView {
    uint8_t* k;
    uint8_t* v;
    uint16_t* ks;
    uint16_t* vs;
    int pages, page, heads;
};

inline bool cache_ok(const gptq_cache* c) {
    return c && c->k && c->v && c->k_scale && c->v_scale && c->pages >= 1 &&
           c->pages <= ((int64_t)1 << 31) - 1 && c->page >= 16 && c->page <= (1 << 20) && c->page % 16 == 0 &&
           c->heads >= 1 && c->heads <= 65535 &&
           c->pages <= ((int64_t)1 << 40) / ((int64_t)c->page * c->heads) && (c->dim == 64 || c->dim == 128 || c->dim == 256) && al16(c->k) &&
           al16(c->v) && al16(c->k_scale) && al16(c->v_scale);
}
inline bool batch_sizes_ok(const gptq_batch* b) {
    return b && b->seqs >= 1 && b->seqs <= (1 << 20) && b->width >= 1 && b->width <= (1 << 24) && b->rows >= 0 &&
           b->rows <= (1 << 23) && (b->start || b->rows == b->seqs);
}
// Positions of a sequence stay below 2^30.
inline bool table_ok(const gptq_cache* c, const gptq_batch* b) {
    return (int64_t)b->width * c->page <= (1 << 30);
}
inline bool batch_ok(const gptq_batch* b) {
    return batch_sizes_ok(b) && b->table && b->len &&
           (((uintptr_t)b->table | (uintptr_t)b->len | (uintptr_t)b->start) & 3u) == 0;
}
// A tensor of rows x heads x dim elements at strides ld, ldh, in either order: 16-byte vectors
// everywhere, no element twice.
inline bool heads_ok(const void* p, int64_t rows, int64_t ld, int64_t ldh, int64_t heads, int dim, int es) {
    const int64_t a = 16 / es, most = (int64_t)1 << 36;
    return al16(p) && ld % a == 0 && ldh % a == 0 && ldh >= dim && ld >= dim && ld <= most && ldh <= most &&
           (ld >= (heads - 1) * ldh + dim || ldh >= (rows - 1) * ld + dim);
}
inline size_t heads_bytes(int64_t rows, int64_t ld, int64_t ldh, int64_t heads, int dim, int es) {
    return (size_t)((rows - 1) * ld + (heads - 1) * ldh + dim) * (size_t)es;
}
// Such a tensor, its heads side by side, as rows of memory; one with other heads is not compared (no rows).
inline RowSet heads_rows(const void* p, int64_t rows, int64_t ld, int64_t ldh, int64_t heads, int dim, int es) {
    return RowSet{p, ld * es, p && (ldh == dim || heads == 1) ? rows : 0, heads * dim * es};
}
// Does a set share a byte with one of the cache's planes?
inline bool meets_cache(const RowSet& t, const gptq_cache* c) {
    const int64_t tokens = c->pages * c->page * c->heads, codes = tokens * (c->dim / 2), scales = tokens * (c->dim / 16);
    return rows_meet(t, RowSet{c->k, codes, 1, codes}) || rows_meet(t, RowSet{c->v, codes, 1, codes}) ||
           rows_meet(t, RowSet{c->k_scale, scales, 1, scales}) || rows_meet(t, RowSet{c->v_scale, scales, 1, scales});
}
inline CacheView cache_view(const gptq_cache* c) {
    return CacheView{c->k, c->v, c->k_scale, c->v_scale, (int)c->pages, c->page, c->heads};
}
inline Batch batch_view(const gptq_batch* b) {
    return Batch{b->table, b->len, b->start, b->seqs, b->width, b->rows};
}
inline void check_cache(const gptq_cache* c, const gptq_batch* b) {
    const size_t tok = (size_t)c->pages * (size_t)c->page * (size_t)c->heads;
    check_buffer(c->k, tok * (size_t)(c->dim / 2), "k");
    check_buffer(c->v, tok * (size_t)(c->dim / 2), "v");
    check_buffer(c->k_scale, tok * (size_t)(c->dim / 16), "k_scale");
    check_buffer(c->v_scale, tok * (size_t)(c->dim / 16), "v_scale");
    check_buffer(b->table, 4 * (size_t)b->seqs * (size_t)b->width, "table");
    check_buffer(b->len, 4 * (size_t)b->seqs, "len");
    if (b->start) check_buffer(b->start, 4 * (size_t)(b->seqs + 1), "start");
}
// Spans of a whole cache plane and of the batch's arrays.
inline Span plane(const void* p, const gptq_cache* c, int64_t per_token, bool write) {
    const int64_t rows = c->pages * c->heads;
    return Span{p, c->page * per_token, rows, c->page * per_token, 1, write, false};
}
inline Span batch_span(const gptq_batch* b, int which) {
    if (which == 0) return rd(b->table, b->width, b->seqs, b->width);
    if (which == 1) return rd(b->len, b->seqs, 1, b->seqs);
    return rd(b->start ? b->start : b->len, b->seqs + 1, b->start ? 1 : 0, b->seqs + 1);
}

// Division by d = page / 16 (up to 2^16) as a product: with 2^b >= d, m = ceil(2^(26 + b) / d) and n < 2^26,
// n m >> 26 + b = floor(n / d), since m d - 2^(26 + b) < d <= 2^b.  A sequence's n, tokens / 16, stay below.
struct PageDiv {
    uint32_t m;
    int shift;
};
inline PageDiv page_div(int page) {
    const uint32_t d = (uint32_t)page / 16;
    int b = 0;
    while ((1u << b) < d) ++b;
    return PageDiv{(uint32_t)(((1ull << (26 + b)) + d - 1) / d), 26 + b};
}

// Index of the (page, head, token) row a position of sequence b is kept in, or -1 where there is
// no such place.
__host__ __device__ __forceinline__ int64_t cache_row(const CacheView& c, const Batch& q, int b, int64_t pos, int head) {
    if (pos < 0 || pos >= (int64_t)q.width * c.page) return -1;
    const int blk = (int)pos / c.page;
    const int page = q.table[(int64_t)b * q.width + blk];
    if ((unsigned)page >= (unsigned)c.pages) return -1;
    return ((int64_t)page * c.heads + head) * c.page + ((int)pos - blk * c.page);
}

}  // namespace gptq
