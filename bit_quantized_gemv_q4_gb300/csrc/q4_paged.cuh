// Device view of the paged key / value cache (q4.h section 7) and what its
// kernels share: where a position's row is, and which rows a sequence has.
#pragma once

#include <stdint.h>

#include "q4_device.cuh"
#include "q4_internal.h"

namespace q4p {

// Unsigned division of a position (< 2^31) by the page size: q = n / d by one
// high product and a shift.  With s = ceil(log2 d) and m = ceil(2^(31+s) / d)
// (below 2^32, as 2^s / d < 2), n m / 2^(31+s) exceeds n / d by less than
// n / 2^(31+s) <= 1 / 2^s <= 1 / d, so its floor is the quotient.
struct PageDiv {
    uint32_t d = 1, m = 0, s = 0;
};

inline PageDiv page_div(uint32_t d) {
    PageDiv r;
    r.d = d;
    while ((1ull << r.s) < d) ++r.s;
    r.m = (uint32_t)(((1ull << (31 + r.s)) + d - 1) / d);
    return r;
}

__device__ __forceinline__ uint32_t page_of(const PageDiv& v, uint32_t n) {
    return (uint32_t)(((unsigned long long)n * v.m) >> (31 + v.s));
}

struct View {
    uint16_t *k, *v;
    const int32_t* table;
    const int32_t* ctx_len;
    const int32_t* row_start;
    int n_pages, H, S, max_pages, rows;
    PageDiv div;
    int* err;
};

struct Seq {
    int start, n, ctx;  // first row, rows, cached positions
};

// Sizes of sequence s; n = -1 (and `bad` set) where they do not fit.
__device__ __forceinline__ Seq seq_of(const View& w, int s, bool& bad) {
    Seq q;
    q.start = w.row_start[s];
    const int end = w.row_start[s + 1];
    q.ctx = w.ctx_len[s];
    q.n = end - q.start;
    const long long room = (long long)w.max_pages * w.div.d;
    bad = q.start < 0 || end < q.start || end > w.rows || q.ctx < 0 || (long long)q.ctx + q.n > room;
    if (bad) q.n = -1;
    return q;
}

// Element offset of (position, head)'s row in a pool of head_dim D, or -1
// where the page number is outside the pool.
template <typename I>
__device__ __forceinline__ long long row_at(const View& w, int s, I pos, int h, int D) {
    const uint32_t pg = page_of(w.div, (uint32_t)pos);
    const int id = w.table[(size_t)s * w.max_pages + pg];
    if ((uint32_t)id >= (uint32_t)w.n_pages) return -1;
    return (((long long)id * w.H + h) * w.div.d + ((uint32_t)pos - pg * w.div.d)) * D;
}

}  // namespace q4p

namespace q4i {

// Host checks every call on the cache makes; fills the device view.
inline q4_status paged_view(const q4_paged_cache& c, const int32_t* ctx_len, const int32_t* row_start, int rows,
                            q4p::View* w) {
    if (!c.k || !c.v || !c.page_table || !ctx_len || !row_start) return fail(Q4_ERR_INVALID_ARG, "NULL pointer argument");
    if (c.n_pages < 1 || c.page_size < 1 || c.n_kv_heads < 1 || c.n_seqs < 1 || c.max_pages < 1 || rows < 0)
        return fail(Q4_ERR_INVALID_ARG, "n_pages=%d page_size=%d n_kv_heads=%d n_seqs=%d max_pages=%d rows=%d", c.n_pages,
                    c.page_size, c.n_kv_heads, c.n_seqs, c.max_pages, rows);
    if (c.head_dim != 64 && c.head_dim != 128) return fail(Q4_ERR_UNSUPPORTED, "head_dim=%d (64 or 128)", c.head_dim);
    if ((long long)c.n_kv_heads * c.head_dim > (1 << 24) || c.n_seqs > (1 << 27))
        return fail(Q4_ERR_UNSUPPORTED, "%d kv heads of %d, %d sequences", c.n_kv_heads, c.head_dim, c.n_seqs);
    // (the attention's tiles of up to 128 positions then end below 2^31 as well)
    if ((long long)c.max_pages * c.page_size > (1ll << 31) - 128)
        return fail(Q4_ERR_UNSUPPORTED, "max_pages=%d x page_size=%d positions (at most 2^31 - 128)", c.max_pages, c.page_size);
    if (!aligned4(c.page_table, ctx_len, row_start))
        return fail(Q4_ERR_MISALIGNED, "page_table, ctx_len and row_start must be aligned to their elements");
    if (!aligned16(c.k) || !aligned16(c.v)) return fail(Q4_ERR_MISALIGNED, "the cache's pools must be 16-byte aligned");
    w->k = c.k;
    w->v = c.v;
    w->table = c.page_table;
    w->ctx_len = ctx_len;
    w->row_start = row_start;
    w->n_pages = c.n_pages;
    w->H = c.n_kv_heads;
    w->S = c.n_seqs;
    w->max_pages = c.max_pages;
    w->rows = rows;
    w->div = q4p::page_div((uint32_t)c.page_size);
    w->err = nullptr;
    return Q4_OK;
}

// A row matrix [rows][width] with stride ld (0: packed).
inline q4_status row_matrix(const char* name, const void* p, int width, int* ld) {
    if (!*ld) *ld = width;
    if (*ld < width) return fail(Q4_ERR_INVALID_ARG, "row stride of %s is %d, a row has %d elements", name, *ld, width);
    if (*ld % 8 || !aligned16(p)) return fail(Q4_ERR_MISALIGNED, "%s must be 16-byte aligned, its row stride a multiple of 8", name);
    return Q4_OK;
}

}  // namespace q4i
