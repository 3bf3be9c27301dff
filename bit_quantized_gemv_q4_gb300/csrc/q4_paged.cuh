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

// Sequence of a row: the number of sequences whose end is at or before it, by
// a search 32 ways wide (one load per lane and level).  All lanes get it.  Where
// the starts are not in order it can be another (or none): the caller checks.
__device__ __forceinline__ int seq_of_row(const View& w, int row, int lane) {
    int lo = 0, len = w.S;
    while (len > 0) {
        const int stride = (len + 31) / 32;
        const int i = lane * stride + stride - 1;
        const bool before = i < len && w.row_start[lo + i + 1] <= row;
        const int c = __popc(__ballot_sync(0xffffffffu, before));
        lo += c * stride;
        len = min(stride - 1, len - c * stride);
    }
    return lo;
}

__device__ __forceinline__ bool holds(const View& w, int s, int row, Seq& q) {
    bool bad;
    q = seq_of(w, s, bad);
    return !bad && row >= q.start && row < q.start + q.n;
}

// ---- acceptance: blocks of a sequence's cluster, and the path ---------------
constexpr int kAcceptThreads = 512;
constexpr int kAcceptCluster = 8;
constexpr int kMaxTree = 4096;

// By a whole block: the accepted path of a tree of n rows (n <= kMaxTree) into
// `path`, its length into *len.  Every row in parallel looks whether it
// continues its parent (its token is the one sampled there), the smallest such
// row of a parent wins (an integer minimum, the same in any order), then one
// thread follows the pointers.
__device__ __forceinline__ void walk_tree(const int32_t* draft, const int32_t* parents, const int32_t* sampled, int n,
                                          int32_t* next, int32_t* path, int* len) {
    const int tid = threadIdx.x;
    for (int i = tid; i < n; i += kAcceptThreads) next[i] = 0x7fffffff;
    __syncthreads();
    for (int i = 1 + tid; i < n; i += kAcceptThreads) {
        const int up = parents[i];
        if (up >= 0 && up < i) {
            const int t = sampled[up];
            if (t >= 0 && t == draft[i]) atomicMin(&next[up], i);
        }
    }
    __syncthreads();
    if (tid == 0) {
        int k = 0;
        for (int at = 0; at < n; at = next[at]) path[k++] = at;  // ascending: next[at] > at
        *len = k;
    }
    __syncthreads();
}

// ---- the cache in 8 bits (q4.h section 9) -------------------------------------
constexpr int kBlock = Q4_CACHE8_BLOCK;

struct View8 {
    View w;  // its pools are not used
    uint8_t *k, *v;
    float *ks, *vs;
    int nb;  // blocks of a page
};

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

// Likewise for the cache in 8 bits.
inline q4_status paged_view8(const q4_paged_cache8& c, const int32_t* ctx_len, const int32_t* row_start, int rows,
                             q4p::View8* w) {
    const q4_paged_cache pools = {reinterpret_cast<uint16_t*>(c.k), reinterpret_cast<uint16_t*>(c.v), c.page_table, c.n_pages,
                                  c.page_size, c.n_kv_heads, c.head_dim, c.n_seqs, c.max_pages};
    const q4_status st = paged_view(pools, ctx_len, row_start, rows, &w->w);
    if (st != Q4_OK) return st;
    if (!c.k_scales || !c.v_scales) return fail(Q4_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned4(c.k_scales, c.v_scales)) return fail(Q4_ERR_MISALIGNED, "the scales must be 4-byte aligned");
    w->k = c.k;
    w->v = c.v;
    w->ks = c.k_scales;
    w->vs = c.v_scales;
    w->nb = (c.page_size - 1) / q4p::kBlock + 1;
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
