// Attention over the paged cache in 8 bits (q4.h 9d): the call.  The
// mathematics, the schedule and the kernel for few rows stand in
// q4_tree_attn.cuh.
#include "q4_tree_attn.cuh"

using namespace q4i;

extern "C" q4_status q4_tree_attention8(const q4_tree_attention8_desc* desc, q4_stream_t stream) {
    clear_error();
    if (!desc) return fail(Q4_ERR_INVALID_ARG, "desc is NULL");
    q4_tree_attention8_desc d = *desc;
    q4x::Args a;
    q4p::View8 w8;
    q4_status st = paged_view8(d.cache, d.ctx_len, d.row_start, d.rows, &w8);
    if (st != Q4_OK) return st;
    a.w = w8.w;
    a.ks = w8.ks;
    a.vs = w8.vs;
    a.nb = w8.nb;
    const int D = d.cache.head_dim;
    if ((d.rows > 0 && (!d.q || !d.out)) || !d.workspace) return fail(Q4_ERR_INVALID_ARG, "NULL pointer argument");
    const DeviceInfo* dev = nullptr;
    if ((st = q4x::attention_args(a, d.mask, d.mask_words, d.q, d.out, d.ldq, d.ldo, d.n_q_heads, d.cache.n_kv_heads, D, d.rows,
                                  d.scale, d.workspace, d.workspace_bytes)) != Q4_OK)
        return st;
    if ((st = current_device(&dev)) != Q4_OK) return st;
    if (d.rows == 0) return Q4_OK;
    a.w.err = dev->err_word;
    const long long avg = ((long long)d.rows * a.G + d.cache.n_seqs - 1) / d.cache.n_seqs;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const q4x::Pools pools = q4x::pools_of(d.cache);
    const char* what = "q4_tree_attention8 launch";
    // TMA boxes as in the fp16 cache; the pools' rows are half as long.
    const int even = d.cache.page_size & -d.cache.page_size;
    const long long pool_rows = (long long)d.cache.n_pages * d.cache.n_kv_heads * d.cache.page_size;
    const bool tma = even >= 8 && pool_rows < (1ll << 31) - 1;
    const int box = !tma ? 0 : even < q4x::kKeys ? even : q4x::kKeys;
    // Rows per kv head of the average sequence choose the kernel.  us of 32
    // sequences up to 4000 (500) positions, 8 kv heads of 128, by mean rows:
    //          jobs of 16   tcgen05
    //   10     51           111
    //   18     63           103
    //   26     64           95
    //   32     86 (34)      115 (35)
    //   40     92           104
    //   67     126 (50)     100 (39)
    //   97     205          117
    // (jobs of 32 rows, two CTAs per SM: 74, 70, 74, 111 (32), 102, 135 (42), 213)
    // Of the tcgen05 kernel's forms the one whose keys stay e4m3 converts half as
    // much, and needs more for the products and for each job's query.  us of 16
    // sequences, the longest 6000 (400) positions, 8 kv heads of 128, by mean rows:
    //          keys e4m3    keys fp16
    //   110    100 (31)     118 (26)
    //   175    111          129
    //   250    127 (42)     141 (34)
    //   350    169          179
    //   490    224 (66)     207 (55)
    //   700    337          306
    // so it has up to 384 rows, where the page table holds long contexts.
    if (avg > 48) {
        const int rows = even < 32 ? even : 32;
        const bool lengthy = (long long)d.cache.max_pages * d.cache.page_size >= 2048;
        if (D == 128 && tma && d.cache.page_size % q4p::kBlock == 0 && avg <= 384 && lengthy)
            return q4x::launch_tc<128, 2>(a, pools, d.workspace, dev->sms, rows, s, what);
        return D == 128 ? q4x::launch_tc<128, 1>(a, pools, d.workspace, dev->sms, rows, s, what)
                        : q4x::launch_tc<64, 1>(a, pools, d.workspace, dev->sms, rows, s, what);
    }
    return D == 128 ? q4x::launch<128, 1, true>(a, pools, d.workspace, dev->sms, box, s, what)
                    : q4x::launch<64, 1, true>(a, pools, d.workspace, dev->sms, box, s, what);
}
