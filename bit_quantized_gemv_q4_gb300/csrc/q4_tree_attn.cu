// Attention over the paged fp16 cache (q4.h 7c): the call.  The mathematics, the
// schedule and the kernels stand in q4_tree_attn.cuh.
#include "q4_tree_attn.cuh"

using namespace q4i;

extern "C" size_t q4_tree_attention_workspace_bytes(int head_dim) {
    clear_error();
    if (head_dim != 64 && head_dim != 128) {
        fail(Q4_ERR_UNSUPPORTED, "head_dim=%d (64 or 128)", head_dim);
        return 0;
    }
    return head_dim == 128 ? q4x::workspace_bytes<128>() : q4x::workspace_bytes<64>();
}

extern "C" q4_status q4_tree_attention(const q4_tree_attention_desc* desc, q4_stream_t stream) {
    clear_error();
    if (!desc) return fail(Q4_ERR_INVALID_ARG, "desc is NULL");
    q4_tree_attention_desc d = *desc;
    q4x::Args a;
    q4_status st = paged_view(d.cache, d.ctx_len, d.row_start, d.rows, &a.w);
    if (st != Q4_OK) return st;
    const int D = d.cache.head_dim;
    if ((d.rows > 0 && (!d.q || !d.out)) || !d.workspace) return fail(Q4_ERR_INVALID_ARG, "NULL pointer argument");
    if ((st = q4x::attention_args(a, d.mask, d.mask_words, d.q, d.out, d.ldq, d.ldo, d.n_q_heads, d.cache.n_kv_heads, D, d.rows,
                                  d.scale, d.workspace, d.workspace_bytes)) != Q4_OK)
        return st;
    const DeviceInfo* dev = nullptr;
    if ((st = current_device(&dev)) != Q4_OK) return st;
    if (d.rows == 0) return Q4_OK;
    a.w.err = dev->err_word;
    a.ks = a.vs = nullptr;
    a.nb = 0;
    // Rows per kv head of the average sequence choose the kernel.  us of 32
    // sequences up to 4000 (500) positions, 8 kv heads of 128, by mean rows:
    //          jobs of 16   of 32       of 64      tcgen05
    //   11     62 (21)      63 (22)     85 (28)    72 (30)
    //   16     67 (24)      58 (24)     76 (31)    65 (34)
    //   27     78 (30)      61 (27)     73 (32)    62 (32)
    //   32     123 (37)     87 (33)     92 (33)    75 (33)
    //   43     130 (41)     82 (33)     83 (35)    68 (35)
    // The tcgen05 kernel needs TMA; without it 64 beat 32 from some 50 rows on
    // (230 against 265 us at 86).
    const long long avg = ((long long)d.rows * a.G + d.cache.n_seqs - 1) / d.cache.n_seqs;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const q4x::Pools pools = q4x::pools_of(d.cache);
    const char* what = "q4_tree_attention launch";
    // TMA boxes: the greatest power of two that divides a page, 8 at least (a
    // swizzled row group).  TMA / cp.async, us: 40 contexts up to 12000, pages of
    // 8 105 / 121, of 16 94 / 107, of 64 93 / 96; one user's 16000 positions 20 / 29.
    const int even = d.cache.page_size & -d.cache.page_size;
    const long long pool_rows = (long long)d.cache.n_pages * d.cache.n_kv_heads * d.cache.page_size;
    const bool tma = even >= 8 && pool_rows < (1ll << 31) - 1;
    const int ring_box = !tma ? 0 : even < q4x::kKeys ? even : q4x::kKeys;
    if (avg > 32 && tma) {
        const int box = even < q4x::kTcKeys ? even : q4x::kTcKeys;
        return D == 128 ? q4x::launch_tc<128, 0>(a, pools, d.workspace, dev->sms, box, s, what)
                        : q4x::launch_tc<64, 0>(a, pools, d.workspace, dev->sms, box, s, what);
    }
    if (D == 128)
        return avg <= 16   ? q4x::launch<128, 1>(a, pools, d.workspace, dev->sms, ring_box, s, what)
               : avg <= 32 ? q4x::launch<128, 2>(a, pools, d.workspace, dev->sms, ring_box, s, what)
                           : q4x::launch<128, 4>(a, pools, d.workspace, dev->sms, ring_box, s, what);
    return avg <= 16   ? q4x::launch<64, 1>(a, pools, d.workspace, dev->sms, ring_box, s, what)
           : avg <= 32 ? q4x::launch<64, 2>(a, pools, d.workspace, dev->sms, ring_box, s, what)
                       : q4x::launch<64, 4>(a, pools, d.workspace, dev->sms, ring_box, s, what);
}
