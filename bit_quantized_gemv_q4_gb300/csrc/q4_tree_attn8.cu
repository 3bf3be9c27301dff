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
    // Rows per kv head of the average sequence choose the kernel, and, of the
    // tcgen05 kernel's forms, with the page table's length whether the keys stay
    // e4m3: that converts half as much, and needs more for the products of 256 rows
    // and for a job's query.  us of 16 sequences, 8 kv heads of 128, the longest
    // 20000 / 6000 / 2000 / 500 positions, by mean rows (which vary by a tenth or
    // so between the lengths):
    //         jobs of 16             keys e4m3              keys fp16
    //   38    176 / 69 / 37 / 22     159 / 73 / 44 / 31     244 / 86 / 46 / 25
    //   51    241 / 92 / 41 / 27     166 / 78 / 45 / 30     248 / 90 / 42 / 25
    //   85    326 / 120 / 52 / 35    150 / 74 / 43 / 26     214 / 85 / 42 / 26
    //   117   436 / 184 / 68 / 40    173 / 96 / 49 / 33     217 / 93 / 47 / 29
    //   135   528 / 191 / 74 / 48    204 / 97 / 49 / 35     227 / 99 / 47 / 29
    //   175   698 / 215 / 93 / 53    214 / 104 / 55 / 33    192 / 94 / 50 / 29
    // (jobs of 32 rows instead of 16, two CTAs per SM, were slower at all sizes; at
    // 38 rows over 20000 positions the border of 48 is the slower side by a tenth)
    // Heads of 64, jobs of 16 / keys fp16:
    //   21    79 / 135, 28 / 50, 19 / 33, 14 / 20
    //   39    105 / 125, 35 / 45, 26 / 31, 16 / 20
    //   52    109 / 120, 54 / 56, 26 / 31, 18 / 20
    //   78    164 / 132, 63 / 53, 29 / 31, 22 / 21
    //   116   298 / 152, 106 / 65, 51 / 39, 26 / 24
    // Sequences without rows count in the average, as the host does not see the
    // sizes: 4 sequences of up to 64 rows over 6000 positions 40 us, among 60 idle
    // places, in jobs of 16 rows, 91.
    if (avg > 48) {
        const int rows = even < 32 ? even : 32;
        const bool lengthy = (long long)d.cache.max_pages * d.cache.page_size >= 4096;
        if (D == 128 && tma && d.cache.page_size % q4p::kBlock == 0 && avg <= 168 && lengthy)
            return q4x::launch_tc<128, 2>(a, pools, d.workspace, dev->sms, rows, s, what);
        return D == 128 ? q4x::launch_tc<128, 1>(a, pools, d.workspace, dev->sms, rows, s, what)
                        : q4x::launch_tc<64, 1>(a, pools, d.workspace, dev->sms, rows, s, what);
    }
    return D == 128 ? q4x::launch<128, 1, true>(a, pools, d.workspace, dev->sms, box, s, what)
                    : q4x::launch<64, 1, true>(a, pools, d.workspace, dev->sms, box, s, what);
}
