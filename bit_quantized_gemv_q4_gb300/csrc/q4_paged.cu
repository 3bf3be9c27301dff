// The paged key / value cache: rotary frequencies, the append that rotates,
// and the acceptance of a drafted tree (q4.h 7a, 7b, 7d).
//
// BaseRT: optimal LLM inference on Apple Silicon with native Metal, §3.3
// lists RoPE among the decode kernels and §3.2 preallocates the cache; the
// pages describe neither a cache of pages nor drafted tokens.
#include <cuda_fp16.h>
#include <math.h>

#include "q4_paged.cuh"

namespace q4p {

// ------------------------------------------------------------- frequencies ---
// Once per model, so plain fp64: turns f / 2 pi < 1, scaled to 2^64.  The
// relative error of the fp64 power (a few 2^-53) times a position stays below
// 2^-20 turns up to position 2^31.
__global__ void rope_freq_kernel(q4_rope_desc d, uint64_t* __restrict__ out) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= d.rot_dim / 2) return;
    double f = pow(d.theta, -2.0 * i / d.rot_dim) * 0.15915494309189533577;  // / 2 pi
    if (d.factor > 1.0) {
        double c = 0.0;
        if (d.orig_len > 0) c = fmin(1.0, fmax(0.0, (d.orig_len * f - d.alpha) / (d.beta - d.alpha)));
        f = f * c + f / d.factor * (1.0 - c);
    }
    out[i] = (uint64_t)rint(f * 18446744073709551616.0);
}

// ------------------------------------------------------------------ append ---
// One block per row.  The angle of pair i is the fraction of a turn
// (position * freqs[i]) mod 2^64, exact in integers; its upper 32 bits, signed,
// are x 2^-31 half turns in [-1, 1), which sincospif takes without any
// reduction (an error of 2^-32 turns = 1.5e-9 rad from the bits left off).
// The table of a row's (cos, sin) is built once in shared memory and used by
// every head.
constexpr int kAppendThreads = 256;

struct AppendArgs {
    View w;
    const int32_t* positions;
    const uint16_t *k, *v, *q;
    uint16_t* q_out;
    long long ldk, ldv, ldq, ldqo;
    int Hq;
    const uint64_t* freqs;
    int rot;
    float amplitude;
    PageDiv by_per;  // division by a rotated head's items
};

// Where a row goes.
constexpr int kNobody = 0x7fffffff;
struct At {
    long long base;  // head 0's row in the pools (-1: no memory)
    int slot;        // position
    int seq;         // sequence (kNobody: nobody's row)
};

__device__ __forceinline__ void place(const View& w, const Seq& q, int row, int D, At& at) {
    at.slot = q.ctx + (row - q.start);
    at.base = row_at(w, at.seq, at.slot, 0, D);
    if (at.base < 0) atomicOr(w.err, q4d::kErrDeviceCheck);
}

// By the whole block, where the search has found nobody: a row that is nobody's,
// or a search led astray by a sequence that does not fit.  Takes the first of all
// sequences that holds the row, false if none does.
__device__ __noinline__ bool find_holder(const View& w, int row, int D, At& at) {
    __syncthreads();  // all have seen that it found nobody
    Seq q;
    for (int s = threadIdx.x; s < w.S; s += kAppendThreads)
        if (holds(w, s, row, q)) atomicMin(&at.seq, s);
    __syncthreads();
    if (at.seq == kNobody) return false;
    if (threadIdx.x == 0 && holds(w, at.seq, row, q)) place(w, q, row, D, at);
    __syncthreads();
    return true;
}

__device__ __forceinline__ float h2f(uint32_t w, int hi) {
    return __half2float(__ushort_as_half((uint16_t)(hi ? w >> 16 : w)));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// kPairs: how a 16-byte chunk finds its partners.  0: neighbours (the chunk
// holds whole pairs); 1: the halves of the rotated part are whole chunks, a
// thread turns a chunk of each; 2: halves of any even length, element by
// element.
//
// What bounds it: the bytes, once the latency of a block is covered.  A block
// lives for a chain of dependent loads (the row's sequence, its sizes, the
// page, and beside that the frequencies), so each thread fetches its first
// kAhead items of data before anything else, one warp looks the row up and
// two others compute the angles meanwhile.
//
// Measured: 6767 rows of 32 query and 8 kv heads of 128 (166 MB in and out)
// 30.7 us = 5.4 TB/s, 80 % of the measured copy rate; 478 rows 3.6 us, one row
// 2.8 us, which is a launch.  kAhead 1 / 2 / 4: 31.4 / 30.5 / 42 us (4 spills);
// 8 blocks per SM or 6: 30.5 / 31.9 us (both before the last 0.5 us).
constexpr int kAhead = 2;

template <int D, int kPairs>
__global__ void __launch_bounds__(kAppendThreads, 8) append_kernel(const __grid_constant__ AppendArgs p) {
    __shared__ __align__(16) float2 cs[D / 2];
    __shared__ At at_s;
    const int row = blockIdx.x, tid = threadIdx.x;
    constexpr int NC = D / 8;
    const int half = p.rot / 2, rc = half / 8;          // kPairs 1: chunks of a half
    const int per = kPairs == 1 ? NC - rc : NC;         // items of a rotated head
    const int nq = p.Hq * per, nk = p.w.H * per, items = nq + nk + p.w.H * NC;
    // Item x: a chunk (with its partner, kPairs 1) of a query or key head, or
    // a chunk of the values.
    struct Item {
        int h, c;   // head, chunk
        int kind;   // 0 query, 1 key, 2 value
    };
    const auto item = [&](int x) {
        Item t;
        const int y = x < nq ? x : x < nq + nk ? x - nq : x - nq - nk;
        t.kind = x < nq ? 0 : x < nq + nk ? 1 : 2;
        if (t.kind == 2) {
            t.h = y / NC;
            t.c = y % NC;
        } else {
            t.h = (int)page_of(p.by_per, y);
            t.c = y - t.h * per;
        }
        return t;
    };
    const auto source = [&](const Item& t) {
        const uint16_t* m = t.kind == 0 ? p.q + row * p.ldq : t.kind == 1 ? p.k + row * p.ldk : p.v + row * p.ldv;
        return m + (long long)t.h * D;
    };
    const auto fetch = [&](const Item& t, uint4& a, uint4& b) {
        const uint16_t* src = source(t);
        if (kPairs == 1 && t.kind != 2) {
            if (t.c < rc) b = *reinterpret_cast<const uint4*>(src + 8 * (t.c + rc));
            a = *reinterpret_cast<const uint4*>(src + 8 * (t.c < rc ? t.c : t.c + rc));
        } else if (kPairs != 2 || t.kind == 2) {
            a = *reinterpret_cast<const uint4*>(src + 8 * t.c);
        }
    };
    uint4 a0[kAhead], b0[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (tid + i * kAppendThreads < items) fetch(item(tid + i * kAppendThreads), a0[i], b0[i]);

    const auto angle = [&](int i, long long pos) {
        const uint64_t turn = (uint64_t)pos * p.freqs[i];
        float sn, cn;
        sincospif((float)(int32_t)(uint32_t)(turn >> 32) * 4.656612873077393e-10f, &sn, &cn);
        cs[i] = make_float2(cn * p.amplitude, sn * p.amplitude);
    };
    if (tid < 32) {
        const int s = seq_of_row(p.w, row, tid);
        if (tid == 0) {
            Seq q;
            const bool mine = s < p.w.S && holds(p.w, s, row, q);
            at_s.seq = mine ? s : kNobody;
            if (mine) place(p.w, q, row, D, at_s);
        }
    } else if (tid >= 64 && tid < 64 + half && p.positions) {
        angle(tid - 64, p.positions[row]);
    } else if (tid >= 128 && row == 0) {
        // the first row's block latches the sequences that do not fit
        for (int s = tid - 128; s < p.w.S; s += kAppendThreads - 128) {
            bool bad;
            seq_of(p.w, s, bad);
            if (bad) atomicOr(p.w.err, q4d::kErrDeviceCheck);
        }
    }
    __syncthreads();
    if (at_s.seq == kNobody && !find_holder(p.w, row, D, at_s)) return;
    const int slot = at_s.slot;
    if (!p.positions && half > 0) {
        if (tid < half) angle(tid, slot);
        __syncthreads();
    }
    const long long base = at_s.base, head_step = (long long)p.w.div.d * D;
    const auto finish = [&](const Item& t, uint4 a, const uint4& b) {
        uint16_t* dst = t.kind == 0   ? p.q_out + row * p.ldqo + (long long)t.h * D
                        : t.kind == 1 ? p.w.k + base + t.h * head_step
                                      : p.w.v + base + t.h * head_step;
        if (t.kind != 0 && base < 0) return;
        if (t.kind == 2) {
            *reinterpret_cast<uint4*>(dst + 8 * t.c) = a;
            return;
        }
        uint32_t wa[4] = {a.x, a.y, a.z, a.w};
        if constexpr (kPairs == 1) {
            if (t.c >= rc) {  // behind the rotated part
                *reinterpret_cast<uint4*>(dst + 8 * (t.c + rc)) = a;
                return;
            }
            const uint32_t wb[4] = {b.x, b.y, b.z, b.w};
            uint32_t oa[4], ob[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 r = *reinterpret_cast<const float4*>(&cs[8 * t.c + 2 * e]);
                const float x0 = h2f(wa[e], 0), x1 = h2f(wa[e], 1), y0 = h2f(wb[e], 0), y1 = h2f(wb[e], 1);
                oa[e] = pack2(x0 * r.x - y0 * r.y, x1 * r.z - y1 * r.w);
                ob[e] = pack2(y0 * r.x + x0 * r.y, y1 * r.z + x1 * r.w);
            }
            *reinterpret_cast<uint4*>(dst + 8 * t.c) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
            *reinterpret_cast<uint4*>(dst + 8 * (t.c + rc)) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
        } else if constexpr (kPairs == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * t.c + e;  // pair
                if (i < half) {
                    const float2 r = cs[i];
                    const float x = h2f(wa[e], 0), y = h2f(wa[e], 1);
                    wa[e] = pack2(x * r.x - y * r.y, y * r.x + x * r.y);
                }
            }
            *reinterpret_cast<uint4*>(dst + 8 * t.c) = make_uint4(wa[0], wa[1], wa[2], wa[3]);
        } else {
            // pairs (i, i + half) cross the chunks; in place (q_out == q) a
            // thread must own both elements of a pair, so an item is every
            // NC-th pair here, and every NC-th element behind them
            const uint16_t* src = source(t);
            for (int i = t.c; i < half; i += NC) {
                const float x = __half2float(__ushort_as_half(src[i]));
                const float y = __half2float(__ushort_as_half(src[i + half]));
                const float2 r = cs[i];
                dst[i] = __half_as_ushort(__float2half_rn(x * r.x - y * r.y));
                dst[i + half] = __half_as_ushort(__float2half_rn(y * r.x + x * r.y));
            }
            for (int i = p.rot + t.c; i < D; i += NC) dst[i] = src[i];
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (tid + i * kAppendThreads < items) finish(item(tid + i * kAppendThreads), a0[i], b0[i]);
    for (int x = tid + kAhead * kAppendThreads; x < items; x += kAppendThreads) {
        const Item t = item(x);
        uint4 a = {}, b = {};
        fetch(t, a, b);
        finish(t, a, b);
    }
}

// -------------------------------------------------------------- acceptance ---
// A cluster of 8 blocks per sequence.  Each block finds the path for itself:
// every row in parallel looks whether it continues its parent (its token is
// the one sampled there) and the smallest such row of a parent wins (an
// integer minimum, the same in any order), then one thread follows the
// pointers.  The blocks share the columns (layer, keys or values, head,
// 16-byte chunk) to move: a thread moves its column's rows of the whole path,
// and as paths ascend (path[i] >= i, path[j] > path[i] for j > i) no row is
// written before the same column's later sources are past it.  ctx_out may be
// ctx_len, so it is written after every block of the cluster has read it.
//
// What bounds it: a chain of dependent loads (sizes, the tokens and parents, the
// path, its pages, its rows) and, for many sequences, the rows' bytes.  28
// layers of 8 heads of 128, one sequence of 16 rows 5.3 us, 32 of up to 64 rows
// (27 MB) 10.7 us = 2.5 TB/s, 8.4 us where the rows lie in L2.  Clusters of 1 / 4 / 8: 11.5 / 5.9 / 5.0 and 18.7 /
// 8.8 / 8.7 us.
constexpr int kMoves = 8;  // rows whose addresses are staged, and whose copies are in flight, together

struct AcceptArgs {
    View w;
    const int32_t *draft, *parents, *sampled;
    int32_t *accepted, *path, *next_token;
    int32_t* ctx_out;
    int layers, D;
    long long layer_stride;
};

__global__ void __cluster_dims__(kAcceptCluster, 1, 1) __launch_bounds__(kAcceptThreads)
    accept_kernel(const AcceptArgs p) {
    __shared__ int32_t next[kMaxTree];
    __shared__ int32_t path[kMaxTree];
    __shared__ int len_s;
    __shared__ long long src_s[kMoves], dst_s[kMoves];
    const int s = blockIdx.x / kAcceptCluster, rank = blockIdx.x % kAcceptCluster, tid = threadIdx.x;
    bool bad;
    Seq q = seq_of(p.w, s, bad);
    if (q.n > kMaxTree) {
        bad = true;
        q.n = -1;
    }
    if (bad && rank == 0 && tid == 0) atomicOr(p.w.err, q4d::kErrDeviceCheck);
    const int n = q.n;
    walk_tree(p.draft + q.start, p.parents + q.start, p.sampled + q.start, n, next, path, &len_s);
    const int len = len_s;
    // what is moved: path[i] -> i for the rows that are not in place
    const int cols = p.D / 8, per_layer = 2 * p.w.H * cols;
    const long long total = (long long)p.layers * per_layer;
    const long long head_step = (long long)p.w.div.d * p.D;
    int first = 1;
    while (first < len && path[first] == first) ++first;
    for (int i0 = first; i0 < len && total > 0; i0 += kMoves) {
        const int m = min(kMoves, len - i0);
        __syncthreads();
        if (tid < m) {
            const long long a = row_at(p.w, s, q.ctx + path[i0 + tid], 0, p.D);
            const long long b = row_at(p.w, s, q.ctx + i0 + tid, 0, p.D);
            if (a < 0 || b < 0) atomicOr(p.w.err, q4d::kErrDeviceCheck);
            src_s[tid] = a;
            dst_s[tid] = a < 0 ? -1 : b;
        }
        __syncthreads();
        for (long long x = (long long)rank * kAcceptThreads + tid; x < total; x += kAcceptCluster * kAcceptThreads) {
            const long long l = x / per_layer;
            const int y = (int)(x - l * per_layer), c = y % cols, h = y / cols % p.w.H;
            uint16_t* pool = (y >= p.w.H * cols ? p.w.v : p.w.k) + l * p.layer_stride + h * head_step + 8 * c;
            uint4 r[kMoves];
#pragma unroll
            for (int i = 0; i < kMoves; ++i)
                if (i < m && dst_s[i] >= 0) r[i] = *reinterpret_cast<const uint4*>(pool + src_s[i]);
#pragma unroll
            for (int i = 0; i < kMoves; ++i)
                if (i < m && dst_s[i] >= 0) *reinterpret_cast<uint4*>(pool + dst_s[i]) = r[i];
        }
    }
    if (rank == 0 && n >= 0)
        for (int i = tid; i < n; i += kAcceptThreads) p.path[q.start + i] = i < len ? path[i] : -1;
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (rank == 0 && tid == 0 && n >= 0) {
        p.accepted[s] = len;
        p.next_token[s] = len > 0 ? p.sampled[q.start + path[len - 1]] : -1;
        p.ctx_out[s] = q.ctx + len;
    }
}

}  // namespace q4p

using namespace q4i;

extern "C" q4_status q4_rope_frequencies(const q4_rope_desc* desc, uint64_t* freqs, q4_stream_t stream) {
    clear_error();
    if (!desc || !freqs) return fail(Q4_ERR_INVALID_ARG, "NULL pointer argument");
    const q4_rope_desc& d = *desc;
    if (d.rot_dim < 2 || d.rot_dim > 1024 || d.rot_dim % 2)
        return fail(Q4_ERR_INVALID_ARG, "rot_dim=%d (even, 2 .. 1024)", d.rot_dim);
    if (!(d.theta > 1.0) || !(d.theta < INFINITY) || !(d.factor >= 1.0) || !(d.factor < INFINITY) || d.orig_len < 0)
        return fail(Q4_ERR_INVALID_ARG, "theta=%g factor=%g orig_len=%d", d.theta, d.factor, d.orig_len);
    if (d.factor > 1.0 && d.orig_len > 0 && !(d.alpha >= 0.0 && d.beta > d.alpha && d.beta < INFINITY))
        return fail(Q4_ERR_INVALID_ARG, "alpha=%g beta=%g (0 <= alpha < beta)", d.alpha, d.beta);
    if (reinterpret_cast<uintptr_t>(freqs) & 7u) return fail(Q4_ERR_MISALIGNED, "freqs must be 8-byte aligned");
    const DeviceInfo* dev = nullptr;
    const q4_status st = current_device(&dev);
    if (st != Q4_OK) return st;
    const int n = d.rot_dim / 2;
    q4p::rope_freq_kernel<<<(n + 63) / 64, 64, 0, reinterpret_cast<cudaStream_t>(stream)>>>(d, freqs);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "q4_rope_frequencies launch");
}

extern "C" q4_status q4_paged_append(const q4_paged_append_desc* desc, q4_stream_t stream) {
    clear_error();
    if (!desc) return fail(Q4_ERR_INVALID_ARG, "desc is NULL");
    q4_paged_append_desc d = *desc;
    q4p::AppendArgs a;
    q4_status st = paged_view(d.cache, d.ctx_len, d.row_start, d.rows, &a.w);
    if (st != Q4_OK) return st;
    const int D = d.cache.head_dim;
    if ((d.rows > 0 && (!d.k || !d.v)) || (d.q && !d.q_out) || (d.q_out && !d.q)) return fail(Q4_ERR_INVALID_ARG, "NULL pointer argument");
    if (d.q ? d.n_q_heads < 1 : d.n_q_heads < 0) return fail(Q4_ERR_INVALID_ARG, "n_q_heads=%d", d.n_q_heads);
    if ((long long)d.n_q_heads * D > (1 << 24)) return fail(Q4_ERR_UNSUPPORTED, "%d query heads", d.n_q_heads);
    if (d.rot_dim < 0 || d.rot_dim > D || d.rot_dim % 2) return fail(Q4_ERR_INVALID_ARG, "rot_dim=%d of %d", d.rot_dim, D);
    if ((d.rot_dim > 0) != (d.freqs != nullptr)) return fail(Q4_ERR_INVALID_ARG, "freqs and rot_dim go together");
    if (d.layout != Q4_ROPE_HALF && d.layout != Q4_ROPE_INTERLEAVED) return fail(Q4_ERR_INVALID_ARG, "layout=%d", (int)d.layout);
    if (!(d.amplitude >= 0.f) || !(d.amplitude < INFINITY)) return fail(Q4_ERR_INVALID_ARG, "amplitude=%g", d.amplitude);
    if (reinterpret_cast<uintptr_t>(d.freqs) & 7u) return fail(Q4_ERR_MISALIGNED, "freqs must be 8-byte aligned");
    if (!aligned4(d.positions)) return fail(Q4_ERR_MISALIGNED, "positions must be 4-byte aligned");
    const int wk = d.cache.n_kv_heads * D, wq = d.n_q_heads * D;
    if ((st = row_matrix("k", d.k, wk, &d.ldk)) != Q4_OK || (st = row_matrix("v", d.v, wk, &d.ldv)) != Q4_OK) return st;
    if (d.q && ((st = row_matrix("q", d.q, wq, &d.ldq)) != Q4_OK || (st = row_matrix("q_out", d.q_out, wq, &d.ldqo)) != Q4_OK))
        return st;
    if (d.q == d.q_out && d.q && d.ldq != d.ldqo) return fail(Q4_ERR_INVALID_ARG, "q_out is q with another row stride");
    const DeviceInfo* dev = nullptr;
    if ((st = current_device(&dev)) != Q4_OK) return st;
    if (d.rows == 0) return Q4_OK;
    a.w.err = dev->err_word;
    a.positions = d.positions;
    a.k = d.k;
    a.v = d.v;
    a.q = d.q;
    a.q_out = d.q_out;
    a.ldk = d.ldk;
    a.ldv = d.ldv;
    a.ldq = d.ldq;
    a.ldqo = d.ldqo;
    a.Hq = d.q ? d.n_q_heads : 0;
    a.freqs = d.freqs;
    a.rot = d.rot_dim;
    a.amplitude = d.amplitude == 0.f ? 1.f : d.amplitude;
    // chunks of 8: neighbours always pair up within one; halves do where they
    // are whole chunks (rot_dim a multiple of 16; 30.3 us where element by
    // element takes 40.9, 6767 rows)
    const int pairs = d.layout == Q4_ROPE_INTERLEAVED ? 0 : d.rot_dim % 16 == 0 ? 1 : 2;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    void (*kern)(q4p::AppendArgs) =
        D == 128 ? (pairs == 0 ? q4p::append_kernel<128, 0> : pairs == 1 ? q4p::append_kernel<128, 1> : q4p::append_kernel<128, 2>)
                 : (pairs == 0 ? q4p::append_kernel<64, 0> : pairs == 1 ? q4p::append_kernel<64, 1> : q4p::append_kernel<64, 2>);
    a.by_per = q4p::page_div((uint32_t)(pairs == 1 ? D / 8 - d.rot_dim / 16 : D / 8));
    kern<<<d.rows, q4p::kAppendThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "q4_paged_append launch");
}

extern "C" q4_status q4_tree_accept(const q4_tree_accept_desc* desc, q4_stream_t stream) {
    clear_error();
    if (!desc) return fail(Q4_ERR_INVALID_ARG, "desc is NULL");
    const q4_tree_accept_desc& d = *desc;
    q4p::AcceptArgs a;
    q4_status st = paged_view(d.cache, d.ctx_len, d.row_start, d.rows, &a.w);
    if (st != Q4_OK) return st;
    if (!d.accepted || !d.next_token || !d.ctx_out || (d.rows > 0 && (!d.draft || !d.parents || !d.sampled || !d.path)))
        return fail(Q4_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned4(d.draft, d.parents, d.sampled, d.accepted, d.path, d.next_token, d.ctx_out))
        return fail(Q4_ERR_MISALIGNED, "the int32 arrays must be 4-byte aligned");
    if (d.n_layers < 0 || d.n_layers > (1 << 16)) return fail(Q4_ERR_INVALID_ARG, "n_layers=%d", d.n_layers);
    if (d.layer_stride % 8) return fail(Q4_ERR_MISALIGNED, "layer_stride must be a multiple of 8");
    const unsigned long long pool =
        (unsigned long long)d.cache.n_pages * d.cache.page_size * d.cache.n_kv_heads * d.cache.head_dim;
    if (d.n_layers > 1 && d.layer_stride < pool)
        return fail(Q4_ERR_INVALID_ARG, "layer_stride=%zu, a layer's pool has %llu elements", d.layer_stride, pool);
    const DeviceInfo* dev = nullptr;
    if ((st = current_device(&dev)) != Q4_OK) return st;
    a.w.err = dev->err_word;
    a.draft = d.draft;
    a.parents = d.parents;
    a.sampled = d.sampled;
    a.accepted = d.accepted;
    a.path = d.path;
    a.next_token = d.next_token;
    a.ctx_out = d.ctx_out;
    a.layers = d.n_layers;
    a.D = d.cache.head_dim;
    a.layer_stride = (long long)d.layer_stride;
    q4p::accept_kernel<<<d.cache.n_seqs * q4p::kAcceptCluster, q4p::kAcceptThreads, 0,
                         reinterpret_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "q4_tree_accept launch");
}
