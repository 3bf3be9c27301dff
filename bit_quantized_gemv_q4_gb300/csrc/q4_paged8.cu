// The paged key / value cache in 8 bits: the append that rounds to it, reading
// it back, the acceptance of a drafted tree in it; and the append (to either
// cache) that normalises queries and keys (q4.h 9a, 9b, 9c, 9e).
//
// BaseRT: optimal LLM inference on Apple Silicon with native Metal, §3.3
// fuses the operator sequences of the attention path; the pages describe
// neither a cache in 8 bits nor the norms of heads.
//
// Mathematics of the format: e4m3 is a float of 3 + 1 significant bits, so a
// scale finer than a power of two would win no relative accuracy, while with
// powers of two a block whose scale grows is rewritten exactly (its exponents
// shift; only what falls below 2^-6 of the new scale is rounded again) and
// code * scale is an fp16 number: at least 2^-15 * 2^-9 = 2^-24, at most
// 2^8 * 240, as the elements are limited to that.
#include <cuda_fp16.h>
#include <math.h>

#include "q4_paged8.cuh"

namespace q4p {

// The least scale 2^e, e of -15 .. 8, for elements up to t <= 61440: with t =
// m 2^k, 1 <= m < 2, and 448 = 1.75 * 2^8, e is k - 8, or k - 7 where m > 1.75,
// which the carry into the exponent adds.
__device__ __forceinline__ float scale_for(float t) {
    const int e = (int)((__float_as_uint(t) + 0x1fffffu) >> 23) - (127 + 8);
    return __uint_as_float((uint32_t)(127 + max(e, -15)) << 23);
}

constexpr float kGreatest = 61440.f;
__device__ __forceinline__ float limited(float x) { return x != x ? x : fminf(fmaxf(x, -kGreatest), kGreatest); }

// Four codes times a ratio of scales, as codes.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    const float2 a = e4m3_f32(w), b = e4m3_f32(w >> 16);
    return f32_e4m3(a.x * ratio, a.y * ratio) | f32_e4m3(b.x * ratio, b.y * ratio) << 16;
}

// ------------------------------------------------------------------ append ---
// A block of threads looks after `win` rows: it finds their sequences, and
// takes every run of rows that begins among them - in the 8-bit cache the new
// rows of one block of 16 positions (they share a scale, so one thread block
// has to have them all), else single rows.  gridDim.y blocks share a window's
// heads.  NC = D / 8 lanes hold a head of a row, 8 elements each: its mean of
// squares is a sum over them, and the partner of an element lies in the same
// lane (neighbours) or the same element of another lane (halves of whole
// 16-byte chunks), else it is read once more.
constexpr int kRowThreads = 256;
constexpr int kWin = 16;                    // rows of a window at most
constexpr int kCover = kWin + kBlock - 1;   // rows that runs beginning in it may have

struct RowsArgs {
    View8 c;               // append_norm: c.w alone, its pools
    const int32_t* positions;
    const uint16_t *k, *v, *q;
    uint16_t* q_out;
    long long ldk, ldv, ldq, ldqo;
    int Hq;
    const uint64_t* freqs;
    int rot;
    float amplitude;
    const uint16_t *qw, *kw;
    int q_norm, k_norm;
    float eps;
    int win;
};

// Rows of one sequence that share a block of positions.
struct Run {
    int row, m;       // first row, rows
    int slot, old;    // its position; cached positions before it in the block
    long long base;   // head 0's row of that position in the pools (-1: no memory)
    long long scale;  // head 0's scale
};

// By a warp: the sequence that holds a row, false if none does.  A search led
// astray by a sequence that does not fit is made good by looking at all.
__device__ __forceinline__ bool find_row(const View& w, int row, int lane, int& s, Seq& q) {
    s = seq_of_row(w, row, lane);
    if (s < w.S && holds(w, s, row, q)) return true;
    int first = 0x7fffffff;
    for (int i = lane; i < w.S && first == 0x7fffffff; i += 32)
        if (holds(w, i, row, q)) first = i;
    s = __reduce_min_sync(0xffffffffu, first);
    return s != 0x7fffffff && holds(w, s, row, q);
}

template <int D, int kPairs, bool k8>
__global__ void __launch_bounds__(kRowThreads, 4) append_rows_kernel(const __grid_constant__ RowsArgs p) {
    constexpr int NC = D / 8, G = kRowThreads / NC;  // lanes of a head, heads at a time
    constexpr int kMost = k8 ? kCover : kWin;
    constexpr int kPass = k8 ? (kCover + G - 1) / G : 1;
    __shared__ Run run_s[kWin];
    __shared__ int row_run[kMost];                   // run of each covered row ...
    __shared__ int row_at_run[kMost];                // ... and its place in it
    __shared__ int rows_s;
    __shared__ __align__(16) float2 cs[kMost][D / 2];
    __shared__ __align__(16) float wq_s[D], wk_s[D];
    __shared__ uint32_t top_s[3][kWin];              // greatest magnitudes of the runs, as bits
    const View& w = p.c.w;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r0 = blockIdx.x * p.win;

    if (tid < D) {
        if (p.q_norm) wq_s[tid] = p.qw ? __half2float(__ushort_as_half(p.qw[tid])) : 1.f;
        if (p.k_norm) wk_s[tid] = p.kw ? __half2float(__ushort_as_half(p.kw[tid])) : 1.f;
    }
    if (tid < 3 * kWin) top_s[tid / kWin][tid % kWin] = 0u;
    for (int i = warp; i < kWin; i += kRowThreads / 32) {
        const int row = r0 + i;
        Run r = {0, 0, 0, 0, -1, 0};
        int s;
        Seq q;
        if (i < p.win && row < w.rows && find_row(w, row, lane, s, q)) {
            r.row = row;
            r.slot = q.ctx + (row - q.start);
            const uint32_t pg = page_of(w.div, (uint32_t)r.slot);
            const int at = r.slot - (int)(pg * w.div.d), in = at % kBlock;
            const bool first = row == q.start;
            if constexpr (k8) {
                if (first || in == 0) r.m = min(min(kBlock - in, (int)w.div.d - at), q.start + q.n - row);
                r.old = first ? in : 0;
            } else {
                r.m = 1;
            }
            const int id = w.table[(size_t)s * w.max_pages + pg];
            if ((uint32_t)id < (uint32_t)w.n_pages) {
                r.base = ((long long)id * w.H * w.div.d + at) * D;
                if constexpr (k8) r.scale = (long long)id * w.H * p.c.nb + at / kBlock;
            } else if (lane == 0 && r.m > 0) {
                atomicOr(w.err, q4d::kErrDeviceCheck);
            }
        }
        if (lane == 0) run_s[i] = r;
    }
    if (r0 == 0 && blockIdx.y == 0) {
        // the first block latches the sequences that do not fit
        for (int s = tid; s < w.S; s += kRowThreads) {
            bool bad;
            seq_of(w, s, bad);
            if (bad) atomicOr(w.err, q4d::kErrDeviceCheck);
        }
    }
    __syncthreads();
    if (warp == 0) {
        const int m = lane < kWin ? run_s[lane].m : 0;
        int sum = m;
#pragma unroll
        for (int x = 1; x < kWin; x <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, x);
            if (lane >= x) sum += y;
        }
        if (lane == kWin - 1) rows_s = sum;
        for (int j = 0; j < m; ++j) {
            row_run[sum - m + j] = lane;
            row_at_run[sum - m + j] = j;
        }
    }
    __syncthreads();
    const int T = rows_s;
    if (T == 0) return;
    const int half = p.rot / 2;
    for (int x = tid; x < T * half; x += kRowThreads) {
        const int t = x / half, i = x - t * half;
        const Run& r = run_s[row_run[t]];
        const int j = row_at_run[t];
        const long long pos = p.positions ? p.positions[r.row + j] : r.slot + j;
        const uint64_t turn = (uint64_t)pos * p.freqs[i];
        float sn, cn;
        sincospif((float)(int32_t)(uint32_t)(turn >> 32) * 4.656612873077393e-10f, &sn, &cn);
        cs[t][i] = make_float2(cn * p.amplitude, sn * p.amplitude);
    }
    __syncthreads();

    const int g = tid / NC, c = tid % NC, rc = half / 8;
    // A head of covered row t, loaded by its NC lanes (all lanes of the warp come
    // here; those without one pass live = false), normalised and rotated.
    const auto turned = [&](const uint16_t* src, bool live, int t, bool norm, const float* weight, float (&x)[8]) {
        const uint4 a = live ? *reinterpret_cast<const uint4*>(src + 8 * c) : make_uint4(0, 0, 0, 0);
        unpack8(a, x);
        float inv = 1.f;
        if (norm) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = NC / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float v = ss * (1.f / D) + p.eps;
            inv = v == 0.f ? 0.f : 1.f / sqrtf(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * weight[8 * c + e];
        }
        if (half == 0) return;
        if constexpr (kPairs == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * c + e;
                if (i < half) {
                    const float2 r = cs[t][i];
                    const float u = x[2 * e], v = x[2 * e + 1];
                    x[2 * e] = u * r.x - v * r.y;
                    x[2 * e + 1] = v * r.x + u * r.y;
                }
            }
        } else if constexpr (kPairs == 1) {
            const int partner = c < rc ? c + rc : c < 2 * rc ? c - rc : c;
            const int i0 = 8 * min(c, partner);
            const float sign = c < rc ? -1.f : 1.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = __shfl_sync(0xffffffffu, x[e], partner, NC);
                if (partner != c) {
                    const float2 r = cs[t][i0 + e];
                    x[e] = x[e] * r.x + sign * y * r.y;
                }
            }
        } else {
            // pairs (i, i + half) across the chunks
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = 8 * c + e;
                if (i < 2 * half && live) {
                    const int o = i < half ? i + half : i - half;
                    float y = __half2float(__ushort_as_half(src[o]));
                    if (norm) y = y * inv * weight[o];
                    const float2 r = cs[t][min(i, o)];
                    x[e] = i < half ? x[e] * r.x - y * r.y : x[e] * r.x + y * r.y;
                }
            }
            __syncwarp();  // in place (q_out == q): every partner is read before any is written
        }
    };

    const int part = blockIdx.y, parts = gridDim.y;
    // queries
    {
        const int h0 = (int)((long long)p.Hq * part / parts), nh = (int)((long long)p.Hq * (part + 1) / parts) - h0;
        const int items = T * nh;
        for (int x0 = 0; x0 < items; x0 += G) {
            const int x = x0 + g, t = min(x, items - 1) / nh, h = h0 + min(x, items - 1) - t * nh;
            const bool live = x < items;
            const long long row = run_s[row_run[t]].row + row_at_run[t];
            float y[8];
            turned(p.q + row * p.ldq + (long long)h * D, live, t, p.q_norm, wq_s, y);
            if (live) *reinterpret_cast<uint4*>(p.q_out + row * p.ldqo + (long long)h * D + 8 * c) = pack8(y);
        }
    }
    // keys (heads 0 ..) and values (heads H ..)
    const int x0 = (int)(2ll * w.H * part / parts), x1 = (int)(2ll * w.H * (part + 1) / parts);
    if constexpr (!k8) {
        const int nh = x1 - x0, items = T * nh;
        for (int i0 = 0; i0 < items; i0 += G) {
            const int i = i0 + g, t = min(i, items - 1) / nh, x = x0 + min(i, items - 1) - t * nh;
            const bool live = i < items;
            const Run& r = run_s[row_run[t]];
            const int h = x < w.H ? x : x - w.H;
            const uint16_t* src = x < w.H ? p.k + r.row * p.ldk + (long long)h * D : p.v + r.row * p.ldv + (long long)h * D;
            // (a warp may hold keys and values at once: the values go through unchanged)
            float y[8];
            turned(src, live, t, p.k_norm, wk_s, y);
            const uint4 a = x < w.H ? pack8(y) : live ? *reinterpret_cast<const uint4*>(src + 8 * c) : make_uint4(0, 0, 0, 0);
            if (live && r.base >= 0)
                *reinterpret_cast<uint4*>((x < w.H ? w.k : w.v) + r.base + (long long)h * w.div.d * D + 8 * c) = a;
        }
    } else {
        for (int x = x0; x < x1; ++x) {
            const bool key = x < w.H;
            const int h = key ? x : x - w.H, n = (x - x0) % 3;
            uint8_t* pool = key ? p.c.k : p.c.v;
            float* scales = key ? p.c.ks : p.c.vs;
            float y[kPass][8], was[kPass];
#pragma unroll
            for (int e = 0; e < kPass; ++e) {
                const int t = e * G + g;
                const bool live = t < T;
                const Run& r = run_s[row_run[live ? t : 0]];
                const long long row = r.row + row_at_run[live ? t : 0];
                if (key) {
                    turned(p.k + row * p.ldk + (long long)h * D, live, live ? t : 0, p.k_norm, wk_s, y[e]);
                } else {
                    const uint4 a = live ? *reinterpret_cast<const uint4*>(p.v + row * p.ldv + (long long)h * D + 8 * c)
                                         : make_uint4(0, 0, 0, 0);
                    unpack8(a, y[e]);
                }
                was[e] = live && r.old > 0 && r.base >= 0 ? scales[r.scale + (long long)h * p.c.nb] : 0.f;
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[e][i] = limited(y[e][i]);
                    top = fmaxf(top, fabsf(y[e][i]));  // (NaN loses)
                }
#pragma unroll
                for (int o = NC / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (live && c == 0) atomicMax(&top_s[n][row_run[t]], __float_as_uint(top));
            }
            // Three sets of tops: this head's is read behind the barrier, the next
            // head's was cleared before it, and the one before may still be read.
            if (tid < kWin) top_s[(n + 1) % 3][tid] = 0u;
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kPass; ++e) {
                const int t = e * G + g;
                if (t >= T) continue;
                const Run& r = run_s[row_run[t]];
                if (r.base < 0) continue;
                const int j = row_at_run[t];
                const float scale = fmaxf(scale_for(__uint_as_float(top_s[n][row_run[t]])), was[e]);
                const float inv = 1.f / scale;
                uint8_t* at = pool + r.base + (long long)h * w.div.d * D + 8 * c;
#pragma unroll
                for (int i = 0; i < 8; ++i) y[e][i] *= inv;
                *reinterpret_cast<uint2*>(at + (long long)j * D) =
                    make_uint2(f32_e4m3(y[e][0], y[e][1]) | f32_e4m3(y[e][2], y[e][3]) << 16,
                               f32_e4m3(y[e][4], y[e][5]) | f32_e4m3(y[e][6], y[e][7]) << 16);
                if (j == 0 && (r.old == 0 || scale != was[e])) {
                    if (c == 0) scales[r.scale + (long long)h * p.c.nb] = scale;
                    const float ratio = was[e] * inv;
                    for (int o = 1; o <= r.old; ++o) {
                        uint2* const from = reinterpret_cast<uint2*>(at - (long long)o * D);
                        const uint2 v = *from;
                        *from = make_uint2(rescale4(v.x, ratio), rescale4(v.y, ratio));
                    }
                }
            }
        }
    }
}

// -------------------------------------------------------------------- read ---
// A warp per row: 16 codes a lane.  What bounds it: bytes.
constexpr int kReadThreads = 256;

struct ReadArgs {
    View8 c;
    uint16_t *k, *v;
    long long ldk, ldv;
};

template <int D>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadArgs p) {
    const View& w = p.c.w;
    const int lane = threadIdx.x & 31, row = (int)(blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5));
    if (blockIdx.x == 0) {
        for (int s = threadIdx.x; s < w.S; s += kReadThreads) {
            bool bad;
            seq_of(w, s, bad);
            if (bad) atomicOr(w.err, q4d::kErrDeviceCheck);
        }
    }
    int s;
    Seq q;
    if (row >= w.rows || !find_row(w, row, lane, s, q)) return;
    const int slot = q.ctx + (row - q.start);
    const uint32_t pg = page_of(w.div, (uint32_t)slot);
    const int at = slot - (int)(pg * w.div.d);
    const int id = w.table[(size_t)s * w.max_pages + pg];
    const bool there = (uint32_t)id < (uint32_t)w.n_pages;
    if (!there && lane == 0) atomicOr(w.err, q4d::kErrDeviceCheck);
    constexpr int NC = D / 16;
    const int items = w.H * NC;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        uint16_t* out = kv ? p.v : p.k;
        if (!out) continue;
        out += row * (kv ? p.ldv : p.ldk);
        const uint8_t* pool = kv ? p.c.v : p.c.k;
        const float* scales = kv ? p.c.vs : p.c.ks;
#pragma unroll 4
        for (int x = lane; x < items; x += 32) {
            const int h = x / NC, c = x % NC;
            uint4 a = make_uint4(0, 0, 0, 0);
            float f = 0.f;
            if (there) {
                const long long hd = (long long)id * w.H + h;
                a = *reinterpret_cast<const uint4*>(pool + (hd * w.div.d + at) * D + 16 * c);
                f = scales[hd * p.c.nb + at / kBlock];
            }
            const uint32_t ws[4] = {a.x, a.y, a.z, a.w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 u = e4m3_f32(ws[e]), v = e4m3_f32(ws[e] >> 16);
                o[2 * e] = pack_half2(u.x * f, u.y * f);
                o[2 * e + 1] = pack_half2(v.x * f, v.y * f);
            }
            uint4* dst = reinterpret_cast<uint4*>(out + (long long)h * D + 16 * c);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

// -------------------------------------------------------------- acceptance ---
// As for the fp16 cache a cluster of 8 blocks per sequence, each of which finds
// the path for itself.  Then, destination block by destination block (16
// positions with one scale), the warps of the cluster share the (layer, keys or
// values, head) columns: a warp reads all rows of its column's block that will
// be written before it writes any.  Paths ascend, so a row whose place a block
// gives up moves within that block: no later block reads what an earlier one
// has written.
struct Accept8Args {
    View8 c;
    const int32_t *draft, *parents, *sampled;
    int32_t *accepted, *path, *next_token;
    int32_t* ctx_out;
    int layers;
    long long layer_stride, scale_stride;
};

template <int D>
__global__ void __cluster_dims__(kAcceptCluster, 1, 1) __launch_bounds__(kAcceptThreads)
    accept8_kernel(const __grid_constant__ Accept8Args p) {
    __shared__ int32_t next[kMaxTree];
    __shared__ int32_t path[kMaxTree];
    __shared__ int len_s;
    __shared__ long long src_s[kBlock], scale_s[kBlock];  // head 0's row and scale that come to each place (src -1: none)
    const View& w = p.c.w;
    const int s = blockIdx.x / kAcceptCluster, rank = blockIdx.x % kAcceptCluster, tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    bool bad;
    Seq q = seq_of(w, s, bad);
    if (q.n > kMaxTree) {
        bad = true;
        q.n = -1;
    }
    if (bad && rank == 0 && tid == 0) atomicOr(w.err, q4d::kErrDeviceCheck);
    const int n = q.n;
    walk_tree(p.draft + q.start, p.parents + q.start, p.sampled + q.start, n, next, path, &len_s);
    const int len = len_s;
    int first = 1;  // path[i] == i before it, path[i] > i from there on
    while (first < len && path[first] == first) ++first;
    const int page = (int)w.div.d;
    const long long columns = 2ll * w.H * p.layers;
    constexpr int NC = D / 16, PER = 32 / NC, kPass = kBlock / PER;  // lanes of a row, rows at a time
    const int c = lane % NC, g = lane / NC;
    for (int i0 = first; i0 < len && columns > 0;) {
        // the block that path row i0 moves into
        const int slot = q.ctx + i0;
        const uint32_t pg = page_of(w.div, (uint32_t)slot);
        const int at = slot - (int)(pg * w.div.d), lo = at / kBlock * kBlock;
        const int count = min(min(kBlock, page - lo), q.n - (i0 - (at - lo)));  // its places up to the last new row
        const int i1 = min(len, i0 + count - (at - lo));                        // path rows that move into it: i0 .. i1 - 1
        const int id = w.table[(size_t)s * w.max_pages + pg];
        const bool there = (uint32_t)id < (uint32_t)w.n_pages;
        __syncthreads();
        if (tid < kBlock) {
            const int i = i0 + tid - (at - lo);
            src_s[tid] = -1;
            if (i >= i0 && i < i1) {
                const int from = q.ctx + path[i];
                const uint32_t fp = page_of(w.div, (uint32_t)from);
                const int fid = w.table[(size_t)s * w.max_pages + fp], fat = from - (int)(fp * w.div.d);
                if ((uint32_t)fid < (uint32_t)w.n_pages) {
                    src_s[tid] = ((long long)fid * w.H * page + fat) * D;
                    scale_s[tid] = (long long)fid * w.H * p.c.nb + fat / kBlock;
                }
                if (!there || src_s[tid] < 0) atomicOr(w.err, q4d::kErrDeviceCheck);
            }
        }
        __syncthreads();
        const long long base = ((long long)id * w.H * page + lo) * D, own = (long long)id * w.H * p.c.nb + lo / kBlock;
        i0 = i1;
        if (!there) continue;
        constexpr int kWarps = kAcceptThreads / 32;
        for (long long x = rank * kWarps + warp; x < columns; x += kAcceptCluster * kWarps) {
            const long long l = x / (2 * w.H);
            const int y = (int)(x - l * (2 * w.H)), h = y < w.H ? y : y - w.H;
            uint8_t* pool = (y < w.H ? p.c.k : p.c.v) + l * p.layer_stride + (long long)h * page * D;
            float* scales = (y < w.H ? p.c.ks : p.c.vs) + l * p.scale_stride + (long long)h * p.c.nb;
            const float was = scales[own];
            float from[kPass], most = was;
            uint4 r[kPass];
#pragma unroll
            for (int e = 0; e < kPass; ++e) {
                const int j = e * PER + g;
                from[e] = was;
                if (src_s[j] >= 0) {
                    from[e] = scales[scale_s[j]];
                    r[e] = *reinterpret_cast<const uint4*>(pool + src_s[j] + 16 * c);
                }
                most = fmaxf(most, from[e]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            const bool grown = most != was;
#pragma unroll
            for (int e = 0; e < kPass; ++e) {
                const int j = e * PER + g;
                if (src_s[j] < 0 && grown && j < count) r[e] = *reinterpret_cast<const uint4*>(pool + base + (long long)j * D + 16 * c);
            }
            __syncwarp();  // everything is read
#pragma unroll
            for (int e = 0; e < kPass; ++e) {
                const int j = e * PER + g;
                if (src_s[j] < 0 && !(grown && j < count)) continue;
                if (from[e] != most) {
                    const float ratio = from[e] / most;
                    r[e] = make_uint4(rescale4(r[e].x, ratio), rescale4(r[e].y, ratio), rescale4(r[e].z, ratio),
                                      rescale4(r[e].w, ratio));
                }
                *reinterpret_cast<uint4*>(pool + base + (long long)j * D + 16 * c) = r[e];
            }
            if (grown && lane == 0) scales[own] = most;
        }
    }
    if (rank == 0 && n >= 0)
        for (int i = tid; i < n; i += kAcceptThreads) p.path[q.start + i] = i < len ? path[i] : -1;
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (rank == 0 && tid == 0 && n >= 0) {  // ctx_out may be ctx_len: every block has read it
        p.accepted[s] = len;
        p.next_token[s] = len > 0 ? p.sampled[q.start + path[len - 1]] : -1;
        p.ctx_out[s] = q.ctx + len;
    }
}

}  // namespace q4p

using namespace q4i;

namespace {

// The arguments that the appends to both caches share (7b's checks); a.c.w is set.
q4_status rows_args(const q4_paged_append8_desc& given, const q4_head_norm* norm, q4p::RowsArgs* a) {
    q4_paged_append8_desc d = given;
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
    q4_status st;
    if ((st = row_matrix("k", d.k, wk, &d.ldk)) != Q4_OK || (st = row_matrix("v", d.v, wk, &d.ldv)) != Q4_OK) return st;
    if (d.q && ((st = row_matrix("q", d.q, wq, &d.ldq)) != Q4_OK || (st = row_matrix("q_out", d.q_out, wq, &d.ldqo)) != Q4_OK))
        return st;
    if (d.q == d.q_out && d.q && d.ldq != d.ldqo) return fail(Q4_ERR_INVALID_ARG, "q_out is q with another row stride");
    a->q_norm = a->k_norm = 0;
    a->qw = a->kw = nullptr;
    a->eps = 0.f;
    if (norm) {
        if (!(norm->eps >= 0.f) || !(norm->eps < INFINITY)) return fail(Q4_ERR_INVALID_ARG, "norm eps=%g", norm->eps);
        if ((reinterpret_cast<uintptr_t>(norm->q_weight) | reinterpret_cast<uintptr_t>(norm->k_weight)) & 1u)
            return fail(Q4_ERR_MISALIGNED, "the norms' weights must be 2-byte aligned");
        a->q_norm = norm->q_rmsnorm != 0;
        a->k_norm = norm->k_rmsnorm != 0;
        a->qw = norm->q_weight;
        a->kw = norm->k_weight;
        a->eps = norm->eps;
    }
    a->positions = d.positions;
    a->k = d.k;
    a->v = d.v;
    a->q = d.q;
    a->q_out = d.q_out;
    a->ldk = d.ldk;
    a->ldv = d.ldv;
    a->ldq = d.ldq;
    a->ldqo = d.ldqo;
    a->Hq = d.q ? d.n_q_heads : 0;
    a->freqs = d.freqs;
    a->rot = d.rot_dim;
    a->amplitude = d.amplitude == 0.f ? 1.f : d.amplitude;
    return Q4_OK;
}

template <bool k8>
q4_status launch_rows(q4p::RowsArgs& a, int D, q4_rope_layout layout, const DeviceInfo* dev, q4_stream_t stream, const char* what) {
    const int rows = a.c.w.rows;
    a.c.w.err = dev->err_word;
    // halves pair up in whole chunks where rot_dim is a multiple of 16
    const int pairs = layout == Q4_ROPE_INTERLEAVED ? 0 : a.rot % 16 == 0 ? 1 : 2;
    void (*kern)(q4p::RowsArgs) =
        D == 128 ? (pairs == 0   ? q4p::append_rows_kernel<128, 0, k8>
                    : pairs == 1 ? q4p::append_rows_kernel<128, 1, k8>
                                 : q4p::append_rows_kernel<128, 2, k8>)
                 : (pairs == 0   ? q4p::append_rows_kernel<64, 0, k8>
                    : pairs == 1 ? q4p::append_rows_kernel<64, 1, k8>
                                 : q4p::append_rows_kernel<64, 2, k8>);
    a.win = rows >= 2048 ? q4p::kWin : rows >= 512 ? 4 : 1;
    const int windows = (rows - 1) / a.win + 1;
    const int most = 2 * a.c.w.H < 64 ? 2 * a.c.w.H : 64;
    int parts = (6 * dev->sms + windows - 1) / windows;
    parts = parts < 1 ? 1 : parts > most ? most : parts;
    kern<<<dim3((unsigned)windows, (unsigned)parts), q4p::kRowThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, what);
}

}  // namespace

extern "C" q4_status q4_paged_append_norm(const q4_paged_append_desc* desc, const q4_head_norm* norm, q4_stream_t stream) {
    clear_error();
    if (!desc) return fail(Q4_ERR_INVALID_ARG, "desc is NULL");
    const q4_paged_append_desc& d = *desc;
    q4p::RowsArgs a;
    q4_status st = paged_view(d.cache, d.ctx_len, d.row_start, d.rows, &a.c.w);
    if (st != Q4_OK) return st;
    a.c.k = a.c.v = nullptr;
    a.c.ks = a.c.vs = nullptr;
    a.c.nb = 0;
    const q4_paged_cache& c = d.cache;
    const q4_paged_append8_desc same = {
        {nullptr, nullptr, nullptr, nullptr, c.page_table, c.n_pages, c.page_size, c.n_kv_heads, c.head_dim, c.n_seqs, c.max_pages},
        d.ctx_len, d.row_start, d.rows, d.positions, d.k, d.v, d.ldk, d.ldv, d.q, d.q_out, d.ldq, d.ldqo, d.n_q_heads, d.freqs,
        d.rot_dim, d.layout, d.amplitude};
    if ((st = rows_args(same, norm, &a)) != Q4_OK) return st;
    const DeviceInfo* dev = nullptr;
    if ((st = current_device(&dev)) != Q4_OK) return st;
    if (d.rows == 0) return Q4_OK;
    return launch_rows<false>(a, c.head_dim, d.layout, dev, stream, "q4_paged_append_norm launch");
}

extern "C" q4_status q4_paged_append8(const q4_paged_append8_desc* desc, const q4_head_norm* norm, q4_stream_t stream) {
    clear_error();
    if (!desc) return fail(Q4_ERR_INVALID_ARG, "desc is NULL");
    const q4_paged_append8_desc& d = *desc;
    q4p::RowsArgs a;
    q4_status st = paged_view8(d.cache, d.ctx_len, d.row_start, d.rows, &a.c);
    if (st != Q4_OK) return st;
    if ((st = rows_args(d, norm, &a)) != Q4_OK) return st;
    const DeviceInfo* dev = nullptr;
    if ((st = current_device(&dev)) != Q4_OK) return st;
    if (d.rows == 0) return Q4_OK;
    return launch_rows<true>(a, d.cache.head_dim, d.layout, dev, stream, "q4_paged_append8 launch");
}

extern "C" q4_status q4_paged_read8(const q4_paged_read8_desc* desc, q4_stream_t stream) {
    clear_error();
    if (!desc) return fail(Q4_ERR_INVALID_ARG, "desc is NULL");
    q4_paged_read8_desc d = *desc;
    q4p::ReadArgs a;
    q4_status st = paged_view8(d.cache, d.first, d.row_start, d.rows, &a.c);
    if (st != Q4_OK) return st;
    const int width = d.cache.n_kv_heads * d.cache.head_dim;
    if ((st = row_matrix("k", d.k, width, &d.ldk)) != Q4_OK || (st = row_matrix("v", d.v, width, &d.ldv)) != Q4_OK) return st;
    const DeviceInfo* dev = nullptr;
    if ((st = current_device(&dev)) != Q4_OK) return st;
    if (d.rows == 0 || (!d.k && !d.v)) return Q4_OK;
    a.c.w.err = dev->err_word;
    a.k = d.k;
    a.v = d.v;
    a.ldk = d.ldk;
    a.ldv = d.ldv;
    const unsigned grid = (unsigned)((d.rows - 1) / (q4p::kReadThreads / 32) + 1);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (d.cache.head_dim == 128) q4p::read_kernel<128><<<grid, q4p::kReadThreads, 0, s>>>(a);
    else q4p::read_kernel<64><<<grid, q4p::kReadThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "q4_paged_read8 launch");
}

extern "C" q4_status q4_tree_accept8(const q4_tree_accept8_desc* desc, q4_stream_t stream) {
    clear_error();
    if (!desc) return fail(Q4_ERR_INVALID_ARG, "desc is NULL");
    const q4_tree_accept8_desc& d = *desc;
    q4p::Accept8Args a;
    q4_status st = paged_view8(d.cache, d.ctx_len, d.row_start, d.rows, &a.c);
    if (st != Q4_OK) return st;
    if (!d.accepted || !d.next_token || !d.ctx_out || (d.rows > 0 && (!d.draft || !d.parents || !d.sampled || !d.path)))
        return fail(Q4_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned4(d.draft, d.parents, d.sampled, d.accepted, d.path, d.next_token, d.ctx_out))
        return fail(Q4_ERR_MISALIGNED, "the int32 arrays must be 4-byte aligned");
    if (d.n_layers < 0 || d.n_layers > (1 << 16)) return fail(Q4_ERR_INVALID_ARG, "n_layers=%d", d.n_layers);
    if (d.layer_stride % 16) return fail(Q4_ERR_MISALIGNED, "layer_stride must be a multiple of 16");
    const unsigned long long heads = (unsigned long long)d.cache.n_pages * d.cache.n_kv_heads;
    const unsigned long long pool = heads * d.cache.page_size * d.cache.head_dim, blocks = heads * a.c.nb;
    if (d.n_layers > 1 && (d.layer_stride < pool || d.scale_stride < blocks))
        return fail(Q4_ERR_INVALID_ARG, "layer_stride=%zu scale_stride=%zu, a layer has %llu elements and %llu scales", d.layer_stride,
                    d.scale_stride, pool, blocks);
    const DeviceInfo* dev = nullptr;
    if ((st = current_device(&dev)) != Q4_OK) return st;
    a.c.w.err = dev->err_word;
    a.draft = d.draft;
    a.parents = d.parents;
    a.sampled = d.sampled;
    a.accepted = d.accepted;
    a.path = d.path;
    a.next_token = d.next_token;
    a.ctx_out = d.ctx_out;
    a.layers = d.n_layers;
    a.layer_stride = (long long)d.layer_stride;
    a.scale_stride = (long long)d.scale_stride;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)d.cache.n_seqs * q4p::kAcceptCluster;
    if (d.cache.head_dim == 128) q4p::accept8_kernel<128><<<grid, q4p::kAcceptThreads, 0, s>>>(a);
    else q4p::accept8_kernel<64><<<grid, q4p::kAcceptThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "q4_tree_accept8 launch");
}
