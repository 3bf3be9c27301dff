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
// A block of threads looks after a window of rows: it finds their sequences, and
// takes every run of rows that begins among them - in the 8-bit cache the new
// rows of one block of 16 positions (they share a scale, so one thread block
// has to have them all), else single rows.  gridDim.y blocks share a window's
// heads.  D / 16 lanes hold a head of a row, 16 elements each, the halves of
// rotated pairs together where they are whole 16-byte chunks: its mean of
// squares is a sum over them.
//
// What bounds it: the smallest calls the chain of look-ups (row, sequence, page,
// cached scale), the largest bytes and that chain, which four blocks per SM do
// not quite cover (issue slots 47 .. 54 % busy).  Measured, 32 query and 8 kv heads
// of 128: one row with norms (16 query heads) 4.6 us, 40 rows into 8 bits 5.4
// (10.2 where every one of their blocks takes a greater scale: up to 15 cached
// rows rewritten one after another by the lanes of the block's first new row);
// 6767 rows with norms into fp16 (166 MB in and out) 33.8 us = 4.9 TB/s, 72 % of
// the measured copy rate, into 8 bits (152 MB) 38.6 = 3.9 TB/s, 58 %
// (with three blocks per SM 38.0 and 39.0, with five 34.4 and 42.9).
constexpr int kRowThreads = 256, kAhead = 2;
constexpr int kWin = 8;                     // rows of a window
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
};

// Places of pair i's angle and of element i's weight in shared memory: lanes of
// a head that read 16 bytes each find them side by side.
template <int D>
__device__ __forceinline__ int angle_at(int i) {
    return ((i & 7) / 2 * (D / 16) + i / 8) * 2 + (i & 1);
}
template <int D>
__device__ __forceinline__ int weight_at(int i) {
    return ((i & 7) / 4 * (D / 8) + i / 8) * 4 + (i & 3);
}

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
    constexpr int NJ = D / 16, G = kRowThreads / NJ;  // lanes of a head, heads at a time
    constexpr int kMost = k8 ? kCover : kWin;
    static_assert(kMost <= G, "a head of all covered rows at a time");
    __shared__ Run run_s[kWin];
    __shared__ int row_run[kMost];                   // run of each covered row ...
    __shared__ int row_at_run[kMost];                // ... its place in it ...
    __shared__ int row_s[kMost];                     // ... and number
    __shared__ int rows_s;
    __shared__ __align__(16) float2 cs[kMost][D / 2];
    __shared__ __align__(16) float wq_s[D], wk_s[D];
    constexpr int kHeads = G / kBlock;
    __shared__ uint32_t top_s[3][kHeads][kWin];      // greatest magnitudes of the runs, as bits
    const View& w = p.c.w;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r0 = blockIdx.x * kWin;

    if (tid < D) {
        if (p.q_norm) wq_s[weight_at<D>(tid)] = p.qw ? __half2float(__ushort_as_half(p.qw[tid])) : 1.f;
        if (p.k_norm) wk_s[weight_at<D>(tid)] = p.kw ? __half2float(__ushort_as_half(p.kw[tid])) : 1.f;
    }
    if (tid < 3 * kHeads * kWin) top_s[tid / kWin / kHeads][tid / kWin % kHeads][tid % kWin] = 0u;
    for (int i = warp; i < kWin; i += kRowThreads / 32) {
        const int row = r0 + i;
        Run r = {0, 0, 0, 0, -1, 0};
        int s;
        Seq q;
        if (i < kWin && row < w.rows && find_row(w, row, lane, s, q)) {
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
        // (runs of one window overlap, and are more than kMost rows, only where the
        // starts are not in order, which is latched above: what is past it is left out)
        if (lane == kWin - 1) rows_s = min(sum, kMost);
        for (int j = 0; j < m && sum - m + j < kMost; ++j) {
            row_run[sum - m + j] = lane;
            row_at_run[sum - m + j] = j;
            row_s[sum - m + j] = run_s[lane].row + j;
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
        // The fraction of a turn in 2^-32, exact in integers: the nearest quarter
        // and what is left of it, at most an eighth, whose float is off by 2^-28
        // turns at most.
        const uint32_t turn = (uint32_t)((uint64_t)pos * p.freqs[i] >> 32), quarter = (turn + 0x20000000u) >> 30;
        float sn, cn;
        sincospif((float)(int32_t)(turn - (quarter << 30)) * 4.656612873077393e-10f, &sn, &cn);
        const float co = quarter & 1u ? -sn : cn, si = quarter & 1u ? cn : sn, sign = quarter & 2u ? -p.amplitude : p.amplitude;
        cs[t][angle_at<D>(i)] = make_float2(co * sign, si * sign);
    }
    __syncthreads();

    // Lane j of a head's NJ holds two 16-byte chunks of it: the two halves of
    // eight rotated pairs, or neighbours (which hold whole pairs, or none).
    const int g = tid / NJ, j = tid % NJ, rc = half / 8;
    const int c0 = kPairs == 1 && j < rc ? j : 2 * j, c1 = kPairs == 1 && j < rc ? j + rc : 2 * j + 1;
    struct Head {
        uint4 a, b;
    };
    const auto fetch = [&](const uint16_t* src, bool live) {
        const uint4 z = make_uint4(0, 0, 0, 0);
        return Head{live ? *reinterpret_cast<const uint4*>(src + 8 * c0) : z, live ? *reinterpret_cast<const uint4*>(src + 8 * c1) : z};
    };
    // A head of covered row t, which its lanes hold, normalised and rotated (all
    // lanes of the warp come here; those without a head pass live = false).
    const auto turned = [&](const Head& a, const uint16_t* src, bool live, int t, bool norm, const float* weight, float (&x)[16]) {
        unpack8(a.a, x);
        unpack8(a.b, x + 8);
        float inv = 1.f;
        if (norm) {
            float ss = 0.f, s2 = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(x[e], x[e], ss);
                s2 = fmaf(x[8 + e], x[8 + e], s2);
            }
            ss += s2;
#pragma unroll
            for (int o = NJ / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float v = fmaf(ss, 1.f / D, p.eps);
            inv = v == 0.f ? 0.f : rsqrtf(v);  // (2 ulp; a sixteenth of a step of fp16)
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 u = *reinterpret_cast<const float4*>(weight + weight_at<D>(8 * c0 + e));
                const float4 v = *reinterpret_cast<const float4*>(weight + weight_at<D>(8 * c1 + e));
                const float us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[e + i] *= inv * us[i];
                    x[8 + e + i] *= inv * vs[i];
                }
            }
        }
        if (half == 0) return;
        if constexpr (kPairs == 0) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float4 f = *reinterpret_cast<const float4*>(&cs[t][angle_at<D>(8 * j + e)]);
                const float2 rs[2] = {{f.x, f.y}, {f.z, f.w}};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 r = 8 * j + e + i < half ? rs[i] : make_float2(1.f, 0.f);
                    const float u = x[2 * (e + i)], v = x[2 * (e + i) + 1];
                    x[2 * (e + i)] = u * r.x - v * r.y;
                    x[2 * (e + i) + 1] = v * r.x + u * r.y;
                }
            }
        } else if constexpr (kPairs == 1) {
            if (j < rc) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 f = *reinterpret_cast<const float4*>(&cs[t][angle_at<D>(8 * j + e)]);
                    const float2 rs[2] = {{f.x, f.y}, {f.z, f.w}};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float u = x[e + i], v = x[8 + e + i];
                        x[e + i] = u * rs[i].x - v * rs[i].y;
                        x[8 + e + i] = v * rs[i].x + u * rs[i].y;
                    }
                }
            }
        } else {
            // pairs (i, i + half) across the chunks
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int i = 16 * j + e;
                if (i < 2 * half && live) {
                    const int o = i < half ? i + half : i - half;
                    float y = __half2float(__ushort_as_half(src[o]));
                    if (norm) y *= inv * weight[weight_at<D>(o)];
                    const float2 r = cs[t][angle_at<D>(min(i, o))];
                    x[e] = i < half ? x[e] * r.x - y * r.y : x[e] * r.x + y * r.y;
                }
            }
            __syncwarp();  // in place (q_out == q): every partner is read before any is written
        }
    };
    const auto put = [&](uint16_t* dst, const uint4& a, const uint4& b) {
        *reinterpret_cast<uint4*>(dst + 8 * c0) = a;
        *reinterpret_cast<uint4*>(dst + 8 * c1) = b;
    };
    // items of `count` heads: row of the window's, head (small numbers: by one product)
    const auto split = [&](int x, int count, uint32_t by, int& t, int& h) {
        t = x < 65536 && count < 65536 ? (int)__umulhi((uint32_t)x, by) : x / count;
        if (count == 1) t = x;
        h = x - t * count;
    };

    const int part = blockIdx.y, parts = gridDim.y;
    // queries, kAhead heads of a thread's on their way together
    const int q0 = (int)((long long)p.Hq * part / parts), nq = (int)((long long)p.Hq * (part + 1) / parts) - q0;
    if (nq > 0) {
        const int items = T * nq;
        const uint32_t by = 0xffffffffu / (uint32_t)nq + 1u;
        for (int i0 = 0; i0 < items; i0 += G * kAhead) {
            Head a[kAhead];
            int t[kAhead], h[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int i = i0 + e * G + g;
                split(min(i, items - 1), nq, by, t[e], h[e]);
                a[e] = fetch(p.q + (long long)row_s[t[e]] * p.ldq + (long long)(q0 + h[e]) * D, i < items);
            }
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                if (i0 + e * G >= items) break;
                const bool live = i0 + e * G + g < items;
                const long long row = row_s[t[e]], at = (long long)(q0 + h[e]) * D;
                float y[16];
                turned(a[e], p.q + row * p.ldq + at, live, t[e], p.q_norm, wq_s, y);
                if (live) put(p.q_out + row * p.ldqo + at, pack8(y), pack8(y + 8));
            }
        }
    }
    // keys (heads 0 ..) and values (heads H ..)
    const int x0 = (int)(2ll * w.H * part / parts), x1 = (int)(2ll * w.H * (part + 1) / parts);
    if (x0 == x1) return;
    const auto source = [&](int x, int t) {
        const long long row = row_s[t];
        return x < w.H ? p.k + row * p.ldk + (long long)x * D : p.v + row * p.ldv + (long long)(x - w.H) * D;
    };
    if constexpr (!k8) {
        const auto all = [&](int first, int count, bool key) {  // rows of heads first .. of the keys or values
            if (count <= 0) return;
            const int items = T * count;
            const uint32_t by = 0xffffffffu / (uint32_t)count + 1u;
            for (int i0 = 0; i0 < items; i0 += G * kAhead) {
                Head a[kAhead];
                int t[kAhead], h[kAhead];
#pragma unroll
                for (int e = 0; e < kAhead; ++e) {
                    const int i = i0 + e * G + g;
                    split(min(i, items - 1), count, by, t[e], h[e]);
                    h[e] += first;
                    a[e] = fetch((key ? p.k + row_s[t[e]] * p.ldk : p.v + row_s[t[e]] * p.ldv) + (long long)h[e] * D, i < items);
                }
#pragma unroll
                for (int e = 0; e < kAhead; ++e) {
                    if (i0 + e * G >= items) break;
                    const bool live = i0 + e * G + g < items;
                    const long long base = run_s[row_run[t[e]]].base;
                    uint16_t* const to = (key ? w.k : w.v) + base + (long long)h[e] * w.div.d * D;
                    if (key) {
                        float y[16];
                        turned(a[e], p.k + row_s[t[e]] * p.ldk + (long long)h[e] * D, live, t[e], p.k_norm, wk_s, y);
                        if (live && base >= 0) put(to, pack8(y), pack8(y + 8));
                    } else if (live && base >= 0) {
                        put(to, a[e].a, a[e].b);
                    }
                }
            }
        };
        all(x0, min(x1, w.H) - x0, true);
        all(max(x0 - w.H, 0), x1 - w.H - max(x0 - w.H, 0), false);
    } else {
        // a few heads at a time, all their covered rows together; the next heads'
        // are on their way while these are rounded
        const int wide = T <= kBlock ? kBlock : G < 2 * kBlock ? G : 2 * kBlock, heads = G / wide;
        const int mine = g / wide, t = min(g % wide, T - 1);
        const Run& r = run_s[row_run[t]];
        const int in_run = row_at_run[t];
        const bool has = g % wide < T;
        Head a = fetch(source(min(x0 + mine, x1 - 1), t), has && x0 + mine < x1);
        for (int xb = x0, n = 0; xb < x1; xb += heads, n = n == 2 ? 0 : n + 1) {
            const bool live = has && xb + mine < x1;
            const int x = min(xb + mine, x1 - 1);
            const bool key = x < w.H;
            const int h = key ? x : x - w.H;
            float* const scale_at = (key ? p.c.ks : p.c.vs) + r.scale + (long long)h * p.c.nb;
            const Head now = a;
            a = fetch(source(min(x + heads, x1 - 1), t), has && x + heads < x1);
            const float was = live && r.old > 0 && r.base >= 0 ? *scale_at : 0.f;
            float y[16];
            if (__any_sync(0xffffffffu, key)) turned(now, source(x, t), live && key, t, p.k_norm, wk_s, y);
            if (!key) {
                unpack8(now.a, y);
                unpack8(now.b, y + 8);
            }
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                y[i] = limited(y[i]);
                top = fmaxf(top, fabsf(y[i]));  // (NaN loses)
            }
#pragma unroll
            for (int o = NJ / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (live && j == 0) atomicMax(&top_s[n][mine][row_run[t]], __float_as_uint(top));
            // Three sets of tops: this step's is read behind the barrier, the next
            // one's was cleared before it, and the one before may still be read.
            if (tid < kHeads * kWin) top_s[n == 2 ? 0 : n + 1][tid / kWin][tid % kWin] = 0u;
            __syncthreads();
            if (!live || r.base < 0) continue;
            const float scale = fmaxf(scale_for(__uint_as_float(top_s[n][mine][row_run[t]])), was);
            const float inv = 1.f / scale;
            uint8_t* const at = (key ? p.c.k : p.c.v) + r.base + (long long)h * w.div.d * D;
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = f32_e4m3(y[4 * i] * inv, y[4 * i + 1] * inv) | f32_e4m3(y[4 * i + 2] * inv, y[4 * i + 3] * inv) << 16;
            *reinterpret_cast<uint2*>(at + in_run * D + 8 * c0) = make_uint2(o[0], o[1]);
            *reinterpret_cast<uint2*>(at + in_run * D + 8 * c1) = make_uint2(o[2], o[3]);
            if (in_run == 0 && (r.old == 0 || scale != was)) {
                if (j == 0) *scale_at = scale;
                const float ratio = was * inv;
                for (int b = 1; b <= r.old; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint2* const from = reinterpret_cast<uint2*>(at - b * D + 8 * (i ? c1 : c0));
                        const uint2 v = *from;
                        *from = make_uint2(rescale4(v.x, ratio), rescale4(v.y, ratio));
                    }
            }
        }
    }
}

// -------------------------------------------------------------------- read ---
// A warp per row, 16 codes a lane.  What bounds it: bytes.  Measured: 31982 rows
// of 8 heads of 128 (197 MB in and out) 36.7 us = 5.4 TB/s, 79 % of the measured
// copy rate, with six blocks per SM (40 registers; five 38.1, eight 36.9).  With
// five: 8 codes a lane (whole sectors at a store) 41 us, 4 rows a warp that share
// their look-ups 42, blocks of 128 / 512 threads 37.9 / 43.
constexpr int kReadThreads = 256;

struct ReadArgs {
    View8 c;
    uint16_t *k, *v;
    long long ldk, ldv;
};

template <int D>
__global__ void __launch_bounds__(kReadThreads, 6) read_kernel(const __grid_constant__ ReadArgs p) {
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
            const uint32_t f2 = pack_half2(f, f);  // (a power of two: exact, and so are the products)
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[2 * e] = mul2(e4m3_half2(ws[e]), f2);
                o[2 * e + 1] = mul2(e4m3_half2_hi(ws[e]), f2);
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
// has written.  What bounds it: dependent loads (tree, path, page, scales, codes)
// behind one another.  Measured, 28 layers of 8 heads of 128: one sequence of 16
// rows 6.9 us, 32 sequences (1426 rows) 13.8 (8.0 and 16.6 where the scales of
// one destination in ten grow, which a repeated call does not see).
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
    // As many parts of the heads as give each SM a few blocks.  us, windows of 16 /
    // 8 / 4 rows: 6767 rows with norms 36.3 / 34.6 / 36, into 8 bits 40.3 / 39.2 / 50,
    // 40 rows into 8 bits 6.6 / 5.6 / 5.6.
    const int windows = (rows - 1) / q4p::kWin + 1;
    const int most = 2 * a.c.w.H < 64 ? 2 * a.c.w.H : 64;
    int parts = (8 * dev->sms + windows - 1) / windows;
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
