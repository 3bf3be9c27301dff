// Sampling a token per row of logits with temperature, top-k, top-p and
// min-p from given random numbers (q4.h section 8; BaseRT: optimal LLM
// inference on Apple Silicon with native Metal, §3.3 lists sampling among the
// decode kernels).
//
// Mathematics: in the order (logit descending, index ascending) every limit
// keeps a beginning, and the choice itself is the first place where a running
// sum passes a bound.  So each step is one search: the place where the count
// (top-k) or the weight (top-p, the choice) of what stands before it reaches
// a target.
//
// Weights are integers, round(2^44 2^-t) with t = (max - l) log2(e) / T: their
// sums are exact in any order (2^19 of them stay below 2^63), so neither
// atomics nor the split of the work can change a token.  A weight carries an
// error near 2^-31 of itself (t as a float pair, below), where a plain fp32
// exponential's 2^-23 would move the borders of the tail's tokens, which are
// narrower than that.
//
// GB300 design: a cluster of up to 16 CTAs per row, so that one row alone
// still uses 16 SMs; the CTAs' tops, sums and lists meet in distributed shared
// memory and the whole call is one launch.  The row comes from memory once and
// from L2 after that:
//   1. the greatest logit (and each thread's own greatest);
//   2. a threshold that leaves about as many tokens as can matter: the bin of
//      t that holds the N-th greatest of the threads' greatest logits (at
//      least N tokens are as great), N = top_k or kWanted;
//   3. the tokens above it into lists, and, unless top_k makes it needless,
//      the weight of all; one CTA sorts the list (a few hundred), scans its
//      weights and finds every limit in it.
// What does not end inside the list (a flat distribution, the tail's share of
// u) goes on: a histogram of counts and weights over 1536 bins of t, then the
// tokens of the bin that holds the target, sorted as before; and where one
// bin holds more than the list (thousands of equal logits), eight bits of the
// key at a time.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include "q4_device.cuh"
#include "q4_internal.h"

namespace q4s {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxVocab = 1 << 19;
constexpr int kMaxCluster = 16;
constexpr int kWanted = 512;         // tokens the list aims at without top_k
constexpr int kMostK = 1024;         // top_k up to which the list is tried
constexpr int kList = 1024;          // tokens of a CTA's list
constexpr int kAll = 2048;           // tokens of the joined list
constexpr int kCut = 512;            // bins of the threshold: 16 per octave
constexpr int kBins = 1536;          // bins of the histogram: 32 per octave, 48 octaves (weights end at 45)
constexpr u64 kOne = 1ull << 44;     // the weight of the greatest logit
constexpr uint32_t kLeast = 0x007FFFFFu;  // key of -inf: takes no part

struct Args {
    const void* logits;
    int vocab;
    long long ld;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t* top_k;
    int32_t* tokens;
    float* probs;
    int cluster;
};

struct Shared {
    u64 xch[2][kMaxCluster][2];  // exchange between the CTAs, double-buffered
    u64 red[kWarps + 1];
    u64 result[4];
    u64 all[kAll];    // the joined list, sorted
    u64 pre[kAll];    // its running weights
    u64 list[kList];  // this CTA's tokens: key << 32 | ~index
    u64 mw[kBins];    // the cluster's histogram, then its running sums
    uint32_t mc[kBins];
    uint32_t cnt[kBins], lo[kBins], hi[kBins];  // this CTA's histogram; cnt is also the threshold's
    uint32_t pow64[64];
    uint32_t count;  // of list
    int cut;
};

// Greater float, greater key; -0 counts as +0, NaN as -inf.
__device__ __forceinline__ uint32_t key_of(float f) {
    uint32_t b = __float_as_uint(f);
    if ((b & 0x7fffffffu) > 0x7f800000u) return kLeast;
    if (b == 0x80000000u) b = 0;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

struct Scale {
    float max, hi, lo;  // log2(e) / T = hi + lo
};

// t in fp32, as the bins see it: monotone in the logit.
__device__ __forceinline__ float coarse_t(float l, const Scale& c) { return l == c.max ? 0.f : (c.max - l) * c.hi; }

__device__ __forceinline__ u64 weight_of(float l, const Scale& c, const uint32_t* pow64) {
    if (l == c.max) return kOne;
    // d + de = max - l exactly (the error of a difference is a float)
    const float d = c.max - l;
    // t + te = (d + de) (hi + lo) to about 2^-46 of it
    const float t = d * c.hi;
    if (!(t < 46.f)) return 0;
    const float b = d - c.max;
    const float de = (c.max - (d - b)) + (-l - b);
    const float te = fmaf(d, c.hi, -t) + fmaf(d, c.lo, de * c.hi);
    const float n = floorf(t);
    const float f = t - n;                    // exact
    const int j = (int)(f * 64.f);            // 2^-f = 2^(-j/64) 2^-r
    const float r = (f - (float)j * 0.015625f) + te;  // the difference is exact; |r| < 2^-6 + a little
    // 2^-r = 1 - y, y = z - z^2 / 2 + z^3 / 6 - z^4 / 24, z = r ln 2; the next
    // term is below 2^-39
    const float z = r * 0.69314718f;
    const float y = z * (1.f - z * (0.5f - z * (0.16666667f - z * 0.041666668f)));
    const uint32_t p = pow64[j];
    const long long m = (long long)p - (long long)__float2int_rn((float)p * y);  // units of 2^-32, about 2^31 .. 2^32
    // 2^44 2^-n m 2^-32, rounded
    const int sh = 12 - (int)n;
    if (sh >= 0) return (u64)(m << sh);
    return (u64)((m + (1ll << (-sh - 1))) >> -sh);
}

// This CTA's part of a row: 16-byte vectors v0 .. v1 - 1 behind `head` single
// elements (the first CTA's) and before the last ones (the last CTA's), so
// that the CTAs' parts are in index order.
template <bool HALF>
struct Part {
    using E = typename std::conditional<HALF, uint16_t, float>::type;
    static constexpr int VE = HALF ? 8 : 4;
    const E* row;
    int vocab, head, v0, v1, tail, rank, ranks;

    __device__ Part(const Args& a, int r, int rank_) : vocab(a.vocab), rank(rank_), ranks(a.cluster) {
        row = static_cast<const E*>(a.logits) + r * a.ld;
        const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(E));
        head = min(vocab, (VE - off) % VE);
        const int nv = (vocab - head) / VE;
        v0 = (int)((long long)nv * rank / ranks);
        v1 = (int)((long long)nv * (rank + 1) / ranks);
        tail = head + nv * VE;
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (HALF) return __half2float(__ushort_as_half(row[i]));
        else return row[i];
    }
    // f(value, index) for every element of the part, four vectors in flight
    // per thread; a thread's indices ascend.
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        if (rank == 0 && (int)threadIdx.x < head) f(at(threadIdx.x), (int)threadIdx.x);
        const uint4* vec = reinterpret_cast<const uint4*>(row + head);
        for (int v = v0 + threadIdx.x; v < v1; v += 4 * kThreads) {
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v + i * kThreads < v1) w[i] = vec[v + i * kThreads];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (v + i * kThreads >= v1) break;
                const int at0 = head + (v + i * kThreads) * VE;
                const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                if constexpr (HALF) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f(__half2float(__ushort_as_half((uint16_t)(x[e >> 1] >> (16 * (e & 1))))), at0 + e);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) f(__uint_as_float(x[e]), at0 + e);
                }
            }
        }
        if (rank == ranks - 1 && tail + (int)threadIdx.x < vocab) f(at(tail + threadIdx.x), tail + (int)threadIdx.x);
    }
};

__device__ __forceinline__ u64 block_sum(u64 x, Shared& s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = x;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) t += s.red[i];
    return t;
}

// Inclusive running sum of one value per thread.
__device__ __forceinline__ u64 block_scan(u64 x, Shared& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += t;
    }
    __syncthreads();
    if (lane == 31) s.red[warp] = x;
    __syncthreads();
    for (int i = 0; i < warp; ++i) x += s.red[i];
    return x;
}

struct Pair {
    u64 a, b;
};

// What the cluster's CTAs share: `mine` (the same in all threads of a CTA)
// goes to every CTA; the values of rank r are then xch[phase][r].  The buffers
// alternate: one is written again only after the next exchange, at which
// every CTA has read it.
struct Cluster {
    cg::cluster_group g;
    int rank, ranks, phase;
    __device__ const u64 (*exchange(Shared& s, Pair mine))[2] {
        if ((int)threadIdx.x < ranks) {
            u64* dst = g.map_shared_rank(&s.xch[phase][rank][0], threadIdx.x);
            dst[0] = mine.a;
            dst[1] = mine.b;
        }
        g.sync();
        const u64(*r)[2] = s.xch[phase];
        phase ^= 1;
        return r;
    }
};

// Sorts all[0 .. n) descending (bitonic, padded with zeros to a power of two)
// and leaves the running weights in pre[].
__device__ void sort_and_scan(Shared& s, int n, const Scale& c) {
    int m = 2;
    while (m < n) m *= 2;
    for (int i = n + threadIdx.x; i < m; i += kThreads) s.all[i] = 0;
    __syncthreads();
    for (int size = 2; size <= m; size *= 2)
        for (int step = size / 2; step > 0; step /= 2) {
            for (int i = threadIdx.x; i < m / 2; i += kThreads) {
                const int a = 2 * i - (i & (step - 1)), b = a + step;
                const u64 x = s.all[a], y = s.all[b];
                if ((x < y) == ((a & size) == 0)) {
                    s.all[a] = y;
                    s.all[b] = x;
                }
            }
            __syncthreads();
        }
    constexpr int P = kAll / kThreads;
    u64 w[P], t = 0;
#pragma unroll
    for (int e = 0; e < P; ++e) {
        const int i = P * threadIdx.x + e;
        if (i < n) t += weight_of(key_value((uint32_t)(s.all[i] >> 32)), c, s.pow64);
        w[e] = t;
    }
    const u64 before = block_scan(t, s) - t;
#pragma unroll
    for (int e = 0; e < P; ++e)
        if (P * (int)threadIdx.x + e < n) s.pre[P * threadIdx.x + e] = before + w[e];
    __syncthreads();
}

// First place of pre[0 .. n) that reaches target (there is one), to all threads.
__device__ int reach(Shared& s, int n, u64 target) {
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (s.pre[i] >= target && (i == 0 || s.pre[i - 1] < target)) s.result[3] = i;
    __syncthreads();
    const int i = (int)s.result[3];
    __syncthreads();
    return i;
}

// The joined list into rank 0's all[], from every CTA's list.
__device__ void gather(Shared& s, Cluster& cl, const u64 (*counts)[2]) {
    int at = 0;
    for (int r = 0; r < cl.ranks; ++r) {
        const u64* src = cl.g.map_shared_rank(&s.list[0], r);
        const int n = (int)counts[r][0];
        for (int i = threadIdx.x; i < n; i += kThreads) s.all[at + i] = src[i];
        at += n;
    }
    __syncthreads();
}

__device__ __forceinline__ void append(Shared& s, uint32_t key, int index) {
    const uint32_t i = atomicAdd(&s.count, 1u);
    if (i < kList) s.list[i] = (u64)key << 32 | (uint32_t)~index;
}

// Histogram of a CTA: counts and weights as 32-bit halves with the carry
// passed on, a run of equal bins added at once (logits that are all equal
// would otherwise queue at one address).
struct Tally {
    int bin = -1;
    uint32_t n = 0;
    u64 w = 0;
    __device__ __forceinline__ void flush(Shared& s) {
        if (n == 0) return;
        atomicAdd(&s.cnt[bin], n);
        const uint32_t l = (uint32_t)w;
        const uint32_t old = atomicAdd(&s.lo[bin], l);
        const uint32_t h = (uint32_t)(w >> 32) + (old + l < old ? 1u : 0u);
        if (h) atomicAdd(&s.hi[bin], h);
        n = 0;
        w = 0;
    }
    __device__ __forceinline__ void add(Shared& s, int b, u64 x) {
        if (b != bin) {
            flush(s);
            bin = b;
        }
        ++n;
        w += x;
    }
};

// Every CTA's histogram of `bins` bins (descending logits), joined and summed
// up from the front, into every CTA's mc[], mw[] (at offset `at`).
__device__ void join_histogram(Shared& s, Cluster& cl, int bins) {
    cl.g.sync();  // all histograms done
    const int b0 = bins * cl.rank / cl.ranks, b1 = bins * (cl.rank + 1) / cl.ranks;
    for (int b = b0 + threadIdx.x; b < b1; b += kThreads) {
        uint32_t n = 0;
        u64 w = 0;
        for (int r = 0; r < cl.ranks; ++r) {
            n += *cl.g.map_shared_rank(&s.cnt[b], r);
            w += (u64)*cl.g.map_shared_rank(&s.lo[b], r) + ((u64)*cl.g.map_shared_rank(&s.hi[b], r) << 32);
        }
        for (int r = 0; r < cl.ranks; ++r) {
            *cl.g.map_shared_rank(&s.mc[b], r) = n;
            *cl.g.map_shared_rank(&s.mw[b], r) = w;
        }
    }
    cl.g.sync();
    constexpr int P = kBins / kThreads;
    u64 n[P], w[P], tn = 0, tw = 0;
#pragma unroll
    for (int e = 0; e < P; ++e) {
        const int b = P * threadIdx.x + e;
        if (b < bins) {
            tn += s.mc[b];
            tw += s.mw[b];
        }
        n[e] = tn;
        w[e] = tw;
    }
    const u64 bn = block_scan(tn, s) - tn, bw = block_scan(tw, s) - tw;
#pragma unroll
    for (int e = 0; e < P; ++e) {
        const int b = P * threadIdx.x + e;
        if (b < bins) {
            s.mc[b] = (uint32_t)(bn + n[e]);
            s.mw[b] = bw + w[e];
        }
    }
    __syncthreads();
}

// First bin whose running count or weight reaches target (there is one).
__device__ int reach_bin(Shared& s, int bins, bool by_count, u64 target) {
    for (int b = threadIdx.x; b < bins; b += kThreads) {
        const u64 x = by_count ? s.mc[b] : s.mw[b];
        const u64 y = b == 0 ? 0 : by_count ? s.mc[b - 1] : s.mw[b - 1];
        if (x >= target && y < target) s.result[2] = b;
    }
    __syncthreads();
    const int b = (int)s.result[2];
    __syncthreads();
    return b;
}

__device__ __forceinline__ void clear_histogram(Shared& s, int bins) {
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kThreads) s.cnt[b] = s.lo[b] = s.hi[b] = 0;
    __syncthreads();
}

__device__ __forceinline__ int bin_of(float l, const Scale& c) {
    return (int)fminf(coarse_t(l, c) * 32.f, (float)(kBins - 1));
}

struct Hit {
    u64 weight;  // of everything up to the place, and of the token there
    u64 own;
    int token;
};

// The place where the count or weight of the tokens of `bin` reaches target
// (what stands before the bin already taken off): its running weight within
// the bin and, if asked, its token.
template <bool HALF>
__device__ Hit search_bin(const Part<HALF>& row, Shared& s, Cluster& cl, const Scale& c, int bin, bool by_count,
                          u64 target) {
    __syncthreads();
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
    row.each([&](float l, int i) {
        const uint32_t k = key_of(l);
        if (k != kLeast && bin_of(l, c) == bin) append(s, k, i);
    });
    __syncthreads();
    const u64(*n)[2] = cl.exchange(s, {s.count, 0});
    u64 total = 0;
    bool fits = true;
    for (int r = 0; r < cl.ranks; ++r) {
        total += n[r][0];
        fits = fits && n[r][0] <= kList;
    }
    Hit h;
    if (fits && total <= kAll) {
        u64 place = 0, pre = 0, own = 0;
        if (cl.rank == 0) {
            gather(s, cl, n);
            sort_and_scan(s, (int)total, c);
            place = by_count ? target - 1 : reach(s, (int)total, target);
            pre = s.pre[place];
            own = pre - (place ? s.pre[place - 1] : 0);
            place = (uint32_t)~(uint32_t)s.all[place];
        }
        const u64(*x)[2] = cl.exchange(s, {pre, place});
        h.weight = x[0][0];
        h.token = (int)x[0][1];
        const u64(*y)[2] = cl.exchange(s, {own, 0});
        h.own = y[0][0];
        return h;
    }
    // eight bits of the key at a time, the greatest first
    uint32_t prefix = 0;
    u64 wb = 0, nb = 0, equal = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        clear_histogram(s, 256);
        Tally t;
        row.each([&](float l, int i) {
            const uint32_t k = key_of(l);
            if (k == kLeast || bin_of(l, c) != bin || (shift < 24 && k >> (shift + 8) != prefix >> (shift + 8))) return;
            t.add(s, 255 - (int)(k >> shift & 255u), weight_of(key_value(k), c, s.pow64));
        });
        t.flush(s);
        join_histogram(s, cl, 256);
        const int b = reach_bin(s, 256, by_count, target - (by_count ? nb : wb));
        const u64 n0 = b ? s.mc[b - 1] : 0, w0 = b ? s.mw[b - 1] : 0;
        equal = s.mc[b] - n0;
        nb += n0;
        wb += w0;
        prefix |= (uint32_t)(255 - b) << shift;
    }
    h.own = weight_of(key_value(prefix), c, s.pow64);
    u64 place = by_count ? target - nb - 1 : h.own ? (target - wb - 1) / h.own : 0;  // among the equal keys
    if (place >= equal) place = equal - 1;
    h.weight = wb + (place + 1) * h.own;
    // its index: the parts are in index order, and a CTA walks its part so
    u64 mine = 0;
    row.each([&](float l, int) { mine += key_of(l) == prefix; });
    mine = block_sum(mine, s);
    const u64(*x)[2] = cl.exchange(s, {mine, 0});
    u64 before = 0;
    for (int r = 0; r < cl.rank; ++r) before += x[r][0];
    u64 found = 0;
    if (before <= place && place < before + mine) {
        const int i0 = row.rank == 0 ? 0 : row.head + row.v0 * Part<HALF>::VE;
        const int i1 = row.rank == row.ranks - 1 ? row.vocab : row.head + row.v1 * Part<HALF>::VE;
        u64 seen = before;
        for (int i = i0; i < i1 && seen <= place; i += kThreads) {
            const bool eq = i + (int)threadIdx.x < i1 && key_of(row.at(i + threadIdx.x)) == prefix;
            const u64 run = block_scan(eq, s);
            if (eq && seen + run == place + 1) s.result[1] = i + threadIdx.x + 1;
            __syncthreads();
            if (threadIdx.x == kThreads - 1) s.result[0] = run;
            __syncthreads();
            seen += s.result[0];
        }
        found = s.result[1];
    }
    const u64(*y)[2] = cl.exchange(s, {found, 0});
    h.token = -1;
    for (int r = 0; r < cl.ranks; ++r)
        if (y[r][0]) h.token = (int)y[r][0] - 1;
    return h;
}

__device__ __forceinline__ u64 share_target(double share, u64 W) {  // least integer at or above share * W, 1 .. W
    const double want = ceil(fmax(share, 0.0) * (double)W);
    return want < 1.0 ? 1 : want > (double)W ? W : (u64)want;
}

template <bool HALF>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const Args a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& s = *reinterpret_cast<Shared*>(smem);
    Cluster cl{cg::this_cluster(), 0, a.cluster, 0};
    cl.rank = (int)cl.g.block_rank();
    const int r = blockIdx.x / a.cluster, tid = threadIdx.x;
    const Part<HALF> row(a, r, cl.rank);
    if (tid < 64) s.pow64[tid] = (uint32_t)fmin(4294967295.0, rint(exp2(-tid / 64.0) * 4294967296.0));
    for (int b = tid; b < kCut; b += kThreads) s.cnt[b] = 0;
    if (tid == 0) s.count = 0;
    const auto finish = [&](int token, double prob) {
        if (cl.rank == 0 && tid == 0) {
            a.tokens[r] = token;
            if (a.probs) a.probs[r] = (float)prob;
        }
    };

    // 1. the greatest logit, at its lowest index
    float best = -INFINITY;
    int best_at = 0;
    row.each([&](float l, int i) {
        if (l > best) {
            best = l;
            best_at = i;
        }
    });
    const bool any = best > -INFINITY;
    {
        u64 m = any ? (u64)key_of(best) << 32 | (uint32_t)~best_at : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const u64 t = __shfl_xor_sync(0xffffffffu, m, o);
            m = t > m ? t : m;
        }
        if ((tid & 31) == 0) s.red[tid >> 5] = m;
        __syncthreads();
    }
    u64 top = 0;
    for (int i = 0; i < kWarps; ++i) top = s.red[i] > top ? s.red[i] : top;
    cl.g.sync();  // every CTA of the cluster runs: its shared memory can be written
    {
        const u64(*x)[2] = cl.exchange(s, {top, 0});
        for (int i = 0; i < cl.ranks; ++i) top = x[i][0] > top ? x[i][0] : top;
    }
    const float T = a.temperature ? a.temperature[r] : 1.f;
    const int k = a.top_k ? a.top_k[r] : 0;
    if (top == 0 || !a.u || !(T > 0.f) || k == 1) {
        if (top == 0) finish(-1, 0.0);
        else finish((int)(uint32_t)~(uint32_t)top, 1.0);
        cl.g.sync();  // no CTA leaves while another may still write to it
        return;
    }
    Scale c;
    {
        c.max = key_value((uint32_t)(top >> 32));
        const double f = fmin(1.4426950408889634 / (double)T, 1e30);
        c.hi = (float)f;
        c.lo = (float)(f - (double)c.hi);
    }
    const bool with_k = k > 0 && k < a.vocab;
    const float p = a.top_p ? a.top_p[r] : 1.f;
    const float mp = a.min_p ? a.min_p[r] : 0.f;
    const double least = mp > 0.f ? (double)fminf(mp, 1.f) * (double)kOne : 0.0;
    const double u = fmin(fmax((double)a.u[r], 0.0), 1.0);

    // 2. the threshold
    if (any) atomicAdd(&s.cnt[(int)fminf(coarse_t(best, c) * 16.f, (float)(kCut - 1))], 1u);
    cl.g.sync();
    {
        uint32_t n = 0;
        for (int i = 0; i < cl.ranks; ++i) n += *cl.g.map_shared_rank(&s.cnt[tid], i);
        const u64 wanted = with_k && k <= kMostK ? k : kWanted;
        const u64 run = block_scan(n, s);
        if (tid == 0) s.cut = kCut - 1;
        __syncthreads();
        if (run >= wanted && run - n < wanted) s.cut = tid;
        __syncthreads();
    }
    static_assert(kCut == kThreads, "a bin per thread");
    const float cut = (float)(s.cut + 1);

    // 3. the list, and the weight of all
    u64 all = 0, rest = 0;
    row.each([&](float l, int i) {
        const float t = coarse_t(l, c) * 16.f;
        if (t < cut) {
            append(s, key_of(l), i);
        } else if (l > -INFINITY) {
            ++rest;
        }
        if (!with_k && l > -INFINITY) all += weight_of(l, c, s.pow64);
    });
    all = block_sum(all, s);
    rest = block_sum(rest, s);
    u64 n_list = 0, W = 0;
    bool fits = true, done = false;
    const u64(*n)[2] = cl.exchange(s, {s.count, rest});
    rest = 0;
    for (int i = 0; i < cl.ranks; ++i) {
        n_list += n[i][0];
        rest += n[i][1];
        fits = fits && n[i][0] <= kList;
    }
    fits = fits && n_list <= kAll;
    if (fits && cl.rank == 0) gather(s, cl, n);
    {
        const u64(*x)[2] = cl.exchange(s, {all, 0});
        for (int i = 0; i < cl.ranks; ++i) W += x[i][0];
    }
    if (fits && cl.rank == 0) {
        const int N = (int)n_list;
        sort_and_scan(s, N, c);
        const u64 W_list = s.pre[N - 1];
        bool ok = true;
        if (with_k) {
            ok = k <= N || rest == 0;
            W = s.pre[min(k, N) - 1];
        }
        if (ok && p < 1.f) {
            const u64 target = share_target((double)p, W);
            ok = target <= W_list;
            if (ok) W = s.pre[reach(s, N, target)];
        }
        if (ok && least > 0.0) {
            int m = 0;  // the ones that min_p keeps
            for (int i0 = 0; i0 < N; i0 += kThreads) {
                const int i = i0 + tid;
                m += __syncthreads_count(i < N && (double)(s.pre[i] - (i ? s.pre[i - 1] : 0)) >= least);
            }
            if (m < N || rest == 0) W = min(W, s.pre[m - 1]);
            else ok = W <= W_list;
        }
        if (ok) {
            const u64 target = min(W, (u64)(u * (double)W) + 1);
            ok = target <= W_list;
            if (ok) {
                const int i = reach(s, N, target);
                finish((int)(uint32_t)~(uint32_t)s.all[i], (double)(s.pre[i] - (i ? s.pre[i - 1] : 0)) / (double)W);
            }
        }
        done = ok;
    }
    {
        const u64(*x)[2] = cl.exchange(s, {done, 0});
        done = x[0][0] != 0;
    }
    if (!done) {
        // what the list does not decide: the histogram over all
        clear_histogram(s, kBins);
        u64 some = 0;
        Tally t;
        row.each([&](float l, int) {
            if (!(l > -INFINITY)) return;
            const u64 w = weight_of(l, c, s.pow64);
            if (w == 0) return;
            if ((double)w >= least) some += w;
            t.add(s, bin_of(l, c), w);
        });
        t.flush(s);
        some = block_sum(some, s);
        {
            const u64(*x)[2] = cl.exchange(s, {some, 0});
            some = 0;
            for (int i = 0; i < cl.ranks; ++i) some += x[i][0];
        }
        join_histogram(s, cl, kBins);
        // the running sums are needed for up to three searches, which use the
        // same arrays where a bin overflows the list: the last one's bin and
        // target are found before that, the others' leave a sum only
        W = s.mw[kBins - 1];
        const auto before = [&](int b, bool by_count) -> u64 {
            return b == 0 ? 0 : by_count ? (u64)s.mc[b - 1] : s.mw[b - 1];
        };
        const auto again = [&]() {  // the histogram, where a search has used its arrays
            clear_histogram(s, kBins);
            Tally t2;
            row.each([&](float l, int) {
                if (!(l > -INFINITY)) return;
                const u64 w = weight_of(l, c, s.pow64);
                if (w) t2.add(s, bin_of(l, c), w);
            });
            t2.flush(s);
            join_histogram(s, cl, kBins);
        };
        if (with_k && (u64)k < s.mc[kBins - 1]) {
            const int b = reach_bin(s, kBins, true, k);
            const u64 wb = before(b, false);
            const u64 nb = before(b, true);
            const bool big = s.mc[b] - nb > kList;  // may not fit the list
            W = wb + search_bin<HALF>(row, s, cl, c, b, true, k - nb).weight;
            if (big) again();
        }
        if (p < 1.f) {
            const u64 target = share_target((double)p, W);
            const int b = reach_bin(s, kBins, false, target);
            const u64 wb = before(b, false);
            const bool big = s.mc[b] - before(b, true) > kList;
            W = wb + search_bin<HALF>(row, s, cl, c, b, false, target - wb).weight;
            if (big) again();
        }
        if (least > 0.0) W = min(W, some);
        const u64 target = min(W, (u64)(u * (double)W) + 1);
        const int b = reach_bin(s, kBins, false, target);
        const Hit h = search_bin<HALF>(row, s, cl, c, b, false, target - before(b, false));
        finish(h.token, (double)h.own / (double)W);
    }
    cl.g.sync();  // no CTA leaves while another may still use its shared memory
}

template <bool HALF>
cudaError_t launch(Args& a, int rows, int sms, cudaStream_t stream) {
    // As many CTAs per row as two per SM allow, each with at least 2048
    // tokens.  16 CTAs need the non-portable cluster size.
    int c = kMaxCluster;
    while (c > 1 && ((long long)rows * c > 2 * sms || a.vocab < 2048 * c / 2 + 1)) c /= 2;
    a.cluster = c;
    static std::atomic<int> marks[64], wide[64];
    const void* kern = reinterpret_cast<const void*>(sample_kernel<HALF>);
    cudaError_t e = q4i::ensure_smem_attr(kern, marks, (int)sizeof(Shared));
    if (e != cudaSuccess) return e;
    int dev = 0;
    cudaGetDevice(&dev);
    if (c > 8 && !wide[dev & 63].load(std::memory_order_acquire)) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
        wide[dev & 63].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * c));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)c;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<HALF>, a);
}

}  // namespace q4s

using namespace q4i;

extern "C" q4_status q4_sample(const q4_sample_desc* desc, q4_stream_t stream) {
    clear_error();
    if (!desc) return fail(Q4_ERR_INVALID_ARG, "desc is NULL");
    const q4_sample_desc& d = *desc;
    if (d.dtype != Q4_F32 && d.dtype != Q4_F16) return fail(Q4_ERR_INVALID_ARG, "bad dtype");
    if (d.rows < 0 || d.vocab < 1) return fail(Q4_ERR_INVALID_ARG, "rows=%d vocab=%d", d.rows, d.vocab);
    if (d.vocab > q4s::kMaxVocab) return fail(Q4_ERR_UNSUPPORTED, "vocab=%d above %d", d.vocab, q4s::kMaxVocab);
    if (d.ld != 0 && d.ld < d.vocab) return fail(Q4_ERR_INVALID_ARG, "row stride %d, vocab=%d", d.ld, d.vocab);
    if (!d.logits || !d.tokens) return fail(Q4_ERR_INVALID_ARG, "NULL pointer argument");
    if (reinterpret_cast<uintptr_t>(d.logits) & (d.dtype == Q4_F16 ? 1u : 3u))
        return fail(Q4_ERR_MISALIGNED, "logits must be aligned to their elements");
    const DeviceInfo* dev = nullptr;
    const q4_status st = current_device(&dev);
    if (st != Q4_OK) return st;
    if (d.rows == 0) return Q4_OK;
    q4s::Args a;
    a.logits = d.logits;
    a.vocab = d.vocab;
    a.ld = d.ld ? d.ld : d.vocab;
    a.temperature = d.temperature;
    a.top_p = d.top_p;
    a.min_p = d.min_p;
    a.u = d.u;
    a.top_k = d.top_k;
    a.tokens = d.tokens;
    a.probs = d.probs;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = d.dtype == Q4_F16 ? q4s::launch<true>(a, d.rows, dev->sms, s) : q4s::launch<false>(a, d.rows, dev->sms, s);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "q4_sample launch");
}
