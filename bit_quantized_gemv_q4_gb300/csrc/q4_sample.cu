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
// error near 2^-30 of itself (t as a float pair, below), where a plain fp32
// exponential's 2^-23 would move the borders of the tail's tokens, which are
// narrower than that.
//
// GB300 design: a cluster of up to 8 CTAs per row, so that one row alone
// still uses 8 SMs; the CTAs' tops, sums and lists meet in distributed shared
// memory and the whole call is one launch.  The row comes from memory once and
// from L2 after that:
//   1. the greatest logit (and each thread's own greatest);
//   2. a threshold that leaves about as many tokens as can matter: the bin of
//      t that holds the N-th greatest of the threads' greatest logits (at
//      least N tokens are as great), N = top_k or kWanted;
//   3. the tokens above it into lists, and, unless top_k makes it needless,
//      the weight of all and a histogram of the weights below it (1536 bins of
//      t); one CTA sorts the list (a few hundred), scans its weights and finds
//      in it whatever limit ends there.
// A target below the list (a flat distribution's nucleus, the tail's share of
// u) is found in the histogram; the tokens of its bin are collected and
// sorted as before.  Where one bin holds more than such a list (thousands of
// equal logits), and where the list itself overflows, the search goes eight
// bits of the key at a time.
//
// What bounds it: the passes' instructions (35 a token in pass 3: the weight,
// its step's bin, the list), and behind them a chain of exchanges, barriers and
// short passes; DRAM is read once.  Measured: 256 rows of 50257 fp16 logits,
// top_p 0.9 in all, 56 us (26 MB, 0.5 TB/s), 51 where the rows lie in L2: the
// greatest logit and the threshold 12, pass 3 18 (5 of them the histogram's
// atomics, 1 the rounding error of max - l), the list 3, the rest what the tail
// needs; SMs with two rows issue in up to 93 % of their cycles.  61 rows of
// 151936 with every setting in turn 55 us, 45 from L2; one row with top_k 50
// 14 us.  Both kernels stand at 64 registers (two CTAs of 512 threads per SM)
// and spill: 72 bytes stored and 200 loaded (fp32), 48 and 156 (fp16).
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
constexpr int kMaxCluster = 8;
constexpr int kWanted = 96;          // tokens the list aims at without top_k (256 rows, of 63 us: 320 74, 160 65, 40 63)
constexpr int kMostK = 1024;         // top_k up to which the list is tried
constexpr int kList = 1024;          // tokens of a CTA's list
constexpr int kAll = 2048;           // tokens of the joined list
constexpr int kBinList = 1024;       // tokens of a bin that are sorted together
constexpr int kCounting = 256;       // up to here a sort counts, per token, the greater ones (one row 14 us, bitonic 19)
// Tokens of a CTA, so that sums of 15-bit parts of their weights stay below 2^32:
// with its last vector and up to 7 single elements a part has 2^17 - 1 at most.
constexpr int kMostPart = (1 << 17) - 8;
constexpr int kCut = 512;            // bins of the threshold: 16 per octave (4 steps)
constexpr int kBins = 1536;          // bins of a histogram: a step each from the threshold on, or two steps from t = 0 on
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
    u64 xch[2][kMaxCluster][4];  // exchange between the CTAs, double-buffered
    u64 red[4][kWarps];
    u64 result[4];
    u64 all[kAll];         // the joined list, sorted
    u64 pre[kAll];         // its running weights
    u64 bin_all[kBinList];  // likewise a bin's tokens
    u64 bin_pre[kBinList];
    u64 list[kList];  // this CTA's tokens: key << 32 | ~index
    u64 mw[kBins];    // the cluster's histogram, then its running sums
    uint32_t mc[kBins];
    uint32_t h0[kBins], h1[kBins], h2[kBins];  // this CTA's histogram: two parts of short weights, or (count, low, high)
    uint32_t cut_count[kCut];                  // the threads' greatest logits
    float2 pow64[64];  // 2^(-j/64) in units of 2^-29 (short_weight)
    uint32_t count;    // of list
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

// Adding 1.5 2^23 rounds a float below 2^22 to an integer in its low mantissa
// bits, which keeps conversions off the slow pipe.
constexpr float kMagic = 12582912.f;
__device__ __forceinline__ int magic_int(float x) { return __float_as_int(x) - __float_as_int(kMagic); }

// Steps of a logit: 64 t to the nearest integer, kSteps from t = 46 on (no
// weight there).  Monotone in the logit; every bin is a range of steps.
constexpr float kEnd = 46.f;
constexpr int kSteps = 64 * 46 + 1;
constexpr float kLast = kMagic + 64.f * 46.f;  // (that step's weight rounds to zero)
__device__ __forceinline__ int steps_of(float l, const Scale& c) {
    const float d = l == c.max ? 0.f : c.max - l;
    return d * c.hi < kEnd ? magic_int(fmaf(d, c.hi * 64.f, kMagic)) : kSteps;
}

// round(2^29 2^(-j/64))
__constant__ uint32_t kPow64[64] = {
    536870912u, 531087746u, 525366875u, 519707630u, 514109347u, 508571368u, 503093043u, 497673732u,
    492312797u, 487009610u, 481763549u, 476573998u, 471440350u, 466362000u, 461338355u, 456368824u,
    451452825u, 446589781u, 441779122u, 437020283u, 432312707u, 427655840u, 423049137u, 418492057u,
    413984066u, 409524635u, 405113241u, 400749367u, 396432500u, 392162134u, 387937769u, 383758908u,
    379625062u, 375535746u, 371490480u, 367488790u, 363530205u, 359614263u, 355740503u, 351908471u,
    348117717u, 344367798u, 340658272u, 336988706u, 333358668u, 329767733u, 326215479u, 322701490u,
    319225354u, 315786663u, 312385013u, 309020006u, 305691246u, 302398344u, 299140913u, 295918571u,
    292730940u, 289577647u, 286458320u, 283372595u, 280320109u, 277300504u, 274313427u, 271358526u,
};

// A weight 2^44 2^(-k/64) (1 - y), rounded (kf = kMagic + k, k >= 0, |y| <
// 0.0056), is short_weight << left(k), and short_weight is below 2^29 + 2^22.
// The table holds an integer's bits, with those of kMagic added, and a float.
constexpr uint32_t kMagicBits = 0x4B400000u;  // kMagic; its low six bits are zero
__device__ __forceinline__ int left(int k) { return max(15 - (k >> 6), 0); }
__device__ __forceinline__ uint32_t short_weight(float kf, float y, const float2* pow64) {
    const uint32_t bits = __float_as_uint(kf);
    const float2 p = pow64[bits & 63];
    // units of 2^-29: 2^28 .. 2^29; |p y| < 2^22
    const uint32_t m = __float_as_uint(p.x) - __float_as_uint(fmaf(p.y, y, kMagic));
    const int sh = max((int)(bits >> 6) - (int)(kMagicBits >> 6) - 15, 0);
    return (m + ((1u << sh) >> 1)) >> sh;
}

constexpr float kZ1 = 0.0108304247f, kZ2 = -5.86490495e-05f, kZ3 = 2.11731307e-07f;  // ln2/64, -its square / 2, its cube / 6

// round(2^44 2^-t).  The passes over a row (two_of below) do the same
// operations on two logits at a time, so a token has one weight.
__device__ __forceinline__ u64 weight_of(float l, const Scale& c, const float2* pow64) {
    if (l == c.max) return kOne;
    // d + de = max - l exactly (the error of a difference is a float)
    const float d = c.max - l;
    if (!(d * c.hi < kEnd)) return 0;
    const float b = d - c.max;
    const float de = (c.max - (d - b)) + (-l - b);
    // 64 t = k + r, |r| <= 1/2 and a little: the product less k is one fused
    // operation, so nothing of it is lost; then its smaller parts
    const float hi = c.hi * 64.f, lo = c.lo * 64.f;  // exact
    const float kf = fmaf(d, hi, kMagic);
    float r = fmaf(d, hi, -(kf - kMagic));
    r = fmaf(de, hi, r);
    r = fmaf(d, lo, r);
    // 2^(-r/64) = 1 - y, y = z - z^2 / 2 + z^3 / 6, z = r ln2 / 64 < 0.0055;
    // the next term is below 2^-34
    const float y = r * fmaf(r, fmaf(r, kZ3, kZ2), kZ1);
    return (u64)short_weight(kf, y, pow64) << left(magic_int(kf));
}

// k (as kMagic + k) and y of two logits (max finite).  The difference's rounding
// error counts for half-precision logits as well: some 2^13 times smaller than
// the greatest they lose bits in it, up to 2^-20 of a weight.
struct Two {
    float2 kf, y;
};
__device__ __forceinline__ Two two_of(float2 l, const Scale& c) {
    const float2 mx = make_float2(c.max, c.max), neg = make_float2(-1.f, -1.f);
    const float2 hi = make_float2(c.hi * 64.f, c.hi * 64.f), lo = make_float2(c.lo * 64.f, c.lo * 64.f);
    const float2 mg = make_float2(kMagic, kMagic);
    const float2 d = __ffma2_rn(l, neg, mx);
    const float2 kf = __ffma2_rn(d, hi, mg);
    float2 r = __ffma2_rn(d, hi, __ffma2_rn(kf, neg, mg));
    const float2 b = __fadd2_rn(d, make_float2(-c.max, -c.max));
    const float2 db = __ffma2_rn(b, neg, d);                  // d - b
    const float2 e0 = __ffma2_rn(db, neg, mx);                // max - (d - b)
    const float2 e1 = __ffma2_rn(__fadd2_rn(l, b), neg, e0);  // ... + (-l - b)
    r = __ffma2_rn(e1, hi, r);
    r = __ffma2_rn(d, lo, r);
    const float2 q = __ffma2_rn(r, __ffma2_rn(r, make_float2(kZ3, kZ3), make_float2(kZ2, kZ2)), make_float2(kZ1, kZ1));
    return {kf, __fmul2_rn(r, q)};
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
    // f(vector, index of its first element) for the part's vectors, N in flight
    // per thread, and one(value, index) for the single elements; a thread's
    // indices ascend.
    template <int N, typename F, typename G>
    __device__ __forceinline__ void vectors(F f, G one) const {
        if (rank == 0 && (int)threadIdx.x < head) one(at(threadIdx.x), (int)threadIdx.x);
        const uint4* vec = reinterpret_cast<const uint4*>(row + head);
        uint4 next[N];  // the loads of the turn after this one are on their way meanwhile
        const auto load = [&](int v) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (v + i * kThreads < v1) next[i] = vec[v + i * kThreads];
        };
        load(v0 + threadIdx.x);
#pragma unroll 1
        for (int v = v0 + threadIdx.x; v < v1; v += N * kThreads) {
            uint4 w[N];
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = next[i];
            load(v + N * kThreads);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (v + i * kThreads >= v1) break;
                f(w[i], head + (v + i * kThreads) * VE);
            }
        }
        if (rank == ranks - 1 && tail + (int)threadIdx.x < vocab) one(at(tail + threadIdx.x), tail + (int)threadIdx.x);
    }
    // f(two values, index of the first).  Single elements come with a -inf, which
    // takes no part.
    template <int N, typename F>
    __device__ __forceinline__ void pairs(F f) const {
        vectors<N>(
            [&](uint4 w, int i) {
                if constexpr (HALF) {
                    f(__half22float2(*reinterpret_cast<const __half2*>(&w.x)), i);
                    f(__half22float2(*reinterpret_cast<const __half2*>(&w.y)), i + 2);
                    f(__half22float2(*reinterpret_cast<const __half2*>(&w.z)), i + 4);
                    f(__half22float2(*reinterpret_cast<const __half2*>(&w.w)), i + 6);
                } else {
                    f(make_float2(__uint_as_float(w.x), __uint_as_float(w.y)), i);
                    f(make_float2(__uint_as_float(w.z), __uint_as_float(w.w)), i + 2);
                }
            },
            [&](float x, int i) { f(make_float2(x, -INFINITY), i); });
    }
    // This thread's greatest logit (NaN left out), -inf without any.
    __device__ __forceinline__ float greatest() const {
        float best = -INFINITY;
        __half2 two = __floats2half2_rn(-INFINITY, -INFINITY);  // (a maximum of halves needs no conversion)
        vectors<4>(
            [&](uint4 w, int) {
                if constexpr (HALF) {
                    const __half2 x = __hmax2(*reinterpret_cast<const __half2*>(&w.x), *reinterpret_cast<const __half2*>(&w.y));
                    const __half2 y = __hmax2(*reinterpret_cast<const __half2*>(&w.z), *reinterpret_cast<const __half2*>(&w.w));
                    two = __hmax2(two, __hmax2(x, y));
                } else {
                    best = fmaxf(best, fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)),
                                             fmaxf(__uint_as_float(w.z), __uint_as_float(w.w))));
                }
            },
            [&](float x, int) { best = fmaxf(best, x); });
        if constexpr (HALF) best = fmaxf(best, fmaxf(__low2float(two), __high2float(two)));
        return best;
    }
    // f(value, index), one at a time (the added -inf among them).
    template <int N, typename F>
    __device__ __forceinline__ void each(F f) const {
        pairs<N>([&](float2 l, int i) {
            f(l.x, i);
            f(l.y, i + 1);
        });
    }
};

// Sums of N values over the CTA, to all threads.
template <int N>
__device__ __forceinline__ void block_sum(u64 (&x)[N], Shared& s) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) s.red[i][threadIdx.x >> 5] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        u64 t = threadIdx.x % 32 < kWarps ? s.red[i][threadIdx.x % 32] : 0;
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        x[i] = __shfl_sync(0xffffffffu, t, 0);
    }
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
    if (lane == 31) s.red[0][warp] = x;
    __syncthreads();
    for (int i = 0; i < warp; ++i) x += s.red[0][i];
    return x;
}

struct Four {
    u64 v[4];
};

// What the cluster's CTAs share: `mine` (the same in all threads of a CTA)
// goes to every CTA; the values of rank r are then xch[phase][r].  The buffers
// alternate: one is written again only after the next exchange, at which
// every CTA has read it.
struct Cluster {
    cg::cluster_group g;
    int rank, ranks, phase;
    __device__ const u64 (*exchange(Shared& s, Four mine))[4] {
        if ((int)threadIdx.x < 4 * ranks) {
            u64* dst = g.map_shared_rank(&s.xch[phase][rank][0], threadIdx.x / 4);
            const int i = threadIdx.x % 4;
            dst[i] = i == 0 ? mine.v[0] : i == 1 ? mine.v[1] : i == 2 ? mine.v[2] : mine.v[3];
        }
        sync();
        const u64(*r)[4] = s.xch[phase];
        phase ^= 1;
        return r;
    }
    __device__ void sync() {
        if (ranks > 1) g.sync();
        else __syncthreads();
    }
};

// Sorts all[0 .. n) descending and leaves the running weights in pre[].
template <bool HALF>
__device__ void sort_and_scan(Shared& s, u64* all, u64* pre, int n, const Scale& c) {
    if (n <= kCounting) {
        // every token's place is the number of greater ones (no two are
        // equal): two threads per token look at half of them each
        const int i = threadIdx.x >> 1, part = threadIdx.x & 1;
        const u64 x = i < n ? all[i] : 0;
        int place = 0;
        if (i < n)
            for (int j = part; j < n; j += 2) place += all[j] > x;
        place += __shfl_xor_sync(0xffffffffu, place, 1);
        __syncthreads();
        if (i < n && part == 0) all[place] = x;
        __syncthreads();
    } else {
        // bitonic, padded with zeros to a power of two
        int m = 2 * kCounting;
        while (m < n) m *= 2;
        for (int i = n + threadIdx.x; i < m; i += kThreads) all[i] = 0;
        __syncthreads();
        for (int size = 2; size <= m; size *= 2)
            for (int step = size / 2; step > 0; step /= 2) {
                for (int i = threadIdx.x; i < m / 2; i += kThreads) {
                    const int a = 2 * i - (i & (step - 1)), b = a + step;
                    const u64 x = all[a], y = all[b];
                    if ((x < y) == ((a & size) == 0)) {
                        all[a] = y;
                        all[b] = x;
                    }
                }
                __syncthreads();
            }
    }
    u64 before = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        const u64 w = i < n ? weight_of(key_value((uint32_t)(all[i] >> 32)), c, s.pow64) : 0;
        const u64 run = before + block_scan(w, s);
        if (i < n) pre[i] = run;
        __syncthreads();
        before = pre[min(n, i0 + kThreads) - 1];
    }
    __syncthreads();
}

// First place of pre[0 .. n) that reaches target (there is one; else the last), to all threads.
__device__ int reach(Shared& s, const u64* pre, int n, u64 target) {
    if (threadIdx.x == 0) s.result[3] = n - 1;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (pre[i] >= target && (i == 0 || pre[i - 1] < target)) s.result[3] = i;
    __syncthreads();
    const int i = (int)s.result[3];
    __syncthreads();
    return i;
}

// The joined list into rank 0's `all`, from every CTA's list.
__device__ void gather(Shared& s, Cluster& cl, const u64 (*counts)[4], u64* all) {
    int total = 0;
    for (int r = 0; r < cl.ranks; ++r) total += (int)counts[r][0];
    for (int i = threadIdx.x; i < total; i += kThreads) {  // (a thread per token: the remote loads overlap)
        int r = 0, j = i;
        while (j >= (int)counts[r][0]) j -= (int)counts[r++][0];
        all[i] = *cl.g.map_shared_rank(&s.list[j], r);
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
        atomicAdd(&s.h0[bin], n);
        const uint32_t l = (uint32_t)w;
        const uint32_t old = atomicAdd(&s.h1[bin], l);
        const uint32_t h = (uint32_t)(w >> 32) + (old + l < old ? 1u : 0u);
        if (h) atomicAdd(&s.h2[bin], h);
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

// A short weight into the tail's histogram, in parts of 15 bits (no result is
// waited for): the tokens of a bin are of one step, which shifts their sum, and
// the last bin's, from a step above 16 * 64 on, are not shifted.
__device__ __forceinline__ void add_tail(Shared& s, int bin, uint32_t w) {
    atomicAdd(&s.h0[bin], w & 0x7fffu);
    atomicAdd(&s.h1[bin], w >> 15);
}
static_assert(kBins > 16 * 64, "the last bin's shift");

// Every CTA's histogram of `bins` bins (descending logits), joined and summed
// up from the front, into every CTA's mc[] and mw[].
__device__ void join_histogram(Shared& s, Cluster& cl, int bins) {
    cl.sync();  // all histograms done
    const int b0 = bins * cl.rank / cl.ranks, b1 = bins * (cl.rank + 1) / cl.ranks;
    for (int b = b0 + threadIdx.x; b < b1; b += kThreads) {
        uint32_t n = 0;
        u64 w = 0;
        for (int r = 0; r < cl.ranks; ++r) {
            const u64 x = *cl.g.map_shared_rank(&s.h0[b], r), y = *cl.g.map_shared_rank(&s.h1[b], r),
                      z = *cl.g.map_shared_rank(&s.h2[b], r);
            n += (uint32_t)x;
            w += y + (z << 32);
        }
        for (int r = 0; r < cl.ranks; ++r) {
            *cl.g.map_shared_rank(&s.mc[b], r) = n;
            *cl.g.map_shared_rank(&s.mw[b], r) = w;
        }
    }
    cl.sync();
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

// The tail's histogram of all CTAs, by rank 0 for itself (every CTA's is done):
// running sums of the weights into mw[].
__device__ void join_tail(Shared& s, Cluster& cl, int cut) {
    constexpr int P = kBins / kThreads;
    u64 w[P] = {};
    for (int r = 0; r < cl.ranks; ++r) {
        const uint32_t* h0 = cl.g.map_shared_rank(&s.h0[P * threadIdx.x], r);
        const uint32_t* h1 = cl.g.map_shared_rank(&s.h1[P * threadIdx.x], r);
#pragma unroll
        for (int e = 0; e < P; ++e) w[e] += (u64)h0[e] + ((u64)h1[e] << 15);
    }
#pragma unroll
    for (int e = 0; e < P; ++e) w[e] <<= left(cut + P * threadIdx.x + e);
#pragma unroll
    for (int e = 1; e < P; ++e) w[e] += w[e - 1];
    const u64 before = block_scan(w[P - 1], s) - w[P - 1];
#pragma unroll
    for (int e = 0; e < P; ++e) s.mw[P * threadIdx.x + e] = before + w[e];
    __syncthreads();
}
// The weight of this CTA's tail, a part of it per thread.
__device__ __forceinline__ u64 tail_weight(const Shared& s, int cut) {
    u64 w = 0;
    for (int b = threadIdx.x; b < kBins; b += kThreads) w += ((u64)s.h0[b] + ((u64)s.h1[b] << 15)) << left(cut + b);
    return w;
}

// First bin whose running count or weight reaches target (there is one; else the last).
__device__ int reach_bin(Shared& s, int bins, bool by_count, u64 target) {
    if (threadIdx.x == 0) s.result[2] = bins - 1;
    __syncthreads();
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
    for (int b = threadIdx.x; b < bins; b += kThreads) s.h0[b] = s.h1[b] = s.h2[b] = 0;
    __syncthreads();
}

struct Hit {
    u64 weight;  // of everything up to the place, and of the token there
    u64 own;
    int token;
    bool by_digits;  // the search used the histogram's arrays
};

// The place where the count or weight of the tokens of steps s0 .. s1 - 1
// reaches target (what stands before them already taken off): its running
// weight among them and its token.
template <bool HALF>
__device__ Hit search_bin(const Part<HALF>& row, Shared& s, Cluster& cl, const Scale& c, int s0, int s1,
                          bool by_count, u64 target) {
    __syncthreads();
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
    // most tokens are ruled out by two comparisons, a step wider than the range
    // (without a limit where the scale is zero)
    const float step = 1.f / (c.hi * 64.f);
    const float most = s0 > 0 ? c.max - (float)(s0 - 1) * step : INFINITY;
    const float fewest = c.hi > 0.f ? c.max - (float)(s1 + 1) * step : -INFINITY;
    const auto one = [&](float x, int i) {
        if (x <= most && x >= fewest && x > -INFINITY) {
            const int st = steps_of(x, c);
            if (st >= s0 && st < s1) append(s, key_of(x), i);
        }
    };
    const __half2 hi = __half2half2(__float2half_ru(most)), lo = __half2half2(__float2half_rd(fewest));
    row.template vectors<2>(
        [&](uint4 w, int i) {
            uint32_t in;  // a bit per element of the vector
            if constexpr (HALF) {
                const auto between = [&](uint32_t x) {
                    const __half2 h = *reinterpret_cast<const __half2*>(&x);
                    return __hle2_mask(h, hi) & __hge2_mask(h, lo);
                };
                in = (between(w.x) & 0x00010001u) | (between(w.y) & 0x00020002u) | (between(w.z) & 0x00040004u) |
                     (between(w.w) & 0x00080008u);
            } else {
                const auto between = [&](uint32_t x) { return __uint_as_float(x) <= most && __uint_as_float(x) >= fewest; };
                in = (between(w.x) ? 1u : 0u) | (between(w.y) ? 2u : 0u) | (between(w.z) ? 4u : 0u) | (between(w.w) ? 8u : 0u);
            }
#pragma unroll 1
            while (in) {
                const int b = __ffs((int)in) - 1, word = b & 15;
                in &= in - 1;
                const uint32_t x = word == 0 ? w.x : word == 1 ? w.y : word == 2 ? w.z : w.w;
                if constexpr (HALF) one(__half2float(__ushort_as_half((uint16_t)(b < 16 ? x : x >> 16))), i + 2 * word + (b >> 4));
                else one(__uint_as_float(x), i + word);
            }
        },
        one);
    __syncthreads();
    const u64(*n)[4] = cl.exchange(s, {{s.count, 0, 0, 0}});
    u64 total = 0;
    bool fits = true;
    for (int r = 0; r < cl.ranks; ++r) {
        total += n[r][0];
        fits = fits && n[r][0] <= kList;
    }
    Hit h;
    h.by_digits = !(fits && total <= kBinList);
    if (total == 0) {  // (no target lies in an empty bin)
        h.weight = h.own = 0;
        h.token = -1;
        return h;
    }
    if (!h.by_digits) {
        u64 place = 0, pre = 0, own = 0;
        if (cl.rank == 0) {
            gather(s, cl, n, s.bin_all);
            sort_and_scan<HALF>(s, s.bin_all, s.bin_pre, (int)total, c);
            place = by_count ? min(target - 1, total - 1) : reach(s, s.bin_pre, (int)total, target);
            pre = s.bin_pre[place];
            own = pre - (place ? s.bin_pre[place - 1] : 0);
            place = (uint32_t)~(uint32_t)s.bin_all[place];
        }
        const u64(*x)[4] = cl.exchange(s, {{pre, place, own, 0}});
        h.weight = x[0][0];
        h.token = (int)x[0][1];
        h.own = x[0][2];
        return h;
    }
    // eight bits of the key at a time, the greatest first
    uint32_t prefix = 0;
    u64 wb = 0, nb = 0, equal = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        clear_histogram(s, 256);
        Tally t;
        row.template each<1>([&](float l, int) {
            const uint32_t k = key_of(l);
            const int st = steps_of(l, c);
            if (k == kLeast || st < s0 || st >= s1 || (shift < 24 && k >> (shift + 8) != prefix >> (shift + 8))) return;
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
    u64 same[1] = {0};
    row.template each<1>([&](float l, int) { same[0] += key_of(l) == prefix; });
    block_sum(same, s);
    const u64 mine = same[0];
    const u64(*x)[4] = cl.exchange(s, {{mine, 0, 0, 0}});
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
    const u64(*y)[4] = cl.exchange(s, {{found, 0, 0, 0}});
    h.token = -1;
    for (int r = 0; r < cl.ranks; ++r)
        if (y[r][0]) h.token = (int)y[r][0] - 1;
    return h;
}

// floor(x W) and whether anything is left over, for 0 <= x <= 1: a float is a
// 24-bit integer and a power of two, so the product is exact in 128 bits.
__device__ __forceinline__ u64 share_floor(float x, u64 W, bool& rest) {
    if (x >= 1.f) {
        rest = false;
        return W;
    }
    const uint32_t b = __float_as_uint(x);
    const int e = (int)(b >> 23);
    const u64 m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const int sh = 150 - (e ? e : 1);  // x = m 2^-sh; 24 .. 149
    const u64 lo = W * m, hi = __umul64hi(W, m);  // hi below 2^24
    if (sh < 64) {
        rest = (lo & ((1ull << sh) - 1)) != 0;
        return lo >> sh | hi << (64 - sh);
    }
    rest = lo != 0 || (sh < 128 ? (hi & ((1ull << (sh - 64)) - 1)) != 0 : hi != 0);
    return sh - 64 < 64 ? hi >> (sh - 64) : 0;
}
__device__ __forceinline__ u64 nucleus_target(float p, u64 W) {  // least integer at or above p W, at least 1
    bool rest;
    const u64 t = share_floor(fmaxf(p, 0.f), W, rest);
    return max(t + rest, 1ull);
}
__device__ __forceinline__ u64 token_target(float u, u64 W) {  // least integer above u W, at most W
    bool rest;
    return min(share_floor(u, W, rest) + 1, W);
}

template <bool HALF>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& s = *reinterpret_cast<Shared*>(smem);
    Cluster cl{cg::this_cluster(), 0, a.cluster, 0};
    cl.rank = (int)cl.g.block_rank();
    const int r = blockIdx.x / a.cluster, tid = threadIdx.x;
    const Part<HALF> row(a, r, cl.rank);
    const auto finish = [&](int token, u64 own, u64 of) {
        if (cl.rank == 0 && tid == 0) {
            a.tokens[r] = token;
            if (a.probs) a.probs[r] = of ? (float)((double)own / (double)of) : 0.f;
        }
    };

    // 1. the greatest logit
    const float best = row.greatest();
    const bool any = best > -INFINITY;
    // (while the loads are on their way: the tables)
    if (tid < 64) s.pow64[tid] = make_float2(__uint_as_float(kPow64[tid] + kMagicBits), (float)kPow64[tid]);
    for (int b = tid; b < kCut; b += kThreads) s.cut_count[b] = 0;
    for (int b = tid; b < kBins; b += kThreads) s.h0[b] = s.h1[b] = s.h2[b] = 0;
    if (tid == 0) {
        s.count = 0;
        s.cut = kCut - 1;
    }
    {
        const uint32_t m = __reduce_max_sync(0xffffffffu, any ? key_of(best) : 0u);
        if ((tid & 31) == 0) s.red[0][tid >> 5] = m;
    }
    cl.sync();  // every CTA of the cluster runs: its shared memory can be written
    uint32_t top = __reduce_max_sync(0xffffffffu, (tid & 31) < kWarps ? (uint32_t)s.red[0][tid & 31] : 0u);
    if (cl.ranks > 1) {
        const u64(*x)[4] = cl.exchange(s, {{top, 0, 0, 0}});
        for (int i = 0; i < cl.ranks; ++i) top = max(top, (uint32_t)x[i][0]);
    }
    const float T = a.temperature ? a.temperature[r] : 1.f;
    const int k = a.top_k ? a.top_k[r] : 0;
    if (top == 0) {
        finish(-1, 0, 0);
        cl.sync();  // no CTA leaves while another may still write to it
        return;
    }
    Scale c;
    c.max = key_value(top);
    if (!a.u || !(T > 0.f) || k == 1) {
        // its lowest index: the threads that have met it look once more
        if (tid == 0) s.cut = 0x7fffffff;
        __syncthreads();
        if (any && best == c.max)
            row.template each<1>([&](float l, int i) {
                if (l == best) atomicMin(&s.cut, i);
            });
        __syncthreads();
        const u64(*x)[4] = cl.exchange(s, {{(u64)s.cut, 0, 0, 0}});
        u64 at = x[0][0];
        for (int i = 1; i < cl.ranks; ++i) at = min(at, x[i][0]);
        finish((int)at, 1, 1);
        cl.sync();
        return;
    }
    {
        // log2(e) / T as a float pair: the quotient, and what it leaves over
        const float f = 1.44269502f / T;
        c.hi = fminf(f, 1e30f);
        const float left = fmaf(-f, T, 1.44269502f) + 1.92596299e-8f;
        c.lo = f > 1e-30f && f < 1e30f ? left / T : 0.f;
    }
    const bool with_k = k > 0 && k < a.vocab;
    const float p = a.top_p ? a.top_p[r] : 1.f;
    const float mp = a.min_p ? a.min_p[r] : 0.f;
    const u64 least_w = mp > 0.f ? __float2ull_ru(fminf(mp, 1.f) * 17592186044416.f) : 0;  // 2^44 min_p, exact
    const float u = fminf(fmaxf(a.u[r], 0.f), 1.f);

    // 2. the threshold
    if (any) atomicAdd(&s.cut_count[min(steps_of(best, c) >> 2, kCut - 1)], 1u);
    cl.sync();
    {
        static_assert(kCut == kThreads, "a bin per thread");
        uint32_t n = 0;
        if (cl.ranks > 1) {
            for (int i = 0; i < cl.ranks; ++i) n += *cl.g.map_shared_rank(&s.cut_count[tid], i);
        } else {
            n = s.cut_count[tid];
        }
        const u64 wanted = with_k && k <= kMostK ? k : kWanted;
        const u64 run = block_scan(n, s);
        if (run >= wanted && run - n < wanted) s.cut = tid;
        __syncthreads();
    }
    const int cut = 4 * (s.cut + 1);  // the list's steps: 0 .. cut - 1

    // 3. the list; without top_k the histogram and the weight of what is not in
    // it, and of that the weight that min_p keeps
    u64 sums[3] = {0, 0, 0};  // outside the list: valid tokens (top_k), weight, kept weight
    const bool top_inf = isinf(c.max);
    if (with_k || top_inf) {
        // (any beginning of the order will do: one comparison per token)
        const float least_l = c.max - (float)cut / (c.hi * 64.f);
        row.template pairs<2>([&](float2 l, int i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = e ? l.y : l.x;
                if (x >= least_l && x > -INFINITY) append(s, key_of(x), i + e);
                else sums[0] += x > -INFINITY;
            }
        });
    } else {
        // (whether min_p keeps any of the tail: by the greatest weight of its first step)
        const bool keeps = least_w && (u64)short_weight(kMagic + (float)cut, -0.0055f, s.pow64) << left(cut) >= least_w;
        row.template pairs<1>([&](float2 l, int i) {
            const Two x = two_of(l, c);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float kf = e ? x.kf.y : x.kf.x;
                if (!(kf <= kLast)) continue;  // no weight (-inf and NaN among them)
                if (kf < kMagic + (float)cut) {
                    append(s, key_of(e ? l.y : l.x), i + e);
                } else {
                    const uint32_t w = short_weight(kf, e ? x.y.y : x.y.x, s.pow64);
                    add_tail(s, min(magic_int(kf) - cut, kBins - 1), w);
                    if (keeps) {
                        const u64 all = (u64)w << left(magic_int(kf));
                        if (all >= least_w) sums[2] += all;
                    }
                }
            }
        });
        __syncthreads();
        sums[1] = tail_weight(s, cut);
    }
    block_sum(sums, s);
    u64 n_list = 0, rest = 0, W = 0, some = 0;  // W, some: the tail's as yet
    bool fits = true;
    const u64(*n)[4] = cl.exchange(s, {{s.count, sums[0], sums[1], sums[2]}});
    for (int i = 0; i < cl.ranks; ++i) {
        n_list += n[i][0];
        rest += n[i][1];
        W += n[i][2];
        some += n[i][3];
        fits = fits && n[i][0] <= kList;
    }
    fits = fits && n_list > 0 && n_list <= kAll && !top_inf;

    // Rank 0 decides: the list holds everything; the nucleus ends below it; the
    // token stands below it (then in which bin, by the histogram); the list
    // does not do.
    enum : u64 { kDone, kNucleus, kToken, kNoList };
    u64 state = kNoList, target = 0, W_list = 0;
    int bin = 0;
    const auto choose = [&]() {  // the token, W being known
        if (least_w) W = min(W, some);
        target = token_target(u, W);
        if (target > W_list) {
            state = kToken;
            return;
        }
        state = kDone;
        const int i = reach(s, s.pre, (int)n_list, target);
        finish((int)(uint32_t)~(uint32_t)s.all[i], s.pre[i] - (i ? s.pre[i - 1] : 0), W);
    };
    const auto find_bin = [&]() {  // takes what stands before it off the target
        target -= W_list;
        bin = reach_bin(s, kBins, false, target);
        if (bin) target -= s.mw[bin - 1];
    };
    if (fits && cl.rank == 0) {
        const int N = (int)n_list;
        gather(s, cl, n, s.all);
        sort_and_scan<HALF>(s, s.all, s.pre, N, c);
        W_list = s.pre[N - 1];
        if (!with_k || k <= N || rest == 0) {
            if (with_k) W = s.pre[min(k, N) - 1];  // top_k ends in the list
            else W += W_list;
            if (least_w) {
                int kept = 0;
                for (int i0 = 0; i0 < N; i0 += kThreads) {
                    const int i = i0 + tid;
                    kept += __syncthreads_count(i < N && s.pre[i] - (i ? s.pre[i - 1] : 0) >= least_w);
                }
                some = (with_k ? 0 : some) + s.pre[kept - 1];  // (the greatest is kept)
            }
            state = kDone;
            if (p < 1.f) {
                target = nucleus_target(p, W);
                if (target <= W_list) W = s.pre[reach(s, s.pre, N, target)];
                else state = kNucleus;
            }
            if (state == kDone) choose();
            if (state != kDone) {
                join_tail(s, cl, cut);
                find_bin();
            }
        }
    }
    const auto tell = [&]() {
        const u64(*x)[4] = cl.exchange(s, {{state, target, (u64)bin, W}});
        state = x[0][0];
        target = x[0][1];
        bin = (int)x[0][2];
        if (state != kNoList) W = x[0][3];
    };
    tell();
    if (state == kDone) return;  // (every CTA has read what it reads of the others)
    if (state == kNucleus || state == kToken) {
        // below the list, without top_k
        Hit h = search_bin<HALF>(row, s, cl, c, cut + bin, bin < kBins - 1 ? cut + bin + 1 : kSteps, false, target);
        if (state == kNucleus) {
            if (h.by_digits) {  // the search has used the histogram's arrays
                clear_histogram(s, kBins);
                row.template each<1>([&](float l, int) {
                    const int st = steps_of(l, c);
                    if (st >= cut && st < kSteps)
                        add_tail(s, min(st - cut, kBins - 1), (uint32_t)(weight_of(l, c, s.pow64) >> left(st)));
                });
                cl.sync();
            }
            if (cl.rank == 0) {
                if (h.by_digits) join_tail(s, cl, cut);
                W = W_list + (bin ? s.mw[bin - 1] : 0) + h.weight;
                choose();
                if (state == kToken) find_bin();
            }
            tell();
            if (state == kDone) return;
            h = search_bin<HALF>(row, s, cl, c, cut + bin, bin < kBins - 1 ? cut + bin + 1 : kSteps, false, target);
        }
        finish(h.token, h.own, W);
    } else if (state == kNoList) {
        // the list has overflowed (a flat top), or top_k is larger than one:
        // counts and weights of all, by bins
        const auto histogram = [&]() {
            clear_histogram(s, kBins);
            Tally t;
            row.template each<1>([&](float l, int) {
                if (!(l > -INFINITY)) return;
                const u64 w = weight_of(l, c, s.pow64);
                if (w == 0) return;
                t.add(s, steps_of(l, c) >> 1, w);
            });
            t.flush(s);
            join_histogram(s, cl, kBins);
        };
        histogram();
        if (least_w) {
            sums[0] = 0;
            row.template each<1>([&](float l, int) {
                if (!(l > -INFINITY)) return;
                const u64 w = weight_of(l, c, s.pow64);
                if (w >= least_w) sums[0] += w;
            });
            u64 one[1] = {sums[0]};
            block_sum(one, s);
            const u64(*x)[4] = cl.exchange(s, {{one[0], 0, 0, 0}});
            some = 0;
            for (int i = 0; i < cl.ranks; ++i) some += x[i][0];
        }
        W = s.mw[kBins - 1];
        const auto at = [&](bool by_count, u64 t) {
            const int b = reach_bin(s, kBins, by_count, t);
            const u64 nb = b ? s.mc[b - 1] : 0, wb = b ? s.mw[b - 1] : 0;
            Hit h = search_bin<HALF>(row, s, cl, c, 2 * b, 2 * b + 2, by_count, t - (by_count ? nb : wb));
            h.weight += wb;
            return h;
        };
        bool stale = false;
        if (with_k && (u64)k < s.mc[kBins - 1]) {
            const Hit h = at(true, (u64)k);
            W = h.weight;
            stale = h.by_digits;
        }
        if (p < 1.f) {
            if (stale) histogram();
            const Hit h = at(false, nucleus_target(p, W));
            W = h.weight;
            stale = h.by_digits;
        }
        if (least_w) W = min(W, some);
        if (stale) histogram();
        const Hit h = at(false, token_target(u, W));
        finish(h.token, h.own, W);
    }
    cl.sync();  // no CTA leaves while another may still use its shared memory
}

template <bool HALF>
cudaError_t launch(Args& a, int rows, int sms, cudaStream_t stream) {
    // As many CTAs per row as the GPU holds for all rows at once (a GB300
    // places 36 clusters of 8 CTAs, 74 of 4, 152 of 2), each with at least 2048
    // tokens and at most kMostPart.  us of rows of 151936 with top_k 50: 1 row 13.6
    // at 8 CTAs, 14.8 at 4; 36 rows 17.7 and 16.3.  With every setting in turn: 16
    // rows 34 at 8, 38 at 4, 44 at 16 (clusters that wait for others); 61 rows 54
    // at 4, 63 at 2.  One row of 8000: 9.0 at 2, 10.9 at 4.
    const auto held = [&](int x) { return x > 2 ? 2 * sms - 2 * x : 2 * sms; };
    int c = kMaxCluster;
    while (c > 1 && ((long long)rows * c > held(c) || a.vocab <= 2048 * c) && a.vocab <= kMostPart * (c / 2)) c /= 2;
    a.cluster = c;
    static std::atomic<int> marks[64];
    const void* kern = reinterpret_cast<const void*>(sample_kernel<HALF>);
    const cudaError_t e = q4i::ensure_smem_attr(kern, marks, (int)sizeof(Shared));
    if (e != cudaSuccess) return e;
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
    if (d.rows > (1 << 26)) return fail(Q4_ERR_UNSUPPORTED, "rows=%d above %d", d.rows, 1 << 26);
    if (d.rows > 0 && (!d.logits || !d.tokens)) return fail(Q4_ERR_INVALID_ARG, "NULL pointer argument");
    if (reinterpret_cast<uintptr_t>(d.logits) & (d.dtype == Q4_F16 ? 1u : 3u))
        return fail(Q4_ERR_MISALIGNED, "logits must be aligned to their elements");
    if (!aligned4(d.temperature, d.top_k, d.top_p, d.min_p, d.u, d.tokens, d.probs))
        return fail(Q4_ERR_MISALIGNED, "the rows' arrays must be 4-byte aligned");
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
