// Attention of several sequences' new rows over a paged key / value cache, in
// fp16 (q4_tree_attn.cu) or in 8 bits (q4_tree_attn8.cu):
// drafted trees by a bit mask, prompt chunks and batched decoding causally
// (q4.h 7c).
//
// Mathematics: for a kv head the G = Hq / Hkv query heads of a sequence's n
// rows are n G rows of one product, S = Q K^T over the same keys, so they are
// taken together: row r is token r / G, head r % G.  One pass over the keys
// keeps a running maximum m, sum l and output O of each row,
//   m' = max(m, s c),  p = 2^(s c - m'),  l' = l 2^(m-m') + sum p,
//   O' = O 2^(m-m') + p V,      c = scale log2 e,
// and parts over different keys join the same way.
//
// What bounds it: up to a few dozen rows per kv head the bytes of the cache
// (each read once: 4 D bytes per position and head, in 8 bits 2 D and half a
// byte of scales), beyond that the products.  The positions are the long axis,
// and there are often fewer (sequence, head) pairs than SMs, so the work is cut
// by positions: every (sequence, head, block of rows) is a job of tiles (of 64
// positions, on tcgen05 and on the line in 8 bits of 128), all jobs' tiles stand
// in one line, and the CTA c of C takes its C-th part of the line.  A job that lies in one CTA's part is finished there; of a job that
// several share, each leaves (m, l, O) in the workspace (at most two per CTA:
// one job begun by another, one left unfinished), and a second kernel joins
// them in the order of the CTAs, so the bits do not depend on timing.
#pragma once

#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "q4_paged8.cuh"
#include "q4_tc.cuh"

namespace q4x {

namespace cg = cooperative_groups;
using q4p::Seq;
using q4p::View;

constexpr int kKeys = 64;      // positions per tile
constexpr int kMaxRows = 64;   // rows of a job
constexpr int kMaxCtas = 512;
constexpr int kTcRows = 256, kMaxTcCtas = 160;
// P = 2^(s - m + kShift): fp16 keeps 11 bits of a probability down to 2^-26
// of the row's greatest (below, it is off by 2^-37 of that at most), and O / l
// is the same quotient.  The tcgen05 kernel lets the greatest score exceed m by
// kLag, so P reaches 2^15, over the fp16 cache alone: a P that decides its row is
// rounded then, but is 2^12 exactly where m is the greatest score.  8 bits with
// and without a lag, error against 64 bits and time: the trees 2.09e-4 and 104.7
// us / 2.02e-4 and 105.2 us, the chunks 2.16e-4 and 179 us / 2.05e-4 and 181 us
// (rounding the outputs alone: 2.00e-4).
constexpr float kShift = 12.f, kLag = 3.f;

struct Args {
    View w;           // 8 bits: its pools are those of the codes
    const float *ks, *vs;  // 8 bits: the scales
    int nb;                // ... of a page and head
    const uint32_t* mask;
    int mask_words;
    const uint16_t* q;
    uint16_t* out;
    long long ldq, ldo;
    int G;       // query heads per kv head
    q4p::PageDiv by_g;  // division by G
    float c;     // scale * log2(e)
    int ctas;    // CTAs that share the line
    int BM, KT;  // rows of a job, positions of a tile (1 << KT_log2)
    int KT_log2;
    int cost_full, cost_half;  // units of a tile for a row block with more than BM / 2 rows, and for others
    int lead;                  // units of a job before its first tile
    float* po;   // workspace: [2 CTAs][BM][D] outputs
    float2* pml; // [2 CTAs][BM] (m, l)
    int4* rec;   // [CTAs] tcgen05: the job that begins in the CTA and ends in a later one
};

template <int D>
__device__ __forceinline__ float* part_o(const Args& a, int slot) {
    return a.po + (size_t)slot * a.BM * D;
}
__device__ __forceinline__ float2* part_ml(const Args& a, int slot) { return a.pml + (size_t)slot * a.BM; }

// ---------------------------------------------------------------- schedule ---
// Tiles of a sequence's row block `rb`: with a mask every row may see every
// new row; causally the block's last token is the last key.
__device__ __forceinline__ int block_tiles(const Args& a, const Seq& q, int rb) {
    const int last = min((int)q4p::page_of(a.by_g, (rb + 1) * a.BM - 1), q.n - 1);
    const int keys = q.ctx + (a.mask ? q.n : last + 1);
    return (keys + a.KT - 1) >> a.KT_log2;
}

// A tile's units of the line: what it costs.
__device__ __forceinline__ int tile_cost(const Args& a, const Seq& q, int rb) {
    return q.n * a.G - rb * a.BM > a.BM / 2 ? a.cost_full : a.cost_half;
}

// Units of one head of a sequence (all row blocks).
__device__ __forceinline__ unsigned long long head_units(const Args& a, const Seq& q) {
    unsigned long long t = 0;
#pragma unroll 1
    for (int b = 0; b * a.BM < q.n * a.G; b += 4)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if ((b + e) * a.BM < q.n * a.G) t += (unsigned)(a.lead + block_tiles(a, q, b + e) * tile_cost(a, q, b + e));
    return t;
}

// A job's tiles tile .. tiles - 1; tile t stands at unit start + t * cost of the line.
struct Place {
    int s, h, rb, tile, tiles, cost;
    unsigned start;
    Seq q;
};

// The line's length; `sums` gets the threads' running shares: each thread adds
// up a contiguous share of the sequences.  The line has fewer than 2^31 units:
// a call beyond that (10^14 operations and more) is left out, with the error
// latched.
static __device__ __noinline__ unsigned line_scan(const Args& a, unsigned* sums, int threads) {
    __shared__ unsigned long long wsum[32];
    const int per = (int)((unsigned)(a.w.S + threads - 1) / (unsigned)threads);
    const int lo = min(a.w.S, (int)threadIdx.x * per), hi = min(a.w.S, lo + per);
    unsigned long long t = 0;
#pragma unroll 1
    for (int s = lo; s < hi; ++s) {
        bool bad;
        const Seq q = q4p::seq_of(a.w, s, bad);
        if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.w.err, q4d::kErrDeviceCheck);
        t += head_units(a, q) * a.w.H;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long u = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += u;
    }
    if (lane == 31) wsum[warp] = t;
    __syncthreads();
    unsigned long long all = 0;
#pragma unroll 1
    for (int i = 0; i < threads / 32; ++i) {
        if (i == warp) t += all;
        all += wsum[i];
    }
    sums[threadIdx.x] = (unsigned)t;
    __syncthreads();
    if (all < (1ull << 31)) return (unsigned)all;
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.w.err, q4d::kErrDeviceCheck);
    return 0;
}

// A CTA's share of the line (CTA c: units c * share ..): a tile belongs to the
// CTA in whose share its first unit lies.  At least two tiles: one, so that a
// CTA between two others of a job has a part of it, and another, as fewer
// parts join faster (one user's 2000 positions: 14.3 -> 11.6 us).
__device__ __forceinline__ unsigned line_share(const Args& a, unsigned line) {
    return max((line + (unsigned)a.ctas - 1) / (unsigned)a.ctas, 2u * (unsigned)max(a.cost_full, a.cost_half));
}

// The job that holds unit x (x < the line's length), from its first tile on.
static __device__ __noinline__ Place line_find(const Args& a, const unsigned* sums, int threads, unsigned x) {
    int lo = 0, hi = threads - 1;  // first thread whose running sum exceeds x
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (sums[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    const unsigned before = lo > 0 ? sums[lo - 1] : 0u;
    unsigned rest = x - before;
    Place p;
    unsigned head = 0;
    bool bad;
    if (a.w.S <= threads) {  // a thread's share was one sequence
        p.s = lo;
        p.q = q4p::seq_of(a.w, p.s, bad);
        head = (sums[lo] - before) / (unsigned)a.w.H;
    } else {
        p.s = lo * (int)((unsigned)(a.w.S + threads - 1) / (unsigned)threads);
#pragma unroll 1
        while (true) {
            p.q = q4p::seq_of(a.w, p.s, bad);
            head = (unsigned)head_units(a, p.q);
            if (rest < head * (unsigned)a.w.H) break;  // (below 2^31: the line is)
            rest -= head * (unsigned)a.w.H;
            ++p.s;
        }
    }
    p.h = (int)(rest / head);
    rest -= (unsigned)p.h * head;
#pragma unroll 1
    for (p.rb = 0;; ++p.rb) {
        p.tiles = block_tiles(a, p.q, p.rb);
        p.cost = tile_cost(a, p.q, p.rb);
        if (rest < (unsigned)(a.lead + p.tiles * p.cost)) break;
        rest -= (unsigned)(a.lead + p.tiles * p.cost);
    }
    p.start = x - rest + a.lead;
    p.tile = 0;
    return p;
}

// The next job (there is one).
__device__ __forceinline__ void next_job(const Args& a, Place& p) {
    p.start += (unsigned)(p.tiles * p.cost + a.lead);
    p.tile = 0;
    if (++p.rb * a.BM >= p.q.n * a.G) {
        p.rb = 0;
        if (++p.h == a.w.H) {
            p.h = 0;
            do {
                bool bad;
                p.q = q4p::seq_of(a.w, ++p.s, bad);
            } while (p.q.n <= 0);
        }
    }
    p.tiles = block_tiles(a, p.q, p.rb);
    p.cost = tile_cost(a, p.q, p.rb);
}

// First tile of the job at or behind unit x: 0 .. tiles.
__device__ __forceinline__ int tile_at(const Place& p, unsigned x) {
    const unsigned d = x - p.start + (unsigned)p.cost - 1;
    return x <= p.start ? 0 : min(p.tiles, (int)(d / (unsigned)p.cost));
}

// A CTA's part x0 .. x1 of the line as segments, each a run of one job's
// tiles p.tile .. end - 1.
struct Walk {
    Place p;
    int end;
    unsigned x1;
    // false: the CTA has no tiles
    __device__ __forceinline__ bool begin(const Args& a, const unsigned* sums, int threads, unsigned line) {
        const unsigned share = line_share(a, line), x0 = share * blockIdx.x;  // below 2^31 + ctas (1024 at most) * 20: two tiles' cost
        x1 = min(line, x0 + share);
        if (x0 >= x1) return false;
        p = line_find(a, sums, threads, x0);
        p.tile = tile_at(p, x0);
        if (p.tile == p.tiles) {  // x0 lies in the last tile's units
            if (!more(a)) return false;
            next_job(a, p);
        }
        end = tile_at(p, x1);
        return p.tile < end;  // (the part may lie in what leads a job)
    }
    // whether the next job's first tile lies in the part (the line's end has none behind it)
    __device__ __forceinline__ bool more(const Args& a) const { return p.start + (unsigned)(p.tiles * p.cost + a.lead) < x1; }
    __device__ __forceinline__ void next(const Args& a) {
        next_job(a, p);
        end = tile_at(p, x1);
    }
};

// ----------------------------------------------------------------- devices ---
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {  // 16-byte chunk c of row r in a [rows][D] fp16 tile
    return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
    const uint32_t n = live ? 16u : 0u;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ bool finite16(uint16_t h) { return (h & 0x7C00u) != 0x7C00u; }

// Whether new row j (0 <= j < n) is seen by row i of a sequence that starts at row `start`.
__device__ __forceinline__ bool sees(const Args& a, int start, int i, int j) {
    if (!a.mask) return j <= i;
    const int word = j >> 5;
    return word < a.mask_words && (a.mask[(size_t)(start + i) * a.mask_words + word] >> (j & 31) & 1u);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}

// Place of the scale of (position, head) in the scales, -1 where the page number is outside the pool.
__device__ __forceinline__ long long scale_of(const Args& a, int s, int pos, int h) {
    const uint32_t pg = q4p::page_of(a.w.div, (uint32_t)pos);
    const int id = a.w.table[(size_t)s * a.w.max_pages + pg];
    if ((uint32_t)id >= (uint32_t)a.w.n_pages) return -1;
    return ((long long)id * a.w.H + h) * a.nb + ((uint32_t)pos - pg * a.w.div.d) / q4p::kBlock;
}

// Adds to columns c0 .. c1 - 1 of a written row (fp16 `out`, else fp32 `part`)
// the infinities and NaN of the new rows it sees in the segment's T tiles.
template <int D, bool k8>
__device__ __noinline__ void add_odd(const Args& a, const Place& p, int T, int tok, int c0, int c1, uint16_t* out,
                                     float* part) {
    const int n0 = max(0, p.tile * a.KT - p.q.ctx), n1 = min(p.q.n, (p.tile + T) * a.KT - p.q.ctx);
    for (int nj = n0; nj < n1; ++nj) {
        if (!sees(a, p.q.start, tok, nj)) continue;
        const long long at = q4p::row_at(a.w, p.s, p.q.ctx + nj, p.h, D);
        if (at < 0) continue;
        for (int c = c0; c < c1; ++c) {
            float f;
            if constexpr (k8) {
                if ((reinterpret_cast<const uint8_t*>(a.w.v)[at + c] & 0x7f) != 0x7f) continue;  // (NaN alone is not finite)
                f = NAN;
            } else {
                const uint16_t v = a.w.v[at + c];
                if (finite16(v)) continue;
                f = __half2float(__ushort_as_half(v));
            }
            if (out) out[c] = __half_as_ushort(__float2half_rn(__half2float(__ushort_as_half(out[c])) + f));
            else part[c] += f;
        }
    }
}

// ------------------------------------------------- mma.sync: few rows per job ---
// WM warps along the job's 16 WM rows, WN = 4 / WM along the tile's
// positions, and a fifth warp that brings the tiles: by TMA where a page is a
// multiple of 8 rows (boxes of `box` rows, the greatest power of two up to 64
// that divides the page; a page that does not exist is read outside the map,
// where TMA fills in zeros), else by 16-byte cp.async from row to row.  The
// consumers never meet while they walk a job: a stage is handed over by its
// "full" and "empty" barriers alone.
// Fragment layouts of mma.m16n8k16 (g = lane / 4, u = lane % 4): A covers rows
// g, g + 8 and columns 2u, 2u+1, 2u+8, 2u+9; B rows 2u, 2u+1, 2u+8, 2u+9 of
// column g; an accumulator rows g, g + 8, columns 2u, 2u+1, so two
// neighbouring score tiles are the A operand of a 16-position step of P V.
//
// Measured: 40 users' tokens over contexts up to 12000 (8 query heads on each
// of 4 kv heads of 128, 549 MB of cache) 95 us = 5.8 TB/s, 85 % of the measured
// copy rate; a short line is bound by its chain of waits: a job's sizes, its
// first pages, the first tiles, the parts' way through L2 and the joining
// kernel, 9.5 us with one tile of work.
//
// kClustered: few jobs (a few users' decoding), where latency counts.  The
// CTAs of a cluster take a job's tiles together and join their parts through
// distributed shared memory: one launch, and no line to walk.  One user's
// token over 1000 positions (16 heads on 8): 8.1 us, sizes, pages and one tile
// per CTA behind one another (the line: 10.6).
constexpr int kConsumers = 128, kThreads = 160;
// Units of a tile, and of a job before its tiles: the way to a new job's first
// tile costs a CTA about four tiles' time.  us with lead 0 / 8 / 16: 24 users'
// tokens up to 2000 positions 37 / 30 / 29, 100 users' up to 500 56 / 38 / 36,
// 40 up to 12000 94 / 94 / 94.
constexpr int kRingCost = 4, kRingLead = 16;
// 8 bits, whose tiles are twice as long: lead 4 / 8 / 12 / 16 / 24: 48 users' tokens
// up to 14000 positions 181 / 175 / 176 / 176 / 180, up to 4000 64 / 62 / 63 / 64 / 67.
constexpr int kRing8Lead = 8;

// Positions of a tile.  8 bits, the line: 128, as a tile's fixed cost (waits,
// statistics) weighs twice as much against half the bytes (48 users' tokens up
// to 14000 positions: 188 us, with 64 200).
template <bool kClustered, bool k8>
constexpr int ring_keys() {
    return k8 && !kClustered ? 128 : kKeys;
}

template <int D, bool k8, int KEYS>
struct Ring {
    static constexpr int kStages = !k8 ? 3 : KEYS == 64 ? 4 : 2;
    static constexpr uint32_t kTile = KEYS * D * (k8 ? 1 : 2);       // keys or values of a tile
    static constexpr uint32_t kScales = k8 ? 2 * KEYS * 4 : 0;       // scales of its positions, keys' and values'
    static constexpr uint32_t kQuery = k8 ? 16 * D * 2 : 0;          // a 16-row job's query
    static constexpr size_t kSmem = 1024 + (size_t)kStages * (2 * kTile + kScales) + kQuery + 256;
};

constexpr int kMaxStages = 4;
struct RingBars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    volatile int abort;
    volatile int odd[2];  // last segment (by parity) that met infinities or NaN among its new rows' values
};

// Byte offset of row r, 16-byte chunk c in a tile of 128-byte-wide swizzled
// slabs of 64 rows; 64-byte rows (8 bits, D = 64) swizzle by pairs of rows.
template <int D, bool k8>
__device__ __forceinline__ uint32_t ring_off(int r, int c) {
    if constexpr (k8 && D == 64) return (uint32_t)(r * 64 + ((c ^ (r >> 1 & 3)) << 4));
    return (uint32_t)((c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Clears the NaN among four e4m3 codes.
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
    const uint32_t nan = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;  // 1 in the bytes that are 0x7f or 0xff
    return w & ~(nan * 0xffu);
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool live) {
    const uint32_t n = live ? 4u : 0u;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ bool ring_wait(RingBars& B, uint64_t& bar, uint32_t parity, int* err) {
    if (B.abort) return false;
    if (q4d::mbar_wait(q4d::smem_addr(&bar), parity, err)) return true;
    B.abort = 1;
    return false;
}

struct MapArgs {
    Args a;
    int box;       // rows per TMA box
    int zero_row;  // a row outside the maps
    int cluster, cluster_log2;  // CTAs per job: 4, 8 or 16 (0: the line)
};

// Sequence and row block of the call's block-th row block, false if there are
// fewer: a warp looks through 32 sequences at a time.
__device__ __forceinline__ bool find_block(const Args& a, int block, Place& p) {
    const int lane = threadIdx.x & 31;
    if (a.w.S == 1) {  // (one user's token: 0.3 us)
        bool bad;
        p.s = 0;
        p.rb = block;
        p.q = q4p::seq_of(a.w, 0, bad);
        return block * a.BM < p.q.n * a.G;
    }
#pragma unroll 1
    for (int s0 = 0; s0 < a.w.S; s0 += 32) {
        Seq q = {0, 0, 0};
        if (s0 + lane < a.w.S) {
            bool bad;
            q = q4p::seq_of(a.w, s0 + lane, bad);
        }
        const int own = q.n > 0 ? (q.n * a.G + a.BM - 1) / a.BM : 0;
        int sum = own;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, x);
            if (lane >= x) sum += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, block < sum);
        if (past) {
            const int from = __ffs((int)past) - 1;
            p.s = s0 + from;
            p.rb = block - __shfl_sync(0xffffffffu, sum - own, from);
            p.q.start = __shfl_sync(0xffffffffu, q.start, from);
            p.q.n = __shfl_sync(0xffffffffu, q.n, from);
            p.q.ctx = __shfl_sync(0xffffffffu, q.ctx, from);
            return true;
        }
        block -= __shfl_sync(0xffffffffu, sum, 31);
    }
    return false;
}

// Latches sequences whose sizes do not fit.  find_block stops at its own
// sequence, so the blocks share all of them: a warp of each looks at every
// gridDim.x-th 32.
__device__ __forceinline__ void latch_bad(const Args& a) {
#pragma unroll 1
    for (int s = 32 * blockIdx.x + (threadIdx.x & 31); s < a.w.S; s += 32 * gridDim.x) {
        bool bad;
        q4p::seq_of(a.w, s, bad);
        if (bad) atomicOr(a.w.err, q4d::kErrDeviceCheck);
    }
}

//
// k8: the tiles hold e4m3 codes, a 16-byte chunk 16 elements, and the scales of
// their positions come beside them by 4-byte cp.async.  Codes become fp16 in
// registers: a thread's word of a key chunk holds elements 4u .. 4u+3, which
// take the places 2u, 2u+1, 2u+8, 2u+9 of the contraction (the query lies in
// shared memory in the same order), and the scores take the keys' scales in
// fp32.  A transposed word of a value chunk holds elements 2g, 2g+1 of two
// positions; apart they are the B operands of an even and an odd column tile,
// which take the values' scales (powers of two: exact) before the product.
// Half the bytes for the same products and more instructions: what bounds it
// is issue and waits as much as the bytes, so three CTAs share an SM.  48
// users' tokens over contexts up to 14000 (32 query heads on 8 of 128, 911 MB)
// 171 us = 5.3 TB/s, 78 % of the measured copy rate, with pages of 64 164 us
// (of 16: more and smaller copies); two CTAs with three stages 232 us (before
// the last 17).  The pages looked up a tile ahead brought nothing.  Heads of 64
// leave room for four: 119 us against 139 with three (457 MB = 3.8 TB/s: a tile
// is half the bytes for as many waits, look-ups, scores and exponentials).
// At 128 registers (heads of 64: 96) it spills, 276 bytes stored and 268 loaded
// (116 / 164; by cp.async 264 / 256 and 152 / 252), in the tile loop too: the
// five warps of a CTA load 47 and store 28 registers a tile in that batch (34
// and 22).
template <int D, bool k8>
constexpr int kRingCtas = !k8 ? 2 : D == 64 ? 4 : 3;
template <int D, int WM, bool kTma, bool kClustered, bool k8>
__global__ void __launch_bounds__(kThreads, kRingCtas<D, k8>)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ MapArgs t) {
    constexpr int BM = 16 * WM, WN = 4 / WM;
    constexpr int NCH = k8 ? D / 16 : D / 8, KS = D / 16, DN = D / 8, SLABS = k8 ? 1 : D / 64;  // chunks of a row ...
    constexpr int KEYS = ring_keys<kClustered, k8>();
    constexpr int KW = KEYS / WN, NT = KW / 8;  // a warp's positions of a tile, 8-wide tiles of them
    constexpr uint32_t TB = Ring<D, k8, KEYS>::kTile;
    constexpr int kStages = Ring<D, k8, KEYS>::kStages;
    constexpr auto off = ring_off<D, k8>;
    const Args& a = t.a;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ unsigned sums[kThreads];
    __shared__ float2 ml_s[4 * 16], fin_s[kClustered ? BM : 1];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* scales_s = reinterpret_cast<float*>(smem + kStages * 2 * TB);  // [stage][keys, values][position]
    uint8_t* query_s = reinterpret_cast<uint8_t*>(scales_s + kStages * Ring<D, k8, KEYS>::kScales / 4);
    RingBars& B = *reinterpret_cast<RingBars*>(query_s + Ring<D, k8, KEYS>::kQuery);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            // by cp.async every lane of the producing warp arrives
            q4d::mbar_init(q4d::smem_addr(&B.full[i]), (kTma ? 1 : 0) + (!kTma || k8 ? 32 : 0));
            q4d::mbar_init(q4d::smem_addr(&B.empty[i]), 4);
        }
        B.abort = 0;
        B.odd[0] = B.odd[1] = 0;
        q4d::fence_mbar_init();
    }
    Walk w;
    bool any;
    int rank = 0;
    if constexpr (kClustered) {
        const int job = (int)(blockIdx.x >> t.cluster_log2);
        rank = (int)blockIdx.x & (t.cluster - 1);
        Place& p = w.p;
        p.h = job % a.w.H;
        if (!find_block(a, job / a.w.H, p)) {  // (the whole cluster)
            if (warp == 4) latch_bad(a);
            return;
        }
        p.tiles = block_tiles(a, p.q, p.rb);
        p.tile = (int)((unsigned)(p.tiles * rank) >> t.cluster_log2);  // tiles * 16 stays below 2^31
        w.end = (int)((unsigned)(p.tiles * (rank + 1)) >> t.cluster_log2);
        p.cost = 1;
        p.start = 0;
        w.x1 = 0;  // no more segments
        any = p.tile < w.end;
        __syncthreads();
    } else {
        any = w.begin(a, sums, kThreads, line_scan(a, sums, kThreads));
        q4d::pdl_trigger();  // the joining kernel's blocks may start; they wait for this grid's end
        if (!any) return;
    }
    Place& p = w.p;

    if (warp == 4) {
        // ------------------------------------------------- tiles
        bool ok = true, rest = any;
        uint32_t kt = 0;
        while (rest && ok) {
            const int len = p.q.ctx + p.q.n;
            for (; p.tile < w.end && ok; ++p.tile, ++kt) {
                const int st = kt % kStages;
                const uint32_t fb = q4d::smem_addr(&B.full[st]);
                uint8_t* kv = smem + st * 2 * TB;
                // the scales of positions lane, lane + 32, ..
                long long scale_at[KEYS / 32];
                if constexpr (k8) {
#pragma unroll
                    for (int e = 0; e < KEYS / 32; ++e) {
                        const int key = p.tile * KEYS + e * 32 + lane;
                        scale_at[e] = key < len ? scale_of(a, p.s, key, p.h) : -1;
                    }
                }
                const auto bring_scales = [&]() {
                    const uint32_t to = q4d::smem_addr(scales_s) + (uint32_t)(st * Ring<D, k8, KEYS>::kScales + lane * 4);
#pragma unroll
                    for (int e = 0; e < KEYS / 32; ++e) {
                        const long long x = scale_at[e] < 0 ? 0 : scale_at[e];
                        cp4(to + e * 128, a.ks + x, scale_at[e] >= 0);
                        cp4(to + KEYS * 4 + e * 128, a.vs + x, scale_at[e] >= 0);
                    }
                };
                if constexpr (kTma) {
                    // the first NB lanes: boxes of keys, the next: of values
                    constexpr int NB = KEYS / 8;
                    const int b = lane % NB, key = p.tile * KEYS + b * t.box;
                    const bool mine = lane < 2 * NB && b * t.box < KEYS;
                    int y = t.zero_row;
                    if (mine && key < len) {
                        const long long at = q4p::row_at(a.w, p.s, key, p.h, 1);
                        if (at >= 0) y = (int)at;
                        else atomicOr(a.w.err, q4d::kErrDeviceCheck);
                    }
                    if (kt >= kStages) ok = ring_wait(B, B.empty[st], (kt / kStages - 1) & 1, a.w.err);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) q4d::mbar_arrive_expect_tx(fb, 2 * TB);
                    __syncwarp();
                    if (mine) {
                        const uint32_t dst = q4d::smem_addr(kv + (lane / NB) * TB) + (uint32_t)(b * t.box) * (k8 ? D : 128);
#pragma unroll
                        for (int sl = 0; sl < SLABS; ++sl)
                            q4t::tma_load_2d(dst + sl * (KEYS * 128), lane < NB ? &tmK : &tmV, 64 * sl, y, fb);
                    }
                    if constexpr (k8) {
                        bring_scales();
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(fb) : "memory");
                    }
                } else {
                    if (kt >= kStages) ok = ring_wait(B, B.empty[st], (kt / kStages - 1) & 1, a.w.err);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    // a lane looks two rows up; the lanes of a row share it
                    const uint32_t kb = q4d::smem_addr(kv);
                    constexpr int PER = 32 / NCH;
                    const int c = lane % NCH;
#pragma unroll 1
                    for (int half = 0; half < KEYS / 32; ++half) {
                        const int key = p.tile * KEYS + half * 32 + lane;
                        long long at = -1;
                        if (key < len) {
                            at = q4p::row_at(a.w, p.s, key, p.h, D);
                            if (at < 0) atomicOr(a.w.err, q4d::kErrDeviceCheck);
                        }
#pragma unroll 4
                        for (int e = 0; e < 32; e += PER) {
                            const int r = e + lane / NCH;
                            const long long row = __shfl_sync(0xffffffffu, at, r);
                            const long long x = (row < 0 ? 0 : row) + (k8 ? 16 : 8) * c;
                            const uint32_t to = kb + off(half * 32 + r, c);
                            if constexpr (k8) {
                                cp16(to, reinterpret_cast<const uint8_t*>(a.w.k) + x, row >= 0);
                                cp16(to + TB, reinterpret_cast<const uint8_t*>(a.w.v) + x, row >= 0);
                            } else {
                                cp16(to, a.w.k + x, row >= 0);
                                cp16(to + TB, a.w.v + x, row >= 0);
                            }
                        }
                    }
                    if constexpr (k8) bring_scales();
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(fb) : "memory");
                }
            }
            rest = w.more(a);
            if (rest && ok) w.next(a);
        }
        if constexpr (!kTma || k8) asm volatile("cp.async.wait_all;" ::: "memory");
        if (kTma && !ok)  // copies still in flight land before the CTA can exit
            for (uint32_t i = kt > kStages ? kt - kStages : 0; i < kt; ++i)
                q4d::mbar_wait(q4d::smem_addr(&B.full[i % kStages]), (i / kStages) & 1, nullptr);
        if constexpr (!kClustered) return;
        latch_bad(a);  // (while the others take the last tiles)
    }

    // ----------------------------------------------------- scores and values
    // A failed wait (latched) does not leave the loops: the results are void,
    // but every warp still comes to the barriers the others wait at.
    const int g = lane >> 2, u = lane & 3;
    const int wm = warp / WN, wn = warp % WN;
    static_assert(!k8 || WM == 1, "jobs of 16 rows");
    constexpr bool kTwoChains = k8 && NT == 2;
    // 8 bits: an infinity in a query counts as NaN.  All its scores can be -inf,
    // which would look as if the row saw nothing; finite queries have none, as
    // their sums stay below 2^40.  So a seen score of -inf makes the row NaN (48
    // users' tokens 171 us, with the infinities taken out of the query 175); with
    // heads of 64, where that costs registers that the tile loop lacks, the query
    // goes in with NaN for infinities (95 against 99 us).
    constexpr bool kInfSeen = k8 && D == 128;
    uint32_t qf[k8 ? 1 : KS][4];  // (8 bits: in shared memory, so that three CTAs' registers fit an SM)
    int tok[2] = {0, 0};             // tokens of this thread's rows
    float o[DN][4], m[2], l[2];
    bool fresh = true;              // the job's first tile in this CTA
    bool begun = p.tile == 0;       // ... and in the line
    const int row0 = wm * 16 + g;   // this thread's rows of the job: row0, row0 + 8
    const auto col = [&](int dn) { return k8 ? 16 * (dn >> 1) + 4 * u + 2 * (dn & 1) : 8 * dn + 2 * u; };  // of o[dn]'s pairs
    uint32_t seg = 0, kt = 0;
    int seg_tile = p.tile;          // the segment's first tile
    const bool consume = warp < 4 && any;
    while (consume) {
        const int st = kt % kStages;
        const int R = min(BM, p.q.n * a.G - p.rb * BM);
        if (!k8 || fresh) {
#pragma unroll
            for (int e = 0; e < 2; ++e) tok[e] = (int)q4p::page_of(a.by_g, p.rb * BM + min(row0 + 8 * e, R - 1));
        }
        if (fresh) {
            if constexpr (k8) {
                // Four rows a warp.  A chunk of 16 elements is laid down in the order
                // in which the codes' words take them, elements 4u, 4u+1 before all
                // 4u+2, 4u+3, so that ldmatrix finds the fragments.
                const int r = 4 * warp + (lane >> 3);
                const bool live = r < R;
                const int rr = p.rb * BM + min(r, R - 1), tk = (int)q4p::page_of(a.by_g, rr);
                const uint16_t* src = a.q + (size_t)(p.q.start + tk) * a.ldq + (size_t)(p.h * a.G + rr - tk * a.G) * D;
#pragma unroll
                for (int kk = lane & 7; kk < KS; kk += 8) {
                    const uint4 z = make_uint4(0, 0, 0, 0);
                    uint4 x = live ? *reinterpret_cast<const uint4*>(src + 16 * kk) : z;
                    uint4 y = live ? *reinterpret_cast<const uint4*>(src + 16 * kk + 8) : z;
                    if constexpr (!kInfSeen) x = q4p::without_infinities(x), y = q4p::without_infinities(y);
                    *reinterpret_cast<uint4*>(query_s + swz<D>(r, 2 * kk)) = make_uint4(x.x, x.z, y.x, y.z);
                    *reinterpret_cast<uint4*>(query_s + swz<D>(r, 2 * kk + 1)) = make_uint4(x.y, x.w, y.y, y.w);
                }
                q4d::named_bar(1, kConsumers);  // (they have met at the last segment's end, behind its last use)
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool live = !k8 && row0 + 8 * e < R;
                const int rr = p.rb * BM + min(row0 + 8 * e, R - 1);
                const uint16_t* src = a.q + (size_t)(p.q.start + tok[e]) * a.ldq + (size_t)(p.h * a.G + rr - tok[e] * a.G) * D + 2 * u;
#pragma unroll
                for (int kk = 0; kk < (k8 ? 0 : KS); ++kk) {
                    qf[kk][e] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * kk) : 0u;
                    qf[kk][2 + e] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * kk + 8) : 0u;
                }
                m[e] = -INFINITY;
                l[e] = 0.f;
            }
#pragma unroll
            for (int dn = 0; dn < DN; ++dn) o[dn][0] = o[dn][1] = o[dn][2] = o[dn][3] = 0.f;
            fresh = false;
            seg_tile = p.tile;
        }
        const uint32_t kb = q4d::smem_addr(smem + st * 2 * TB), vb = kb + TB;
        ring_wait(B, B.full[st], (kt / kStages) & 1, a.w.err);
        __syncwarp();
        const int key0 = p.tile * KEYS;
        const bool tail = key0 + KEYS > p.q.ctx;  // the tile holds new rows, or the end
        if (tail) {
            // A new row's value reaches only the rows that see it, and what
            // lies behind the sequence nobody: those rows are cleared, or
            // their infinities and NaN, which are added back at the end where
            // they are seen.  (Warps of the same positions write the same.)
            bool found = false;
            for (int y = lane; y < KW * NCH; y += 32) {
                const int r = wn * KW + y / NCH, c = y % NCH, nj = key0 + r - p.q.ctx;
                if (nj < 0) continue;
                uint4* at = reinterpret_cast<uint4*>(smem + st * 2 * TB + TB + off(r, c));
                if (nj >= p.q.n) {
                    *at = make_uint4(0, 0, 0, 0);
                    continue;
                }
                const uint4 v = *at;
                uint32_t ws[4] = {v.x, v.y, v.z, v.w};
                bool bad = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (k8) {
                        const uint32_t x = without_nan(ws[e]);
                        bad |= x != ws[e];
                        ws[e] = x;
                    } else {
                        if (!finite16((uint16_t)ws[e])) ws[e] &= 0xffff0000u, bad = true;
                        if (!finite16((uint16_t)(ws[e] >> 16))) ws[e] &= 0x0000ffffu, bad = true;
                    }
                }
                if (bad) *at = make_uint4(ws[0], ws[1], ws[2], ws[3]);
                found |= bad;
            }
            if (found) B.odd[seg & 1] = (int)seg + 1;
            __syncwarp();
        }
        // scores
        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        if constexpr (k8) {
            float sd[kTwoChains ? NT : 1][4] = {};  // (two chains of products where there are few tiles)
            const uint32_t qs = q4d::smem_addr(query_s);
#pragma unroll
            for (int kk = 0; kk < KS; kk += 2) {
                uint32_t qa[2][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) ldsm4(qs + swz<D>(lane & 15, 2 * (kk + e) + (lane >> 4)), qa[e]);
#pragma unroll
                for (int nt = 0; nt < NT; nt += 2) {
                    uint32_t b[4];  // two chunks of two position tiles
                    ldsm4(kb + off(wn * KW + (nt + (lane >> 4)) * 8 + (lane & 7), kk + (lane >> 3 & 1)), b);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mma(kTwoChains && (e & 1) ? sd[kTwoChains ? nt + (e >> 1) : 0] : sc[nt + (e >> 1)], qa[e & 1],
                            q4p::e4m3_half2(b[e]), q4p::e4m3_half2_hi(b[e]));
                }
            }
            if constexpr (kTwoChains)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[nt][e] += sd[nt][e];
            const float* ks = scales_s + st * (Ring<D, k8, KEYS>::kScales / 4) + wn * KW + 2 * u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 f = *reinterpret_cast<const float2*>(ks + nt * 8);
                sc[nt][0] *= f.x;
                sc[nt][1] *= f.y;
                sc[nt][2] *= f.x;
                sc[nt][3] *= f.y;
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < KS; kk += 2) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t b[4];
                    ldsm4(kb + off(wn * KW + nt * 8 + (lane & 7), 2 * kk + (lane >> 3)), b);
                    mma(sc[nt], qf[kk], b[0], b[1]);
                    mma(sc[nt], qf[kk + 1], b[2], b[3]);
                }
            }
        }
        if (tail) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int nj = key0 + wn * KW + nt * 8 + 2 * u + (e & 1) - p.q.ctx;
                    if (nj >= 0 && (nj >= p.q.n || !sees(a, p.q.start, tok[e >> 1], nj))) sc[nt][e] = -INFINITY;
                    else if (kInfSeen && sc[nt][e] == -INFINITY) sc[nt][e] = NAN;
                }
        }
        uint32_t pa[NT / 2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mx = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(sc[nt][2 * e], sc[nt][2 * e + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            if (kInfSeen && !tail && mx == -INFINITY) l[e] = NAN;
            const float mn = fmaxf(m[e], mx * a.c);  // (c is positive: checked on the host)
            const float ms = mn == -INFINITY ? 0.f : mn;
            const float f = ex2(m[e] - ms);
            m[e] = mn;
            float sum = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float p0 = ex2(fmaf(sc[nt][2 * e], a.c, kShift - ms));
                const float p1 = ex2(fmaf(sc[nt][2 * e + 1], a.c, kShift - ms));
                sum += p0 + p1;
                pa[nt >> 1][(nt & 1) * 2 + e] = pack2(p0, p1);
            }
            l[e] = fmaf(l[e], f, sum);
            if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
                for (int dn = 0; dn < DN; ++dn) {
                    o[dn][2 * e] *= f;
                    o[dn][2 * e + 1] *= f;
                }
            }
        }
#pragma unroll
        for (int kj = 0; kj < KW / 16; ++kj) {
            if constexpr (k8) {
                const float* vs = scales_s + st * (Ring<D, k8, KEYS>::kScales / 4) + KEYS + wn * KW + kj * 16 + 2 * u;
                const float2 f0 = *reinterpret_cast<const float2*>(vs), f1 = *reinterpret_cast<const float2*>(vs + 8);
                const uint32_t s0 = pack2(f0.x, f0.y), s1 = pack2(f1.x, f1.y);
#pragma unroll
                for (int ch = 0; ch < NCH; ch += 2) {
                    uint32_t b[4];
                    ldsm4_t(vb + off(wn * KW + kj * 16 + (lane & 15), ch + (lane >> 4)), b);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t x = __byte_perm(b[2 * e], 0u, 0x3120), y = __byte_perm(b[2 * e + 1], 0u, 0x3120);
                        const int dn = 2 * (ch + e);
                        mma(o[dn], pa[kj], q4p::mul2(q4p::e4m3_half2(x), s0), q4p::mul2(q4p::e4m3_half2(y), s1));
                        mma(o[dn + 1], pa[kj], q4p::mul2(q4p::e4m3_half2_hi(x), s0), q4p::mul2(q4p::e4m3_half2_hi(y), s1));
                    }
                }
            } else {
#pragma unroll
                for (int dn = 0; dn < DN; dn += 2) {
                    uint32_t b[4];
                    ldsm4_t(vb + off(wn * KW + kj * 16 + (lane & 15), dn + (lane >> 4)), b);
                    mma(o[dn], pa[kj], b[0], b[1]);
                    mma(o[dn + 1], pa[kj], b[2], b[3]);
                }
            }
        }

        const bool job_end = p.tile + 1 == p.tiles, seg_end = p.tile + 1 == w.end;
        if (seg_end) {
            if constexpr (k8) {
                // columns 16 c + 4u, + 2 (even tile) and + 1, + 3 (odd) as two neighbouring pairs
#pragma unroll
                for (int dn = 0; dn < DN; dn += 2)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float x = o[dn][e + 1];
                        o[dn][e + 1] = o[dn + 1][e];
                        o[dn + 1][e] = x;
                    }
            }
            // the row sums over the quad's columns, then over the WN warps
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            }
            // The warps' outputs meet in this tile's stage, [WN][BM][D] fp32
            // (at most 32 KB), which is still ours; a cluster's CTA has
            // consumed all it loads, and takes stage 0, so that the others
            // know the place.  (8 bits: a stage is half as large, so they meet
            // in pairs.)
            float* ob = reinterpret_cast<float*>(smem + (kClustered ? 0 : st * 2 * TB));
            static_assert((size_t)(k8 ? (WN + 1) / 2 : WN) * BM * D * 4 <= 2 * TB, "joining space");
            // Nobody reads the tiles any more, and every warp's note of
            // infinities or NaN among the values (B.odd) is there: a warp
            // that finds a row cleared by another one has none of its own.
            // As no warp is more than a segment ahead, two notes suffice.
            q4d::named_bar(1, kConsumers);
            if constexpr (WN > 1) {
                if (u == 0) {
                    ml_s[warp * 16 + g] = make_float2(m[0], l[0]);
                    ml_s[warp * 16 + g + 8] = make_float2(m[1], l[1]);
                }
                q4d::named_bar(1, kConsumers);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = g + 8 * e;
                    float mm = -INFINITY, ls = 0.f;
#pragma unroll
                    for (int i = 0; i < WN; ++i) mm = fmaxf(mm, ml_s[(wm * WN + i) * 16 + r].x);
                    const float ms = mm == -INFINITY ? 0.f : mm;
#pragma unroll
                    for (int i = 0; i < WN; ++i) ls = fmaf(ml_s[(wm * WN + i) * 16 + r].y, ex2(ml_s[(wm * WN + i) * 16 + r].x - ms), ls);
                    const float f = ex2(m[e] - ms);
                    float* dst = ob + ((size_t)wn * BM + wm * 16 + r) * D;
                    if constexpr (k8) {
#pragma unroll
                        for (int dn = 0; dn < DN; ++dn) {
                            o[dn][2 * e] *= f;
                            o[dn][2 * e + 1] *= f;
                        }
                    } else {
#pragma unroll
                        for (int dn = 0; dn < DN; ++dn)
                            *reinterpret_cast<float2*>(dst + col(dn)) = make_float2(o[dn][2 * e] * f, o[dn][2 * e + 1] * f);
                    }
                    m[e] = mm;
                    l[e] = ls;
                }
                if constexpr (k8) {
                    // warps WN / 2 .. give theirs to the others, and so on
#pragma unroll
                    for (int half = WN / 2; half >= 1; half /= 2) {
                        float* at = ob + ((size_t)(wn % half) * BM + wm * 16 + g) * D;
                        if (wn >= half && wn < 2 * half) {
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int dn = 0; dn < DN; ++dn)
                                    *reinterpret_cast<float2*>(at + 8 * e * D + col(dn)) = make_float2(o[dn][2 * e], o[dn][2 * e + 1]);
                        }
                        q4d::named_bar(1, kConsumers);
                        if (wn < half) {
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int dn = 0; dn < DN; ++dn) {
                                    const float2 x = *reinterpret_cast<const float2*>(at + 8 * e * D + col(dn));
                                    o[dn][2 * e] += x.x;
                                    o[dn][2 * e + 1] += x.y;
                                }
                        }
                        if (half > 1) q4d::named_bar(1, kConsumers);
                    }
                } else {
                    q4d::named_bar(1, kConsumers);
                }
                if (!k8 && wn == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int dn = 0; dn < DN; ++dn) {
                            float2 v = make_float2(0.f, 0.f);
#pragma unroll
                            for (int i = 0; i < WN; ++i) {
                                const float2 x = *reinterpret_cast<const float2*>(
                                    ob + ((size_t)i * BM + wm * 16 + g + 8 * e) * D + col(dn));
                                v.x += x.x;
                                v.y += x.y;
                            }
                            o[dn][2 * e] = v.x;
                            o[dn][2 * e + 1] = v.y;
                        }
                }
            }
            if (kClustered && wn == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = row0 + 8 * e;
                    if (u == 0) fin_s[r] = make_float2(m[e], l[e]);
#pragma unroll
                    for (int dn = 0; dn < DN; ++dn)  // (over this thread's own elements of the warps' outputs)
                        *reinterpret_cast<float2*>(ob + (size_t)r * D + col(dn)) = make_float2(o[dn][2 * e], o[dn][2 * e + 1]);
                }
            }
            if (!kClustered && wn == 0) {
                const bool whole = begun && job_end;
                const int slot = 2 * blockIdx.x + (begun ? 1 : 0);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = row0 + 8 * e, rr = p.rb * BM + r;
                    if (r >= R) continue;
                    const float inv = !whole ? 1.f : l[e] == 0.f ? 0.f : 1.f / l[e];
                    uint16_t* out = a.out + (size_t)(p.q.start + tok[e]) * a.ldo + (size_t)(p.h * a.G + rr - tok[e] * a.G) * D;
                    float* part = part_o<D>(a, slot) + (size_t)r * D;
                    if (!whole && u == 0) part_ml(a, slot)[r] = make_float2(m[e], l[e]);
#pragma unroll
                    for (int dn = 0; dn < DN; ++dn) {
                        const float x = o[dn][2 * e] * inv, y = o[dn][2 * e + 1] * inv;
                        if (whole) *reinterpret_cast<uint32_t*>(out + col(dn)) = pack2(x, y);
                        else *reinterpret_cast<float2*>(part + col(dn)) = make_float2(x, y);
                    }
                }
                if (B.odd[seg & 1] == (int)seg + 1) {
                    __syncwarp();  // the rows are written
                    Place from = p;
                    from.tile = seg_tile;
                    for (int e = 0; e < 2; ++e) {
                        const int r = row0 + 8 * e, rr = p.rb * BM + r;
                        if (r >= R || u != 0) continue;
                        add_odd<D, k8>(a, from, p.tile + 1 - seg_tile, tok[e], 0, D,
                                   whole ? a.out + (size_t)(p.q.start + tok[e]) * a.ldo + (size_t)(p.h * a.G + rr - tok[e] * a.G) * D : nullptr,
                                   part_o<D>(a, slot) + (size_t)r * D);
                    }
                }
            }
            fresh = true;
            begun = true;
            ++seg;
        }
        // the stage goes back (what this thread did to it stands before the next copy)
        if (kTma && (tail || seg_end)) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.empty[st]));
        ++kt;
        if (++p.tile == w.end) {
            if (!w.more(a)) break;
            w.next(a);
        }
    }
    if constexpr (kClustered) {
        // ------------------------------------------------- the cluster's parts
        const int R = min(BM, p.q.n * a.G - p.rb * BM);
        float* ob = reinterpret_cast<float*>(smem);
        if (!any) {
            for (int y = tid; y < R * D; y += kThreads) ob[y] = 0.f;
            for (int r = tid; r < R; r += kThreads) fin_s[r] = make_float2(-INFINITY, 0.f);
        }
        __syncwarp();
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        // a warp per row, the rows spread over the CTAs
        for (int r = rank * 4 + warp; warp < 4 && r < R; r += 4 * t.cluster) {
            float2 ml = make_float2(-INFINITY, 0.f);
            bool odd = false;
            if (lane < t.cluster) {
                ml = *cl.map_shared_rank(&fin_s[r], lane);
                odd = *cl.map_shared_rank(const_cast<int*>(&B.odd[0]), lane) != 0;
            }
            float mm = ml.x;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
            const float f = ex2(ml.x - (mm == -INFINITY ? 0.f : mm));
            float ls = lane < t.cluster ? ml.y * f : 0.f;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
            constexpr int E = D / 32;
            float acc[E] = {};
            const auto add = [&](auto size) {  // (all parts' loads in flight together)
                constexpr int N = decltype(size)::value;
                float v[N][E];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float* src = cl.map_shared_rank(ob + (size_t)r * D + E * lane, i);
                    if constexpr (E == 4) {
                        const float4 x = *reinterpret_cast<const float4*>(src);
                        v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
                    } else {
                        const float2 x = *reinterpret_cast<const float2*>(src);
                        v[i][0] = x.x, v[i][1] = x.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float fi = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(v[i][e], fi, acc[e]);
                }
            };
            if (t.cluster == 16) add(std::integral_constant<int, 16>{});
            else if (t.cluster == 8) add(std::integral_constant<int, 8>{});
            else add(std::integral_constant<int, 4>{});
            const float inv = ls == 0.f ? 0.f : 1.f / ls;
            const int rr = p.rb * BM + r, tok = (int)q4p::page_of(a.by_g, rr);
            uint16_t* out = a.out + (size_t)(p.q.start + tok) * a.ldo + (size_t)(p.h * a.G + rr - tok * a.G) * D;
            uint32_t y[E / 2];
#pragma unroll
            for (int e = 0; e < E; e += 2) y[e / 2] = pack2(acc[e] * inv, acc[e + 1] * inv);
            if constexpr (E == 4) *reinterpret_cast<uint2*>(out + E * lane) = make_uint2(y[0], y[1]);
            else *reinterpret_cast<uint32_t*>(out + E * lane) = y[0];
            if (__any_sync(0xffffffffu, odd)) {
                __syncwarp();  // the row is written
                Place from = p;
                from.tile = 0;
                if (lane == 0) add_odd<D, k8>(a, from, p.tiles, tok, 0, D, out, nullptr);
            }
        }
        cl.sync();  // no CTA leaves while another reads its part
    }
}

// A job that several CTAs share: first row of its sequence, head, row block,
// rows, and the CTAs it is in, b ..  parts 0: no such job.
struct Shared {
    int start, h, rb, rows, b, parts;
};
__device__ __forceinline__ Shared shared_job(const Args& a, const Place& p, unsigned share, int b) {
    const int last = (int)((p.start + (unsigned)((p.tiles - 1) * p.cost)) / share);  // CTA of the last tile
    return {p.q.start, p.h, p.rb, (int)min((long long)a.BM, (long long)p.q.n * a.G - (long long)p.rb * a.BM), b, last - b + 1};
}

// Joins the parts of kRows rows of a job.  kRows rows and kParts parts are
// taken at a time, their loads in flight together; a lane holds (m, l) of
// every 32nd part.
template <int D, int kRows, int kParts>
__device__ __forceinline__ void join_rows(const Args& a, const Shared& job, int r0) {
    static_assert(32 % kParts == 0, "");
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, rows = job.rows, b = job.b, last = b + job.parts - 1;
    // CTA b has the job's beginning (slot 2 b + 1), later CTAs their slot 2 c
    const auto slot_of = [&](int c) { return 2 * c + (c == b); };
    float m[kRows], l[kRows], f[kRows], o[kRows][E];
    float2 ml[kRows];
    const auto load_ml = [&](int c, int i) {  // of this lane's part
        return c + lane <= last && r0 + i < rows ? part_ml(a, slot_of(c + lane))[r0 + i] : make_float2(-INFINITY, 0.f);
    };
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        ml[i] = load_ml(b, i);
        m[i] = ml[i].x;
        l[i] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] = 0.f;
    }
    for (int c = b; c <= last; c += kParts) {
        float v[kParts][kRows][E];
#pragma unroll
        for (int j = 0; j < kParts; ++j) {
            const float* src = part_o<D>(a, slot_of(c + j)) + (size_t)r0 * D + E * lane;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                if (c + j > last || r0 + i >= rows) {
#pragma unroll
                    for (int e = 0; e < E; ++e) v[j][i][e] = 0.f;
                } else if constexpr (E == 4) {
                    const float4 t = *reinterpret_cast<const float4*>(src + i * D);
                    v[j][i][0] = t.x, v[j][i][1] = t.y, v[j][i][2] = t.z, v[j][i][3] = t.w;
                } else {
                    const float2 t = *reinterpret_cast<const float2*>(src + i * D);
                    v[j][i][0] = t.x, v[j][i][1] = t.y;
                }
            }
        }
        if (c == b) {  // (with the first parts' rows on their way)
            for (int y = b + 32; y <= last; y += 32)
#pragma unroll
                for (int i = 0; i < kRows; ++i) m[i] = fmaxf(m[i], load_ml(y, i).x);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], s));
                if (m[i] == -INFINITY) m[i] = 0.f;
            }
        }
        if (((c - b) & 31) == 0) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                if (c > b) ml[i] = load_ml(c, i);  // (read again)
                f[i] = ex2(ml[i].x - m[i]);
                l[i] = fmaf(ml[i].y, f[i], l[i]);
            }
        }
#pragma unroll
        for (int j = 0; j < kParts; ++j)
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const float fi = __shfl_sync(0xffffffffu, f[i], (c - b + j) & 31);  // 0 behind the last part
#pragma unroll
                for (int e = 0; e < E; ++e) o[i][e] = fmaf(v[j][i][e], fi, o[i][e]);
            }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (r0 + i >= rows) break;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], s);
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const int rr = job.rb * a.BM + r0 + i, tok = (int)q4p::page_of(a.by_g, rr);
        uint16_t* dst = a.out + (size_t)(job.start + tok) * a.ldo + (size_t)(job.h * a.G + rr - tok * a.G) * D + E * lane;
        uint32_t w[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2) w[e / 2] = pack2(o[i][e] * inv, o[i][e + 1] * inv);
        if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(dst) = w[0];
    }
}

// Two rows at a time where there are few parts, else one.
constexpr int kFewParts = 8;  // (trees: 85 us, with 4 87, with 2 88)
__device__ __forceinline__ int join_items(const Shared& job) {
    return job.parts == 0 ? 0 : job.parts <= kFewParts ? (job.rows + 1) / 2 : job.rows;
}
template <int D>
__device__ __forceinline__ void join_item(const Args& a, const Shared& job, int i) {
    if (job.parts <= kFewParts) join_rows<D, 2, 2>(a, job, 2 * i);
    else join_rows<D, 1, 8>(a, job, i);
}

constexpr int kJoinThreads = 256;

// Behind the ring's kernel, where a job has few rows: block b looks at the
// border behind CTA b, for a job that has begun there, while the attention's
// last CTAs run.
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 4) tree_join_kernel(const __grid_constant__ Args a) {
    __shared__ unsigned sums[kJoinThreads];
    const unsigned line = line_scan(a, sums, kJoinThreads);
    const unsigned share = line_share(a, line), xb = share * blockIdx.x, x = xb + share;
    Shared job = {};
    if (x < line) {
        const Place p = line_find(a, sums, kJoinThreads, x);
        // begun in CTA b, not ended there
        if (p.start >= xb && p.start < x && p.start + (unsigned)((p.tiles - 1) * p.cost) >= x)
            job = shared_job(a, p, share, blockIdx.x);
    }
    // the parts are written (and no grid that follows this one starts before
    // the attention's end, so blocks without work wait as well)
    q4d::pdl_wait();
    const int items = join_items(job);
    for (int i = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5); i < items; i += gridDim.y * (kJoinThreads / 32))
        join_item<D>(a, job, i);
}

// Behind the tcgen05 kernel, where a job has up to 256 rows: CTAs leave records
// of the jobs they begin, every block counts all records' items, and the warps
// of the grid share them.  One user's 61 x 4 rows over 4000 positions: 28 us,
// with the kernel above 36.  Behind the ring's kernel it is the other way: 24
// users' tokens 22.0 us, with this one 23.6, as the records can be read only
// when the attention has ended.  With heads of 128 it spills (80 bytes stored,
// 132 loaded, at 64 registers for four blocks per SM).
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 4) tree_join_many_kernel(const __grid_constant__ Args a) {
    constexpr int kWarps = kJoinThreads / 32;
    static_assert(kMaxTcCtas <= kJoinThreads, "a record per thread");
    __shared__ int before[kJoinThreads];  // items of the records before
    __shared__ int wsum[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    q4d::pdl_wait();
    const auto read = [&](int b) {
        const int4 r = a.rec[b];
        return Shared{r.x, r.y, r.z, r.w & 0xffff, b, r.w >> 16};
    };
    const int items = tid < a.ctas ? join_items(read(tid)) : 0;
    int run = items;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, run, x);
        if (lane >= x) run += y;
    }
    if (lane == 31) wsum[warp] = run;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) run += wsum[i];
        all += wsum[i];
    }
    before[tid] = run - items;
    __syncthreads();
    for (int i = blockIdx.x * kWarps + warp; i < all; i += gridDim.x * kWarps) {
        int b = 0;  // the last record with before[b] <= i
#pragma unroll
        for (int x = kJoinThreads / 2; x > 0; x >>= 1)
            if (before[b + x] <= i) b += x;
        join_item<D>(a, read(b), i - before[b]);
    }
}
__device__ __forceinline__ void write_record(const Args& a, const Place& p, unsigned share) {
    const Shared j = shared_job(a, p, share, blockIdx.x);
    a.rec[blockIdx.x] = make_int4(j.start, j.h, j.rb, j.rows | j.parts << 16);
}

// The parts' places in the workspace.
template <int D>
size_t parts_bytes(int ctas, int BM) {
    return (size_t)2 * ctas * BM * (D + 2) * 4 + (size_t)ctas * sizeof(int4);
}
template <int D>
void place_parts(Args& a, void* workspace) {
    a.po = static_cast<float*>(workspace);
    a.pml = reinterpret_cast<float2*>(a.po + (size_t)2 * a.ctas * a.BM * D);
    a.rec = reinterpret_cast<int4*>(a.pml + (size_t)2 * a.ctas * a.BM);
}
template <int D>
size_t workspace_bytes() {
    const size_t x = parts_bytes<D>(kMaxCtas, kMaxRows), y = parts_bytes<D>(kMaxTcCtas, kTcRows);
    return x > y ? x : y;
}

// The joining kernel starts while the attention's last CTAs run (programmatic
// dependent launch).
inline cudaError_t launch_join(void (*kern)(Args), dim3 grid, const Args& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// What a launch has to know of either cache.
struct Pools {
    const void *k, *v;
    int n_pages, page_size, n_kv_heads, head_dim, n_seqs, max_pages;
};
template <class C>
inline Pools pools_of(const C& c) {
    return {c.k, c.v, c.n_pages, c.page_size, c.n_kv_heads, c.head_dim, c.n_seqs, c.max_pages};
}

// The pools as 2-D maps [rows][D], boxes of 128 bytes x box (8 bits: whole rows x box).
template <bool k8>
inline q4_status pool_maps(CUtensorMap* k, CUtensorMap* v, const Pools& c, uint32_t box) {
    const uint64_t rows = (uint64_t)c.n_pages * c.n_kv_heads * c.page_size, D = (uint64_t)c.head_dim;
    if constexpr (k8) {
        const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
        const q4_status st = q4i::make_map(k, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.k, D, rows, D, (uint32_t)D, box, sw);
        if (st != Q4_OK) return st;
        return q4i::make_map(v, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.v, D, rows, D, (uint32_t)D, box, sw);
    }
    const q4_status st = q4i::make_map(k, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, c.k, D, rows, D * 2, 64, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != Q4_OK) return st;
    return q4i::make_map(v, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, c.v, D, rows, D * 2, 64, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, int WM, bool kTma, bool kClustered, bool k8>
cudaError_t launch_kernel(const CUtensorMap& k, const CUtensorMap& v, const MapArgs& t, int grid, cudaStream_t s) {
    static std::atomic<int> marks[64];
    const auto kern = tree_attn_kernel<D, WM, kTma, kClustered, k8>;
    using R = Ring<D, k8, ring_keys<kClustered, k8>()>;
    const void* fn = reinterpret_cast<const void*>(kern);
    cudaError_t e = q4i::ensure_smem_attr(fn, marks, (int)R::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = R::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    if (kClustered) {
        if (t.cluster > 8) {
            static std::atomic<int> wide[64];
            if ((e = q4i::ensure_wide_clusters(fn, wide)) != cudaSuccess) return e;
        }
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)t.cluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, kern, k, v, t);
}

// CTAs of a job's cluster, where the GPU holds all clusters at once (a GB300
// places 14 of 16 CTAs, 36 of 8 and 74 of 4, two per SM); 0: the line.  us of a
// token's step, 8 kv heads of 128, clusters / line, contexts up to
//              100        1000       4000      16000    64000
//   1 user     7.9 / 9.4  8.0 / 11   10 / 15   21 / 25  54 / 52  (16 CTAs; of 8: 7.0, 7.4, 11, 28, 88)
//   2 users    7.3 / 9.4  8.8 / 11   13 / 16   32 / 32  94 / 69  (8)
//   4 users    8.4 / 9.5  9.5 / 12   17 / 19   34 / 31  114 / 104
//   8 users    8.5 / 9.6  11 / 13    22 / 24   64 / 64  209 / 182  (4)
// The host sees the contexts' bound alone, the table's width.  A cluster looks
// for its job through all sequences, the line's threads share them: 4 users
// over 1000 positions among 512 places 14.5 / 16.8 us, among 1024 20 / 18.
inline int cluster_size(long long jobs, int seqs, long long positions, int sms) {
    if (seqs > 512) return 0;
    if (jobs * 16 <= 3 * sms / 2) return 16;
    if (positions > 8192) return 0;
    return jobs * 8 <= 2 * sms - 16 ? 8 : jobs * 4 <= 2 * sms - 8 ? 4 : 0;
}

// box 0: no TMA.  (64 rows a job only without it: with it as many go to tcgen05.)
template <int D, int WM, bool k8 = false>
q4_status launch(Args& a, const Pools& c, void* workspace, int sms, int box, cudaStream_t s, const char* what) {
    MapArgs t;
    CUtensorMap k = {}, v = {};
    a.BM = 16 * WM;
    a.cost_full = a.cost_half = kRingCost;
    a.lead = k8 ? kRing8Lead : kRingLead;
    // (8 bits: jobs of 16 rows, whose parts are smaller)
    static_assert(2 * 16 < kMaxRows, "the parts of twice as many CTAs fit the workspace");
    const int resident = kRingCtas<D, k8> * sms, most = k8 ? 2 * kMaxCtas : kMaxCtas;
    a.ctas = resident < most ? resident : most;
    place_parts<D>(a, workspace);
    if (box) {
        const q4_status st = pool_maps<k8>(&k, &v, c, (uint32_t)box);
        if (st != Q4_OK) return st;
    }
    t.box = box;
    t.zero_row = (int)((long long)c.n_pages * c.n_kv_heads * c.page_size);
    // (n rows in S sequences that have some make at most S + (n - S) / BM blocks)
    const long long seqs = c.n_seqs < a.w.rows ? c.n_seqs : a.w.rows;
    const long long jobs = (seqs + ((long long)a.w.rows * a.G - seqs) / a.BM) * c.n_kv_heads;
    t.cluster = cluster_size(jobs, c.n_seqs, (long long)c.max_pages * c.page_size, sms);
    t.cluster_log2 = t.cluster == 16 ? 4 : t.cluster == 8 ? 3 : 2;
    a.KT = t.cluster ? ring_keys<true, k8>() : ring_keys<false, k8>();
    a.KT_log2 = a.KT == 128 ? 7 : 6;
    t.a = a;
    const auto run = [&](auto tma) {
        constexpr bool T = decltype(tma)::value;
        return t.cluster ? launch_kernel<D, WM, T, true, k8>(k, v, t, (int)jobs * t.cluster, s)
                         : launch_kernel<D, WM, T, false, k8>(k, v, t, a.ctas, s);
    };
    cudaError_t e;
    if constexpr (WM == 4) e = run(std::false_type{});
    else e = box ? run(std::true_type{}) : run(std::false_type{});
    if (!t.cluster && e == cudaSuccess) e = launch_join(tree_join_kernel<D>, dim3((unsigned)a.ctas - 1, (unsigned)WM), a, s);
    return e == cudaSuccess ? Q4_OK : q4i::cuda_fail(e, what);
}

// The arguments that both caches' calls share (7c's checks).
inline q4_status attention_args(Args& a, const uint32_t* mask, int mask_words, const uint16_t* q, uint16_t* out, int ldq, int ldo,
                                int n_q_heads, int n_kv_heads, int D, int rows, float scale, const void* workspace,
                                size_t workspace_bytes_given) {
    using namespace q4i;
    if (n_q_heads < n_kv_heads || n_q_heads % n_kv_heads)
        return fail(Q4_ERR_INVALID_ARG, "n_q_heads=%d is not a multiple of n_kv_heads=%d", n_q_heads, n_kv_heads);
    if ((long long)n_q_heads * D > (1 << 24)) return fail(Q4_ERR_UNSUPPORTED, "%d query heads", n_q_heads);
    const int G = n_q_heads / n_kv_heads;
    if ((long long)rows * G > (1ll << 30)) return fail(Q4_ERR_UNSUPPORTED, "rows=%d x %d query heads per kv head", rows, G);
    if (mask && mask_words < 1) return fail(Q4_ERR_INVALID_ARG, "mask_words=%d", mask_words);
    a.c = (scale == 0.f ? 1.f / sqrtf((float)D) : scale) * 1.4426950408889634f;
    if (!(a.c >= 1e-30f && a.c <= 1e30f)) return fail(Q4_ERR_INVALID_ARG, "scale=%g", scale);
    if (!aligned4(mask)) return fail(Q4_ERR_MISALIGNED, "mask must be 4-byte aligned");
    q4_status st;
    if ((st = row_matrix("q", q, n_q_heads * D, &ldq)) != Q4_OK) return st;
    if ((st = row_matrix("out", out, n_q_heads * D, &ldo)) != Q4_OK) return st;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return fail(Q4_ERR_MISALIGNED, "the workspace must be 256-byte aligned");
    const size_t need = D == 128 ? workspace_bytes<128>() : workspace_bytes<64>();
    if (workspace_bytes_given < need) return fail(Q4_ERR_INVALID_ARG, "workspace %zu bytes, need %zu", workspace_bytes_given, need);
    a.mask = mask;
    a.mask_words = mask_words;
    a.q = q;
    a.out = out;
    a.ldq = ldq;
    a.ldo = ldo;
    a.G = G;
    a.by_g = q4p::page_div((uint32_t)G);
    return Q4_OK;
}

// ------------------------------------------------- tcgen05: many rows per job ---
// From a few dozen rows per kv head on the products bound the work, and they
// belong to the 5th-generation tensor cores.  A CTA takes a job of up to 256
// rows and 128-position tiles as two streams of 128 rows (the MMA's M):
//   more than 128 rows: stream i has rows 128 i .. and every tile, so a tile
//     of keys and values is read once for 256 rows;
//   else: both streams have the same rows and alternate tiles, and their
//     (m, l, O) are joined at the end.
// Per stream a warpgroup computes the softmax (thread = row = TMEM lane) while
// the tensor cores work for the other stream, and one warp issues, in order,
//   S(0) | PVa(0) PVb(0) S(1) | PVa(1) PVb(1) S(2) | ...
// S = Q K^T (128 x 128, Q and K from shared memory) and O += P V (P, fp16,
// from tensor memory over the scores it came from, V read MN-major; a, b: the
// positions 0 .. 63 and 64 .. 127, each as soon as its P is there).  MMAs of
// one thread run in order, so S(k + 1) may overwrite what P V(k) reads, and
// the commit behind S(k + 1) tells the softmax that O holds step k's product.
// Tensor memory (512 columns): S 0 and 1 (128 each), O 0 and 1.
// The reference maximum of a row moves only when its maximum exceeds it by
// more than kLag (a factor 2^3; 8 bits: at all); then O and l are rescaled.
// Key and value tiles come by TMA as boxes of `box` rows (the greatest power
// of two, 8 .. 128, that divides the page): a box lies in one page.  A page
// that does not exist is read outside the map, where TMA fills in zeros.
//
// Measured: a chunk of 1024 and one of 532 rows over 6000 and 4100 positions
// (32 query heads on 8 kv heads of 128) 134 us = 1.10 PFLOP/s, 58 % of the
// measured matrix rate, the tensor pipe active half of the time: the softmax
// of a stream is not always done when the other's products are; 14 us are the
// joining of the parts.  Trees of up to 61 rows over 8 contexts up to 20000:
// 86 us = 4.4 TB/s of cache (375 MB).  A job's beginning and end (queries in,
// tensor memory out: some 5 us) are what short contexts cost.
constexpr int kTcKeys = 128;
// warps 0..3, 4..7: softmax of stream 0, 1; 8: keys, 9: values, 10, 11: MMA of stream 0, 1; 8 bits: 12..15: keys and values
constexpr int kTcThreads = 384, kTc8Threads = 512;
// Units of a tile, with two row streams and with alternate tiles (8 : 8 instead:
// trees 101 us, 8 : 4: 96), and of a job before its tiles.  us with lead 0 / 16 /
// 32: 64 trees of 30 over 1000 positions 113 / 66 / 64, 8 trees of 40 up to 8000
// 67 / 49 / 48, the chunks 137 / 135 / 132.
constexpr int kTcCostFull = 8, kTcCostHalf = 5, kTcLead = 32;
// 8 bits, keys made fp16 (kCache 1 below): the conversions of a tile take as long
// for 128 rows as for 256, and nothing runs beside them (2.9 us against 2.2).  us
// of the chunks and of 16 sequences up to 256 rows (6000 positions) with half a
// tile at 5 / 8 / 10 / 11 : 8: 210 / 183 / 179 / 179, 308 / 284 / 280 / 282.  Heads
// of 64: 1.5 against 1.8; at 6 / 8 / 10 : 8 137 / 138 / 139, 213 / 219 / 222.
// (With m following at once, kLag above, the chunks are at 180, of heads of 64 at 140.)
// Keys as they are (kCache 2): 1.5 us against 2.5; lead 16 / 32 / 48 / 64: 8 trees
// of 61 up to 20000 positions 113 / 108 / 105 / 107.
template <int D>
constexpr int kTc8CostHalf = D == 64 ? 7 : 10;
constexpr int kTc8Lead = 40, kTcE4Lead = 48;

template <int D>
struct TcShape {
    static constexpr uint32_t kTile = 128 * D * 2;      // a 128 x D fp16 tile: D / 64 swizzled slabs of 16 KB
    static constexpr int kStages = D == 128 ? 2 : 4;    // of keys, and of values
    static constexpr size_t kSmem = 1024 + (2 + 2 * kStages) * (size_t)kTile + 512 + 8 * 2048;  // tiles, barriers, staging
};

// 8 bits: a slot for 32 positions' codes per converting warp, instead of the
// outputs' staging.
constexpr int kTcSlots = kTc8Threads / 32 - 10;  // (kCache 2: one is not used)
template <int D>
struct Tc8Shape : TcShape<D> {
    static constexpr uint32_t kSlot = 32 * D;
    static constexpr size_t kSmem = 1024 + (2 + 2 * TcShape<D>::kStages) * (size_t)TcShape<D>::kTile + 512 + kTcSlots * kSlot + (32 + 256) * 4;
};

struct TcBars {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t v_clean[4];  // two row streams: stream 0 has cleared what stream 1's products must not meet
    // per stream: a step's scores; its P, positions 0 .. 63 and 64 .. 127; its turn
    uint64_t s_full[2], pa_full[2], pb_full[2], turn[2], drain[2];
    uint64_t q_full, o_full, x_full, x_done;
    uint64_t raw_full[kTcSlots];  // 8 bits
    uint32_t tmem_base;
    volatile int abort;
    volatile int odd[8];  // last segment (modulo kOdd) that met infinities or NaN among its new rows' values
};

__device__ __forceinline__ bool tc_wait(TcBars& B, uint64_t& bar, uint32_t parity, int* err) {
    if (B.abort) return false;
    if (!q4d::mbar_wait(q4d::smem_addr(&bar), parity, err)) {
        B.abort = 1;
        return false;
    }
    return true;
}

__device__ __forceinline__ uint32_t sw_off(int r, int c) {  // row r, 16-byte chunk c < 8 of a swizzled slab
    return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

// 32 consecutive 32-bit columns of this thread's tensor-memory lane.
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Bits 0 .. 31: which of the positions behind new row j0 (negative: cached)
// row `tok` of a sequence sees.
__device__ __forceinline__ uint32_t sees_word(const Args& a, const Seq& q, int tok, int j0) {
    if (j0 >= q.n) return 0u;
    if (j0 + 32 <= 0) return 0xffffffffu;
    uint32_t bits;
    const int lo = j0 < 0 ? 0 : j0;
    if (!a.mask) {
        const int n = tok - lo + 1;  // rows lo .. tok
        bits = n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
    } else {
        const uint32_t* m = a.mask + (size_t)(q.start + tok) * a.mask_words;
        const int w = lo >> 5, s = lo & 31;
        const uint32_t w0 = w < a.mask_words ? m[w] : 0u, w1 = s && w + 1 < a.mask_words ? m[w + 1] : 0u;
        bits = s ? (w0 >> s) | (w1 << (32 - s)) : w0;
    }
    if (q.n - lo < 32) bits &= (1u << (q.n - lo)) - 1u;
    return j0 < 0 ? (bits << -j0) | ((1u << -j0) - 1u) : bits;
}

// New rows that every row of the job sees.
__device__ __forceinline__ int all_see(const Args& a, const Place& p) {
    return a.mask ? 0 : (int)q4p::page_of(a.by_g, p.rb * a.BM) + 1;
}

// Elements 8 c .. of row e of a stream's query, 16 lanes a row, from fp16 (two
// slabs of swizzled 128-byte rows) to three e4m3 parts (three, 16 KB apart, the
// first two in the same place) of the query times a power of two, whose inverse
// goes to *scale.  A row with an infinity becomes NaN, as its scores would be.
__device__ __forceinline__ void split_query(uint8_t* dst, int e, int c, float* scale) {
    const uint4 q = *reinterpret_cast<const uint4*>(dst + (c >> 3) * 16384 + sw_off(e, c & 7));
    __syncwarp();
    uint32_t x[4] = {q.x, q.y, q.z, q.w};
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top2 = q4p::max2(top2, x[i] & 0x7fff7fffu);  // (NaN loses: it makes its element NaN)
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top2 = q4p::max2(top2, __shfl_xor_sync(0xffffffffu, top2, o));
    const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
    // top = m 2^k, 1 <= m < 2, k >= -14 (a lesser one counts as 2^-14): times
    // 2^(7 - k) = 2^up 2^(7 - k - up), of which fp16 has both
    const int k = max((int)(top >> 10), 1) - 15, up = min(7 - k, 15);
    const uint32_t f0 = (top >> 10) == 31 ? 0x7e007e00u : (uint32_t)(15 + up) * 0x04000400u, f1 = (uint32_t)(15 + 7 - k - up) * 0x04000400u;
    if (c == 0) *scale = __uint_as_float((uint32_t)(127 - 7 + k) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = q4p::mul2(q4p::mul2(x[i], f0), f1);
    uint8_t* const to = dst + sw_off(e, c >> 1) + 8 * (c & 1);
#pragma unroll
    for (int part = 0; part < 3; ++part) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = q4p::half2_e4m3(x[i]);
            if (part < 2) x[i] = q4p::sub2(x[i], q4p::e4m3_half2(w[i]));  // exact
        }
        *reinterpret_cast<uint2*>(to + part * 16384) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    }
}

// Clears row `row` of a value tile, or only its infinities and NaN; whether there were any.
template <int D>
__device__ __noinline__ bool clean_row(uint8_t* tile, int row, bool all) {
    bool found = false;
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
        uint4* at = reinterpret_cast<uint4*>(tile + (c >> 3) * 16384 + sw_off(row, c & 7));
        if (all) {
            *at = make_uint4(0, 0, 0, 0);
            continue;
        }
        const uint4 w = *at;
        uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!finite16((uint16_t)ws[e])) ws[e] &= 0xffff0000u, bad = true;
            if (!finite16((uint16_t)(ws[e] >> 16))) ws[e] &= 0x0000ffffu, bad = true;
        }
        if (bad) *at = make_uint4(ws[0], ws[1], ws[2], ws[3]);
        found |= bad;
    }
    return found;
}

//
// kCache 1 (8 bits): warps 8, 9 and 12 .. 15 bring the codes and make them fp16,
// 32 positions of a tile at a time, in turn, first the keys', then the values'.
// Each has a slot of its own in shared memory: it waits for a copy, takes it
// into registers, sets the next copy going (bulk copies of the rows that lie
// together in a page) and, when the tile that the MMA reads is free, stores the
// rows into it with the scales multiplied in (exact).  It also clears what must
// not reach every row, so that the softmax has nothing to do with the tiles.
// kCache 2 (heads of 128, pages of whole blocks): the keys stay e4m3, tiles that
// warp 8's TMA brings and the MMA takes as they are, and five converting warps
// have the values alone.  The query is split: a power of two times it, whose
// greatest element then lies in 128 .. 256, is the sum of three e4m3 numbers but
// for 2^-10 (2^-17 of the greatest), S = Q1 K + Q2 K + Q3 K in one accumulator,
// half as long again as the fp16 product.  The blocks' scales (16 columns of S
// each) and the row's enter the maximum and the exponent.
//
// What bounds it: the converting warps (some 2900 cycles for 32 positions: a
// warp's instructions one after another, fetched anew beside the other roles')
// where a tile has 128 rows, the softmax and the products where it has 256.
// Measured, contexts and heads as above: the chunks 180 us (kCache 1), the trees
// 104 us (kCache 2; 1 takes 119).  It spills 28 .. 44 bytes at 128 registers, outside
// the loops over tiles (a warp loads 11 registers in the whole of the chunks).  Keys and values by turns in one body; tried in
// kCache 1 (trees / chunks, before the tiles' costs were weighed: 150 / 215): a
// warp that brings the slots of all 197 / 311, four converting warps 215 / 328,
// five 148 / 237, pairs of a key and a value quarter 155 / 291, 16 positions at a
// time 212 / 280.  In kCache 2: keys of 128 rows or fewer alone as they are, by
// the converting warps themselves, 158 / 260; the tiles asked into L2 ahead 113.
template <int D, int kCache>
__global__ void __launch_bounds__(kCache ? kTc8Threads : kTcThreads, 1)
    tree_attn_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ MapArgs t) {
    constexpr bool k8 = kCache > 0, kRaw = kCache == 2;
    using Sh = std::conditional_t<k8, Tc8Shape<D>, TcShape<D>>;
    static_assert(sizeof(TcBars) <= 512, "barriers");
    constexpr uint32_t kTile = Sh::kTile;
    constexpr int NST = Sh::kStages, SLABS = D / 64;
    static_assert(!kRaw || (D == 128 && NST == 2), "keys as they are: heads of 128");
    constexpr int kThr = k8 ? kTc8Threads : kTcThreads;
    // Notes of infinities and NaN: the warps that find them run ahead of the
    // ones that read them by less than so many segments (the softmax by one; the
    // tiles' warps by the stages as well, 4 at most, of a tile each, and by the
    // positions in their registers).
    constexpr uint32_t kOdd = k8 ? 8 : 2;
    constexpr uint32_t kColS = 0, kColO = 256;
    const Args& a = t.a;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ unsigned share_s;
    __shared__ __align__(16) unsigned sums[2 * 256];  // the threads' running sums; later (m, l) of both streams' rows, float2
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr uint32_t kPart = 128 * 128;             // kRaw: a part of a stream's query, a tile of keys
    constexpr uint32_t kQuery = kRaw ? 3 * kPart : kTile, kKeyTile = kRaw ? kPart : kTile;
    uint8_t* q_s = base;                              // two tiles (kRaw: of three parts)
    uint8_t* k_s = base + 2 * kQuery;
    uint8_t* v_s = k_s + NST * kKeyTile;
    static_assert(2 * kQuery + NST * kKeyTile == (2 + NST) * kTile, "the same room");
    TcBars& B = *reinterpret_cast<TcBars*>(v_s + NST * kTile);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int* err = a.w.err;

    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            q4d::mbar_init(q4d::smem_addr(&B.k_full[i]), kRaw ? 33 : k8 ? 4 : 1);  // kRaw: TMA's bytes, every lane's copies
            q4d::mbar_init(q4d::smem_addr(&B.k_empty[i]), 2);  // both streams' MMAs
            q4d::mbar_init(q4d::smem_addr(&B.v_full[i]), k8 ? 4 : 1);
            q4d::mbar_init(q4d::smem_addr(&B.v_empty[i]), 2);
            q4d::mbar_init(q4d::smem_addr(&B.v_clean[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            q4d::mbar_init(q4d::smem_addr(&B.s_full[i]), 1);
            q4d::mbar_init(q4d::smem_addr(&B.pa_full[i]), 4);
            q4d::mbar_init(q4d::smem_addr(&B.pb_full[i]), 4);
            q4d::mbar_init(q4d::smem_addr(&B.turn[i]), 4);
            q4d::mbar_init(q4d::smem_addr(&B.drain[i]), 1);
        }
        for (int i = 0; i < (int)kOdd; ++i) B.odd[i] = 0;
        if constexpr (k8)
            for (int i = 0; i < kTcSlots; ++i) q4d::mbar_init(q4d::smem_addr(&B.raw_full[i]), 1);
        q4d::mbar_init(q4d::smem_addr(&B.q_full), 8);
        q4d::mbar_init(q4d::smem_addr(&B.o_full), 2);
        q4d::mbar_init(q4d::smem_addr(&B.x_full), 8);
        q4d::mbar_init(q4d::smem_addr(&B.x_done), 8);
        B.abort = 0;
        q4d::fence_mbar_init();
    }
    if (warp == 11) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         q4d::smem_addr(&B.tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const unsigned line = line_scan(a, sums, kThr);
    q4t::fence_before();
    __syncthreads();
    q4t::fence_after();
    q4d::pdl_trigger();
    const uint32_t tmem = B.tmem_base;

    if (tid == 0) {  // (the thread that may write a record later)
        a.rec[blockIdx.x] = make_int4(0, 0, 0, 0);
        share_s = line_share(a, line);
    }

    Walk w;
    if (w.begin(a, sums, kThr, line)) {
        // Every role walks the same segments.
        Place& p = w.p;
        bool rest = true;     // segments to do
        uint32_t seg = 0;   // segments done
        uint32_t tiles0 = 0;  // tiles before this segment

        // kRaw: [4 tiles][8 blocks] key scales, [2 streams][128] what a row's
        // scores are to be multiplied by.  (Tile kt's scales are written once
        // the scores of tile kt - 2 are there; those wait until their stream has
        // read the step before, tile kt - 4 or later, and the first of a segment
        // until both streams have ended the one before.)
        float* const key_scales = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(&B) + 512 + kTcSlots * Tc8Shape<D>::kSlot);
        float* const row_scales = key_scales + 32;
        if (k8 && ((!kRaw && warp == 8) || warp == 9 || warp >= 12)) {
            // --------------------------------------------- codes to fp16
            if constexpr (k8) {
                constexpr int NC = D / 8, PER = 32 / NC, NL = 32 / PER;  // lanes of a row (8 codes each), rows at a time, loads
                constexpr uint32_t kConv = kRaw ? kTcSlots - 1 : kTcSlots;
                const int c = lane % NC, g = lane / NC, own = (warp < 10 ? warp - 8 : warp - 10) - (kRaw ? 1 : 0);
                uint8_t* const slot = reinterpret_cast<uint8_t*>(&B) + 512 + own * Sh::kSlot;
                const uint32_t slot_s = q4d::smem_addr(slot) + lane * D, fb = q4d::smem_addr(&B.raw_full[own]);
                // Quarters of the line's tiles, 4 each; lane = position.  A quarter
                // is looked up while the one before it is copied and the one before
                // that stored.  The cursor p stands at the tile of quarter `next`,
                // the last one looked up.
                uint32_t next = own, kt = 0;
                int id = -1, key = 0;
                bool live = false;
                const auto look_up = [&]() {  // (the page number is used later)
                    key = p.tile * kTcKeys + 32 * (int)(next & 3) + lane;
                    live = key < p.q.ctx + p.q.n;
                    if (live) id = a.w.table[(size_t)p.s * a.w.max_pages + q4p::page_of(a.w.div, (uint32_t)key)];
                };
                // moves the cursor on, to quarter `next` (false: there is none)
                const auto advance = [&]() {
                    while (next >= 4 * kt + 4) {
                        ++kt;
                        if (++p.tile < w.end) continue;
                        ++seg;
                        if (!w.more(a)) return false;
                        w.next(a);
                    }
                    return true;
                };
                // number, segment, rows that exist, first new row (32 and more:
                // none); this lane's row (offset) and scales
                struct Quarter {
                    uint32_t at, seg, there;
                    int fresh;
                    long long row;
                    float ks, vs;
                };
                const auto resolve = [&]() {
                    Quarter x;
                    const bool mine = live && (uint32_t)id < (uint32_t)a.w.n_pages;
                    if (live && !mine) atomicOr(err, q4d::kErrDeviceCheck);
                    const int in_page = (int)((uint32_t)key - q4p::page_of(a.w.div, (uint32_t)key) * a.w.div.d);
                    const long long head = (long long)id * a.w.H + p.h, at = head * a.nb + in_page / q4p::kBlock;
                    x.row = (head * a.w.div.d + in_page) * D;
                    x.ks = mine ? a.ks[at] : 0.f;
                    x.vs = mine ? a.vs[at] : 0.f;
                    x.there = __ballot_sync(0xffffffffu, mine);
                    x.at = next;
                    x.seg = seg;
                    x.fresh = p.q.ctx - (key - lane);
                    return x;
                };
                const auto leads = [&](const Quarter& x) { return (x.there >> lane & 1u) && (lane & (t.box - 1)) == 0; };
                const auto copy = [&](const Quarter& x, const uint16_t* pool) {
                    const bool mine = leads(x);
                    const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
                    if (lane == 0) q4d::mbar_arrive_expect_tx(fb, (uint32_t)(boxes * t.box * D));
                    __syncwarp();
                    if (mine) q4d::bulk_g2s(slot_s, reinterpret_cast<const uint8_t*>(pool) + x.row, (uint32_t)(t.box * D), fb);
                };
                bool more = advance();
                Quarter now = {}, then = {};
                if (more) {
                    look_up();
                    now = resolve();
                    copy(now, kRaw ? a.w.v : a.w.k);
                    next += kConv;
                }
                bool further = more && advance(), again = false;
                if (further) look_up();
                // `turns` copies have been taken: keys and values by turns.  (One
                // body for both: the code's length costs instruction fetches.)
                uint32_t turns = 0;
                bool flying = more;  // a copy is on its way
#pragma unroll 1
                while (more) {
                    const bool values = kRaw || (turns & 1);
                    const uint32_t tile = now.at >> 2, st = tile % NST;
                    if (!__all_sync(0xffffffffu, tc_wait(B, B.raw_full[own], turns & 1, err))) break;
                    ++turns;
                    uint2 r[NL];
#pragma unroll
                    for (int e = 0; e < NL; ++e) r[e] = *reinterpret_cast<const uint2*>(slot + e * 256 + lane * 8);
                    const float scale = values ? now.vs : now.ks;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the next copy may write the slot
                    __syncwarp();
                    if (now.there != 0xffffffffu) {
#pragma unroll
                        for (int e = 0; e < NL; ++e)
                            if (!(now.there >> (e * PER + g) & 1u)) r[e] = make_uint2(0u, 0u);
                    }
                    if (kRaw || !values) again = further;
                    if (kRaw) {
                        if (further) then = resolve();
                        next += kConv;
                    }
                    flying = !values || again;
                    if (flying) copy(values ? then : now, values && !kRaw ? a.w.k : a.w.v);
                    if (!values) {
                        if (further) then = resolve();
                        next += kConv;
                    } else {
                        if (further && (further = advance())) look_up();
                        if (now.fresh < 32) {  // new rows' NaN
                            bool found = false;
#pragma unroll
                            for (int e = 0; e < NL; ++e) {
                                if (e * PER + g < now.fresh) continue;
                                const uint2 x = make_uint2(without_nan(r[e].x), without_nan(r[e].y));
                                found |= x.x != r[e].x || x.y != r[e].y;
                                r[e] = x;
                            }
                            if (found) B.odd[now.seg & (kOdd - 1)] = (int)now.seg + 1;
                            __syncwarp();
                        }
                    }
                    uint64_t* empty = values ? B.v_empty : B.k_empty;
                    if (tile >= (uint32_t)NST && !__all_sync(0xffffffffu, tc_wait(B, empty[st], (tile / NST - 1) & 1, err))) break;
                    // row y = e * PER + g at (y / 8) * 1024 + (y % 8) * 128, chunk c of its slab
                    uint8_t* const to = (values ? v_s : k_s) + st * kTile + (c >> 3) * 16384 + 4096 * (now.at & 3);
                    const uint32_t f2 = pack2(scale, scale);
#pragma unroll
                    for (int e = 0; e < NL; ++e) {
                        const uint32_t f = __shfl_sync(0xffffffffu, f2, e * PER + g);
                        *reinterpret_cast<uint4*>(to + sw_off(e * PER + g, c & 7)) =
                            make_uint4(q4p::mul2(q4p::e4m3_half2(r[e].x), f), q4p::mul2(q4p::e4m3_half2_hi(r[e].x), f),
                                       q4p::mul2(q4p::e4m3_half2(r[e].y), f), q4p::mul2(q4p::e4m3_half2_hi(r[e].y), f));
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(values ? &B.v_full[st] : &B.k_full[st]));
                    if (values) {
                        now = then;
                        more = again;
                    }
                }
                if (flying) q4d::mbar_wait(fb, turns & 1, nullptr);  // a copy in flight lands before the CTA can exit
            }
        } else if (kRaw && warp == 8) {
            // --------------------------------------------- tiles of keys as they are
            if constexpr (kRaw) {
                const int boxes = kTcKeys / t.box;
                bool ok = true;
                uint32_t kt = 0;
                while (rest && ok) {
                    const int len = p.q.ctx + p.q.n;
                    for (; p.tile < w.end && ok; ++p.tile, ++kt) {
                        const uint32_t st = kt % NST, fb = q4d::smem_addr(&B.k_full[st]);
                        // the first lanes a box each, and the first 8 a block's scale
                        const int key = p.tile * kTcKeys + lane * t.box, block = p.tile * kTcKeys + lane * q4p::kBlock;
                        int y = t.zero_row;
                        if (lane < boxes && key < len) {
                            const long long at = q4p::row_at(a.w, p.s, key, p.h, 1);
                            if (at >= 0) y = (int)at;
                            else atomicOr(err, q4d::kErrDeviceCheck);
                        }
                        const long long scale = lane < 8 && block < len ? scale_of(a, p.s, block, p.h) : -1;
                        if (kt >= (uint32_t)NST) ok = __all_sync(0xffffffffu, tc_wait(B, B.k_empty[st], (kt / NST - 1) & 1, err));
                        if (!ok) break;
                        if (lane == 0) q4d::mbar_arrive_expect_tx(fb, kPart);
                        __syncwarp();
                        if (lane < boxes) q4t::tma_load_2d(q4d::smem_addr(k_s + st * kPart) + lane * t.box * 128, &tmK, 0, y, fb);
                        if (lane < 8)
                            cp4(q4d::smem_addr(key_scales + (kt & 3) * 8 + lane), a.ks + (scale < 0 ? 0 : scale), scale >= 0);
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(fb) : "memory");
                    }
                    rest = w.more(a);
                    if (rest && ok) w.next(a);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                if (!ok) {  // copies still in flight land before the CTA can exit
                    for (uint32_t i = kt > (uint32_t)NST ? kt - NST : 0; i < kt; ++i)
                        q4d::mbar_wait(q4d::smem_addr(&B.k_full[i % NST]), (i / NST) & 1, nullptr);
                }
            }
        } else if (!k8 && (warp == 8 || warp == 9)) {
            // --------------------------------------------- key / value tiles
            const bool keys = warp == 8;
            uint64_t* full = keys ? B.k_full : B.v_full;
            uint64_t* empty = keys ? B.k_empty : B.v_empty;
            uint8_t* dst0 = keys ? k_s : v_s;
            const CUtensorMap* map = keys ? &tmK : &tmV;
            const int boxes = kTcKeys / t.box;
            bool ok = true;
            uint32_t kt = 0;
            while (rest && ok) {
                const int T = w.end - p.tile;
                const int len = p.q.ctx + p.q.n;
                for (int j = 0; j < T && ok; ++j, ++kt) {
                    const uint32_t st = kt % NST;
                    if (kt >= (uint32_t)NST) ok = __all_sync(0xffffffffu, tc_wait(B, empty[st], (kt / NST - 1) & 1, err));
                    if (!ok) break;
                    const uint32_t fb = q4d::smem_addr(&full[st]);
                    if (lane == 0) q4d::mbar_arrive_expect_tx(fb, kTile);
                    __syncwarp();
                    for (int b = lane; b < boxes; b += 32) {
                        const int key = (p.tile + j) * kTcKeys + b * t.box;
                        int y = t.zero_row;
                        if (key < len) {
                            const long long at = q4p::row_at(a.w, p.s, key, p.h, 1);
                            if (at >= 0) y = (int)at;
                            else atomicOr(err, q4d::kErrDeviceCheck);
                        }
                        const uint32_t dst = q4d::smem_addr(dst0 + st * kTile) + (uint32_t)(b * t.box) * 128u;
#pragma unroll
                        for (int sl = 0; sl < SLABS; ++sl) q4t::tma_load_2d(dst + sl * 16384, map, 64 * sl, y, fb);
                    }
                }
                rest = w.more(a);
                if (rest && ok) w.next(a);
            }
            if (!ok) {  // copies still in flight land before the CTA can exit
                for (uint32_t i = kt > (uint32_t)NST ? kt - NST : 0; i < kt; ++i)
                    q4d::mbar_wait(q4d::smem_addr(&full[i % NST]), (i / NST) & 1, nullptr);
            }
        } else if (warp == 10 || warp == 11) {
            // ------------------------------------------------- MMA issue
            // One warp per stream (a completed wait costs an issuing thread
            // about as much as four MMAs, so the streams' waits run side by
            // side), one elected lane issuing.
            const int i = warp - 10;
            const bool leader = elect_one();
            const uint32_t id_s = q4t::idesc_f16_m128(kTcKeys, 0), id_o = q4t::idesc_f16_m128(D, 1);
            const uint64_t dq = q4t::sw128_desc(q4d::smem_addr(q_s), 16, 1024);
            const uint64_t dk = q4t::sw128_desc(q4d::smem_addr(k_s), 16, 1024);
            const uint64_t dv = q4t::sw128_desc(q4d::smem_addr(v_s), 16384, 1024);
            const uint32_t sd = tmem + kColS + 128 * i, od = tmem + kColO + 128 * i;
            bool ok = true;
            uint32_t n_p = 0;     // steps done: the phases of pa_full and pb_full
            uint32_t cleans = 0;  // parity of the v_clean phases passed, a bit per stage
            while (rest && ok) {
                const int T = w.end - p.tile;
                const bool two = p.q.n * a.G - p.rb * a.BM > 128;
                const int steps = two ? T : (T - i + 1) / 2;
                const uint64_t ad = dq + (uint64_t)((two ? i : 0) * (kQuery / 16));
                const auto tile_of = [&](int k) { return tiles0 + (two ? k : 2 * k + i); };
                // the scores of step k (its keys have landed)
                const auto issue_s = [&](int k) {
                    const uint32_t st = tile_of(k) % NST;
                    const uint64_t bd = dk + (uint64_t)(st * (kKeyTile / 16));
                    if (leader) {
                        if constexpr (kRaw) {
                            // (the instruction descriptor's types: e4m3 is 0 here as fp16 is there)
#pragma unroll
                            for (int kk = 0; kk < 12; ++kk)
                                q4t::mma_ss_e4m3(sd, ad + (uint64_t)((kk >> 2) * (kPart / 16) + (kk & 3) * 2), bd + (uint64_t)((kk & 3) * 2), id_s,
                                                 kk > 0 ? 1u : 0u);
                        } else {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint64_t off = (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) / 16);
                                q4t::mma_ss(sd, ad + off, bd + off, id_s, kk > 0 ? 1u : 0u);
                            }
                        }
                        q4t::commit(q4d::smem_addr(&B.s_full[i]));
                        q4t::commit(q4d::smem_addr(&B.k_empty[st]));
                        if (!two) q4t::commit(q4d::smem_addr(&B.k_empty[st]));  // the barrier counts both streams
                    }
                    __syncwarp();
                };
                // half h of O += P V of step k: its positions 64 h ..
                const auto issue_pv = [&](int k, int h) {
                    const uint64_t bd = dv + (uint64_t)((tile_of(k) % NST) * (kTile / 16));
                    if (leader) {
#pragma unroll
                        for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                            q4t::mma_ts(od, sd + 8 * kk, bd + (uint64_t)(kk * 2048 / 16), id_o, (k > 0 || kk > 0) ? 1u : 0u);
                    }
                    __syncwarp();
                };
                const auto wait_k = [&](int k) {
                    const uint32_t kt = tile_of(k);
                    return tc_wait(B, B.k_full[kt % NST], (kt / NST) & 1, err);
                };
                ok = tc_wait(B, B.q_full, seg & 1, err);
                if (ok && steps > 0) {
                    ok = wait_k(0);
                    q4t::fence_after();
                    if (ok) issue_s(0);
                }
                for (int k = 0; k < steps && ok; ++k) {
                    const uint32_t kt = tile_of(k), st = kt % NST;
                    const bool more = k + 1 < steps;
                    ok = tc_wait(B, B.v_full[st], (kt / NST) & 1, err) && (!more || wait_k(k + 1)) &&
                         tc_wait(B, B.pa_full[i], n_p & 1, err);
                    if (!k8 && ok && two && i == 1 && (p.tile + k + 1) * kTcKeys > p.q.ctx + all_see(a, p)) {
                        ok = tc_wait(B, B.v_clean[st], cleans >> st & 1, err);
                        cleans ^= 1u << st;
                    }
                    if (!ok) break;
                    q4t::fence_after();
                    issue_pv(k, 0);
                    if (!(ok = tc_wait(B, B.pb_full[i], n_p & 1, err))) break;
                    q4t::fence_after();
                    issue_pv(k, 1);
                    ++n_p;
                    if (more) issue_s(k + 1);
                    if (leader) {
                        q4t::commit(q4d::smem_addr(&B.v_empty[st]));
                        if (!two) q4t::commit(q4d::smem_addr(&B.v_empty[st]));
                        if (!more) q4t::commit(q4d::smem_addr(&B.o_full));
                    }
                    __syncwarp();
                }
                if (steps == 0 && leader) q4d::mbar_arrive(q4d::smem_addr(&B.o_full));
                tiles0 += T;
                ++seg;
                rest = w.more(a);
                if (rest && ok) w.next(a);
            }
            if (!ok) B.abort = 1;
            // every MMA this warp issued has finished before the CTA winds down
            if (leader) q4t::commit(q4d::smem_addr(&B.drain[i]));
            __syncwarp();
            q4d::mbar_wait(q4d::smem_addr(&B.drain[i]), 0, nullptr);
        } else if (warp < 8) {
            // ------------------------------------------------- softmax
            const int i = warp >> 2, wr = warp & 3;  // stream, TMEM lane quarter
            const int row = wr * 32 + lane;
            const uint32_t lt = tmem + ((uint32_t)(wr * 32) << 16);
            const uint32_t ts = lt + kColS + 128 * i, to = lt + kColO + 128 * i;
            const float2 cc = make_float2(a.c, a.c);
            float* ml_x = reinterpret_cast<float*>(sums);  // [2 streams][128] (m, l), for joins
            uint32_t n_s = 0;    // steps done: the phases of s_full
            uint32_t turns = 0;  // turns taken
            uint32_t joins = 0;  // joined segments so far
            bool joined = false;  // the last segment was one
            bool ok = true;
            // The job's row of this thread (none: -1), as token and head, and
            // its query into the stream's tile.  Both streams share stream 0's
            // tile where the job has 128 rows or fewer.
            const auto job_row = [&](const Place& w) {
                const int R = min(a.BM, w.q.n * a.G - w.rb * a.BM);
                const int r = (R > 128 ? 128 * i : 0) + row;
                return r < R ? r : -1;
            };
            const auto put_query = [&](const Place& w) {
                const bool two = w.q.n * a.G - w.rb * a.BM > 128;
                if (two || i == 0) {
                    // this warp's 32 rows, whole rows at a time
                    const int R = min(a.BM, w.q.n * a.G - w.rb * a.BM);
                    uint8_t* dst = q_s + (two ? i : 0) * kQuery;
                    constexpr int NC = D / 8, PER = 32 / NC;  // chunks of a row, rows per load
                    const int c = lane % NC;
                    const uint32_t col = q4d::smem_addr(dst) + (uint32_t)(c >> 3) * 16384u;
                    // (asynchronous loads in a loop: code that runs once per
                    // segment costs its instruction fetches)
#pragma unroll 4
                    for (int e = wr * 32 + lane / NC; e < wr * 32 + 32; e += PER) {
                        const int r = (two ? 128 * i : 0) + e;
                        const int rr = w.rb * a.BM + min(r, R - 1), tk = (int)q4p::page_of(a.by_g, rr);
                        cp16(col + sw_off(e, c & 7),
                             a.q + (size_t)(w.q.start + tk) * a.ldq + (size_t)(w.h * a.G + rr - tk * a.G) * D + 8 * c, r < R);
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    if constexpr (kRaw) {
#pragma unroll 4
                        for (int e = wr * 32 + lane / NC; e < wr * 32 + 32; e += PER)
                            split_query(dst, e, c, row_scales + (two ? 128 * i : 0) + e);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.q_full));
            };
            // The streams take turns at the exponentials: one computes them
            // while the tensor cores work for the other.  Left alone they fall
            // into step and both wait for each other's MMAs.
            const auto take_turn = [&]() {
                const bool open = i == 0 && turns == 0;  // stream 0 begins
                const bool go = open || tc_wait(B, B.turn[i], (turns - (i == 0)) & 1, err);
                ++turns;
                return (bool)__all_sync(0xffffffffu, go);
            };
            const auto pass_turn = [&]() {
                __syncwarp();
                if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.turn[1 - i]));
            };
            put_query(p);
            while (rest) {
                const int T = w.end - p.tile;
                const bool two = p.q.n * a.G - p.rb * a.BM > 128;
                const int r = job_row(p);
                const int tok = (int)q4p::page_of(a.by_g, p.rb * a.BM + max(r, 0));
                const int steps = two ? T : (T - i + 1) / 2;
                const int seen_by_all = p.q.ctx + all_see(a, p);
                float m = -INFINITY, l = 0.f;
                float c_row = 0.f;  // kRaw: scale log2 e times what the row's query was divided by
                for (int j = 0; j < steps; ++j) {
                    const int tj = two ? j : 2 * j + i;  // tile of the segment
                    const int key0 = (p.tile + tj) * kTcKeys;
                    const uint32_t kt = tiles0 + tj, st = kt % NST;
                    // some row of the job does not see some position of the tile
                    const bool tail = key0 + kTcKeys > seen_by_all;
                    // The row in halves, so that it fits the registers: the
                    // maximum of the second, of the first, P of the first, the
                    // second once more, P of the second.
                    uint32_t seen = 0;  // what this row sees of the tile, some bits of it (kCache 1, tail)
                    uint32_t s[64];
                    float x4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    const auto load_half = [&](int h) {
                        ld32(ts + 64 * h, s);
                        ld32(ts + 64 * h + 32, s + 32);
                        q4t::ld_wait();
                        if (tail) {
#pragma unroll
                            for (int w = 0; w < 2; ++w) {
                                const uint32_t bits = sees_word(a, p.q, tok, key0 + 64 * h + 32 * w - p.q.ctx);
                                if (kCache == 1) seen |= bits;
                                if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!(bits >> e & 1u)) s[32 * w + e] = 0xff800000u;
                            }
                        }
                    };
                    // kRaw: the scales of half h's four blocks (0, of one that does not
                    // exist, counts as 1: its scores are ruled out or 0)
                    float ks[4];
                    const auto load_scales = [&](int h) {
                        const float4 f = *reinterpret_cast<const float4*>(key_scales + (kt & 3) * 8 + 4 * h);
                        ks[0] = f.x == 0.f ? 1.f : f.x;
                        ks[1] = f.y == 0.f ? 1.f : f.y;
                        ks[2] = f.z == 0.f ? 1.f : f.z;
                        ks[3] = f.w == 0.f ? 1.f : f.w;
                    };
                    const auto max_half = [&](int h) {
                        if constexpr (kRaw) {
                            load_scales(h);
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                float y[4];
#pragma unroll
                                for (int f = 0; f < 4; ++f) {
                                    const uint32_t* z = s + 16 * b + f;
                                    y[f] = fmaxf(fmaxf(__uint_as_float(z[0]), __uint_as_float(z[4])),
                                                 fmaxf(__uint_as_float(z[8]), __uint_as_float(z[12])));
                                }
                                x4[b] = fmaxf(x4[b], fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * ks[b]);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 64; e += 8)
#pragma unroll
                                for (int f = 0; f < 4; ++f)
                                    x4[f] = fmaxf(x4[f], fmaxf(__uint_as_float(s[e + f]), __uint_as_float(s[e + 4 + f])));
                        }
                    };
                    ok = __all_sync(0xffffffffu, tc_wait(B, B.s_full[i], n_s & 1, err));
                    if (!ok) break;
                    ++n_s;
                    q4t::fence_after();
                    if (kRaw && j == 0) c_row = a.c * row_scales[(two ? 128 * i : 0) + row];
                    load_half(1);
                    max_half(1);
                    load_half(0);
                    max_half(0);
                    const float top = fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3]));
                    // an infinity in the query whose products are all of the other sign
                    // (finite ones stay below 2^40): NaN, not a row that sees nothing
                    if (kCache == 1 && top == -INFINITY && (!tail || seen)) l = NAN;
                    const float mx = top * (kRaw ? c_row : a.c);
                    float corr = 1.f;
                    if (mx > (k8 ? m : m + kLag)) {
                        corr = m == -INFINITY ? 1.f : ex2(m - mx);  // nothing seen yet: O and l are zero
                        m = mx;
                    }
                    const float sub = kShift - (m == -INFINITY ? 0.f : m);
                    const float2 ss = make_float2(sub, sub);
                    float2 sum = make_float2(0.f, 0.f), sum2 = make_float2(0.f, 0.f);
                    const auto exp_half = [&](int h) {
                        if constexpr (kRaw) load_scales(h);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float cb = kRaw ? c_row * ks[e >> 3] : 0.f;
                            float2 v = __ffma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])),
                                                  kRaw ? make_float2(cb, cb) : cc, ss);
                            v.x = ex2(v.x);
                            v.y = ex2(v.y);
                            if (e & 1) sum2 = __fadd2_rn(sum2, v);
                            else sum = __fadd2_rn(sum, v);
                            s[e] = pack2(v.x, v.y);
                        }
                        st32(ts + 32 * h, s);
                    };
                    if (!(ok = take_turn())) break;
                    exp_half(0);
                    // (this step's scores are in, so the step before is in O)
                    if (j > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            ld32(to + c0, s);
                            q4t::ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) * corr);
                            st32(to + c0, s);
                        }
                    }
                    // A new row's value reaches only the rows that see it, and
                    // what lies behind the sequence nobody: this thread clears
                    // its row of the value tile there, or its infinities and
                    // NaN, which the epilogue adds back where they are seen.
                    if (!k8 && tail && !(two && i == 1)) {
                        ok = __all_sync(0xffffffffu, tc_wait(B, B.v_full[st], (kt / NST) & 1, err));
                        if (!ok) break;
                        const int nj = key0 + row - p.q.ctx;
                        if (nj >= 0 && clean_row<D>(v_s + st * kTile, row, nj >= p.q.n)) B.odd[seg & (kOdd - 1)] = (int)seg + 1;
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        if (two) {
                            __syncwarp();
                            if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.v_clean[st]));
                        }
                    }
                    q4t::st_wait();
                    if (j == 0 && joined) {  // the other stream's threads have read this one's O
                        ok = __all_sync(0xffffffffu, tc_wait(B, B.x_done, (joins - 1) & 1, err));
                        if (!ok) break;
                    }
                    q4t::fence_before();
                    __syncwarp();
                    if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.pa_full[i]));
                    load_half(1);
                    exp_half(1);
                    pass_turn();
                    l = fmaf(l, corr, (sum.x + sum2.x) + (sum.y + sum2.y));
                    q4t::st_wait();
                    q4t::fence_before();
                    __syncwarp();
                    if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.pb_full[i]));
                }
                if (ok && !two && steps < (T + 1) / 2) {  // the other stream's last step has no partner here
                    ok = take_turn();
                    pass_turn();
                }
                if (!ok) break;
                ok = __all_sync(0xffffffffu, tc_wait(B, B.o_full, seg & 1, err));
                if (!ok) break;
                q4t::fence_after();
                // The next segment's queries go in first: its scores are
                // computed while this one's results are written.
                const Place done = p;
                const uint32_t seg_done = seg;
                tiles0 += T;
                ++seg;
                rest = w.more(a);
                if (rest) {
                    w.next(a);
                    put_query(p);
                }
                const bool job_begin = done.tile == 0, whole = job_begin && done.tile + T == done.tiles;
                if (tid == 0 && job_begin && !whole) write_record(a, done, share_s);
                // Of a job on alternate tiles every thread has half the row's
                // columns, of both streams' parts.
                const bool join = !two && T > 1;
                float f0 = 1.f, f1 = 0.f;
                if (join) {
                    *reinterpret_cast<float2*>(ml_x + 2 * (128 * i + row)) = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.x_full));
                    ok = __all_sync(0xffffffffu, tc_wait(B, B.x_full, joins & 1, err));
                    if (!ok) break;
                    ++joins;
                    const float2 u = *reinterpret_cast<const float2*>(ml_x + 2 * row);
                    const float2 v = *reinterpret_cast<const float2*>(ml_x + 2 * (128 + row));
                    m = fmaxf(u.x, v.x);
                    const float ms = m == -INFINITY ? 0.f : m;
                    f0 = ex2(u.x - ms);
                    f1 = ex2(v.x - ms);
                    l = u.y * f0 + v.y * f1;
                }
                if (join || two || i == 0) {
                    const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
                    const int slot = 2 * blockIdx.x + (job_begin ? 1 : 0);
                    const int R = min(a.BM, done.q.n * a.G - done.rb * a.BM);
                    const int rw = (two ? 128 * i : 0) + wr * 32;  // the warp's first row of the job
                    if (!whole && r >= 0 && (!join || i == 0)) part_ml(a, slot)[r] = make_float2(m, l);
                    const int c1 = join ? D / 2 * (i + 1) : D;
                    const uint32_t t0 = join ? lt + kColO : to;
                    // 16 columns at a time by way of shared memory, so that a
                    // warp stores whole sectors: 4 lanes per row.  (8 bits: whose
                    // room the codes' slots take: by shuffles.)
                    float* stage = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(&B) + 512) + warp * 512;
                    const auto write = [&](int ry, int col, const float4& v) {
                        if (ry >= R) return;
                        if (whole) {
                            const int rr = done.rb * a.BM + ry, tk = (int)q4p::page_of(a.by_g, rr);
                            *reinterpret_cast<uint2*>(a.out + (size_t)(done.q.start + tk) * a.ldo +
                                                      (size_t)(done.h * a.G + rr - tk * a.G) * D + col) =
                                make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
                        } else {
                            *reinterpret_cast<float4*>(part_o<D>(a, slot) + (size_t)ry * D + col) = v;
                        }
                    };
#pragma unroll 1
                    for (int c0 = join ? D / 2 * i : 0; c0 < c1; c0 += 16) {
                        uint32_t w[16];
                        float o[16];
                        q4t::ld16(t0 + c0, w);
                        q4t::ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(w[e]) * (f0 * inv);
                        if (join) {
                            q4t::ld16(t0 + 128 + c0, w);
                            q4t::ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = fmaf(__uint_as_float(w[e]), f1 * inv, o[e]);
                        }
                        if constexpr (k8) {
                            // 4 x 4 chunks of 4 lanes: chunk e of lane x goes to lane e, as chunk x
#pragma unroll
                            for (int b = 2; b > 0; b >>= 1) {
                                const bool up = lane & b;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    if (e & b) continue;
#pragma unroll
                                    for (int f = 0; f < 4; ++f) {
                                        const float give = up ? o[4 * e + f] : o[4 * (e + b) + f];
                                        const float got = __shfl_xor_sync(0xffffffffu, give, b);
                                        o[4 * e + f] = up ? got : o[4 * e + f];
                                        o[4 * (e + b) + f] = up ? o[4 * (e + b) + f] : got;
                                    }
                                }
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                write(rw + (lane & ~3) + e, c0 + 4 * (lane & 3), make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                *reinterpret_cast<float4*>(stage + lane * 16 + ((e ^ (lane >> 1 & 3)) * 4)) =
                                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                            __syncwarp();
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int y = e * 8 + (lane >> 2), c = lane & 3;
                                write(rw + y, c0 + 4 * c, *reinterpret_cast<const float4*>(stage + y * 16 + ((c ^ (y >> 1 & 3)) * 4)));
                            }
                            __syncwarp();
                        }
                    }
                    // (what comes next is a lane's own row, which others of the warp have written)
                    if constexpr (k8) __syncwarp();
                    if (B.odd[seg_done & (kOdd - 1)] == (int)seg_done + 1 && r >= 0) {
                        const int rr = done.rb * a.BM + r;
                        add_odd<D, k8>(a, done, T, tok, join ? D / 2 * i : 0, c1,
                                       whole ? a.out + (size_t)(done.q.start + tok) * a.ldo + (size_t)(done.h * a.G + rr - tok * a.G) * D
                                             : nullptr,
                                       part_o<D>(a, slot) + (size_t)r * D);
                    }
                }
                q4t::fence_before();  // O is read before this warp releases the next segment's products
                joined = join;
                if (join) {
                    __syncwarp();
                    if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.x_done));
                }
            }
        }
    }
    q4t::fence_before();
    __syncthreads();
    if (warp == 11) {
        q4t::fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// box: rows that lie together in a page (8 bits: 1, 2 .. 32).
template <int D, int kCache>
q4_status launch_tc(Args& a, const Pools& c, void* workspace, int sms, int box, cudaStream_t s, const char* what) {
    MapArgs t;
    a.ctas = sms < kMaxTcCtas ? sms : kMaxTcCtas;
    a.BM = kTcRows;
    a.KT = kTcKeys;
    a.KT_log2 = 7;
    a.cost_full = kTcCostFull;
    a.lead = kCache == 1 ? kTc8Lead : kCache == 2 ? kTcE4Lead : kTcLead;
    a.cost_half = kCache == 1 ? kTc8CostHalf<D> : kTcCostHalf;
    place_parts<D>(a, workspace);
    t.a = a;
    t.box = box;
    t.zero_row = (int)((long long)c.n_pages * c.n_kv_heads * c.page_size);
    CUtensorMap tmK = {}, tmV = {};
    constexpr bool k8 = kCache > 0;
    if constexpr (kCache != 1) {
        const q4_status st = pool_maps<k8>(&tmK, &tmV, c, (uint32_t)box);
        if (st != Q4_OK) return st;
    }
    using Sh = std::conditional_t<k8, Tc8Shape<D>, TcShape<D>>;
    constexpr int kThr = k8 ? kTc8Threads : kTcThreads;
    const auto kern = tree_attn_tc_kernel<D, kCache>;
    static std::atomic<int> marks[64];
    cudaError_t e = q4i::ensure_smem_attr(reinterpret_cast<const void*>(kern), marks, (int)Sh::kSmem);
    if (e == cudaSuccess) {
        kern<<<a.ctas, kThr, Sh::kSmem, s>>>(tmK, tmV, t);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = launch_join(tree_join_many_kernel<D>, dim3((unsigned)(4 * sms)), a, s);
    return e == cudaSuccess ? Q4_OK : q4i::cuda_fail(e, what);
}

}  // namespace q4x
