// Attention of several sequences' new rows over a paged key / value cache:
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
// (each read once: 4 D bytes per position and head), beyond that the
// products.  The positions are the long axis, and there are often fewer
// (sequence, head) pairs than SMs, so the work is cut by positions: every
// (sequence, head, block of rows) is a job of 64-position tiles, all jobs'
// tiles stand in one line, and the CTA c of C takes its C-th part of the
// line.  A job that lies in one CTA's part is finished there; of a job that
// several share, each leaves (m, l, O) in the workspace (at most two per CTA:
// one job begun by another, one left unfinished), and a second kernel joins
// them in the order of the CTAs, so the bits do not depend on timing.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "q4_paged.cuh"
#include "q4_tc.cuh"

namespace q4x {

namespace cg = cooperative_groups;
using q4p::Seq;
using q4p::View;

constexpr int kKeys = 64;      // positions per tile
constexpr int kStages = 3;
constexpr int kMaxRows = 64;   // rows of a job
constexpr int kMaxCtas = 512;
constexpr int kTcRows = 256, kMaxTcCtas = 160;
// P = 2^(s - m + kShift): fp16 keeps 11 bits of a probability down to 2^-26
// of the row's greatest (below, it is off by 2^-37 of that at most), and O / l
// is the same quotient.  The tcgen05 kernel lets the greatest score exceed m by
// kLag, so P reaches 2^15.
constexpr float kShift = 12.f, kLag = 3.f;

struct Args {
    View w;
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
__device__ __noinline__ unsigned line_scan(const Args& a, unsigned* sums, int threads) {
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
    return max((line + (unsigned)a.ctas - 1) / (unsigned)a.ctas, 2u * (unsigned)a.cost_full);
}

// The job that holds unit x (x < the line's length), from its first tile on.
__device__ __noinline__ Place line_find(const Args& a, const unsigned* sums, int threads, unsigned x) {
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
        const unsigned share = line_share(a, line), x0 = share * blockIdx.x;  // below 2^31 + 512 * cost
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

// Adds to columns c0 .. c1 - 1 of a written row (fp16 `out`, else fp32 `part`)
// the infinities and NaN of the new rows it sees in the segment's T tiles.
template <int D>
__device__ __noinline__ void add_odd(const Args& a, const Place& p, int T, int tok, int c0, int c1, uint16_t* out,
                                     float* part) {
    const int n0 = max(0, p.tile * a.KT - p.q.ctx), n1 = min(p.q.n, (p.tile + T) * a.KT - p.q.ctx);
    for (int nj = n0; nj < n1; ++nj) {
        if (!sees(a, p.q.start, tok, nj)) continue;
        const long long at = q4p::row_at(a.w, p.s, p.q.ctx + nj, p.h, D);
        if (at < 0) continue;
        for (int c = c0; c < c1; ++c) {
            const uint16_t v = a.w.v[at + c];
            if (finite16(v)) continue;
            const float f = __half2float(__ushort_as_half(v));
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

template <int D>
struct Ring {
    static constexpr uint32_t kTile = kKeys * D * 2;  // keys or values of a tile
    static constexpr size_t kSmem = 1024 + (size_t)kStages * 2 * kTile + 256;
};

struct RingBars {
    uint64_t full[kStages], empty[kStages];
    volatile int abort;
    volatile int odd[2];  // last segment (by parity) that met infinities or NaN among its new rows' values
};

// Byte offset of row r, 16-byte chunk c in a tile of 64-wide swizzled slabs of 64 rows.
__device__ __forceinline__ uint32_t ring_off(int r, int c) {
    return (uint32_t)((c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
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

template <int D, int WM, bool kTma, bool kClustered>
__global__ void __launch_bounds__(kThreads, 2)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ MapArgs t) {
    constexpr int BM = 16 * WM, WN = 4 / WM;
    constexpr int NCH = D / 8, KS = D / 16, DN = D / 8, SLABS = D / 64;
    constexpr int KW = kKeys / WN, NT = KW / 8;  // a warp's positions of a tile, 8-wide tiles of them
    constexpr uint32_t TB = Ring<D>::kTile;
    const Args& a = t.a;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ unsigned sums[kThreads];
    __shared__ float2 ml_s[4 * 16], fin_s[kClustered ? BM : 1];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    RingBars& B = *reinterpret_cast<RingBars*>(smem + kStages * 2 * TB);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            // by cp.async every lane of the producing warp arrives
            q4d::mbar_init(q4d::smem_addr(&B.full[i]), kTma ? 1 : 32);
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
                if constexpr (kTma) {
                    // lanes 0 .. 7: boxes of keys, 8 .. 15: of values
                    const int b = lane & 7, key = p.tile * kKeys + b * t.box;
                    const bool mine = lane < 16 && b * t.box < kKeys;
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
                        const uint32_t dst = q4d::smem_addr(kv + (lane >> 3) * TB) + (uint32_t)(b * t.box) * 128u;
#pragma unroll
                        for (int sl = 0; sl < SLABS; ++sl)
                            q4t::tma_load_2d(dst + sl * (kKeys * 128), lane < 8 ? &tmK : &tmV, 64 * sl, y, fb);
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
                    for (int half = 0; half < 2; ++half) {
                        const int key = p.tile * kKeys + half * 32 + lane;
                        long long at = -1;
                        if (key < len) {
                            at = q4p::row_at(a.w, p.s, key, p.h, D);
                            if (at < 0) atomicOr(a.w.err, q4d::kErrDeviceCheck);
                        }
#pragma unroll 4
                        for (int e = 0; e < 32; e += PER) {
                            const int r = e + lane / NCH;
                            const long long row = __shfl_sync(0xffffffffu, at, r);
                            const long long off = (row < 0 ? 0 : row) + 8 * c;
                            const uint32_t to = kb + ring_off(half * 32 + r, c);
                            cp16(to, a.w.k + off, row >= 0);
                            cp16(to + TB, a.w.v + off, row >= 0);
                        }
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(fb) : "memory");
                }
            }
            rest = w.more(a);
            if (rest && ok) w.next(a);
        }
        if constexpr (!kTma) asm volatile("cp.async.wait_all;" ::: "memory");
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
    uint32_t qf[KS][4];
    float o[DN][4], m[2], l[2];
    bool fresh = true;              // the job's first tile in this CTA
    bool begun = p.tile == 0;       // ... and in the line
    const int row0 = wm * 16 + g;   // this thread's rows of the job: row0, row0 + 8
    uint32_t seg = 0, kt = 0;
    int seg_tile = p.tile;          // the segment's first tile
    const bool consume = warp < 4 && any;
    while (consume) {
        const int st = kt % kStages;
        const int R = min(BM, p.q.n * a.G - p.rb * BM);
        int tok[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) tok[e] = (int)q4p::page_of(a.by_g, p.rb * BM + min(row0 + 8 * e, R - 1));
        if (fresh) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool live = row0 + 8 * e < R;
                const int rr = p.rb * BM + min(row0 + 8 * e, R - 1);
                const uint16_t* src = a.q + (size_t)(p.q.start + tok[e]) * a.ldq + (size_t)(p.h * a.G + rr - tok[e] * a.G) * D + 2 * u;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
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
        const int key0 = p.tile * kKeys;
        const bool tail = key0 + kKeys > p.q.ctx;  // the tile holds new rows, or the end
        if (tail) {
            // A new row's value reaches only the rows that see it, and what
            // lies behind the sequence nobody: those rows are cleared, or
            // their infinities and NaN, which are added back at the end where
            // they are seen.  (Warps of the same positions write the same.)
            bool found = false;
            for (int y = lane; y < KW * NCH; y += 32) {
                const int r = wn * KW + y / NCH, c = y % NCH, nj = key0 + r - p.q.ctx;
                if (nj < 0) continue;
                uint4* at = reinterpret_cast<uint4*>(smem + st * 2 * TB + TB + ring_off(r, c));
                if (nj >= p.q.n) {
                    *at = make_uint4(0, 0, 0, 0);
                    continue;
                }
                const uint4 v = *at;
                uint32_t ws[4] = {v.x, v.y, v.z, v.w};
                bool bad = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (!finite16((uint16_t)ws[e])) ws[e] &= 0xffff0000u, bad = true;
                    if (!finite16((uint16_t)(ws[e] >> 16))) ws[e] &= 0x0000ffffu, bad = true;
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
#pragma unroll
        for (int kk = 0; kk < KS; kk += 2) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint32_t b[4];
                ldsm4(kb + ring_off(wn * KW + nt * 8 + (lane & 7), 2 * kk + (lane >> 3)), b);
                mma(sc[nt], qf[kk], b[0], b[1]);
                mma(sc[nt], qf[kk + 1], b[2], b[3]);
            }
        }
        if (tail) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int nj = key0 + wn * KW + nt * 8 + 2 * u + (e & 1) - p.q.ctx;
                    if (nj >= 0 && (nj >= p.q.n || !sees(a, p.q.start, tok[e >> 1], nj))) sc[nt][e] = -INFINITY;
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
        for (int kj = 0; kj < KW / 16; ++kj)
#pragma unroll
            for (int dn = 0; dn < DN; dn += 2) {
                uint32_t b[4];
                ldsm4_t(vb + ring_off(wn * KW + kj * 16 + (lane & 15), dn + (lane >> 4)), b);
                mma(o[dn], pa[kj], b[0], b[1]);
                mma(o[dn + 1], pa[kj], b[2], b[3]);
            }

        const bool job_end = p.tile + 1 == p.tiles, seg_end = p.tile + 1 == w.end;
        if (seg_end) {
            // the row sums over the quad's columns, then over the WN warps
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            }
            // The warps' outputs meet in this tile's stage, [WN][BM][D] fp32
            // (at most 32 KB), which is still ours; a cluster's CTA has
            // consumed all it loads, and takes stage 0, so that the others
            // know the place.
            float* ob = reinterpret_cast<float*>(smem + (kClustered ? 0 : st * 2 * TB));
            static_assert((size_t)WN * BM * D * 4 <= 2 * TB, "joining space");
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
                    float* dst = ob + ((size_t)wn * BM + wm * 16 + r) * D + 2 * u;
#pragma unroll
                    for (int dn = 0; dn < DN; ++dn)
                        *reinterpret_cast<float2*>(dst + 8 * dn) = make_float2(o[dn][2 * e] * f, o[dn][2 * e + 1] * f);
                    m[e] = mm;
                    l[e] = ls;
                }
                q4d::named_bar(1, kConsumers);
                if (wn == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int dn = 0; dn < DN; ++dn) {
                            float2 v = make_float2(0.f, 0.f);
#pragma unroll
                            for (int i = 0; i < WN; ++i) {
                                const float2 x = *reinterpret_cast<const float2*>(
                                    ob + ((size_t)i * BM + wm * 16 + g + 8 * e) * D + 2 * u + 8 * dn);
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
                        *reinterpret_cast<float2*>(ob + (size_t)r * D + 2 * u + 8 * dn) = make_float2(o[dn][2 * e], o[dn][2 * e + 1]);
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
                        if (whole) *reinterpret_cast<uint32_t*>(out + 8 * dn + 2 * u) = pack2(x, y);
                        else *reinterpret_cast<float2*>(part + 8 * dn + 2 * u) = make_float2(x, y);
                    }
                }
                if (B.odd[seg & 1] == (int)seg + 1) {
                    __syncwarp();  // the rows are written
                    Place from = p;
                    from.tile = seg_tile;
                    for (int e = 0; e < 2; ++e) {
                        const int r = row0 + 8 * e, rr = p.rb * BM + r;
                        if (r >= R || u != 0) continue;
                        add_odd<D>(a, from, p.tile + 1 - seg_tile, tok[e], 0, D,
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
                if (lane == 0) add_odd<D>(a, from, p.tiles, tok, 0, D, out, nullptr);
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

// The pools as 2-D maps [rows][D], boxes of 64 x box elements.
inline q4_status pool_maps(CUtensorMap* k, CUtensorMap* v, const q4_paged_cache& c, uint32_t box) {
    const uint64_t rows = (uint64_t)c.n_pages * c.n_kv_heads * c.page_size, D = (uint64_t)c.head_dim;
    const q4_status st = q4i::make_map(k, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, c.k, D, rows, D * 2, 64, box, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != Q4_OK) return st;
    return q4i::make_map(v, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, c.v, D, rows, D * 2, 64, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, int WM, bool kTma, bool kClustered>
cudaError_t launch_kernel(const CUtensorMap& k, const CUtensorMap& v, const MapArgs& t, int grid, cudaStream_t s) {
    static std::atomic<int> marks[64];
    const auto kern = tree_attn_kernel<D, WM, kTma, kClustered>;
    const void* fn = reinterpret_cast<const void*>(kern);
    cudaError_t e = q4i::ensure_smem_attr(fn, marks, (int)Ring<D>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Ring<D>::kSmem;
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
template <int D, int WM>
q4_status launch(Args& a, const q4_paged_cache& c, void* workspace, int sms, int box, cudaStream_t s) {
    MapArgs t;
    CUtensorMap k = {}, v = {};
    a.BM = 16 * WM;
    a.KT = kKeys;
    a.KT_log2 = 6;
    a.cost_full = a.cost_half = kRingCost;
    a.lead = kRingLead;
    a.ctas = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
    place_parts<D>(a, workspace);
    if (box) {
        const q4_status st = pool_maps(&k, &v, c, (uint32_t)box);
        if (st != Q4_OK) return st;
    }
    t.box = box;
    t.zero_row = (int)((long long)c.n_pages * c.n_kv_heads * c.page_size);
    // (n rows in S sequences that have some make at most S + (n - S) / BM blocks)
    const long long seqs = c.n_seqs < a.w.rows ? c.n_seqs : a.w.rows;
    const long long jobs = (seqs + ((long long)a.w.rows * a.G - seqs) / a.BM) * c.n_kv_heads;
    t.cluster = cluster_size(jobs, c.n_seqs, (long long)c.max_pages * c.page_size, sms);
    t.cluster_log2 = t.cluster == 16 ? 4 : t.cluster == 8 ? 3 : 2;
    t.a = a;
    const auto run = [&](auto tma) {
        constexpr bool T = decltype(tma)::value;
        return t.cluster ? launch_kernel<D, WM, T, true>(k, v, t, (int)jobs * t.cluster, s)
                         : launch_kernel<D, WM, T, false>(k, v, t, a.ctas, s);
    };
    cudaError_t e;
    if constexpr (WM == 4) e = run(std::false_type{});
    else e = box ? run(std::true_type{}) : run(std::false_type{});
    if (!t.cluster && e == cudaSuccess) e = launch_join(tree_join_kernel<D>, dim3((unsigned)a.ctas - 1, (unsigned)WM), a, s);
    return e == cudaSuccess ? Q4_OK : q4i::cuda_fail(e, "q4_tree_attention launch");
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
// more than kLag (a factor 2^3); then O and l are rescaled.
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
constexpr int kTcThreads = 384;  // warps 0..3, 4..7: softmax of stream 0, 1; 8: keys, 9: values, 10, 11: MMA of stream 0, 1
// Units of a tile, with two row streams and with alternate tiles (8 : 8 instead:
// trees 101 us, 8 : 4: 96), and of a job before its tiles.  us with lead 0 / 16 /
// 32: 64 trees of 30 over 1000 positions 113 / 66 / 64, 8 trees of 40 up to 8000
// 67 / 49 / 48, the chunks 137 / 135 / 132.
constexpr int kTcCostFull = 8, kTcCostHalf = 5, kTcLead = 32;

template <int D>
struct TcShape {
    static constexpr uint32_t kTile = 128 * D * 2;      // a 128 x D fp16 tile: D / 64 swizzled slabs of 16 KB
    static constexpr int kStages = D == 128 ? 2 : 4;    // of keys, and of values
    static constexpr size_t kSmem = 1024 + (2 + 2 * kStages) * (size_t)kTile + 512 + 8 * 2048;  // tiles, barriers, staging
};

struct TcBars {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t v_clean[4];  // two row streams: stream 0 has cleared what stream 1's products must not meet
    // per stream: a step's scores; its P, positions 0 .. 63 and 64 .. 127; its turn
    uint64_t s_full[2], pa_full[2], pb_full[2], turn[2], drain[2];
    uint64_t q_full, o_full, x_full, x_done;
    uint32_t tmem_base;
    volatile int abort;
    volatile int odd[2];  // last segment (by parity) that met infinities or NaN among its new rows' values
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

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_attn_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ MapArgs t) {
    using Sh = TcShape<D>;
    constexpr uint32_t kTile = Sh::kTile;
    constexpr int NST = Sh::kStages, SLABS = D / 64;
    constexpr uint32_t kColS = 0, kColO = 256;
    const Args& a = t.a;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ unsigned share_s;
    __shared__ __align__(16) unsigned sums[2 * 256];  // kTcThreads running sums; later (m, l) of both streams' rows, float2
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* q_s = base;                              // two tiles; between segments, stream 1's O (fp32)
    uint8_t* k_s = base + 2 * kTile;
    uint8_t* v_s = k_s + NST * kTile;
    TcBars& B = *reinterpret_cast<TcBars*>(v_s + NST * kTile);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int* err = a.w.err;

    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            q4d::mbar_init(q4d::smem_addr(&B.k_full[i]), 1);
            q4d::mbar_init(q4d::smem_addr(&B.k_empty[i]), 2);  // both streams' MMAs
            q4d::mbar_init(q4d::smem_addr(&B.v_full[i]), 1);
            q4d::mbar_init(q4d::smem_addr(&B.v_empty[i]), 2);
            q4d::mbar_init(q4d::smem_addr(&B.v_clean[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            q4d::mbar_init(q4d::smem_addr(&B.s_full[i]), 1);
            q4d::mbar_init(q4d::smem_addr(&B.pa_full[i]), 4);
            q4d::mbar_init(q4d::smem_addr(&B.pb_full[i]), 4);
            q4d::mbar_init(q4d::smem_addr(&B.turn[i]), 4);
            q4d::mbar_init(q4d::smem_addr(&B.drain[i]), 1);
            B.odd[i] = 0;
        }
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
    const unsigned line = line_scan(a, sums, kTcThreads);
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
    if (w.begin(a, sums, kTcThreads, line)) {
        // Every role walks the same segments.
        Place& p = w.p;
        bool rest = true;     // segments to do
        uint32_t seg = 0;   // segments done
        uint32_t tiles0 = 0;  // tiles before this segment

        if (warp == 8 || warp == 9) {
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
        } else if (warp >= 10) {
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
                const uint64_t ad = dq + (uint64_t)((two ? i : 0) * (kTile / 16));
                const auto tile_of = [&](int k) { return tiles0 + (two ? k : 2 * k + i); };
                // the scores of step k (its keys have landed)
                const auto issue_s = [&](int k) {
                    const uint32_t st = tile_of(k) % NST;
                    const uint64_t bd = dk + (uint64_t)(st * (kTile / 16));
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t off = (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) / 16);
                            q4t::mma_ss(sd, ad + off, bd + off, id_s, kk > 0 ? 1u : 0u);
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
                    if (ok && two && i == 1 && (p.tile + k + 1) * kTcKeys > p.q.ctx + all_see(a, p)) {
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
                    uint8_t* dst = q_s + (two ? i : 0) * kTile;
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
                for (int j = 0; j < steps; ++j) {
                    const int tj = two ? j : 2 * j + i;  // tile of the segment
                    const int key0 = (p.tile + tj) * kTcKeys;
                    const uint32_t kt = tiles0 + tj, st = kt % NST;
                    // some row of the job does not see some position of the tile
                    const bool tail = key0 + kTcKeys > seen_by_all;
                    // The row in halves, so that it fits the registers: the
                    // maximum of the second, of the first, P of the first, the
                    // second once more, P of the second.
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
                                if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!(bits >> e & 1u)) s[32 * w + e] = 0xff800000u;
                            }
                        }
                    };
                    const auto max_half = [&]() {
#pragma unroll
                        for (int e = 0; e < 64; e += 8)
#pragma unroll
                            for (int f = 0; f < 4; ++f)
                                x4[f] = fmaxf(x4[f], fmaxf(__uint_as_float(s[e + f]), __uint_as_float(s[e + 4 + f])));
                    };
                    ok = __all_sync(0xffffffffu, tc_wait(B, B.s_full[i], n_s & 1, err));
                    if (!ok) break;
                    ++n_s;
                    q4t::fence_after();
                    load_half(1);
                    max_half();
                    load_half(0);
                    max_half();
                    const float mx = fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * a.c;
                    float corr = 1.f;
                    if (mx > m + kLag) {
                        corr = m == -INFINITY ? 1.f : ex2(m - mx);  // nothing seen yet: O and l are zero
                        m = mx;
                    }
                    const float sub = kShift - (m == -INFINITY ? 0.f : m);
                    const float2 ss = make_float2(sub, sub);
                    float2 sum = make_float2(0.f, 0.f), sum2 = make_float2(0.f, 0.f);
                    const auto exp_half = [&](int h) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float2 v = __ffma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), cc, ss);
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
                    if (tail && !(two && i == 1)) {
                        ok = __all_sync(0xffffffffu, tc_wait(B, B.v_full[st], (kt / NST) & 1, err));
                        if (!ok) break;
                        const int nj = key0 + row - p.q.ctx;
                        if (nj >= 0 && clean_row<D>(v_s + st * kTile, row, nj >= p.q.n)) B.odd[seg & 1] = (int)seg + 1;
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
                    // warp stores whole sectors: 4 lanes per row
                    float* stage = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(&B) + 512) + warp * 512;
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
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<float4*>(stage + lane * 16 + ((e ^ (lane >> 1 & 3)) * 4)) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int y = e * 8 + (lane >> 2), c = lane & 3;
                            const float4 v = *reinterpret_cast<const float4*>(stage + y * 16 + ((c ^ (y >> 1 & 3)) * 4));
                            const int ry = rw + y;
                            if (ry >= R) continue;
                            if (whole) {
                                const int rr = done.rb * a.BM + ry, tk = (int)q4p::page_of(a.by_g, rr);
                                *reinterpret_cast<uint2*>(a.out + (size_t)(done.q.start + tk) * a.ldo +
                                                          (size_t)(done.h * a.G + rr - tk * a.G) * D + c0 + 4 * c) =
                                    make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
                            } else {
                                *reinterpret_cast<float4*>(part_o<D>(a, slot) + (size_t)ry * D + c0 + 4 * c) = v;
                            }
                        }
                        __syncwarp();
                    }
                    if (B.odd[seg_done & 1] == (int)seg_done + 1 && r >= 0) {
                        const int rr = done.rb * a.BM + r;
                        add_odd<D>(a, done, T, tok, join ? D / 2 * i : 0, c1,
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

template <int D>
q4_status launch_tc(Args& a, const q4_paged_cache& c, void* workspace, int sms, int box, cudaStream_t s) {
    MapArgs t;
    a.ctas = sms < kMaxTcCtas ? sms : kMaxTcCtas;
    a.BM = kTcRows;
    a.KT = kTcKeys;
    a.KT_log2 = 7;
    a.cost_full = kTcCostFull;
    a.lead = kTcLead;
    a.cost_half = kTcCostHalf;
    place_parts<D>(a, workspace);
    t.a = a;
    t.box = box;
    t.zero_row = (int)((long long)c.n_pages * c.n_kv_heads * c.page_size);
    CUtensorMap tmK, tmV;
    const q4_status st = pool_maps(&tmK, &tmV, c, (uint32_t)box);
    if (st != Q4_OK) return st;
    static std::atomic<int> marks[64];
    cudaError_t e = q4i::ensure_smem_attr(reinterpret_cast<const void*>(tree_attn_tc_kernel<D>), marks, (int)TcShape<D>::kSmem);
    if (e == cudaSuccess) {
        tree_attn_tc_kernel<D><<<a.ctas, kTcThreads, TcShape<D>::kSmem, s>>>(tmK, tmV, t);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = launch_join(tree_join_many_kernel<D>, dim3((unsigned)(4 * sms)), a, s);
    return e == cudaSuccess ? Q4_OK : q4i::cuda_fail(e, "q4_tree_attention launch");
}

}  // namespace q4x

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
    if (d.n_q_heads < d.cache.n_kv_heads || d.n_q_heads % d.cache.n_kv_heads)
        return fail(Q4_ERR_INVALID_ARG, "n_q_heads=%d is not a multiple of n_kv_heads=%d", d.n_q_heads, d.cache.n_kv_heads);
    if ((long long)d.n_q_heads * D > (1 << 24)) return fail(Q4_ERR_UNSUPPORTED, "%d query heads", d.n_q_heads);
    const int G = d.n_q_heads / d.cache.n_kv_heads;
    if ((long long)d.rows * G > (1ll << 30)) return fail(Q4_ERR_UNSUPPORTED, "rows=%d x %d query heads per kv head", d.rows, G);
    if (d.mask && d.mask_words < 1) return fail(Q4_ERR_INVALID_ARG, "mask_words=%d", d.mask_words);
    a.c = (d.scale == 0.f ? 1.f / sqrtf((float)D) : d.scale) * 1.4426950408889634f;
    if (!(a.c >= 1e-30f && a.c <= 1e30f)) return fail(Q4_ERR_INVALID_ARG, "scale=%g", d.scale);
    if (!aligned4(d.mask)) return fail(Q4_ERR_MISALIGNED, "mask must be 4-byte aligned");
    if ((st = row_matrix("q", d.q, d.n_q_heads * D, &d.ldq)) != Q4_OK) return st;
    if ((st = row_matrix("out", d.out, d.n_q_heads * D, &d.ldo)) != Q4_OK) return st;
    if (reinterpret_cast<uintptr_t>(d.workspace) & 255u) return fail(Q4_ERR_MISALIGNED, "the workspace must be 256-byte aligned");
    const size_t need = D == 128 ? q4x::workspace_bytes<128>() : q4x::workspace_bytes<64>();
    if (d.workspace_bytes < need) return fail(Q4_ERR_INVALID_ARG, "workspace %zu bytes, need %zu", d.workspace_bytes, need);
    const DeviceInfo* dev = nullptr;
    if ((st = current_device(&dev)) != Q4_OK) return st;
    if (d.rows == 0) return Q4_OK;
    a.w.err = dev->err_word;
    a.mask = d.mask;
    a.mask_words = d.mask_words;
    a.q = d.q;
    a.out = d.out;
    a.ldq = d.ldq;
    a.ldo = d.ldo;
    a.G = G;
    a.by_g = q4p::page_div((uint32_t)G);
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
    const long long avg = ((long long)d.rows * G + d.cache.n_seqs - 1) / d.cache.n_seqs;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // TMA boxes: the greatest power of two that divides a page, 8 at least (a
    // swizzled row group).  TMA / cp.async, us: 40 contexts up to 12000, pages of
    // 8 105 / 121, of 16 94 / 107, of 64 93 / 96; one user's 16000 positions 20 / 29.
    const int even = d.cache.page_size & -d.cache.page_size;
    const long long pool_rows = (long long)d.cache.n_pages * d.cache.n_kv_heads * d.cache.page_size;
    const bool tma = even >= 8 && pool_rows < (1ll << 31) - 1;
    const int ring_box = !tma ? 0 : even < q4x::kKeys ? even : q4x::kKeys;
    if (avg > 32 && tma) {
        const int box = even < q4x::kTcKeys ? even : q4x::kTcKeys;
        return D == 128 ? q4x::launch_tc<128>(a, d.cache, d.workspace, dev->sms, box, s)
                        : q4x::launch_tc<64>(a, d.cache, d.workspace, dev->sms, box, s);
    }
    if (D == 128)
        return avg <= 16   ? q4x::launch<128, 1>(a, d.cache, d.workspace, dev->sms, ring_box, s)
               : avg <= 32 ? q4x::launch<128, 2>(a, d.cache, d.workspace, dev->sms, ring_box, s)
                           : q4x::launch<128, 4>(a, d.cache, d.workspace, dev->sms, ring_box, s);
    return avg <= 16   ? q4x::launch<64, 1>(a, d.cache, d.workspace, dev->sms, ring_box, s)
           : avg <= 32 ? q4x::launch<64, 2>(a, d.cache, d.workspace, dev->sms, ring_box, s)
                       : q4x::launch<64, 4>(a, d.cache, d.workspace, dev->sms, ring_box, s);
}
