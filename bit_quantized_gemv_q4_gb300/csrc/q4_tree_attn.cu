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
#include <cuda_fp16.h>
#include <math.h>

#include "q4_paged.cuh"

namespace q4x {

using q4p::Seq;
using q4p::View;

constexpr int kKeys = 64;      // positions per tile
constexpr int kThreads = 128;  // 4 warps: WM of them along the rows, 4 / WM along the positions
constexpr int kStages = 3;
constexpr int kMaxRows = 64;   // rows of a job
constexpr int kMaxCtas = 512;
// P = 2^(s - m + kShift): fp16 keeps 11 bits of a probability down to 2^-26
// of the row's greatest, and O / l is the same quotient.
constexpr float kShift = 12.f;

struct Args {
    View w;
    const uint32_t* mask;
    int mask_words;
    const uint16_t* q;
    uint16_t* out;
    long long ldq, ldo;
    int G;       // query heads per kv head
    float c;     // scale * log2(e)
    float* part; // workspace: [2 CTAs][kMaxRows][D] outputs, then [2 CTAs][kMaxRows] (m, l)
    int ctas;
};

template <int D>
__device__ __forceinline__ float* part_o(const Args& a, int slot) {
    return a.part + (size_t)slot * kMaxRows * D;
}
template <int D>
__device__ __forceinline__ float2* part_ml(const Args& a, int slot) {
    return reinterpret_cast<float2*>(a.part + (size_t)2 * kMaxCtas * kMaxRows * D) + (size_t)slot * kMaxRows;
}

// ---------------------------------------------------------------- schedule ---
// Tiles of a sequence's row block `rb` (BM rows): with a mask every row may
// see every new row; causally the block's last token is the last key.
__device__ __forceinline__ int block_tiles(const Args& a, const Seq& q, int rb, int BM) {
    const int last = min(((rb + 1) * BM - 1) / a.G, q.n - 1);
    const int keys = q.ctx + (a.mask ? q.n : last + 1);
    return (keys + kKeys - 1) / kKeys;
}

// Tiles of one head of a sequence (all row blocks).
__device__ __forceinline__ long long head_tiles(const Args& a, const Seq& q, int BM) {
    if (q.n <= 0) return 0;
    const int blocks = (int)(((long long)q.n * a.G + BM - 1) / BM);
    if (a.mask) return (long long)blocks * block_tiles(a, q, 0, BM);
    long long t = 0;
    for (int b = 0; b < blocks; ++b) t += block_tiles(a, q, b, BM);
    return t;
}

// A place in the line of tiles.
struct Place {
    int s, h, rb, tile, tiles;  // tile of the job's `tiles`
    Seq q;
};

// The job line's length, and the place of tile x (by every thread; `sums`
// holds the threads' shares).  Each thread adds up a contiguous share of the
// sequences; the share that holds x is then walked.
__device__ __forceinline__ long long line_scan(const Args& a, int BM, long long* sums, int threads) {
    const int per = (a.w.S + threads - 1) / threads;
    const int lo = min(a.w.S, (int)threadIdx.x * per), hi = min(a.w.S, lo + per);
    long long t = 0;
    for (int s = lo; s < hi; ++s) {
        bool bad;
        const Seq q = q4p::seq_of(a.w, s, bad);
        if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.w.err, q4d::kErrDeviceCheck);
        t += head_tiles(a, q, BM);
    }
    t *= a.w.H;
    // inclusive scan over the threads
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += u;
    }
    __shared__ long long wsum[32];
    if (lane == 31) wsum[warp] = t;
    __syncthreads();
    for (int i = 0; i < warp; ++i) t += wsum[i];
    sums[threadIdx.x] = t;
    __syncthreads();
    return sums[threads - 1];
}

// Place of tile x (x < the line's length).
__device__ __forceinline__ Place line_find(const Args& a, int BM, const long long* sums, int threads, long long x) {
    int lo = 0, hi = threads - 1;  // first thread whose inclusive sum exceeds x
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (sums[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    if (lo > 0) x -= sums[lo - 1];
    const int per = (a.w.S + threads - 1) / threads;
    Place p;
    bool bad;
    long long head = 0;
    for (p.s = lo * per;; ++p.s) {
        p.q = q4p::seq_of(a.w, p.s, bad);
        head = head_tiles(a, p.q, BM);
        if (x < head * a.w.H) break;
        x -= head * a.w.H;
    }
    p.h = (int)(x / head);
    x -= p.h * head;
    for (p.rb = 0;; ++p.rb) {
        p.tiles = block_tiles(a, p.q, p.rb, BM);
        if (x < p.tiles) break;
        x -= p.tiles;
    }
    p.tile = (int)x;
    return p;
}

// The next tile's place (there is one).
__device__ __forceinline__ void step(const Args& a, int BM, Place& p) {
    if (++p.tile < p.tiles) return;
    p.tile = 0;
    if ((long long)++p.rb * BM >= (long long)p.q.n * a.G) {
        p.rb = 0;
        if (++p.h == a.w.H) {
            p.h = 0;
            do {
                bool bad;
                p.q = q4p::seq_of(a.w, ++p.s, bad);
            } while (p.q.n <= 0);
        }
    }
    p.tiles = block_tiles(a, p.q, p.rb, BM);
}

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

template <int D>
constexpr size_t attn_smem() {
    return (size_t)kStages * 2 * kKeys * D * 2;
}

// ------------------------------------------------------------------ kernel ---
// WM warps along the job's 16 WM rows, WN = 4 / WM along the tile's
// positions.  Fragment layouts of mma.m16n8k16 (g = lane / 4, u = lane % 4):
// A covers rows g, g + 8 and columns 2u, 2u+1, 2u+8, 2u+9; B rows 2u, 2u+1,
// 2u+8, 2u+9 of column g; an accumulator rows g, g + 8, columns 2u, 2u+1, so
// two neighbouring score tiles are the A operand of a 16-position step of P V.
template <int D, int WM>
__global__ void __launch_bounds__(kThreads, 2) tree_attn_kernel(const Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long sums[kThreads];
    __shared__ float2 ml_s[4][16];
    constexpr int BM = 16 * WM, WN = 4 / WM;
    constexpr int NCH = D / 8, KS = D / 16, DN = D / 8;
    constexpr int KW = kKeys / WN, NT = KW / 8;  // a warp's positions of a tile, 8-wide tiles of them
    constexpr uint32_t TB = kKeys * D * 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, u = lane & 3;
    const int wm = warp / WN, wn = warp % WN;
    const long long line = line_scan(a, BM, sums, kThreads);
    const long long x0 = line * blockIdx.x / a.ctas, x1 = line * (blockIdx.x + 1) / a.ctas;
    if (x0 >= x1) return;
    Place cur = line_find(a, BM, sums, kThreads, x0);
    Place ld = cur;
    const uint32_t sm0 = q4d::smem_addr(smem);

    // Tile `ld` into stage st: a thread takes one 16-byte chunk column of
    // every (kThreads / NCH)-th row.  Positions behind the sequence (stale
    // rows hold anything, and 0 * NaN would reach the sums) become zeros.
    auto load = [&](int st) {
        const uint32_t kb = sm0 + (uint32_t)st * 2u * TB, vb = kb + TB;
        const int c = tid % NCH, r0 = tid / NCH;
        const int len = ld.q.ctx + ld.q.n;
#pragma unroll
        for (int i = 0; i < kKeys * NCH / kThreads; ++i) {
            const int r = r0 + i * (kThreads / NCH);
            const int key = ld.tile * kKeys + r;
            long long at = -1;
            if (key < len) {
                at = q4p::row_at(a.w, ld.s, key, ld.h, D);
                if (at < 0) atomicOr(a.w.err, q4d::kErrDeviceCheck);
            }
            const bool live = at >= 0;
            const long long off = (live ? at : 0) + 8 * c;
            cp16(kb + swz<D>(r, c), a.w.k + off, live);
            cp16(vb + swz<D>(r, c), a.w.v + off, live);
        }
    };
    long long loaded = x0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (loaded < x1) {
            load(i);
            if (++loaded < x1) step(a, BM, ld);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    uint32_t qf[KS][4];
    float o[DN][4], m[2], l[2];
    bool fresh = true;   // the job's first tile in this CTA
    bool begun = cur.tile == 0;  // ... and in the line
    const int row0 = wm * 16 + g;  // this thread's rows of the job: row0, row0 + 8
    for (long long x = x0; x < x1; ++x) {
        const int st = (int)((x - x0) % kStages);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();
        if (loaded < x1) {
            load((int)((loaded - x0) % kStages));
            if (++loaded < x1) step(a, BM, ld);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        const uint32_t kb = sm0 + (uint32_t)st * 2u * TB, vb = kb + TB;
        const int R = min(BM, (int)min((long long)BM, (long long)cur.q.n * a.G - (long long)cur.rb * BM));
        if (fresh) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = row0 + 8 * e, rr = cur.rb * BM + r;
                const int tok = rr / a.G, head = cur.h * a.G + rr % a.G;
                const uint16_t* src = a.q + (cur.q.start + tok) * a.ldq + (long long)head * D + 2 * u;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    qf[kk][e] = r < R ? *reinterpret_cast<const uint32_t*>(src + 16 * kk) : 0u;
                    qf[kk][2 + e] = r < R ? *reinterpret_cast<const uint32_t*>(src + 16 * kk + 8) : 0u;
                }
                m[e] = -INFINITY;
                l[e] = 0.f;
            }
#pragma unroll
            for (int dn = 0; dn < DN; ++dn) o[dn][0] = o[dn][1] = o[dn][2] = o[dn][3] = 0.f;
            fresh = false;
        }
        const int key0 = cur.tile * kKeys;
        const bool tail = key0 + kKeys > cur.q.ctx;  // the tile holds new rows, or the end
        const int tok[2] = {(cur.rb * BM + row0) / a.G, (cur.rb * BM + row0 + 8) / a.G};
        if (tail) {
            // A new row's value reaches only the rows that see it: infinities
            // and NaN of the tile are added to those by hand and then
            // cleared, as their products with a zero probability would be NaN.
            bool odd = false;
            for (int y = tid; y < kKeys * NCH; y += kThreads) {
                const int r = y / NCH, c = y % NCH;
                if (key0 + r < cur.q.ctx) continue;
                const uint4 w = *reinterpret_cast<const uint4*>(smem + (vb - sm0) + swz<D>(r, c));
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) odd |= !finite16((uint16_t)ws[e]) || !finite16((uint16_t)(ws[e] >> 16));
            }
            if (__syncthreads_or(odd)) {
                for (int j = 0; j < KW; ++j) {
                    const int r = wn * KW + j, nj = key0 + r - cur.q.ctx;
                    if (nj < 0 || nj >= cur.q.n) continue;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (row0 + 8 * e >= R || !sees(a, cur.q.start, tok[e], nj)) continue;
#pragma unroll
                        for (int dn = 0; dn < DN; ++dn) {
                            const uint32_t w = *reinterpret_cast<const uint32_t*>(smem + (vb - sm0) + swz<D>(r, dn) + 4 * u);
                            const uint16_t lo = (uint16_t)w, hi = (uint16_t)(w >> 16);
                            if (!finite16(lo)) o[dn][2 * e] += __half2float(__ushort_as_half(lo));
                            if (!finite16(hi)) o[dn][2 * e + 1] += __half2float(__ushort_as_half(hi));
                        }
                    }
                }
                __syncthreads();
                for (int y = tid; y < kKeys * D; y += kThreads) {
                    const int r = y / D, d = y % D;
                    if (key0 + r < cur.q.ctx) continue;
                    uint16_t* v = reinterpret_cast<uint16_t*>(smem + (vb - sm0) + swz<D>(r, d / 8)) + d % 8;
                    if (!finite16(*v)) *v = 0;
                }
                __syncthreads();
            }
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
                ldsm4(kb + swz<D>(wn * KW + nt * 8 + (lane & 7), 2 * kk + (lane >> 3)), b);
                mma(sc[nt], qf[kk], b[0], b[1]);
                mma(sc[nt], qf[kk + 1], b[2], b[3]);
            }
        }
        if (tail) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int nj = key0 + wn * KW + nt * 8 + 2 * u + (e & 1) - cur.q.ctx;
                    if (nj >= 0 && (nj >= cur.q.n || row0 + 8 * (e >> 1) >= R || !sees(a, cur.q.start, tok[e >> 1], nj)))
                        sc[nt][e] = -INFINITY;
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
            // a negative scale turns the order round: the greatest of s c
            // then comes from the smallest s; c > 0 is checked on the host
            const float mn = fmaxf(m[e], mx * a.c);
            const float ms = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[e] - ms);
            m[e] = mn;
            float sum = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float p0 = exp2f(fmaf(sc[nt][2 * e], a.c, kShift - ms));
                const float p1 = exp2f(fmaf(sc[nt][2 * e + 1], a.c, kShift - ms));
                sum += p0 + p1;
                pa[nt >> 1][(nt & 1) * 2 + e] = pack2(p0, p1);
            }
            l[e] = fmaf(l[e], f, sum);
#pragma unroll
            for (int dn = 0; dn < DN; ++dn) {
                o[dn][2 * e] *= f;
                o[dn][2 * e + 1] *= f;
            }
        }
#pragma unroll
        for (int kj = 0; kj < KW / 16; ++kj)
#pragma unroll
            for (int dn = 0; dn < DN; dn += 2) {
                uint32_t b[4];
                ldsm4_t(vb + swz<D>(wn * KW + kj * 16 + (lane & 15), dn + (lane >> 4)), b);
                mma(o[dn], pa[kj], b[0], b[1]);
                mma(o[dn + 1], pa[kj], b[2], b[3]);
            }

        const bool job_end = cur.tile + 1 == cur.tiles;
        if (job_end || x + 1 == x1) {
            // the row sums over the quad's columns, then over the WN warps
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            }
            if constexpr (WN > 1) {
                // this tile's stage is free until the next iteration's barrier:
                // the warps' outputs meet there, [WN][BM][D] fp32 (at most 32 KB)
                static_assert((size_t)WN * BM * D * 4 <= 2 * TB, "joining space");
                if (u == 0) {
                    ml_s[warp][g] = make_float2(m[0], l[0]);
                    ml_s[warp][g + 8] = make_float2(m[1], l[1]);
                }
                __syncthreads();
                float* ob = reinterpret_cast<float*>(smem + (kb - sm0));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = g + 8 * e;
                    float mm = -INFINITY, ls = 0.f;
#pragma unroll
                    for (int i = 0; i < WN; ++i) mm = fmaxf(mm, ml_s[wm * WN + i][r].x);
                    const float ms = mm == -INFINITY ? 0.f : mm;
#pragma unroll
                    for (int i = 0; i < WN; ++i) ls = fmaf(ml_s[wm * WN + i][r].y, exp2f(ml_s[wm * WN + i][r].x - ms), ls);
                    const float f = exp2f(m[e] - ms);
                    float* dst = ob + ((size_t)wn * BM + wm * 16 + r) * D + 2 * u;
#pragma unroll
                    for (int dn = 0; dn < DN; ++dn)
                        *reinterpret_cast<float2*>(dst + 8 * dn) = make_float2(o[dn][2 * e] * f, o[dn][2 * e + 1] * f);
                    m[e] = mm;
                    l[e] = ls;
                }
                __syncthreads();
                if (wn == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int dn = 0; dn < DN; ++dn) {
                            float2 t = make_float2(0.f, 0.f);
#pragma unroll
                            for (int i = 0; i < WN; ++i) {
                                const float2 v = *reinterpret_cast<const float2*>(
                                    ob + ((size_t)i * BM + wm * 16 + g + 8 * e) * D + 2 * u + 8 * dn);
                                t.x += v.x;
                                t.y += v.y;
                            }
                            o[dn][2 * e] = t.x;
                            o[dn][2 * e + 1] = t.y;
                        }
                }
            }
            if (wn == 0) {
                if (begun && job_end) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = row0 + 8 * e, rr = cur.rb * BM + r;
                        if (r >= R) continue;
                        const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
                        uint16_t* dst = a.out + (long long)(cur.q.start + rr / a.G) * a.ldo +
                                        (long long)(cur.h * a.G + rr % a.G) * D + 2 * u;
#pragma unroll
                        for (int dn = 0; dn < DN; ++dn)
                            *reinterpret_cast<uint32_t*>(dst + 8 * dn) = pack2(o[dn][2 * e] * inv, o[dn][2 * e + 1] * inv);
                    }
                } else {
                    const int slot = 2 * blockIdx.x + (begun ? 1 : 0);
                    float* po = part_o<D>(a, slot);
                    float2* pm = part_ml<D>(a, slot);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = row0 + 8 * e;
                        if (r >= R) continue;
                        if (u == 0) pm[r] = make_float2(m[e], l[e]);
#pragma unroll
                        for (int dn = 0; dn < DN; ++dn)
                            *reinterpret_cast<float2*>(po + (size_t)r * D + 8 * dn + 2 * u) =
                                make_float2(o[dn][2 * e], o[dn][2 * e + 1]);
                    }
                }
            }
            fresh = true;
            begun = true;
        }
        if (x + 1 < x1) step(a, BM, cur);
    }
}

// Joins the parts of the jobs that several CTAs shared.  Block b looks at the
// border between CTAs b and b + 1; it works if that is the first border inside
// its job.  A warp per row; grid.y covers the rows.
template <int D>
__global__ void __launch_bounds__(256) tree_join_kernel(const Args a, int BM) {
    __shared__ long long sums[256];
    const long long line = line_scan(a, BM, sums, 256);
    const int b = blockIdx.x;
    const long long x = line * (b + 1) / a.ctas, xb = line * b / a.ctas;
    if (x <= xb || x >= line) return;  // CTA b has no tiles, or the line ends
    const Place p = line_find(a, BM, sums, 256, x);
    const long long j0 = x - p.tile, j1 = j0 + p.tiles;  // the job's tiles
    if (p.tile == 0 || xb > j0) return;                   // no job across this border, or an earlier border's
    const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const long long rr = (long long)p.rb * BM + r;
    if (r >= BM || rr >= (long long)p.q.n * a.G) return;
    // CTA b has the job's beginning (slot 2 b + 1), later CTAs their slot 2 c
    constexpr int E = D / 32;
    float m = -INFINITY;
    int last = b;
    for (int c = b; c < a.ctas && line * c / a.ctas < j1; ++c) {
        if (line * (c + 1) / a.ctas == line * c / a.ctas) continue;
        m = fmaxf(m, part_ml<D>(a, 2 * c + (c == b))[r].x);
        last = c;
    }
    const float ms = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[E] = {};
    for (int c = b; c <= last; ++c) {
        if (line * (c + 1) / a.ctas == line * c / a.ctas) continue;
        const int slot = 2 * c + (c == b);
        const float2 t = part_ml<D>(a, slot)[r];
        const float f = exp2f(t.x - ms);
        l = fmaf(t.y, f, l);
        const float* src = part_o<D>(a, slot) + (size_t)r * D + E * lane;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(src[e], f, o[e]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* dst = a.out + (p.q.start + rr / a.G) * a.ldo + (p.h * a.G + rr % a.G) * D + E * lane;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack2(o[e] * inv, o[e + 1] * inv);
}

template <int D>
size_t workspace_bytes() {
    return (size_t)2 * kMaxCtas * kMaxRows * (D + 2) * 4;
}

template <int D, int WM>
cudaError_t launch(Args& a, int sms, cudaStream_t s) {
    static std::atomic<int> marks[64];
    cudaError_t e = q4i::ensure_smem_attr(reinterpret_cast<const void*>(tree_attn_kernel<D, WM>), marks, (int)attn_smem<D>());
    if (e != cudaSuccess) return e;
    a.ctas = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
    tree_attn_kernel<D, WM><<<a.ctas, kThreads, attn_smem<D>(), s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    tree_join_kernel<D><<<dim3(a.ctas - 1, 2 * WM), 256, 0, s>>>(a, 16 * WM);
    return cudaGetLastError();
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
    if (!d.q || !d.out || !d.workspace) return fail(Q4_ERR_INVALID_ARG, "NULL pointer argument");
    if (d.n_q_heads < d.cache.n_kv_heads || d.n_q_heads % d.cache.n_kv_heads)
        return fail(Q4_ERR_INVALID_ARG, "n_q_heads=%d is not a multiple of n_kv_heads=%d", d.n_q_heads, d.cache.n_kv_heads);
    if ((long long)d.n_q_heads * D > (1 << 24)) return fail(Q4_ERR_UNSUPPORTED, "%d query heads", d.n_q_heads);
    const int G = d.n_q_heads / d.cache.n_kv_heads;
    if ((long long)d.rows * G > (1ll << 30)) return fail(Q4_ERR_UNSUPPORTED, "rows=%d x %d query heads per kv head", d.rows, G);
    if (d.mask && d.mask_words < 1) return fail(Q4_ERR_INVALID_ARG, "mask_words=%d", d.mask_words);
    a.c = (d.scale == 0.f ? 1.f / sqrtf((float)D) : d.scale) * 1.4426950408889634f;
    if (!(a.c >= 1e-30f && a.c <= 1e30f)) return fail(Q4_ERR_INVALID_ARG, "scale=%g", d.scale);
    if (reinterpret_cast<uintptr_t>(d.mask) & 3u) return fail(Q4_ERR_MISALIGNED, "mask must be 4-byte aligned");
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
    a.part = static_cast<float*>(d.workspace);
    // rows per job: the average sequence's, by 16, 32 or 64
    const long long avg = ((long long)d.rows * G + d.cache.n_seqs - 1) / d.cache.n_seqs;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (D == 128)
        e = avg <= 16 ? q4x::launch<128, 1>(a, dev->sms, s) : avg <= 32 ? q4x::launch<128, 2>(a, dev->sms, s) : q4x::launch<128, 4>(a, dev->sms, s);
    else
        e = avg <= 16 ? q4x::launch<64, 1>(a, dev->sms, s) : avg <= 32 ? q4x::launch<64, 2>(a, dev->sms, s) : q4x::launch<64, 4>(a, dev->sms, s);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "q4_tree_attention launch");
}
