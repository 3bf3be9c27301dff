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
#include "q4_tc.cuh"

namespace q4x {

using q4p::Seq;
using q4p::View;

constexpr int kKeys = 64;      // positions per tile
constexpr int kThreads = 128;  // 4 warps: WM of them along the rows, 4 / WM along the positions
constexpr int kStages = 3;
constexpr int kMaxRows = 64;   // rows of a job
constexpr int kMaxCtas = 512;
constexpr int kTcRows = 256, kMaxTcCtas = 160;
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
    int ctas;    // CTAs that share the line
    int BM, KT;  // rows of a job, positions of a tile
    float* po;   // workspace: [2 CTAs][BM][D] outputs
    float2* pml; // [2 CTAs][BM] (m, l)
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
    const int last = min(((rb + 1) * a.BM - 1) / a.G, q.n - 1);
    const int keys = q.ctx + (a.mask ? q.n : last + 1);
    return (keys + a.KT - 1) / a.KT;
}

// Tiles of one head of a sequence (all row blocks).
__device__ __forceinline__ long long head_tiles(const Args& a, const Seq& q) {
    if (q.n <= 0) return 0;
    const int blocks = (int)(((long long)q.n * a.G + a.BM - 1) / a.BM);
    if (a.mask || blocks == 1) return (long long)blocks * block_tiles(a, q, blocks - 1);
    long long t = 0;
    for (int b = 0; b < blocks; ++b) t += block_tiles(a, q, b);
    return t;
}

// A place in the line of tiles.
struct Place {
    int s, h, rb, tile, tiles;  // tile of the job's `tiles`
    Seq q;
};

// The line's length; `sums` gets the threads' running shares: each thread adds
// up a contiguous share of the sequences.
__device__ __forceinline__ long long line_scan(const Args& a, long long* sums, int threads) {
    const int per = (a.w.S + threads - 1) / threads;
    const int lo = min(a.w.S, (int)threadIdx.x * per), hi = min(a.w.S, lo + per);
    long long t = 0;
    for (int s = lo; s < hi; ++s) {
        bool bad;
        const Seq q = q4p::seq_of(a.w, s, bad);
        if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.w.err, q4d::kErrDeviceCheck);
        t += head_tiles(a, q);
    }
    t *= a.w.H;
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

// A CTA's share of the line: as even as whole tiles allow.
__device__ __forceinline__ long long line_share(const Args& a, long long line) {
    if (line < (1ll << 31)) return ((unsigned)line + (unsigned)a.ctas - 1) / (unsigned)a.ctas;
    return (line + a.ctas - 1) / a.ctas;
}

// Place of tile x (x < the line's length).
__device__ __forceinline__ Place line_find(const Args& a, const long long* sums, int threads, long long x) {
    int lo = 0, hi = threads - 1;  // first thread whose running sum exceeds x
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
        head = head_tiles(a, p.q);
        if (x < head * a.w.H) break;
        x -= head * a.w.H;
    }
    p.h = x < (1ll << 31) && head < (1ll << 31) ? (int)((unsigned)x / (unsigned)head) : (int)(x / head);
    x -= p.h * head;
    for (p.rb = 0;; ++p.rb) {
        p.tiles = block_tiles(a, p.q, p.rb);
        if (x < p.tiles) break;
        x -= p.tiles;
    }
    p.tile = (int)x;
    return p;
}

// The next job's first tile (there is one).
__device__ __forceinline__ void next_job(const Args& a, Place& p) {
    p.tile = 0;
    if ((long long)++p.rb * a.BM >= (long long)p.q.n * a.G) {
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
}

// The next tile's place (there is one).
__device__ __forceinline__ void step(const Args& a, Place& p) {
    if (++p.tile == p.tiles) next_job(a, p);
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
    const long long line = line_scan(a, sums, kThreads);
    const long long share = line_share(a, line), x0 = share * blockIdx.x, x1 = min(line, x0 + share);
    q4d::pdl_trigger();  // the joining kernel's blocks may start; they wait for this grid's end
    if (x0 >= x1) return;
    Place cur = line_find(a, sums, kThreads, x0);
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
            if (++loaded < x1) step(a, ld);
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
            if (++loaded < x1) step(a, ld);
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
                    float2* pm = part_ml(a, slot);
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
        if (x + 1 < x1) step(a, cur);
    }
}

// Joins the parts of the jobs that several CTAs shared.  Block b looks at the
// border between CTAs b and b + 1; it works if that is the first border inside
// its job.  A warp per row; a lane holds (m, l) of every 32nd part, so the
// loads are in flight together.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const Args a) {
    __shared__ long long sums[kJoinThreads];
    const long long line = line_scan(a, sums, kJoinThreads);
    const long long share = line_share(a, line);
    const int b = blockIdx.x;
    const long long xb = share * b, x = xb + share;
    Place p;
    long long j0 = 0;  // the job's first tile
    bool work = x < line;
    if (work) {
        p = line_find(a, sums, kJoinThreads, x);
        j0 = x - p.tile;
        work = p.tile != 0 && xb <= j0;  // a job across this border, and no earlier border in it
    }
    // the parts are written (and no grid that follows this one starts before
    // the attention's end, so blocks without work wait as well)
    q4d::pdl_wait();
    if (!work) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = (int)min((long long)a.BM, (long long)p.q.n * a.G - (long long)p.rb * a.BM);
    // CTA b has the job's beginning (slot 2 b + 1), later CTAs their slot 2 c
    const int last = (int)((j0 + p.tiles - 1) / share);  // CTA of the job's last tile
    const auto slot_of = [&](int c) { return 2 * c + (c == b); };
    for (int r = blockIdx.y * (kJoinThreads / 32) + warp; r < rows; r += gridDim.y * (kJoinThreads / 32)) {
        const long long rr = (long long)p.rb * a.BM + r;
        float m = -INFINITY;
        for (int c = b + lane; c <= last; c += 32) m = fmaxf(m, part_ml(a, slot_of(c))[r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ms = m == -INFINITY ? 0.f : m;
        constexpr int E = D / 32;
        float l = 0.f, o[E] = {};
        for (int c0 = b; c0 <= last; c0 += 32) {
            float f = 0.f;
            if (c0 + lane <= last) {
                const float2 t = part_ml(a, slot_of(c0 + lane))[r];
                f = exp2f(t.x - ms);
                l = fmaf(t.y, f, l);
            }
            const int n = min(32, last - c0 + 1);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float fi = __shfl_sync(0xffffffffu, f, i);
                const float* src = part_o<D>(a, slot_of(c0 + i)) + (size_t)r * D + E * lane;
                float v[E];
                if constexpr (E == 4) {
                    const float4 t = *reinterpret_cast<const float4*>(src);
                    v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
                } else {
                    const float2 t = *reinterpret_cast<const float2*>(src);
                    v[0] = t.x, v[1] = t.y;
                }
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(v[e], fi, o[e]);
            }
        }
#pragma unroll
        for (int o2 = 16; o2 > 0; o2 >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o2);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* dst = a.out + (p.q.start + rr / a.G) * a.ldo + (p.h * a.G + rr % a.G) * D + E * lane;
        uint32_t w[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2) w[e / 2] = pack2(o[e] * inv, o[e + 1] * inv);
        if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(dst) = w[0];
    }
}

// The parts' places in the workspace.
template <int D>
size_t parts_bytes(int ctas, int BM) {
    return (size_t)2 * ctas * BM * (D + 2) * 4;
}
template <int D>
void place_parts(Args& a, void* workspace) {
    a.po = static_cast<float*>(workspace);
    a.pml = reinterpret_cast<float2*>(a.po + (size_t)2 * a.ctas * a.BM * D);
}
template <int D>
size_t workspace_bytes() {
    const size_t x = parts_bytes<D>(kMaxCtas, kMaxRows), y = parts_bytes<D>(kMaxTcCtas, kTcRows);
    return x > y ? x : y;
}

// The joining kernel starts while the attention's last CTAs run (programmatic
// dependent launch) and has its place in the line by the time they end.
template <int D>
cudaError_t launch_join(const Args& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.ctas - 1, (unsigned)(a.BM <= 32 ? 1 : a.BM <= 64 ? 2 : 4));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<D>, a);
}

template <int D, int WM>
cudaError_t launch(Args& a, void* workspace, int sms, cudaStream_t s) {
    static std::atomic<int> marks[64];
    cudaError_t e = q4i::ensure_smem_attr(reinterpret_cast<const void*>(tree_attn_kernel<D, WM>), marks, (int)attn_smem<D>());
    if (e != cudaSuccess) return e;
    a.ctas = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
    a.BM = 16 * WM;
    a.KT = kKeys;
    place_parts<D>(a, workspace);
    tree_attn_kernel<D, WM><<<a.ctas, kThreads, attn_smem<D>(), s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_join<D>(a, s);
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
// the tensor cores work for the other stream, and one thread issues, in order,
//   S(0) | P V(0) S(1) | P V(1) S(2) | ...
// S = Q K^T (128 x 128, Q and K from shared memory) and O += P V (P, fp16,
// from tensor memory over the scores it came from, V read MN-major).  MMAs of
// one thread run in order, so S(k + 1) may overwrite what P V(k) reads, and
// the commit behind S(k + 1) tells the softmax that O holds step k's product.
// Tensor memory (512 columns): S 0 and 1 (128 each), O 0 and 1.
// The reference maximum of a row moves only when its maximum exceeds it by
// more than 8 (a factor 2^8); then O and l are rescaled.  With kTcShift P
// reaches 2^15 and keeps 11 bits down to 2^-29 of the row's greatest at worst.
// Key and value tiles come by TMA as boxes of `box` rows (the greatest power
// of two, 8 .. 128, that divides the page): a box lies in one page.  A page
// that does not exist is read outside the map, where TMA fills in zeros.
constexpr int kTcKeys = 128;
constexpr int kTcThreads = 384;  // warps 0..3, 4..7: softmax of stream 0, 1; 8: keys, 9: values, 10, 11: MMA of stream 0, 1
constexpr float kTcShift = 7.f;

template <int D>
struct TcShape {
    static constexpr uint32_t kTile = 128 * D * 2;      // a 128 x D fp16 tile: D / 64 swizzled slabs of 16 KB
    static constexpr int kStages = D == 128 ? 2 : 4;    // of keys, and of values
    static constexpr size_t kSmem = 1024 + (2 + 2 * kStages) * (size_t)kTile + 512;
};

struct TcBars {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t v_clean[4];  // two row streams: stream 0 has cleared what stream 1's products must not meet
    uint64_t s_full[2], p_full[2], q_full, o_full, x_full, x_empty, drain[2];
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

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
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

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

struct TcArgs {
    Args a;
    int box;            // rows per TMA box
    int zero_row;       // a row outside the maps
};

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_attn_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const TcArgs t) {
    using Sh = TcShape<D>;
    constexpr uint32_t kTile = Sh::kTile;
    constexpr int NST = Sh::kStages, SLABS = D / 64;
    constexpr uint32_t kColS = 0, kColO = 256;
    const Args& a = t.a;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ long long sums[kTcThreads];
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
            q4d::mbar_init(q4d::smem_addr(&B.p_full[i]), 4);
            q4d::mbar_init(q4d::smem_addr(&B.drain[i]), 1);
            B.odd[i] = 0;
        }
        q4d::mbar_init(q4d::smem_addr(&B.q_full), 8);
        q4d::mbar_init(q4d::smem_addr(&B.o_full), 2);
        q4d::mbar_init(q4d::smem_addr(&B.x_full), 4);
        q4d::mbar_init(q4d::smem_addr(&B.x_empty), 4);
        B.abort = 0;
        q4d::fence_mbar_init();
    }
    if (warp == 11) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         q4d::smem_addr(&B.tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const long long line = line_scan(a, sums, kTcThreads);
    const long long share = line_share(a, line), x0 = share * blockIdx.x, x1 = min(line, x0 + share);
    q4t::fence_before();
    __syncthreads();
    q4t::fence_after();
    q4d::pdl_trigger();
    const uint32_t tmem = B.tmem_base;

    if (x0 < x1) {
        // Every role walks the same segments: the part of each job that lies
        // in x0 .. x1 - 1.
        Place p = line_find(a, sums, kTcThreads, x0);
        long long x = x0;
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
            while (x < x1 && ok) {
                const int T = (int)min((long long)(p.tiles - p.tile), x1 - x);
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
                x += T;
                if (x < x1 && ok) next_job(a, p);
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
            uint32_t n_p = 0;    // p_full phases passed
            uint32_t cleans = 0;  // parity of the v_clean phases passed, a bit per stage
            while (x < x1 && ok) {
                const int T = (int)min((long long)(p.tiles - p.tile), x1 - x);
                const bool two = (long long)p.q.n * a.G - (long long)p.rb * a.BM > 128;
                const int steps = two ? T : (T - i + 1) / 2;
                const uint64_t ad = dq + (uint64_t)((two ? i : 0) * (kTile / 16));
                const auto tile_of = [&](int k) { return tiles0 + (two ? k : 2 * k + i); };
                // S of step k (its keys have landed)
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
                        if (!two) q4t::commit(q4d::smem_addr(&B.k_empty[st]));  // the other stream's share
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
                         tc_wait(B, B.p_full[i], n_p & 1, err);
                    if (ok && two && i == 1 && (p.tile + k + 1) * kTcKeys > p.q.ctx + (a.mask ? 0 : p.rb * a.BM / a.G + 1)) {
                        ok = tc_wait(B, B.v_clean[st], cleans >> st & 1, err);
                        cleans ^= 1u << st;
                    }
                    if (!ok) break;
                    ++n_p;
                    q4t::fence_after();
                    const uint64_t bd = dv + (uint64_t)(st * (kTile / 16));
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < kTcKeys / 16; ++kk)
                            q4t::mma_ts(od, sd + 8 * kk, bd + (uint64_t)(kk * 2048 / 16), id_o, (k > 0 || kk > 0) ? 1u : 0u);
                    }
                    __syncwarp();
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
                x += T;
                if (x < x1 && ok) next_job(a, p);
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
            uint32_t n_s = 0;      // s_full phases passed
            uint32_t joins = 0;    // joined segments so far
            bool ok = true;
            while (x < x1) {
                const int T = (int)min((long long)(p.tiles - p.tile), x1 - x);
                const int R = (int)min((long long)a.BM, (long long)p.q.n * a.G - (long long)p.rb * a.BM);
                const bool two = R > 128;
                const int r = (two ? 128 * i : 0) + row;  // row of the job
                const bool live = r < R;  // the others run along with queries of zero
                const int rr = p.rb * a.BM + (live ? r : 0), tok = rr / a.G;
                const size_t q_row = (size_t)(p.q.start + tok), q_col = (size_t)(p.h * a.G + rr % a.G) * D;
                const int steps = two ? T : (T - i + 1) / 2;
                const bool join = !two && T > 1;
                // new rows that every row of the job sees
                const int all_see = a.mask ? 0 : p.rb * a.BM / a.G + 1;
                // the row's query into the stream's tile (both streams share stream
                // 0's), once every warp of stream 0 has read the last join's part there
                if (joins > 0) ok = __all_sync(0xffffffffu, ok && tc_wait(B, B.x_empty, (joins - 1) & 1, err));
                if (!ok) break;
                if (two || i == 0) {
                    uint8_t* dst = q_s + (two ? i : 0) * kTile;
                    const uint4* src = reinterpret_cast<const uint4*>(a.q + q_row * a.ldq + q_col);
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 w = live ? src[c] : make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + sw_off(row, c & 7)) = w;
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.q_full));

                float m = -INFINITY, l = 0.f;
                for (int j = 0; j < steps; ++j) {
                    const int tj = two ? j : 2 * j + i;  // tile of the segment
                    const int key0 = (p.tile + tj) * kTcKeys;
                    const uint32_t kt = tiles0 + tj, st = kt % NST;
                    ok = __all_sync(0xffffffffu, tc_wait(B, B.s_full[i], n_s & 1, err));
                    if (!ok) break;
                    ++n_s;
                    q4t::fence_after();
                    // The row in halves, so that it fits the registers: the
                    // second one's maximum, the first one's, P of the first
                    // (over scores that are read), the second one again.
                    // Some row of the job does not see some position of the tile:
                    const bool tail = key0 + kTcKeys > p.q.ctx + all_see;
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
                    load_half(1);
                    max_half();
                    load_half(0);
                    max_half();
                    const float mx = fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * a.c;
                    float corr = 1.f;
                    if (mx > m + 8.f) {
                        corr = m == -INFINITY ? 1.f : ex2(m - mx);  // nothing seen yet: O and l are zero
                        m = mx;
                    }
                    const float sub = kTcShift - (m == -INFINITY ? 0.f : m);
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
                    exp_half(0);
                    load_half(1);
                    exp_half(1);
                    l = fmaf(l, corr, (sum.x + sum2.x) + (sum.y + sum2.y));
                    if (j > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll
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
                        if (nj >= 0) {
                            uint8_t* vt = v_s + st * kTile;
                            bool found = false;
#pragma unroll
                            for (int c = 0; c < D / 8; ++c) {
                                uint4* at = reinterpret_cast<uint4*>(vt + (c >> 3) * 16384 + sw_off(row, c & 7));
                                if (nj >= p.q.n) {
                                    *at = make_uint4(0, 0, 0, 0);
                                    continue;
                                }
                                uint4 w = *at;
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
                            if (found) B.odd[seg & 1] = (int)seg + 1;
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        if (two) {
                            __syncwarp();
                            if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.v_clean[st]));
                        }
                    }
                    q4t::st_wait();
                    q4t::fence_before();
                    __syncwarp();
                    if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.p_full[i]));
                }
                if (!ok) break;
                ok = __all_sync(0xffffffffu, tc_wait(B, B.o_full, seg & 1, err));
                if (!ok) break;
                q4t::fence_after();
                const bool job_begin = p.tile == 0, job_end = p.tile + T == p.tiles;
                const bool odd = B.odd[seg & 1] == (int)seg + 1;
                if (join && i == 1) {
                    // stream 1's part, fp32, into the query tiles' place (16-byte
                    // chunks of a row spread over the banks); (m, l) into sums, done with
                    float* ob = reinterpret_cast<float*>(q_s);
                    constexpr int NC = D / 4;
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t o[16];
                        q4t::ld16(to + c0, o);
                        q4t::ld_wait();
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            *reinterpret_cast<uint4*>(ob + row * D + (((c0 / 4 + c) ^ (row & (NC - 1))) * 4)) =
                                make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                    }
                    sums[2 * row] = __float_as_int(m);
                    sums[2 * row + 1] = __float_as_int(l);
                    __syncwarp();
                    if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.x_full));
                } else if (two || i == 0) {
                    float f0 = 1.f, f1 = 0.f;
                    if (join) {
                        ok = __all_sync(0xffffffffu, tc_wait(B, B.x_full, joins & 1, err));
                        if (!ok) break;
                        const float m1 = __int_as_float((int)sums[2 * row]), l1 = __int_as_float((int)sums[2 * row + 1]);
                        const float mm = fmaxf(m, m1), ms = mm == -INFINITY ? 0.f : mm;
                        f0 = ex2(m - ms);
                        f1 = ex2(m1 - ms);
                        l = l * f0 + l1 * f1;
                        m = mm;
                    }
                    const bool whole = job_begin && job_end;
                    const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
                    const int slot = 2 * blockIdx.x + (job_begin ? 1 : 0);
                    const float* ob = reinterpret_cast<const float*>(q_s);
                    constexpr int NC = D / 4;
                    if (!whole && live) part_ml(a, slot)[r] = make_float2(m, l);
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t w[16];
                        float o[16];
                        q4t::ld16(to + c0, w);
                        q4t::ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(w[e]);
                        if (join) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const float4 v = *reinterpret_cast<const float4*>(
                                    ob + row * D + (((c0 / 4 + c) ^ (row & (NC - 1))) * 4));
                                o[4 * c] = fmaf(v.x, f1, o[4 * c] * f0);
                                o[4 * c + 1] = fmaf(v.y, f1, o[4 * c + 1] * f0);
                                o[4 * c + 2] = fmaf(v.z, f1, o[4 * c + 2] * f0);
                                o[4 * c + 3] = fmaf(v.w, f1, o[4 * c + 3] * f0);
                            }
                        }
                        if (odd && live) {
                            const int n0 = max(0, p.tile * kTcKeys - p.q.ctx), n1 = min(p.q.n, (p.tile + T) * kTcKeys - p.q.ctx);
                            for (int nj = n0; nj < n1; ++nj) {
                                if (!sees(a, p.q.start, tok, nj)) continue;
                                const long long at = q4p::row_at(a.w, p.s, p.q.ctx + nj, p.h, D);
                                if (at < 0) continue;
                                for (int e = 0; e < 16; ++e) {
                                    const uint16_t v = a.w.v[at + c0 + e];
                                    if (!finite16(v)) o[e] += __half2float(__ushort_as_half(v));
                                }
                            }
                        }
                        if (!live) continue;
                        if (whole) {
                            uint32_t y[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = pack2(o[2 * e] * inv, o[2 * e + 1] * inv);
                            uint4* dst = reinterpret_cast<uint4*>(a.out + q_row * a.ldo + q_col + c0);
                            dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
                            dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
                        } else {
                            float4* dst = reinterpret_cast<float4*>(part_o<D>(a, slot) + (size_t)r * D + c0);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                    }
                    if (join) {
                        __syncwarp();
                        if (lane == 0) q4d::mbar_arrive(q4d::smem_addr(&B.x_empty));
                    }
                }
                q4t::fence_before();  // O is read before the next segment's queries release its MMAs
                if (join) ++joins;
                tiles0 += T;
                ++seg;
                x += T;
                if (x < x1) next_job(a, p);
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
    TcArgs t;
    a.ctas = sms < kMaxTcCtas ? sms : kMaxTcCtas;
    a.BM = kTcRows;
    a.KT = kTcKeys;
    place_parts<D>(a, workspace);
    t.a = a;
    t.box = box;
    const uint64_t rows = (uint64_t)c.n_pages * c.n_kv_heads * c.page_size;
    t.zero_row = (int)rows;
    CUtensorMap tmK, tmV;
    q4_status st;
    if ((st = q4i::make_map(&tmK, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, c.k, D, rows, D * 2, 64, (uint32_t)box, CU_TENSOR_MAP_SWIZZLE_128B)) != Q4_OK)
        return st;
    if ((st = q4i::make_map(&tmV, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, c.v, D, rows, D * 2, 64, (uint32_t)box, CU_TENSOR_MAP_SWIZZLE_128B)) != Q4_OK)
        return st;
    static std::atomic<int> marks[64];
    cudaError_t e = q4i::ensure_smem_attr(reinterpret_cast<const void*>(tree_attn_tc_kernel<D>), marks, (int)TcShape<D>::kSmem);
    if (e == cudaSuccess) {
        tree_attn_tc_kernel<D><<<a.ctas, kTcThreads, TcShape<D>::kSmem, s>>>(tmK, tmV, t);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = launch_join<D>(a, s);
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
    // rows per job: the average sequence's, by 16, 32 or 64
    const long long avg = ((long long)d.rows * G + d.cache.n_seqs - 1) / d.cache.n_seqs;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int box = d.cache.page_size % 128 == 0 ? 128 : d.cache.page_size & -d.cache.page_size;
    const long long pool_rows = (long long)d.cache.n_pages * d.cache.n_kv_heads * d.cache.page_size;
    if (avg > 32 && box >= 8 && pool_rows < (1ll << 31) - 1)
        return D == 128 ? q4x::launch_tc<128>(a, d.cache, d.workspace, dev->sms, box, s)
                        : q4x::launch_tc<64>(a, d.cache, d.workspace, dev->sms, box, s);
    cudaError_t e;
    if (D == 128)
        e = avg <= 16 ? q4x::launch<128, 1>(a, d.workspace, dev->sms, s) : avg <= 32 ? q4x::launch<128, 2>(a, d.workspace, dev->sms, s) : q4x::launch<128, 4>(a, d.workspace, dev->sms, s);
    else
        e = avg <= 16 ? q4x::launch<64, 1>(a, d.workspace, dev->sms, s) : avg <= 32 ? q4x::launch<64, 2>(a, d.workspace, dev->sms, s) : q4x::launch<64, 4>(a, d.workspace, dev->sms, s);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "q4_tree_attention launch");
}
