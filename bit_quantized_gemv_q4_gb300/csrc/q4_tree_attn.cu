// Attention over the paged fp16 cache (q4.h 7c): the tcgen05 kernel for many
// rows per kv head, and the call.  The mathematics, the schedule and the kernel
// for few rows stand in q4_tree_attn.cuh.
#include "q4_tree_attn.cuh"

namespace q4x {

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
                        add_odd<D, false>(a, done, T, tok, join ? D / 2 * i : 0, c1,
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
q4_status launch_tc(Args& a, const Pools& c, void* workspace, int sms, int box, cudaStream_t s) {
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
    const q4_status st = pool_maps<false>(&tmK, &tmV, c, (uint32_t)box);
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
    if ((st = q4x::attention_args(a, d.mask, d.mask_words, d.q, d.out, d.ldq, d.ldo, d.n_q_heads, d.cache.n_kv_heads, D, d.rows,
                                  d.scale, d.workspace, d.workspace_bytes)) != Q4_OK)
        return st;
    const DeviceInfo* dev = nullptr;
    if ((st = current_device(&dev)) != Q4_OK) return st;
    if (d.rows == 0) return Q4_OK;
    a.w.err = dev->err_word;
    a.ks = a.vs = nullptr;
    a.nb = 0;
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
    const long long avg = ((long long)d.rows * a.G + d.cache.n_seqs - 1) / d.cache.n_seqs;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const q4x::Pools pools = q4x::pools_of(d.cache);
    const char* what = "q4_tree_attention launch";
    // TMA boxes: the greatest power of two that divides a page, 8 at least (a
    // swizzled row group).  TMA / cp.async, us: 40 contexts up to 12000, pages of
    // 8 105 / 121, of 16 94 / 107, of 64 93 / 96; one user's 16000 positions 20 / 29.
    const int even = d.cache.page_size & -d.cache.page_size;
    const long long pool_rows = (long long)d.cache.n_pages * d.cache.n_kv_heads * d.cache.page_size;
    const bool tma = even >= 8 && pool_rows < (1ll << 31) - 1;
    const int ring_box = !tma ? 0 : even < q4x::kKeys ? even : q4x::kKeys;
    if (avg > 32 && tma) {
        const int box = even < q4x::kTcKeys ? even : q4x::kTcKeys;
        return D == 128 ? q4x::launch_tc<128>(a, pools, d.workspace, dev->sms, box, s)
                        : q4x::launch_tc<64>(a, pools, d.workspace, dev->sms, box, s);
    }
    if (D == 128)
        return avg <= 16   ? q4x::launch<128, 1>(a, pools, d.workspace, dev->sms, ring_box, s, what)
               : avg <= 32 ? q4x::launch<128, 2>(a, pools, d.workspace, dev->sms, ring_box, s, what)
                           : q4x::launch<128, 4>(a, pools, d.workspace, dev->sms, ring_box, s, what);
    return avg <= 16   ? q4x::launch<64, 1>(a, pools, d.workspace, dev->sms, ring_box, s, what)
           : avg <= 32 ? q4x::launch<64, 2>(a, pools, d.workspace, dev->sms, ring_box, s, what)
                       : q4x::launch<64, 4>(a, pools, d.workspace, dev->sms, ring_box, s, what);
}
