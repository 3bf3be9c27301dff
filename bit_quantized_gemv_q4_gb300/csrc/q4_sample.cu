// Sampling a token per row of logits with temperature, top-k, top-p and
// min-p from given random numbers (q4.h section 8; BaseRT: optimal LLM
// inference on Apple Silicon with native Metal, §3.3 lists sampling among the
// decode kernels).
//
// Mathematics: in the order (logit descending, index ascending) every limit
// keeps a beginning, and the choice itself is the first place where a running
// sum passes a bound.  So all steps are one search: the place where the count
// (top-k) or the weight (top-p, the choice) of everything before it reaches a
// target.  It goes digit by digit over an order-preserving 32-bit key of the
// logit, eight bits at a time: histogram the keys that share the digits found
// so far, walk the histogram from the top, descend.  Equal keys at the end
// have equal weights and go by index.
//
// Weights are integers, round(2^44 2^-t) with t = (max - l) log2(e) / T: their
// sums are exact in any order (2^19 of them stay below 2^63), so neither the
// atomics nor the split of the work can change a token, and a sum is as good
// as the weights.  A weight carries an error near 2^-31 of itself (t as a
// float pair, below), where a plain fp32 exponential's 2^-23 would move the
// borders of the tail's tokens, which are narrower than that.
#include <cuda_fp16.h>
#include <math.h>

#include "q4_device.cuh"
#include "q4_internal.h"

namespace q4s {

constexpr int kThreads = 1024;
constexpr int kMaxVocab = 1 << 19;
constexpr unsigned long long kOne = 1ull << 44;  // the weight of the greatest logit
constexpr uint32_t kLeast = 0x007FFFFFu;          // key of -inf: takes no part

struct Args {
    const void* logits;
    int vocab;
    long long ld;
    const float *temperature, *top_p, *min_p, *u;
    const int32_t* top_k;
    int32_t* tokens;
    float* probs;
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

// 2^-x for 0 <= x < 1 starts from a table of 2^(-j/64) in units of 2^-32.
struct Scale {
    float max, hi, lo;  // log2(e) / T = hi + lo
};

__device__ __forceinline__ unsigned long long weight_of(float l, const Scale& c, const uint32_t* pow64) {
    if (l == c.max) return kOne;
    // d + de = max - l exactly (the error of a difference is a float)
    const float d = c.max - l;
    const float b = d - c.max;
    const float de = (c.max - (d - b)) + (-l - b);
    // t + te = (d + de) (hi + lo) to about 2^-46 of it
    const float t = d * c.hi;
    if (!(t < 46.f)) return 0;
    const float te = fmaf(d, c.hi, -t) + fmaf(d, c.lo, de * c.hi);
    const float n = floorf(t);
    const float f = t - n;                    // exact
    const int j = (int)(f * 64.f);
    const float r = (f - (float)j * 0.015625f) + te;  // the first difference exact; |r| < 2^-6 + a little
    // 2^-r = 1 - y, y = r ln2 - (r ln2)^2 / 2 + (r ln2)^3 / 6 - ...; the fifth
    // term is below 2^-37
    const float z = r * 0.69314718f;
    const float y = z * (1.f - z * (0.5f - z * (0.16666667f - z * 0.041666668f)));
    const uint32_t p = pow64[j];
    const long long m = (long long)p - (long long)rintf((float)p * y);  // units of 2^-32, about 2^31 .. 2^32
    // 2^44 2^-n m 2^-32, rounded
    const int sh = 12 - (int)n;
    if (sh >= 0) return (unsigned long long)(m << sh);
    return (unsigned long long)((m + (1ll << (-sh - 1))) >> -sh);
}

template <bool HALF>
__device__ __forceinline__ float logit(const Args& a, const void* row, int i) {
    return HALF ? __half2float(static_cast<const __half*>(row)[i]) : static_cast<const float*>(row)[i];
}

struct Found {
    uint32_t key;            // the key at the target
    unsigned long long before;  // weight of the greater keys
    unsigned long long n_before, n_equal;  // their number, and that of the equal ones
};

// The first place, in descending key order, where the running count (BY_COUNT)
// or weight reaches `target` (>= 1, at most the total).
template <bool HALF, bool BY_COUNT>
__device__ Found search(const Args& a, const void* row, const Scale& c, const uint32_t* pow64,
                        unsigned long long target, unsigned long long* hw, unsigned int* hn, Found* out) {
    uint32_t prefix = 0;
    unsigned long long wb = 0, nb = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += blockDim.x) {
            hw[i] = 0;
            hn[i] = 0;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.vocab; i += blockDim.x) {
            const float l = logit<HALF>(a, row, i);
            const uint32_t k = key_of(l);
            if (k == kLeast || (shift < 24 && (k >> (shift + 8)) != (prefix >> (shift + 8)))) continue;
            const uint32_t b = (k >> shift) & 255u;
            atomicAdd(&hw[b], weight_of(key_value(k), c, pow64));
            atomicAdd(&hn[b], 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned long long w = wb, n = nb;
            int b = 255;
            int lastb = 255;
            for (; b >= 0; --b) {
                if (hn[b]) lastb = b;
                const unsigned long long run = BY_COUNT ? n + hn[b] : w + hw[b];
                if (run >= target) break;
                w += hw[b];
                n += hn[b];
            }
            if (b < 0) {  // not reached: the last one that holds anything
                b = lastb;
                w -= hw[b];
                n -= hn[b];
            }
            out->key = prefix | (uint32_t)b << shift;
            out->before = w;
            out->n_before = n;
            out->n_equal = hn[b];
        }
        __syncthreads();
        prefix = out->key;
        wb = out->before;
        nb = out->n_before;
    }
    const Found f = *out;
    __syncthreads();
    return f;
}

template <bool HALF>
__global__ void __launch_bounds__(kThreads) sample_kernel(const Args a) {
    __shared__ uint32_t pow64[64];
    __shared__ unsigned long long hw[256];
    __shared__ unsigned int hn[256];
    __shared__ Found found;
    __shared__ uint32_t red[32];
    __shared__ unsigned long long sum_s[2];
    __shared__ int count_s[33];
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const void* row = HALF ? (const void*)(static_cast<const __half*>(a.logits) + r * a.ld)
                           : (const void*)(static_cast<const float*>(a.logits) + r * a.ld);
    if (tid < 64) pow64[tid] = (uint32_t)fmin(4294967295.0, rint(exp2(-tid / 64.0) * 4294967296.0));
    if (tid < 2) sum_s[tid] = 0;
    uint32_t top = 0;
    for (int i = tid; i < a.vocab; i += kThreads) top = max(top, key_of(logit<HALF>(a, row, i)));
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) red[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, red[lane]);
    if (top <= kLeast) {  // nothing to choose from
        if (tid == 0) {
            a.tokens[r] = -1;
            if (a.probs) a.probs[r] = 0.f;
        }
        return;
    }
    const float T = a.temperature ? a.temperature[r] : 1.f;
    const bool greedy = !a.u || !(T > 0.f);
    Scale c;
    {
        c.max = key_value(top);
        const double s = fmin(1.4426950408889634 / (greedy ? 1.0 : (double)T), 1e30);
        c.hi = (float)s;
        c.lo = (float)(s - (double)c.hi);
    }
    uint32_t key = top;
    unsigned long long rank = 0, w_kept = kOne, w_key = kOne;
    if (!greedy) {
        // the weight of all, and of those that min_p keeps
        const float mp = a.min_p ? a.min_p[r] : 0.f;
        const double least = mp > 0.f ? (double)fminf(mp, 1.f) * (double)kOne : 0.0;
        unsigned long long all = 0, some = 0;
        for (int i = tid; i < a.vocab; i += kThreads) {
            const uint32_t k = key_of(logit<HALF>(a, row, i));
            if (k == kLeast) continue;
            const unsigned long long w = weight_of(key_value(k), c, pow64);
            all += w;
            if ((double)w >= least) some += w;
        }
        atomicAdd(&sum_s[0], all);
        atomicAdd(&sum_s[1], some);
        __syncthreads();
        unsigned long long W = sum_s[0];
        const int k = a.top_k ? a.top_k[r] : 0;
        if (k > 0 && k < a.vocab) {
            const Found f = search<HALF, true>(a, row, c, pow64, k, hw, hn, &found);
            const unsigned long long left = (unsigned long long)k > f.n_before ? k - f.n_before : 0;
            W = f.before + (left < f.n_equal ? left : f.n_equal) * weight_of(key_value(f.key), c, pow64);
        }
        const float p = a.top_p ? a.top_p[r] : 1.f;
        if (p < 1.f) {
            const double want = ceil((double)fmaxf(p, 0.f) * (double)W);
            const unsigned long long target = want < 1.0 ? 1 : want > (double)W ? W : (unsigned long long)want;
            const Found f = search<HALF, false>(a, row, c, pow64, target, hw, hn, &found);
            const unsigned long long w = weight_of(key_value(f.key), c, pow64);
            const unsigned long long m = w ? (target - f.before + w - 1) / w : 0;
            W = f.before + (m < f.n_equal ? m : f.n_equal) * w;
        }
        if (least > 0.0 && sum_s[1] < W) W = sum_s[1];
        w_kept = W;
        const double u = fmin(fmax((double)a.u[r], 0.0), 1.0);
        unsigned long long target = (unsigned long long)(u * (double)W) + 1;
        if (target > W) target = W;
        const Found f = search<HALF, false>(a, row, c, pow64, target, hw, hn, &found);
        key = f.key;
        w_key = weight_of(key_value(key), c, pow64);
        rank = w_key ? (target - f.before - 1) / w_key : 0;
        if (rank >= f.n_equal) rank = f.n_equal - 1;
    }
    // the rank-th token, by index, that has the key
    unsigned long long seen = 0;
    for (int i0 = 0; i0 < a.vocab; i0 += kThreads) {
        const int i = i0 + tid;
        const bool eq = i < a.vocab && key_of(logit<HALF>(a, row, i)) == key;
        const unsigned b = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) count_s[warp] = __popc(b);
        __syncthreads();
        unsigned long long before = seen;
        for (int j = 0; j < warp; ++j) before += count_s[j];
        if (eq && before + __popc(b & ((1u << lane) - 1u)) == rank) {
            a.tokens[r] = i;
            if (a.probs) a.probs[r] = (float)((double)w_key / (double)w_kept);
        }
        for (int j = 0; j < kThreads / 32; ++j) seen += count_s[j];
        __syncthreads();
        if (seen > rank) break;
    }
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
    if (d.dtype == Q4_F16)
        q4s::sample_kernel<true><<<d.rows, q4s::kThreads, 0, s>>>(a);
    else
        q4s::sample_kernel<false><<<d.rows, q4s::kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? Q4_OK : cuda_fail(e, "q4_sample launch");
}
