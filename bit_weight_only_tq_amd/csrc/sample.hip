// Sampling: one token a row from its logits, temperature, top-k, min-p, top-p
// and a given random number.
//
// With the weights w_i = exp((x_i - max x) / T) and the tokens ranked by
// (logit, lowest index first), the kept tokens are a prefix of the ranking:
// the first k, of these the ones with w >= min_p, of these the ones whose
// weight before them is below top_p times the weight of them all.  The token
// drawn is the first index at which the running weight of the kept tokens, in
// index order, passes u times their total.
//
// A prefix of the ranking is a cut: a logit (as an order-preserving 32-bit
// key) and how many of the tokens with that logit are in, lowest index first.
// The cuts are found by radix selection on the keys with histograms of counts
// and weights, no sort.  A kept set hangs on comparisons of weight sums, so
// weights are computed in fp64 and summed as 64-bit fixed point: such sums do
// not depend on their order, so atomics and any split of the row give the same
// bits, and their error (2^-44 of the largest weight each) is far below any
// token's share.

#include <math.h>

#include "tq_device.h"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;

struct LogitF32 {
    static constexpr int VEC = 4;
    typedef uint32_t raw;
    static __device__ __forceinline__ float value(const uint32_t (&w)[4], int i) { return __uint_as_float(w[i]); }
    static __device__ __forceinline__ float one(const void* row, int64_t i) { return static_cast<const float*>(row)[i]; }
};
template <class E>
struct Logit16 {
    static constexpr int VEC = 8;
    typedef uint16_t raw;
    static __device__ __forceinline__ float value(const uint32_t (&w)[4], int i) {
        return E::to_f32((uint16_t)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]));
    }
    static __device__ __forceinline__ float one(const void* row, int64_t i) {
        return E::to_f32(static_cast<const uint16_t*>(row)[i]);
    }
};

// Order-preserving key of a logit; NaN counts as -inf and -0 as +0.  No logit
// has key 0, which stands for "no token".
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float(key ^ ((key & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}

// VEC logits from element i on (keys; 0 past the row's end).  Rows of an odd
// vocabulary start anywhere, so the load asks for the alignment of one value.
template <class L>
__device__ __forceinline__ void load_keys(const void* row, int i, int V, uint32_t (&key)[L::VEC]) {
    constexpr int VEC = L::VEC;
    if (i + VEC <= V) {
        struct __attribute__((packed, aligned(sizeof(typename L::raw)))) Vec {
            uint32_t w[4];
        };
        const Vec v = *reinterpret_cast<const Vec*>(static_cast<const typename L::raw*>(row) + i);
        uint32_t w[4] = {v.w[0], v.w[1], v.w[2], v.w[3]};
#pragma unroll
        for (int e = 0; e < VEC; ++e) key[e] = key_of(L::value(w, e));
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) key[e] = i + e < V ? key_of(L::one(row, i + e)) : 0u;
    }
}

struct Row {
    double max, inv_t;  // largest logit, 1 / T
    uint32_t kmax;
    double fix;         // 2^S: fixed-point unit of the weights
    __device__ __forceinline__ double weight(uint32_t key) const {
        if (key == kmax) return 1.0;             // also +inf
        if (key <= 0x007FFFFFu) return 0.0;      // -inf or no token
        return exp(((double)logit_of(key) - max) * inv_t);
    }
    __device__ __forceinline__ uint64_t fixed(double w) const { return (uint64_t)(w * fix + 0.5); }
};

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor((unsigned long long)v, d, 64);
    return v;
}

struct Shared {
    uint32_t count[kBins];
    unsigned long long weight[kBins];
    unsigned long long scan_w[kWaves];
    uint32_t scan_c[kWaves];
    // results of a search
    uint32_t bin, found, before_c;
    unsigned long long before_w, total_w;
    unsigned long long best;
    uint32_t first;
    int seg;
    uint32_t seg_ties;
    unsigned long long seg_before;
};

// Exclusive prefix sums over the workgroup's threads of (c, w), in thread order; the totals go to *tc, *tw.
__device__ __forceinline__ void block_scan(Shared& sh, uint32_t c, uint64_t w, uint32_t* bc, uint64_t* bw, uint32_t* tc,
                                           uint64_t* tw) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t ic = c;
    unsigned long long iw = w;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t oc = __shfl_up(ic, d, 64);
        const unsigned long long ow = __shfl_up(iw, d, 64);
        if (lane >= d) {
            ic += oc;
            iw += ow;
        }
    }
    __syncthreads();
    if (lane == 63) {
        sh.scan_c[wave] = ic;
        sh.scan_w[wave] = iw;
    }
    __syncthreads();
    uint32_t pc = 0, sc = 0;
    uint64_t pw = 0, sw = 0;
    for (int i = 0; i < kWaves; ++i) {
        if (i == wave) {
            pc = sc;
            pw = sw;
        }
        sc += sh.scan_c[i];
        sw += sh.scan_w[i];
    }
    *bc = pc + ic - c;
    *bw = pw + iw - w;
    *tc = sc;
    *tw = sw;
}

// A cut of the ranking being refined, digit by digit: the keys whose top bits
// are `prefix` hold the border, `c` tokens of weight `w` rank above them.
struct Cut {
    uint32_t prefix;
    int bits;  // of the prefix
    uint32_t c;
    uint64_t w;
};

// Histogram (count and weight) of the next digit of the keys in `cut`'s bin
// that are at least `floor_key`.
template <class L>
__device__ __forceinline__ void histogram(Shared& sh, const void* row, int V, const Row& r, const Cut& cut, int digit,
                                          double min_w, uint32_t floor_key) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        sh.count[i] = 0;
        sh.weight[i] = 0;
    }
    __syncthreads();
    const int shift = 32 - cut.bits - digit;
    for (int i = threadIdx.x * L::VEC; i < V; i += kThreads * L::VEC) {
        uint32_t key[L::VEC];
        load_keys<L>(row, i, V, key);
#pragma unroll
        for (int e = 0; e < L::VEC; ++e) {
            if (key[e] == 0 || key[e] < floor_key || (cut.bits && (key[e] >> (32 - cut.bits)) != cut.prefix)) continue;
            const double w = r.weight(key[e]);
            if (w < min_w) continue;
            const uint32_t b = (key[e] >> shift) & ((1u << digit) - 1);
            atomicAdd(&sh.count[b], 1u);
            atomicAdd(&sh.weight[b], (unsigned long long)r.fixed(w));
        }
    }
    __syncthreads();
}

// The bin, from the largest key down, in which the ranking's prefix ends: the
// one that holds token number `k` (by count), or the first after which the
// weight is no longer below `limit`.  Without one everything is in the prefix.
__device__ __forceinline__ bool search(Shared& sh, Cut& cut, int digit, bool by_count, uint32_t k, double limit,
                                       uint64_t* total) {
    if (threadIdx.x == 0) sh.found = 0;
    constexpr int PER = kBins / kThreads;
    uint32_t c = 0;
    uint64_t w = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = kBins - 1 - (threadIdx.x * PER + i);
        c += sh.count[b];
        w += sh.weight[b];
    }
    uint32_t bc, tc;
    uint64_t bw, tw;
    block_scan(sh, c, w, &bc, &bw, &tc, &tw);
    bc += cut.c;
    bw += cut.w;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = kBins - 1 - (threadIdx.x * PER + i);
        const uint32_t nc = bc + sh.count[b];
        const uint64_t nw = bw + sh.weight[b];
        const bool here = sh.count[b] && (by_count ? (bc < k && k <= nc) : ((double)bw < limit && !((double)nw < limit)));
        if (here) {
            sh.found = 1;
            sh.bin = b;
            sh.before_c = bc;
            sh.before_w = bw;
        }
        bc = nc;
        bw = nw;
    }
    __syncthreads();
    if (total) *total = cut.w + tw;
    if (!sh.found) return false;
    cut.prefix = (cut.prefix << digit) | sh.bin;
    cut.bits += digit;
    cut.c = sh.before_c;
    cut.w = sh.before_w;
    return true;
}

template <class L>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
    __shared__ Shared sh;
    extern __shared__ unsigned long long seg_mem[];  // per segment: weight, then ties
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int V = a.V;
    const int64_t b = blockIdx.x;
    const void* row = static_cast<const typename L::raw*>(a.logits) + b * a.row_stride;
    constexpr int VEC = L::VEC, SEG = 64 * VEC;

    // largest logit, lowest index
    if (tid == 0) {
        sh.best = 0;
        sh.first = 0xFFFFFFFFu;
    }
    __syncthreads();
    unsigned long long best = 0;
    for (int i = tid * VEC; i < V; i += kThreads * VEC) {
        uint32_t key[VEC];
        load_keys<L>(row, i, V, key);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const unsigned long long x = ((unsigned long long)key[e] << 32) | (uint32_t)~(i + e);
            best = key[e] && x > best ? x : best;
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const unsigned long long o = __shfl_xor(best, d, 64);
        best = o > best ? o : best;
    }
    if (lane == 0) atomicMax(&sh.best, best);
    __syncthreads();
    best = sh.best;
    Row r;
    r.kmax = (uint32_t)(best >> 32);
    const int top = (int)~(uint32_t)best;
    if (r.kmax <= 0x007FFFFFu) {  // every logit is -inf or NaN
        if (tid == 0) {
            a.tokens[b] = -1;
            if (a.logprobs) a.logprobs[b] = -INFINITY;
        }
        return;
    }
    const float T = a.temperature ? a.temperature[b] : 1.0f;
    const float p = a.top_p ? a.top_p[b] : 1.0f;
    const float min_p = a.min_p ? a.min_p[b] : 0.0f;
    int k = a.top_k ? a.top_k[b] : 0;
    if (k <= 0 || k > V) k = V;
    float u = a.u[b];
    u = u > 0.0f ? fminf(u, 0.99999994f) : 0.0f;
    if (!(T > 0.0f) || k == 1 || !(p > 0.0f) || !(min_p <= 1.0f)) {  // the best token alone is kept
        if (tid == 0) {
            a.tokens[b] = top;
            if (a.logprobs) a.logprobs[b] = 0.0f;
        }
        return;
    }
    r.max = (double)logit_of(r.kmax);
    r.inv_t = 1.0 / (double)T;
    r.fix = a.fix;

    // the cut: tokens with keys above `ckey`, and the first `cties` with it
    const double min_w = min_p > 0.0f ? (double)min_p : 0.0;
    uint32_t ckey = 0, cties = 0;
    const bool by_k = k < V, by_p = p < 1.0f;
    if (by_k || by_p) {
        Cut root{0, 0, 0, 0};
        uint64_t total = 0;
        const int digits[3] = {11, 11, 10};
        if (by_k) {
            Cut cut = root;
            bool in = true;
            for (int d = 0; d < 3 && in; ++d) {
                histogram<L>(sh, row, V, r, cut, digits[d], min_w, 0);
                in = search(sh, cut, digits[d], true, (uint32_t)k, 0.0, &total);
            }
            if (in) {  // otherwise fewer than k tokens are left, and `total` is their weight
                ckey = cut.prefix;
                cties = (uint32_t)k - cut.c;
                total = cut.w + cties * r.fixed(r.weight(ckey));
            }
        }
        if (by_p) {
            Cut cut = root;
            bool in = true;
            const uint32_t floor_key = ckey;
            double limit = 0.0;
            for (int d = 0; d < 3 && in; ++d) {
                histogram<L>(sh, row, V, r, cut, digits[d], min_w, floor_key);
                if (d == 0) {
                    if (!by_k) {
                        uint64_t all;
                        Cut none = root;
                        search(sh, none, digits[d], true, 0xFFFFFFFFu, 0.0, &all);
                        total = all;
                        __syncthreads();
                    }
                    limit = (double)p * (double)total;
                }
                in = search(sh, cut, digits[d], false, 0, limit, nullptr);
            }
            if (in) {
                const uint64_t one = r.fixed(r.weight(cut.prefix));
                const double n = one ? ceil((limit - (double)cut.w) / (double)one) : 1.0;
                uint32_t ties = n < 1.0 ? 1u : n > 2147483647.0 ? 0x7FFFFFFFu : (uint32_t)n;
                if (cut.prefix == ckey && ties > cties) ties = cties;
                ckey = cut.prefix;
                cties = ties;
            }
        }
    }

    // weights of the kept tokens by segments of the row
    const int segs = (V + SEG - 1) / SEG;
    unsigned long long* seg_w = seg_mem;
    uint32_t* seg_t = reinterpret_cast<uint32_t*>(seg_mem + segs);
    uint32_t first = 0xFFFFFFFFu;  // first kept index of positive weight
    for (int s = wave; s < segs; s += kWaves) {
        uint32_t key[VEC];
        const int i = s * SEG + lane * VEC;
        load_keys<L>(row, i, V, key);
        uint64_t w = 0;
        uint32_t ties = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (key[e] < ckey || key[e] == 0) continue;
            const double x = r.weight(key[e]);
            if (x < min_w) continue;
            if (x > 0.0) first = min(first, (uint32_t)(i + e));
            if (key[e] == ckey) ++ties;
            else w += r.fixed(x);
        }
        w = wave_sum_u64(w);
        for (int d = 32; d > 0; d >>= 1) ties += __shfl_xor(ties, d, 64);
        if (lane == 0) {
            seg_w[s] = w;
            seg_t[s] = ties;
        }
    }
    for (int d = 32; d > 0; d >>= 1) first = min(first, (uint32_t)__shfl_xor((int)first, d, 64));
    if (lane == 0) atomicMin(&sh.first, first);
    __syncthreads();
    const uint64_t one = ckey ? r.fixed(r.weight(ckey)) : 0;
    const int per = (segs + kThreads - 1) / kThreads;
    const int s0 = min(segs, tid * per), s1 = min(segs, s0 + per);
    uint32_t tc = 0, bt, all_t;
    uint64_t bw, all_w;
    for (int s = s0; s < s1; ++s) tc += seg_t[s];
    block_scan(sh, tc, 0, &bt, &bw, &all_t, &all_w);
    uint64_t mine = 0;
    {
        uint32_t t = bt;
        for (int s = s0; s < s1; ++s) {
            const uint32_t in = t < cties ? min(cties - t, seg_t[s]) : 0;
            mine += seg_w[s] + in * one;
            t += seg_t[s];
        }
    }
    uint32_t d0, d1;
    block_scan(sh, 0, mine, &d0, &bw, &d1, &all_w);
    const double target = (double)u * (double)all_w;
    {
        uint32_t t = bt;
        uint64_t before = bw;
        for (int s = s0; s < s1; ++s) {
            const uint32_t in = t < cties ? min(cties - t, seg_t[s]) : 0;
            const uint64_t next = before + seg_w[s] + in * one;
            if (!((double)before > target) && (double)next > target) {
                sh.seg = s;
                sh.seg_ties = t;
                sh.seg_before = before;
            }
            t += seg_t[s];
            before = next;
        }
    }
    __syncthreads();
    if (wave != 0) return;
    // the token inside its segment
    const int i = sh.seg * SEG + lane * VEC;
    uint32_t key[VEC];
    load_keys<L>(row, i, V, key);
    uint32_t ties = 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) ties += ckey && key[e] == ckey;
    uint32_t it = ties;
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(it, d, 64);
        if (lane >= d) it += o;
    }
    uint32_t t = sh.seg_ties + it - ties;
    uint64_t w[VEC], sum = 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        w[e] = 0;
        if (key[e] < ckey || key[e] == 0) continue;
        if (ckey && key[e] == ckey && t++ >= cties) continue;
        const double x = r.weight(key[e]);
        if (x >= min_w) w[e] = r.fixed(x);
        sum += w[e];
    }
    unsigned long long is = sum;
    for (int d = 1; d < 64; d <<= 1) {
        const unsigned long long o = __shfl_up(is, d, 64);
        if (lane >= d) is += o;
    }
    uint64_t before = sh.seg_before + is - sum;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const uint64_t next = before + w[e];
        const bool here = u > 0.0f ? (!((double)before > target) && (double)next > target) : false;
        if (here) {
            a.tokens[b] = i + e;
            if (a.logprobs) a.logprobs[b] = (float)log(r.weight(key[e]) / ((double)all_w / r.fix));
        }
        before = next;
    }
    if (u == 0.0f && lane == 0) {
        const uint32_t f = sh.first;
        a.tokens[b] = (int32_t)f;
        if (a.logprobs) a.logprobs[b] = (float)log(r.weight(key_of(L::one(row, f))) / ((double)all_w / r.fix));
    }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& args, hipStream_t s) {
    SampleArgs a = args;
    int bits = 0;
    while (((int64_t)1 << bits) < a.V) ++bits;
    a.fix = ldexp(1.0, 62 - bits);
    const int seg = a.dtype == 2 ? 64 * LogitF32::VEC : 64 * 8;
    const size_t lds = (size_t)((a.V + seg - 1) / seg) * 12 + 8;
    static DeviceFlags r32, rh, rb;
    const int most = (int)(kSampleMaxVocab / 256) * 12 + 8;
    hipError_t e = hipSuccess;
    const dim3 grid((unsigned)a.B), block(kThreads);
    if (a.dtype == 2) {
        e = raise_lds_limit(reinterpret_cast<const void*>(sample_kernel<LogitF32>), most, r32);
        if (e == hipSuccess) sample_kernel<LogitF32><<<grid, block, lds, s>>>(a);
    } else if (a.dtype == 1) {
        e = raise_lds_limit(reinterpret_cast<const void*>(sample_kernel<Logit16<BF16>>), most, rb);
        if (e == hipSuccess) sample_kernel<Logit16<BF16>><<<grid, block, lds, s>>>(a);
    } else {
        e = raise_lds_limit(reinterpret_cast<const void*>(sample_kernel<Logit16<F16>>), most, rh);
        if (e == hipSuccess) sample_kernel<Logit16<F16>><<<grid, block, lds, s>>>(a);
    }
    return e != hipSuccess ? e : hipGetLastError();
}

}  // namespace tq
