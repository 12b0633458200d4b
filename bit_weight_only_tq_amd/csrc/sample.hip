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
// Cuts are found by radix selection on the keys with histograms of counts and
// weights, no sort.  A kept set hangs on comparisons of weight sums, so
// weights are computed in fp64 and summed as 64-bit fixed point: such sums do
// not depend on their order, so atomics and any split of the row give the same
// bits, and their error (2^-43 of the largest weight each, at most) is far below any
// token's share.
//
// One workgroup a row.  What it costs is the passes over the row and the
// exponentials, so the selection runs on a short list in LDS wherever one
// holds every token that can be kept (sample_kernel tells which):
//  * up to 4096 logits: the whole row, or the part of it that these leave;
//  * top-k with k <= 1024: the k-th largest of 2048 maxima, two of each
//    thread's share, is a logit that at least k tokens reach, and not many
//    more do;
//  * min-p: the tokens of at least min_p;
//  * top-p alone: the tokens of one of 2048 even steps of the logits, the one
//    in which the weights pass top_p of their total.
// A list that overflows leaves the selection to passes over the row.
//
// Times of a call among others, on other logits each time.  One row of 32000
// with top-k of 50 and top-p: 12 us, in which every phase is a few microseconds
// of latency.  64 rows of 128000 (16 bits), top-k of 200 and top-p: 23 us, two
// passes over a row by one compute unit taking 13.  256 rows of 129281 (fp32),
// min-p and top-p: 34 us, 3.9 TB/s of logits (29 us, 4.5 TB/s, where they are
// the last call's and lie in the card's cache).  By histograms over the whole
// row the three took 67, 192 and 174 us.  64 rows of 129281, top-p alone: 113 us,
// without a cut 78 us: a 12-term series a logit on 64 of 256 compute units.

#include <math.h>

#include "tq_device.h"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr int kList = 4096;  // tokens of a list

struct LogitF32 {
    static constexpr int VEC = 4, FLIGHT = 8;  // FLIGHT: vectors a thread reads at a time
    typedef uint32_t raw;
    static __device__ __forceinline__ float value(const uint32_t (&w)[4], int i) { return __uint_as_float(w[i]); }
    static __device__ __forceinline__ float one(const void* row, int64_t i) { return static_cast<const float*>(row)[i]; }
};
template <class E>
struct Logit16 {
    static constexpr int VEC = 8, FLIGHT = 4;
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

// The logits x of a row for which pre(x, place in its vector)
// holds, as f(x, index), U vectors a
// thread in flight.  Vectors past the end are read from the last whole one and
// their values dropped.  `from`, `to`: of the row, whole rounds of U vectors a
// thread, without either the whole row.
template <class L, int U, class P, class F>
__device__ __forceinline__ void each_logit(const void* row, int V, P pre, F f, int from = 0, int to = INT32_MAX) {
    constexpr int VEC = L::VEC, STEP = kThreads * VEC;
    const typename L::raw* x = static_cast<const typename L::raw*>(row);
    if (V < VEC) {
        if (from == 0 && (int)threadIdx.x < V && pre(L::one(row, threadIdx.x), 0)) f(L::one(row, threadIdx.x), (int)threadIdx.x);
        return;
    }
    struct __attribute__((packed, aligned(sizeof(typename L::raw)))) Vec {
        uint32_t w[4];
    };
    for (int base = from + (int)threadIdx.x * VEC; base < min(V, to); base += U * STEP) {
        Vec v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const Vec*>(x + min(base + u * STEP, V - VEC));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = base + u * STEP, at = min(i, V - VEC);
            const uint32_t w[4] = {v[u].w[0], v[u].w[1], v[u].w[2], v[u].w[3]};
            if (i + VEC <= V) {
                uint32_t hits = 0;
#pragma unroll
                for (int e = 0; e < VEC; ++e) hits |= pre(L::value(w, e), e) ? 1u << e : 0u;
                for (; hits; hits &= hits - 1) {
                    const int e = __ffs((int)hits) - 1;
                    float x = L::value(w, 0);
#pragma unroll
                    for (int o = 1; o < VEC; ++o) x = e == o ? L::value(w, o) : x;
                    f(x, i + e);
                }
            } else if (i < V) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (at + e >= i && pre(L::value(w, e), e)) f(L::value(w, e), at + e);
            }
        }
    }
}

// 2^f for |f| <= 1/2 by its series: the first term left out is
// (f ln 2)^13 / 13!, at most 1.7e-16, 2^-51 of the sum.
__device__ __forceinline__ double exp2_series(double f) {
    constexpr double L = 0.69314718055994531, L2 = L * L, L3 = L2 * L, L4 = L2 * L2;
    double s = L4 * L4 * L4 / 479001600.0;
    s = fma(s, f, L4 * L4 * L3 / 39916800.0);
    s = fma(s, f, L4 * L4 * L2 / 3628800.0);
    s = fma(s, f, L4 * L4 * L / 362880.0);
    s = fma(s, f, L4 * L4 / 40320.0);
    s = fma(s, f, L4 * L3 / 5040.0);
    s = fma(s, f, L4 * L2 / 720.0);
    s = fma(s, f, L4 * L / 120.0);
    s = fma(s, f, L4 / 24.0);
    s = fma(s, f, L3 / 6.0);
    s = fma(s, f, L2 / 2.0);
    s = fma(s, f, L);
    return fma(s, f, 1.0);
}

struct Row {
    double max, per_t;  // largest logit, log2(e) / T
    uint32_t kmax;
    int fix;            // weights are summed in units of 2^-fix, fix <= 52
    // weight * 2^shift
    __device__ __forceinline__ double scaled(uint32_t key, int shift) const {
        if (key <= 0x007FFFFFu) return 0.0;  // -inf or no token
        // also of the largest, +inf and overflow: the maximum of the fp64
        // exponent's -1100 and NaN is -1100
        const double y = key == kmax ? 0.0 : fmax(((double)logit_of(key) - max) * per_t, -1100.0);
        const double n = rint(y);
        return ldexp(exp2_series(y - n), (int)n + shift);
    }
    __device__ __forceinline__ double weight(uint32_t key) const { return scaled(key, 0); }
    // The weight in units of 2^-fix, to the nearest: the low bits of 2^52 plus it.
    __device__ __forceinline__ uint64_t fixed(uint32_t key) const { return units(scaled(key, fix)); }
    __device__ __forceinline__ uint64_t fixed(double weight) const { return units(ldexp(weight, fix)); }
    static __device__ __forceinline__ uint64_t units(double x) {
        return (uint64_t)__double_as_longlong(x + 4503599627370496.0) - 0x4330000000000000ull;
    }
    __device__ __forceinline__ double of_units(uint64_t x) const { return ldexp((double)x, -fix); }
    // Even steps of the logits below the largest, as bins that rise with the
    // logit: 2048 over the 32 T in which a weight can add to a sum, or over 64
    // where that is less.  Rounding keeps the order, so equal logits share a
    // bin and larger ones never have a lower one.
    __device__ __forceinline__ float step(float T) const { return (float)kBins / fminf(32.0f * T, 64.0f); }
    // The lower end of a bin (above 0), less a margin that covers the roundings.
    __device__ __forceinline__ float step_end(int bin, float step) const {
        return top() - (float)(kBins - bin) / step - (fabsf(top()) + 64.0f) * 1e-6f;
    }
    __device__ __forceinline__ float top() const { return logit_of(kmax); }
    __device__ __forceinline__ int bin(uint32_t key, float step) const {
        if (key == kmax) return kBins - 1;  // also +inf
        return kBins - 1 - (int)fminf((logit_of(kmax) - logit_of(key)) * step, (float)(kBins - 1));
    }
};

// Inclusive prefix sums over the 64 lanes, by lane shifts within rows of 16 and
// two broadcasts between rows: no LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {  // 0 where there is none
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t from_lane(uint64_t v) {
    return (uint64_t)from_lane<CTRL, ROWS>((uint32_t)v) | (uint64_t)from_lane<CTRL, ROWS>((uint32_t)(v >> 32)) << 32;
}
template <class N>
__device__ __forceinline__ N wave_scan(N v) {
    v += from_lane<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
    v += from_lane<0x112, 0xF>(v);
    v += from_lane<0x114, 0xF>(v);
    v += from_lane<0x118, 0xF>(v);
    v += from_lane<0x142, 0xA>(v);  // last lane of rows 0 and 2 to rows 1 and 3
    v += from_lane<0x143, 0xC>(v);  // lane 31 to rows 2 and 3
    return v;
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }
__device__ __forceinline__ uint64_t lane_of(uint64_t v, int lane) {
    return (uint64_t)lane_of((uint32_t)v, lane) | (uint64_t)lane_of((uint32_t)(v >> 32), lane) << 32;
}

struct Shared {
    uint32_t count[kBins];
    unsigned long long weight[kBins];
    unsigned long long scan_w[kWaves];
    uint32_t scan_c[kWaves];
    // results of a search
    uint32_t bin, found, before_c;
    unsigned long long before_w, total_w;
    uint32_t best, first;
    int seg;
    uint32_t seg_ties;
    unsigned long long seg_before;
    uint32_t n;  // tokens of the list, also past its end
};

// The list: keys (0: dropped) and indexes, behind which the segments of a
// drawing over the row lie where there is no list.
struct List {
    uint32_t key[kList], idx[kList];
};

// Exclusive prefix sums over the workgroup's threads of (c, w), in thread order; the totals go to *tc, *tw.
__device__ __forceinline__ void block_scan(Shared& sh, uint32_t c, uint64_t w, uint32_t* bc, uint64_t* bw, uint32_t* tc,
                                           uint64_t* tw) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t ic = wave_scan(c);
    const uint64_t iw = wave_scan(w);
    __syncthreads();
    if (lane == 63) {
        sh.scan_c[wave] = ic;
        sh.scan_w[wave] = iw;
    }
    __syncthreads();
    // every wave scans the sums of the waves in its first lanes
    static_assert(kWaves == 16, "one row of lanes");
    const uint32_t sc = wave_scan(lane < kWaves ? sh.scan_c[lane] : 0u);
    const uint64_t sw = wave_scan(lane < kWaves ? (uint64_t)sh.scan_w[lane] : (uint64_t)0);
    const int before = __builtin_amdgcn_readfirstlane(wave) - 1;
    *bc = (before < 0 ? 0u : lane_of(sc, before)) + ic - c;
    *bw = (before < 0 ? 0ull : lane_of(sw, before)) + iw - w;
    *tc = lane_of(sc, kWaves - 1);
    *tw = lane_of(sw, kWaves - 1);
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
    uint32_t c = 0, cs[PER];
    uint64_t w = 0, ws[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = kBins - 1 - (threadIdx.x * PER + i);
        c += cs[i] = sh.count[b];
        w += ws[i] = sh.weight[b];
    }
    uint32_t bc, tc;
    uint64_t bw, tw;
    block_scan(sh, c, w, &bc, &bw, &tc, &tw);
    bc += cut.c;
    bw += cut.w;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t nc = bc + cs[i];
        const uint64_t nw = bw + ws[i];
        const bool here = cs[i] && (by_count ? (bc < k && k <= nc) : ((double)bw < limit && !((double)nw < limit)));
        if (here) {
            sh.found = 1;
            sh.bin = kBins - 1 - (threadIdx.x * PER + i);
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

// The same over the first n tokens of the list.
__device__ __forceinline__ void histogram_list(Shared& sh, const List& list, int n, const Row& r, const Cut& cut, int digit,
                                               uint32_t floor_key) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        sh.count[i] = 0;
        sh.weight[i] = 0;
    }
    __syncthreads();
    const int shift = 32 - cut.bits - digit;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint32_t key = list.key[i];
        if (key == 0 || key < floor_key || (cut.bits && (key >> (32 - cut.bits)) != cut.prefix)) continue;
        const uint32_t b = (key >> shift) & ((1u << digit) - 1);
        atomicAdd(&sh.count[b], 1u);
        atomicAdd(&sh.weight[b], (unsigned long long)r.fixed(key));
    }
    __syncthreads();
}

// How many of the tokens with the cut's logit are in, by weight.
__device__ __forceinline__ uint32_t ties_in(const Row& r, const Cut& cut, double limit) {
    const uint64_t one = r.fixed(cut.prefix);
    const double n = one ? ceil((limit - (double)cut.w) / (double)one) : 1.0;
    return n < 1.0 ? 1u : n > 2147483647.0 ? 0x7FFFFFFFu : (uint32_t)n;
}

__device__ __forceinline__ void append(Shared& sh, List& list, uint32_t key, int i) {
    const uint32_t at = atomicAdd(&sh.n, 1u);
    if (at < (uint32_t)kList) {
        list.key[at] = key;
        list.idx[at] = (uint32_t)i;
    }
}

// A logit that at least k tokens reach: the lower end of the step that holds
// the k-th largest of the threads' 2 * kThreads maxima, which are logits of
// different tokens.  The lowest finite one if there is no such step.
__device__ __forceinline__ uint32_t floor_of_best(Shared& sh, const Row& r, const float (&most)[2], uint32_t k) {
    const float step = (float)kBins / 64.0f;
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
        sh.count[i] = 0;
        sh.weight[i] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (most[i] > -INFINITY) atomicAdd(&sh.count[r.bin(key_of(most[i]), step)], 1u);
    __syncthreads();
    Cut cut{0, 0, 0, 0};
    if (!search(sh, cut, 0, true, k, 0.0, nullptr) || sh.bin == 0) return 0x00800000u;
    return max(key_of(r.step_end((int)sh.bin, step)), 0x00800000u);
}

// A logit that every token of weight min_p or more reaches, by a margin that
// covers the roundings of fp64 and of the logarithm many times over.
__device__ __forceinline__ uint32_t floor_of(const Row& r, double T, double min_p) {
    const double d = T * log(min_p), x = r.max + d;
    const double low = x - 1e-9 * (fabs(r.max) + fabs(d) + T);
    if (!(low > -3.0e38)) return 0x00800000u;  // every finite logit
    float f = (float)low;
    f -= fabsf(f) * 1e-6f + 1e-37f;
    return f > -3.0e38f ? key_of(f) : 0x00800000u;
}

// Cuts and the drawing where the list holds every token that can be kept, at
// most kFew.  Every token's place by rank and by index is counted, all pairs
// spread over the workgroup's threads; then two prefix sums of the weights, in
// the one order and in the other, give the cut and the token.  Against passes
// of histograms this is a few short loops: code that runs once is bound by its
// own fetch and by the workgroup's barriers.
constexpr int kFew = 512;
__device__ __forceinline__ void draw_from_few(Shared& sh, const List& list, int n, const Row& r, double min_w, int k, float p,
                                              float u, int32_t* token, float* logprob) {
    const int tid = threadIdx.x;
    struct Few {
        uint64_t rank[kFew], by_rank[kFew], by_idx[kFew];
        uint32_t place[kFew];  // by rank, and << 16 by index
    };
    static_assert(sizeof(Few) <= sizeof(sh.count) + sizeof(sh.weight), "the bins' memory");
    Few& few = *reinterpret_cast<Few*>(sh.count);
    int width = 64;
    while (width < n) width *= 2;
    bool in = false;
    uint32_t key = 0, at = 0xFFFFFFFFu;
    uint64_t w = 0;
    double x = 0.0;
    __syncthreads();
    if (tid < width) {
        if (tid < n) {
            key = list.key[tid];
            at = list.idx[tid];
            x = r.weight(key);
            in = x > 0.0 && !(x < min_w);
            w = in ? r.fixed(x) : 0ull;
        }
        // larger: a better rank; the low word falls with the index also where
        // the token is out (no key), and is 0 past the list
        few.rank[tid] = (uint64_t)(in ? key : 0u) << 32 | (uint32_t)~at;
        few.by_rank[tid] = few.by_idx[tid] = 0;
        few.place[tid] = 0;
    }
    __syncthreads();
    {
        const int mine = tid & (width - 1), part = tid / width, parts = kThreads / width;
        const int per = ((width / 4 + parts - 1) / parts) * 4, j1 = min(width, (part + 1) * per);
        const uint64_t rank = few.rank[mine];
        uint32_t place = 0;
#pragma unroll 1
        for (int j = part * per; j < j1; j += 4) {
            uint64_t other[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) other[e] = few.rank[j + e];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                place += (other[e] > rank ? 1u : 0u) + ((uint32_t)other[e] > (uint32_t)rank ? 0x10000u : 0u);
        }
        atomicAdd(&few.place[mine], place);
    }
    __syncthreads();
    uint32_t by_rank = 0, by_idx = 0, none_c, all_c;
    if (tid < n) {
        by_rank = few.place[tid] & 0xFFFFu;
        by_idx = few.place[tid] >> 16;
        in = in && by_rank < (uint32_t)k;
        if (in) few.by_rank[by_rank] = w;
    }
    if (p < 1.0f) {
        uint64_t before, total;
        __syncthreads();
        block_scan(sh, 0u, tid < width ? few.by_rank[tid] : (uint64_t)0, &none_c, &before, &all_c, &total);
        if (tid < width) few.by_rank[tid] = before;
        __syncthreads();
        in = in && (double)few.by_rank[by_rank] < (double)p * (double)total;
    }
    if (in) {
        few.by_idx[by_idx] = w;
        atomicMin(&sh.first, by_idx);
    }
    __syncthreads();
    const uint64_t one = tid < width ? few.by_idx[tid] : (uint64_t)0;
    uint64_t past, total;
    block_scan(sh, 0u, one, &none_c, &past, &all_c, &total);
    const double target = (double)u * (double)total;
    if (u > 0.0f && !((double)past > target) && (double)(past + one) > target) sh.first = (uint32_t)tid;
    __syncthreads();
    if (in && by_idx == sh.first) {  // u = 0: the first token that is kept
        *token = (int32_t)at;
        if (logprob) *logprob = (float)log(x / r.of_units(total));
    }
}

// Cuts and the drawing where the list holds every token that can be kept.
__device__ __forceinline__ void draw_from_list(Shared& sh, List& list, int n, const Row& r, double min_w, int k, bool by_k,
                                               float p, float u, int V, int32_t* token, float* logprob) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int digits[3] = {11, 11, 10};
    // tokens without weight, or below min_p, are out; what is left and its weight
    uint32_t c = 0, bc, left;
    uint64_t w = 0, bw, total;
    for (int i = tid; i < n; i += kThreads) {
        const double x = r.weight(list.key[i]);
        if (!(x > 0.0) || x < min_w) list.key[i] = 0;
        else ++c, w += r.fixed(x);
    }
    block_scan(sh, c, w, &bc, &bw, &left, &total);
    // the cut, as in sample_kernel; `ties`: how many tokens have its logit
    uint32_t ckey = 0, cties = 0, ties = 0;
    if (by_k && (uint32_t)k < left) {
        Cut cut{0, 0, 0, 0};
        for (int d = 0; d < 3; ++d) {
            histogram_list(sh, list, n, r, cut, digits[d], 0);
            search(sh, cut, digits[d], true, (uint32_t)k, 0.0, nullptr);
        }
        ckey = cut.prefix;
        cties = (uint32_t)k - cut.c;
        ties = sh.count[sh.bin];
        total = cut.w + cties * r.fixed(ckey);
    }
    if (p < 1.0f) {
        const double limit = (double)p * (double)total;
        Cut cut{0, 0, 0, 0};
        bool in = true;
        for (int d = 0; d < 3 && in; ++d) {
            histogram_list(sh, list, n, r, cut, digits[d], ckey);
            in = search(sh, cut, digits[d], false, 0, limit, nullptr);
        }
        if (in) {
            uint32_t t = ties_in(r, cut, limit);
            if (cut.prefix == ckey && t > cties) t = cties;
            ckey = cut.prefix;
            cties = t;
            ties = sh.count[sh.bin];
        }
    }
    uint32_t gone = 0;  // bit e: this thread's e-th token is a tie past the cut
    if (ties > cties) {  // the lowest indexes of a tie are in: gathered, and each counted against the others
        uint32_t* tied = reinterpret_cast<uint32_t*>(sh.weight);
        static_assert(sizeof(sh.weight) >= kList * sizeof(uint32_t), "room for a list of ties");
        __syncthreads();
        if (tid == 0) sh.n = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads)
            if (list.key[i] == ckey) tied[atomicAdd(&sh.n, 1u)] = list.idx[i];
        __syncthreads();
        const int m = (int)sh.n;
        for (int i = tid, e = 0; i < n; i += kThreads, ++e) {
            if (list.key[i] != ckey) continue;
            const uint32_t at = list.idx[i];
            uint32_t before = 0;
            int j = 0;
            for (; j + 4 <= m; j += 4) {
                const uint32_t t0 = tied[j], t1 = tied[j + 1], t2 = tied[j + 2], t3 = tied[j + 3];
                before += (t0 < at) + (t1 < at) + (t2 < at) + (t3 < at);
            }
            for (; j < m; ++j) before += tied[j] < at;
            if (before >= cties) gone |= 1u << e;
        }
    }
    // what the cut leaves, by steps of the row's index: kBins at most
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) sh.weight[i] = 0;
    if (tid == 0) sh.n = 0;
    __syncthreads();
    int shift = 0;
    while ((V - 1) >> shift >= kBins) ++shift;
    uint32_t first = 0xFFFFFFFFu;
    for (int i = tid, e = 0; i < n; i += kThreads, ++e) {
        const uint32_t key = list.key[i], at = list.idx[i];
        if (key == 0 || gone >> e & 1) continue;
        if (key < ckey) {
            gone |= 1u << e;
            continue;
        }
        first = min(first, at);
        atomicAdd(&sh.weight[at >> shift], (unsigned long long)r.fixed(key));
    }
    for (int d = 32; d > 0; d >>= 1) first = min(first, (uint32_t)__shfl_xor((int)first, d, 64));
    if (lane == 0 && first != 0xFFFFFFFFu) atomicMin(&sh.first, first);
    __syncthreads();
    for (int i = tid, e = 0; i < n; i += kThreads, ++e)
        if (gone >> e & 1) list.key[i] = 0;
    constexpr int PER = kBins / kThreads;
    uint64_t mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += sh.weight[tid * PER + i];
    block_scan(sh, 0, mine, &bc, &bw, &left, &total);
    const double target = (double)u * (double)total;
    uint64_t before = bw;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint64_t next = before + sh.weight[tid * PER + i];
        if (!((double)before > target) && (double)next > target) {
            sh.seg = tid * PER + i;
            sh.seg_before = before;
        }
        before = next;
    }
    __syncthreads();
    // the token inside its step, of whose tokens (V / kBins at most) one
    // thread each sums the ones before; u = 0 takes the first that is kept
    static_assert(kSampleMaxVocab / kBins <= kThreads, "a thread for every token of a step");
    const uint32_t seg = (uint32_t)sh.seg;
    for (int i = tid; i < n; i += kThreads) {
        const uint32_t key = list.key[i], at = list.idx[i];
        if (key == 0 || (u > 0.0f ? at >> shift != seg : at != sh.first)) continue;
        const uint32_t place = atomicAdd(&sh.n, 1u);
        sh.count[place] = (uint32_t)i;
        sh.weight[place] = (unsigned long long)r.fixed(key);
    }
    __syncthreads();
    const int m = (int)sh.n;
    if (tid >= m) return;
    const uint32_t key = list.key[sh.count[tid]], at = list.idx[sh.count[tid]];
    uint64_t past = sh.seg_before;
    for (int j = 0; j < m; ++j)
        if (list.idx[sh.count[j]] < at) past += sh.weight[j];
    if (u > 0.0f && ((double)past > target || !((double)(past + sh.weight[tid]) > target))) return;
    *token = (int32_t)at;
    if (logprob) *logprob = (float)log(r.weight(key) / r.of_units(total));
}

template <class L>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
    __shared__ Shared sh;
    extern __shared__ unsigned long long seg_mem[];  // the list, or per segment of the row: weight, then ties
    List& list = *reinterpret_cast<List*>(seg_mem);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int V = a.V;
    const int64_t b = blockIdx.x;
    const void* row = static_cast<const typename L::raw*>(a.logits) + b * a.row_stride;
    constexpr int VEC = L::VEC, SEG = 64 * VEC;

    // largest logit
    if (tid == 0) {
        sh.best = 0;
        sh.first = 0xFFFFFFFFu;
        sh.n = 0;
    }
    __syncthreads();
    // One pass takes the largest logits of two halves of each thread's share
    // (every value updates a maximum in `pre`, two instructions each).  A long
    // row with min-p begins its list in the same pass: the tokens that pass
    // min-p pass it against the largest logit of the row's first round too.
    float most[2] = {-INFINITY, -INFINITY};
    const auto largest = [&](float x, int e) {
        float& m = most[e & 1];
        m = x > m ? x : m;
        return false;
    };
    const auto workgroup_best = [&] {
        uint32_t best = key_of(fmaxf(most[0], most[1]));
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) best = max(best, (uint32_t)__shfl_xor((int)best, d, 64));
        if (lane == 0) atomicMax(&sh.best, best);
        __syncthreads();
        return sh.best;
    };
    constexpr int ROUND = L::FLIGHT * VEC * kThreads;
    const float T = a.temperature ? a.temperature[b] : 1.0f;
    const float min_p = a.min_p ? a.min_p[b] : 0.0f;
    const double min_w = min_p > 0.0f ? (double)min_p : 0.0;
    const bool early = V > 2 * ROUND && T > 0.0f && min_p > 0.0f && min_p <= 1.0f;
    if (early) {
        each_logit<L, L::FLIGHT>(row, V, largest, [](float, int) {}, 0, ROUND);
        Row first;
        first.kmax = workgroup_best();
        first.max = (double)logit_of(first.kmax);
        // without a logit above -inf in that round: every finite one
        const float x0 = logit_of(first.kmax > 0x007FFFFFu ? floor_of(first, (double)T, min_w) : 0x00800000u);
        each_logit<L, L::FLIGHT>(row, V, [&](float x, int e) {
            largest(x, e);
            return x >= x0;
        }, [&](float x, int i) { append(sh, list, key_of(x), i); }, ROUND);
    } else {
        each_logit<L, L::FLIGHT>(row, V, largest, [](float, int) {});
    }
    workgroup_best();
    const uint32_t my_key = key_of(fmaxf(most[0], most[1]));
    Row r;
    r.kmax = sh.best;
    if (r.kmax <= 0x007FFFFFu) {  // every logit is -inf or NaN
        if (tid == 0) {
            a.tokens[b] = -1;
            if (a.logprobs) a.logprobs[b] = -INFINITY;
        }
        return;
    }
    const float p = a.top_p ? a.top_p[b] : 1.0f;
    int k = a.top_k ? a.top_k[b] : 0;
    if (k <= 0 || k > V) k = V;
    float u = a.u[b];
    u = u > 0.0f ? fminf(u, 0.99999994f) : 0.0f;
    if (!(T > 0.0f) || k == 1 || !(p > 0.0f) || !(min_p <= 1.0f)) {  // the best token alone is kept
        const float x0 = logit_of(r.kmax);
        uint32_t at = 0xFFFFFFFFu;
        if (my_key == r.kmax)
            each_logit<L, L::FLIGHT>(row, V, [&](float x, int) { return x == x0; }, [&](float, int i) { at = min(at, (uint32_t)i); });
        if (at != 0xFFFFFFFFu) atomicMin(&sh.first, at);
        __syncthreads();
        if (tid == 0) {
            a.tokens[b] = (int32_t)sh.first;
            if (a.logprobs) a.logprobs[b] = 0.0f;
        }
        return;
    }
    r.max = (double)logit_of(r.kmax);
    r.per_t = 1.4426950408889634 / (double)T;
    r.fix = a.fix;

    // the cut: tokens with keys above `ckey`, and the first `cties` with it
    uint32_t ckey = 0, cties = 0;
    const bool by_k = k < V, by_p = p < 1.0f;
    const int digits[3] = {11, 11, 10};

    // A list of every token that can be kept, where a bound of their logits is
    // known: the whole of a short row, the best k, the ones of min_p
    uint32_t bound = 0;
    if (V <= kList) bound = 0x00800000u;
    if (V > kFew) {
        if (min_w > 0.0) bound = max(bound, floor_of(r, (double)T, min_w));
        if (by_k && k <= kThreads) bound = max(bound, floor_of_best(sh, r, most, (uint32_t)k));
    }
    bool listed = false;
    if (bound) {
        const float x0 = logit_of(bound);
        // of the list begun above, what the first round adds; otherwise, or if it overflowed, all of it
        const bool begun = early && sh.n <= (uint32_t)kList;
        __syncthreads();
        if (!begun && tid == 0) sh.n = 0;
        __syncthreads();
        each_logit<L, L::FLIGHT>(row, V, [&](float x, int) { return x >= x0; },
                                 [&](float x, int i) { append(sh, list, key_of(x), i); }, 0, begun ? ROUND : INT32_MAX);
        __syncthreads();
        listed = sh.n <= (uint32_t)kList;
        if (begun && listed && sh.n > 64u) {
            // the list was begun with a lower bound: what this one leaves of it
            constexpr int PER = kList / kThreads;
            uint32_t keys[PER], at[PER];
            const int n = (int)sh.n;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int i = tid + e * kThreads;
                keys[e] = i < n ? list.key[i] : 0u;
                at[e] = i < n ? list.idx[i] : 0u;
            }
            __syncthreads();
            if (tid == 0) sh.n = 0;
            __syncthreads();
#pragma unroll
            for (int e = 0; e < PER; ++e)
                if (keys[e] >= bound) append(sh, list, keys[e], (int)at[e]);
            __syncthreads();
        }
    }
    if (listed && sh.n <= (uint32_t)kFew) {
        draw_from_few(sh, list, (int)sh.n, r, min_w, k, p, u, a.tokens + b, a.logprobs ? a.logprobs + b : nullptr);
        return;
    }
    if (listed) {
        draw_from_list(sh, list, (int)sh.n, r, min_w, k, by_k, p, u, V, a.tokens + b, a.logprobs ? a.logprobs + b : nullptr);
        return;
    }

    bool cut_found = false;
    if (by_p && !by_k) {
        // the step of the logits in which the cut lies, then its tokens as a list
        const float step = r.step(T);
        __syncthreads();
        for (int i = tid; i < kBins; i += kThreads) {
            sh.count[i] = 0;
            sh.weight[i] = 0;
        }
        if (tid == 0) sh.n = 0;
        __syncthreads();
        // Tokens of less than (1 - p) / V of the total (at least 1, the best
        // token's weight) add up to less than 1 - p of it: they lie past the
        // cut, and only count in the total.
        const uint64_t small = r.fixed((1.0 - (double)p) / (double)V * 0.999);
        uint64_t rest = 0;
        each_logit<L, 2>(row, V, [](float, int) { return true; }, [&](float x, int) {
            const uint32_t key = key_of(x);
            const double w = r.weight(key);
            const uint64_t f = r.fixed(w);
            if (w < min_w) return;
            if (f < small || f == 0) {
                rest += f;
                return;
            }
            const int bin = r.bin(key, step);
            atomicAdd(&sh.count[bin], 1u);
            atomicAdd(&sh.weight[bin], (unsigned long long)f);
        });
        uint32_t none_c, all_c;
        uint64_t none_w, all_rest;
        block_scan(sh, 0u, rest, &none_c, &none_w, &all_c, &all_rest);
        __syncthreads();
        Cut none{0, 0, 0, 0}, cut{0, 0, 0, 0};
        uint64_t total = 0;
        search(sh, none, 0, true, 0xFFFFFFFFu, 0.0, &total);
        const double limit = (double)p * (double)(total + all_rest);
        __syncthreads();
        if (search(sh, cut, 0, false, 0, limit, nullptr)) {
            const int bin = (int)sh.bin;
            const Cut above{0, 0, sh.before_c, sh.before_w};
            // the step's ends, a little wider than their rounding
            const float lo = bin == 0 ? -INFINITY : r.step_end(bin, step);
            const float hi = bin == kBins - 1 ? INFINITY : r.step_end(bin + 1, step) + (fabsf(r.top()) + 64.0f) * 2e-6f;
            each_logit<L, L::FLIGHT>(row, V, [&](float x, int) { return x >= lo && x <= hi; }, [&](float x, int i) {
                const uint32_t key = key_of(x);
                if (key <= 0x007FFFFFu || r.bin(key, step) != bin) return;
                const double w = r.weight(key);
                const uint64_t f = r.fixed(w);
                if (w >= min_w && f >= small && f != 0) append(sh, list, key, i);
            });
            __syncthreads();
            if (sh.n <= (uint32_t)kList) {
                const int n = (int)sh.n;
                cut = above;
                bool in = true;
                for (int d = 0; d < 3 && in; ++d) {
                    histogram_list(sh, list, n, r, cut, digits[d], 0);
                    in = search(sh, cut, digits[d], false, 0, limit, nullptr);
                }
                cut_found = in;
                if (in) {
                    ckey = cut.prefix;
                    cties = ties_in(r, cut, limit);
                }
            }
        }
        __syncthreads();  // the list's memory is the segments' from here on
    }
    if (!cut_found && (by_k || by_p)) {
        Cut root{0, 0, 0, 0};
        uint64_t total = 0;
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
                total = cut.w + cties * r.fixed(ckey);
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
                uint32_t ties = ties_in(r, cut, limit);
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
        w = wave_scan(w);
        if (__any(ties != 0)) ties = wave_scan(ties);
        if (lane == 63) {
            seg_w[s] = w;
            seg_t[s] = ties;
        }
    }
    for (int d = 32; d > 0; d >>= 1) first = min(first, (uint32_t)__shfl_xor((int)first, d, 64));
    if (lane == 0) atomicMin(&sh.first, first);
    __syncthreads();
    const uint64_t one = ckey ? r.fixed(ckey) : 0;
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
            if (a.logprobs) a.logprobs[b] = (float)log(r.weight(key[e]) / r.of_units(all_w));
        }
        before = next;
    }
    if (u == 0.0f && lane == 0) {
        const uint32_t f = sh.first;
        a.tokens[b] = (int32_t)f;
        if (a.logprobs) a.logprobs[b] = (float)log(r.weight(key_of(L::one(row, f))) / r.of_units(all_w));
    }
}

}  // namespace

// The rows of one launch.
static hipError_t launch_sample_part(SampleArgs a, hipStream_t s) {
    int bits = 0;
    while (((int64_t)1 << bits) < a.V) ++bits;
    a.fix = bits < 10 ? 52 : 62 - bits;  // V weights of 2^fix at most: sums stay below 2^63
    const int seg = a.dtype == 2 ? 64 * LogitF32::VEC : 64 * 8;
    size_t lds = (size_t)((a.V + seg - 1) / seg) * 12 + 8;
    if (lds < sizeof(List)) lds = sizeof(List);
    static DeviceFlags r32, rh, rb;
    const int most = (int)(kSampleMaxVocab / 256) * 12 + 8;  // more than a list
    static_assert((kSampleMaxVocab / 256) * 12 + 8 >= sizeof(List), "the raised limit covers the list");
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

hipError_t launch_sample(const SampleArgs& args, hipStream_t s) {
    const int64_t size = args.dtype == 2 ? 4 : 2;
    const auto from = [](auto* p, int64_t b) { return p ? p + b : p; };
    for (int64_t b = 0; b < args.B; b += kMaxGroups) {
        SampleArgs a = args;
        a.B = args.B - b < kMaxGroups ? args.B - b : kMaxGroups;
        a.logits = static_cast<const char*>(a.logits) + b * a.row_stride * size;
        a.u += b;
        a.temperature = from(a.temperature, b);
        a.top_k = from(a.top_k, b);
        a.top_p = from(a.top_p, b);
        a.min_p = from(a.min_p, b);
        a.tokens += b;
        a.logprobs = from(a.logprobs, b);
        const hipError_t e = launch_sample_part(a, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace tq
