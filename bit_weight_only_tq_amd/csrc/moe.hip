// The rows of a mixture of experts around its products (experts.hip): the
// router that chooses each token's experts and sorts the pairs (token, expert)
// by expert, and the weighted sum of each token's rows afterwards.
//
// Router.  A token's logits lie in the registers of 16 lanes (64 where there are
// more than 256 experts or more than 16 chosen ones): V of them a lane, as
// integers ordered like the values.  Each of the k rounds takes the largest
// value of the group and, of the lanes that hold it, the lowest index, so equal
// logits go to the lowest index whatever their place.  exp and sums are fp32.
//
// Sorting by expert is a counting sort that keeps the pairs' order: a pair's
// place is the number of pairs of smaller experts plus the number of earlier
// pairs of its own, so the result does not depend on the schedule.  Up to 64
// tokens are routed and sorted by one workgroup; beyond, a first launch routes
// chunks of tokens and leaves each chunk's counts in the workspace, and a second
// one, a workgroup a chunk again, sums the counts before its own.  Bound by latency:
// 1 token of 8 experts 5.5 us (the kernel 4.1), 64 tokens of 64 experts, 8 chosen, 6.3
// and 65 tokens 9.9, 16383 of 128 14 us (a launch 2.5).

#include "tq_device.h"
#include "tq_internal.h"
#include "tq_tiles.h"

namespace tq {

namespace {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / kWave;

struct F32 {
    static constexpr bool kShort = false;
    static __device__ __forceinline__ float load(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
};
struct H16 {
    static constexpr bool kShort = true;
    static constexpr uint32_t kMinusInf = 0xFC00u;
    static __device__ __forceinline__ float value(uint16_t h) { return f16_bits_to_f32(h); }
};
struct B16 {
    static constexpr bool kShort = true;
    static constexpr uint32_t kMinusInf = 0xFF80u;
    static __device__ __forceinline__ float value(uint16_t h) { return bf16_bits_to_f32(h); }
};

// Integers ordered like the values; 0 for what is never chosen (NaN, -inf).  For a
// 16-bit type the same with its own 16 bits.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 is 0
    if (!(x > -__builtin_inff())) return 0u;
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint32_t order16_of(uint16_t h, uint32_t minus_inf) {
    const uint32_t u = (h & 0x7FFFu) ? h : 0u;  // -0 is 0
    const uint32_t inf = minus_inf & 0x7FFFu;
    if ((u & 0x7FFFu) > inf || u == minus_inf) return 0u;
    return (u >> 15) ? ~u & 0xFFFFu : (u | 0x8000u);
}
__device__ __forceinline__ uint16_t bits16_of(uint32_t o) { return (uint16_t)((o >> 15) ? (o & 0x7FFFu) : ~o); }
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float((o >> 31) ? (o & 0x7FFFFFFFu) : ~o);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

// Over the LANES lanes of a token's group (16: one row of lanes; 64: the wave);
// every lane has the result.  Swaps of neighbours and pairs, then mirrors.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    v = umax(v, dpp<0xB1>(v));
    v = umax(v, dpp<0x4E>(v));
    v = umax(v, dpp<0x141>(v));
    v = umax(v, dpp<0x140>(v));
    if constexpr (LANES == 64) {
        v = umax(v, (uint32_t)__shfl_xor((int)v, 16, kWave));
        v = umax(v, (uint32_t)__shfl_xor((int)v, 32, kWave));
    }
    return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
    v = umin(v, dpp<0xB1>(v));
    v = umin(v, dpp<0x4E>(v));
    v = umin(v, dpp<0x141>(v));
    v = umin(v, dpp<0x140>(v));
    if constexpr (LANES == 64) {
        v = umin(v, (uint32_t)__shfl_xor((int)v, 16, kWave));
        v = umin(v, (uint32_t)__shfl_xor((int)v, 32, kWave));
    }
    return v;
}
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
    if constexpr (LANES == 64) return wave_sum(v);
    else return row16_sum(v);
}

// A lane's logits of token t, experts sub + LANES v, and the best of what is left.
// 16-bit types: value and index (downwards) in one word, so a round is one maximum.
// fp32: the largest value, then the lowest index of the lanes that hold it.
struct Best {
    uint32_t key;    // order of the value, 0: none
    uint32_t index;
};
template <class L, int LANES, int V>
struct Logits {
    uint32_t key[V];
    int sub;
    __device__ __forceinline__ void load(const RouteArgs& a, int64_t row) {
        sub = (int)threadIdx.x & (LANES - 1);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = sub + LANES * v;
            const bool in = e < a.E;
            if constexpr (L::kShort) {
                const uint32_t o = in ? order16_of(static_cast<const uint16_t*>(a.logits)[row + e], L::kMinusInf) : 0u;
                key[v] = o ? (o << 16) | (0xFFFFu - (uint32_t)e) : 0u;
            } else {
                key[v] = in ? order_of(L::load(a.logits, row + e)) : 0u;
            }
        }
    }
    static __device__ __forceinline__ float value(uint32_t k) {
        if constexpr (L::kShort) return L::value(bits16_of(k));
        else return value_of(k);
    }
    // order of a key that is not 0
    __device__ __forceinline__ uint32_t order(int v) const { return L::kShort ? key[v] >> 16 : key[v]; }
    __device__ __forceinline__ Best take() {
        uint32_t best = 0u;
        if constexpr (L::kShort) {
#pragma unroll
            for (int v = 0; v < V; ++v) best = umax(best, key[v]);
            best = group_max<LANES>(best);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (key[v] == best) key[v] = 0u;
            return Best{best >> 16, 0xFFFFu - (best & 0xFFFFu)};
        } else {
            int at = 0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (key[v] > best) best = key[v], at = v;
            const uint32_t m = group_max<LANES>(best);
            const uint32_t i = group_min<LANES>(m && best == m ? (uint32_t)(sub + LANES * at) : 0xFFFFFFFFu);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if ((uint32_t)(sub + LANES * v) == i) key[v] = 0u;
            return Best{m, i};
        }
    }
};

// Routes token t (the same for the LANES lanes of a group; t >= T does nothing
// but goes along): writes its experts and weights; -> lane j < k has expert j,
// E where there is none.
template <class L, int LANES, int V>
__device__ __forceinline__ int route_token(const RouteArgs& a, int64_t t) {
    typedef Logits<L, LANES, V> Keys;
    const int sub = (int)threadIdx.x & (LANES - 1);
    const bool live = t < a.T;
    Keys keys;
    keys.load(a, (live ? t : a.T - 1) * a.row_stride);
    uint32_t top = 0u, mine = 0u;
    uint32_t expert = (uint32_t)a.E;
    float all = 0.0f;
    if (!a.renormalize) {  // the sum over all, before any is taken
        uint32_t m = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) m = umax(m, keys.key[v] ? keys.order(v) : 0u);
        top = group_max<LANES>(m);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (keys.key[v]) all += keys.order(v) == top ? 1.0f : expf(Keys::value(keys.order(v)) - Keys::value(top));
        all = group_sum<LANES>(all);
    }
    for (int j = 0; j < a.k; ++j) {
        const Best b = keys.take();
        if (j == 0) top = b.key;
        if (sub == j && b.key) mine = b.key, expert = b.index;
    }
    // equal largest logits, infinite ones among them, weigh the same
    const float w = mine == 0u ? 0.0f : mine == top ? 1.0f : expf(Keys::value(mine) - Keys::value(top));
    const float total = a.renormalize ? group_sum<LANES>(w) : all;
    if (live && sub < a.k) {
        a.experts[t * a.k + sub] = mine ? (int32_t)expert : -1;
        a.weights[t * a.k + sub] = mine ? w / total : 0.0f;
    }
    return (int)expert;
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = (uint32_t)__shfl_up((int)v, d, kWave);
        if (lane >= d) v += o;
    }
    return v;
}

__device__ __forceinline__ uint32_t wave_sum_u32(uint32_t v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += (uint32_t)__shfl_xor((int)v, d, kWave);
    return v;
}

// Exclusive sum over the workgroup's threads; *total has the whole.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* scratch, uint32_t* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t in = wave_scan(v);
    if (lane == 63) scratch[wave] = in;
    __syncthreads();
    uint32_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) {
        const uint32_t s = scratch[w];
        if (w < wave) before += s;
        sum += s;
    }
    __syncthreads();
    *total = sum;
    return before + in - v;
}

// The pairs [p0, p0 + n) are dealt to the waves in contiguous shares of whole
// 64s.  hist [waves][E + 1] first counts each share's pairs by class (expert, E:
// none), then holds the next place of each class in each share; places are taken
// 64 pairs at a time, a lane's rank among its class's lanes by ballots of the
// class's bits.  base(e): the class's first place of these pairs.
template <class Id, class Base>
__device__ __forceinline__ void sort_pairs(const RouteArgs& a, int64_t p0, int64_t n, uint32_t* hist, Id id_of, Base base) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int E1 = a.E + 1;
    const int64_t share = (n + kRouteThreads - 1) / kRouteThreads * 64;
    const int64_t from = wave * share < n ? wave * share : n;
    const int64_t to = from + share < n ? from + share : n;
    for (int i = threadIdx.x; i < kRouteWaves * E1; i += kRouteThreads) hist[i] = 0;
    __syncthreads();
    for (int64_t i = from + lane; i < to; i += 64) atomicAdd(&hist[wave * E1 + id_of(i)], 1u);
    __syncthreads();
    for (int e = threadIdx.x; e < E1; e += kRouteThreads) {
        uint32_t at = base(e), c[kRouteWaves];
#pragma unroll
        for (int w = 0; w < kRouteWaves; ++w) c[w] = hist[w * E1 + e];
#pragma unroll
        for (int w = 0; w < kRouteWaves; ++w) {
            hist[w * E1 + e] = at;
            at += c[w];
        }
    }
    __syncthreads();
    volatile uint32_t* next = hist + wave * E1;
    int bits = 0;
    while ((1 << bits) < E1) ++bits;
    for (int64_t i0 = from; i0 < to; i0 += 64) {
        const bool in = i0 + lane < to;
        const int id = in ? id_of(i0 + lane) : 0;
        uint64_t same = __ballot(in);
        for (int b = 0; b < bits; ++b) {
            const uint64_t one = __ballot((id >> b) & 1);
            same &= ((id >> b) & 1) ? one : ~one;
        }
        if (in) {
            const int rank = __popcll(same & ((1ull << lane) - 1));
            const uint32_t at = next[id] + (uint32_t)rank;
            __builtin_amdgcn_wave_barrier();
            if (rank == 0) next[id] = at + (uint32_t)__popcll(same);
            const int64_t pair = p0 + i0 + lane;
            a.rows[at] = (int32_t)pair;
            a.places[pair] = id < a.E ? (int32_t)at : -1;
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Up to 64 tokens: routing and sorting in one workgroup.
template <class L, int LANES, int V>
__global__ __launch_bounds__(kRouteThreads) void route_one_kernel(RouteArgs a) {
    extern __shared__ uint32_t smem_route[];
    uint32_t* hist = smem_route;                                  // [waves][E + 1]
    uint32_t* first = hist + kRouteWaves * (a.E + 1);             // [E + 1]
    uint32_t* scratch = first + a.E + 1;                          // [waves]
    int16_t* ids = reinterpret_cast<int16_t*>(scratch + kRouteWaves);  // [T k]
    constexpr int kTokens = kRouteThreads / LANES;
    const int sub = (int)threadIdx.x & (LANES - 1);
    for (int t0 = 0; t0 < (int)a.T; t0 += kTokens) {
        const int t = t0 + (int)threadIdx.x / LANES;
        const int e = route_token<L, LANES, V>(a, t);
        if (t < (int)a.T && sub < a.k) ids[t * a.k + sub] = (int16_t)e;
    }
    const int n = (int)a.T * a.k;
    for (int e = threadIdx.x; e <= a.E; e += kRouteThreads) first[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kRouteThreads) atomicAdd(&first[ids[i]], 1u);
    __syncthreads();
    uint32_t total;
    const uint32_t before = block_scan((int)threadIdx.x < a.E ? first[threadIdx.x] : 0u, scratch, &total);
    if ((int)threadIdx.x < a.E) {
        first[threadIdx.x] = before;
        a.offsets[threadIdx.x] = (int32_t)before;
    }
    if (threadIdx.x == 0) {
        first[a.E] = total;
        a.offsets[a.E] = (int32_t)total;
    }
    __syncthreads();
    sort_pairs(a, 0, n, hist, [&](int64_t i) { return (int)ids[i]; }, [&](int e) { return first[e]; });
}

// A chunk of tokens a workgroup: routing, and the chunk's counts by expert.
template <class L, int LANES, int V>
__global__ __launch_bounds__(kRouteThreads) void route_chunk_kernel(RouteArgs a) {
    __shared__ uint32_t count[kRouteMaxExperts + 1];
    constexpr int kTokens = kRouteThreads / LANES;
    const int sub = (int)threadIdx.x & (LANES - 1);
    for (int e = threadIdx.x; e <= a.E; e += kRouteThreads) count[e] = 0;
    __syncthreads();
    const int64_t from = (int64_t)blockIdx.x * a.chunk;
    const int64_t to = from + a.chunk < a.T ? from + a.chunk : a.T;
    for (int64_t t0 = from; t0 < to; t0 += kTokens) {
        const int64_t t = t0 + (int)threadIdx.x / LANES;
        const int e = route_token<L, LANES, V>(a, t < to ? t : a.T);
        if (t < to && sub < a.k) atomicAdd(&count[e], 1u);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) a.counts[(int64_t)blockIdx.x * a.E + e] = count[e];
}

// The places of a chunk's pairs.  Thread (s, e) sums the counts of expert e over
// the chunks s, s + S, ...: all of them and those before its own.
__global__ __launch_bounds__(kRouteThreads) void sort_chunk_kernel(RouteArgs a) {
    extern __shared__ uint32_t smem_sort[];
    uint32_t* hist = smem_sort;                           // [waves][E + 1]
    uint32_t* first = hist + kRouteWaves * (a.E + 1);     // [E + 1]
    uint32_t* scratch = first + a.E + 1;                  // [waves]
    uint32_t* part = scratch + kRouteWaves;               // [2][1024]
    int16_t* held = reinterpret_cast<int16_t*>(part + 2 * kRouteThreads);  // [1024] the chunk's experts, if they fit
    const int64_t t0 = (int64_t)blockIdx.x * a.chunk;
    const int64_t t1 = t0 + a.chunk < a.T ? t0 + a.chunk : a.T;
    const int32_t* ids = a.experts + t0 * a.k;
    const int64_t n = (t1 - t0) * a.k;
    int id = 0;
    if (n <= kRouteThreads && threadIdx.x < n) id = ids[threadIdx.x];  // beside the counts
    int width = 16;
    while (width < a.E) width *= 2;
    const int S = kRouteThreads / width, s = (int)threadIdx.x / width, e = (int)threadIdx.x & (width - 1);
    const int chunks = (int)gridDim.x, mine = (int)blockIdx.x;
    uint32_t before = 0, all = 0;
    if (e < a.E) {
        const uint32_t* p = a.counts + e;
#pragma unroll 16
        for (int c = s; c < chunks; c += S) {
            const uint32_t v = p[(int64_t)c * a.E];
            all += v;
            if (c < mine) before += v;
        }
    }
    part[threadIdx.x] = before;
    part[kRouteThreads + threadIdx.x] = all;
    __syncthreads();
    before = all = 0;
    if ((int)threadIdx.x < a.E) {  // thread e of the first S: all slices of expert e
        for (int i = 0; i < S; ++i) {
            before += part[i * width + threadIdx.x];
            all += part[kRouteThreads + i * width + threadIdx.x];
        }
    }
    // places of the experts' first pairs, and how many of the pairs before this chunk
    // have an expert
    uint32_t total, chosen_before = wave_sum_u32(before);
    if ((threadIdx.x & 63) == 0) hist[threadIdx.x >> 6] = chosen_before;  // read behind block_scan's barriers
    const uint32_t start = block_scan(all, scratch, &total);
    chosen_before = 0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) chosen_before += hist[w];
    if ((int)threadIdx.x < a.E) {
        first[threadIdx.x] = start + before;
        if (mine == 0) a.offsets[threadIdx.x] = (int32_t)start;
    }
    if (threadIdx.x == 0) {
        first[a.E] = total + (uint32_t)(t0 * a.k) - chosen_before;
        if (mine == 0) a.offsets[a.E] = (int32_t)total;
    }
    if (n <= kRouteThreads) {
        if (threadIdx.x < n) held[threadIdx.x] = (int16_t)(id < 0 ? a.E : id);
        __syncthreads();
        sort_pairs(a, t0 * a.k, n, hist, [&](int64_t i) { return (int)held[i]; }, [&](int c) { return first[c]; });
    } else {
        __syncthreads();
        sort_pairs(a, t0 * a.k, n, hist,
                   [&](int64_t i) {
                       const int e1 = ids[i];
                       return e1 < 0 ? a.E : e1;
                   },
                   [&](int c) { return first[c]; });
    }
}

template <class L, int LANES, int V>
hipError_t route_variant(const RouteArgs& a, hipStream_t s) {
    const size_t lds = (size_t)(kRouteWaves * (a.E + 1) + a.E + 1 + kRouteWaves) * 4;
    static DeviceFlags one_set, sort_set;
    hipError_t e;
    if (a.chunk == 0) {
        const size_t bytes = lds + (((size_t)a.T * a.k * 2 + 3) & ~(size_t)3);
        e = raise_lds_limit(reinterpret_cast<const void*>(&route_one_kernel<L, LANES, V>), kRouteMaxLds, one_set);
        if (e != hipSuccess) return e;
        route_one_kernel<L, LANES, V><<<1, kRouteThreads, bytes, s>>>(a);
        return hipGetLastError();
    }
    const unsigned chunks = (unsigned)((a.T + a.chunk - 1) / a.chunk);
    route_chunk_kernel<L, LANES, V><<<chunks, kRouteThreads, 0, s>>>(a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    e = raise_lds_limit(reinterpret_cast<const void*>(&sort_chunk_kernel), kRouteMaxLds, sort_set);
    if (e != hipSuccess) return e;
    sort_chunk_kernel<<<chunks, kRouteThreads, lds + 2 * kRouteThreads * 4 + kRouteThreads * 2, s>>>(a);
    return hipGetLastError();
}

// 16 lanes a token as long as they hold its logits and its choices: 2048 tokens of
// 64 experts, 8 chosen, 10.5 us with 16 lanes and 28 with 64; 16383 of 200, 21 and 36.
template <class L>
hipError_t route_type(const RouteArgs& a, hipStream_t s) {
    if (a.E > 256 || a.k > 16) return route_variant<L, 64, 16>(a, s);
    if (a.E > 128) return route_variant<L, 16, 16>(a, s);
    if (a.E > 64) return route_variant<L, 16, 8>(a, s);
    return route_variant<L, 16, 4>(a, s);
}

// ------------------------------------------------------------------ combine

template <class T>
__device__ __forceinline__ void add8(float (&acc)[8], const uint4& v, float w) {
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(w, T::to_f32((uint16_t)d[i]), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w, T::to_f32((uint16_t)(d[i] >> 16)), acc[2 * i + 1]);
    }
}

// Eight values at any address (the memory mode of this platform allows vectors
// there), or the n of them that a row still has.
struct __attribute__((packed, aligned(2))) Eight {
    uint32_t d[4];
};
template <bool WHOLE>
__device__ __forceinline__ uint4 load8(const uint16_t* p, int n) {
    if constexpr (WHOLE) {
        const Eight v = *reinterpret_cast<const Eight*>(p);
        return make_uint4(v.d[0], v.d[1], v.d[2], v.d[3]);
    } else {
        uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) d[i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
        return make_uint4(d[0], d[1], d[2], d[3]);
    }
}

template <class T, bool WHOLE>
__device__ __forceinline__ void combine_columns(const CombineArgs& a, int64_t t, int64_t c, int n) {
    const int32_t* places = a.places + t * a.k;
    const float* weights = a.weights + t * a.k;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    if (a.add) add8<T>(acc, load8<WHOLE>(a.add + t * a.add_stride + c, n), 1.0f);
    constexpr int U = WHOLE ? 8 : 1;  // rows in flight
    for (int j0 = 0; j0 < a.k; j0 += U) {
        int32_t p[U];
        float w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u < a.k ? j0 + u : a.k - 1;
            p[u] = places[j];
            w[u] = weights[j];
        }
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u >= a.k) break;
            const bool in = p[u] >= 0 && p[u] < a.P;
            v[u] = load8<WHOLE>(a.y + (int64_t)(in ? p[u] : 0) * a.N + c, n);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u >= a.k) break;
            if (p[u] >= 0 && p[u] < a.P) add8<T>(acc, v[u], w[u]);
        }
    }
    uint16_t* dst = a.out + t * a.N + c;
    Eight out;
#pragma unroll
    for (int i = 0; i < 4; ++i) out.d[i] = round_pair<T>(acc[2 * i], acc[2 * i + 1]);
    if constexpr (WHOLE) {
        *reinterpret_cast<Eight*>(dst) = out;
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) dst[i] = (uint16_t)(out.d[i / 2] >> (16 * (i % 2)));
    }
}

// out[t] = add[t] + sum over j of weights[t, j] y[places[t, j]], in fp32, in the
// order of j, rounded once.  Bound by the read of the rows.  A thread has 8 columns
// of one token (the last of a row what is left of it); the k rows' loads are
// independent and eight of them in flight together.  Measured: 8191 tokens, 6 rows of
// 2048, 45 us, 5.2 TB/s; one token 4.6 us, a launch.
template <class T>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
    const int64_t cols = (a.N + 7) / 8;
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (item >= a.T * cols) return;
    const int64_t t = item / cols, c = (item - t * cols) * 8;
    if (c + 8 <= a.N) combine_columns<T, true>(a, t, c, 8);
    else combine_columns<T, false>(a, t, c, (int)(a.N - c));
}

template <class T>
hipError_t combine_type(const CombineArgs& a, hipStream_t s) {
    const int64_t per_token = (a.N + 7) / 8;
    // whole tokens a launch, fewer than 2^32 threads each
    const int64_t most = kMaxGroups * 256 / per_token;
    for (int64_t t = 0; t < a.T; t += most) {
        CombineArgs b = a;
        b.T = a.T - t < most ? a.T - t : most;
        b.places = a.places + t * a.k;
        b.weights = a.weights + t * a.k;
        b.out = a.out + t * a.N;
        if (a.add) b.add = a.add + t * a.add_stride;
        const unsigned groups = (unsigned)((b.T * per_token + 255) / 256);
        combine_kernel<T><<<groups, 256, 0, s>>>(b);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

int64_t route_chunk(int64_t T) {
    if (T <= kRouteOneTokens) return 0;
    const int64_t c = (T + kRouteMaxChunks - 1) / kRouteMaxChunks;
    return c <= 64 ? 64 : (c + 63) / 64 * 64;
}

hipError_t launch_moe_route(const RouteArgs& args, hipStream_t s) {
    RouteArgs a = args;
    a.chunk = route_chunk(a.T);
    switch (a.dtype) {
        case 0: return route_type<H16>(a, s);
        case 1: return route_type<B16>(a, s);
        default: return route_type<F32>(a, s);
    }
}

hipError_t launch_moe_combine(const CombineArgs& args, hipStream_t s) {
    CombineArgs a = args;
    if (a.P == 0) a.k = 0;  // no place has a row
    return a.bf16 ? combine_type<BF16>(a, s) : combine_type<F16>(a, s);
}

}  // namespace tq
