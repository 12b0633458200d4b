// Attention of each request's new tokens over the pages of its cache.
//
// For query row i (position p) and key j of its request, with the scores
// t_ij = scale log2(e) q_i . k_j of the visible keys (j <= p; with a window
// w: p - j < w or j < sinks),
//   out_i = sum_j 2^(t_ij - m_i) v_j / l_i,   l_i = sum_j 2^(t_ij - m_i),
//   lse_i = ln 2 (m_i + log2 l_i),
// in one pass over the keys with a running m_i near the maximum (any m_i gives
// the same result).  Maxima, sums and outputs are held in fp32; the weights
// 2^(t - m) are rounded to the cache's type, as the output is.  The matrix
// cores take both operands of a product in one type, and a second product with
// what a rounding leaves would double the work on V.  The rounding is what
// the result loses against one in fp32: its error against fp64 is 1.04 to 1.4
// times as large.
//
// The query heads that share a KV head are rows of one matrix: row r of a
// request and KV head is token r / G, head r % G of the group of G.

#include <math.h>

#include <type_traits>

#include "tq_device.h"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr float kLn2 = 0.69314718055994531f;

// Element types: the matrix products, the rounding of two weights to a
// dword, the exponent step that carries a non-finite value's magnitude into
// bit 15, and kLift: m_i is held that far below the running maximum.  fp16 has
// its full step down to 2^-14 and nothing below 2^-25, so with m_i the maximum
// itself many small weights behind a large one lost their bits, or vanished,
// while l_i summed them whole.  2^7 is the room it has: weights reach 2^8 times
// what they are at the maximum before m_i is raised, and 2^15 fits.
struct AttnF16 {
    static __device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack2(float x, float y) {
        return __builtin_bit_cast(uint32_t, f16x2{(_Float16)x, (_Float16)y});
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w).x; }
    static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w).y; }
    static constexpr uint32_t kExpStep = 0x04000400u;
    static constexpr float kLift = 7.f;
};
struct AttnBF16 {
    static __device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack2(float x, float y) {
        return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x, (__bf16)y});
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
    static constexpr uint32_t kExpStep = 0x00800080u;
    static constexpr float kLift = 0.f;
};

template <class E>
__device__ __forceinline__ uint32_t nonfinite(uint32_t w) {
    return ((w & 0x7FFF7FFFu) + E::kExpStep) & 0x80008000u;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Page tables are read as constant memory, through the scalar cache: such loads
// wait for no vector load or DMA in flight.
typedef const __attribute__((address_space(4))) int32_t* const_i32;

// One request as the kernels see it: its new tokens and the keys in reach of
// its table.  A request whose offsets do not lie in [0, T] has no tokens.
struct Request {
    int t0, n;       // first token, number of new tokens
    int first;       // position of the first new token
    int keys;        // keys that can be read
};
__device__ __forceinline__ Request request_of(const AttnArgs& a, int b) {
    Request r;
    const int c0 = a.cu[b], c1 = a.cu[b + 1];
    const int kv = max(a.kv[b], 0);
    const bool ok = c0 >= 0 && c1 <= a.T && c1 > c0;
    r.t0 = c0;
    r.n = ok ? c1 - c0 : 0;
    r.first = kv - r.n;
    const int64_t reach = (int64_t)a.width << a.shift;
    r.keys = kv < reach ? kv : (int)reach;
    return r;
}

// The key blocks (2^LOG keys, aligned) a run of positions p0 .. p1 can see:
// `head` blocks of sinks from key 0, then [main0, main1).
struct Blocks {
    int head, main0, count;
    __device__ __forceinline__ int at(int i) const { return i < head ? i : main0 + (i - head); }
};
template <int LOG>
__device__ __forceinline__ Blocks blocks_of(const AttnArgs& a, const Request& r, int p0, int p1) {
    Blocks k;
    const int end = min(p1, r.keys - 1) + 1;  // first key nobody sees
    const int main1 = end > 0 ? (int)(((uint32_t)end + (1u << LOG) - 1u) >> LOG) : 0;
    int lo = 0;
    if (a.window > 0) lo = (int)max((int64_t)p0 - a.window + 1, (int64_t)0);
    k.main0 = min(lo >> LOG, main1);
    k.head = min((int)(((uint32_t)a.sinks + (1u << LOG) - 1u) >> LOG), k.main0);
    k.count = k.head + (main1 - k.main0);
    return k;
}
__device__ __forceinline__ bool sees(const AttnArgs& a, int p, int j) {
    return j <= p && (a.window <= 0 || p - j < a.window || j < a.sinks);
}

// ---- rows kernel: 16 rows a wave.
//
// A wave takes 16 rows and runs over blocks of 32 keys with no LDS: K and V
// come from their pages into the registers in which the matrix cores want
// them.  S^T = K Q^T with the keys of a block dealt to the two 16-row tiles
// so that lane (g, c) (g = lane / 16, c = lane % 16) gets the scores of row c
// for the keys 8 g .. 8 g + 7; rounded, these are the second operand of
// O^T = V^T P^T as they stand.  V is read in whole rows (lane c holds D / 16
// consecutive values of 8 keys) and transposed by one byte-permute a dword.
// Row statistics and outputs of a row stay in the lanes of that row.
//
// Decode is bound by the read of the cache, so the waves of a workgroup take
// different key blocks, and the blocks of all requests are dealt to the
// workgroups in even shares; the last one to finish a request joins the partial
// results in order.  64 requests of 33 to 8191 keys with 64 + 8 heads of 128:
// 200 us, 5.4 TB/s of cache; two of 100001 and 131071 keys with 32 + 8 heads:
// 170 us, 5.6 TB/s (a streaming read reaches as much).  The same with splits of
// a fixed length, whose workgroups came in rounds: 226 and 187 us.
constexpr int kRowsThreads = 256;
constexpr int kWaves = kRowsThreads / 64;
constexpr int kRowsMost = 16;  // rows (new tokens times the group's heads) of a request that the rows kernel takes
constexpr int kBlockKeys = 32;

// Dword t of a lane's V values of one key.
template <int VD>
struct VRow {
    uint32_t w[VD];
};
template <int VD>
__device__ __forceinline__ VRow<VD> load_vrow(const uint16_t* p) {
    VRow<VD> r;
    if constexpr (VD == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        r.w[0] = x.x;
        r.w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < VD / 4; ++i) {
            const uint4 x = *reinterpret_cast<const uint4*>(p + 8 * i);
            r.w[4 * i] = x.x;
            r.w[4 * i + 1] = x.y;
            r.w[4 * i + 2] = x.z;
            r.w[4 * i + 3] = x.w;
        }
    }
    return r;
}

// Two values of a partial result (see store_partial), 8-byte aligned.
__device__ __forceinline__ void store_pair(float* p, float x, float y) {
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), (uint64_t)__float_as_uint(x) | (uint64_t)__float_as_uint(y) << 32,
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Joins the partial results of a workgroup tile's splits, in split order, by
// the last workgroup to arrive (256 threads): weights of the splits from their
// row statistics ([row][2] at the front of each slab), then the weighted sum
// of their outputs ([row][D] from `out_at` on).  Split s lies at slabs.at(s).
// `wgt` has room for rows * nsplit floats.
struct Slabs {
    const float *first, *base;
    int64_t stride;
    __device__ __forceinline__ const float* at(int s) const { return s == 0 ? first : base + s * stride; }
};
template <class E, int D>
__device__ __forceinline__ void join_splits(const AttnArgs& a, const Request& rq, int h, int64_t row0, int rows, int out_at,
                                            const Slabs& slabs, int nsplit, float* wgt, float* row_m, float* row_l) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, G = a.G;
    for (int row = wave; row < rows; row += 4) {
        float M = -INFINITY;
        for (int s = lane; s < nsplit; s += 64)
            M = fmaxf(M, __hip_atomic_load(slabs.at(s) + 2 * row, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
#pragma unroll
        for (int x = 32; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor(M, x, 64));
        const float ms = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        for (int s = lane; s < nsplit; s += 64) {
            const float ps = __hip_atomic_load(slabs.at(s) + 2 * row, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const float pl = __hip_atomic_load(slabs.at(s) + 2 * row + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const float f = exp2_fast(ps - ms);
            wgt[row * nsplit + s] = f;
            L += f * pl;
        }
        L = wave_sum(L);
        if (lane == 0) {
            row_m[row] = M;
            row_l[row] = L;
        }
    }
    __syncthreads();
    // Pairs of values, U pairs of RS splits in flight a thread: these loads go
    // past the L2 and take a microsecond or two each, so a join is bound by how
    // many of them wait at once.  Many rows fill that with pairs, few with splits.
    const int pairs = rows * (D / 2);
    const auto join = [&](auto units, auto round) {
        constexpr int U = decltype(units)::value, RS = decltype(round)::value;
        for (int u0 = tid; u0 < pairs; u0 += U * kRowsThreads) {
            float x0[U], x1[U];
            int rw[U], at_d[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int p = min(u0 + u * kRowsThreads, pairs - 1);
                rw[u] = p / (D / 2);
                at_d[u] = out_at + 2 * p;
                x0[u] = x1[u] = 0.f;
            }
            for (int s0 = 0; s0 < nsplit; s0 += RS) {
                uint64_t v[RS][U];
#pragma unroll
                for (int s = 0; s < RS; ++s)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        v[s][u] = __hip_atomic_load(reinterpret_cast<const uint64_t*>(slabs.at(min(s0 + s, nsplit - 1)) + at_d[u]),
                                                    __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
                for (int s = 0; s < RS; ++s)
                    if (s0 + s < nsplit) {
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const float f = wgt[rw[u] * nsplit + s0 + s];
                            x0[u] += f * __uint_as_float((uint32_t)v[s][u]);
                            x1[u] += f * __uint_as_float((uint32_t)(v[s][u] >> 32));
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u0 + u * kRowsThreads >= pairs) break;
                const float L = row_l[rw[u]];
                const int64_t r = row0 + rw[u];
                const int tok = (int)(r / G), d = at_d[u] - out_at - rw[u] * D;
                const int64_t at = (int64_t)(rq.t0 + tok) * a.Hq + h * G + (int)(r - (int64_t)tok * G);
                const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : NAN);
                *reinterpret_cast<uint32_t*>(a.out + at * D + d) = E::pack2(x0[u] * inv, x1[u] * inv);
                if (d == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : kLn2 * (row_m[rw[u]] + log2f(L));
            }
        }
    };
    using std::integral_constant;
    if (pairs > 4 * kRowsThreads) join(integral_constant<int, 8>{}, integral_constant<int, 2>{});
    else if (pairs > kRowsThreads) join(integral_constant<int, 4>{}, integral_constant<int, 4>{});
    else join(integral_constant<int, 1>{}, integral_constant<int, 16>{});
}

// Even shares: the requests' blocks lie one after another (start[b], start[B]
// in all), and every workgroup of a KV head takes as many of them, so that one
// round of workgroups ends together whatever the lengths.  -> blocks of a
// share: kShareBlocks (one a wave) at least; so many that no request has more
// than a.split_most shares; and no fewer than where the longest request's join
// costs what its blocks do.  N blocks in shares of x take 0.3 us x, and the
// join of N / x partial results, 32 KiB of them in flight for 1.5 us,
// 1.5 us rows D 4 B / 32 KiB each: x = sqrt(N rows D 6e-4).  All threads of the
// workgroup.
constexpr int kShareRequests = 1024;
constexpr int kShareBlocks = 4;
constexpr int kSplitBlocks = 8;  // calls whose requests have no more blocks are not shared out
// x / y for x >= 0, y > 0; 64-bit division is a long loop, and seldom needed.
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
    return (x | y) >> 32 == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}
template <class F>
__device__ __forceinline__ int64_t even_shares(const AttnArgs& a, int64_t* start, int64_t* word, F blocks) {
    __shared__ int64_t sums[4], most_of[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const auto share_of = [&](int64_t total, int64_t most) {
        const int64_t share = divide(total + a.workers - 1, a.workers);
        const int64_t joined = (int64_t)sqrtf((float)most * a.join_cost);
        return max(max(share, joined), max(divide(most + a.split_most - 2, a.split_most - 1), (int64_t)kShareBlocks));
    };
    if (a.B == 1) {  // nothing to add up
        const int64_t n = blocks(0);
        if (tid == 0) {
            start[0] = 0;
            start[1] = n;
        }
        __syncthreads();
        return share_of(n, n);
    }
    const int per = (a.B + kRowsThreads - 1) / kRowsThreads, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int64_t sum = 0, most = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = blocks(b);
        start[b] = sum;  // from this thread's first on
        sum += n;
        most = max(most, (int64_t)n);
    }
    int64_t upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up((long long)upto, d, 64), x = __shfl_xor((long long)most, d, 64);
        if (lane >= d) upto += o;
        most = max(most, x);
    }
    if (lane == 63) {
        sums[wave] = upto;
        most_of[wave] = most;
    }
    __syncthreads();
    int64_t before = upto - sum, total = 0;
    for (int w = 0; w < 4; ++w) {
        if (w < wave) before += sums[w];
        total += sums[w];
        most = max(most, most_of[w]);
    }
    for (int b = b0; b < b1; ++b) start[b] += before;
    if (tid == 0) {
        start[a.B] = total;
        *word = share_of(total, most);
    }
    __syncthreads();
    return *word;
}

template <class E, int D>
__global__ __launch_bounds__(kRowsThreads, D == 64 ? 3 : 2) void rows_kernel(AttnArgs a) {
    constexpr int ST = D / 32, DV = D / 16, VD = DV / 2;
    constexpr int LD = D + 4;  // LDS row stride (floats): rows of a quad of lanes fall into different banks
    __shared__ float lds_o[4 * 16 * LD];
    __shared__ float lds_ml[4 * 16 * 2];
    __shared__ float row_m[kRowsMost], row_l[kRowsMost];
    __shared__ uint32_t word;
    __shared__ int64_t start[kShareRequests + 1], share_word;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c = lane & 15;
    const int G = a.G;
    const int h = (int)(blockIdx.x % (unsigned)a.Hkv), worker = (int)(blockIdx.x / (unsigned)a.Hkv);

    // What request b asks of a KV head: its rows and the key blocks they see.
    auto rows_of = [&](const Request& rq) {
        const int64_t all = (int64_t)min(rq.n, a.max_q) * G;
        return all > a.rows_most ? 0 : (int)all;  // the tile kernel's
    };
    auto seen_by = [&](const Request& rq, int rows) { return blocks_of<5>(a, rq, rq.first, rq.first + (rows - 1) / G); };

    // This workgroup's run of blocks of all the requests' together, or all of one request's
    int b = worker;
    int64_t r0 = 0, r1 = 0, share = 1;
    if (a.workers > 0) {
        share = even_shares(a, start, &share_word, [&](int i) {
            const Request rq = request_of(a, i);
            const int rows = rows_of(rq);
            return rows > 0 ? max(seen_by(rq, rows).count, 1) : 0;
        });
        r0 = worker * share;
        r1 = min(start[a.B], r0 + share);
        if (r0 >= r1) return;
        int lo = 0, hi = a.B;  // the last request that begins at or before r0
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= r0) lo = mid;
            else hi = mid;
        }
        b = lo;
    }
    for (;; ++b) {
        if (a.workers > 0 && (b >= a.B || start[b] >= r1)) return;
        const Request rq = request_of(a, b);
        const int rows = rows_of(rq);
        if (rows == 0) {
            if (a.workers > 0) continue;
            return;
        }
        const Blocks bl = seen_by(rq, rows);
        int i0 = 0, i1 = bl.count, nsplit = 1;
        float* slab = nullptr;  // this split's partial result: [rows][2], then [rows][D]
        Slabs slabs{nullptr, nullptr, 0};
        if (a.workers > 0) {
            // A workgroup has at most two partial results: of the request its
            // run begins in, and of the one it ends in.
            const int64_t s0 = start[b], s1 = start[b + 1];
            i0 = (int)(max(r0, s0) - s0);
            i1 = min(bl.count, (int)(min(r1, s1) - s0));
            const int first = (int)divide(s0, share);
            nsplit = (int)divide(s1 - 1, share) - first + 1;
            auto slab_of = [&](int w, int which) { return a.partials + (((int64_t)w * a.Hkv + h) * 2 + which) * a.slab; };
            slab = slab_of(worker, s0 <= r0 ? 0 : 1);
            slabs = Slabs{slab_of(first, s0 > first * share ? 1 : 0), slab_of(first, 0), (int64_t)a.Hkv * 2 * a.slab};
        }

        const bool row_ok = c < rows;
        const int my_tok = (row_ok ? c : 0) / G;
        const int my_head = h * G + (row_ok ? c : 0) - my_tok * G;
        const int my_pos = row_ok ? rq.first + my_tok : INT32_MIN;
        // positions of the first and the last row
        const int tile_p0 = rq.first;
        const int tile_p1 = rq.first + (rows - 1) / G;

        uint4 qf[ST];
        {
            const uint16_t* src = a.q + (int64_t)(rq.t0 + my_tok) * a.q_stride + my_head * a.q_head + 8 * g;
#pragma unroll
            for (int s = 0; s < ST; ++s) {
                qf[s] = *reinterpret_cast<const uint4*>(src + 32 * s);
                if (!row_ok) qf[s] = make_uint4(0, 0, 0, 0);
            }
        }
        f32x4 o[DV];
#pragma unroll
        for (int j = 0; j < DV; ++j) o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        float m = -INFINITY, l = 0.f;

        const const_i32 trow = (const_i32)(uintptr_t)(a.table + (int64_t)b * a.table_stride);
        const int last_key = rq.keys - 1;
        const int page_mask = (1 << a.shift) - 1;
        const int kperm = 8 * (c >> 2) + (c & 3);  // key of tile t's row c: kperm + 4 t
        // A block's two runs of 16 keys lie in a page each.  Page ids come through
        // the scalar cache one block ahead; the K of the next block is loaded into
        // the registers of this one's as soon as its scores are there, and V after
        // the products, so that loads are in flight all the time.
        struct Pages {
            int lo, hi;
        };
        auto pages_at = [&](int i) {
            const int key0 = bl.at(i < i1 ? i : i1 - 1) * kBlockKeys;
            return Pages{trow[min(key0, last_key) >> a.shift], trow[min(key0 + 16, last_key) >> a.shift]};
        };
        auto there = [&](int id) { return (uint32_t)id < (uint32_t)a.pages; };
        auto base_of = [&](int id) { return (int64_t)(there(id) ? id : 0) * a.page_stride + ((int64_t)h << a.shift) * D; };
        uint4 kf[2][ST];
        VRow<VD> vr[8];
        auto load_k = [&](int key0, const Pages& pg) {
            const uint16_t* kbase = a.k + (c >= 8 ? base_of(pg.hi) : base_of(pg.lo)) + 8 * g;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint16_t* p = kbase + (uint32_t)(((key0 + kperm + 4 * t) & page_mask) * D);
#pragma unroll
                for (int s = 0; s < ST; ++s) kf[t][s] = *reinterpret_cast<const uint4*>(p + 32 * s);
            }
        };
        auto load_v = [&](int key0, const Pages& pg) {
            const uint16_t* vbase = a.v + (g >= 2 ? base_of(pg.hi) : base_of(pg.lo)) + DV * c + (uint32_t)(((key0 + 8 * g) & page_mask) * D);
#pragma unroll
            for (int e = 0; e < 8; ++e) vr[e] = load_vrow<VD>(vbase + e * D);
        };
        if (i0 + wave < i1) {
            int i = i0 + wave, key0 = bl.at(i) * kBlockKeys;
            Pages now = pages_at(i);
            load_k(key0, now);
            load_v(key0, now);
            Pages next = pages_at(i + kWaves);
            for (;;) {
                const bool more = i + kWaves < i1;
                const int key1 = more ? bl.at(i + kWaves) * kBlockKeys : key0;
                const bool okv = there(g >= 2 ? now.hi : now.lo);
                float t8[8];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    f32x4 s4 = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < ST; ++s) s4 = E::mfma16(kf[t][s], qf[s], s4);
#pragma unroll
                    for (int r = 0; r < 4; ++r) t8[4 * t + r] = s4[r] * a.scale_log2;
                }
                if (more) load_k(key1, next);
                // blocks that every row of the tile sees whole need no mask
                bool whole = key0 + kBlockKeys - 1 <= min(tile_p0, last_key);
                if (a.window > 0) whole = whole && (tile_p1 - key0 < a.window || key0 + kBlockKeys <= a.sinks);
                const bool masked = !whole || !there(now.lo) || !there(now.hi);
                bool poisoned = false;
                if (masked) {
                    uint32_t bad = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int j = key0 + 8 * g + e;
                        const bool held = okv && j <= last_key;
                        if (!held || !sees(a, my_pos, j)) t8[e] = -INFINITY;
                        // a key that no row of the tile sees may hold anything
                        const bool hidden = !held || j > tile_p1 ||
                                            (a.window > 0 && tile_p0 - j >= a.window && j >= a.sinks);
#pragma unroll
                        for (int w = 0; w < VD; ++w) {
                            if (hidden) vr[e].w[w] = 0;
                            bad |= nonfinite<E>(vr[e].w[w]);
                        }
                    }
                    poisoned = __any(bad != 0);
                }
                // running maximum less kLift, shared by the four lanes of a row;
                // raised only when a score passes the maximum by more than 2^8,
                // so that most blocks rescale nothing
                float mx = t8[0];
#pragma unroll
                for (int e = 1; e < 8; ++e) mx = fmaxf(mx, t8[e]);
                if (__any(mx > m + (E::kLift + 8.f))) {
                    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
                    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
                    const float mn = fmaxf(m, mx - E::kLift);
                    const float f = mn == -INFINITY ? 1.f : exp2_fast(m - mn);
                    m = mn;
                    l *= f;
#pragma unroll
                    for (int j = 0; j < DV; ++j) o[j] *= f;
                }
                const float ms = m == -INFINITY ? 0.f : m;
                uint32_t pw[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p0 = exp2_fast(t8[2 * e] - ms), p1 = exp2_fast(t8[2 * e + 1] - ms);
                    l += p0 + p1;
                    pw[e] = E::pack2(p0, p1);
                }
                if (!poisoned) {
                    const uint4 pf = make_uint4(pw[0], pw[1], pw[2], pw[3]);
#pragma unroll
                    for (int j = 0; j < DV; ++j) {
                        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
                        uint4 vf;
                        vf.x = __builtin_amdgcn_perm(vr[1].w[j / 2], vr[0].w[j / 2], sel);
                        vf.y = __builtin_amdgcn_perm(vr[3].w[j / 2], vr[2].w[j / 2], sel);
                        vf.z = __builtin_amdgcn_perm(vr[5].w[j / 2], vr[4].w[j / 2], sel);
                        vf.w = __builtin_amdgcn_perm(vr[7].w[j / 2], vr[6].w[j / 2], sel);
                        o[j] = E::mfma16(vf, pf, o[j]);
                    }
                } else {
                    // A value that some rows see and others do not is not finite:
                    // 0 times it would spoil the rows it is hidden from, so the
                    // block is added key by key, to the rows that see each.
                    // Lane (g, c) owns row c, values D / 4 g .. of V.
                    for (int gg = 0; gg < 4; ++gg) {
                        const int src = gg * 16;
                        const int pid = gg >= 2 ? now.hi : now.lo;
                        for (int e = 0; e < 8; ++e) {
                            const int j = key0 + 8 * gg + e;
                            float p = 0.f;
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const float px = (x & 1) ? E::hi(pw[x / 2]) : E::lo(pw[x / 2]);
                                const float got = __shfl(px, src + c, 64);
                                if (x == e) p = got;
                            }
                            if (!there(pid) || j > last_key || !sees(a, my_pos, j)) continue;
                            const uint16_t* vp = a.v + (int64_t)pid * a.page_stride +
                                                 (((int64_t)h << a.shift) + (j & page_mask)) * D + 4 * DV * g;
#pragma unroll
                            for (int r = 0; r < 4; ++r)
#pragma unroll
                                for (int jj = 0; jj < DV; ++jj) {
                                    const uint32_t w = vp[DV * r + jj];
                                    o[jj][r] = fmaf(p, E::lo(w), o[jj][r]);
                                }
                        }
                    }
                }
                if (!more) break;
                load_v(key1, next);
                i += kWaves;
                key0 = key1;
                now = next;
                next = pages_at(i + kWaves);
            }
            l += __shfl_xor(l, 16, 64);
            l += __shfl_xor(l, 32, 64);
        }

        // join the waves
        {
            float* dst = lds_o + (wave * 16 + c) * LD + 4 * DV * g;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < DV; j += 4)
                    *reinterpret_cast<float4*>(dst + DV * r + j) = make_float4(o[j][r], o[j + 1][r], o[j + 2][r], o[j + 3][r]);
            if (g == 0) {
                lds_ml[(wave * 16 + c) * 2] = m;
                lds_ml[(wave * 16 + c) * 2 + 1] = l;
            }
        }
        __syncthreads();
        const bool parts = nsplit > 1;
        constexpr int EPT = 4;                                             // values a thread joins at a time
        for (int u = tid; u < rows * (D / EPT); u += kRowsThreads) {
            const int row = u / (D / EPT), d = (u - row * (D / EPT)) * EPT;
            float M = -INFINITY, L = 0.f;
            for (int w = 0; w < kWaves; ++w) M = fmaxf(M, lds_ml[(w * 16 + row) * 2]);
            const float ms = M == -INFINITY ? 0.f : M;
            float acc[EPT] = {0.f, 0.f, 0.f, 0.f};
            for (int w = 0; w < kWaves; ++w) {
                const int base = w * 16 + row;
                const float f = exp2_fast(lds_ml[base * 2] - ms);
                L += f * lds_ml[base * 2 + 1];
                const float4 x = *reinterpret_cast<const float4*>(lds_o + base * LD + d);
                acc[0] += f * x.x;
                acc[1] += f * x.y;
                acc[2] += f * x.z;
                acc[3] += f * x.w;
            }
            if (parts) {
#pragma unroll
                    for (int e = 0; e < EPT; e += 2) store_pair(slab + 2 * rows + row * D + d + e, acc[e], acc[e + 1]);
                if (d == 0) {
                    store_partial(slab + 2 * row, M);
                    store_partial(slab + 2 * row + 1, L);
                }
            } else {
                const int tok = row / G;
                const int64_t at = (int64_t)(rq.t0 + tok) * a.Hq + h * G + row - tok * G;
                const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : NAN);
                *reinterpret_cast<uint2*>(a.out + at * D + d) =
                    make_uint2(E::pack2(acc[0] * inv, acc[1] * inv), E::pack2(acc[2] * inv, acc[3] * inv));
                if (d == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : kLn2 * (M + log2f(L));
            }
        }
        if (parts && split_last_arrival(a.flags, (uint32_t)(b * a.Hkv + h), nsplit, &word))
            join_splits<E, D>(a, rq, h, 0, rows, 2 * rows, slabs, nsplit, lds_o, row_m, row_l);
        if (a.workers == 0) return;
        __syncthreads();  // LDS is the next request's
    }
}

// ---- tile kernel: 32 rows a wave, 128 a workgroup, keys in tiles of 64.
//
// Prompt chunks are bound by the matrix cores.  K and V tiles go from their
// pages to LDS by DMA, one tile ahead, and are shared by the four waves; the
// transposed products are as in the rows kernel, with 32 x 32 matrix tiles:
// S^T = K Q^T leaves row n = lane % 32 of the queries in lanes n and n + 32,
// each with 4 of every 8 keys, and these scores, rounded, are the second
// operand of O^T = V^T P^T with the keys of a step of 16 dealt as
// (4 h .. 4 h + 3, 8 + 4 h .. 8 + 4 h + 3), h = lane / 32.  V^T comes from
// LDS through the transposing read, which gives a lane four keys of one
// column.  So the weights never leave their registers, and a row's maximum
// and sum need no exchange between lanes but where the maximum is raised.
//
// 16-byte chunks of a row are stored at chunk ^ f(key) (kswz, vswz), so that 8
// or 16 lanes of a K read, and 16 or 32 of a V read (4 keys, 32 or 64 bytes of
// each), fall into different banks.
//
// The scores of tile i + 1 are computed in the same run of instructions as the
// exponentials and the products with V of tile i, so that the matrix cores and
// the vector unit work at once within a wave: K runs one tile ahead of V.
//
// 8192 tokens over 12288 keys, 32 + 8 heads of 128, bf16: 1030 to 1090 us, 1010
// to 1070 TFLOP/s; without the overlap of scores and weights 1220 us.  The
// matrix cores are busy 56 % of the cycles, at a clock that the card's power
// holds at 1.7 GHz under this load.  Heads of 64, three waves a SIMD: 168
// registers, of which 2 spill (12 bytes of scratch a lane, stored before the key
// loop and read back after it); 24 decoding requests beside 9 chunks, a window of 2047: 131 to 146 us.
// There the vector unit counts as much as the matrix cores: 3.5e8 exponentials
// at a quarter of its rate take 36 us of it, four or five more operations a
// score 45 us, where the products alone take 72 us of the matrix cores.
constexpr int kTileKeys = 64;
constexpr int kTileRows = 128;
constexpr int kTileThreads = 256;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) char lds_char;

// 8 bytes a lane from LDS, transposed over 16 lanes: lane i of the 16 gives
// the address of 4 values of row i / 4, columns 4 (i % 4) .. + 3, and gets the
// values of column i in the four rows.
__device__ __forceinline__ uint2 lds_transposed(const lds_char* p) {
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

// N DMAs of 16 bytes a lane from a wave-uniform base (see dma16s): run u from
// base + 1024 u + off[u] to lds_addr + 1024 u + 16 * lane.
template <int N>
__device__ __forceinline__ void dma_runs(const void* base, const uint32_t (&off)[N], uint32_t lds_addr) {
    static_assert(N == 2 || N == 4, "runs of a wave's 16 keys");
    if constexpr (N == 4)
        asm volatile("s_mov_b32 m0, %5\n\ts_nop 0\n\t"
                     "global_load_lds_dwordx4 %0, %4\n\tglobal_load_lds_dwordx4 %1, %4 offset:1024\n\t"
                     "global_load_lds_dwordx4 %2, %4 offset:2048\n\tglobal_load_lds_dwordx4 %3, %4 offset:0xC00"
                     :: "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "s"(base), "s"(lds_addr) : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\t"
                     "global_load_lds_dwordx4 %0, %2\n\tglobal_load_lds_dwordx4 %1, %2 offset:1024"
                     :: "v"(off[0]), "v"(off[1]), "s"(base), "s"(lds_addr) : "memory", "m0");
}

template <int D>
struct TileGeom {
    static constexpr int kRowBytes = D * 2;
    static constexpr int kMatBytes = kTileKeys * kRowBytes;  // one of K and V
    static constexpr int kLdsBytes = 4 * kMatBytes;          // two of K, then two of V
    static __device__ __forceinline__ int kswz(int key) {
        return D == 128 ? (key & 15) : ((key & 7) ^ ((key >> 3) & 1));
    }
    static __device__ __forceinline__ int vswz(int key) {
        return D == 128 ? 2 * ((key & 3) ^ ((key & 3) << 1)) : 2 * (key & 3);
    }
};

// The request of tile `t` of a call: request b's tiles begin at
// floor(cu[b] G / 128) + b, which leaves room for the ceil(n G / 128) it
// needs.  Finds the last b that begins at or before t (offsets ascending);
// 64 places a round, so that a batch of 64 costs one read.
__device__ __forceinline__ int64_t tiles_before(const AttnArgs& a, int b) {
    const int c = min(max(a.cu[b], 0), a.T);
    return (int64_t)c * a.G / kTileRows + b;
}
__device__ __forceinline__ int request_of_tile(const AttnArgs& a, int64_t t) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = a.B;  // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int probe = lo + lane * step;
        const bool in = lane * step < n && tiles_before(a, probe) <= t;
        const int last = 63 - __clzll((long long)(__ballot(in) | 1ull));
        n = min(step, n - last * step);
        lo += last * step;
    }
    return lo;
}

template <class E, int D>
__global__ __launch_bounds__(kTileThreads, D == 64 ? 3 : 2) void tile_kernel(AttnArgs a) {
    using TG = TileGeom<D>;
    constexpr int KS = D / 16;        // steps of S^T = K Q^T
    constexpr int DB = D / 32;        // 32-column blocks of O
    constexpr int CPR = D / 8;        // chunks of a row
    constexpr int RPD = 64 / CPR;     // rows a DMA of one wave fills
    extern __shared__ uint4 smem_tile[];
    __shared__ uint32_t ctrl[3];
    __shared__ float row_m[kTileRows], row_l[kTileRows];
    const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem_tile;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, half = lane >> 5;
    // workgroup -> KV head (fastest), split, tile (the last rows, which see most keys, first)
    int64_t id = blockIdx.x;
    const int h = (int)(id % a.Hkv);
    id /= a.Hkv;
    const int split = (int)(id % a.splits);
    id /= a.splits;
    const int64_t t = a.tiles - 1 - id;
    const int b = __builtin_amdgcn_readfirstlane(request_of_tile(a, t));
    const Request rq = request_of(a, b);
    const int G = a.G;
    const int64_t rows_all = (int64_t)min(rq.n, a.max_q) * G;
    const int64_t row0 = (t - tiles_before(a, b)) * kTileRows;
    if (row0 < 0 || row0 >= rows_all || rows_all <= a.rows_most) return;
    const int rows = (int)(rows_all - row0 < kTileRows ? rows_all - row0 : kTileRows);
    const int wg_p0 = rq.first + (int)(row0 / G), wg_p1 = rq.first + (int)((row0 + rows - 1) / G);
    const Blocks bl = blocks_of<6>(a, rq, wg_p0, wg_p1);
    int per = a.split_blocks;
    if ((int64_t)per * a.splits < bl.count) per = (bl.count + a.splits - 1) / a.splits;
    const int nsplit = bl.count > per ? (bl.count + per - 1) / per : 1;
    if (split >= nsplit) return;

    const int64_t my_row = row0 + 32 * wave + n;
    const bool row_ok = my_row < rows_all;
    const int my_tok = (int)((row_ok ? my_row : row0) / G);
    const int my_head = h * G + (int)((row_ok ? my_row : row0) - (int64_t)my_tok * G);
    const int my_pos = row_ok ? rq.first + my_tok : INT32_MIN;
    const bool wave_ok = 32 * wave < rows;
    const int64_t last_row = row0 + 32 * wave + 31 < rows_all ? row0 + 32 * wave + 31 : rows_all - 1;
    const int p0 = rq.first + (int)((row0 + 32 * wave) / G), p1 = rq.first + (int)(last_row / G);

    uint4 qf[KS];
    {
        const uint16_t* src = a.q + (int64_t)(rq.t0 + my_tok) * a.q_stride + my_head * a.q_head + 8 * half;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            qf[s] = *reinterpret_cast<const uint4*>(src + 16 * s);
            if (!row_ok) qf[s] = make_uint4(0, 0, 0, 0);
        }
    }
    f32x16 o[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] = 0.f;
    float m = -INFINITY, l = 0.f;

    const int i0 = split * per, i1 = min(bl.count, i0 + per);
    const const_i32 trow = (const_i32)(uintptr_t)(a.table + (int64_t)b * a.table_stride);
    const int last_key = rq.keys - 1;
    const int page_mask = (1 << a.shift) - 1;

    // DMA of a tile: wave w fills keys 16 w .. 16 w + 15, which lie in one
    // page; lane -> (row lane / CPR, chunk lane % CPR) of each run of RPD rows.
    // Byte offsets in the run, which begins 1024 u behind the wave's first key
    // in the page and in LDS alike.
    constexpr int RUNS = 16 / RPD;
    uint32_t dma_k[RUNS], dma_v[RUNS];
#pragma unroll
    for (int u = 0; u < RUNS; ++u) {
        const int r = lane / CPR, c = lane % CPR;
        dma_k[u] = (uint32_t)(r * TG::kRowBytes + ((c ^ TG::kswz(u * RPD + r)) << 4));
        dma_v[u] = (uint32_t)(r * TG::kRowBytes + ((c ^ TG::vswz(u * RPD + r)) << 4));
    }
    // The page of keys j .. j + 15 (j a multiple of 16), -1 where there is none
    auto page_at = [&](int j) {
        if (j > last_key) return -1;
        const int pg = trow[j >> a.shift];
        return (uint32_t)pg < (uint32_t)a.pages ? pg : -1;
    };
    // Set for good by the first value that is not finite in a tile that not every
    // row sees whole.
    uint32_t* poison = &ctrl[0];
    // The first tile of which a page is not there.  Waves look their pages up at
    // different times, up to two tiles ahead, and the waves must agree on which
    // tiles have gaps (a barrier hangs on it): so a wave posts the tile's number
    // and a tile i asks for one of at most i.  What was posted for the tiles up
    // to i lies a barrier or more back when i is asked for, and what is posted
    // meanwhile, for later tiles, does not change the answer.
    uint32_t* absent = &ctrl[1];
    // A tile: its first key, and where this wave's run lies in the caches.
    // The page id is read one tile before it is used (id_of, then tile_at).
    struct Tile {
        int key0;
        int64_t at;
    };
    const int64_t head_at = ((int64_t)h << a.shift) * D;
    auto first_key = [&](int i) { return bl.at(i < i1 ? i : i1 - 1) * kTileKeys; };
    auto id_of = [&](int i) { return trow[min(first_key(i) + 16 * wave, last_key) >> a.shift]; };
    auto tile_at = [&](int i, int id) {
        Tile t;
        t.key0 = first_key(i);
        const int j = t.key0 + 16 * wave;
        if ((uint32_t)id >= (uint32_t)a.pages) {
            id = 0;
            atomicMin(absent, (uint32_t)i);
        }
        t.at = (int64_t)id * a.page_stride + head_at + (uint32_t)((j & page_mask) * D);
        return t;
    };
    auto issue_k = [&](const Tile& t, int i) {
        dma_runs(a.k + t.at, dma_k, lds + (uint32_t)((i & 1) * TG::kMatBytes + 16 * wave * TG::kRowBytes));
    };
    auto issue_v = [&](const Tile& t, int i) {
        dma_runs(a.v + t.at, dma_v, lds + (uint32_t)((2 + (i & 1)) * TG::kMatBytes + 16 * wave * TG::kRowBytes));
    };
    // this lane's operands: byte offsets in a K and in a V tile
    uint32_t kaddr[KS], vaddr[DB];
#pragma unroll
    for (int s = 0; s < KS; ++s) kaddr[s] = (uint32_t)(n * TG::kRowBytes + (((2 * s + half) ^ TG::kswz(n)) << 4));
    {
        const int key = 4 * half + ((lane & 15) >> 2);
        const int x = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
#pragma unroll
        for (int d = 0; d < DB; ++d)
            vaddr[d] = (uint32_t)(key * TG::kRowBytes + (((4 * d + x) ^ TG::vswz(key)) << 4) + 8 * (lane & 1));
    }
    char* smem = reinterpret_cast<char*>(smem_tile);
    if (tid == 0) {
        *poison = 0u;
        *absent = 0xFFFFFFFFu;
    }
    __syncthreads();
    const int wg_whole = min(wg_p0, last_key) - (kTileKeys - 1);  // tiles up to here are seen whole but for a window

    f32x16 s[2];  // scores of the tile to come
    auto scores = [&](int i) {
        const char* st = smem + (i & 1) * TG::kMatBytes;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kt][r] = 0.f;
#pragma unroll
            for (int x = 0; x < KS; ++x) {
                const uint4 kf = *reinterpret_cast<const uint4*>(st + kaddr[x] + 32 * kt * TG::kRowBytes);
                s[kt] = E::mfma32(kf, qf[x], s[kt]);
            }
        }
    };
    Tile cur{}, next{};
    if (i0 < i1) {
        cur = tile_at(i0, id_of(i0));
        issue_k(cur, i0);
        next = tile_at(i0 + 1, id_of(i0 + 1));
        int id = id_of(i0 + 2);
        issue_v(cur, i0);
        if (i0 + 1 < i1) {
            issue_k(next, i0 + 1);
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * (16 / RPD)) : "memory");  // K of the first tile is in LDS
        } else {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(16 / RPD) : "memory");
        }
        __syncthreads();
        scores(i0);
        for (int i = i0; i < i1; ++i) {
            const int key0 = cur.key0;
            const bool gaps = *absent <= (uint32_t)i;
            cur = next;
            next = tile_at(i + 2, id);
            id = id_of(i + 3);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's part of V of tile i and of K of tile i + 1
            __syncthreads();                                  // everybody's, and what the next DMAs replace is read
            if (i + 2 < i1) issue_k(next, i + 2);  // no DMA is in flight when the loop ends
            if (i + 1 < i1) issue_v(cur, i + 1);

            // Tiles that not every row sees whole: a weight of 0 times a value that
            // is not finite would be NaN, so such values leave the tile first; the
            // ones that some row sees are added in the end.
            bool masked = gaps || key0 > wg_whole;
            if (a.window > 0) masked = masked || (wg_p1 - key0 >= a.window && key0 + kTileKeys > a.sinks);
            bool hide = false;
            uint32_t there = 15u;  // bit x: keys key0 + 16 x .. have a page (or lie past the last key)
            if (masked) {
                if (gaps) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (page_at(key0 + 16 * x) < 0) there &= ~(1u << x);
                }
                // does this wave have a row that does not see the tile whole?
                hide = there != 15u || key0 + kTileKeys - 1 > min(p0, last_key);
                if (a.window > 0) hide = hide || (p1 - key0 >= a.window && key0 + kTileKeys > a.sinks);
                const int end = min(wg_p1, last_key);
                char* st = smem + (2 + (i & 1)) * TG::kMatBytes;
                int u0 = tid;
                asm volatile("" : "+v"(u0));  // nothing of this path is held in registers through the loop
                for (int u = u0; u < kTileKeys * CPR; u += kTileThreads) {
                    uint4* at = reinterpret_cast<uint4*>(st) + u;
                    const uint4 v = *at;
                    const uint32_t bx = nonfinite<E>(v.x), by = nonfinite<E>(v.y), bz = nonfinite<E>(v.z), bw = nonfinite<E>(v.w);
                    if (bx | by | bz | bw) {
                        *at = make_uint4(v.x & ~((bx >> 15) * 0xFFFFu), v.y & ~((by >> 15) * 0xFFFFu),
                                         v.z & ~((bz >> 15) * 0xFFFFu), v.w & ~((bw >> 15) * 0xFFFFu));
                        const int x = u / CPR, j = key0 + x;
                        if (j <= end && ((there >> (x >> 4)) & 1u) && !(a.window > 0 && wg_p0 - j >= a.window && j >= a.sinks))
                            *poison = 1u;
                    }
                }
                __syncthreads();
            }
            if (!wave_ok) continue;  // no rows: this wave only helps to fill the tiles
            if (hide) {
                // Key x of the tile (x - 4 half below, a constant) is seen up to
                // `most`, with a window not from `sink` to `low`, and only where
                // it has a page.
                const int64_t base = key0 + 4 * half;
                auto in_tile = [&](int64_t x) { return (int)(x < -1 ? -1 : x > kTileKeys ? kTileKeys : x); };
                const int most = in_tile((int64_t)min(my_pos, last_key) - base);
                const auto each = [&](auto hidden) {
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                        for (int r = 0; r < 16; ++r) s[kt][r] = hidden(32 * kt + 8 * (r >> 2) + (r & 3)) ? -INFINITY : s[kt][r];
                };
                each([&](int x) { return x > most; });
                if (a.window > 0) {
                    const int sink = in_tile((int64_t)a.sinks - base), low = in_tile((int64_t)my_pos - a.window - base);
                    const uint32_t gap = (uint32_t)max(low - sink + 1, 0);
                    each([&](int x) { return (uint32_t)(x - sink) < gap; });
                }
                if (there != 15u) each([&](int x) { return !((there >> (x >> 4)) & 1u); });
            }
            // running maximum of the scaled scores, held and raised as in the rows kernel
            float mx = s[0][0];
#pragma unroll
            for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[0][r]);
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[1][r]);
            mx *= a.scale_log2;
            if (__any(mx > m + (E::kLift + 8.f))) {
                mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
                const float mn = fmaxf(m, mx - E::kLift);
                const float f = mn == -INFINITY ? 1.f : exp2_fast(m - mn);
                m = mn;
                l *= f;
#pragma unroll
                for (int d = 0; d < DB; ++d) o[d] *= f;
            }
            const float ms = m == -INFINITY ? 0.f : m;
            const f32x16 sc[2] = {s[0], s[1]};
            scores(i + 1);  // past the last tile: of what its buffer holds, not used
            uint32_t pw[16];
            float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    const float x0 = exp2_fast(fmaf(sc[kt][r], a.scale_log2, -ms)), x1 = exp2_fast(fmaf(sc[kt][r + 1], a.scale_log2, -ms));
                    add[r & 2] += x0;
                    add[(r & 2) + 1] += x1;
                    pw[8 * kt + r / 2] = E::pack2(x0, x1);
                }
            l += (add[0] + add[1]) + (add[2] + add[3]);

            // step x: keys 16 x .. 16 x + 15
            const lds_char* vt[DB];
#pragma unroll
            for (int d = 0; d < DB; ++d)
                vt[d] = (const lds_char*)smem_tile + (2 + (i & 1)) * TG::kMatBytes + vaddr[d];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint4 pf = make_uint4(pw[4 * x], pw[4 * x + 1], pw[4 * x + 2], pw[4 * x + 3]);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    const uint2 lo = lds_transposed(vt[d] + 16 * x * TG::kRowBytes);
                    const uint2 hi = lds_transposed(vt[d] + (16 * x + 8) * TG::kRowBytes);
                    o[d] = E::mfma32(make_uint4(lo.x, lo.y, hi.x, hi.y), pf, o[d]);
                }
            }
            if (masked && *poison) {
                // A value that some rows see and others do not is not finite (it
                // is zero in LDS): such values are added one by one, from their
                // page, to the rows that see them.  Lane (n, half) owns row n,
                // columns 8 y + 4 half .. + 3.
                int n_ = n, half_ = half;
                asm volatile("" : "+v"(n_), "+v"(half_));  // as above
                for (int x = 0; x < kTileKeys; ++x) {
                    const int j = key0 + x, src = n_ + 32 * ((x >> 2) & 1), pg = page_at(j);
                    float p = 0.f;
#pragma unroll
                    for (int w = 0; w < 16; ++w) {
                        // dword w holds keys 32 (w / 8) + 8 ((w % 8) / 2) + 4 half + 2 (w % 2) and the next
                        const int k = 32 * (w >> 3) + 8 * ((w & 7) >> 1) + 2 * (w & 1);
                        const uint32_t got = __shfl(pw[w], src, 64);
                        if (k == (x & ~5)) p = (x & 1) ? E::hi(got) : E::lo(got);
                    }
                    if (pg < 0 || !sees(a, my_pos, j)) continue;
                    const uint16_t* row = a.v + (int64_t)pg * a.page_stride + (((int64_t)h << a.shift) + (j & page_mask)) * D;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const uint32_t w = row[32 * d + 8 * (r >> 2) + 4 * half_ + (r & 3)];
                            if (nonfinite<E>(w) & 0x8000u) o[d][r] = fmaf(p, E::lo(w), o[d][r]);
                        }
                }
            }
        }
    }
    l += __shfl_xor(l, 32, 64);

    const bool parts = nsplit > 1;
    const int64_t wg_tile = t * a.Hkv + h;
    if (!parts) {
        if (!row_ok) return;
        const int64_t at = (int64_t)(rq.t0 + my_tok) * a.Hq + my_head;
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : NAN);
        uint16_t* dst = a.out + at * D + 4 * half;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                *reinterpret_cast<uint2*>(dst + 32 * d + 8 * y) =
                    make_uint2(E::pack2(o[d][4 * y] * inv, o[d][4 * y + 1] * inv), E::pack2(o[d][4 * y + 2] * inv, o[d][4 * y + 3] * inv));
        if (half == 0 && a.lse) a.lse[at] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
        return;
    }
    float* slab = a.partials + (wg_tile * a.splits + split) * a.slab;  // [128][2], then [128][D]
    if (row_ok) {
        const int row = 32 * wave + n;
        if (half == 0) {
            store_partial(slab + 2 * row, m);
            store_partial(slab + 2 * row + 1, l);
        }
        float* dst = slab + 2 * kTileRows + row * D + 4 * half;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 2) store_pair(dst + 32 * d + 8 * (r >> 2) + (r & 3), o[d][r], o[d][r + 1]);
    }
    if (!split_last_arrival(a.flags, (uint32_t)wg_tile, nsplit, &ctrl[2])) return;
    const float* slabs = a.partials + wg_tile * a.splits * a.slab;
    join_splits<E, D>(a, rq, h, row0, rows, 2 * kTileRows, Slabs{slabs, slabs, a.slab}, nsplit,
                      reinterpret_cast<float*>(smem_tile), row_m, row_l);
}

}  // namespace

// Schedule of a call.
//
// Requests of more than kRowsMost rows go to the tile kernel, the others to the
// rows kernel.  A call that may hold both kinds launches both, unless there is
// one request or none reads more than kShortKeys keys: the tile kernel then
// takes them all, a decoding row in a tile of 128 costing less than the second
// launch and its tail (24 decoding requests beside 9 chunks, a window of 2047:
// 143 us against 165; 44 requests of up to 401 keys, 13 of them chunks of 23
// tokens at most: 14 against 31; 60 decoding requests of up to 8191 keys beside
// 4 chunks: 697 against 728).  The same holds, at any length, where the largest
// request has 64 rows at most (64 requests of up to 8191 keys and 3 tokens: 233
// against 310).
//
// Which side is faster hangs on how even the lengths are, which the host does
// not see, more than on the longest of them: the tile kernel has no even shares,
// so a decoding request much longer than the others is one long run of tiles.
// Us in one launch and in two, by the longest request's keys:
//                                      4096      8192     12000     16000     32000
//   32 requests, 2 chunks of 512,
//     lengths spread evenly           92/105   174/206   249/288   327/372   645/711
//     one long, the others 1/16       81/42    155/51    227/64    297/75    592/141
//   8 requests, 1 chunk of 512, even  62/67    110/106   157/152   202/189   390/370
//   33 requests, 9 of 300, 24 + 8
//     heads of 64, even               73/85    135/145   186/210   248/269   483/506
//     one long                        59/29    110/42    159/52    208/57    408/91
//   4 requests, 1 chunk of 1000, even 85/55    161/86    233/114   306/145   608/260
// (32 + 8 heads of 128 but where given.)  kShortKeys is no crossing, then: it
// keeps the gain of even batches up to there, and bounds what an uneven one loses.
//
// Rows kernel: with a workspace, the two
// workgroups a compute unit holds take even shares of all blocks, 4 at least (a
// block a wave).  Without one, or where
// the requests are more than the counters, a request is one workgroup's.
//
// Tile kernel: keys are split only while that keeps the grid within the two
// workgroups a compute unit holds, into no less than 8 tiles each.
constexpr int64_t kShortKeys = 12288;
constexpr int64_t kTileSplitMost = 64;  // the join's weights: splits * 128 floats of LDS, 32 KiB for D = 64

AttnPlan attn_plan(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q, int64_t max_kv, int64_t window,
                   int64_t sinks, int compute_units) {
    AttnPlan p{};
    const int64_t G = Hq / Hkv;
    if (max_q > T) max_q = T;
    int64_t rows = max_q * G;
    const bool large = rows > kRowsMost;
    // the keys that a run of `r` rows reads, at most
    auto reach = [&](int64_t r) {
        const int64_t w = window + sinks + (r + G - 1) / G + 2 * kTileKeys;
        return window > 0 && w < max_kv ? w : max_kv;
    };
    size_t bytes = 0;
    if (large) {
        p.rows_most = B > 1 && rows > 64 && reach(kTileRows) > kShortKeys ? kRowsMost : 0;
        p.tiles = T * G / kTileRows + B;
        const int64_t blocks = (reach(kTileRows) + kTileKeys - 1) / kTileKeys;
        int64_t n = 2 * compute_units / (p.tiles * Hkv);
        if (n > blocks / 8) n = blocks / 8;
        if (n > kTileSplitMost) n = kTileSplitMost;
        if (n < 1 || p.tiles * Hkv > kMaxFlags) n = 1;
        p.tile_split_blocks = blocks > 0 ? (blocks + n - 1) / n : 1;
        p.tile_splits = blocks > 0 ? (blocks + p.tile_split_blocks - 1) / p.tile_split_blocks : 1;
        p.tile_slab = kTileRows * (D + 2);
        if (p.tile_splits > 1) bytes = (size_t)(p.tiles * Hkv * p.tile_splits * p.tile_slab) * 4;
        rows = kRowsMost;
    } else {
        p.rows_most = rows;
    }
    if (p.rows_most > 0) {
        p.slab = rows * (D + 2);
        const int64_t blocks = (reach(rows) + kBlockKeys - 1) / kBlockKeys;
        p.split_most = 4096 / rows;  // the join's weights: splits * rows <= 4096 floats of LDS
        p.join_cost = (float)(rows * D) * 6e-4f;
        int64_t w = B * blocks / kShareBlocks + 1;
        if (w > 2 * compute_units / Hkv) w = 2 * compute_units / Hkv;
        if (w > 1 && blocks > kSplitBlocks && B <= kShareRequests && B * Hkv <= kMaxFlags) {
            p.workers = w;
            const size_t need = (size_t)(w * Hkv * 2 * p.slab) * 4;
            if (need > bytes) bytes = need;
        }
    }
    p.data_bytes = bytes;
    return p;
}

namespace {

template <class E, int D>
hipError_t launch_rows(const AttnArgs& a, unsigned grid, hipStream_t s) {
    rows_kernel<E, D><<<dim3(grid), dim3(kRowsThreads), 0, s>>>(a);
    return hipGetLastError();
}

template <class E, int D>
hipError_t launch_tiles(const AttnArgs& a, unsigned grid, hipStream_t s) {
    static DeviceFlags raised;
    const hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&tile_kernel<E, D>), TileGeom<D>::kLdsBytes, raised);
    if (e != hipSuccess) return e;
    tile_kernel<E, D><<<dim3(grid), dim3(kTileThreads), TileGeom<D>::kLdsBytes, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention(const AttnArgs& args, const AttnPlan& plan, hipStream_t s) {
    AttnArgs a = args;
    a.rows_most = plan.rows_most;
    if (plan.tiles > 0) {
        a.tiles = plan.tiles;
        a.splits = a.partials ? (int)plan.tile_splits : 1;
        a.split_blocks = (int)plan.tile_split_blocks;
        a.slab = plan.tile_slab;
        const int64_t grid = plan.tiles * a.splits * a.Hkv;
        if (grid <= 0 || grid > 0x7FFFFFFF) return hipErrorInvalidValue;
        const unsigned gd = (unsigned)grid;
        const hipError_t e = a.bf16 ? (a.D == 64 ? launch_tiles<AttnBF16, 64>(a, gd, s) : launch_tiles<AttnBF16, 128>(a, gd, s))
                                    : (a.D == 64 ? launch_tiles<AttnF16, 64>(a, gd, s) : launch_tiles<AttnF16, 128>(a, gd, s));
        if (e != hipSuccess) return e;
    }
    if (plan.rows_most == 0) return hipSuccess;
    a.workers = a.partials ? (int)plan.workers : 0;
    a.split_most = (int)plan.split_most;
    a.join_cost = plan.join_cost;
    a.slab = plan.slab;
    const int64_t grid = (a.workers > 0 ? a.workers : (int64_t)a.B) * a.Hkv;
    if (grid <= 0 || grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    const unsigned gd = (unsigned)grid;
    if (a.bf16) return a.D == 64 ? launch_rows<AttnBF16, 64>(a, gd, s) : launch_rows<AttnBF16, 128>(a, gd, s);
    return a.D == 64 ? launch_rows<AttnF16, 64>(a, gd, s) : launch_rows<AttnF16, 128>(a, gd, s);
}

}  // namespace tq
