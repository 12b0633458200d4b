// Low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + scale[l] (x[t] A[l]^T) B[l]^T,  l = ids[t],
// and out[t] = base[t] where l names no adapter.
//
// Both thin products of a block of rows are one workgroup's work, so nothing
// passes through memory between them.  Rows stay in the order of the call: a
// workgroup takes one adapter of its block at a time and leaves the others' rows
// out, so one launch serves any mixture, prompts of one adapter as well as
// decoding rows of many, without sorting.
//
// The first product's sums are fp32.  They enter the second one whole, as three
// 16-bit numbers each after a scaling of the row by a power of two: the rounded
// value, the rounded rest and the rest of that.  Each takes as many bits of the
// sum's 24 as the type has (8 of bf16, 11 of fp16), so nothing is left but, in fp16,
// what lies 2^-39 below the row's largest sum: its third number is a multiple of
// 2^-24, of sums scaled to 2^15.  (Two numbers keep 16 bits in bf16 and are 1 to 3 %
// faster, 75 instead of 77 us for 8191 rows of rank 64, but one output in 600 is then
// not what the fp32 sum rounds to.)
//
// What bounds it: a decoding row's call two trips to memory (ids, then all else): 8.9
// us for one row of rank 16, 4096 x 4096; 64 rows of 32 adapters, 6144 x 4096, the
// adapters' reads through L2, 11.5 us; a prompt the rows' loads, see below.
//
// Rows of any alignment are read and written in 16-byte vectors (the memory mode of
// this platform allows any address), but for the last columns of a row.
//
// Rows, ranks and columns that are not there are read through buffer descriptors
// at an offset past their end, which gives zeros and drops stores: no load waits
// for a mask, and nothing branches.

#include <initializer_list>

#include "tq_device.h"
#include "tq_internal.h"
#include "tq_lora_index.h"
#include "tq_tiles.h"

namespace tq {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A buffer of fewer than 2^31 bytes (kNowhere lies past any of them).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}

// What is in flight, as far as registers go: D steps of 32 S columns of x and A,
// kAhead steps of 32 columns of B and base.
template <int MB, int RT, int W>
struct Depth {
    static constexpr int S = RT <= 8 ? 2 : 1;
    static constexpr int D = RT == 1 ? (MB == 1 ? 4 : 3) : RT == 2 ? 3 : RT == 4 ? (MB == 1 ? 3 : 2) : 1;
    static constexpr int kAhead = RT <= 2 ? (W == 16 ? 2 : 4) : RT == 4 ? 2 : 1;
    // the first columns of B and base are asked for before x, as far as registers go
    static constexpr bool kEarly = MB * RT < 16;
    static constexpr int kLd = 16 * RT + 4;  // words of a row of sums in LDS
};

// Rows of sums [16 MB][kLd] in LDS as operands of the second product: lane
// 16 g + i has row i, ranks 32 s + 8 g .. + 7, as three numbers whose sum is the sum
// times 2^-e, and `scale` 2^e.
constexpr int kParts = 3;
template <class T, int MB, int RT>
__device__ __forceinline__ void split_sums16(const float* lds, int ld, float scale, u32x4 (&h16)[kParts][MB][(RT + 1) / 2],
                                             float (&factor)[MB]) {
    constexpr int kKs = (RT + 1) / 2;
    constexpr int kTop = std::is_same<T, F16>::value ? 15 : 0;  // the row's largest sum becomes 2^kTop at most
    const int g = (threadIdx.x & 63) >> 4, i16 = threadIdx.x & 15;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const float* sums = lds + (16 * m + i16) * ld;
        f32x4 h[kKs][2];
        float most = 0.0f;
#pragma unroll
        for (int s = 0; s < kKs; ++s)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                // ranks past 16 RT (RT = 1 alone): zeros
                const int j = 32 * s + 8 * g + 4 * q;
                h[s][q] = *reinterpret_cast<const f32x4*>(sums + (RT > 1 || j < 16 ? j : 0));
                if (RT == 1 && j >= 16) h[s][q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = fabsf(h[s][q][e]);
                    most = fmaxf(most, v < __builtin_inff() ? v : 0.0f);
                }
            }
        most = fmaxf(most, __shfl_xor(most, 16, kWave));
        most = fmaxf(most, __shfl_xor(most, 32, kWave));
        int ex = most > 0.0f ? __builtin_amdgcn_frexp_expf(most) - kTop : 0;  // most = f 2^(ex + kTop), 1/2 <= f < 1
        ex = ex < -100 ? -100 : ex > 120 ? 120 : ex;                          // 2^ex is a normal number
        factor[m] = ldexpf(scale, ex);
#pragma unroll
        for (int s = 0; s < kKs; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v0 = ldexpf(h[s][e / 2][2 * (e % 2)], -ex), v1 = ldexpf(h[s][e / 2][2 * (e % 2) + 1], -ex);
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    const uint32_t part = round_pair<T>(v0, v1);
                    h16[p][m][s][e] = part;
                    v0 = fabsf(v0) < __builtin_inff() ? v0 - T::to_f32((uint16_t)part) : 0.0f;
                    v1 = fabsf(v1) < __builtin_inff() ? v1 - T::to_f32((uint16_t)(part >> 16)) : 0.0f;
                }
            }
    }
}

// The second product may be NaN because an infinite B met a sum's rest, which is 0 or
// of the other sign: there the product of the sums' first numbers alone, first(m, t),
// decides.  The test is an instruction for two values; what follows it is run by
// waves with a NaN only.
template <int MB>
__device__ __forceinline__ bool any_nan(const f32x4 (&d)[MB][2]) {
    bool odd = false;
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int t = 0; t < 2; ++t)
            odd |= (bool)__builtin_isunordered(d[m][t][0], d[m][t][1]) | (bool)__builtin_isunordered(d[m][t][2], d[m][t][3]);
    return odd;
}
template <int MB, class First>
__device__ __forceinline__ void take_first(f32x4 (&d)[MB][2], First first) {
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const f32x4 f = first(m, t);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[m][t][e] = d[m][t][e] != d[m][t][e] ? f[e] : d[m][t][e];
        }
}

// The rows `mine` of the block at t0, all of adapter l (-1: none), and the columns
// of the chunk.  W waves deal the columns of x in steps of 32 S (whole cache lines
// of a row), then those of the output in steps of 32.  Both loops have the next
// steps' loads in flight under this one's products, and the first columns of B and
// base are asked for before x, so that a call of few rows waits for memory twice:
// for the ids, then for everything else.
// LDS: [W][16 MB][kLd] fp32 sums of the waves' columns.
template <class T, int MB, int RT, int W>
__device__ __forceinline__ void update(const LoraArgs& a, int64_t t0, uint32_t chunk, int l, uint64_t mine) {
    typedef typename Mfma<T>::vec vec;
    typedef Depth<MB, RT, W> Q;
    constexpr int kThreads = W * kWave, kRows = 16 * MB;
    constexpr int kKs = (RT + 1) / 2;  // 32-deep steps of the second product
    constexpr int S = Q::S, D = Q::D, kAhead = Q::kAhead, kLd = Q::kLd;
    extern __shared__ __attribute__((aligned(16))) float smem_lora[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, i16 = lane & 15;
    const int N = (int)a.N, K = (int)a.K;
    const int n_lo = (int)chunk * (int)a.cols;
    const int n_hi = n_lo + (int)a.cols < N ? n_lo + (int)a.cols : N;
    const int rows = a.T - t0 < kRows ? (int)(a.T - t0) : kRows;
    const bool some = l >= 0;
    const auto from = buffer(a.base + t0 * a.base_stride, ((rows - 1) * a.base_stride + N) * 2);
    const auto to = buffer(a.out + t0 * a.out_stride, ((rows - 1) * a.out_stride + N) * 2);
    const auto bbuf = buffer(a.B + (int64_t)(some ? l : 0) * a.N * a.r, (int64_t)N * a.r * 2);
    uint32_t from_row[MB], to_row[MB];  // columns 8 g .. 8 g + 7 of this lane's rows
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const bool live = (mine >> (16 * m + i16)) & 1;
        from_row[m] = live ? (uint32_t)((16 * m + i16) * a.base_stride + 8 * g) * 2u : kNowhere;
        to_row[m] = live ? (uint32_t)((16 * m + i16) * a.out_stride + 8 * g) * 2u : kNowhere;
    }
    uint32_t b_lane[2][kKs];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int st = 0; st < kKs; ++st) b_lane[t][st] = lora_b_lane(a.r, i16, g, t, st);
    // Output columns n .. n + 31
    struct Cols {
        u32x4 b[2][kKs], base[MB];
    };
    auto load_cols = [&](int n, Cols& c) {
        if (some) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int st = 0; st < kKs; ++st)
                    c.b[t][st] = __builtin_amdgcn_raw_buffer_load_b128(bbuf, b_lane[t][st] + lora_b_step(a.r, n), 0, 0);
        }
#pragma unroll
        for (int m = 0; m < MB; ++m)
            c.base[m] = __builtin_amdgcn_raw_buffer_load_b128(from, n + 8 * g + 8 <= n_hi ? from_row[m] : kNowhere, n * 2, 0);
    };
    auto at = [&](int i) { return lora_step(n_lo, (int)a.cols, W, wave, i); };
    Cols cols[kAhead];
    if (Q::kEarly && at(0) < n_hi) load_cols(at(0), cols[0]);

    u32x4 h16[kParts][MB][kKs];  // operands of the second product: lane 16 g + i, row i, ranks 32 s + 8 g ..
    float factor[MB];
    if (some) {
        const float* scale_at = a.scale ? a.scale + l : nullptr;
        // x A^T
        f32x4 acc[MB][RT];
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[m][r] = f32x4{0.f, 0.f, 0.f, 0.f};
        const auto xbuf = buffer(a.x + t0 * a.x_stride, ((rows - 1) * a.x_stride + K) * 2);
        const auto abuf = buffer(a.A + (int64_t)l * a.r * a.K, (int64_t)a.r * K * 2);
        uint32_t xr[MB], ar[RT];
#pragma unroll
        for (int m = 0; m < MB; ++m)
            xr[m] = ((mine >> (16 * m + i16)) & 1) ? (uint32_t)((16 * m + i16) * a.x_stride + 8 * g) * 2u : kNowhere;
#pragma unroll
        for (int r = 0; r < RT; ++r) ar[r] = 16 * r + i16 < a.r ? (uint32_t)((16 * r + i16) * K + 8 * g) * 2u : kNowhere;
        struct Step {
            u32x4 x[S][MB], a[S][RT];
        };
        auto load_step = [&](int k0, Step& s, bool part) {
#pragma unroll
            for (int u = 0; u < S; ++u) {
                const bool in = !part || k0 + 32 * u + 8 * g < K;
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    s.x[u][m] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, in ? xr[m] + 64u * u : kNowhere, 2 * k0, 0);
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    s.a[u][r] = __builtin_amdgcn_raw_buffer_load_b128(abuf, in ? ar[r] + 64u * u : kNowhere, 2 * k0, 0);
            }
        };
        auto products = [&](const Step& s) {
#pragma unroll
            for (int u = 0; u < S; ++u)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        acc[m][r] = Mfma<T>::mma(__builtin_bit_cast(vec, s.x[u][m]), __builtin_bit_cast(vec, s.a[u][r]), acc[m][r]);
        };
        const int whole = K & ~(32 * S - 1);
        constexpr int kNext = 32 * S * W;
        Step st[D];
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (32 * S * wave + d * kNext < whole) load_step(32 * S * wave + d * kNext, st[d], false);
        for (int k0 = 32 * S * wave; k0 < whole; k0 += D * kNext) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (k0 + d * kNext < whole) products(st[d]);
                if (k0 + (d + D) * kNext < whole) load_step(k0 + (d + D) * kNext, st[d], false);
            }
        }
        if (whole < K && wave == W - 1) {  // the rest, a multiple of 8 columns
            load_step(whole, st[0], true);
            products(st[0]);
        }
        const float scale = scale_at ? *scale_at : 1.0f;
        // lane 16 g + i: rows 4 g .. 4 g + 3, rank 16 r + i
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) smem_lora[(wave * kRows + 16 * m + 4 * g + e) * kLd + 16 * r + i16] = acc[m][r][e];
        __syncthreads();
        // the waves' sums, in their order; ranks past r count as 0 (an infinite x has
        // NaN there, times the zeros of A)
        for (int i = threadIdx.x; i < kRows * 4 * RT; i += kThreads) {
            const int j = 4 * (i % (4 * RT));
            f32x4* p = reinterpret_cast<f32x4*>(smem_lora + (i / (4 * RT)) * kLd + j);
            f32x4 v = *p;
#pragma unroll
            for (int w = 1; w < W; ++w) v += p[w * kRows * kLd / 4];
            *p = j < a.r ? v : f32x4{0.f, 0.f, 0.f, 0.f};  // r is a multiple of 8
        }
        __syncthreads();
        split_sums16<T, MB, RT>(smem_lora, kLd, scale, h16, factor);
    }

    auto finish = [&](int n, const Cols& c) {
        f32x4 d[MB][2];
#pragma unroll
        for (int m = 0; m < MB; ++m) d[m][0] = d[m][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (some) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int st = 0; st < kKs; ++st) {
                    const vec bv = __builtin_bit_cast(vec, c.b[t][st]);
#pragma unroll
                    for (int m = 0; m < MB; ++m)
#pragma unroll
                        for (int p = 0; p < kParts; ++p) d[m][t] = Mfma<T>::mma(bv, __builtin_bit_cast(vec, h16[p][m][st]), d[m][t]);
                }
            if (__builtin_expect(__ballot(any_nan<MB>(d)) != 0, 0))
                take_first<MB>(d, [&](int m, int t) {
                    f32x4 f = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int st = 0; st < kKs; ++st)
                        f = Mfma<T>::mma(__builtin_bit_cast(vec, c.b[t][st]), __builtin_bit_cast(vec, h16[0][m][st]), f);
                    return f;
                });
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            u32x4 v = c.base[m];
            // the columns of a row's end that are no whole vector, one by one
            const bool end = n + 32 > n_hi, part = n + 8 * g + 8 > n_hi;
            if (end) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t one = __builtin_amdgcn_raw_buffer_load_b16(
                        from, part && n + 8 * g + e < n_hi ? from_row[m] + 2u * e : kNowhere, n * 2, 0);
                    v[e / 2] |= one << (16 * (e % 2));
                }
            }
            if (some) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = round_pair<T>(fmaf(factor[m], d[m][e / 2][2 * (e % 2)], T::to_f32((uint16_t)v[e])),
                                         fmaf(factor[m], d[m][e / 2][2 * (e % 2) + 1], T::to_f32((uint16_t)(v[e] >> 16))));
            }
            __builtin_amdgcn_raw_buffer_store_b128(v, to, part ? kNowhere : to_row[m], n * 2, 0);
            if (end) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(v[e / 2] >> (16 * (e % 2))), to,
                                                          part && n + 8 * g + e < n_hi ? to_row[m] + 2u * e : kNowhere, n * 2, 0);
            }
        }
    };
    // h B^T
#pragma unroll
    for (int d = Q::kEarly ? 1 : 0; d < kAhead; ++d)
        if (at(d) < n_hi) load_cols(at(d), cols[d]);
    for (int i = 0; at(i) < n_hi; i += kAhead) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
            if (at(i + d) < n_hi) finish(at(i + d), cols[d]);
            if (at(i + d + kAhead) < n_hi) load_cols(at(i + d + kAhead), cols[d]);
        }
    }
}

// MB blocks of 16 rows, rank up to 16 RT, W waves.
template <class T, int MB, int RT, int W>
__global__ __launch_bounds__(W * kWave) void lora_kernel(LoraArgs a) {
    const int lane = threadIdx.x & 63;
    // Workgroups go to the XCDs in turn: the chunks of columns of one block and
    // adapter are on one of them, whose L2 then has the adapter and the rows.
    const uint32_t chunks = (uint32_t)a.chunks, turn = blockIdx.x >> 3;
    const uint32_t unit = turn / chunks * 8 + (blockIdx.x & 7), chunk = turn % chunks;
    const uint32_t slot = unit / (uint32_t)a.blocks;
    if (slot >= (uint32_t)a.slots) return;
    const int64_t t0 = (int64_t)(unit - slot * (uint32_t)a.blocks) * (16 * MB);

    // the slot-th different adapter of the rows, or all of them in turn; -1: none
    int id = -2;
    if (lane < 16 * MB && t0 + lane < a.T) {
        id = a.ids[t0 + lane];
        if (id < 0 || id >= a.L) id = -1;
    }
    uint64_t left = __ballot(id > -2);
    uint32_t skip = slot;
    do {
        const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t mine = __ballot(id == l);
        left &= ~mine;
        if (skip == 0 && !(l < 0 && a.out == a.base)) {
            update<T, MB, RT, W>(a, t0, chunk, l, mine);
            if (a.slots == 1 && left) __syncthreads();  // the sums in LDS have been read
        }
        if (a.slots > 1 && skip-- == 0) return;
    } while (left);
}

// ---------------------------------------------------------------- long prompts
//
// The same for 32 rows a workgroup and rank up to 64, with every operand brought to
// LDS by DMA in whole cache lines.  Read straight into matrix operands (16 rows x
// 64 bytes, neighbouring lanes in different rows) a compute unit gets 37 GB/s from
// its L2, in lines of 128 bytes 119; the adapter alone is read once per 32 rows.
// Each wave has a ring of its own of S stages, so the loops have no barrier:
//  - first product: 64 columns of 32 rows of x and of the 16 RT rows of A;
//  - second: 64 rows of B, which lie in a row, and 64 columns of base.
// Chunk c (16 bytes) of row r of a 128-byte row lies at c ^ (r / 2 % 8).  The sum
// takes the place of base in LDS and leaves from there, in lines again.
// Rows and ranks past the end are the last one again (ranks past it count as 0).
// Needs N % 8 == 0 and 16-byte aligned rows.  Measured: 8191 rows of 5 prompts, 4096
// x 4096, rank 64, 81 us (direct loads 109), 2.4 TB/s of rows; of one prompt 55: a
// block in which a prompt ends has two adapters and takes twice as long as the
// others, one a compute unit, that wait for it.
template <int RT>
struct Stage {
    static constexpr int W = RT <= 2 ? 8 : 4, S = RT == 2 ? 2 : 3;
    static constexpr int kBytes = 4096 + 2048 * RT;  // x and A, or base and 64 rows of B
    static constexpr int kRing = W * S * kBytes;
    static constexpr int kLd = 16 * RT + 4;
    static_assert(W * 32 * kLd * 4 <= kRing, "the sums take the ring's place");
};

__device__ __forceinline__ int line_swizzle(int r) { return (r >> 1) & 7; }

template <class T, int RT>
__device__ __forceinline__ void update_staged(const LoraArgs& a, int64_t t0, uint32_t chunk, int l, uint64_t mine) {
    typedef typename Mfma<T>::vec vec;
    typedef Stage<RT> Q;
    constexpr int W = Q::W, S = Q::S, kKs = (RT + 1) / 2, kLd = Q::kLd;
    extern __shared__ __attribute__((aligned(16))) float smem_lora[];
    uint8_t* lds = reinterpret_cast<uint8_t*>(smem_lora);
    const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem_lora;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, i16 = lane & 15;
    const int N = (int)a.N, K = (int)a.K, r = a.r;
    const int n_lo = (int)chunk * (int)a.cols;
    const int n_hi = n_lo + (int)a.cols < N ? n_lo + (int)a.cols : N;
    const int rows = a.T - t0 < 32 ? (int)(a.T - t0) : 32;
    const bool some = l >= 0;
    uint8_t* const ring = lds + wave * (S * Q::kBytes);
    const uint32_t ring_at = lds_base + (uint32_t)(wave * (S * Q::kBytes));

    u32x4 h16[kParts][2][kKs];  // operands of the second product: lane 16 g + i, row i, ranks 32 s + 8 g ..
    float factor[2];
    if (some) {
        f32x4 acc[2][RT];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < RT; ++q) acc[m][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        const uint16_t* x = a.x + t0 * a.x_stride;
        const uint16_t* A = a.A + (int64_t)l * r * a.K;
        uint32_t x_off[4], a_off[2 * RT];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int row = 8 * u + (lane >> 3);
            x_off[u] = (uint32_t)((row < rows ? row : rows - 1) * a.x_stride) * 2u + 16u * ((lane & 7) ^ line_swizzle(row));
        }
#pragma unroll
        for (int u = 0; u < 2 * RT; ++u) {
            const int row = 8 * u + (lane >> 3);
            a_off[u] = (uint32_t)((row < r ? row : r - 1) * K) * 2u + 16u * ((lane & 7) ^ line_swizzle(row));
        }
        constexpr int kCount = 4 + 2 * RT;  // transfers of a stage
        auto issue = [&](int k0, int stage) {
            const uint32_t to = ring_at + (uint32_t)(stage * Q::kBytes);
#pragma unroll
            for (int u = 0; u < 4; ++u) dma16s(x + k0, x_off[u], to + 1024u * u);
#pragma unroll
            for (int u = 0; u < 2 * RT; ++u) dma16s(A + k0, a_off[u], to + 4096u + 1024u * u);
        };
        const int steps = K / 64;
        const int own = steps > wave ? (steps - wave + W - 1) / W : 0;  // steps wave, wave + W, ...
#pragma unroll
        for (int d = 0; d < S - 1; ++d)
            if (d < own) issue(64 * (wave + W * d), d);
        int stage = 0;
        for (int k = 0; k < own; ++k) {
            // the stage read last is free: its reads have been used
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (k + S - 1 < own) {
                issue(64 * (wave + W * (k + S - 1)), stage == 0 ? S - 1 : stage - 1);
                asm volatile("s_waitcnt vmcnt(%0)" :: "n"((S - 1) * kCount) : "memory");
            } else {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
            const uint8_t* p = ring + stage * Q::kBytes;
            stage = stage == S - 1 ? 0 : stage + 1;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                vec xv[2], av[RT];
                const int at = i16 * 128 + 16 * ((4 * u + g) ^ line_swizzle(i16));
#pragma unroll
                for (int m = 0; m < 2; ++m) xv[m] = __builtin_bit_cast(vec, *reinterpret_cast<const u32x4*>(p + 2048 * m + at));
#pragma unroll
                for (int q = 0; q < RT; ++q) av[q] = __builtin_bit_cast(vec, *reinterpret_cast<const u32x4*>(p + 4096 + 2048 * q + at));
#pragma unroll
                for (int q = 0; q < RT; ++q)
#pragma unroll
                    for (int m = 0; m < 2; ++m) acc[m][q] = Mfma<T>::mma(xv[m], av[q], acc[m][q]);
            }
        }
        const int whole = K & ~63;
        if (whole < K && wave == W - 1) {  // the rest, a multiple of 8 columns, through buffer bounds
            const auto xbuf = buffer(x, ((rows - 1) * a.x_stride + K) * 2);
            const auto abuf = buffer(A, (int64_t)r * K * 2);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int k = whole + 32 * u + 8 * g;
                vec xv[2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    xv[m] = __builtin_bit_cast(vec, __builtin_amdgcn_raw_buffer_load_b128(
                        xbuf, k < K && 16 * m + i16 < rows ? (uint32_t)((16 * m + i16) * a.x_stride + k) * 2u : kNowhere, 0, 0));
#pragma unroll
                for (int q = 0; q < RT; ++q) {
                    const vec av = __builtin_bit_cast(vec, __builtin_amdgcn_raw_buffer_load_b128(
                        abuf, k < K && 16 * q + i16 < r ? (uint32_t)((16 * q + i16) * K + k) * 2u : kNowhere, 0, 0));
#pragma unroll
                    for (int m = 0; m < 2; ++m) acc[m][q] = Mfma<T>::mma(xv[m], av, acc[m][q]);
                }
            }
        }
        __syncthreads();  // the rings are idle
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < RT; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) smem_lora[(wave * 32 + 16 * m + 4 * g + e) * kLd + 16 * q + i16] = acc[m][q][e];
        __syncthreads();
        for (int i = threadIdx.x; i < 32 * 4 * RT; i += W * kWave) {
            const int j = 4 * (i % (4 * RT));
            f32x4* p = reinterpret_cast<f32x4*>(smem_lora + (i / (4 * RT)) * kLd + j);
            f32x4 v = *p;
#pragma unroll
            for (int w = 1; w < W; ++w) v += p[w * 32 * kLd / 4];
            *p = j < r ? v : f32x4{0.f, 0.f, 0.f, 0.f};  // r is a multiple of 8
        }
        __syncthreads();
        const float scale = a.scale ? a.scale[l] : 1.0f;
        split_sums16<T, 2, RT>(smem_lora, kLd, scale, h16, factor);
        __syncthreads();  // the sums have been read: the rings again
    }

    // 64 columns of the output from n on.  Rows of B as they lie in memory, r values
    // each; for r = 64 chunk c of row n at c ^ (n / 2 % 2 + 2 (n / 8 % 4)), so that the
    // 16 rows of a matrix operand meet 16 different places.
    const uint16_t* base = a.base + t0 * a.base_stride;
    uint16_t* out = a.out + t0 * a.out_stride;
    const uint16_t* B = some ? a.B + (int64_t)l * a.N * r : a.base;
    const int b_count = some ? r / 8 : 0;  // transfers: 64 rows of 2 r bytes
    uint32_t base_off[4];
    int base_col[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int row = 8 * u + (lane >> 3);
        base_off[u] = (uint32_t)((row < rows ? row : rows - 1) * a.base_stride) * 2u;
        base_col[u] = 8 * ((lane & 7) ^ line_swizzle(row));
    }
    auto row_swizzle = [&](int n) { return ((n >> 1) & 1) | (((n >> 3) & 3) << 1); };
    const uint32_t b_end = (uint32_t)N * (uint32_t)r * 2u - 16u;
    auto issue_base = [&](int n, uint32_t to) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = n + base_col[u] < N ? n + base_col[u] : N - 8;
            dma16s(base, base_off[u] + 2u * col, to + 1024u * u);
        }
    };
    auto issue = [&](int n, int stage) {
        const uint32_t to = ring_at + (uint32_t)(stage * Q::kBytes);
        issue_base(n, to);
#pragma unroll
        for (int u = 0; u < 2 * RT; ++u)
            if (u < b_count) {
                uint32_t off = (uint32_t)n * r * 2u + 1024u * u + 16u * lane;
                if (r == 64) off ^= 16u * row_swizzle(8 * u + (lane >> 3));
                dma16s(B, off < b_end ? off : b_end, to + 4096u + 1024u * u);
            }
    };
    // ranks 32 st + 8 g .. of the row of tile t and a half of the columns; past r: zeros
    auto read_b = [&](const uint8_t* p, int half, int t, int st) {
        const int row = 32 * half + 8 * (i16 >> 2) + 4 * t + (i16 & 3), j = 32 * st + 8 * g;
        uint32_t off = (uint32_t)row * r * 2u + (j < r ? 2u * j : 0u);
        if (r == 64) off ^= 16u * row_swizzle(row);
        u32x4 b = *reinterpret_cast<const u32x4*>(p + 4096 + off);
        const uint32_t keep = j < r ? ~0u : 0u;
        b &= keep;
        return b;
    };
    auto at = [&](int i) { return n_lo + 64 * (wave + W * i); };
    int own = 0;
    while (at(own) < n_hi) ++own;
#pragma unroll
    for (int d = 0; d < S - 1; ++d)
        if (d < own) issue(at(d), d);
    int stage = 0;
    for (int i = 0; i < own; ++i) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the stage read last is free
        if (i + S - 1 < own) issue(at(i + S - 1), stage == 0 ? S - 1 : stage - 1);
        // Stores are counted with the transfers: with the four of the last step behind
        // this stage's, all that was issued before them has landed.
        if (i + S - 1 < own) {
            if (some) {
                if (r == 16 * RT) asm volatile("s_waitcnt vmcnt(%0)" :: "n"((S - 1) * (4 + 2 * RT)) : "memory");
                else asm volatile("s_waitcnt vmcnt(%0)" :: "n"((S - 1) * 5) : "memory");
            } else {
                asm volatile("s_waitcnt vmcnt(%0)" :: "n"((S - 1) * 4) : "memory");
            }
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        uint8_t* p = ring + stage * Q::kBytes;
        const uint32_t p_at = ring_at + (uint32_t)(stage * Q::kBytes);
        stage = stage == S - 1 ? 0 : stage + 1;
        const int n = at(i);
        // 32 columns of the sum, in base's place; -> whether there is a NaN before base
        auto add_half = [&](auto mend, int half) {
            f32x4 d[2][2];
#pragma unroll
            for (int m = 0; m < 2; ++m) d[m][0] = d[m][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int st = 0; st < kKs; ++st) {
                    const u32x4 b = read_b(p, half, t, st);
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int q = 0; q < kParts; ++q)
                            d[m][t] = Mfma<T>::mma(__builtin_bit_cast(vec, b), __builtin_bit_cast(vec, h16[q][m][st]), d[m][t]);
                }
            const bool odd = any_nan<2>(d);
            if constexpr (decltype(mend)::value)
                take_first<2>(d, [&](int m, int t) {
                    f32x4 f = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int st = 0; st < kKs; ++st)
                        f = Mfma<T>::mma(__builtin_bit_cast(vec, read_b(p, half, t, st)), __builtin_bit_cast(vec, h16[0][m][st]), f);
                    return f;
                });
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                u32x4* q = reinterpret_cast<u32x4*>(p + (16 * m + i16) * 128 + 16 * ((4 * half + g) ^ line_swizzle(i16)));
                u32x4 v = *q;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = round_pair<T>(fmaf(factor[m], d[m][e / 2][2 * (e % 2)], T::to_f32((uint16_t)v[e])),
                                         fmaf(factor[m], d[m][e / 2][2 * (e % 2) + 1], T::to_f32((uint16_t)(v[e] >> 16))));
                *q = v;
            }
            return odd;
        };
        if (some) {
            const bool odd0 = add_half(std::false_type{}, 0), odd1 = add_half(std::false_type{}, 1);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (__builtin_expect(__ballot(odd0 || odd1) != 0, 0)) {  // once more, from base as it was
                issue_base(n, p_at);
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                add_half(std::true_type{}, 0);
                add_half(std::true_type{}, 1);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int row = 8 * u + (lane >> 3);
            const u32x4 v = *reinterpret_cast<const u32x4*>(p + 1024 * u + 16 * lane);
            if (((mine >> row) & 1) && n + base_col[u] < n_hi)
                *reinterpret_cast<u32x4*>(out + (int64_t)row * a.out_stride + n + base_col[u]) = v;
        }
    }
}

template <class T, int RT>
__global__ __launch_bounds__(Stage<RT>::W * kWave) void staged_kernel(LoraArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t0 = (int64_t)(blockIdx.x / (uint32_t)a.chunks) * 32;
    const uint32_t chunk = blockIdx.x % (uint32_t)a.chunks;
    int id = -2;
    if (lane < 32 && t0 + lane < a.T) {
        id = a.ids[t0 + lane];
        if (id < 0 || id >= a.L) id = -1;
    }
    uint64_t left = __ballot(id > -2);
    do {
        const int l = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t mine = __ballot(id == l);
        left &= ~mine;
        if (!(l < 0 && a.out == a.base)) {
            update_staged<T, RT>(a, t0, chunk, l, mine);
            if (left) __syncthreads();  // every wave's ring is idle
        }
    } while (left);
}

// Up to so many rows a block's adapters are spread over workgroups; beyond, the rows
// are taken for prompts, few adapters a block, and one workgroup takes them in turn.
// For rows that each have another adapter that is slow: 256 rows of 32 adapters, rank
// 16, 4096 x 4096, 17 us and 257 rows 104; sorted by adapter, 512 rows take 14.
constexpr int64_t kLoraDecodeRows = 256;

// Columns of a workgroup, in whole passes of its waves.  Each workgroup makes the
// first product again and reads its columns of the second, so its time goes with
// K + cols, and with the workgroups of a compute unit where there are more than
// one.  How many of a block's slots have an adapter is known on the device alone:
// the sum of the times for one and for all of them is what is made small.  (Two
// workgroups a compute unit in any case: 64 rows of 32 adapters, 6144 x 4096, rank
// 16, 19.4 us instead of 11.6; one in any case: 229 rows of 10 prompts, 8840 x 704,
// 22.3 instead of 11.2.)
int64_t chunk_columns(const LoraArgs& a, int64_t pass) {
    const int64_t passes = (a.N + pass - 1) / pass, units = compute_units();
    int64_t best = 0;
    double best_time = 0;
    for (const int64_t live : {a.blocks, a.blocks * a.slots})
        for (int64_t fill = 1; fill <= 2; ++fill) {
            int64_t c = fill * units / ((live + 7) / 8 * 8);
            c = c < 1 ? 1 : c > passes ? passes : c;
            const int64_t cols = (passes + c - 1) / c * pass;
            double time = 0;
            for (const int64_t l : {a.blocks, a.blocks * a.slots}) {
                const double share = (double)((l + 7) / 8 * 8 * c) / (double)units;
                time += (share > 1.0 ? share : 1.0) * (double)(a.K + cols);
            }
            if (best == 0 || time < best_time) {
                best = cols;
                best_time = time;
            }
        }
    return best;
}

template <class T, int MB, int RT, int W>
hipError_t launch_variant(const LoraArgs& args, hipStream_t s) {
    constexpr int lds = W * 16 * MB * Depth<MB, RT, W>::kLd * 4;
    static DeviceFlags set;
    hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&lora_kernel<T, MB, RT, W>), lds, set);
    if (e != hipSuccess) return e;
    constexpr int64_t kMostRows = (int64_t)1 << 20;  // of a launch: at most 2^22 workgroups
    for (int64_t t = 0; t < args.T; t += kMostRows) {
        LoraArgs a = args;
        a.T = args.T - t < kMostRows ? args.T - t : kMostRows;
        a.x += t * a.x_stride;
        a.base += t * a.base_stride;
        a.out += t * a.out_stride;
        a.ids += t;
        a.blocks = (a.T + 16 * MB - 1) / (16 * MB);
        // Decoding rows have many adapters: a workgroup for each that a block can
        // have.  Prompts have few: a workgroup takes its block's in turn.
        a.slots = 1;
        if (a.T <= kLoraDecodeRows) {
            a.slots = 16 * MB;
            if (a.slots > a.L + 1) a.slots = a.L + 1;
            if (a.slots > a.T) a.slots = a.T;
        }
        const int64_t pass = 32 * W;
        a.cols = chunk_columns(a, pass);
        a.chunks = (a.N + a.cols - 1) / a.cols;
        const int64_t groups = (a.blocks * a.slots + 7) / 8 * 8 * a.chunks;
        lora_kernel<T, MB, RT, W><<<(unsigned)groups, W * kWave, lds, s>>>(a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T, int RT>
hipError_t launch_staged(const LoraArgs& args, hipStream_t s) {
    typedef Stage<RT> Q;
    static DeviceFlags set;
    hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&staged_kernel<T, RT>), Q::kRing, set);
    if (e != hipSuccess) return e;
    constexpr int64_t kMostRows = (int64_t)1 << 20;
    for (int64_t t = 0; t < args.T; t += kMostRows) {
        LoraArgs a = args;
        a.T = args.T - t < kMostRows ? args.T - t : kMostRows;
        a.x += t * a.x_stride;
        a.base += t * a.base_stride;
        a.out += t * a.out_stride;
        a.ids += t;
        a.blocks = (a.T + 31) / 32;
        // one workgroup a compute unit (its rings take most of the LDS)
        const int64_t pass = 64 * Q::W, passes = (a.N + pass - 1) / pass;
        int64_t want = (compute_units() + a.blocks - 1) / a.blocks;
        if (want > passes) want = passes;
        a.cols = (passes + want - 1) / want * pass;
        a.chunks = (a.N + a.cols - 1) / a.cols;
        staged_kernel<T, RT><<<(unsigned)(a.blocks * a.chunks), Q::W * kWave, Q::kRing, s>>>(a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

// Rows of whole 16-byte vectors go through LDS where a block of 32 has few
// adapters (300 rows of 3 prompts, 4096 x 4096, rank 64: 25 us instead of 43; rank
// 16 from 2048 rows on, 1200 rows 25 and 22.5).  Else, for many rows, blocks of 32
// read an adapter half as often as those of 16.  Few rows of a small rank: 16 waves,
// so that one pass of loads covers 4096 columns.
template <class T>
hipError_t launch_type(const LoraArgs& a, hipStream_t s) {
    const bool vec = a.N % 8 == 0 && ((a.base_stride | a.out_stride) & 7) == 0 &&
                     ((reinterpret_cast<uintptr_t>(a.base) | reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0;
    const bool many = a.T >= 2048;
    if (vec && a.r <= 64 && a.K >= 64 && (many || (a.r > 16 && a.T > kLoraDecodeRows))) {
        if (a.r <= 16) return launch_staged<T, 1>(a, s);
        if (a.r <= 32) return launch_staged<T, 2>(a, s);
        return launch_staged<T, 4>(a, s);
    }
    if (a.r <= 16) return many ? launch_variant<T, 2, 1, 8>(a, s) : launch_variant<T, 1, 1, 16>(a, s);
    if (a.r <= 32) return many ? launch_variant<T, 2, 2, 8>(a, s) : launch_variant<T, 1, 2, 8>(a, s);
    if (a.r <= 64) return many ? launch_variant<T, 2, 4, 8>(a, s) : launch_variant<T, 1, 4, 8>(a, s);
    if (a.r <= 128) return many ? launch_variant<T, 2, 8, 8>(a, s) : launch_variant<T, 1, 8, 8>(a, s);
    return launch_variant<T, 1, 16, 8>(a, s);
}

}  // namespace

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) { return a.bf16 ? launch_type<BF16>(a, s) : launch_type<F16>(a, s); }

}  // namespace tq
