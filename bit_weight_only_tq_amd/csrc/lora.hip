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
// The first product's sums are fp32.  They enter the second one as two 16-bit
// numbers each, the rounded value and the rounded rest, after a scaling of the
// row by a power of two to at most 1: together they keep at least 16 bits of the
// row's largest value, so that the adapter's update is rounded once, with the sum.
//
// Rows, ranks and columns that are not there are read through buffer descriptors
// at an offset past their end, which gives zeros and drops stores: no load waits
// for a mask, and nothing branches.

#include "tq_device.h"
#include "tq_internal.h"
#include "tq_tiles.h"

namespace tq {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// A buffer of fewer than 2^31 bytes, and an offset that lies past any of them.
constexpr uint32_t kNowhere = 0x80000000u;
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
    static constexpr bool kEarly = RT <= 8;  // the first columns of B and base are asked for before x
    static constexpr int kLd = 16 * RT + 4;  // words of a row of sums in LDS
};

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
    extern __shared__ float smem_lora[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, i16 = lane & 15;
    const int N = (int)a.N, K = (int)a.K;
    const int n_lo = (int)chunk * (int)a.cols;
    const int n_hi = n_lo + (int)a.cols < N ? n_lo + (int)a.cols : N;
    const int rows = a.T - t0 < kRows ? (int)(a.T - t0) : kRows;
    const bool some = l >= 0;
    const bool vec_ok = N % 8 == 0 && ((a.base_stride | a.out_stride) & 7) == 0 &&
                        ((reinterpret_cast<uintptr_t>(a.base) | reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0;

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
    // Output columns n .. n + 31: matrix row 4 g' + e of tile c is column
    // n + 8 g' + 4 c + e, so that a lane ends with 8 columns in a row of one row.
    const uint32_t b_row = (uint32_t)((8 * (i16 >> 2) + (i16 & 3)) * a.r + 8 * g) * 2u;
    struct Cols {
        u32x4 b[2][kKs], base[MB];
    };
    auto load_cols = [&](int n, Cols& c) {
        if (some) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int st = 0; st < kKs; ++st)
                    c.b[t][st] = __builtin_amdgcn_raw_buffer_load_b128(
                        bbuf, 32 * st + 8 * g < a.r ? b_row + 8u * t * a.r + 64u * st : kNowhere, n * a.r * 2, 0);
        }
        if (vec_ok) {
#pragma unroll
            for (int m = 0; m < MB; ++m)
                c.base[m] = __builtin_amdgcn_raw_buffer_load_b128(from, n + 8 * g < n_hi ? from_row[m] : kNowhere, n * 2, 0);
        }
    };
    // Step i of a wave: two in a row where there are enough columns for every wave,
    // so that a wave's stores fill the cache lines that they begin.
    const bool pairs = a.cols >= 64 * W;
    auto at = [&](int i) { return n_lo + (pairs ? 64 * wave + 32 * (i & 1) + (i >> 1) * (64 * W) : 32 * wave + i * (32 * W)); };
    Cols cols[kAhead];
    if constexpr (Q::kEarly) load_cols(at(0), cols[0]);

    u32x4 hi[MB][kKs], lo[MB][kKs];  // operands of the second product: lane 16 g + i, row i, ranks 32 s + 8 g ..
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
        // the waves' sums, in their order
        for (int i = threadIdx.x; i < kRows * 4 * RT; i += kThreads) {
            f32x4* p = reinterpret_cast<f32x4*>(smem_lora + (i / (4 * RT)) * kLd + 4 * (i % (4 * RT)));
            f32x4 v = *p;
#pragma unroll
            for (int w = 1; w < W; ++w) v += p[w * kRows * kLd / 4];
            *p = v;
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const float* sums = smem_lora + (16 * m + i16) * kLd;
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
            int ex = most > 0.0f ? __builtin_amdgcn_frexp_expf(most) : 0;  // most = f 2^ex, 1/2 <= f < 1
            ex = ex < -100 ? -100 : ex > 120 ? 120 : ex;                   // 2^ex is a normal number
            factor[m] = ldexpf(scale, ex);
#pragma unroll
            for (int s = 0; s < kKs; ++s) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v0 = ldexpf(h[s][e / 2][2 * (e % 2)], -ex), v1 = ldexpf(h[s][e / 2][2 * (e % 2) + 1], -ex);
                    const uint32_t top = round_pair<T>(v0, v1);
                    const float r0 = v0 - T::to_f32((uint16_t)top), r1 = v1 - T::to_f32((uint16_t)(top >> 16));
                    hi[m][s][e] = top;
                    lo[m][s][e] = round_pair<T>(fabsf(v0) < __builtin_inff() ? r0 : 0.0f, fabsf(v1) < __builtin_inff() ? r1 : 0.0f);
                }
            }
        }
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
                    for (int m = 0; m < MB; ++m) {
                        d[m][t] = Mfma<T>::mma(bv, __builtin_bit_cast(vec, hi[m][st]), d[m][t]);
                        d[m][t] = Mfma<T>::mma(bv, __builtin_bit_cast(vec, lo[m][st]), d[m][t]);
                    }
                }
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (vec_ok) {
                u32x4 v = c.base[m];
                if (some) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = round_pair<T>(fmaf(factor[m], d[m][e / 2][2 * (e % 2)], T::to_f32((uint16_t)v[e])),
                                             fmaf(factor[m], d[m][e / 2][2 * (e % 2) + 1], T::to_f32((uint16_t)(v[e] >> 16))));
                }
                __builtin_amdgcn_raw_buffer_store_b128(v, to, n + 8 * g < n_hi ? to_row[m] : kNowhere, n * 2, 0);
            } else {
                uint16_t v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = __builtin_amdgcn_raw_buffer_load_b16(from, n + 8 * g + e < n_hi ? from_row[m] + 2u * e : kNowhere, n * 2, 0);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (some) v[e] = round_one<T>(fmaf(factor[m], d[m][e / 4][e % 4], T::to_f32(v[e])));
                    __builtin_amdgcn_raw_buffer_store_b16(v[e], to, n + 8 * g + e < n_hi ? to_row[m] + 2u * e : kNowhere, n * 2, 0);
                }
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

constexpr int64_t kLoraDecodeRows = 256;

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
        // columns of a workgroup: all of them where the blocks alone fill the compute
        // units, else chunks of whole passes of the waves
        const int64_t pass = 32 * W, passes = (a.N + pass - 1) / pass;
        int64_t want = (2 * compute_units() + a.blocks * a.slots - 1) / (a.blocks * a.slots);
        if (want > passes) want = passes;
        a.cols = (passes + want - 1) / want * pass;
        a.chunks = (a.N + a.cols - 1) / a.cols;
        const int64_t groups = (a.blocks * a.slots + 7) / 8 * 8 * a.chunks;
        lora_kernel<T, MB, RT, W><<<(unsigned)groups, W * kWave, lds, s>>>(a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

// Few rows: 16 waves, so that one pass of loads covers 4096 columns.  Many: 32
// rows, so that an adapter is read half as often.
template <class T>
hipError_t launch_type(const LoraArgs& a, hipStream_t s) {
    if (a.T >= 2048) {
        if (a.r <= 16) return launch_variant<T, 2, 1, 8>(a, s);
        if (a.r <= 32) return launch_variant<T, 2, 2, 8>(a, s);
        if (a.r <= 64) return launch_variant<T, 2, 4, 8>(a, s);
        if (a.r <= 128) return launch_variant<T, 2, 8, 8>(a, s);
        return launch_variant<T, 1, 16, 8>(a, s);
    }
    if (a.r <= 16) return launch_variant<T, 1, 1, 16>(a, s);
    if (a.r <= 32) return launch_variant<T, 1, 2, 8>(a, s);
    if (a.r <= 64) return launch_variant<T, 1, 4, 8>(a, s);
    if (a.r <= 128) return launch_variant<T, 1, 8, 8>(a, s);
    return launch_variant<T, 1, 16, 8>(a, s);
}

}  // namespace

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) { return a.bf16 ? launch_type<BF16>(a, s) : launch_type<F16>(a, s); }

}  // namespace tq
