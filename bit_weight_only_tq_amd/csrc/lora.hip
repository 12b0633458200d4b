// Low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + scale[l] (x[t] A[l]^T) B[l]^T,  l = ids[t],
// and out[t] = base[t] where l names no adapter.
//
// Both thin products of a block of rows are one workgroup's work, so nothing
// passes through memory between them.  Rows stay in the order of the call: a
// workgroup takes the s-th different adapter of its block (blockIdx.y = s) and
// masks the others' rows, so one launch serves any mixture, prompts of one
// adapter as well as decoding rows of many, without sorting.
//
// The first product's sums are fp32.  They enter the second one as two 16-bit
// numbers each, the rounded value and the rounded rest, after a scaling of the
// row by a power of two to at most 1: together they keep at least 16 bits of the
// row's largest value, so that the adapter's update is rounded once, with the sum.

#include "tq_device.h"
#include "tq_internal.h"
#include "tq_tiles.h"

namespace tq {

namespace {

constexpr int kLoraWaves = 4;
constexpr int kLoraThreads = kLoraWaves * kWave;

template <class T>
__device__ __forceinline__ float round_to(float v) {
    return T::to_f32(T::from_f32_fast(v));
}

// MB blocks of 16 rows, rank up to 16 RT.  LDS: [waves][16 MB][16 RT] fp32 sums
// of the waves' columns.
template <class T, int MB, int RT>
__global__ __launch_bounds__(kLoraThreads) void lora_kernel(LoraArgs a, int cols) {
    typedef typename Mfma<T>::vec vec;
    constexpr int kRank = 16 * RT, kKs = (RT + 1) / 2;  // 32-deep steps of the second product
    extern __shared__ float smem_lora[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, i16 = lane & 15;
    const int64_t t0 = (int64_t)blockIdx.x * (16 * MB);

    // the s-th different adapter of the rows, -1: none; `mine`: its rows
    int id = -2;
    if (lane < 16 * MB && t0 + lane < a.T) {
        id = a.ids[t0 + lane];
        if (id < 0 || id >= a.L) id = -1;
    }
    uint64_t left = __ballot(id > -2), mine = 0;
    int l = -2;
    for (int s = 0; s <= (int)blockIdx.y; ++s) {
        if (!left) return;
        l = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        mine = __ballot(id == l);
        left &= ~mine;
    }
    if (l < 0 && a.out == a.base) return;
    const int64_t n_lo = (int64_t)blockIdx.z * cols;
    const int64_t n_hi = n_lo + cols < a.N ? n_lo + cols : a.N;
    const bool vec_ok = a.N % 8 == 0 && ((a.base_stride | a.out_stride) & 7) == 0 &&
                        ((reinterpret_cast<uintptr_t>(a.base) | reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0;

    uint4 hi[MB][kKs], lo[MB][kKs];  // operands of the second product: lane 16 g + i, row i, ranks 32 s + 8 g ..
    float factor[MB];
    if (l >= 0) {
        // x A^T: wave w takes the 32-column steps w, w + waves, ...
        f32x4 acc[MB][RT];
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[m][r] = f32x4{0.f, 0.f, 0.f, 0.f};
        const uint16_t* xr[MB];
        bool live[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            live[m] = (mine >> (16 * m + i16)) & 1;
            xr[m] = a.x + (live[m] ? t0 + 16 * m + i16 : t0) * a.x_stride;
        }
        const uint16_t* ar[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int j = 16 * r + i16 < a.r ? 16 * r + i16 : a.r - 1;
            ar[r] = a.A + ((int64_t)l * a.r + j) * a.K;
        }
        for (int64_t k0 = 32 * wave; k0 < a.K; k0 += 32 * kLoraWaves) {
            const int64_t k = k0 + 8 * g;
            const bool in = k < a.K;  // K is a multiple of 8
            uint4 xv[MB], av[RT];
#pragma unroll
            for (int m = 0; m < MB; ++m)
                xv[m] = in && live[m] ? *reinterpret_cast<const uint4*>(xr[m] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < RT; ++r) av[r] = in ? *reinterpret_cast<const uint4*>(ar[r] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    acc[m][r] = Mfma<T>::mma(__builtin_bit_cast(vec, xv[m]), __builtin_bit_cast(vec, av[r]), acc[m][r]);
        }
        // lane 16 g + i: rows 4 g .. 4 g + 3, rank 16 r + i
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    smem_lora[(wave * 16 * MB + 16 * m + 4 * g + e) * kRank + 16 * r + i16] = acc[m][r][e];
        __syncthreads();
        // the waves' sums, in their order
        for (int i = threadIdx.x; i < 16 * MB * kRank; i += kLoraThreads) {
            float v = smem_lora[i];
            for (int w = 1; w < kLoraWaves; ++w) v += smem_lora[w * 16 * MB * kRank + i];
            smem_lora[i] = i % kRank < a.r ? v : 0.0f;
        }
        __syncthreads();
        const float s = a.scale ? a.scale[l] : 1.0f;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const float* row = smem_lora + (16 * m + i16) * kRank;
            float h[kKs][8], most = 0.0f;
#pragma unroll
            for (int st = 0; st < kKs; ++st)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = 32 * st + 8 * g + e;
                    h[st][e] = j < kRank ? row[j] : 0.0f;
                    const float v = fabsf(h[st][e]);
                    if (v < __builtin_inff()) most = fmaxf(most, v);
                }
            most = fmaxf(most, __shfl_xor(most, 16, kWave));
            most = fmaxf(most, __shfl_xor(most, 32, kWave));
            int ex = 0;
            if (most > 0.0f) frexpf(most, &ex);  // most = f 2^ex, 1/2 <= f < 1
            ex = ex < -100 ? -100 : ex > 120 ? 120 : ex;  // 2^ex is a normal number
            factor[m] = ldexpf(s, ex);
#pragma unroll
            for (int st = 0; st < kKs; ++st) {
                uint32_t dh[4], dl[4];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = ldexpf(h[st][e], -ex);
                    const float top = round_to<T>(v);
                    const float rest = fabsf(v) < __builtin_inff() ? v - top : 0.0f;
                    const uint32_t bh = T::from_f32_fast(top), bl = T::from_f32_fast(rest);
                    dh[e / 2] = e % 2 ? dh[e / 2] | (bh << 16) : bh;
                    dl[e / 2] = e % 2 ? dl[e / 2] | (bl << 16) : bl;
                }
                hi[m][st] = make_uint4(dh[0], dh[1], dh[2], dh[3]);
                lo[m][st] = make_uint4(dl[0], dl[1], dl[2], dl[3]);
            }
        }
    }

    // h B^T, 32 columns a step of a wave: matrix row 4 g' + e of tile c is column
    // n + 8 g' + 4 c + e, so a lane ends with 8 columns in a row of one output row
    for (int64_t n = n_lo + 32 * wave; n < n_hi; n += 32 * kLoraWaves) {
        f32x4 d[MB][2];
#pragma unroll
        for (int m = 0; m < MB; ++m) d[m][0] = d[m][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (l >= 0) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                int64_t col = n + 8 * (i16 >> 2) + 4 * c + (i16 & 3);
                if (col >= a.N) col = a.N - 1;
                const uint16_t* br = a.B + ((int64_t)l * a.N + col) * a.r;
#pragma unroll
                for (int st = 0; st < kKs; ++st) {
                    const int j = 32 * st + 8 * g;
                    const uint4 b = j < a.r ? *reinterpret_cast<const uint4*>(br + j) : make_uint4(0, 0, 0, 0);
                    const vec bv = __builtin_bit_cast(vec, b);
#pragma unroll
                    for (int m = 0; m < MB; ++m) {
                        d[m][c] = Mfma<T>::mma(bv, __builtin_bit_cast(vec, hi[m][st]), d[m][c]);
                        d[m][c] = Mfma<T>::mma(bv, __builtin_bit_cast(vec, lo[m][st]), d[m][c]);
                    }
                }
            }
        }
        const int64_t c0 = n + 8 * g;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (!((mine >> (16 * m + i16)) & 1) || c0 >= n_hi) continue;
            const int64_t t = t0 + 16 * m + i16;
            const uint16_t* src = a.base + t * a.base_stride + c0;
            uint16_t* dst = a.out + t * a.out_stride + c0;
            if (vec_ok) {
                const uint4 v = *reinterpret_cast<const uint4*>(src);
                if (l < 0) {
                    *reinterpret_cast<uint4*>(dst) = v;
                    continue;
                }
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w = dword_of(v, e);
                    const float y0 = fmaf(factor[m], d[m][e / 2][2 * (e % 2)], T::to_f32((uint16_t)w));
                    const float y1 = fmaf(factor[m], d[m][e / 2][2 * (e % 2) + 1], T::to_f32((uint16_t)(w >> 16)));
                    o[e] = (uint32_t)T::from_f32_fast(y0) | ((uint32_t)T::from_f32_fast(y1) << 16);
                }
                *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (c0 + e >= n_hi) break;
                    dst[e] = l < 0 ? src[e] : T::from_f32_fast(fmaf(factor[m], d[m][e / 4][e % 4], T::to_f32(src[e])));
                }
            }
        }
    }
}

template <class T, int MB, int RT>
hipError_t launch_variant(const LoraArgs& a, hipStream_t s) {
    constexpr int lds = kLoraWaves * 16 * MB * 16 * RT * 4;
    static DeviceFlags set;
    hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&lora_kernel<T, MB, RT>), lds, set);
    if (e != hipSuccess) return e;
    const int64_t blocks = (a.T + 16 * MB - 1) / (16 * MB);
    int64_t slots = 16 * MB;
    if (slots > a.L + 1) slots = a.L + 1;
    if (slots > a.T) slots = a.T;
    int64_t cols = 512;
    const int64_t chunks = (a.N + cols - 1) / cols;
    const dim3 grid((unsigned)blocks, (unsigned)slots, (unsigned)chunks);
    lora_kernel<T, MB, RT><<<grid, kLoraThreads, lds, s>>>(a, (int)cols);
    return hipGetLastError();
}

template <class T>
hipError_t launch_type(const LoraArgs& a, hipStream_t s) {
    if (a.r <= 16) return launch_variant<T, 1, 1>(a, s);
    if (a.r <= 32) return launch_variant<T, 1, 2>(a, s);
    if (a.r <= 64) return launch_variant<T, 1, 4>(a, s);
    if (a.r <= 128) return launch_variant<T, 1, 8>(a, s);
    return launch_variant<T, 1, 16>(a, s);
}

}  // namespace

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) { return a.bf16 ? launch_type<BF16>(a, s) : launch_type<F16>(a, s); }

}  // namespace tq
