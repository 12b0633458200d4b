// Products grouped by expert: row p of C, offsets[e] <= p < offsets[e + 1], is a
// row of A times expert e's packed weights (ternary or W4A16), fp32 sums.
//
// The numbers of rows are known on the device alone.  A launch has workgroups
// for as many blocks of rows as P rows of E experts can make at most; each finds
// its expert and rows by a scan over the offsets and leaves if there are none.

#include "tq_device.h"
#include "tq_internal.h"
#include "tq_tiles.h"

namespace tq {

namespace {

// Block `y` of BM rows among all experts' blocks (an expert's last one may have
// fewer rows): its expert, first row and number of rows; rows 0: no such block.
// Offsets are held to [0, P], so nothing outside A and C is named by any values.
struct Block {
    int expert;
    int64_t row;
    int rows;
};
__device__ __forceinline__ Block find_block(const int32_t* offsets, int E, int64_t P, int BM, int64_t y) {
    const int lane = threadIdx.x & 63;
    int64_t before = 0;  // blocks of the experts before this 64
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        int64_t lo = 0, hi = 0;
        if (e < E) {
            lo = offsets[e];
            hi = offsets[e + 1];
            lo = lo < 0 ? 0 : lo > P ? P : lo;
            hi = hi < lo ? lo : hi > P ? P : hi;
        }
        const int n = (int)((hi - lo + BM - 1) / BM);
        int sum = n;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(sum, d, kWave);
            if (lane >= d) sum += o;
        }
        const uint64_t past = __ballot(before + sum > y);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int64_t first = before + __shfl(sum - n, l, kWave);
            const int64_t row = (int64_t)__shfl((int)lo, l, kWave) + (y - first) * BM;
            const int64_t end = (int64_t)__shfl((int)hi, l, kWave);
            return Block{__builtin_amdgcn_readfirstlane(e0 + l), row, (int)(end - row < BM ? end - row : BM)};
        }
        before += __shfl(sum, 63, kWave);
    }
    return Block{0, 0, 0};
}

// The row of A that row p of C is made from; entries of `rows` outside [0, P)
// are held to it.
__device__ __forceinline__ int64_t source_row(const ExpertArgs& a, int64_t p) {
    if (!a.rows) return p;
    const int32_t pair = a.rows[p];
    const int32_t most = (int32_t)(a.P - 1);
    return (pair < 0 ? 0 : pair > most ? most : pair) / a.fan;
}

__device__ __forceinline__ float gate(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// ---------------------------------------------------------------- few rows
//
// 16 rows of one expert and R blocks of 16 weight rows a workgroup, its waves
// dealing the columns.  A wave reads weights and activations straight into
// matrix operands: lane 16 g + i has 16 bytes of codes of weight row i and the
// activations of the same columns of row i (natural order, tq_tiles.h).
// W4A16: a step is one scale group of 128 columns, its sum starts from zero and
// is scaled into the result; ternary: 256 columns, scaled at the end.  The waves'
// results meet in LDS and are summed in the waves' order.
// Gated: the first half of the R blocks are rows of the gate, the second half the
// same rows of the up projection.
constexpr int kStreamWaves = 8;

template <class T, int FMT, bool ASYM, bool GATED, int R>
__global__ __launch_bounds__(kStreamWaves * kWave) void stream_kernel(ExpertArgs a) {
    typedef typename Mfma<T>::vec vec;
    constexpr int kCols = FMT == 0 ? 256 : 128;  // of a step
    constexpr int kUnits = FMT == 0 ? 8 : 4;     // 8-column units a lane and step
    constexpr int kOut = GATED ? R / 2 : R;      // blocks of 16 output columns
    __shared__ f32x4 red[kStreamWaves][R][kWave];
    const int64_t id = a.first + blockIdx.x;
    const int64_t tiles = ((GATED ? a.N / 2 : a.N) + 16 * kOut - 1) / (16 * kOut);
    const Block blk = find_block(a.offsets, (int)a.E, a.P, 16, id / tiles);
    if (blk.rows == 0) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int g = lane >> 4, i16 = lane & 15;
    const int64_t N = a.N, K = a.K;
    const int64_t width = GATED ? N / 2 : N;       // output columns
    const int64_t n0 = id % tiles * (16 * kOut);
    const int64_t rb = FMT == 0 ? K / 4 : K / 2;   // code bytes of a weight row
    const int64_t G = K / 128;
    const bool live = i16 < blk.rows;
    const uint16_t* arow = a.A + (live ? source_row(a, blk.row + i16) : 0) * K;
    int64_t wr[R];  // weight rows (past the end: the last)
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t c = n0 + 16 * (r % kOut) + i16;
        wr[r] = (int64_t)blk.expert * N + (c < width ? c : width - 1) + (r >= kOut ? width : 0);
    }
    const int steps = (int)((K + kCols - 1) / kCols);
    const int from = (int)((int64_t)steps * wave / kStreamWaves), to = (int)((int64_t)steps * (wave + 1) / kStreamWaves);
    const uint32_t magic_v = vgpr_const<kMagic2>();
    const uint32_t mask_v = sgpr_const<0x00F0000Fu>();
    const f16x2 mul = __builtin_bit_cast(f16x2, 0x2C003C00u);  // (1, 1/16)
    const NatConsts nat = nat_consts();
    f32x4 acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int step = from; step < to; ++step) {
        const int64_t c0 = (int64_t)step * kCols + g * (kCols / 4);  // this lane's columns
        const bool in = FMT == 1 || c0 < K;                          // ternary: K is a multiple of 64 alone
        uint4 q[R], av[kUnits];
#pragma unroll
        for (int r = 0; r < R; ++r)
            q[r] = in ? *reinterpret_cast<const uint4*>(a.w + wr[r] * rb + (FMT == 0 ? c0 / 4 : c0 / 2)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            av[u] = in && live ? *reinterpret_cast<const uint4*>(arow + c0 + 8 * u) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if constexpr (FMT == 0) {
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    const uint32_t x = dword_of(q[r], u / 2);
                    const uint4 b = u % 2 ? nat_quad<1>(x, magic_v, nat) : nat_quad<0>(x, magic_v, nat);
                    acc[r] = Mfma<T>::mma(__builtin_bit_cast(vec, av[u]), __builtin_bit_cast(vec, b), acc[r]);
                }
            } else {
                f16x2 sub = w4_nat_sub(8u);
                if constexpr (ASYM) sub = w4_nat_sub(a.zeros[wr[r] * G + step]);
                f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    const uint4 b = nat_w4_quad<T>(dword_of(q[r], u), mask_v, magic_v, mul, sub);
                    sum = Mfma<T>::mma(__builtin_bit_cast(vec, av[u]), __builtin_bit_cast(vec, b), sum);
                }
                const float s = f16_bits_to_f32(a.scale[wr[r] * G + step]);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][i] = fmaf(s, sum[i], acc[r][i]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) red[wave][r][lane] = acc[r];
    __syncthreads();
    for (int t = threadIdx.x; t < kOut * kWave; t += kStreamWaves * kWave) {
        const int r = t / kWave, l = t % kWave;
        const int64_t c = n0 + 16 * r + (l & 15);
        if (c >= width) continue;
        f32x4 v = red[0][r][l];
        for (int w = 1; w < kStreamWaves; ++w) v += red[w][r][l];
        f32x4 u = v;
        if constexpr (GATED) {
            u = red[0][r + kOut][l];
            for (int w = 1; w < kStreamWaves; ++w) u += red[w][r + kOut][l];
        }
        const int64_t n = (int64_t)blk.expert * N + c;
        float sv = 1.0f, su = 1.0f;
        if constexpr (FMT == 0) {
            sv = f16_bits_to_f32(a.scale[n]) * Mfma<T>::kUnit;
            if constexpr (GATED) su = f16_bits_to_f32(a.scale[n + width]) * Mfma<T>::kUnit;
        }
        const float bv = a.bias ? T::to_f32(a.bias[n]) : 0.0f;
        const float bu = GATED && a.bias ? T::to_f32(a.bias[n + width]) : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * (l >> 4) + i;
            if (row >= blk.rows) continue;
            float y = fmaf(v[i], sv, bv);
            if constexpr (GATED) y = gate(y, fmaf(u[i], su, bu));
            a.C[(blk.row + row) * width + c] = T::from_f32_fast(y);
        }
    }
}

// Blocks of BM rows that P rows of E experts make at most.
int64_t most_blocks(int64_t P, int64_t E, int64_t BM) {
    const int64_t used = P < E ? P : E;
    return (P + used * (BM - 1)) / BM;
}

template <class T, int FMT, bool ASYM, bool GATED>
hipError_t launch_stream(const ExpertArgs& args, hipStream_t s) {
    constexpr int R = 4;
    constexpr int kOut = GATED ? R / 2 : R;
    const int64_t width = GATED ? args.N / 2 : args.N;
    const int64_t groups = (width + 16 * kOut - 1) / (16 * kOut) * most_blocks(args.P, args.E, 16);
    ExpertArgs a = args;
    for (a.first = 0; a.first < groups; a.first += kMaxGroups) {
        const int64_t n = groups - a.first < kMaxGroups ? groups - a.first : kMaxGroups;
        stream_kernel<T, FMT, ASYM, GATED, R><<<(unsigned)n, kStreamWaves * kWave, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T>
hipError_t launch_type(const ExpertArgs& a, hipStream_t s) {
    if (a.fmt == 0) return a.gated ? launch_stream<T, 0, false, true>(a, s) : launch_stream<T, 0, false, false>(a, s);
    if (a.zeros) return a.gated ? launch_stream<T, 1, true, true>(a, s) : launch_stream<T, 1, true, false>(a, s);
    return a.gated ? launch_stream<T, 1, false, true>(a, s) : launch_stream<T, 1, false, false>(a, s);
}

}  // namespace

hipError_t launch_experts(const ExpertArgs& a, hipStream_t s) {
    return a.bf16 ? launch_type<BF16>(a, s) : launch_type<F16>(a, s);
}

}  // namespace tq
