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
            const int64_t first = before + __builtin_amdgcn_readlane(sum - n, l);
            const int64_t row = __builtin_amdgcn_readlane((int)lo, l) + (y - first) * BM;
            const int64_t end = __builtin_amdgcn_readlane((int)hi, l);
            return Block{e0 + l, row, (int)(end - row < BM ? end - row : BM)};
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return Block{0, 0, 0};
}

// All experts' blocks.
__device__ __forceinline__ int64_t count_blocks(const int32_t* offsets, int E, int64_t P, int BM) {
    const int lane = threadIdx.x & 63;
    int sum = 0;  // a lane's experts: their rows are at most P together where offsets ascend
    for (int e = lane; e < E; e += 64) {
        int64_t lo = offsets[e], hi = offsets[e + 1];
        lo = lo < 0 ? 0 : lo > P ? P : lo;
        hi = hi < lo ? lo : hi > P ? P : hi;
        sum += (int)((hi - lo + BM - 1) / BM);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d, kWave);
    return __builtin_amdgcn_readfirstlane(sum);
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

// ---------------------------------------------------------------- many rows
//
// BM rows of one expert and 256 weight rows a workgroup, four waves of BM x 64.
// Activations and codes come by DMA (no registers) into a ring of three stages of
// 64 columns, two ahead of the matrix cores: BM rows x 128 bytes, 16-byte chunks
// XOR-swizzled (chunk c of row r at c ^ (r % 8)), and 256 weight rows x 16 or 32
// bytes.  Codes are unpacked in registers in the natural order of their columns.
// Two workgroups share a compute unit, so one's barriers lie under the other's
// products.
//
// W4A16: the accumulators hold the sum in units of the current group's scale, so
// entering a group multiplies them by the ratio of the last scale to its own, and
// the operands stay the exact q - z.  (Scaling every group's sum into a second set
// of accumulators costs as many instructions and twice the registers, which
// halves the tile.)  A group whose scale is 0 keeps the last unit, and its code
// words are replaced by those of zero weights.
namespace tile {

constexpr int BN = 256, BK = 64, WN = 64, TN = 4;
constexpr int kWaves = 4, kThreads = kWaves * kWave;
constexpr int kStages = 3;
constexpr int kEpiLd = WN + 8;  // halves of a row staged for its store
constexpr int kGroupRows = 8;   // blocks of rows that pass over all columns together

template <int FMT, int BM>
struct Ring {
    static constexpr int kABytes = BM * BK * 2;
    static constexpr int kBBytes = BN * BK / (FMT == 0 ? 4 : 2);
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kBytes = kStages * kStageBytes;
    static constexpr int AU = BM / 32, BU = kBBytes / 4096;  // 1-KB transfers a wave and stage
    static_assert(kWaves * 32 * kEpiLd * 2 <= kBytes, "epilogue staging must fit in the ring");
};

// Eight columns of a code word as exact operands.  fp16: q - z (add: the packed
// constants of z).  bf16: (q - z) / 16, two nibbles' signed values by the
// converter of offset 4-bit numbers, (n ^ 8) / 16 - 1/2; `add` is (8 - z) / 16.
// keep is 0 where the group's scale is 0 (all ones elsewhere): its words then
// become those of zero weights.
template <class T, bool ASYM>
struct W4Unpack;
template <bool ASYM>
struct W4Unpack<F16, ASYM> {
    static constexpr float kUnit = 1.0f;
    uint32_t keep = ~0u;
    f16x2 add = w4_nat_sub(8u);
    __device__ __forceinline__ void set(uint32_t z, bool zero) {
        keep = zero ? 0u : ~0u;
        if constexpr (ASYM) add = w4_nat_sub(zero ? 0u : z);
    }
    __device__ __forceinline__ uint4 quad(uint32_t x, uint32_t mask_v, uint32_t magic_v) const {
        const uint32_t y = ASYM ? x & keep : (x & keep) | (0x88888888u & ~keep);
        return nat_w4_quad<F16>(y, mask_v, magic_v, __builtin_bit_cast(f16x2, 0x2C003C00u), add);  // (1, 1/16)
    }
};
template <bool ASYM>
struct W4Unpack<BF16, ASYM> {
    static constexpr float kUnit = 16.0f;
    uint32_t keep = ~0u;
    float add = 0.0f;
    __device__ __forceinline__ void set(uint32_t z, bool zero) {
        keep = zero ? 0u : ~0u;
        if constexpr (ASYM) add = zero ? 0.0f : (float)(8 - (int)z) * 0.0625f;
    }
    template <int I>
    __device__ __forceinline__ float one(uint32_t v) const {
        const float f = __builtin_amdgcn_cvt_off_f32_i4((int)__builtin_amdgcn_ubfe(v, 8 * I, 8));
        if constexpr (ASYM) return f + add;
        else return f;
    }
    template <int I>
    __device__ __forceinline__ uint32_t pair(uint32_t lo, uint32_t hi) const {
        return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)one<I>(lo), (__bf16)one<I>(hi)});
    }
    __device__ __forceinline__ uint4 quad(uint32_t x, uint32_t, uint32_t) const {
        uint32_t lo = (x ^ 0x88888888u) & keep;
        uint32_t hi = lo >> 4;
        asm("" : "+v"(lo), "+v"(hi));  // two words of bytes, not eight shifts
        return make_uint4(pair<0>(lo, hi), pair<1>(lo, hi), pair<2>(lo, hi), pair<3>(lo, hi));
    }
};

// The tile of workgroup `id`: workgroups go to the XCDs (each with an L2 of its
// own) in turn, so each XCD takes a contiguous share of the tiles, in the order
// of kGroupRows blocks of rows over all columns.
struct Place {
    Block blk;
    int n_tile;
};
__device__ __forceinline__ Place find_tile(const ExpertArgs& a, int BM, uint32_t tiles_n, uint32_t id) {
    const uint32_t blocks = (uint32_t)count_blocks(a.offsets, (int)a.E, a.P, BM);
    const uint32_t total = blocks * tiles_n;  // below 2^31: the launcher's check
    const uint32_t xcd = id & 7, s = id >> 3, per = total / 8, more = total % 8;
    if (s >= per + (xcd < more ? 1 : 0)) return Place{Block{0, 0, 0}, 0};
    const uint32_t tile = xcd * per + (xcd < more ? xcd : more) + s;
    const uint32_t band = tile / (kGroupRows * tiles_n), in = tile - band * kGroupRows * tiles_n;
    const uint32_t left = blocks - band * kGroupRows;
    const uint32_t rows = left < kGroupRows ? left : kGroupRows;
    const int n_tile = __builtin_amdgcn_readfirstlane((int)(in / rows));
    const int y = __builtin_amdgcn_readfirstlane((int)(band * kGroupRows + in % rows));
    return Place{find_block(a.offsets, (int)a.E, a.P, BM, y), n_tile};
}

template <class T, int FMT, bool ASYM, bool GATED, int BM>
__global__ __launch_bounds__(kThreads, 2) void kernel(ExpertArgs a) {
    typedef typename Mfma<T>::vec vec;
    typedef Ring<FMT, BM> G;
    constexpr int TM = BM / 16, AU = G::AU, BU = G::BU;
    constexpr int kCols = GATED ? BN / 2 : BN;  // output columns of the tile
    extern __shared__ uint4 smem_tile[];
    uint8_t* lds = reinterpret_cast<uint8_t*>(smem_tile);
    const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem_tile;
    const int64_t N = a.N, K = a.K, width = GATED ? N / 2 : N;
    const Place place = find_tile(a, BM, (uint32_t)((width + kCols - 1) / kCols), (uint32_t)a.first + blockIdx.x);
    const Block blk = place.blk;
    if (blk.rows == 0) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, i16 = lane & 15;
    const int64_t c0 = (int64_t)place.n_tile * kCols;
    const int64_t rb = FMT == 0 ? K / 4 : K / 2;
    const int64_t GK = K / 128;
    // weight row of row lr of the tile: 64 a wave; gated: 32 of the gate, then the
    // same 32 of the up projection.  Past the end: the last.
    auto weight_row = [&](int lr) {
        int64_t c;
        int64_t half = 0;
        if constexpr (GATED) {
            c = c0 + (lr >> 6) * 32 + (lr & 31);
            half = (lr & 32) ? width : 0;
        } else {
            c = c0 + lr;
        }
        return (uint32_t)(half + (c < width ? c : width - 1));
    };
    const uint8_t* w_exp = a.w + (int64_t)blk.expert * N * rb;             // this expert's
    const uint16_t* s_exp = a.scale + (int64_t)blk.expert * N * (FMT == 0 ? 1 : GK);
    const uint8_t* z_exp = ASYM ? a.zeros + (int64_t)blk.expert * N * GK : nullptr;

    // DMA sources of this lane: 16 bytes of activation row 8 (AU w + u) + l / 8, and
    // of weight row 64 w + l (ternary) or 32 (2 w + u) + l / 2 (W4A16)
    const uint8_t* a_src[AU];
#pragma unroll
    for (int u = 0; u < AU; ++u) {
        const int r = 8 * (AU * wave + u) + (lane >> 3);
        const int64_t row = source_row(a, blk.row + (r < blk.rows ? r : blk.rows - 1));
        a_src[u] = reinterpret_cast<const uint8_t*>(a.A + row * K) + 16 * ((lane & 7) ^ (lane >> 3));
    }
    uint32_t b_src[BU];  // from the expert's weights: below 2^31 bytes
#pragma unroll
    for (int u = 0; u < BU; ++u) {
        if constexpr (FMT == 0) b_src[u] = weight_row(64 * wave + lane) * (uint32_t)rb;
        else b_src[u] = weight_row(32 * (2 * wave + u) + (lane >> 1)) * (uint32_t)rb + 16 * (lane & 1);
    }
    // The sources run on from stage to stage and stay at the last K-step, so that the
    // counts of transfers in flight stay exact; what is issued past the end goes
    // into a stage that nobody reads any more.
    const uint8_t* b_at = w_exp;
    const int nk = (int)(K / BK);
    int issued = 0;
    uint32_t issue_at = lds_base;  // the stage that the next issue fills
    auto issue = [&]() {
#pragma unroll
        for (int u = 0; u < AU; ++u) dma16(a_src[u], issue_at + 1024u * (AU * wave + u));
#pragma unroll
        for (int u = 0; u < BU; ++u) dma16s(b_at, b_src[u], issue_at + G::kABytes + 1024u * (BU * wave + u));
        issue_at = issue_at == lds_base + (kStages - 1) * G::kStageBytes ? lds_base : issue_at + G::kStageBytes;
        const bool on = ++issued < nk;
        b_at += on ? (FMT == 0 ? BK / 4 : BK / 2) : 0;
#pragma unroll
        for (int u = 0; u < AU; ++u) a_src[u] += on ? 2 * BK : 0;
    };
    // all but the stage issued last have landed
    auto wait_stage = [&]() { asm volatile("s_waitcnt vmcnt(%0)" :: "n"(AU + BU) : "memory"); };

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int a_frag = i16 * (BK * 2);
    const int swz = i16 & 7;
    const int b_frag = G::kABytes + (wave * WN + i16) * (FMT == 0 ? 16 : 32) + (FMT == 0 ? 4 : 8) * g;
    const uint32_t magic_v = vgpr_const<kMagic2>();
    const uint32_t mask_v = sgpr_const<0x00F0000Fu>();
    const NatConsts nat = nat_consts();
    uint32_t sr[TN];  // index of the scales of this lane's weight rows
#pragma unroll
    for (int j = 0; j < TN; ++j) sr[j] = weight_row(wave * WN + 16 * j + i16) * (uint32_t)(FMT == 0 ? 1 : GK);
    W4Unpack<T, ASYM> un[TN];
    float unit[TN];              // scale that the accumulators are in units of
    uint16_t next_s[TN];         // the next group's
    uint8_t next_z[TN];
    auto load_scales = [&](int64_t group) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            next_s[j] = (s_exp + group)[sr[j]];
            if constexpr (ASYM) next_z[j] = (z_exp + group)[sr[j]];
        }
    };

    if constexpr (FMT == 1) {
#pragma unroll
        for (int j = 0; j < TN; ++j) unit[j] = 1.0f;
        load_scales(0);
    }
    issue();
    issue();
    wait_stage();
    stage_barrier();
    uint32_t read_at = 0;  // of the stage that is read
    constexpr int kHalves = FMT == 1 ? 2 : 1;  // K-steps of a scale group
    for (int kt = 0; kt < nk; kt += kHalves) {
        if constexpr (FMT == 1) {  // enter group kt / 2
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const float s = f16_bits_to_f32(next_s[j]);
                const bool zero = s == 0.0f;
                un[j].set(ASYM ? next_z[j] : 8u, zero);
                float r = __builtin_amdgcn_rcpf(s);
                r = unit[j] * fmaf(fmaf(-s, r, 1.0f), r, r);  // a Newton step: within an ulp
                if (zero) r = 1.0f;
                else unit[j] = s;
                if (kt > 0) {
#pragma unroll
                    for (int i = 0; i < TM; ++i) acc[i][j] *= r;
                }
            }
            load_scales(kt + 2 < nk ? kt / 2 + 1 : kt / 2);
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            issue();  // K-step kt + h + 2
            const uint8_t* sbase = lds + read_at;
            read_at = read_at == (kStages - 1) * G::kStageBytes ? 0 : read_at + G::kStageBytes;
            uint2 x[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                if constexpr (FMT == 0) x[j].x = *reinterpret_cast<const uint32_t*>(sbase + b_frag + 16 * 16 * j);
                else x[j] = *reinterpret_cast<const uint2*>(sbase + b_frag + 16 * 32 * j);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (s) asm volatile("" ::: "memory");  // the second half's loads stay behind the first: registers
                const uint8_t* arow = sbase + a_frag + 16 * ((2 * g + s) ^ swz);
                vec bf[TN];
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    uint4 b;
                    if constexpr (FMT == 0) b = s ? nat_quad<1>(x[j].x, magic_v, nat) : nat_quad<0>(x[j].x, magic_v, nat);
                    else b = un[j].quad(s ? x[j].y : x[j].x, mask_v, magic_v);
                    bf[j] = __builtin_bit_cast(vec, b);
                }
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const vec af = __builtin_bit_cast(vec, *reinterpret_cast<const uint4*>(arow + i * 16 * (BK * 2)));
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[i][j] = Mfma<T>::mma(af, bf[j], acc[i][j]);
                }
            }
            wait_stage();     // the next stage has landed
            stage_barrier();  // ... for every wave, and nobody reads this one any more
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();  // the ring is idle from here on

    // epilogue: a wave's 32 rows at a time through an LDS area of its own, so that a
    // lane stores 16 bytes in a row
    uint16_t* stg = reinterpret_cast<uint16_t*>(lds) + wave * 32 * kEpiLd;
    float sc[TN], bi[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        if constexpr (FMT == 0) sc[j] = f16_bits_to_f32(s_exp[sr[j]]) * Mfma<T>::kUnit;
        else sc[j] = unit[j] * W4Unpack<T, ASYM>::kUnit;
        bi[j] = a.bias ? T::to_f32(a.bias[(int64_t)blk.expert * N + weight_row(wave * WN + 16 * j + i16)]) : 0.0f;
    }
    constexpr int kWaveCols = GATED ? WN / 2 : WN;
    constexpr int kLanesPerRow = kWaveCols / 8, kRowsPerPass = 64 / kLanesPerRow;
    const bool vec_ok = width % 8 == 0 && (reinterpret_cast<uintptr_t>(a.C) & 15u) == 0;
#pragma unroll
    for (int slab = 0; slab < TM / 2; ++slab) {
#pragma unroll
        for (int ii = 0; ii < 2; ++ii) {
            const int i = 2 * slab + ii;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                uint16_t* row = stg + (16 * ii + 4 * g + r) * kEpiLd + i16;
                if constexpr (GATED) {
#pragma unroll
                    for (int j = 0; j < TN / 2; ++j)
                        row[16 * j] = T::from_f32_fast(gate(fmaf(acc[i][j][r], sc[j], bi[j]),
                                                            fmaf(acc[i][j + TN / 2][r], sc[j + TN / 2], bi[j + TN / 2])));
                } else {
#pragma unroll
                    for (int j = 0; j < TN; ++j) row[16 * j] = T::from_f32_fast(fmaf(acc[i][j][r], sc[j], bi[j]));
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 32 / kRowsPerPass; ++q) {
            const int row = lane / kLanesPerRow + kRowsPerPass * q;
            const int col = 8 * (lane % kLanesPerRow);
            const int64_t n = c0 + wave * kWaveCols + col;
            if (32 * slab + row >= blk.rows) continue;
            uint16_t* dst = a.C + (blk.row + 32 * slab + row) * width + n;
            const uint4 v = *reinterpret_cast<const uint4*>(stg + row * kEpiLd + col);
            if (vec_ok && n + 8 <= width) {
                *reinterpret_cast<uint4*>(dst) = v;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < width) dst[e] = (uint16_t)(dword_of(v, e / 2) >> (16 * (e % 2)));
            }
        }
    }
}

}  // namespace tile

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

template <class T, int FMT, bool ASYM, bool GATED, int BM>
hipError_t launch_tile(const ExpertArgs& args, hipStream_t s) {
    typedef tile::Ring<FMT, BM> G;
    static DeviceFlags lds_limit_set;
    hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&tile::kernel<T, FMT, ASYM, GATED, BM>), G::kBytes, lds_limit_set);
    if (e != hipSuccess) return e;
    const int64_t width = GATED ? args.N / 2 : args.N, cols = GATED ? tile::BN / 2 : tile::BN;
    const int64_t groups = ((width + cols - 1) / cols * most_blocks(args.P, args.E, BM) + 7) / 8 * 8;
    if (groups >= (int64_t)1 << 31) return hipErrorInvalidValue;  // an output of more than 2^44 values
    ExpertArgs a = args;
    constexpr int64_t kMost = kMaxGroups / 8 * 8;
    for (a.first = 0; a.first < groups; a.first += kMost) {
        const int64_t n = groups - a.first < kMost ? groups - a.first : kMost;
        tile::kernel<T, FMT, ASYM, GATED, BM><<<(unsigned)n, tile::kThreads, G::kBytes, s>>>(a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T, int FMT, bool ASYM, bool GATED>
hipError_t launch_rows(const ExpertArgs& a, hipStream_t s) {
    const int64_t rows = a.P / (a.P < a.E ? a.P : a.E);  // of an expert, on average
    if (rows >= 48) return launch_tile<T, FMT, ASYM, GATED, 128>(a, s);
    if (rows >= 16) return launch_tile<T, FMT, ASYM, GATED, 64>(a, s);
    return launch_stream<T, FMT, ASYM, GATED>(a, s);
}

template <class T>
hipError_t launch_type(const ExpertArgs& a, hipStream_t s) {
    if (a.fmt == 0) return a.gated ? launch_rows<T, 0, false, true>(a, s) : launch_rows<T, 0, false, false>(a, s);
    if (a.zeros) return a.gated ? launch_rows<T, 1, true, true>(a, s) : launch_rows<T, 1, true, false>(a, s);
    return a.gated ? launch_rows<T, 1, false, true>(a, s) : launch_rows<T, 1, false, false>(a, s);
}

}  // namespace

hipError_t launch_experts(const ExpertArgs& a, hipStream_t s) {
    return a.bf16 ? launch_type<BF16>(a, s) : launch_type<F16>(a, s);
}

}  // namespace tq
