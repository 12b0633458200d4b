// Products grouped by expert: row p of C, offsets[e] <= p < offsets[e + 1], is a
// row of A times expert e's packed weights (ternary or W4A16), fp32 sums.
//
// The numbers of rows are known on the device alone.  A launch has workgroups
// for as many blocks of rows as P rows of E experts can make at most; each finds
// its expert and rows by a scan over the offsets and leaves if there are none.

#include "tq.h"
#include "tq_device.h"
#include "tq_internal.h"
#include "tq_tiles.h"

namespace tq {

namespace {

// A block of BM rows (an expert's last one may have fewer): its expert, first row
// and number of rows; rows 0: no such block.
struct Block {
    int expert;
    int64_t row;
    int rows;
};

// Inclusive sum over the wave: shifts within the rows of 16 lanes, then the rows'
// last lanes to the rows behind them.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15 to rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast 31 to rows 2 and 3
    return v;
}

// All experts' blocks: a lane has the blocks of V experts in a row.  Offsets are
// held to [0, P], so nothing outside A and C is named by any values.
struct Blocks {
    int V, sum;  // blocks up to and with this lane's experts
    int own;     // of its own
    int total;
};
struct Rows {
    int lo, hi;
};
__device__ __forceinline__ Rows rows_of(const ExpertArgs& a, int e) {
    const int P = (int)a.P;
    const bool in = (uint32_t)e < (uint32_t)a.E;
    int lo = in ? a.offsets[e] : 0, hi = in ? a.offsets[e + 1] : 0;
    lo = lo < 0 ? 0 : lo > P ? P : lo;
    hi = hi < lo ? lo : hi > P ? P : hi;
    return Rows{lo, hi};
}
__device__ __forceinline__ Blocks count_blocks(const ExpertArgs& a, int BM) {
    const int lane = threadIdx.x & 63;
    Blocks b;
    b.V = ((int)a.E + 63) / 64;
    b.own = 0;
    for (int v = 0; v < b.V; ++v) {
        const Rows r = rows_of(a, lane * b.V + v);
        b.own += (int)(((uint32_t)(r.hi - r.lo) + BM - 1) / (uint32_t)BM);
    }
    b.sum = wave_scan(b.own);
    b.total = __builtin_amdgcn_readlane(b.sum, 63);
    return b;
}
// Block y < total.  Offsets that no routing writes can make more blocks than an int
// counts: what is then no block of an expert's rows has none.
__device__ __forceinline__ Block find_block(const ExpertArgs& a, const Blocks& b, int BM, int y) {
    const int lane = threadIdx.x & 63;
    const uint64_t here = __ballot(b.sum > y);
    if (here == 0) return Block{0, 0, 0};
    const int l = __builtin_ctzll(here);
    int left = y - __builtin_amdgcn_readlane(b.sum - b.own, l);
    // the experts of lane l, 64 at a time (one where V is 1)
    for (int v0 = 0;; v0 += 64) {
        const int v = v0 + lane;
        Rows r = rows_of(a, v < b.V ? l * b.V + v : (int)a.E);
        const int n = (int)(((uint32_t)(r.hi - r.lo) + BM - 1) / (uint32_t)BM);
        const int sum = wave_scan(n);
        const uint64_t past = __ballot(sum > left);
        if (past) {
            const int w = __builtin_ctzll(past);
            const int lo = __builtin_amdgcn_readlane(r.lo, w), end = __builtin_amdgcn_readlane(r.hi, w);
            const uint32_t from = (uint32_t)(left - __builtin_amdgcn_readlane(sum - n, w)) * (uint32_t)BM;
            if (from >= (uint32_t)(end - lo)) return Block{0, 0, 0};
            const int row = lo + (int)from;
            return Block{l * b.V + v0 + w, row, end - row < BM ? end - row : BM};
        }
        left -= __builtin_amdgcn_readlane(sum, 63);
        if (v0 + 64 >= b.V) return Block{0, 0, 0};
    }
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

// Eight columns of a code word as exact operands, for every z of 0 to 255.  fp16: q -
// z (add: -(1024 + z) and -(64 + z), whole numbers below 2^11).  bf16: (q - z) / 16, two nibbles' signed values by the
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
        if constexpr (ASYM) {
            const _Float16 v = (_Float16)(uint16_t)(zero ? 0u : z);
            add = f16x2{(_Float16)-1024.0f, (_Float16)-64.0f} - f16x2{v, v};
        }
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

constexpr int kGroupRows = 8;  // blocks of rows that pass over all columns together

// The tile of workgroup `id`: workgroups go to the XCDs (each with an L2 of its
// own) in turn, so each XCD takes a contiguous share of the tiles, in the order
// of kGroupRows blocks of rows over all columns.
struct Place {
    Block blk;
    int n_tile;
};
__device__ __forceinline__ Place find_tile(const ExpertArgs& a, int BM, uint32_t tiles_n, uint32_t id) {
    const Blocks b = count_blocks(a, BM);
    const uint32_t total = (uint32_t)b.total * tiles_n;  // below 2^31: the launcher's check
    const uint32_t xcd = id & 7, s = id >> 3, per = total / 8, more = total % 8;
    if (s >= per + (xcd < more ? 1 : 0)) return Place{Block{0, 0, 0}, 0};
    const uint32_t tile = xcd * per + (xcd < more ? xcd : more) + s;
    const uint32_t band = tile / (kGroupRows * tiles_n), in = tile - band * kGroupRows * tiles_n;
    const uint32_t left = (uint32_t)b.total - band * kGroupRows;
    const uint32_t rows = left < kGroupRows ? left : kGroupRows;
    const int n_tile = __builtin_amdgcn_readfirstlane((int)(in / rows));
    const int y = __builtin_amdgcn_readfirstlane((int)(band * kGroupRows + in % rows));
    return Place{find_block(a, b, BM, y), n_tile};
}

// ---------------------------------------------------------------- few rows
//
// BM rows of one expert (4 to 64; a matrix tile has 16 in any case) and 32 weight
// rows a wave.  Such calls are bound by the read of the weights, so what counts is
// bytes in flight and whole cache lines: read straight into matrix operands, 16
// rows x 64 bytes an instruction, a compute unit gets 37 GB/s from its L2, in lines
// of 128 bytes 119 GB/s.  So codes and activations go to LDS by DMA, a step of RB
// code bytes a row (128, or 64 where 16 rows of activations and more need the room:
// more workgroups a compute unit hide more than half lines cost, 52.4 instead of 55.2
// us for 48 tokens of 64 experts in blocks of 16 and 57 instead of 67 in blocks of 32),
// into a ring of two steps (three gain nothing where they halve the workgroups, 52.0
// and 52.2 us, nor for one ternary token, 20.9 and 19.6, where as many fit):
//  - codes: [32 rows a wave][RB / 16 chunks of 16 bytes], chunk c of row r at
//    c ^ (r / 2 % 8), or c ^ (r / 4 % 4) of 64 bytes;
//  - activations: [BM rows][BK columns], chunk c of row r at c ^ (r % 16).
// NW waves share a step's activations; KW groups of waves deal the steps where
// there are too few weight rows to fill the compute units, and their sums meet in
// LDS in the groups' order.
// Lane 16 g + i of a wave takes chunk 4 h + g of weight row i (h = 0, and 1 where
// RB is 128) and the activations of the same columns of row i.  W4A16: that is one
// scale group an h, whose sum starts from zero and is scaled into the result.
// Gated: a wave's first 16 weight rows are the gate's, the others the same rows of
// the up projection.
// Measured: 48 tokens, 6 of 64 experts, 2816 x 2048 W4A16 gated, 52 us, 3.6 TB/s of
// codes and scales, the vector unit (unpacking) 68 % busy; one token, 2 of 8 experts,
// 28672 x 4096 ternary, 19 us, 3.1 TB/s; 666 rows of 16 experts, 4096 x 1408 with
// zero points, 27 us, 283 TFLOP/s.
namespace narrow {

template <int FMT, int BM, int KW, int NW, int RB>
struct Ring {
    static constexpr int kStages = 2;
    static constexpr int kWaves = KW * NW, kThreads = kWaves * kWave;
    static constexpr int kRowBytes = RB;                       // of codes, a row and step
    static constexpr int BK = FMT == 0 ? RB * 4 : RB * 2;      // columns of a step
    static constexpr int kHalves = kRowBytes / 64;
    static constexpr int MT = BM <= 16 ? 1 : BM / 16;             // matrix tiles of activation rows
    static constexpr int kABytes = BM * BK * 2;
    static constexpr int kBBytes = NW * 32 * kRowBytes;
    static constexpr int kStageBytes = kABytes + kBBytes;      // of a group of waves
    static constexpr int kBytes = kStages * KW * kStageBytes;
    static constexpr int AU = kABytes / 1024 >= NW ? kABytes / 1024 / NW : 1;  // 1-KB transfers a wave and step
    static constexpr int BU = kRowBytes / 32;
    // scales and zero points held in LDS, at most
    static constexpr int kScaleBytes = FMT == 0 ? 0 : kBytes + 49152 <= 163840 ? 49152 : 163840 - kBytes;
    static_assert(kBytes <= 163840, "a compute unit has 160 KB");
};

template <class T, int FMT, bool ASYM, bool GATED, int BM, int KW, int NW, int RB>
__global__ __launch_bounds__(KW * NW * kWave) void kernel(ExpertArgs a, int scale_bytes) {
    typedef typename Mfma<T>::vec vec;
    typedef Ring<FMT, BM, KW, NW, RB> G;
    constexpr int BK = G::BK, AU = G::AU, BU = G::BU, kStages = G::kStages, MT = G::MT, kRowBytes = G::kRowBytes;
    constexpr int kChunks = kRowBytes / 16;           // of a row's codes
    constexpr int kCols = GATED ? 16 * NW : 32 * NW;  // output columns of the workgroup
    constexpr int kUnits = FMT == 0 ? 8 : 4;          // 8-column units of a 16-byte chunk of codes
    extern __shared__ uint4 smem_narrow[];
    uint8_t* lds = reinterpret_cast<uint8_t*>(smem_narrow);
    const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem_narrow;
    const int64_t N = a.N, width = GATED ? N / 2 : N;
    const int K = (int)a.K;
    const Place place = find_tile(a, BM, (uint32_t)((width + kCols - 1) / kCols), (uint32_t)a.first + blockIdx.x);
    const Block blk = place.blk;
    if (blk.rows == 0) return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kw = wave / NW, nw = wave % NW;
    const int g = lane >> 4, i16 = lane & 15;
    const int64_t c0 = (int64_t)place.n_tile * kCols;
    const uint32_t rb = FMT == 0 ? K / 4 : K / 2;
    const int GK = K / 128;
    // weight row of row lr of the workgroup's 32 NW; past the end: the last
    auto weight_row = [&](int lr) {
        int64_t c, half = 0;
        if constexpr (GATED) {
            c = c0 + (lr >> 5) * 16 + (lr & 15);
            half = (lr & 16) ? width : 0;
        } else {
            c = c0 + lr;
        }
        return (uint32_t)(half + (c < width ? c : width - 1));
    };
    const uint8_t* w_exp = a.w + (int64_t)blk.expert * N * rb;
    const uint16_t* s_exp = a.scale + (int64_t)blk.expert * N * (FMT == 0 ? 1 : GK);
    const uint8_t* z_exp = ASYM ? a.zeros + (int64_t)blk.expert * N * GK : nullptr;

    // steps of this group of waves; the others of the workgroup go along idle
    const int steps = (K + BK - 1) / BK;
    const int from = steps * kw / KW, mine = steps * (kw + 1) / KW - from;
    const int most = (steps + KW - 1) / KW;
    // DMA sources.  Codes: lane l has chunk (l % 8) ^ (row / 2 % 8) of row 8 u + l / 8 of
    // the wave's 32.  Activations: 16-byte chunks of the group's rows in LDS order.
    // In the last step what lies past the row is its last chunk again.
    // swizzle of a row of codes: as many rows span the banks as 256 bytes hold
    auto code_swizzle = [](int r) { return kChunks == 8 ? (r >> 1) & 7 : (r >> 2) & 3; };
    uint32_t b_row[BU];
    const int b_lane = lane / kChunks;  // row of a transfer
#pragma unroll
    for (int u = 0; u < BU; ++u) b_row[u] = weight_row(32 * nw + 64 / kChunks * u + b_lane) * rb;
    auto issue_codes = [&](int step, uint32_t at) {
#pragma unroll
        for (int u = 0; u < BU; ++u) {
            const uint32_t byte = (uint32_t)kRowBytes * (from + step) + 16u * ((lane % kChunks) ^ code_swizzle(64 / kChunks * u + b_lane));
            dma16s(w_exp, b_row[u] + (byte < rb ? byte : rb - 16), at + G::kABytes + 32u * kRowBytes * nw + 1024u * u);
        }
    };
    constexpr int kRowChunks = BK / 8;
    const uint8_t* a_row[AU];
    uint32_t a_chunk[AU];
    auto issue_rows = [&](int step, uint32_t at) {
#pragma unroll
        for (int u = 0; u < AU; ++u) {
            const uint32_t byte = 2u * BK * (from + step) + a_chunk[u];
            dma16(a_row[u] + (byte < 2u * K ? byte : 2u * K - 16), at + 1024u * ((AU * nw + u) % (G::kABytes / 1024)));
        }
    };
    auto stage_at = [&](int stage) { return lds_base + (uint32_t)((stage * KW + kw) * G::kStageBytes); };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k)
        if (k < mine) issue_codes(k, stage_at(k));
    // the scales of the workgroup's rows, [row][GK] as they lie in memory: 16 rows in
    // a row there are 16 in a row here (rows past the end are not used)
    uint8_t* sc_lds = lds + G::kBytes;
    const bool in_lds = FMT == 1 && scale_bytes > 0;
    if (in_lds) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {  // rows 32 nw + 16 p .. + 15, by the groups of waves in turn
            const uint32_t first = weight_row(32 * nw + 16 * p) * (uint32_t)GK;
            const uint32_t end = (uint32_t)N * GK - first;
            const int to = (32 * nw + 16 * p) * GK;
            for (int e = kw * kWave + lane; e < 16 * GK; e += KW * kWave) {
                const uint32_t i = first + ((uint32_t)e < end ? e : 0);
                reinterpret_cast<uint16_t*>(sc_lds)[to + e] = s_exp[i];
                if constexpr (ASYM) sc_lds[64 * NW * GK + to + e] = z_exp[i];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < AU; ++u) {
        const int at = ((AU * nw + u) % (G::kABytes / 1024)) * 64 + lane;  // chunk's place
        const int r = at / kRowChunks;
        a_row[u] = reinterpret_cast<const uint8_t*>(a.A + source_row(a, blk.row + (r < blk.rows ? r : 0)) * K);
        a_chunk[u] = 16u * ((at % kRowChunks) ^ (r & 15));
    }
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k)
        if (k < mine) issue_rows(k, stage_at(k));

    f32x4 acc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int a_frag = (i16 % BM) * (BK * 2), a_swz = i16 % BM;
    const int b_frag = G::kABytes + (32 * nw + i16) * kRowBytes, b_swz = code_swizzle(i16);
    const uint32_t magic_v = vgpr_const<kMagic2>();
    const uint32_t mask_v = sgpr_const<0x00F0000Fu>();
    const NatConsts nat = nat_consts();
    uint32_t sr[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) sr[j] = weight_row(32 * nw + 16 * j + i16);
    // Half h of step k.  PART: a ternary row ends in it; the lanes past its end take
    // weights and activations of 0.
    auto contract = [&](auto part, const uint8_t* sbase, int k, int h) {
        constexpr bool PART = decltype(part)::value;
        const bool past = PART && BK * (from + k) + 16 * kUnits * 2 * h + 64 * g >= K;
        uint4 q[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            q[j] = *reinterpret_cast<const uint4*>(sbase + b_frag + 16 * kRowBytes * j + 16 * ((4 * h + g) ^ b_swz));
            if (past) q[j] = make_uint4(0x55555555u, 0x55555555u, 0x55555555u, 0x55555555u);
        }
        f32x4 sum[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 2; ++j) sum[m][j] = FMT == 1 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[m][j];
        float s[2];
        W4Unpack<T, ASYM> un[2];
        if constexpr (FMT == 1) {
            const int group = G::kHalves * (from + k) + h;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = (32 * nw + 16 * j + i16) * GK + group;
                s[j] = f16_bits_to_f32(in_lds ? reinterpret_cast<const uint16_t*>(sc_lds)[at] : s_exp[(int64_t)sr[j] * GK + group]) *
                       W4Unpack<T, ASYM>::kUnit;
                if constexpr (ASYM) un[j].set(in_lds ? sc_lds[64 * NW * GK + at] : z_exp[(int64_t)sr[j] * GK + group], false);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int chunk = 4 * kUnits * h + kUnits * g + u;
            vec av[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint4 v = *reinterpret_cast<const uint4*>(sbase + a_frag + 16 * m * (BK * 2) + 16 * (chunk ^ a_swz));
                if (past) v = make_uint4(0, 0, 0, 0);
                av[m] = __builtin_bit_cast(vec, v);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint4 b;
                if constexpr (FMT == 0) {
                    const uint32_t x = dword_of(q[j], u / 2);
                    b = u % 2 ? nat_quad<1>(x, magic_v, nat) : nat_quad<0>(x, magic_v, nat);
                } else {
                    b = un[j].quad(dword_of(q[j], u), mask_v, magic_v);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) sum[m][j] = Mfma<T>::mma(av[m], __builtin_bit_cast(vec, b), sum[m][j]);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if constexpr (FMT == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][j][i] = fmaf(s[j], sum[m][j][i], acc[m][j][i]);
                } else {
                    acc[m][j] = sum[m][j];
                }
            }
    };
    auto half = [&](const uint8_t* sbase, int k, int h) {
        if (FMT == 0 && BK * (from + k) + 256 * (h + 1) > K) contract(std::true_type{}, sbase, k, h);
        else contract(std::false_type{}, sbase, k, h);
    };
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    stage_barrier();
    int stage = 0;
    for (int k = 0; k < most; ++k) {
        const bool more = k + kStages - 1 < mine;
        if (more) {
            const int next = stage == 0 ? kStages - 1 : stage - 1;
            issue_codes(k + kStages - 1, stage_at(next));
            issue_rows(k + kStages - 1, stage_at(next));
        }
        if (k < mine) {
            const uint8_t* sbase = lds + (stage * KW + kw) * G::kStageBytes;
            half(sbase, k, 0);
            if (G::kHalves == 2 && BK * (from + k) + BK / 2 < K) half(sbase, k, 1);
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
        // the next step has landed; of the later ones only the last may be on its way
        if (more) asm volatile("s_waitcnt vmcnt(%0)" :: "n"((kStages - 2) * (AU + BU)) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        stage_barrier();
    }

    if constexpr (KW > 1) {  // the groups' sums, in their order
        constexpr int kTiles = NW * MT * 2;
        f32x4* red = reinterpret_cast<f32x4*>(lds) + nw * (MT * 2 * kWave) + lane;  // [KW - 1][NW][MT][2][64]: the ring is idle
        static_assert((KW - 1) * kTiles * 1024 <= G::kBytes, "the sums take the ring's place");
        if (kw > 0) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 2; ++j) red[((kw - 1) * kTiles + 2 * m + j) * kWave] = acc[m][j];
        }
        __syncthreads();
        if (kw > 0) return;
#pragma unroll
        for (int z = 0; z < KW - 1; ++z)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[m][j] += red[(z * kTiles + 2 * m + j) * kWave];
    }
    // lane 16 g + i: rows 4 g .. 4 g + 3, weight row i of each block
    const int64_t bias_row = (int64_t)blk.expert * N;
    float sc[2], bi[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        sc[j] = FMT == 0 ? f16_bits_to_f32(s_exp[sr[j]]) * Mfma<T>::kUnit : 1.0f;
        bi[j] = a.bias ? T::to_f32(a.bias[bias_row + sr[j]]) : 0.0f;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 16 * m + 4 * g + i;
            if (row >= blk.rows || row >= BM) continue;
            uint16_t* dst = a.C + (blk.row + row) * width;
            if constexpr (GATED) {
                const int64_t c = c0 + 16 * nw + i16;
                if (c < width)
                    dst[c] = round_one<T>(gate(fmaf(acc[m][0][i], sc[0], bi[0]), fmaf(acc[m][1][i], sc[1], bi[1])));
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t c = c0 + 32 * nw + 16 * j + i16;
                    if (c < width) dst[c] = round_one<T>(fmaf(acc[m][j][i], sc[j], bi[j]));
                }
            }
        }
}

}  // namespace narrow

// ---------------------------------------------------------------- many rows
//
// 128 rows of one expert and 256 weight rows a workgroup, four waves of 128 x 64.
// Activations and codes come by DMA (no registers) into a ring of three stages of
// 64 columns, two or three ahead of the matrix cores: 128 rows x 128 bytes, 16-byte chunks
// XOR-swizzled (chunk c of row r at c ^ (r / 2 % 8): two rows span the banks, so 16
// rows' reads of a chunk meet 16 different places), and 256 weight rows x 16 or 32
// bytes.  Codes are unpacked in registers in the natural order of their columns.
// Two workgroups share a compute unit, so one's barriers lie under the other's
// products.  Measured: 8192 rows of 8 experts, 28672 x 4096 W4A16 gated, 1.84 to 1.97
// ms, 980 to 1040 TFLOP/s, the matrix cores 53 % and the vector unit 65 % of the cycles
// busy (2.9 vector instructions a product); 4094 rows of 8, 4096 x 14336 ternary,
// 450 us, 1070 TFLOP/s, the matrix cores 77 %.
//
// W4A16: the accumulators hold the sum in units of the current group's scale, so
// entering a group multiplies them by the ratio of the last scale to its own, and
// the operands stay the exact q - z.  (Scaling every group's sum into a second set
// of accumulators costs as many instructions and twice the registers, which
// halves the tile.)  A group whose scale is 0 keeps the last unit, and its code
// words are replaced by those of zero weights.
namespace tile {

constexpr int BM = 128, BN = 256, BK = 64, WN = 64, TN = 4;
constexpr int kWaves = 4, kThreads = kWaves * kWave;
constexpr int kStages = 3;
constexpr int kEpiLd = WN + 8;  // halves of a row staged for its store

template <int FMT>
struct Ring {
    static constexpr int kABytes = BM * BK * 2;
    static constexpr int kBBytes = BN * BK / (FMT == 0 ? 4 : 2);
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kBytes = kStages * kStageBytes;
    static constexpr int kScaleBytes = FMT == 0 ? 0 : 512 * kWaves * 3;  // eight groups of the tile's rows
    static constexpr int AU = BM / 32, BU = kBBytes / 4096;  // 1-KB transfers a wave and stage
    static_assert(kWaves * 32 * kEpiLd * 2 <= kBytes, "epilogue staging must fit in the ring");
};

template <class T, int FMT, bool ASYM, bool GATED>
__global__ __launch_bounds__(kThreads, 2) void kernel(ExpertArgs a) {
    typedef typename Mfma<T>::vec vec;
    typedef Ring<FMT> G;
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
        a_src[u] = reinterpret_cast<const uint8_t*>(a.A + row * K) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
    }
    uint32_t b_src[BU];  // from the expert's weights: below 2^31 bytes
#pragma unroll
    for (int u = 0; u < BU; ++u) {
        if constexpr (FMT == 0) b_src[u] = weight_row(64 * wave + lane) * (uint32_t)rb;
        else b_src[u] = weight_row(32 * (2 * wave + u) + (lane >> 1)) * (uint32_t)rb + 16 * (lane & 1);
    }
    // The sources run on from stage to stage and stay at the last K-step, so that the
    // counts of transfers in flight stay exact; what is issued past the end goes
    // where nobody reads any more.
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

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int a_frag = i16 * (BK * 2);
    const int swz = i16 >> 1;
    const int b_frag = G::kABytes + (wave * WN + i16) * (FMT == 0 ? 16 : 32) + (FMT == 0 ? 4 : 8) * g;
    const uint32_t magic_v = vgpr_const<kMagic2>();
    const uint32_t mask_v = sgpr_const<0x00F0000Fu>();
    const NatConsts nat = nat_consts();
    W4Unpack<T, ASYM> un[TN];
    float unit[TN];  // scale that the accumulators are in units of
    // The wave's 64 rows of scales (and zero points), eight groups at a time, in an
    // LDS area of its own, [8][64]: a lane reads one row's eight at once, so that a
    // line is touched once in sixteen K-steps, and only then waits for memory.
    uint16_t* sc_lds = reinterpret_cast<uint16_t*>(lds + G::kBytes) + 512 * wave;
    uint8_t* zp_lds = lds + G::kBytes + 1024 * kWaves + 512 * wave;
    const uint32_t s_row = weight_row(wave * WN + lane) * (uint32_t)GK;
    auto load_scales = [&](int first) {  // groups first .. first + 7, or the last eight
        const int from = GK < 8 ? 0 : first < (int)GK - 8 ? first : (int)GK - 8;
        uint16_t v[8];
        uint8_t z[8];
        if (GK >= 8) {
            __builtin_memcpy(v, s_exp + from + s_row, 16);
            if constexpr (ASYM) __builtin_memcpy(z, z_exp + from + s_row, 8);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = e < (int)GK ? e : 0;
                v[e] = s_exp[s_row + at];
                if constexpr (ASYM) z[e] = z_exp[s_row + at];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sc_lds[64 * e + lane] = v[e];
            if constexpr (ASYM) zp_lds[64 * e + lane] = z[e];
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's own area: no barrier
        return from;
    };

    // the unpacking constants of the next group, and what takes the sums to its unit
    float ratio[TN];
    int held = 0;  // first group in LDS
    auto enter_group = [&](int group) {
        if ((group & 7) == 0) held = load_scales(group);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int at = 64 * (group - held) + 16 * j + i16;
            const float s = f16_bits_to_f32(sc_lds[at]);
            const bool zero = s == 0.0f;
            un[j].set(ASYM ? zp_lds[at] : 8u, zero);
            float r = __builtin_amdgcn_rcpf(s);
            r = unit[j] * fmaf(fmaf(-s, r, 1.0f), r, r);  // a Newton step: within an ulp
            ratio[j] = zero ? 1.0f : r;
            if (!zero) unit[j] = s;
        }
    };
    uint2 x[TN];      // code words of a K-step: .x its first half (ternary: both)
    uint32_t y[TN];   // of the second half, while x takes the next K-step's
    auto read_codes = [&](const uint8_t* stage) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            if constexpr (FMT == 0) x[j].x = *reinterpret_cast<const uint32_t*>(stage + b_frag + 16 * 16 * j);
            else x[j] = *reinterpret_cast<const uint2*>(stage + b_frag + 16 * 32 * j);
        }
    };
    auto unpack = [&](int half, int j) {
        uint4 b;
        if constexpr (FMT == 0) b = half ? nat_quad<1>(y[j], magic_v, nat) : nat_quad<0>(x[j].x, magic_v, nat);
        else b = un[j].quad(half ? y[j] : x[j].x, mask_v, magic_v);
        return __builtin_bit_cast(vec, b);
    };
    // Half a K-step: 16 weight rows at a time against all activation rows, while the
    // next 16 are unpacked (a product leaves the vector unit three issue slots).  The
    // activations' registers take the next half's as they become free.
    vec af[TM], bf;
    auto read_rows = [&](const uint8_t* stage, int half, int i) {
        af[i] = __builtin_bit_cast(vec, *reinterpret_cast<const uint4*>(stage + a_frag + 16 * ((2 * g + half) ^ swz) + i * 16 * (BK * 2)));
    };
    auto products = [&](auto rescale, int half, const uint8_t* next) {
        constexpr bool kRescale = decltype(rescale)::value;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                if constexpr (kRescale) acc[i][j] *= ratio[j];
                acc[i][j] = Mfma<T>::mma(af[i], bf, acc[i][j]);
                if (j == TN - 1) read_rows(next, half ^ 1, i);
            }
            if (j + 1 < TN) bf = unpack(half, j + 1);
            else if (half == 0) bf = unpack(1, 0);
            if constexpr (FMT == 0) {  // two vector instructions beside each product
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x002, 16 / TM, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    if (j == TN - 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    issue();
    issue();
    issue();
    if constexpr (FMT == 1) {
#pragma unroll
        for (int j = 0; j < TN; ++j) unit[j] = 1.0f;
        enter_group(0);
    }
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(2 * (AU + BU)) : "memory");
    stage_barrier();
    const uint8_t* at = lds;                       // this K-step's stage
    const uint8_t* const last_stage = lds + (kStages - 1) * G::kStageBytes;
    auto second_half = [&]() {
#pragma unroll
        for (int j = 0; j < TN; ++j) y[j] = FMT == 0 ? x[j].x : x[j].y;
    };
    read_codes(at);
#pragma unroll
    for (int i = 0; i < TM; ++i) read_rows(at, 0, i);
    second_half();
    bf = unpack(0, 0);
    constexpr int kSteps = FMT == 1 ? 2 : 1;  // of a scale group
    for (int kt = 0; kt < nk; kt += kSteps) {
#pragma unroll
        for (int h = 0; h < kSteps; ++h) {
            if (FMT == 1 && h == 0) products(std::true_type{}, 0, at);
            else products(std::false_type{}, 0, at);
            // The next stage has landed, for every wave, and everything of this one is
            // in registers: its place takes the third stage from here.
            asm volatile("s_waitcnt vmcnt(%0)" :: "n"(AU + BU) : "memory");
            stage_barrier();
            issue();
            at = at == last_stage ? lds : at + G::kStageBytes;
            read_codes(at);
            products(std::false_type{}, 1, at);
            if (FMT == 1 && h == 1 && kt / 2 + 1 < (int)GK) enter_group(kt / 2 + 1);
            second_half();
            bf = unpack(0, 0);
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
        if constexpr (FMT == 0) sc[j] = f16_bits_to_f32(s_exp[weight_row(wave * WN + 16 * j + i16)]) * Mfma<T>::kUnit;
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

template <class T, int FMT, bool ASYM, bool GATED, int BM, int KW, int NW, int RB>
hipError_t launch_narrow(const ExpertArgs& args, hipStream_t s) {
    typedef narrow::Ring<FMT, BM, KW, NW, RB> G;
    static DeviceFlags lds_limit_set;
    hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&narrow::kernel<T, FMT, ASYM, GATED, BM, KW, NW, RB>),
                                   G::kBytes + G::kScaleBytes, lds_limit_set);
    if (e != hipSuccess) return e;
    const int64_t width = GATED ? args.N / 2 : args.N, cols = (GATED ? 16 : 32) * NW;
    const int64_t groups = ((width + cols - 1) / cols * most_blocks(args.P, args.E, BM) + 7) / 8 * 8;
    if (groups >= (int64_t)1 << 31) return hipErrorInvalidValue;
    const int64_t scales = FMT == 0 ? 0 : 32 * NW * (args.K / 128) * (ASYM ? 3 : 2);
    const int scale_bytes = scales <= G::kScaleBytes ? (int)scales : 0;
    ExpertArgs a = args;
    constexpr int64_t kMost = kMaxGroups / 8 * 8;
    for (a.first = 0; a.first < groups; a.first += kMost) {
        const int64_t n = groups - a.first < kMost ? groups - a.first : kMost;
        narrow::kernel<T, FMT, ASYM, GATED, BM, KW, NW, RB><<<(unsigned)n, G::kThreads, G::kBytes + scale_bytes, s>>>(a, scale_bytes);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T, int FMT, bool ASYM, bool GATED>
hipError_t launch_tile(const ExpertArgs& args, hipStream_t s) {
    typedef tile::Ring<FMT> G;
    static DeviceFlags lds_limit_set;
    hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(&tile::kernel<T, FMT, ASYM, GATED>), G::kBytes + G::kScaleBytes, lds_limit_set);
    if (e != hipSuccess) return e;
    const int64_t width = GATED ? args.N / 2 : args.N, cols = GATED ? tile::BN / 2 : tile::BN;
    const int64_t groups = ((width + cols - 1) / cols * most_blocks(args.P, args.E, tile::BM) + 7) / 8 * 8;
    if (groups >= (int64_t)1 << 31) return hipErrorInvalidValue;  // an output of more than 2^44 values
    ExpertArgs a = args;
    constexpr int64_t kMost = kMaxGroups / 8 * 8;
    for (a.first = 0; a.first < groups; a.first += kMost) {
        const int64_t n = groups - a.first < kMost ? groups - a.first : kMost;
        tile::kernel<T, FMT, ASYM, GATED><<<(unsigned)n, tile::kThreads, G::kBytes + G::kScaleBytes, s>>>(a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

// The workgroups a call can be cut into: rows of activations, weight rows, parts
// the columns are dealt to, bytes of a weight row's codes in a step; and the time
// of a step in us, of a workgroup with a compute unit to itself and for each
// workgroup where several share one (ternary, W4A16, W4A16 with zero points).
struct Cut {
    int rows, weights, parts, bytes;
    float alone[3], shared[3];
};

constexpr Cut kCuts[] = {
    {4, 128, 1, 128, {1.08f, 0.0f, 0.0f}, {0.79f, 0.0f, 0.0f}},  // ternary alone: W4A16 is faster by the next in any case
    {4, 64, 2, 128, {1.18f, 1.06f, 1.35f}, {0.69f, 0.68f, 0.68f}},
    {4, 32, 8, 64, {1.10f, 1.03f, 1.23f}, {0.76f, 0.61f, 0.67f}},
    {16, 128, 1, 64, {0.74f, 0.64f, 1.00f}, {0.48f, 0.39f, 0.41f}},
    {16, 64, 2, 64, {0.81f, 0.67f, 1.02f}, {0.51f, 0.38f, 0.42f}},
    {16, 32, 4, 64, {0.94f, 0.81f, 0.90f}, {0.69f, 0.46f, 0.50f}},
    {32, 128, 1, 64, {0.96f, 0.70f, 1.05f}, {0.66f, 0.48f, 0.59f}},
    {64, 128, 1, 64, {1.35f, 0.93f, 1.28f}, {1.10f, 0.76f, 0.96f}},
    {tile::BM, tile::BN, 1, 0, {0.71f, 1.02f, 1.11f}, {0.85f, 1.13f, 1.09f}},
};
static_assert(sizeof(kCuts) / sizeof(kCuts[0]) == TQ_MOE_CUTS, "tq.h names the number");

// The cut of the shortest estimated time: few rows waste the rows of a large
// block, few blocks leave compute units idle, and a long row takes one workgroup
// many steps.  kCuts was fitted to every cut's time for 253 calls (1 to 4096
// tokens, 1 to 120 experts, 512 to 14336 columns): the one taken here is 3 %
// slower than the best of the nine in the mean and 38 % at worst (80 other calls: 3 %
// and 35 %); by rows an expert alone it is 28 % and fivefold.
int choose_cut(int fmt, bool zeros, int64_t P, int64_t E, int64_t N, int64_t K) {
    const int kind = fmt == 0 ? 0 : zeros ? 2 : 1;
    const int64_t used = P < E ? P : E;
    const int first = fmt == 0 ? 0 : 1;
    int best = first;
    double best_time = 0;
    for (int i = first; i < TQ_MOE_CUTS; ++i) {
        const Cut& c = kCuts[i];
        const bool tiled = c.rows == tile::BM;
        const int64_t bk = tiled ? tile::BK : c.bytes * (fmt == 0 ? 4 : 2);
        const int64_t steps = ((K + bk - 1) / bk + c.parts - 1) / c.parts;
        // an expert's last block is half full; experts of fewer rows than that have one
        const double full = (double)P / (double)(used * c.rows) + 0.5;
        const double share = (full > 1.0 ? full : 1.0) * (double)(used * ((N + c.weights - 1) / c.weights)) / compute_units();
        const double step = share * c.shared[kind] > c.alone[kind] ? share * c.shared[kind] : c.alone[kind];
        // steps' worth of filling the ring and of the results, and the start
        const double time = (double)(steps + (tiled ? 6 : 2)) * step + (tiled ? 5.5 : 2.5);
        if (i == first || time < best_time) {
            best = i;
            best_time = time;
        }
    }
    return best;
}

template <class T, int FMT, bool ASYM, bool GATED, int CUT>
hipError_t launch_cut(const ExpertArgs& a, hipStream_t s) {
    constexpr Cut c = kCuts[CUT];
    return launch_narrow<T, FMT, ASYM, GATED, c.rows, c.parts, c.weights / 32, c.bytes>(a, s);
}

template <class T, int FMT, bool ASYM, bool GATED>
hipError_t launch_rows(const ExpertArgs& a, hipStream_t s) {
    const int cut = choose_cut(a.fmt, a.zeros != nullptr, a.P, a.E, a.N, a.K);
    if constexpr (FMT == 0) {
        if (cut == 0) return launch_cut<T, FMT, ASYM, GATED, 0>(a, s);
    }
    switch (cut) {
        case 1: return launch_cut<T, FMT, ASYM, GATED, 1>(a, s);
        case 2: return launch_cut<T, FMT, ASYM, GATED, 2>(a, s);
        case 3: return launch_cut<T, FMT, ASYM, GATED, 3>(a, s);
        case 4: return launch_cut<T, FMT, ASYM, GATED, 4>(a, s);
        case 5: return launch_cut<T, FMT, ASYM, GATED, 5>(a, s);
        case 6: return launch_cut<T, FMT, ASYM, GATED, 6>(a, s);
        case 7: return launch_cut<T, FMT, ASYM, GATED, 7>(a, s);
        default: return launch_tile<T, FMT, ASYM, GATED>(a, s);
    }
}

template <class T>
hipError_t launch_type(const ExpertArgs& a, hipStream_t s) {
    if (a.fmt == 0) return a.gated ? launch_rows<T, 0, false, true>(a, s) : launch_rows<T, 0, false, false>(a, s);
    if (a.zeros) return a.gated ? launch_rows<T, 1, true, true>(a, s) : launch_rows<T, 1, true, false>(a, s);
    return a.gated ? launch_rows<T, 1, false, true>(a, s) : launch_rows<T, 1, false, false>(a, s);
}

}  // namespace

int select_cut(int fmt, bool zeros, int64_t P, int64_t E, int64_t N, int64_t K) { return choose_cut(fmt, zeros, P, E, N, K); }

hipError_t launch_experts(const ExpertArgs& a, hipStream_t s) {
    return a.bf16 ? launch_type<BF16>(a, s) : launch_type<F16>(a, s);
}

}  // namespace tq
