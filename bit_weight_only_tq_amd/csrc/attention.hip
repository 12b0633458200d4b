// Attention of each request's new tokens over the pages of its cache.
//
// For query row i (position p) and key j of its request, with the scores
// t_ij = scale log2(e) q_i . k_j of the visible keys (j <= p; with a window
// w: p - j < w or j < sinks),
//   out_i = sum_j 2^(t_ij - m_i) v_j / l_i,   l_i = sum_j 2^(t_ij - m_i),
//   lse_i = ln 2 (m_i + log2 l_i),
// in one pass over the keys with a running maximum m_i.  Maxima, sums and
// outputs are held in fp32; the weights 2^(t - m) are rounded to the cache's
// type (the matrix cores' operand), as the output is.
//
// The query heads that share a KV head are rows of one matrix: row r of a
// request and KV head is token r / G, head r % G of the group of G.

#include <math.h>

#include "tq_device.h"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr float kLn2 = 0.69314718055994531f;

// Element types: the matrix products, the rounding of two weights to a
// dword, and the exponent step that carries a non-finite value's magnitude
// into bit 15.
struct AttnF16 {
    static __device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack2(float x, float y) {
        return __builtin_bit_cast(uint32_t, f16x2{(_Float16)x, (_Float16)y});
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w).x; }
    static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w).y; }
    static constexpr uint32_t kExpStep = 0x04000400u;
};
struct AttnBF16 {
    static __device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack2(float x, float y) {
        return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x, (__bf16)y});
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
    static constexpr uint32_t kExpStep = 0x00800080u;
};

template <class E>
__device__ __forceinline__ uint32_t nonfinite(uint32_t w) {
    return ((w & 0x7FFF7FFFu) + E::kExpStep) & 0x80008000u;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

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

// The key blocks (32 keys, aligned) a run of positions p0 .. p1 can see:
// `head` blocks of sinks from key 0, then [main0, main1).
struct Blocks {
    int head, main0, count;
    __device__ __forceinline__ int at(int i) const { return i < head ? i : main0 + (i - head); }
};
__device__ __forceinline__ Blocks blocks_of(const AttnArgs& a, const Request& r, int p0, int p1) {
    Blocks k;
    const int end = min(p1, r.keys - 1) + 1;  // first key nobody sees
    const int main1 = end > 0 ? (int)(((uint32_t)end + 31u) >> 5) : 0;
    int lo = 0;
    if (a.window > 0) lo = max(p0 - a.window + 1, 0);
    k.main0 = min(lo >> 5, main1);
    k.head = min((int)(((uint32_t)a.sinks + 31u) >> 5), k.main0);
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
// different key blocks (R = 1), or different rows of the same keys (R = 2, 4
// for requests with more rows), and the key axis is cut into `a.splits`
// workgroups; the last one to finish joins the partial results in order.
constexpr int kRowsThreads = 256;
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

template <class E, int D>
__global__ __launch_bounds__(kRowsThreads) void rows_kernel(AttnArgs a) {
    constexpr int ST = D / 32, DV = D / 16, VD = DV / 2;
    constexpr int LD = D + 4;  // LDS row stride (floats): rows of a quad of lanes fall into different banks
    __shared__ float lds_o[4 * 16 * LD];
    __shared__ float lds_ml[4 * 16 * 2];
    __shared__ float row_m[64], row_l[64];
    __shared__ uint32_t word;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, c = lane & 15;
    // workgroup -> KV head (fastest), split, row group, request
    int64_t id = blockIdx.x;
    const int h = (int)(id % a.Hkv);
    id /= a.Hkv;
    const int split = (int)(id % a.splits);
    id /= a.splits;
    const int rg = (int)(id % a.row_groups);
    const int b = (int)(id / a.row_groups);
    const Request rq = request_of(a, b);
    const int R = a.R, G = a.G;
    const int64_t rows_all = (int64_t)min(rq.n, a.max_q) * G;
    const int64_t row0 = (int64_t)rg * 16 * R;
    if (row0 >= rows_all) return;
    const int rows = (int)(rows_all - row0 < 16 * R ? rows_all - row0 : 16 * R);  // of this workgroup
    // the keys any of its rows sees, cut into splits
    const Blocks bl = blocks_of(a, rq, rq.first + (int)(row0 / G), rq.first + (int)((row0 + rows - 1) / G));
    int per = a.split_blocks;
    if ((int64_t)per * a.splits < bl.count) per = (bl.count + a.splits - 1) / a.splits;
    const int nsplit = bl.count > per ? (bl.count + per - 1) / per : 1;
    if (split >= nsplit) return;

    const int tile = wave % R, ks = wave / R, KS = 4 / R;
    const int64_t my_row = row0 + tile * 16 + c;
    const bool row_ok = my_row < rows_all;
    const int my_tok = (int)((row_ok ? my_row : row0) / G);
    const int my_head = h * G + (int)((row_ok ? my_row : row0) - (int64_t)my_tok * G);
    const int my_pos = row_ok ? rq.first + my_tok : INT32_MIN;
    // positions of the tile's first and last row
    const int64_t last_row = row0 + tile * 16 + 15 < rows_all ? row0 + tile * 16 + 15 : rows_all - 1;
    const int tile_p0 = rq.first + (int)((row0 + tile * 16) / G);
    const int tile_p1 = rq.first + (int)(last_row / G);
    const bool tile_ok = tile * 16 < rows;

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

    const int i0 = split * per, i1 = min(bl.count, i0 + per);
    const int32_t* trow = a.table + (int64_t)b * a.table_stride;
    const int last_key = rq.keys - 1;
    const int kperm = 8 * (c >> 2) + (c & 3);  // key of tile t's row c: kperm + 4 t
    if (tile_ok) {
        for (int i = i0 + ks; i < i1; i += KS) {
            const int key0 = bl.at(i) * kBlockKeys;
            if (key0 > tile_p1) continue;
            // pages: this lane's K rows lie in one page, its V rows in one page
            const int kk = min(key0 + 8 * (c >> 2), last_key), kv = min(key0 + 8 * g, last_key);
            const int idk = trow[kk >> a.shift], idv = trow[kv >> a.shift];
            const bool okk = (uint32_t)idk < (uint32_t)a.pages, okv = (uint32_t)idv < (uint32_t)a.pages;
            const int page_mask = (1 << a.shift) - 1;
            const uint16_t* kbase = a.k + (int64_t)(okk ? idk : 0) * a.page_stride + ((int64_t)h << a.shift) * D + 8 * g;
            const uint16_t* vbase = a.v + (int64_t)(okv ? idv : 0) * a.page_stride + ((int64_t)h << a.shift) * D + DV * c;
            uint4 kf[2][ST];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint16_t* p = kbase + (int64_t)((key0 + kperm + 4 * t) & page_mask) * D;
#pragma unroll
                for (int s = 0; s < ST; ++s) kf[t][s] = *reinterpret_cast<const uint4*>(p + 32 * s);
            }
            VRow<VD> vr[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) vr[e] = load_vrow<VD>(vbase + (int64_t)((key0 + 8 * g + e) & page_mask) * D);

            float t8[8];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f32x4 s4 = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < ST; ++s) s4 = E::mfma16(kf[t][s], qf[s], s4);
#pragma unroll
                for (int r = 0; r < 4; ++r) t8[4 * t + r] = s4[r] * a.scale_log2;
            }
            // blocks that every row of the tile sees whole need no mask
            bool whole = key0 + kBlockKeys - 1 <= min(tile_p0, last_key);
            if (a.window > 0) whole = whole && (tile_p1 - key0 < a.window || key0 + kBlockKeys <= a.sinks);
            const bool masked = !whole || __any(!okv);
            bool poisoned = false;
            if (masked) {
                uint32_t bad = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = key0 + 8 * g + e;
                    const bool there = okv && j <= last_key;
                    if (!there || !sees(a, my_pos, j)) t8[e] = -INFINITY;
                    // a key that no row of the tile sees may hold anything
                    const bool hidden = !there || j > tile_p1 ||
                                        (a.window > 0 && tile_p0 - j >= a.window && j >= a.sinks);
#pragma unroll
                    for (int w = 0; w < VD; ++w) {
                        if (hidden) vr[e].w[w] = 0;
                        bad |= nonfinite<E>(vr[e].w[w]);
                    }
                }
                poisoned = __any(bad != 0);
            }
            // running maximum, shared by the four lanes of a row; raised only
            // when a score passes it by more than 2^8, so that most blocks
            // rescale nothing (weights up to 256 fit both 16-bit types)
            float mx = t8[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) mx = fmaxf(mx, t8[e]);
            if (__any(mx > m + 8.f)) {
                mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
                mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
                const float mn = fmaxf(m, mx);
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
                    const int pid = __shfl(okv ? idv : -1, src, 64);
                    for (int e = 0; e < 8; ++e) {
                        const int j = key0 + 8 * gg + e;
                        float p = 0.f;
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const float px = (x & 1) ? E::hi(pw[x / 2]) : E::lo(pw[x / 2]);
                            const float got = __shfl(px, src + c, 64);
                            if (x == e) p = got;
                        }
                        if (pid < 0 || j > last_key || !sees(a, my_pos, j)) continue;
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
        }
        l += __shfl_xor(l, 16, 64);
        l += __shfl_xor(l, 32, 64);
    }

    // join the waves of each tile
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
    const int64_t wg_tile = ((int64_t)b * a.row_groups + rg) * a.Hkv + h;
    float* slab = a.partials + (wg_tile * a.splits + split) * a.slab;  // [rows][2], then [rows][D]
    constexpr int EPT = 4;                                             // values a thread joins at a time
    for (int u = tid; u < rows * (D / EPT); u += kRowsThreads) {
        const int row = u / (D / EPT), d = (u - row * (D / EPT)) * EPT;
        const int tl = row >> 4, rr = row & 15;
        float M = -INFINITY, L = 0.f;
        for (int w = 0; w < KS; ++w) M = fmaxf(M, lds_ml[((w * R + tl) * 16 + rr) * 2]);
        const float ms = M == -INFINITY ? 0.f : M;
        float acc[EPT] = {0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < KS; ++w) {
            const int base = (w * R + tl) * 16 + rr;
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
            for (int e = 0; e < EPT; ++e) store_partial(slab + 2 * rows + row * D + d + e, acc[e]);
            if (d == 0) {
                store_partial(slab + 2 * row, M);
                store_partial(slab + 2 * row + 1, L);
            }
        } else {
            const int64_t r = row0 + row;
            const int tok = (int)(r / G);
            const int64_t at = (int64_t)(rq.t0 + tok) * a.Hq + h * G + (int)(r - (int64_t)tok * G);
            const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : NAN);
            *reinterpret_cast<uint2*>(a.out + at * D + d) =
                make_uint2(E::pack2(acc[0] * inv, acc[1] * inv), E::pack2(acc[2] * inv, acc[3] * inv));
            if (d == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : kLn2 * (M + log2f(L));
        }
    }
    if (!parts) return;
    if (!split_last_arrival(a.flags, (uint32_t)wg_tile, nsplit, &word)) return;

    // join the splits, in split order
    const float* slabs = a.partials + wg_tile * a.splits * a.slab;
    float* wgt = lds_o;  // [row][nsplit] weights of the splits; splits * rows <= 4096
    for (int row = wave; row < rows; row += 4) {
        float M = -INFINITY;
        for (int s = lane; s < nsplit; s += 64)
            M = fmaxf(M, __hip_atomic_load(slabs + s * a.slab + 2 * row, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
#pragma unroll
        for (int x = 32; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor(M, x, 64));
        const float ms = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        for (int s = lane; s < nsplit; s += 64) {
            const float ps = __hip_atomic_load(slabs + s * a.slab + 2 * row, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const float pl = __hip_atomic_load(slabs + s * a.slab + 2 * row + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
    for (int u = tid; u < rows * (D / 2); u += kRowsThreads) {
        const int row = u / (D / 2), d = (u - row * (D / 2)) * 2;
        float x0 = 0.f, x1 = 0.f;
        const float* base = slabs + 2 * rows + row * D + d;
        constexpr int RS = 8;  // splits in flight
        for (int s0 = 0; s0 < nsplit; s0 += RS) {
            uint64_t v[RS];
#pragma unroll
            for (int s = 0; s < RS; ++s)
                v[s] = __hip_atomic_load(reinterpret_cast<const uint64_t*>(base + (int64_t)min(s0 + s, nsplit - 1) * a.slab),
                                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int s = 0; s < RS; ++s)
                if (s0 + s < nsplit) {
                    const float f = wgt[row * nsplit + s0 + s];
                    x0 += f * __uint_as_float((uint32_t)v[s]);
                    x1 += f * __uint_as_float((uint32_t)(v[s] >> 32));
                }
        }
        const float L = row_l[row];
        const int64_t r = row0 + row;
        const int tok = (int)(r / G);
        const int64_t at = (int64_t)(rq.t0 + tok) * a.Hq + h * G + (int)(r - (int64_t)tok * G);
        const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : NAN);
        *reinterpret_cast<uint32_t*>(a.out + at * D + d) = E::pack2(x0 * inv, x1 * inv);
        if (d == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : kLn2 * (row_m[row] + log2f(L));
    }
}

}  // namespace

// Schedule of a call.  Row tiles a workgroup holds: as many as the largest
// request needs, up to 4 (its waves then share the keys).  The key axis is
// split until the grid has about 8 workgroups a compute unit (lengths are
// ragged, and short splits even them out), but no split is shorter than
// 8 blocks: below that its partial results cost more than its keys.
AttnPlan attn_plan(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q, int64_t max_kv, int64_t window,
                   int64_t sinks, int compute_units) {
    AttnPlan p{};
    const int64_t G = Hq / Hkv;
    if (max_q > T) max_q = T;
    const int64_t rows = max_q * G;
    p.R = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    p.row_groups = (rows + 16 * p.R - 1) / (16 * p.R);
    const int64_t tiles = B * p.row_groups * Hkv;
    int64_t keys = max_kv;
    if (window > 0) {
        const int64_t reach = window + sinks + (16 * p.R + G - 1) / G + 2 * kBlockKeys;
        if (reach < keys) keys = reach;
    }
    const int64_t blocks = (keys + kBlockKeys - 1) / kBlockKeys;
    p.splits = 1;
    p.split_blocks = blocks > 0 ? blocks : 1;
    if (tiles <= kMaxFlags && blocks > 8) {
        int64_t per = (tiles * blocks + compute_units * 8 - 1) / (compute_units * 8);
        if (per < 8) per = 8;
        int64_t s = (blocks + per - 1) / per;
        const int64_t most = 256 / p.R;  // the join's weights: splits * rows <= 4096 floats of LDS
        if (s > most) s = most;
        per = (blocks + s - 1) / s;
        p.splits = (blocks + per - 1) / per;
        p.split_blocks = per;
    }
    const int64_t held = rows < 16 * p.R ? rows : 16 * p.R;
    p.slab = held * (D + 2);
    p.data_bytes = p.splits > 1 ? (size_t)(tiles * p.splits * p.slab) * 4 : 0;
    return p;
}

hipError_t launch_attention(const AttnArgs& args, const AttnPlan& plan, hipStream_t s) {
    AttnArgs a = args;
    a.R = plan.R;
    a.row_groups = (int)plan.row_groups;
    a.splits = (int)plan.splits;
    a.split_blocks = (int)plan.split_blocks;
    a.slab = plan.slab;
    const int64_t grid = (int64_t)a.B * plan.row_groups * plan.splits * a.Hkv;
    if (grid <= 0 || grid > 0x7FFFFFFF) return hipErrorInvalidValue;
    const dim3 gd((unsigned)grid), bd(kRowsThreads);
    if (a.bf16) {
        if (a.D == 64) rows_kernel<AttnBF16, 64><<<gd, bd, 0, s>>>(a);
        else rows_kernel<AttnBF16, 128><<<gd, bd, 0, s>>>(a);
    } else {
        if (a.D == 64) rows_kernel<AttnF16, 64><<<gd, bd, 0, s>>>(a);
        else rows_kernel<AttnF16, 128><<<gd, bd, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace tq
