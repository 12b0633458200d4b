// Paged-cache kernels of a serving step: the step's plan (page tables, token
// offsets, positions and slots from the requests' lengths) and the append of
// its keys and values, with rotary positions, to the cache.

#include "tq_device.h"
#include "tq_internal.h"

namespace tq {

namespace {

// Sum of two non-negative int32, at most 2^31 - 1 (associative, so a scan
// with it is well defined whatever the lengths hold).
__device__ __forceinline__ int sat_add(int a, int b) {
    const uint32_t s = (uint32_t)a + (uint32_t)b;
    return s > 0x7FFFFFFFu ? 0x7FFFFFFF : (int)s;
}

__device__ __forceinline__ int pages_of(int len, int shift, int width) {
    const int n = (int)(((uint32_t)len + (1u << shift) - 1u) >> shift);
    return n < width ? n : width;
}

// Largest i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
    int lo = 0, hi = n;  // a[lo] <= x, a[hi] > x or hi == n
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// ---- plan.  Request b holds `held` pages and needs `need` after its new
// tokens, so with the exclusive prefix sums of the new tokens (cu) and of the
// new pages (take) every output is local: token t belongs to the last b with
// cu[b] <= t, the i-th fresh page of b is entry head + take[b] + i of the
// free list, and the token that begins a fresh page writes its table entry.
//
// One launch: 2.7 us in the kernel at 8 requests, 7.3 us at 2048 requests with
// 67 thousand new tokens, where empty kernels follow each other every 2.5.  Every
// workgroup scans all B requests by itself (2048 requests are 16 KiB out of L2)
// rather than waiting for a scan kernel: a step this small is bound by launches,
// not by bytes.  Workgroup 0 writes the
// per-request outputs and counts the tokens left without a slot, by ranges of
// tokens instead of token by token; the others take the tokens.
__global__ __launch_bounds__(1024) void plan_kernel(PlanArgs a) {
    extern __shared__ int lds[];
    int* cu = lds;               // [B + 1]
    int* take = lds + a.B + 1;   // [B + 1]
    __shared__ int wave_new[16], wave_pg[16], lost;
    const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 63, wave = tid >> 6;
    const int B = a.B, shift = a.shift, width = a.width;
    if (tid == 0) lost = 0;

    // prefix sums: a run of `per` requests a thread, then lanes, then waves
    const int per = (B + nthr - 1) / nthr;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    int sn = 0, sp = 0;
    for (int b = b0; b < b1; ++b) {
        const int c = max(a.ctx[b], 0), n = max(a.fresh[b], 0);
        sn = sat_add(sn, n);
        sp = sat_add(sp, pages_of(sat_add(c, n), shift, width) - pages_of(c, shift, width));
    }
    int in = sn, ip = sp;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int on = __shfl_up(in, d, 64), op = __shfl_up(ip, d, 64);
        if (lane >= d) {
            in = sat_add(in, on);
            ip = sat_add(ip, op);
        }
    }
    if (lane == 63) {
        wave_new[wave] = in;
        wave_pg[wave] = ip;
    }
    // the lanes before this one; exclusive, so no subtraction of a saturated sum
    int en = __shfl_up(in, 1, 64), ep = __shfl_up(ip, 1, 64);
    if (lane == 0) en = ep = 0;
    __syncthreads();
    int wn = 0, wp = 0;
    for (int w = 0; w < wave; ++w) {
        wn = sat_add(wn, wave_new[w]);
        wp = sat_add(wp, wave_pg[w]);
    }
    en = sat_add(wn, en);
    ep = sat_add(wp, ep);
    for (int b = b0; b < b1; ++b) {
        const int c = max(a.ctx[b], 0), n = max(a.fresh[b], 0), kv = sat_add(c, n);
        cu[b] = en;
        take[b] = ep;
        if (blockIdx.x == 0) {
            a.cu_q[b] = en;
            a.kv_lens[b] = kv;
        }
        en = sat_add(en, n);
        ep = sat_add(ep, pages_of(kv, shift, width) - pages_of(c, shift, width));
    }
    if (b0 < B && b1 == B) {  // the thread with the last request
        cu[B] = en;
        take[B] = ep;
        if (blockIdx.x == 0) a.cu_q[B] = en;
    }
    __syncthreads();

    const int total = cu[B], new_pages = take[B];
    const int head = min(max(*a.free_head, 0), a.n_free);
    const int page = 1 << shift, T = a.T;
    // tokens: positions, slots, and the table entries of the pages they begin
    const int64_t span = max(T, total);
    for (int64_t t64 = (int64_t)(blockIdx.x - 1) * nthr + tid; blockIdx.x > 0 && t64 < span; t64 += (int64_t)(gridDim.x - 1) * nthr) {
        const int t = (int)t64;
        int pos = 0;
        int64_t slot = -1;
        if (t < total) {
            const int b = last_at_most(cu, B, t);
            const int c = max(a.ctx[b], 0);
            pos = sat_add(c, t - cu[b]);
            const int blk = pos >> shift, off = pos & (page - 1);
            if (blk < width) {
                const int held = pages_of(c, shift, width);
                int32_t* entry = a.table + (int64_t)b * a.table_stride + blk;
                int id;
                if (blk < held) {
                    id = *entry;
                } else {
                    const int64_t at = (int64_t)head + take[b] + (blk - held);
                    id = at < a.n_free ? a.free_pages[at] : -1;
                    if (off == 0) *entry = id;
                }
                if (id >= 0) slot = ((int64_t)id << shift) + off;
            }
        }
        if (t < T) {
            a.positions[t] = pos;
            a.slots[t] = slot;
        }
    }

    if (blockIdx.x != 0) return;
    int miss = 0;
    // fresh pages without an id: the tokens t0 .. t1 of the step that lie in them
    for (int f = tid; f < new_pages; f += nthr) {
        const int64_t at = (int64_t)head + f;
        if (at < a.n_free && a.free_pages[at] >= 0) continue;
        const int b = last_at_most(take, B, f);
        const int c = max(a.ctx[b], 0);
        const int64_t p0 = (int64_t)(pages_of(c, shift, width) + (f - take[b])) << shift;
        const int64_t t0 = cu[b] + (p0 - c);
        int64_t t1 = t0 + page;
        if (t1 > cu[b + 1]) t1 = cu[b + 1];
        if (t1 > T) t1 = T;
        if (t1 > t0) miss += (int)(t1 - t0);
    }
    for (int b = tid; b < B; b += nthr) {
        const int c = max(a.ctx[b], 0);
        const int64_t end = min(cu[b + 1], T);
        // tokens past the table's width
        int64_t over = cu[b] + (((int64_t)width << shift) - c);
        if (over < cu[b]) over = cu[b];
        if (end > over) miss += (int)(end - over);
        // tokens in a held page that the table does not name
        if ((c & (page - 1)) && (c >> shift) < width && a.table[(int64_t)b * a.table_stride + (c >> shift)] < 0) {
            int64_t t1 = cu[b] + (page - (c & (page - 1)));
            if (t1 > end) t1 = end;
            if (t1 > cu[b]) miss += (int)(t1 - cu[b]);
        }
    }
    if (tid == 0 && total > T) miss += total - T;
    if (miss) atomicAdd(&lost, miss);  // whole numbers in LDS: any order gives the same sum
    __syncthreads();
    if (tid == 0) {
        a.state[0] = min(sat_add(head, new_pages), a.n_free);
        a.state[1] = lost;
    }
}

// ---- append.  A rotated pair (x, y) becomes (x cos - y sin, y cos + x sin) in
// fp32, rounded once to the cache's type; keys and values go to their slots,
// the queries to q_out.  Bound by memory: everything is read and written once,
// 16383 tokens of 64 + 8 heads of 128 in 125 us, 5.4 TB/s; a large copy reaches
// 4.8 TB/s on this card.

// Eight 16-bit values of a 16-byte vector.
__device__ __forceinline__ uint16_t half_of(const uint4& v, int i) {
    const uint32_t w = dword_of(v, i >> 1);
    return (uint16_t)(i & 1 ? w >> 16 : w);
}
template <class E>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)E::from_f32_fast(x[2 * i]) | ((uint32_t)E::from_f32_fast(x[2 * i + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The angles of one token: its row of the table, or NaN where the position
// lies outside it (the rotated values then are NaN: loud, and nothing is read
// out of bounds).
struct Angles {
    const float* row;
    bool bad;
};
__device__ __forceinline__ Angles angles_of(const AppendArgs& a, int64_t t) {
    Angles g{a.rope, false};
    if (a.rot == 0) return g;
    const int p = a.positions[t];
    if (p < 0 || p >= a.rope_rows) g.bad = true;
    else g.row = a.rope + (int64_t)p * a.rot;
    return g;
}

// Element offset of the first value of a token's head in the cache, or -1.
__device__ __forceinline__ int64_t cache_at(const AppendArgs& a, int64_t t, int h) {
    const int64_t slot = a.slots[t];
    const int64_t pg = slot >> a.shift;
    if (slot < 0 || pg >= a.pages) return -1;
    return pg * a.page_stride + (((int64_t)h << a.shift) + (slot & ((1 << a.shift) - 1))) * a.D;
}

// 16-byte form.  A token's work is a list of items: per rotated head rot / 16
// pairs of vectors (halves) or rot / 8 single vectors (interleaved) and
// (D - rot) / 8 copies, per value head D / 8 copies; a workgroup takes
// `a.tokens_per_group` tokens and its threads run over their items, so that a
// single token of a few heads still spreads over several workgroups' lanes.
template <class E, bool INTER>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
    const int rot_items = INTER ? a.rot / 8 : a.rot / 16;
    const int per_head = rot_items + (a.D - a.rot) / 8;
    const int v_items = a.D / 8;
    const int qk = (a.Hq + a.Hkv) * per_head;
    const int items = qk + a.Hkv * v_items;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_group;
    const int nt = (int)(a.T - t0 < a.tokens_per_group ? a.T - t0 : a.tokens_per_group);
    for (int i = blockIdx.y * 256 + threadIdx.x; i < nt * items; i += gridDim.y * 256) {
        const int tl = i / items, it = i - tl * items;
        const int64_t t = t0 + tl;
        if (it >= qk) {  // a vector of a value head
            const int h = (it - qk) / v_items, c = (it - qk) - h * v_items;
            const int64_t at = cache_at(a, t, h);
            if (at >= 0)
                *reinterpret_cast<uint4*>(a.v_cache + at + 8 * c) =
                    *reinterpret_cast<const uint4*>(a.v + t * a.v_stride + h * a.v_head + 8 * c);
            continue;
        }
        const int hh = it / per_head, c = it - hh * per_head;
        const bool is_q = hh < a.Hq;
        const int h = is_q ? hh : hh - a.Hq;
        const uint16_t* src = is_q ? a.q + t * a.q_stride + h * a.q_head : a.k + t * a.k_stride + h * a.k_head;
        uint16_t* dst;
        if (is_q) {
            dst = a.q_out + (t * a.Hq + h) * a.D;
        } else {
            const int64_t at = cache_at(a, t, h);
            if (at < 0) continue;
            dst = a.k_cache + at;
        }
        if (c >= rot_items) {
            const int e = a.rot + 8 * (c - rot_items);
            *reinterpret_cast<uint4*>(dst + e) = *reinterpret_cast<const uint4*>(src + e);
            continue;
        }
        const Angles g = angles_of(a, t);
        const int half = a.rot >> 1;
        if constexpr (INTER) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * c);
            const float4 cs = *reinterpret_cast<const float4*>(g.row + 4 * c);
            const float4 sn = *reinterpret_cast<const float4*>(g.row + half + 4 * c);
            const float co[4] = {cs.x, cs.y, cs.z, cs.w}, si[4] = {sn.x, sn.y, sn.z, sn.w};
            float r[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = E::to_f32(half_of(v, 2 * j)), y = E::to_f32(half_of(v, 2 * j + 1));
                r[2 * j] = g.bad ? NAN : x * co[j] - y * si[j];
                r[2 * j + 1] = g.bad ? NAN : y * co[j] + x * si[j];
            }
            *reinterpret_cast<uint4*>(dst + 8 * c) = pack8<E>(r);
        } else {
            const uint4 vx = *reinterpret_cast<const uint4*>(src + 8 * c);
            const uint4 vy = *reinterpret_cast<const uint4*>(src + half + 8 * c);
            const float4* cs = reinterpret_cast<const float4*>(g.row + 8 * c);
            const float4* sn = reinterpret_cast<const float4*>(g.row + half + 8 * c);
            const float4 c0 = cs[0], c1 = cs[1], s0 = sn[0], s1 = sn[1];
            const float co[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const float si[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
            float rx[8], ry[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = E::to_f32(half_of(vx, j)), y = E::to_f32(half_of(vy, j));
                rx[j] = g.bad ? NAN : x * co[j] - y * si[j];
                ry[j] = g.bad ? NAN : y * co[j] + x * si[j];
            }
            *reinterpret_cast<uint4*>(dst + 8 * c) = pack8<E>(rx);
            *reinterpret_cast<uint4*>(dst + half + 8 * c) = pack8<E>(ry);
        }
    }
}

// Element form for heads, strides or pointers that 16-byte vectors do not fit:
// one item is a pair of a rotated head or one copied value.  Bound by the number
// of its 2-byte accesses: 16383 tokens of 64 + 8 heads of 128 in rows of 131 take
// 270 us (336 without rotation, whose items are single values), heads of 80 with
// 20 rotated 302 us; a copy of as many bytes takes 142 and 88.  A single token
// takes as long as in vectors (4.8 us a call).
template <class E>
__global__ __launch_bounds__(256) void append_element_kernel(AppendArgs a) {
    const int half = a.rot >> 1;
    const int per_head = half + (a.D - a.rot);
    const int qk = (a.Hq + a.Hkv) * per_head;
    const int items = qk + a.Hkv * a.D;
    const int64_t t = blockIdx.x;
    for (int it = blockIdx.y * 256 + threadIdx.x; it < items; it += gridDim.y * 256) {
        if (it >= qk) {
            const int h = (it - qk) / a.D, d = (it - qk) - h * a.D;
            const int64_t at = cache_at(a, t, h);
            if (at >= 0) a.v_cache[at + d] = a.v[t * a.v_stride + h * a.v_head + d];
            continue;
        }
        const int hh = it / per_head, c = it - hh * per_head;
        const bool is_q = hh < a.Hq;
        const int h = is_q ? hh : hh - a.Hq;
        const uint16_t* src = is_q ? a.q + t * a.q_stride + h * a.q_head : a.k + t * a.k_stride + h * a.k_head;
        uint16_t* dst;
        if (is_q) {
            dst = a.q_out + (t * a.Hq + h) * a.D;
        } else {
            const int64_t at = cache_at(a, t, h);
            if (at < 0) continue;
            dst = a.k_cache + at;
        }
        if (c >= half) {
            const int e = a.rot + (c - half);
            dst[e] = src[e];
            continue;
        }
        const Angles g = angles_of(a, t);
        const float co = g.bad ? NAN : g.row[c], si = g.bad ? NAN : g.row[half + c];
        const int ex = a.interleaved ? 2 * c : c, ey = a.interleaved ? 2 * c + 1 : c + half;
        const float x = E::to_f32(src[ex]), y = E::to_f32(src[ey]);
        dst[ex] = E::from_f32_fast(x * co - y * si);
        dst[ey] = E::from_f32_fast(y * co + x * si);
    }
}

bool vectors_fit(const AppendArgs& a) {
    auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    if (a.D % 8 || a.rot % (a.interleaved ? 8 : 16) || a.page_stride % 8) return false;
    if (a.k_stride % 8 || a.k_head % 8 || a.v_stride % 8 || a.v_head % 8) return false;
    if (!al(a.k) || !al(a.v) || !al(a.k_cache) || !al(a.v_cache)) return false;
    if (a.Hq && (a.q_stride % 8 || a.q_head % 8 || !al(a.q) || !al(a.q_out))) return false;
    return a.rot == 0 || al(a.rope);
}

}  // namespace

hipError_t launch_paged_plan(const PlanArgs& a, hipStream_t s) {
    static DeviceFlags raised;
    const size_t lds = (size_t)(a.B + 1) * 8;
    if (lds > (48u << 10)) {
        const hipError_t e =
            raise_lds_limit(reinterpret_cast<const void*>(plan_kernel), (kPlanMaxRequests + 1) * 8, raised);
        if (e != hipSuccess) return e;
    }
    // a small step is one small workgroup: its waves start and meet sooner
    const int threads = a.B <= 256 && a.T <= 256 ? 256 : 1024;
    const int64_t groups = ((int64_t)a.T + threads - 1) / threads;
    const unsigned grid = 1u + (unsigned)(groups < 1 ? 1 : groups > 512 ? 512 : groups);
    plan_kernel<<<dim3(grid), dim3(threads), lds, s>>>(a);
    return hipGetLastError();
}

// The tokens of one launch.
static hipError_t launch_append_part(AppendArgs a, bool vectors, hipStream_t s) {
    if (!vectors) {
        const int items = (a.Hq + a.Hkv) * (a.D - a.rot / 2) + a.Hkv * a.D;
        const int gy = items > 8 * 256 ? 8 : (items + 255) / 256;
        if (a.bf16) append_element_kernel<BF16><<<dim3((unsigned)a.T, gy), dim3(256), 0, s>>>(a);
        else append_element_kernel<F16><<<dim3((unsigned)a.T, gy), dim3(256), 0, s>>>(a);
        return hipGetLastError();
    }
    const int rot_items = a.interleaved ? a.rot / 8 : a.rot / 16;
    const int items = (a.Hq + a.Hkv) * (rot_items + (a.D - a.rot) / 8) + a.Hkv * (a.D / 8);
    // few tokens: their items spread over workgroups of one item a thread;
    // many: a workgroup has at least two items a thread
    a.tokens_per_group = items >= 512 ? 1 : (512 + items - 1) / items;
    const int64_t gx = (a.T + a.tokens_per_group - 1) / a.tokens_per_group;
    int gy = 1;
    if (gx < 512) {
        const int need = (int)(((int64_t)items * a.tokens_per_group + 255) / 256);
        gy = need < 64 ? need : 64;
    }
    const dim3 grid((unsigned)gx, (unsigned)gy);
    if (a.bf16) {
        if (a.interleaved) append_kernel<BF16, true><<<grid, dim3(256), 0, s>>>(a);
        else append_kernel<BF16, false><<<grid, dim3(256), 0, s>>>(a);
    } else {
        if (a.interleaved) append_kernel<F16, true><<<grid, dim3(256), 0, s>>>(a);
        else append_kernel<F16, false><<<grid, dim3(256), 0, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_kv_append(const AppendArgs& args, hipStream_t s) {
    const bool vectors = vectors_fit(args);
    for (int64_t t = 0; t < args.T; t += kMaxGroups) {
        AppendArgs a = args;
        a.T = args.T - t < kMaxGroups ? args.T - t : kMaxGroups;
        if (a.Hq) {
            a.q += t * a.q_stride;
            a.q_out += t * a.Hq * a.D;
        }
        a.k += t * a.k_stride;
        a.v += t * a.v_stride;
        a.slots += t;
        if (a.rot) a.positions += t;
        const hipError_t e = launch_append_part(a, vectors, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace tq
