// extern "C" entry points of the experts' and adapters' operators: argument
// checks, then one launcher call.  See include/tq.h for the contract.

#include "tq.h"

#include <hip/hip_runtime.h>

#include "tq_checks.h"
#include "tq_internal.h"

namespace {

bool route_sizes_ok(int64_t T, int64_t E, int64_t top_k) {
    return T >= 0 && E > 0 && E <= tq::kRouteMaxExperts && top_k > 0 && top_k <= E && top_k <= tq::kRouteMaxChosen &&
           T <= kInt32Max / top_k;
}

bool expert_sizes_ok(int fmt, int64_t P, int64_t E, int64_t N, int64_t K) {
    return P >= 0 && P <= kInt32Max && E > 0 && E <= 65536 && N > 0 && N <= tq::kMaxK && K > 0 && K <= tq::kMaxK &&
           K % (fmt == 0 ? 64 : 128) == 0 && N * K <= (int64_t)1 << 32;
}

// The checks and the launch of both formats' products.
tq_status moe_gemm(const void* A, tq_dtype dt, int64_t T, int64_t P, int64_t E, int64_t N, int64_t K, int fmt,
                   const void* w, const uint16_t* scale, const uint8_t* zeros, const int32_t* offsets,
                   const int32_t* rows, const void* bias, int gated, void* C, hipStream_t stream) {
    if (dt != TQ_F16 && dt != TQ_BF16) return TQ_ERR_DTYPE;
    if (T < 0 || T > kInt32Max || !expert_sizes_ok(fmt, P, E, N, K) || (gated && N % 2 != 0)) return TQ_ERR_SHAPE;
    if (rows ? (T == 0 ? P != 0 : P % T != 0) : P != T) return TQ_ERR_SHAPE;
    if (P == 0) return TQ_OK;
    if (!A || !w || !scale || !offsets || !C) return TQ_ERR_NULL;
    if (!aligned(A, 16) || !aligned(w, 16) || !aligned(scale, 2) || !aligned(offsets, 4) || !aligned(rows, 4) ||
        !aligned(bias, 2) || !aligned(C, 2))
        return TQ_ERR_ALIGN;
    // rows of C are written while others of A are read
    const int64_t units = fmt == 0 ? 1 : K / 128;  // scales of a weight row
    const Span to{C, P * (gated ? N / 2 : N) * 2};
    const Span from[] = {{A, T * K * 2}, {w, E * N * (K / (fmt == 0 ? 4 : 2))}, {scale, E * N * units * 2},
                         {zeros, zeros ? E * N * units : 0}, {offsets, (E + 1) * 4}, {rows, rows ? P * 4 : 0},
                         {bias, bias ? E * N * 2 : 0}};
    for (const Span& s : from)
        if (to.overlaps(s)) return TQ_ERR_VALUE;
    tq::ExpertArgs a{};
    a.A = static_cast<const uint16_t*>(A);
    a.bf16 = dt == TQ_BF16 ? 1 : 0;
    a.T = T;
    a.P = P;
    a.E = E;
    a.N = N;
    a.K = K;
    a.fmt = fmt;
    a.w = static_cast<const uint8_t*>(w);
    a.scale = scale;
    a.zeros = zeros;
    a.offsets = offsets;
    a.rows = rows;
    a.fan = (int)(P / T);
    a.bias = static_cast<const uint16_t*>(bias);
    a.C = static_cast<uint16_t*>(C);
    a.gated = gated ? 1 : 0;
    return from_hip(tq::launch_experts(a, stream));
}

}  // namespace

extern "C" {

size_t tq_moe_route_workspace_bytes(int64_t T, int64_t E, int64_t top_k) {
    if (!route_sizes_ok(T, E, top_k)) return 0;
    const int64_t chunk = tq::route_chunk(T);
    return chunk ? (size_t)((T + chunk - 1) / chunk) * (size_t)E * 4 : 0;
}

tq_status tq_moe_route(const void* logits, tq_dtype dt, int64_t T, int64_t E, int64_t row_stride, int64_t top_k,
                       int renormalize, int32_t* experts, float* weights, int32_t* offsets, int32_t* rows,
                       int32_t* places, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (dt != TQ_F16 && dt != TQ_BF16 && dt != TQ_F32) return TQ_ERR_DTYPE;
    if (T <= 0 || !route_sizes_ok(T, E, top_k)) return TQ_ERR_SHAPE;
    if (T > 1 && row_stride < E) return TQ_ERR_VALUE;
    if (!logits || !experts || !weights || !offsets || !rows || !places) return TQ_ERR_NULL;
    if (!aligned(logits, dt == TQ_F32 ? 4 : 2) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(offsets, 4) ||
        !aligned(rows, 4) || !aligned(places, 4) || !aligned(workspace, 4))
        return TQ_ERR_ALIGN;
    const size_t need = tq_moe_route_workspace_bytes(T, E, top_k);
    if (need && (!workspace || workspace_bytes < need)) return TQ_ERR_SHAPE;
    // no value is written where another is read or written
    const int64_t pairs = T * top_k * 4;
    const Span span[] = {{experts, pairs}, {weights, pairs}, {offsets, (E + 1) * 4}, {rows, pairs}, {places, pairs},
                         {workspace, (int64_t)need}, {logits, ((T - 1) * row_stride + E) * (dt == TQ_F32 ? 4 : 2)}};
    for (int i = 0; i < 6; ++i)
        for (int j = i + 1; j < 7; ++j)
            if (span[i].overlaps(span[j])) return TQ_ERR_VALUE;
    tq::RouteArgs a{};
    a.logits = logits;
    a.dtype = (int)dt;
    a.T = T;
    a.E = (int)E;
    a.k = (int)top_k;
    a.row_stride = row_stride;
    a.renormalize = renormalize ? 1 : 0;
    a.experts = experts;
    a.weights = weights;
    a.offsets = offsets;
    a.rows = rows;
    a.places = places;
    a.counts = static_cast<uint32_t*>(workspace);
    return from_hip(tq::launch_moe_route(a, stream));
}

tq_status tq_moe_gemm(const void* A, tq_dtype dt, int64_t T, int64_t P, int64_t E, int64_t N, int64_t K,
                      const uint8_t* codes, const uint16_t* scale_f16, const int32_t* offsets, const int32_t* rows,
                      const void* bias, int gated, void* C, hipStream_t stream) {
    return moe_gemm(A, dt, T, P, E, N, K, 0, codes, scale_f16, nullptr, offsets, rows, bias, gated, C, stream);
}

tq_status w4a16_moe_gemm(const void* A, tq_dtype dt, int64_t T, int64_t P, int64_t E, int64_t N, int64_t K,
                         const int32_t* qweight, const uint16_t* scales_f16, const uint8_t* zeros, int64_t group_size,
                         const int32_t* offsets, const int32_t* rows, const void* bias, int gated, void* C,
                         hipStream_t stream) {
    if (group_size != 128) return TQ_ERR_GROUP;
    return moe_gemm(A, dt, T, P, E, N, K, 1, qweight, scales_f16, zeros, offsets, rows, bias, gated, C, stream);
}

int tq_moe_select_cut(int format, int zeros, int64_t P, int64_t E, int64_t N, int64_t K) {
    if ((format != 0 && format != 1) || (format == 0 && zeros) || P < 1 || !expert_sizes_ok(format, P, E, N, K)) return -1;
    return tq::select_cut(format, zeros != 0, P, E, N, K);
}

tq_status tq_moe_combine(const void* y, tq_dtype dt, int64_t T, int64_t P, int64_t N, int64_t top_k,
                         const int32_t* places, const float* weights, const void* add, int64_t add_stride, void* out,
                         hipStream_t stream) {
    if (dt != TQ_F16 && dt != TQ_BF16) return TQ_ERR_DTYPE;
    if (T < 0 || T > kInt32Max || P < 0 || P > kInt32Max || N <= 0 || N > tq::kMaxK || top_k <= 0 || top_k > 65536)
        return TQ_ERR_SHAPE;
    if (add && T > 1 && add_stride < N) return TQ_ERR_VALUE;
    if (T == 0) return TQ_OK;
    if ((P > 0 && !y) || !places || !weights || !out) return TQ_ERR_NULL;
    if (!aligned(y, 2) || !aligned(places, 4) || !aligned(weights, 4) || !aligned(add, 2) || !aligned(out, 2))
        return TQ_ERR_ALIGN;
    const Span to{out, T * N * 2}, from[] = {{y, P * N * 2}, {places, T * top_k * 4}, {weights, T * top_k * 4}};
    for (const Span& s : from)
        if (to.overlaps(s)) return TQ_ERR_VALUE;
    // added rows may be the output's own
    if (add && !(add == out && (T == 1 || add_stride == N)) && to.overlaps(Span{add, ((T - 1) * add_stride + N) * 2}))
        return TQ_ERR_VALUE;
    tq::CombineArgs a{};
    a.y = static_cast<const uint16_t*>(y);
    a.bf16 = dt == TQ_BF16 ? 1 : 0;
    a.T = T;
    a.P = P;
    a.N = N;
    a.k = (int)top_k;
    a.places = places;
    a.weights = weights;
    a.add = static_cast<const uint16_t*>(add);
    a.add_stride = add_stride;
    a.out = static_cast<uint16_t*>(out);
    return from_hip(tq::launch_moe_combine(a, stream));
}

tq_status tq_lora(const void* x, int64_t x_stride, const void* base, int64_t base_stride, tq_dtype dt, int64_t T,
                  int64_t K, int64_t N, int64_t L, int64_t rank, const void* A, const void* B, const int32_t* ids,
                  const float* scale, void* out, int64_t out_stride, hipStream_t stream) {
    if (dt != TQ_F16 && dt != TQ_BF16) return TQ_ERR_DTYPE;
    if (T < 0 || T > ((int64_t)1 << 27) || K <= 0 || K > tq::kMaxK || K % 8 != 0 || N <= 0 || N > tq::kMaxK || L <= 0 ||
        L > kInt32Max || rank <= 0 || rank > 256 || rank % 8 != 0 || rank * K > tq::kLoraMaxAdapter ||
        rank * N > tq::kLoraMaxAdapter)
        return TQ_ERR_SHAPE;
    if (T == 1) x_stride = K, base_stride = out_stride = N;  // not looked at
    for (const int64_t* s : {&x_stride, &base_stride, &out_stride})
        if (*s < (s == &x_stride ? K : N) || *s > tq::kLoraMaxStride) return TQ_ERR_VALUE;
    if (T == 0) return TQ_OK;
    if (!x || !base || !A || !B || !ids || !out) return TQ_ERR_NULL;
    if (!aligned(x, 16) || x_stride % 8 || !aligned(A, 16) || !aligned(B, 16) || !aligned(base, 2) ||
        !aligned(out, 2) || !aligned(ids, 4) || !aligned(scale, 4))
        return TQ_ERR_ALIGN;
    // the update may be made in place; nothing else that is read may be written
    const Span to{out, ((T - 1) * out_stride + N) * 2};
    const Span from[] = {{x, ((T - 1) * x_stride + K) * 2}, {A, L * rank * K * 2}, {B, L * N * rank * 2}, {ids, T * 4},
                         {scale, scale ? L * 4 : 0}};
    for (const Span& s : from)
        if (to.overlaps(s)) return TQ_ERR_VALUE;
    if (!(base == out && base_stride == out_stride) && to.overlaps(Span{base, ((T - 1) * base_stride + N) * 2}))
        return TQ_ERR_VALUE;
    tq::LoraArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.x_stride = x_stride;
    a.base = static_cast<const uint16_t*>(base);
    a.base_stride = base_stride;
    a.bf16 = dt == TQ_BF16 ? 1 : 0;
    a.T = T;
    a.K = K;
    a.N = N;
    a.L = L;
    a.r = (int)rank;
    a.A = static_cast<const uint16_t*>(A);
    a.B = static_cast<const uint16_t*>(B);
    a.ids = ids;
    a.scale = scale;
    a.out = static_cast<uint16_t*>(out);
    a.out_stride = out_stride;
    return from_hip(tq::launch_lora(a, stream));
}

}  // extern "C"
