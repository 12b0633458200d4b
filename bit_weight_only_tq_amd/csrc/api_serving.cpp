// extern "C" entry points of the serving operators: argument checks, then one
// launcher call.  See include/tq.h for the contract.  Like the rest of the
// library they work on the caller's current device and stream and keep no
// state between calls.

#include "tq.h"

#include <hip/hip_runtime.h>
#include <math.h>

#include "tq_internal.h"

namespace {

constexpr int64_t kInt32Max = 0x7FFFFFFF;

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

tq_status from_hip(hipError_t e) { return e == hipSuccess ? TQ_OK : TQ_ERR_HIP; }

// log2 of a page size (a power of two from 16 to 1024), or -1.
int page_shift(int64_t page_size) {
    for (int s = 4; s <= 10; ++s)
        if (page_size == (int64_t)1 << s) return s;
    return -1;
}

// `bytes` bytes of a caller's buffer; empty ones overlap nothing.
struct Span {
    const void* p;
    int64_t bytes;
    bool overlaps(const Span& o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        return bytes > 0 && o.bytes > 0 && a < b + (uintptr_t)o.bytes && b < a + (uintptr_t)bytes;
    }
};

}  // namespace

extern "C" {

tq_status tq_paged_plan(const int32_t* ctx_lens, const int32_t* new_lens, int32_t* page_table, int64_t table_stride,
                        const int32_t* free_pages, const int32_t* free_head, int64_t B, int64_t width, int64_t n_free,
                        int64_t T, int64_t page_size, int32_t* cu_q, int32_t* kv_lens, int32_t* positions,
                        int64_t* slots, int32_t* state, hipStream_t stream) {
    if (!ctx_lens || !new_lens || !page_table || !free_head || !cu_q || !kv_lens || !state) return TQ_ERR_NULL;
    if (n_free > 0 && !free_pages) return TQ_ERR_NULL;
    if (T > 0 && (!positions || !slots)) return TQ_ERR_NULL;
    if (B <= 0 || B > tq::kPlanMaxRequests || width <= 0 || width > kInt32Max || n_free < 0 || n_free > kInt32Max ||
        T < 0 || T > kInt32Max)
        return TQ_ERR_SHAPE;
    const int shift = page_shift(page_size);
    if (shift < 0 || table_stride < width) return TQ_ERR_VALUE;
    if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(page_table, 4) || !aligned(free_pages, 4) ||
        !aligned(free_head, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) || !aligned(positions, 4) ||
        !aligned(slots, 8) || !aligned(state, 4))
        return TQ_ERR_ALIGN;
    // every workgroup reads the lengths and the free list while others write
    const Span span[] = {{page_table, ((B - 1) * table_stride + width) * 4}, {cu_q, (B + 1) * 4}, {kv_lens, B * 4},
                         {positions, T * 4}, {slots, T * 8}, {state, 8},  // written
                         {ctx_lens, B * 4}, {new_lens, B * 4}, {free_pages, n_free * 4}, {free_head, 4}};
    for (int w = 0; w < 6; ++w)
        for (int o = w + 1; o < 10; ++o)
            if (span[w].overlaps(span[o])) return TQ_ERR_VALUE;
    const tq::PlanArgs a{ctx_lens, new_lens, page_table, table_stride, free_pages, free_head, (int)B,     (int)width,
                         (int)n_free, (int)T, shift,     cu_q,         kv_lens,    positions, slots, state};
    return from_hip(tq::launch_paged_plan(a, stream));
}

tq_status tq_kv_append(const void* q, int64_t q_stride, int64_t q_head, const void* k, int64_t k_stride,
                       int64_t k_head, const void* v, int64_t v_stride, int64_t v_head, tq_dtype dt, int64_t T,
                       int64_t Hq, int64_t Hkv, int64_t D, void* k_cache, void* v_cache, int64_t pages,
                       int64_t page_size, int64_t page_stride, const int64_t* slots, const int32_t* positions,
                       const float* rope, int64_t rope_rows, int64_t rot, int interleaved, void* q_out,
                       hipStream_t stream) {
    if (dt != TQ_F16 && dt != TQ_BF16) return TQ_ERR_DTYPE;
    if (T < 0 || T > kInt32Max || Hq < 0 || Hq > 4096 || Hkv <= 0 || Hkv > 4096 || D <= 0 || D > 4096 || pages <= 0 ||
        pages > kInt32Max || rot < 0 || rot > D || rot % 2 != 0)
        return TQ_ERR_SHAPE;
    const int shift = page_shift(page_size);
    if (shift < 0 || page_stride < Hkv * page_size * D) return TQ_ERR_VALUE;
    if (T == 0) return TQ_OK;
    if (!k || !v || !k_cache || !v_cache || !slots) return TQ_ERR_NULL;
    if (Hq > 0 && (!q || !q_out)) return TQ_ERR_NULL;
    if (rot > 0 && (!rope || !positions)) return TQ_ERR_NULL;
    if (rot > 0 && rope_rows <= 0) return TQ_ERR_SHAPE;
    if (!aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(k_cache, 2) || !aligned(v_cache, 2) ||
        !aligned(q_out, 2) || !aligned(slots, 8) || !aligned(positions, 4) || !aligned(rope, 4))
        return TQ_ERR_ALIGN;
    tq::AppendArgs a;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q_stride = q_stride;
    a.q_head = q_head;
    a.k_stride = k_stride;
    a.k_head = k_head;
    a.v_stride = v_stride;
    a.v_head = v_head;
    a.bf16 = dt == TQ_BF16 ? 1 : 0;
    a.T = T;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.D = (int)D;
    a.k_cache = static_cast<uint16_t*>(k_cache);
    a.v_cache = static_cast<uint16_t*>(v_cache);
    a.pages = pages;
    a.page_stride = page_stride;
    a.shift = shift;
    a.slots = slots;
    a.positions = positions;
    a.rope = rope;
    a.rope_rows = rope_rows;
    a.rot = (int)rot;
    a.interleaved = interleaved ? 1 : 0;
    a.q_out = static_cast<uint16_t*>(q_out);
    return from_hip(tq::launch_kv_append(a, stream));
}

static bool attention_sizes_ok(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q, int64_t max_kv) {
    return T >= 0 && T <= kInt32Max && Hkv > 0 && Hkv <= 4096 && Hq > 0 && Hq <= 65536 && Hq % Hkv == 0 &&
           (D == 64 || D == 128) && B > 0 && B <= kInt32Max && max_q >= (T > 0 ? 1 : 0) && max_q <= kInt32Max &&
           max_kv >= 0 && max_kv <= kInt32Max && T * Hq / 128 + B * Hkv < ((int64_t)1 << 24);  // workgroups, of 256 threads
}

size_t tq_paged_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q,
                                          int64_t max_kv, int64_t window, int64_t sinks) {
    if (!attention_sizes_ok(T, Hq, Hkv, D, B, max_q, max_kv) || T == 0 || window < 0 || sinks < 0) return 0;
    const tq::AttnPlan p = tq::attn_plan(T, Hq, Hkv, D, B, max_q, max_kv, window, sinks, tq::compute_units());
    return p.data_bytes ? tq::kFlagBytes + p.data_bytes : 0;
}

tq_status tq_paged_attention(const void* q, int64_t q_stride, int64_t q_head, tq_dtype dt, int64_t T, int64_t Hq,
                             int64_t Hkv, int64_t D, const void* k_cache, const void* v_cache, int64_t pages,
                             int64_t page_size, int64_t page_stride, const int32_t* page_table, int64_t table_stride,
                             int64_t width, const int32_t* cu_q, const int32_t* kv_lens, int64_t B, int64_t max_q,
                             int64_t max_kv, float scale, int64_t window, int64_t sinks, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (dt != TQ_F16 && dt != TQ_BF16) return TQ_ERR_DTYPE;
    if (!attention_sizes_ok(T, Hq, Hkv, D, B, max_q, max_kv) || pages <= 0 || pages > kInt32Max || width <= 0 ||
        width > kInt32Max)
        return TQ_ERR_SHAPE;
    const int shift = page_shift(page_size);
    if (shift < 0 || page_stride < Hkv * page_size * D || table_stride < width) return TQ_ERR_VALUE;
    if (!(scale > 0.0f) || !isfinite(scale)) return TQ_ERR_VALUE;
    if (window < 0 || window > kInt32Max || sinks < 0 || sinks > kInt32Max) return TQ_ERR_VALUE;
    if (T == 0) return TQ_OK;
    if (!q || !k_cache || !v_cache || !page_table || !cu_q || !kv_lens || !out) return TQ_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(workspace, 16) || !aligned(page_table, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) ||
        !aligned(lse, 4) || q_stride % 8 || q_head % 8 || page_stride % 8)
        return TQ_ERR_ALIGN;
    const tq::AttnPlan plan = tq::attn_plan(T, Hq, Hkv, D, B, max_q, max_kv, window, sinks, tq::compute_units());
    tq::AttnArgs a{};
    if (plan.data_bytes && workspace && workspace_bytes >= tq::kFlagBytes + plan.data_bytes) {
        a.flags = static_cast<uint32_t*>(workspace);
        a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + tq::kFlagBytes);
    }
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_stride;
    a.q_head = q_head;
    a.bf16 = dt == TQ_BF16 ? 1 : 0;
    a.T = (int)T;
    a.B = (int)B;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.G = (int)(Hq / Hkv);
    a.D = (int)D;
    a.k = static_cast<const uint16_t*>(k_cache);
    a.v = static_cast<const uint16_t*>(v_cache);
    a.pages = pages;
    a.page_stride = page_stride;
    a.shift = shift;
    a.table = page_table;
    a.table_stride = table_stride;
    a.width = (int)width;
    a.cu = cu_q;
    a.kv = kv_lens;
    a.max_q = (int)max_q;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.window = (int)window;
    a.sinks = (int)sinks;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    return from_hip(tq::launch_attention(a, plan, stream));
}

tq_status tq_sample(const void* logits, tq_dtype dt, int64_t B, int64_t V, int64_t row_stride, const float* u,
                    const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                    int32_t* tokens, float* logprobs, hipStream_t stream) {
    if (dt != TQ_F16 && dt != TQ_BF16 && dt != TQ_F32) return TQ_ERR_DTYPE;
    if (B < 0 || B > kInt32Max || V <= 0 || V > tq::kSampleMaxVocab) return TQ_ERR_SHAPE;
    if (B > 1 && row_stride < V) return TQ_ERR_VALUE;
    if (B == 0) return TQ_OK;
    if (!logits || !u || !tokens) return TQ_ERR_NULL;
    if (!aligned(logits, dt == TQ_F32 ? 4 : 2) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
        !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(logprobs, 4))
        return TQ_ERR_ALIGN;
    tq::SampleArgs a;
    a.logits = logits;
    a.dtype = (int)dt;
    a.B = B;
    a.V = (int)V;
    a.row_stride = row_stride;
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.tokens = tokens;
    a.logprobs = logprobs;
    return from_hip(tq::launch_sample(a, stream));
}

}  // extern "C"
