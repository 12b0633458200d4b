// Python entry of the serving, expert and adapter operators (the module _serving): tensors are
// checked, outputs allocated and the C ABI (tq.h) called on torch's current
// stream, without Python in between.  A serving step makes these calls once a
// layer, often on a few rows, where the host's time is the call's: an append of
// one token took 17 us through ctypes with checks in Python, of which the
// launch itself is 3.
//
// The C ABI takes bare pointers, so everything it cannot see (types, shapes,
// strides, devices) is checked here before any call.  bit_weight_only_tq_amd/
// serving.py and experts.py have the signatures and what the arguments mean.

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "tq.h"

namespace {

using at::Tensor;

[[noreturn]] void type_error(const std::string& s) { throw torch::TypeError(s); }
[[noreturn]] void value_error(const std::string& s) { throw c10::ValueError({__func__, __FILE__, (uint32_t)__LINE__}, s); }

std::string shape_of(const Tensor& t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}
std::string kind_of(const Tensor& t) { return std::to_string(t.dim()) + "-D " + std::string(c10::toString(t.scalar_type())); }

const Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const Tensor* optional(const char* name, PyObject* o) { return o == Py_None ? nullptr : &tensor(name, o); }

int64_t whole(const char* name, PyObject* o) {
    PyObject* i = PyNumber_Index(o);
    if (!i) throw python_error();
    int past = 0;
    const int64_t v = PyLong_AsLongLongAndOverflow(i, &past);
    Py_DECREF(i);
    if (past) value_error(std::string(name) + " does not fit 64 bits");
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

void is(const char* name, const Tensor& t, at::ScalarType type, int64_t dim) {
    if (t.scalar_type() != type || t.dim() != dim)
        type_error(std::string(name) + " must be a " + std::to_string(dim) + "-D " + c10::toString(type) + " tensor, got " +
                   kind_of(t));
}
void contiguous(const char* name, const Tensor& t) {
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
}
// A contiguous vector of n entries (any number for n < 0); -> its address.
void* vector(const char* name, const Tensor& t, at::ScalarType type, int64_t n = -1) {
    is(name, t, type, 1);
    if (n >= 0 && t.size(0) != n)
        value_error(std::string(name) + " must have " + std::to_string(n) + " entries, got " + std::to_string(t.size(0)));
    contiguous(name, t);
    return t.data_ptr();
}
template <class T>
T* vector_of(const char* name, const Tensor& t, int64_t n = -1) {
    return static_cast<T*>(vector(name, t, c10::CppTypeToScalarType<T>::value, n));
}

// All tensors are device tensors of one device (take each, then `index`).
struct OneDevice {
    int index = -1;
    void take(const Tensor& t) {
        if (!t.is_cuda()) value_error("tensors must be device tensors");
        const int i = t.device().index();
        if (index >= 0 && i != index)
            value_error("tensors must live on one device, got " + std::to_string(index) + " and " + std::to_string(i));
        index = i;
    }
    void take(const Tensor* t) {
        if (t) take(*t);
    }
    hipStream_t stream() const { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)index).stream(); }
};

// Elements between the rows of a page table (rows contiguous, not overlapping).
int64_t table_stride(const Tensor& t) {
    const int64_t B = t.size(0), width = t.size(1);
    if (width > 1 && t.stride(1) != 1) value_error("page_table rows must be contiguous");
    const int64_t stride = B > 1 ? t.stride(0) : width;
    if (stride < width) value_error("page_table rows must not overlap");
    return stride;
}

// The caches [pages, Hkv, page_size, D].
struct Cache {
    tq_dtype dt;
    int64_t pages, heads, page, D, stride;
};
Cache cache_of(const Tensor& k, const Tensor& v) {
    Cache c;
    if (k.dim() != 4 || (k.scalar_type() != at::kHalf && k.scalar_type() != at::kBFloat16))
        type_error("k_cache must be a 4-D float16 or bfloat16 tensor [pages, heads, page_size, D]");
    if (v.scalar_type() != k.scalar_type() || v.sizes() != k.sizes() || v.strides() != k.strides())
        value_error("k_cache and v_cache must be alike in shape, type and strides");
    c.dt = k.scalar_type() == at::kHalf ? TQ_F16 : TQ_BF16;
    c.pages = k.size(0);
    c.heads = k.size(1);
    c.page = k.size(2);
    c.D = k.size(3);
    const int64_t body = c.heads * c.page * c.D;
    c.stride = body;
    if (k.is_contiguous()) return c;
    int64_t want = 1;  // the strides inside a page
    for (int i = 3; i > 0; --i) {
        if (k.size(i) != 1 && k.stride(i) != want) value_error("the pages of a cache must be contiguous");
        want *= k.size(i);
    }
    if (c.pages > 1) c.stride = k.stride(0);
    if (c.stride < body) value_error("the pages of a cache must not overlap");
    return c;
}

// [T, heads, D] whose last dimension is contiguous.
struct Heads {
    const void* p = nullptr;
    int64_t n = 0, token = 0, head = 0;
};
Heads heads_of(const char* name, const Tensor& t, at::ScalarType type, int64_t T, int64_t D) {
    is(name, t, type, 3);
    if (t.size(0) != T || t.size(2) != D)
        value_error(std::string(name) + " must be [" + std::to_string(T) + ", heads, " + std::to_string(D) + "], got " + shape_of(t));
    if (D > 1 && t.stride(2) != 1) value_error("the heads of " + std::string(name) + " must be contiguous");
    // a stride over one token or one head leads nowhere and may be any number
    return Heads{t.data_ptr(), t.size(1), T > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
}

Tensor fresh(at::IntArrayRef sizes, const Tensor& like, at::ScalarType type) {
    return at::empty(sizes, like.options().dtype(type));
}

// A vector of n entries at an offset of a buffer's storage: several outputs of
// one allocation (an allocation costs 0.8 us, this 0.1).
Tensor part_of(const Tensor& buffer, int64_t bytes_in, at::ScalarType type, int64_t n) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buffer.storage()), buffer.key_set(),
                                                        c10::scalarTypeToTypeMeta(type));
    const int64_t step = 1;
    t.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(&n, 1), at::IntArrayRef(&step, 1),
                                                   bytes_in / (int64_t)c10::elementSize(type));
    return t;
}

// A call's status as Python sees it: 0, or what _lib._check raises from.
PyObject* with_status(tq_status st, PyObject* result) {
    if (st == TQ_OK) return result;
    Py_DECREF(result);
    return PyLong_FromLong((long)st);
}

template <class F>
tq_status call(F f) {  // other threads run while the launch may block
    tq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return st;
}

void count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) type_error("takes " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

// (ctx_lens, new_lens, page_table, free_pages, free_head, tokens, page_size, out)
PyObject* paged_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8);
    const Tensor &ctx = tensor("ctx_lens", a[0]), &fresh_lens = tensor("new_lens", a[1]), &table = tensor("page_table", a[2]),
                 &free = tensor("free_pages", a[3]), &head = tensor("free_head", a[4]);
    const int64_t tokens = whole("tokens", a[5]), page = whole("page_size", a[6]);
    const int32_t* pc = vector_of<int32_t>("ctx_lens", ctx);
    const int64_t B = ctx.size(0);
    const int32_t* pn = vector_of<int32_t>("new_lens", fresh_lens, B);
    is("page_table", table, at::kInt, 2);
    const int32_t* pf = vector_of<int32_t>("free_pages", free);
    const int32_t* ph = vector_of<int32_t>("free_head", head, 1);
    if (table.size(0) != B)
        value_error("page_table must have " + std::to_string(B) + " rows, got " + std::to_string(table.size(0)));
    if (tokens < 0) value_error("tokens must not be negative");
    const int64_t stride = table_stride(table);
    OneDevice dev;
    static const char* const names[5] = {"out.cu_q", "out.kv_lens", "out.positions", "out.slots", "out.state"};
    const int64_t sizes[5] = {B + 1, B, tokens, tokens, 2};
    Tensor out[5];
    void* p[5];
    const bool given = a[7] != Py_None;
    if (given) {
        if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 5) type_error("out must be a PagedPlan");
        for (int i = 0; i < 5; ++i) {
            out[i] = tensor(names[i], PyTuple_GET_ITEM(a[7], i));
            p[i] = vector(names[i], out[i], i == 3 ? at::kLong : at::kInt, sizes[i]);
        }
    }
    for (const Tensor* t : {&ctx, &fresh_lens, &table, &free, &head}) dev.take(*t);
    if (given) {
        for (const Tensor& t : out) dev.take(t);
    } else {  // the slots first: they are 8 bytes each
        const Tensor buffer = fresh({2 * B + 3 * tokens + 3}, ctx, at::kInt);
        int64_t at = 0;
        for (const int i : {3, 0, 1, 2, 4}) {
            const at::ScalarType type = i == 3 ? at::kLong : at::kInt;
            out[i] = part_of(buffer, at, type, sizes[i]);
            p[i] = out[i].data_ptr();
            at += sizes[i] * (int64_t)c10::elementSize(type);
        }
    }
    const hipStream_t s = dev.stream();
    const tq_status st = call([&] {
        return tq_paged_plan(pc, pn, static_cast<int32_t*>(table.data_ptr()), stride, pf, ph, B, table.size(1), free.size(0),
                             tokens, page, static_cast<int32_t*>(p[0]), static_cast<int32_t*>(p[1]),
                             static_cast<int32_t*>(p[2]), static_cast<int64_t*>(p[3]), static_cast<int32_t*>(p[4]), s);
    });
    PyObject* r;
    if (given) {
        Py_INCREF(a[7]);
        r = a[7];
    } else {
        r = PyTuple_New(5);
        if (!r) throw python_error();
        for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(out[i])));
    }
    return with_status(st, r);
    END_HANDLE_TH_ERRORS
}

// (q, k, v, k_cache, v_cache, slots, positions, rope, interleaved, out)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 10);
    const Tensor *q = optional("q", a[0]), *pos = optional("positions", a[6]), *rope = optional("rope", a[7]),
                 *given = optional("out", a[9]);
    const Tensor &k = tensor("k", a[1]), &v = tensor("v", a[2]), &kc = tensor("k_cache", a[3]), &vc = tensor("v_cache", a[4]),
                 &slots = tensor("slots", a[5]);
    const int inter = PyObject_IsTrue(a[8]);
    if (inter < 0) throw python_error();
    const Cache c = cache_of(kc, vc);
    const at::ScalarType type = kc.scalar_type();
    if (k.dim() != 3) type_error("k must be 3-D [T, heads, D], got " + std::to_string(k.dim()) + "-D");
    const int64_t T = k.size(0);
    const Heads hk = heads_of("k", k, type, T, c.D), hv = heads_of("v", v, type, T, c.D);
    if (hk.n != c.heads || hv.n != c.heads)
        value_error("k and v must have the cache's " + std::to_string(c.heads) + " heads, got " + std::to_string(hk.n) + " and " +
                    std::to_string(hv.n));
    Heads hq;
    if (q) hq = heads_of("q", *q, type, T, c.D);
    const int64_t* ps = vector_of<int64_t>("slots", slots, T);
    if (!rope != !pos) value_error("rope and positions come together");
    const float* pr = nullptr;
    const int32_t* pp = nullptr;
    int64_t rows = 0, rot = 0;
    if (rope) {
        is("rope", *rope, at::kFloat, 2);
        contiguous("rope", *rope);
        pr = static_cast<const float*>(rope->data_ptr());
        pp = vector_of<int32_t>("positions", *pos, T);
        rows = rope->size(0);
        rot = rope->size(1);
        if (rot > c.D || rot % 2)
            value_error("rope must have an even number of columns, at most " + std::to_string(c.D) + ", got " + std::to_string(rot));
    }
    if (given) {
        if (!q) value_error("out needs q");
        is("out", *given, type, 3);
        if (given->sizes() != at::IntArrayRef({T, hq.n, c.D})) value_error("out must have the shape of q, got " + shape_of(*given));
        contiguous("out", *given);
    }
    OneDevice dev;
    dev.take(q);
    for (const Tensor* t : {&k, &v, &kc, &vc, &slots, pos, rope, given}) dev.take(t);
    Tensor out;
    if (given) out = *given;
    else if (q) out = fresh({T, hq.n, c.D}, *q, type);
    void* po = q ? out.data_ptr() : nullptr;
    const hipStream_t s = dev.stream();
    const tq_status st = call([&] {
        return tq_kv_append(hq.p, hq.token, hq.head, hk.p, hk.token, hk.head, hv.p, hv.token, hv.head, c.dt, T, hq.n, c.heads, c.D,
                            kc.data_ptr(), vc.data_ptr(), c.pages, c.page, c.stride, ps, pp, pr, rows, rot, inter, po, s);
    });
    if (!q) Py_INCREF(Py_None);
    return with_status(st, q ? THPVariable_Wrap(std::move(out)) : Py_None);
    END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, page_table, cu_q, kv_lens, max_q, max_kv, scale, window, sinks, return_lse, out, workspace)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 14);
    const Tensor &q = tensor("q", a[0]), &kc = tensor("k_cache", a[1]), &vc = tensor("v_cache", a[2]),
                 &table = tensor("page_table", a[3]), &cu = tensor("cu_q", a[4]), &kv = tensor("kv_lens", a[5]);
    const int64_t max_q = whole("max_q", a[6]), max_kv = whole("max_kv", a[7]), window = whole("window", a[9]),
                  sinks = whole("sinks", a[10]);
    const int want_lse = PyObject_IsTrue(a[11]);
    if (want_lse < 0) throw python_error();
    const bool own_ws = PyUnicode_Check(a[13]);  // "auto"
    const Tensor *given = optional("out", a[12]), *ws = own_ws ? nullptr : optional("workspace", a[13]);
    const Cache c = cache_of(kc, vc);
    double scale = std::pow((double)c.D, -0.5);
    if (a[8] != Py_None) {
        scale = PyFloat_AsDouble(a[8]);
        if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    }
    if (q.dim() != 3) type_error("q must be 3-D [T, heads, D], got " + std::to_string(q.dim()) + "-D");
    const int64_t T = q.size(0);
    const Heads hq = heads_of("q", q, kc.scalar_type(), T, c.D);
    is("page_table", table, at::kInt, 2);
    const int64_t B = table.size(0), width = table.size(1);
    const int32_t* pc = vector_of<int32_t>("cu_q", cu, B + 1);
    const int32_t* pk = vector_of<int32_t>("kv_lens", kv, B);
    const int64_t tab = table_stride(table);
    if (given) {
        is("out", *given, q.scalar_type(), 3);
        if (given->sizes() != q.sizes()) value_error("out must have the shape of q, got " + shape_of(*given));
        contiguous("out", *given);
    }
    OneDevice dev;
    for (const Tensor* t : {&q, &kc, &vc, &table, &cu, &kv, given, ws}) dev.take(t);
    if (ws) contiguous("workspace", *ws);
    Tensor out = given ? *given : fresh({T, hq.n, c.D}, q, q.scalar_type());
    Tensor lse;
    if (want_lse) lse = fresh({T, hq.n}, q, at::kFloat);
    Tensor work;
    if (own_ws) {
        const size_t bytes = tq_paged_attention_workspace_bytes(T, hq.n, c.heads, c.D, B, max_q, max_kv, window, sinks);
        if (bytes) {
            work = fresh({(int64_t)bytes}, q, at::kByte);
            work.narrow(0, 0, TQ_WORKSPACE_FLAG_BYTES).zero_();
            ws = &work;
        }
    }
    const hipStream_t s = dev.stream();
    const tq_status st = call([&] {
        return tq_paged_attention(hq.p, hq.token, hq.head, c.dt, T, hq.n, c.heads, c.D, kc.data_ptr(),
                                  vc.data_ptr(), c.pages, c.page, c.stride, static_cast<const int32_t*>(table.data_ptr()), tab,
                                  width, pc, pk, B, max_q, max_kv, (float)scale, window, sinks, out.data_ptr(),
                                  want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, ws ? ws->data_ptr() : nullptr,
                                  ws ? ws->nbytes() : 0, s);
    });
    PyObject* r = THPVariable_Wrap(std::move(out));
    if (want_lse) {
        PyObject* both = PyTuple_New(2);
        if (!both) throw python_error();
        PyTuple_SET_ITEM(both, 0, r);
        PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(std::move(lse)));
        r = both;
    }
    return with_status(st, r);
    END_HANDLE_TH_ERRORS
}

// (logits, u, temperature, top_k, top_p, min_p, out)
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);
    const Tensor &x = tensor("logits", a[0]), &u = tensor("u", a[1]);
    const Tensor *t = optional("temperature", a[2]), *k = optional("top_k", a[3]), *p = optional("top_p", a[4]),
                 *m = optional("min_p", a[5]);
    if (x.dim() != 2) type_error("logits must be 2-D [B, V], got " + std::to_string(x.dim()) + "-D");
    tq_dtype dt;
    switch (x.scalar_type()) {
        case at::kHalf: dt = TQ_F16; break;
        case at::kBFloat16: dt = TQ_BF16; break;
        case at::kFloat: dt = TQ_F32; break;
        default: type_error("logits must be float16, bfloat16 or float32, got " + std::string(c10::toString(x.scalar_type())));
    }
    const int64_t B = x.size(0), V = x.size(1);
    if (V > 1 && x.stride(1) != 1) value_error("the rows of logits must be contiguous");
    const int64_t stride = B > 1 ? x.stride(0) : V;
    if (stride < V) value_error("the rows of logits must not overlap");
    const float* pu = vector_of<float>("u", u, B);
    const float* pt = t ? vector_of<float>("temperature", *t, B) : nullptr;
    const int32_t* pk = k ? vector_of<int32_t>("top_k", *k, B) : nullptr;
    const float* pp = p ? vector_of<float>("top_p", *p, B) : nullptr;
    const float* pm = m ? vector_of<float>("min_p", *m, B) : nullptr;
    const bool given = a[6] != Py_None;
    Tensor tokens, logprobs;
    if (given) {
        if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 2) type_error("out must be (tokens, logprobs)");
        tokens = tensor("tokens", PyTuple_GET_ITEM(a[6], 0));
        logprobs = tensor("logprobs", PyTuple_GET_ITEM(a[6], 1));
        vector("tokens", tokens, at::kInt, B);
        vector("logprobs", logprobs, at::kFloat, B);
    }
    OneDevice dev;
    for (const Tensor* z : {&x, &u, t, k, p, m}) dev.take(z);
    if (given) {
        dev.take(tokens);
        dev.take(logprobs);
    } else {
        tokens = fresh({B}, u, at::kInt);
        logprobs = fresh({B}, u, at::kFloat);
    }
    const hipStream_t s = dev.stream();
    const tq_status st = call([&] {
        return tq_sample(x.data_ptr(), dt, B, V, stride, pu, pt, pk, pp, pm, static_cast<int32_t*>(tokens.data_ptr()),
                         static_cast<float*>(logprobs.data_ptr()), s);
    });
    PyObject* r = PyTuple_New(2);
    if (!r) throw python_error();
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(tokens)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(logprobs)));
    return with_status(st, r);
    END_HANDLE_TH_ERRORS
}

// ---- experts and adapters

tq_dtype half_type(const char* name, const Tensor& t) {
    if (t.scalar_type() == at::kHalf) return TQ_F16;
    if (t.scalar_type() == at::kBFloat16) return TQ_BF16;
    type_error(std::string(name) + " must be float16 or bfloat16, got " + c10::toString(t.scalar_type()));
}
// [T, n] with contiguous rows of the type; -> elements between rows.
int64_t rows_of(const char* name, const Tensor& t, at::ScalarType type, int64_t T, int64_t n) {
    is(name, t, type, 2);
    if ((T >= 0 && t.size(0) != T) || (n >= 0 && t.size(1) != n))
        value_error(std::string(name) + " must be [" + (T >= 0 ? std::to_string(T) : "rows") + ", " +
                    (n >= 0 ? std::to_string(n) : "columns") + "], got " + shape_of(t));
    const int64_t width = t.size(1);
    if (width > 1 && t.stride(1) != 1) value_error("the rows of " + std::string(name) + " must be contiguous");
    const int64_t stride = t.size(0) > 1 ? t.stride(0) : width;
    if (stride < width) value_error("the rows of " + std::string(name) + " must not overlap");
    return stride;
}
void whole_of(const char* name, const Tensor& t, at::ScalarType type, at::IntArrayRef sizes) {
    is(name, t, type, (int64_t)sizes.size());
    if (t.sizes() != sizes) {
        std::string want;
        for (int64_t s : sizes) want += (want.empty() ? "" : ", ") + std::to_string(s);
        value_error(std::string(name) + " must be (" + want + "), got " + shape_of(t));
    }
    contiguous(name, t);
}

// (logits, top_k, renormalize, out, workspace)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 5);
    const Tensor& x = tensor("logits", a[0]);
    const int64_t k = whole("top_k", a[1]);
    const int renorm = PyObject_IsTrue(a[2]);
    if (renorm < 0) throw python_error();
    if (x.dim() != 2) type_error("logits must be 2-D [T, E], got " + std::to_string(x.dim()) + "-D");
    tq_dtype dt;
    switch (x.scalar_type()) {
        case at::kHalf: dt = TQ_F16; break;
        case at::kBFloat16: dt = TQ_BF16; break;
        case at::kFloat: dt = TQ_F32; break;
        default: type_error("logits must be float16, bfloat16 or float32, got " + std::string(c10::toString(x.scalar_type())));
    }
    const int64_t T = x.size(0), E = x.size(1), stride = rows_of("logits", x, x.scalar_type(), -1, -1);
    // the library's own limits, before anything is allocated by them
    if (T < 1 || E < 1 || E > 1024 || k < 1 || k > E || k > 64 || T > 0x7FFFFFFF / k) return PyLong_FromLong(TQ_ERR_SHAPE);
    const size_t need = tq_moe_route_workspace_bytes(T, E, k);
    static const char* const names[5] = {"out.experts", "out.weights", "out.offsets", "out.rows", "out.places"};
    static const at::ScalarType types[5] = {at::kInt, at::kFloat, at::kInt, at::kInt, at::kInt};
    const bool own_ws = PyUnicode_Check(a[4]);  // "auto"
    const Tensor* ws = own_ws ? nullptr : optional("workspace", a[4]);
    OneDevice dev;
    dev.take(x);
    Tensor out[5];
    const bool given = a[3] != Py_None;
    if (given) {
        if (!PyTuple_Check(a[3]) || PyTuple_GET_SIZE(a[3]) != 5) type_error("out must be a MoeRoute");
        for (int i = 0; i < 5; ++i) {
            out[i] = tensor(names[i], PyTuple_GET_ITEM(a[3], i));
            if (i == 2) vector(names[i], out[i], types[i], E + 1);
            else if (i == 3) vector(names[i], out[i], types[i], T * k);
            else whole_of(names[i], out[i], types[i], {T, k});
            dev.take(out[i]);
        }
    }
    if (ws) {
        contiguous("workspace", *ws);
        dev.take(*ws);
    }
    const c10::DeviceGuard guard(x.device());
    Tensor buffer;
    void* pw = ws ? ws->data_ptr() : nullptr;
    size_t ws_bytes = ws ? ws->nbytes() : 0;
    const int64_t extra = own_ws ? (int64_t)need / 4 : 0;
    if (!given || extra) buffer = fresh({(given ? 0 : 4 * T * k + E + 1) + extra}, x, at::kInt);
    if (!given) {
        int64_t at = 0;
        for (int i = 0; i < 5; ++i) {
            const int64_t len = i == 2 ? E + 1 : T * k;
            out[i] = part_of(buffer, 4 * at, types[i], len);
            if (i != 2 && i != 3) {
                const int64_t sizes[2] = {T, k}, steps[2] = {k, 1};
                out[i].unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(sizes, 2), at::IntArrayRef(steps, 2), at);
            }
            at += len;
        }
    }
    if (own_ws && need) {
        pw = static_cast<int32_t*>(buffer.data_ptr()) + (buffer.numel() - extra);
        ws_bytes = need;
    }
    const hipStream_t s = dev.stream();
    const tq_status st = call([&] {
        return tq_moe_route(x.data_ptr(), dt, T, E, stride, k, renorm, static_cast<int32_t*>(out[0].data_ptr()),
                            static_cast<float*>(out[1].data_ptr()), static_cast<int32_t*>(out[2].data_ptr()),
                            static_cast<int32_t*>(out[3].data_ptr()), static_cast<int32_t*>(out[4].data_ptr()), pw, ws_bytes, s);
    });
    PyObject* r;
    if (given) {
        Py_INCREF(a[3]);
        r = a[3];
    } else {
        r = PyTuple_New(5);
        if (!r) throw python_error();
        for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(out[i])));
    }
    return with_status(st, r);
    END_HANDLE_TH_ERRORS
}

// (A, codes or qweight, scale, zeros, offsets, rows, bias, gated, out, whether they are W4A16's)
PyObject* moe_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 10);
    const Tensor &A = tensor("A", a[0]), &w = tensor("weights", a[1]), &scale = tensor("scale", a[2]),
                 &offsets = tensor("offsets", a[4]);
    const Tensor *zeros = optional("zeros", a[3]), *rows = optional("rows", a[5]), *bias = optional("bias", a[6]),
                 *given = optional("out", a[8]);
    const int gated = PyObject_IsTrue(a[7]);
    if (gated < 0) throw python_error();
    if (A.dim() != 2) type_error("A must be 2-D [T, K], got " + std::to_string(A.dim()) + "-D");
    const tq_dtype dt = half_type("A", A);
    contiguous("A", A);
    const int64_t T = A.size(0), K = A.size(1);
    const bool w4 = a[9] == Py_True;
    if (w.dim() != 3 || w.scalar_type() != (w4 ? at::kInt : at::kByte))
        type_error((w4 ? "qweight must be a 3-D int32 tensor [E, N, K / 8], got " : "codes must be a 3-D uint8 tensor [E, N, K / 4], got ") +
                   kind_of(w));
    const int64_t E = w.size(0), N = w.size(1), G = K / 128;
    if (K % (w4 ? 128 : 64) != 0) value_error("K must be a multiple of " + std::to_string(w4 ? 128 : 64) + ", got " + std::to_string(K));
    whole_of(w4 ? "qweight" : "codes", w, w.scalar_type(), {E, N, w4 ? K / 8 : K / 4});
    if (w4) whole_of("scales", scale, at::kHalf, {E, N, G});
    else whole_of("scale", scale, at::kHalf, {E, N});
    if (zeros) whole_of("zeros", *zeros, at::kByte, {E, N, G});
    vector("offsets", offsets, at::kInt, E + 1);
    int64_t P = T;
    if (rows) {
        vector("rows", *rows, at::kInt);
        P = rows->size(0);
        if (T == 0 ? P != 0 : P % T != 0)
            value_error("rows must have a multiple of A's " + std::to_string(T) + " rows, got " + std::to_string(P));
    }
    if (bias) whole_of("bias", *bias, A.scalar_type(), {E, N});
    if (gated && N % 2) value_error("a gated product needs an even number of weight rows, got " + std::to_string(N));
    const int64_t width = gated ? N / 2 : N;
    if (given) whole_of("out", *given, A.scalar_type(), {P, width});
    OneDevice dev;
    for (const Tensor* t : {&A, &w, &scale, &offsets, zeros, rows, bias, given}) dev.take(t);
    const c10::DeviceGuard guard(A.device());
    Tensor out = given ? *given : fresh({P, width}, A, A.scalar_type());
    const hipStream_t s = dev.stream();
    const int32_t *po = static_cast<const int32_t*>(offsets.data_ptr()),
                  *pr = rows ? static_cast<const int32_t*>(rows->data_ptr()) : nullptr;
    const uint16_t* ps = static_cast<const uint16_t*>(scale.data_ptr());
    const void* pb = bias ? bias->data_ptr() : nullptr;
    const tq_status st = call([&] {
        if (w4)
            return w4a16_moe_gemm(A.data_ptr(), dt, T, P, E, N, K, static_cast<const int32_t*>(w.data_ptr()), ps,
                                  zeros ? static_cast<const uint8_t*>(zeros->data_ptr()) : nullptr, 128, po, pr, pb, gated,
                                  out.data_ptr(), s);
        return tq_moe_gemm(A.data_ptr(), dt, T, P, E, N, K, static_cast<const uint8_t*>(w.data_ptr()), ps, po, pr, pb, gated,
                           out.data_ptr(), s);
    });
    return with_status(st, THPVariable_Wrap(std::move(out)));
    END_HANDLE_TH_ERRORS
}

// (y, places, weights, add, out)
PyObject* moe_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 5);
    const Tensor &y = tensor("y", a[0]), &places = tensor("places", a[1]), &weights = tensor("weights", a[2]);
    const Tensor *add = optional("add", a[3]), *given = optional("out", a[4]);
    if (y.dim() != 2) type_error("y must be 2-D [P, N], got " + std::to_string(y.dim()) + "-D");
    const tq_dtype dt = half_type("y", y);
    contiguous("y", y);
    is("places", places, at::kInt, 2);
    contiguous("places", places);
    const int64_t P = y.size(0), N = y.size(1), T = places.size(0), k = places.size(1);
    whole_of("weights", weights, at::kFloat, {T, k});
    const int64_t stride = add ? rows_of("add", *add, y.scalar_type(), T, N) : 0;
    if (given) whole_of("out", *given, y.scalar_type(), {T, N});
    OneDevice dev;
    for (const Tensor* t : {&y, &places, &weights, add, given}) dev.take(t);
    const c10::DeviceGuard guard(y.device());
    Tensor out = given ? *given : fresh({T, N}, y, y.scalar_type());
    const hipStream_t s = dev.stream();
    const tq_status st = call([&] {
        return tq_moe_combine(y.data_ptr(), dt, T, P, N, k, static_cast<const int32_t*>(places.data_ptr()),
                              static_cast<const float*>(weights.data_ptr()), add ? add->data_ptr() : nullptr, stride,
                              out.data_ptr(), s);
    });
    return with_status(st, THPVariable_Wrap(std::move(out)));
    END_HANDLE_TH_ERRORS
}

// The call has no backward pass: a tensor that wants a gradient would lose it.
void no_gradient(const char* name, const Tensor* t) {
    if (t && t->requires_grad() && at::GradMode::is_enabled())
        value_error(std::string(name) + " requires a gradient, but tq_lora goes forward only: detach it or call under torch.no_grad()");
}

// (x, base, A, B, ids, scale, out)
PyObject* lora(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);
    const Tensor &x = tensor("x", a[0]), &base = tensor("base", a[1]), &A = tensor("A", a[2]), &B = tensor("B", a[3]),
                 &ids = tensor("ids", a[4]);
    const Tensor *scale = optional("scale", a[5]), *given = optional("out", a[6]);
    no_gradient("x", &x);
    no_gradient("base", &base);
    no_gradient("A", &A);
    no_gradient("B", &B);
    no_gradient("scale", scale);
    no_gradient("out", given);
    if (x.dim() != 2) type_error("x must be 2-D [T, K], got " + std::to_string(x.dim()) + "-D");
    const tq_dtype dt = half_type("x", x);
    const at::ScalarType type = x.scalar_type();
    const int64_t T = x.size(0), K = x.size(1), xs = rows_of("x", x, type, T, K);
    const int64_t bs = rows_of("base", base, type, T, -1), N = base.size(1);
    if (A.dim() != 3) type_error("A must be 3-D [L, rank, K], got " + std::to_string(A.dim()) + "-D");
    const int64_t L = A.size(0), r = A.size(1);
    whole_of("A", A, type, {L, r, K});
    whole_of("B", B, type, {L, N, r});
    vector("ids", ids, at::kInt, T);
    if (scale) vector("scale", *scale, at::kFloat, L);
    const int64_t os = given ? rows_of("out", *given, type, T, N) : N;
    OneDevice dev;
    for (const Tensor* t : {&x, &base, &A, &B, &ids, scale, given}) dev.take(t);
    const c10::DeviceGuard guard(x.device());
    Tensor out = given ? *given : fresh({T, N}, x, type);
    const hipStream_t s = dev.stream();
    const tq_status st = call([&] {
        return tq_lora(x.data_ptr(), xs, base.data_ptr(), bs, dt, T, K, N, L, r, A.data_ptr(), B.data_ptr(),
                       static_cast<const int32_t*>(ids.data_ptr()), scale ? static_cast<const float*>(scale->data_ptr()) : nullptr,
                       out.data_ptr(), os, s);
    });
    return with_status(st, THPVariable_Wrap(std::move(out)));
    END_HANDLE_TH_ERRORS
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(paged_plan), ENTRY(kv_append), ENTRY(paged_attention), ENTRY(sample),
                         ENTRY(moe_route), ENTRY(moe_gemm), ENTRY(moe_combine), ENTRY(lora), {nullptr, nullptr, 0, nullptr}};
#undef ENTRY

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__serving() { return PyModule_Create(&module); }
