// Compiled half of the Python binding for the operators around the products
// (norm, cache, attention, log probabilities): argument checks, outputs and
// the C call of qmm.h in one step.  A decode step makes these calls for every
// token and layer on a few rows, where the GPU needs 2 to 8 us and the same
// work in Python took 9 to 18.
//
// Functions take positional arguments only (the Python functions in
// __init__.py give the names, defaults and documentation); None stands for an
// output that is made here.  TypeError and ValueError as the Python half
// raises them, QmmError for a status.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <optional>
#include <string>
#include <vector>

#include "../../include/qmm.h"

namespace {

PyObject *g_error = nullptr;  // QmmError

[[noreturn]] void fail(PyObject *type, const char *format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(type, format, args);
    va_end(args);
    throw python_error();
}

void check_status(qmm_status status, const char *where) {
    if (status == QMM_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "is", (int)status, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

std::string text(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}

// A CUDA tensor of this type.
const at::Tensor &tensor(PyObject *o, at::ScalarType type, const char *name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor (there is no CPU path)", name);
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, "%s must have dtype %s, got %s", name, c10::toString(type),
                               c10::toString(t.scalar_type()));
    return t;
}

void check_shape(const at::Tensor &t, at::IntArrayRef shape, const char *name) {
    if (t.sizes() != shape)
        fail(PyExc_ValueError, "%s must have shape %s, got %s", name, text(shape).c_str(),
                                text(t.sizes()).c_str());
}

void check_dim(const at::Tensor &t, int64_t dim, const char *name) {
    if (t.dim() != dim)
        fail(PyExc_ValueError, "%s must have %d dimensions, got %d", name, (int)dim, (int)t.dim());
}

template <typename T>
T *plane(const at::Tensor &t, at::IntArrayRef shape, const char *name) {
    check_shape(t, shape, name);
    if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
    return static_cast<T *>(t.data_ptr());
}

template <typename T>
T *plane(PyObject *o, at::ScalarType type, at::IntArrayRef shape, const char *name) {
    return plane<T>(tensor(o, type, name), shape, name);
}

// A matrix whose rows are contiguous and do not overlap (one row may be given
// as a vector where `rows` is 1).
struct Rows {
    float *p;
    int64_t ld;
};
Rows rows(const at::Tensor &t, int64_t m, int64_t k, const char *name) {
    if (t.dim() == 1 && m == 1 && t.size(0) == k) {
        if (k > 1 && t.stride(0) != 1) fail(PyExc_ValueError, "%s must have contiguous rows", name);
        return {static_cast<float *>(t.data_ptr()), k};
    }
    check_shape(t, {m, k}, name);
    const int64_t ld = m > 1 ? t.stride(0) : k;
    if ((k > 1 && t.stride(1) != 1) || ld < k) fail(PyExc_ValueError, "%s must have contiguous rows", name);
    return {static_cast<float *>(t.data_ptr()), ld};
}
Rows rows(PyObject *o, int64_t m, int64_t k, const char *name) {
    return rows(tensor(o, at::kFloat, name), m, k, name);
}

// An output: the given tensor, checked, or a new one beside `like`.
at::Tensor out(PyObject *o, at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like,
               const char *name) {
    if (o == Py_None) return at::empty(shape, like.options().dtype(type));
    const at::Tensor &t = tensor(o, type, name);
    plane<void>(t, shape, name);
    return t;
}

// Outputs of one call that share an allocation, each on 64 bytes: an
// allocation costs about 0.4 us of a call's 5 to 7.  Who keeps one of them
// keeps all, so calls with more bytes than kMost give each its own.
struct Shared {
    static constexpr int64_t kMost = 1 << 18;
    at::TensorOptions options;
    at::Tensor buffer;  // undefined: each its own
    int64_t used = 0;
    static int64_t bytes(int64_t count, int64_t size) { return (count * size + 63) & ~(int64_t)63; }
    Shared(const at::Tensor &like, int64_t bytes) : options(like.options()) {
        if (bytes <= kMost) buffer = at::empty({bytes}, options.dtype(at::kByte));
    }
    at::Tensor take(at::IntArrayRef shape, at::ScalarType type) {
        if (!buffer.defined()) return at::empty(shape, options.dtype(type));
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
            c10::Storage(buffer.storage()), buffer.key_set(), c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_storage_offset(used / (int64_t)c10::elementSize(type));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
        used += bytes(t.numel(), (int64_t)c10::elementSize(type));
        return t;
    }
};

int64_t whole(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

void *stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

uint16_t *bits(const at::Tensor &t) { return static_cast<uint16_t *>(t.data_ptr()); }

// Steals nothing, returns a new tuple of tensors (undefined ones as None).
PyObject *tuple(std::initializer_list<at::Tensor> list) {
    PyObject *r = PyTuple_New((Py_ssize_t)list.size());
    if (!r) throw python_error();
    Py_ssize_t i = 0;
    for (const at::Tensor &t : list)
        PyTuple_SET_ITEM(r, i++, t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None));
    return r;
}

void want(Py_ssize_t got, Py_ssize_t n) {
    if (got != n) fail(PyExc_TypeError, "%d arguments are wanted, got %d", (int)n, (int)got);
}

// x [m, k] or [k]; the sum goes to h where it is given or there is a residual.
struct Norm {
    int64_t m, k;
    at::Tensor x, h;
    std::optional<Shared> shared;  // of the outputs that are made here
    Rows xr, rr{nullptr, 0}, hr{nullptr, 0};
    float *w, eps;
};
// a: x, weight, eps, residual, h, then `outputs` more: the codes and, with so
// many bytes for a block of 32 and for a row, the others.
Norm norm_args(PyObject *const *a, int outputs, int64_t per_block, int64_t per_row) {
    Norm n;
    n.x = tensor(a[0], at::kFloat, "x");
    if (n.x.dim() == 1) n.x = n.x.unsqueeze(0);
    check_dim(n.x, 2, "x");
    n.m = n.x.size(0), n.k = n.x.size(1);
    n.xr = rows(n.x, n.m, n.k, "x");
    n.w = plane<float>(a[1], at::kFloat, {n.k}, "weight");
    n.eps = (float)number(a[2]);
    if (a[3] != Py_None) n.rr = rows(a[3], n.m, n.k, "residual");
    bool made = true;
    for (int i = 0; i < outputs; ++i) made &= a[5 + i] == Py_None;
    const bool with_sum = made && a[4] == Py_None && n.rr.p;
    if (made)
        n.shared.emplace(n.x, (with_sum ? Shared::bytes(n.m * n.k, 4) : 0) +
                                  n.m * (n.k + n.k / 32 * per_block + per_row) + 64 * outputs);
    if (a[4] != Py_None) {
        n.h = tensor(a[4], at::kFloat, "h");
        n.hr = rows(n.h, n.m, n.k, "h");
        if (n.h.dim() == 1) n.h = n.h.unsqueeze(0);
    } else if (n.rr.p) {
        n.h = with_sum ? n.shared->take({n.m, n.k}, at::kFloat) : at::empty({n.m, n.k}, n.x.options());
        n.hr = {static_cast<float *>(n.h.data_ptr()), n.k};
    } else {
        n.h = n.x;
    }
    return n;
}

PyObject *rms_norm_q8_0(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    want(count, 8);
    Norm n = norm_args(a, 2, 2, 0);
    at::Tensor aq, ad;
    if (n.shared) {
        aq = n.shared->take({n.m, n.k}, at::kChar);
        ad = n.shared->take({n.m, n.k / 32}, at::kHalf);
    } else {
        aq = out(a[5], {n.m, n.k}, at::kChar, n.x, "aq");
        ad = out(a[6], {n.m, n.k / 32}, at::kHalf, n.x, "ad");
    }
    check_status(qmm_rms_norm_q8_0(n.xr.p, n.xr.ld, n.rr.p, n.rr.ld, n.w, n.eps, n.hr.p, n.hr.ld,
                                   static_cast<int8_t *>(aq.data_ptr()), bits(ad), n.m, n.k,
                                   (int)whole(a[7]), stream()),
                 "qmm_rms_norm_q8_0");
    return tuple({aq, ad, n.h});
    END_HANDLE_TH_ERRORS
}

PyObject *rms_norm_bitnet(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    want(count, 9);
    Norm n = norm_args(a, 3, 0, 4 + 4);
    at::Tensor aq, scale, sum;
    if (n.shared) {
        aq = n.shared->take({n.m, n.k}, at::kChar);
        scale = n.shared->take({n.m}, at::kFloat);
        sum = n.shared->take({n.m}, at::kInt);
    } else {
        aq = out(a[5], {n.m, n.k}, at::kChar, n.x, "aq");
        scale = out(a[6], {n.m}, at::kFloat, n.x, "act_scale");
        sum = out(a[7], {n.m}, at::kInt, n.x, "act_sum");
    }
    check_status(qmm_rms_norm_bitnet(n.xr.p, n.xr.ld, n.rr.p, n.rr.ld, n.w, n.eps, n.hr.p, n.hr.ld,
                                     static_cast<int8_t *>(aq.data_ptr()),
                                     static_cast<float *>(scale.data_ptr()),
                                     static_cast<int32_t *>(sum.data_ptr()), n.m, n.k,
                                     (int)whole(a[8]), stream()),
                 "qmm_rms_norm_bitnet");
    return tuple({aq, scale, sum, n.h});
    END_HANDLE_TH_ERRORS
}

// The planes of a cache: keys, values (f16) or codes and scales of each (Q8_0).
struct Cache {
    int64_t pages, heads, page_size, d;
    void *k, *v;
    uint16_t *kd = nullptr, *vd = nullptr;
};
Cache cache_args(PyObject *const *a, bool q8) {
    const at::ScalarType type = q8 ? at::kChar : at::kHalf;
    const at::Tensor &k = tensor(a[0], type, q8 ? "kq" : "kc");
    check_dim(k, 4, q8 ? "kq" : "kc");
    Cache c{k.size(0), k.size(1), k.size(2), k.size(3), nullptr, nullptr};
    c.k = plane<void>(k, k.sizes(), q8 ? "kq" : "kc");
    c.v = plane<void>(a[q8 ? 2 : 1], type, k.sizes(), q8 ? "vq" : "vc");
    if (q8) {
        const int64_t scales[4] = {c.pages, c.heads, c.page_size, c.d / 32};
        c.kd = plane<uint16_t>(a[1], at::kHalf, scales, "kd");
        c.vd = plane<uint16_t>(a[3], at::kHalf, scales, "vd");
    }
    return c;
}

// k, v, slots, then the planes
template <bool Q8>
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    want(count, Q8 ? 7 : 5);
    const Cache c = cache_args(a + 3, Q8);
    const at::Tensor &k = tensor(a[0], at::kFloat, "k");
    check_dim(k, 2, "k");
    const int64_t m = k.size(0);
    const Rows kr = rows(k, m, c.heads * c.d, "k"), vr = rows(a[1], m, c.heads * c.d, "v");
    const auto *slots = plane<int64_t>(a[2], at::kLong, {m}, "slots");
    if constexpr (Q8)
        check_status(qmm_kv_append_q8_0(kr.p, kr.ld, vr.p, vr.ld, slots, static_cast<int8_t *>(c.k), c.kd,
                                        static_cast<int8_t *>(c.v), c.vd, m, c.heads, c.d, c.pages,
                                        c.page_size, stream()),
                     "qmm_kv_append_q8_0");
    else
        check_status(qmm_kv_append_f16(kr.p, kr.ld, vr.p, vr.ld, slots, static_cast<uint16_t *>(c.k),
                                       static_cast<uint16_t *>(c.v), m, c.heads, c.d, c.pages,
                                       c.page_size, stream()),
                     "qmm_kv_append_f16");
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// q, the planes, table, lens, max_len, scale, window, out, lse, workspace
template <bool Q8>
PyObject *paged_attention(PyObject *, PyObject *const *args, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    constexpr int kPlanes = Q8 ? 4 : 2;
    want(count, 9 + kPlanes);
    const Cache c = cache_args(args + 1, Q8);
    PyObject *const *a = args + 1 + kPlanes;
    const at::Tensor &q = tensor(args[0], at::kFloat, "q");
    check_dim(q, 2, "q");
    const int64_t batch = q.size(0), width = q.size(1);
    if (c.d <= 0 || width % c.d != 0)
        fail(PyExc_ValueError, "q must have a multiple of %lld columns, got %lld", (long long)c.d,
                                (long long)width);
    const int64_t heads = width / c.d;
    const Rows qr = rows(q, batch, width, "q");
    const at::Tensor &table = tensor(a[0], at::kInt, "table");
    check_dim(table, 2, "table");
    const int64_t max_pages = table.size(1);
    const auto *tp = plane<int32_t>(table, {batch, max_pages}, "table");
    const auto *lp = plane<int32_t>(a[1], at::kInt, {batch}, "lens");
    const int64_t max_len = a[2] == Py_None ? max_pages * c.page_size : whole(a[2]);
    const float scale = (float)(a[3] == Py_None ? 1.0 / std::sqrt((double)c.d) : number(a[3]));
    const int64_t window = whole(a[4]);
    at::Tensor o, lse;
    Rows orow;
    if (a[5] == Py_None && a[6] == Py_None) {
        Shared shared(q, Shared::bytes(batch * width, 4) + Shared::bytes(batch * heads, 4));
        o = shared.take({batch, width}, at::kFloat);
        lse = shared.take({batch, heads}, at::kFloat);
        orow = {static_cast<float *>(o.data_ptr()), width};
    } else if (a[5] == Py_None) {
        o = at::empty({batch, width}, q.options());
        orow = {static_cast<float *>(o.data_ptr()), width};
    } else {
        o = tensor(a[5], at::kFloat, "out");
        orow = rows(o, batch, width, "out");
    }
    if (!lse.defined()) lse = out(a[6], {batch, heads}, at::kFloat, q, "lse");
    at::Tensor ws;
    if (a[7] != Py_None) {
        ws = tensor(a[7], at::kByte, "workspace");
        plane<void>(ws, ws.sizes(), "workspace");
    } else {
        const size_t need = qmm_paged_attention_workspace_bytes(batch, heads, c.heads, c.d, max_len);
        // a shape that the query refuses is refused by the call, with its status
        if (need && need != SIZE_MAX) ws = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
    }
    void *wp = ws.defined() ? ws.data_ptr() : nullptr;
    const size_t wb = ws.defined() ? (size_t)ws.numel() : 0;
    auto *lsep = static_cast<float *>(lse.data_ptr());
    if constexpr (Q8)
        check_status(qmm_paged_attention_q8_0(qr.p, qr.ld, static_cast<int8_t *>(c.k), c.kd,
                                              static_cast<int8_t *>(c.v), c.vd, tp, lp, orow.p, orow.ld,
                                              lsep, batch, heads, c.heads, c.d, c.pages, c.page_size,
                                              max_pages, max_len, window, scale, wp, wb, stream()),
                     "qmm_paged_attention_q8_0");
    else
        check_status(qmm_paged_attention_f16(qr.p, qr.ld, static_cast<uint16_t *>(c.k),
                                             static_cast<uint16_t *>(c.v), tp, lp, orow.p, orow.ld, lsep,
                                             batch, heads, c.heads, c.d, c.pages, c.page_size, max_pages,
                                             max_len, window, scale, wp, wb, stream()),
                     "qmm_paged_attention_f16");
    return tuple({o, lse});
    END_HANDLE_TH_ERRORS
}

// logits, tokens, top_k
PyObject *log_probs(PyObject *, PyObject *const *a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    want(count, 3);
    const at::Tensor &x = tensor(a[0], at::kFloat, "logits");
    if (x.dim() != 1) check_dim(x, 2, "logits");
    const int64_t m = x.dim() == 1 ? 1 : x.size(0), n = x.size(-1), top_k = whole(a[2]);
    const Rows xr = rows(x, m, n, "logits");
    if (top_k < 0 || top_k > QMM_TOP_MAX)
        fail(PyExc_ValueError, "top_k must be 0 .. %d, got %lld", QMM_TOP_MAX, (long long)top_k);
    const int32_t *words = nullptr;
    int64_t given = 0;
    const at::Tensor *tokens = nullptr;
    if (a[1] != Py_None) {
        tokens = &tensor(a[1], at::kInt, "tokens");
        if (tokens->dim() != 1) check_dim(*tokens, 2, "tokens");
        given = tokens->dim() == 2 ? tokens->size(1) : 1;
        words = tokens->dim() == 2 ? plane<int32_t>(*tokens, {m, given}, "tokens")
                                   : plane<int32_t>(*tokens, {m}, "tokens");
    }
    Shared shared(x, Shared::bytes(m, 4) + 2 * Shared::bytes(m * top_k, 4) + Shared::bytes(m * given, 4));
    const at::Tensor entropy = shared.take({m}, at::kFloat);
    const at::Tensor ids = shared.take({m, top_k}, at::kInt);
    const at::Tensor top = shared.take({m, top_k}, at::kFloat);
    at::Tensor lp;
    if (tokens) lp = shared.take(tokens->sizes(), at::kFloat);
    check_status(qmm_log_probs(xr.p, xr.ld, m, n, words, given,
                               lp.defined() ? static_cast<float *>(lp.data_ptr()) : nullptr,
                               static_cast<float *>(entropy.data_ptr()), static_cast<int32_t *>(ids.data_ptr()),
                               static_cast<float *>(top.data_ptr()), top_k, stream()),
                 "qmm_log_probs");
    return tuple({lp, entropy, ids, top});
    END_HANDLE_TH_ERRORS
}

PyObject *init(PyObject *, PyObject *error) {
    Py_XSETREF(g_error, Py_NewRef(error));
    Py_RETURN_NONE;
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {{"init", init, METH_O, nullptr},
                          FAST("rms_norm_q8_0", rms_norm_q8_0),
                          FAST("rms_norm_bitnet", rms_norm_bitnet),
                          FAST("kv_append_f16", kv_append<false>),
                          FAST("kv_append_q8_0", kv_append<true>),
                          FAST("paged_attention_f16", paged_attention<false>),
                          FAST("paged_attention_q8_0", paged_attention<true>),
                          FAST("log_probs", log_probs),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_qmm_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmm_torch() { return PyModule_Create(&kModule); }
