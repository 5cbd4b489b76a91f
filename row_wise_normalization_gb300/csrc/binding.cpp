// binding.cpp -- the common case of the head operators' calls, marshalled in C++.
//
// A decoding step waits for the host side of these calls: on GB300's host cores the checks, lookups
// and allocations of one call in Python take 13 to 17 us (the gradient's 30), here 4 to 5 (10), its
// kernel takes 2 to 4. Each function here takes the arguments of the Python function of its name
// (tokens.py), and where they are plain (torch tensors on the current device, of fitting shapes and
// types, outputs to be allocated, the current stream) it allocates the outputs, calls the library and
// returns them as a tuple. In every other case (outputs or a stream given among them) it returns None
// and has done nothing: the Python function then goes its own way, and says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "rownorm.h"

namespace {

// The library's entry points, given by `use`.
struct Entries {
    decltype(&::qk_rope_fwd) qk_rope_fwd;
    decltype(&::qk_rope_bwd) qk_rope_bwd;
    decltype(&::qk_rope_bwd_workspace_size) qk_rope_bwd_workspace_size;
    decltype(&::kv_append) kv_append;
    decltype(&::kv_gather) kv_gather;
    decltype(&::kv_slots) kv_slots;
} C;

using Tensor = at::Tensor;
using Ref = const Tensor*;       // nullptr: None

// An argument that is not plain.
struct NotPlain {};
void need(bool yes) {
    if (!yes) throw NotPlain{};
}

Ref tensor(PyObject* o) {
    if (o == Py_None) return nullptr;
    need(THPVariable_CheckExact(o));
    return &THPVariable_Unpack(o);
}
Ref given(PyObject* o) {
    const Ref t = tensor(o);
    need(t != nullptr);
    return t;
}
bool truth(PyObject* o) {
    need(o == Py_True || o == Py_False);
    return o == Py_True;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw NotPlain{};
    }
    return v;
}
int64_t whole(PyObject* o) {
    need(PyLong_CheckExact(o));
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw NotPlain{};
    }
    return v;
}

int value_code(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return RN_DTYPE_F32;
        case at::kBFloat16: return RN_DTYPE_BF16;
        case at::kHalf: return RN_DTYPE_F16;
        default: throw NotPlain{};
    }
}
int index_code(at::ScalarType t) {
    need(t == at::kInt || t == at::kLong);
    return t == at::kInt ? RN_INDEX_I32 : RN_INDEX_I64;
}

// One call: its device (that of the first tensor, which has to be the current one) and stream.
struct Call {
    int dev;
    explicit Call(const Tensor& t) : dev(t.is_cuda() ? t.get_device() : -1) {
        need(dev >= 0 && dev == c10::cuda::current_device());
    }
    void here(const Tensor& t) const {
        need(t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided);
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
    Tensor make(at::IntArrayRef sizes, at::ScalarType t) const {
        return at::detail::empty_cuda(sizes, t, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev),
                                      c10::nullopt);
    }
    const void* vector(Ref t, int64_t n, at::ScalarType type) const {
        if (!t) return nullptr;
        here(*t);
        need(t->scalar_type() == type && t->numel() == n && t->is_contiguous());
        return t->const_data_ptr();
    }
    const void* ids(const Tensor& t, int64_t n, int* code) const {
        here(t);
        *code = index_code(t.scalar_type());
        need(t.numel() == n && t.is_contiguous());
        return t.const_data_ptr();
    }
};

// Tokens of [tokens, heads, d] or [batch, len, heads, d].
struct Shape {
    int64_t batch, len;
    int dims;
};
Shape shape_of(const Tensor& t) {
    const int64_t n = t.dim();
    need(n == 3 || n == 4);
    return {n == 4 ? t.size(0) : 1, t.size(n - 3), (int)n};
}
rn_heads rows(const Call& c, const Tensor& t, const Shape& s, int64_t d, at::ScalarType type) {
    c.here(t);
    need(t.scalar_type() == type && t.dim() == s.dims);
    const auto z = t.sizes(), st = t.strides();
    const int n = s.dims;
    need(z[n - 1] == d && z[n - 3] == s.len && (n == 3 || z[0] == s.batch) &&
         (st[n - 1] == 1 || t.numel() == 0));
    return {const_cast<void*>(t.const_data_ptr()), z[n - 2], n == 4 ? st[0] : 0, st[n - 3], st[n - 2]};
}
// An output like `like`, contiguous.
rn_heads new_rows(const Call& c, const Tensor& like, Tensor* out) {
    *out = c.make(like.sizes(), like.scalar_type());
    const int n = (int)like.dim();
    const auto st = out->strides();
    return {out->mutable_data_ptr(), like.size(n - 2), n == 4 ? st[0] : 0, st[n - 3], st[n - 2]};
}

// What is done to the rows of q and k (whose data stays to be filled in).
rn_qk describe(const Call& c, const Shape& s, int64_t d, at::ScalarType type, PyObject* positions,
               PyObject* table, PyObject* wq, PyObject* wk, PyObject* eps, PyObject* norm,
               PyObject* interleaved) {
    rn_qk a = {};
    a.batch = s.batch;
    a.len = s.len;
    a.d = d;
    a.dtype = value_code(type);
    a.eps = (float)number(eps);
    a.interleaved = truth(interleaved);
    a.wq = c.vector(tensor(wq), d, type);
    a.wk = c.vector(tensor(wk), d, type);
    a.norm = norm == Py_None ? a.wq || a.wk : truth(norm);
    if (const Ref t = tensor(table)) {
        c.here(*t);
        need(t->scalar_type() == at::kFloat && t->dim() == 2 && t->size(1) > 0 && t->stride(1) == 1);
        a.table = (const float*)t->const_data_ptr();
        a.table_rows = t->size(0);
        a.rot = t->size(1);
        a.table_stride = a.table_rows > 1 ? t->stride(0) : a.rot;
        a.positions = c.ids(*given(positions), s.batch * s.len, &a.itype);
    }
    return a;
}

// A paged cache's [pages, page_size, heads, d] tensors.
rn_cache cache_of(const Call& c, const Tensor& k, const Tensor& v, at::ScalarType type,
                  PyObject* k_scale, PyObject* v_scale, bool written) {
    c.here(k);
    c.here(v);
    const at::ScalarType held = k.scalar_type();
    need(v.scalar_type() == held && k.dim() == 4 && v.dim() == 4);
    const auto zk = k.sizes(), zv = v.sizes(), sk = k.strides(), sv = v.strides();
    need(zk[0] == zv[0] && zk[1] == zv[1] && zk[2] == zv[2] && sk[3] == 1 && sv[3] == 1);
    need(held == type || held == at::kFloat8_e4m3fn);
    rn_cache a = {};
    a.k = written ? k.mutable_data_ptr() : const_cast<void*>(k.const_data_ptr());
    a.v = written ? v.mutable_data_ptr() : const_cast<void*>(v.const_data_ptr());
    a.k_page_stride = sk[0];
    a.k_slot_stride = sk[1];
    a.k_head_stride = sk[2];
    a.v_page_stride = sv[0];
    a.v_slot_stride = sv[1];
    a.v_head_stride = sv[2];
    a.pages = zk[0];
    a.page_size = zk[1];
    a.d_v = zv[3];
    a.dtype = held == at::kFloat8_e4m3fn ? RN_DTYPE_E4M3 : value_code(held);
    a.k_scale = (float)number(k_scale);
    a.v_scale = (float)number(v_scale);
    return a;
}

// The library's status of fn(), called without Python's lock.
template <typename F>
int unlocked(F fn) {
    PyThreadState* const state = PyEval_SaveThread();
    const int st = fn();
    PyEval_RestoreThread(state);
    return st;
}

template <typename... Ts>
PyObject* tuple_of(const Ts&... ts) {
    PyObject* const out = PyTuple_New(sizeof...(Ts));
    if (!out) return nullptr;
    Py_ssize_t i = 0;
    auto put = [&](const Tensor& t) {
        PyObject* const o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
        PyTuple_SET_ITEM(out, i++, o);
        return o != nullptr;
    };
    if (!(put(ts) && ...)) {
        Py_DECREF(out);
        return nullptr;
    }
    return out;
}

// Runs one call; None where it is not plain or has failed (the Python function then does it again,
// or says why it cannot be done).
template <typename F>
PyObject* plain(Py_ssize_t n, Py_ssize_t want, F fn) {
    if (n == want && C.qk_rope_fwd) {
        try {
            PyObject* const out = fn();
            if (out) return out;
            PyErr_Clear();
        } catch (...) {
        }
    }
    Py_RETURN_NONE;
}

// (q, k, positions, table, wq, wk, eps, norm, interleaved)
PyObject* qk_rope_fwd_plain(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return plain(n, 9, [&]() -> PyObject* {
        const Tensor& q = *given(a[0]);
        const Ref k = tensor(a[1]);
        const Call c(q);
        const Shape s = shape_of(q);
        const at::ScalarType type = q.scalar_type();
        const int64_t d = q.size(s.dims - 1);
        rn_qk in = describe(c, s, d, type, a[2], a[3], a[4], a[5], a[6], a[7], a[8]);
        in.q = rows(c, q, s, d, type);
        if (k) in.k = rows(c, *k, s, d, type);
        Tensor qo, ko;
        const rn_heads yq = new_rows(c, q, &qo);
        const rn_heads yk = k ? new_rows(c, *k, &ko) : rn_heads{};
        void* const stream = c.stream();
        if (unlocked([&] { return C.qk_rope_fwd(&in, &yq, &yk, stream); }) != RN_OK) return nullptr;
        return tuple_of(qo, ko);
    });
}

// (dq_out, dk_out, q, k, positions, table, wq, wk, eps, norm, interleaved, param_grads)
PyObject* qk_rope_bwd_plain(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return plain(n, 12, [&]() -> PyObject* {
        const Tensor& gq = *given(a[0]);
        const Ref gk = tensor(a[1]);
        const Call c(gq);
        const Shape s = shape_of(gq);
        const at::ScalarType type = gq.scalar_type();
        const int64_t d = gq.size(s.dims - 1);
        rn_qk in = describe(c, s, d, type, a[4], a[5], a[6], a[7], a[8], a[9], a[10]);
        const rn_heads hq = rows(c, gq, s, d, type);
        const rn_heads hk = gk ? rows(c, *gk, s, d, type) : rn_heads{};
        in.q.heads = hq.heads;
        in.k.heads = hk.heads;
        if (in.norm) {
            in.q = rows(c, *given(a[2]), s, d, type);
            if (gk) in.k = rows(c, *given(a[3]), s, d, type);
            need(in.q.heads == hq.heads && in.k.heads == hk.heads);
        }
        const bool params = truth(a[11]) && in.norm;
        Tensor dq, dk, dwq, dwk, ws;
        const rn_heads yq = new_rows(c, gq, &dq);
        const rn_heads yk = gk ? new_rows(c, *gk, &dk) : rn_heads{};
        size_t bytes = 0;
        if (params && in.wq) dwq = c.make({d}, type);
        if (params && in.wk) dwk = c.make({d}, type);
        if (dwq.defined() || dwk.defined()) {
            need(C.qk_rope_bwd_workspace_size(d, &bytes) == RN_OK);
            ws = c.make({(int64_t)bytes}, at::kByte);
        }
        auto at = [](const Tensor& t) { return t.defined() ? t.mutable_data_ptr() : nullptr; };
        void* const stream = c.stream();
        if (unlocked([&] {
                return C.qk_rope_bwd(&in, &hq, &hk, &yq, &yk, at(dwq), at(dwk), at(ws), bytes, stream);
            }) != RN_OK)
            return nullptr;
        return tuple_of(dq, dk, dwq, dwk);
    });
}

// (k, v, slots, k_cache, v_cache, positions, table, wk, eps, q, wq, norm, interleaved, k_scale, v_scale)
PyObject* kv_append_plain(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return plain(n, 15, [&]() -> PyObject* {
        const Tensor &k = *given(a[0]), &v = *given(a[1]), &kc = *given(a[3]), &vc = *given(a[4]);
        const Ref q = tensor(a[9]);
        need(q || a[10] == Py_None);
        const Call c(k);
        const Shape s = shape_of(k);
        const at::ScalarType type = k.scalar_type();
        const int64_t d = k.size(s.dims - 1);
        rn_qk in = describe(c, s, d, type, a[5], a[6], a[10], a[7], a[8], a[11], a[12]);
        const rn_cache cache = cache_of(c, kc, vc, type, a[13], a[14], true);
        int itype = 0;
        const void* const slots = c.ids(*given(a[2]), s.batch * s.len, &itype);
        need(in.rot == 0 || in.itype == itype);
        in.itype = itype;
        in.k = rows(c, k, s, d, type);
        const rn_heads hv = rows(c, v, s, cache.d_v, type);
        need(kc.size(2) == in.k.heads && kc.size(3) == d);
        Tensor qo;
        rn_heads yq = {};
        if (q) {
            in.q = rows(c, *q, s, d, type);
            yq = new_rows(c, *q, &qo);
        }
        void* const stream = c.stream();
        if (unlocked([&] { return C.kv_append(&in, &yq, &hv, &cache, slots, stream); }) != RN_OK)
            return nullptr;
        return tuple_of(qo);
    });
}

// (k_cache, v_cache, slots, dtype, k_scale, v_scale)
PyObject* kv_gather_plain(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return plain(n, 6, [&]() -> PyObject* {
        const Tensor &kc = *given(a[0]), &vc = *given(a[1]), &slots = *given(a[2]);
        const Call c(kc);
        at::ScalarType type = kc.scalar_type();
        if (a[3] != Py_None) {
            need(THPDtype_Check(a[3]));
            type = reinterpret_cast<THPDtype*>(a[3])->scalar_type;
        } else if (type == at::kFloat8_e4m3fn) {
            type = at::kBFloat16;
        }
        const int code = value_code(type);
        const rn_cache cache = cache_of(c, kc, vc, type, a[4], a[5], false);
        const int64_t tokens = slots.numel(), heads = kc.size(2), d = kc.size(3);
        int itype = 0;
        const void* const at = c.ids(slots, tokens, &itype);
        Tensor k = c.make({tokens, heads, d}, type), v = c.make({tokens, heads, cache.d_v}, type);
        const rn_heads yk = {k.mutable_data_ptr(), heads, 0, heads * d, d};
        const rn_heads yv = {v.mutable_data_ptr(), heads, 0, heads * cache.d_v, cache.d_v};
        void* const stream = c.stream();
        if (unlocked([&] {
                return C.kv_gather(&cache, d, at, itype, tokens, code, &yk, &yv, stream);
            }) != RN_OK)
            return nullptr;
        return tuple_of(k, v);
    });
}

// (page_table, starts, offsets, n, page_size)
PyObject* kv_slots_plain(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return plain(n, 5, [&]() -> PyObject* {
        const Tensor &table = *given(a[0]), &starts = *given(a[1]), &offsets = *given(a[2]);
        const Call c(offsets);
        const at::ScalarType type = offsets.scalar_type();
        c.here(table);
        need(table.scalar_type() == type && table.dim() == 2);
        const int64_t seqs = table.size(0), width = table.size(1), tokens = whole(a[3]);
        need(tokens >= 0 && seqs > 0 && width > 0 && (width == 1 || table.stride(1) == 1));
        int code = 0, other = 0;
        const void* const off = c.ids(offsets, seqs + 1, &code);
        const void* const first = c.ids(starts, seqs, &other);
        need(code == other);
        const int64_t page = whole(a[4]);
        Tensor slots = c.make({tokens}, type), positions = c.make({tokens}, type);
        void* const stream = c.stream();
        if (unlocked([&] {
                return C.kv_slots(code, table.const_data_ptr(), seqs > 1 ? table.stride(0) : width, width,
                                  first, off, seqs, page, slots.mutable_data_ptr(),
                                  positions.mutable_data_ptr(), tokens, stream);
            }) != RN_OK)
            return nullptr;
        return tuple_of(slots, positions);
    });
}

// use(address, ...): the library's entry points, in the order of Entries.
PyObject* use(PyObject*, PyObject* const* a, Py_ssize_t n) {
    constexpr Py_ssize_t want = sizeof(Entries) / sizeof(void*);
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "use() takes %zd addresses", want);
        return nullptr;
    }
    void* at[want];
    for (Py_ssize_t i = 0; i < want; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    static_assert(sizeof(at) == sizeof(C), "entry points");
    memcpy(&C, at, sizeof(C));
    Py_RETURN_NONE;
}

#define METHOD(name, fn) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("use", use),
                         METHOD("qk_rope_fwd", qk_rope_fwd_plain),
                         METHOD("qk_rope_bwd", qk_rope_bwd_plain),
                         METHOD("kv_append", kv_append_plain),
                         METHOD("kv_gather", kv_gather_plain),
                         METHOD("kv_slots", kv_slots_plain),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
    PyObject* const m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
