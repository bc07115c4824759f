// nf4kv_bind.cpp -- the calls of nf4kv.h on torch tensors, for nf4kv.py.
//
// Checks of shapes, types and devices, output and workspace allocation, and the
// call on the current stream; every computation is the library's.  A decode
// step makes a handful of these calls between kernels of a few microseconds,
// so that what a call costs on the host is what it costs altogether: through
// ctypes and checks in Python it was 7 to 13 us, here it is 3.5 to 6 with the launch.
//
// No exception leaves an entry: each is turned into a Python one (ValueError
// for arguments, NF4KVError for a status of the library).
#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/hip/EmptyTensor.h>
#include <Python.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <stdexcept>
#include <string>
#include <vector>

#include "nf4kv.h"

namespace {

PyObject* g_error = nullptr;  // NF4KVError(code, where)
PyObject* g_parts[5];         // the names of an NF4KVCache's parts

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Status {
    int code;
    const char* where;
};
struct PythonError {};  // already set

void need(bool ok, const char* what) {
    if (!ok) throw Refused(what);
}

void check(int code, const char* where) {
    if (code != NF4_OK) throw Status{code, where};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) throw Refused(what);
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}

int32_t int32(PyObject* o, const char* what) {
    const int64_t v = integer(o);
    need(v >= INT32_MIN && v <= INT32_MAX, what);
    return int32_t(v);
}

// An uninitialised tensor on the GPU.  (Without the dispatcher's layers, which
// take as long again: 0.5 us of a call's 3.5 to 6.)
at::Tensor made(at::IntArrayRef sizes, const at::TensorOptions& options) {
    return at::detail::empty_cuda(sizes, options);
}

// The current stream, on whose device all tensors given (None: not given) are.
void* stream_for(std::initializer_list<PyObject*> given) {
    const auto stream = c10::hip::getCurrentHIPStream();
    for (PyObject* o : given)
        if (o != Py_None) {
            const at::Tensor& t = tensor(o, "not a tensor");
            need(t.is_cuda() && t.get_device() == stream.device_index(), "tensors: all on the current GPU");
        }
    return stream.stream();
}

uint16_t* bf16(const at::Tensor& t) { return static_cast<uint16_t*>(t.data_ptr()); }

// An NF4KVCache as it stands at the call: its tensors are ordinary attributes,
// copied, moved, replaced and resized like any others, so that their addresses
// hold for one call only.  (Read and checked anew: 0.2 us.)
struct Held {
    nf4_kv_cache c;
    int64_t device;  // -1: no GPU

    explicit Held(PyObject* cache) {
        for (int i = 0; i < 5; ++i) {
            own[i] = PyObject_GetAttr(cache, g_parts[i]);
            if (!own[i]) {
                drop();
                if (!PyErr_ExceptionMatches(PyExc_AttributeError)) throw PythonError{};
                PyErr_Clear();
                throw Refused("cache: an NF4KVCache");
            }
        }
        try {
            fill();
        } catch (...) {
            drop();
            throw;
        }
    }
    ~Held() { drop(); }
    Held(const Held&) = delete;
    Held& operator=(const Held&) = delete;

   private:
    PyObject* own[5] = {};

    void drop() {
        for (PyObject* o : own) Py_XDECREF(o);
    }

    void fill() {
        const char* const codes = "codes: contiguous uint8 [pages, heads, page, dim/2]";
        const char* const scales = "scales: contiguous bf16 [pages, heads, page, dim/64]";
        const at::Tensor &kc = tensor(own[0], codes), &ks = tensor(own[1], scales), &vc = tensor(own[2], codes),
                         &vs = tensor(own[3], scales);
        need(kc.dim() == 4 && kc.scalar_type() == at::kByte && vc.scalar_type() == at::kByte &&
                 vc.sizes() == kc.sizes() && kc.is_contiguous() && vc.is_contiguous() && kc.size(1) <= 1024 &&
                 kc.size(2) <= 256 && kc.size(3) <= 128,
             codes);
        for (const at::Tensor* s : {&ks, &vs})
            need(s->dim() == 4 && s->scalar_type() == at::kBFloat16 && s->is_contiguous() &&
                     s->size(0) == kc.size(0) && s->size(1) == kc.size(1) && s->size(2) == kc.size(2) &&
                     s->size(3) == kc.size(3) / 32,
                 scales);
        for (const at::Tensor* t : {&ks, &vc, &vs}) need(t->device() == kc.device(), "codes and scales: on one device");
        const bool nf4 = PyUnicode_Check(own[4]) && PyUnicode_CompareWithASCIIString(own[4], "nf4") == 0;
        need(nf4 || (PyUnicode_Check(own[4]) && PyUnicode_CompareWithASCIIString(own[4], "fp4") == 0),
             "quant_type: \"nf4\" or \"fp4\"");
        c = {static_cast<uint8_t*>(kc.data_ptr()), bf16(ks), static_cast<uint8_t*>(vc.data_ptr()), bf16(vs),
             kc.size(0), int32_t(kc.size(1)), int32_t(2 * kc.size(3)), int32_t(kc.size(2)),
             nf4 ? NF4_QUANT_NF4 : NF4_QUANT_FP4};
        device = kc.is_cuda() ? kc.get_device() : -1;
    }
};

void* stream_for(const Held& cache, std::initializer_list<PyObject*> given) {
    void* const stream = stream_for(given);
    need(cache.device == THPVariable_Unpack(*given.begin()).get_device(), "cache: on the tensors' GPU");
    return stream;
}

// A contiguous vector of at least n elements.
template <typename T>
const T* ints(PyObject* o, int64_t n, const char* what) {
    const at::Tensor& t = tensor(o, what);
    need(t.scalar_type() == c10::CppTypeToScalarType<T>::value && t.numel() >= n && t.is_contiguous(), what);
    return static_cast<const T*>(t.data_ptr());
}

// The stride of dimension d, or, since that of a single element may be any
// number, `other` for one.
int64_t stride(const at::Tensor& t, int d, int64_t other) { return t.size(d) == 1 ? other : t.stride(d); }

// bf16 [tokens, heads, dim] with whole heads side by side: its token stride.
int64_t rows(const at::Tensor& t, int64_t tokens, int64_t heads, int64_t dim, const char* what) {
    need(t.dim() == 3 && t.scalar_type() == at::kBFloat16 && t.size(0) == tokens && t.size(1) == heads &&
             t.size(2) == dim && t.stride(2) == 1 && (heads == 1 || t.stride(1) == dim),
         what);
    return stride(t, 0, heads * dim);
}

const at::Tensor& rope_table(PyObject* o) {
    const at::Tensor& t = tensor(o, "table: fp32 [max_pos, rot]");
    need(t.dim() == 2 && t.scalar_type() == at::kFloat && t.is_contiguous(), "table: fp32 [max_pos, rot]");
    return t;
}

// cache(cache) -> the bytes of its nf4_kv_cache
PyObject* cache(PyObject* const* a) {
    const Held own(a[0]);
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&own.c), sizeof(own.c));
}

// rope(x, positions, table, layout, out, backward) -> tensor
PyObject* rope(PyObject* const* a) {
    const char* const what = "x: bf16 or fp32 [tokens, heads, head_dim], a head's elements side by side";
    const at::Tensor& x = tensor(a[0], what);
    need(x.dim() == 3 && (x.scalar_type() == at::kBFloat16 || x.scalar_type() == at::kFloat) && x.stride(2) == 1 &&
             x.size(1) <= INT32_MAX && x.size(2) <= INT32_MAX,
         what);
    const int32_t* positions = ints<int32_t>(a[1], x.size(0), "positions: int32 [tokens]");
    const at::Tensor& t = rope_table(a[2]);
    need(t.size(1) <= INT32_MAX, "table: fp32 [max_pos, rot]");
    void* const stream = stream_for({a[0], a[1], a[2], a[4]});
    at::Tensor y;
    if (a[4] == Py_None) {
        y = made(x.sizes(), x.options());
    } else {
        y = tensor(a[4], "out: as x");
        need(y.sizes() == x.sizes() && y.scalar_type() == x.scalar_type() && y.stride(2) == 1, "out: as x");
    }
    const int64_t xh = stride(x, 1, x.size(2)), xt = stride(x, 0, x.size(1) * xh);
    const int64_t yh = stride(y, 1, y.size(2)), yt = stride(y, 0, y.size(1) * yh);
    const bool back = a[5] == Py_True;
    check((back ? nf4_rope_backward : nf4_rope_forward)(
              x.data_ptr(), xt, xh, y.data_ptr(), yt, yh, x.size(0),
              int32_t(x.size(1)), int32_t(x.size(2)), x.scalar_type() == at::kBFloat16, positions,
              static_cast<const float*>(t.data_ptr()), t.size(0), int32_t(t.size(1)), int32(a[3], "layout"),
              stream),
          back ? "nf4_rope_backward" : "nf4_rope_forward");
    return THPVariable_Wrap(y);
}

// plan(kv_lens, new_lens, block_table, free_pages, free_state, page_size, max_tokens, done)
//   -> (kv_lens, cu_new, slots, positions, free_state, refused)
PyObject* plan(PyObject* const* a) {
    const at::Tensor& table = tensor(a[2], "block_table: int32 [batch, width]");
    need(table.dim() == 2 && table.scalar_type() == at::kInt && table.is_contiguous() && table.size(0) <= INT32_MAX &&
             table.size(1) <= INT32_MAX,
         "block_table: int32 [batch, width]");
    const int64_t batch = table.size(0);
    const int32_t* lens = ints<int32_t>(a[0], batch, "kv_lens: int32 [batch]");
    const int32_t* added = ints<int32_t>(a[1], batch, "new_lens: int32 [batch]");
    const int32_t* ring = ints<int32_t>(a[3], 1, "free_pages: int32 [capacity]");
    const int64_t capacity = THPVariable_Unpack(a[3]).numel();
    need(capacity <= INT32_MAX, "free_pages: int32 [capacity]");
    const int32_t* state = ints<int32_t>(a[4], 2, "free_state: int32 [2]");
    const int32_t page = int32(a[5], "page_size"), most = int32(a[6], "max_tokens");
    need(most >= 0, "max_tokens: not negative");
    const int32_t* done = a[7] == Py_None ? nullptr : ints<int32_t>(a[7], batch, "done: int32 [batch]");
    void* const stream = stream_for({a[0], a[1], a[2], a[3], a[4], a[7]});
    // the int32 outputs share one allocation
    const at::Tensor slots = made({most}, table.options().dtype(at::kLong));
    const at::Tensor own = made({most + 2 * batch + 4}, table.options());
    const std::vector<at::Tensor> part = own.unsafe_split_with_sizes({most, batch, batch + 1, 2, 1});
    int32_t* at_[5];
    for (int i = 0; i < 5; ++i) at_[i] = static_cast<int32_t*>(part[i].data_ptr());
    check(nf4_kv_plan(lens, added, done, int32_t(batch), static_cast<int32_t*>(table.data_ptr()),
                      int32_t(table.size(1)), page, const_cast<int32_t*>(ring), int32_t(capacity), state, most, at_[1],
                      at_[2], static_cast<int64_t*>(slots.data_ptr()), at_[0], at_[3], at_[4], stream),
          "nf4_kv_plan");
    PyObject* const out = PyTuple_New(6);
    if (!out) throw PythonError{};
    const at::Tensor* const given[6] = {&part[1], &part[2], &slots, &part[0], &part[3], &part[4]};
    for (int i = 0; i < 6; ++i) PyTuple_SET_ITEM(out, i, THPVariable_Wrap(*given[i]));
    return out;
}

// append(cache, k, v, slots, positions, table, q, layout, q_out) -> q_out or None
PyObject* append(PyObject* const* a) {
    const Held own(a[0]);
    const nf4_kv_cache* const c = &own.c;
    const char* const kw = "k: bf16 [tokens, heads, head_dim]";
    const at::Tensor &k = tensor(a[1], kw), &v = tensor(a[2], "v: as k");
    need(k.dim() == 3, kw);
    const int64_t tokens = k.size(0);
    const int64_t k_stride = rows(k, tokens, c->n_heads, c->head_dim, kw);
    const int64_t v_stride = rows(v, tokens, c->n_heads, c->head_dim, "v: as k");
    const int64_t* slots = ints<int64_t>(a[3], tokens, "slots: int64 [tokens]");
    const int32_t* positions = nullptr;
    const float* table = nullptr;
    int64_t max_pos = 0, rot = 0;
    if (a[5] != Py_None) {
        const at::Tensor& t = rope_table(a[5]);
        max_pos = t.size(0), rot = t.size(1);
        need(rot > 0 && rot <= INT32_MAX, "table: fp32 [max_pos, rot]");
        table = static_cast<const float*>(t.data_ptr());
        positions = ints<int32_t>(a[4], tokens, "positions: int32 [tokens]");
    }
    at::Tensor q, y;
    int64_t q_stride = 0, y_stride = 0;
    if (a[6] != Py_None) {
        const char* const qw = "q: bf16 [tokens, q_heads, head_dim], as many tokens as k, and rotated by the table";
        q = tensor(a[6], qw);
        need(table && q.dim() == 3 && q.size(1) <= INT32_MAX, qw);
        q_stride = rows(q, tokens, q.size(1), c->head_dim, qw);
    }
    const bool has = q.defined();
    void* const stream = stream_for(own, {a[1], a[2], a[3], table ? a[4] : Py_None, a[5], a[6], a[8]});
    if (has) {
        y = a[8] == Py_None ? made(q.sizes(), q.options()) : tensor(a[8], "q_out: as q");
        y_stride = rows(y, tokens, q.size(1), c->head_dim, "q_out: as q");
    }
    check(nf4_kv_append(c, bf16(k), k_stride, bf16(v), v_stride, slots, tokens, has ? bf16(q) : nullptr,
                        q_stride, has ? bf16(y) : nullptr, y_stride, has ? int32_t(q.size(1)) : 0, positions, table, max_pos, int32_t(rot), int32(a[7], "layout"),
                        stream),
          "nf4_kv_append");
    if (has) return THPVariable_Wrap(y);
    Py_RETURN_NONE;
}

// read(cache, slots) -> (k, v)
PyObject* read(PyObject* const* a) {
    const Held own(a[0]);
    const nf4_kv_cache* const c = &own.c;
    const at::Tensor& s = tensor(a[1], "slots: int64 [tokens]");
    need(s.dim() == 1, "slots: int64 [tokens]");
    const int64_t* slots = ints<int64_t>(a[1], 0, "slots: int64 [tokens]");
    void* const stream = stream_for(own, {a[1]});
    const auto options = s.options().dtype(at::kBFloat16);
    const at::Tensor k = made({s.size(0), c->n_heads, c->head_dim}, options);
    const at::Tensor v = made({s.size(0), c->n_heads, c->head_dim}, options);
    check(nf4_kv_read(c, slots, s.size(0), bf16(k), bf16(v), stream), "nf4_kv_read");
    PyObject* const out = PyTuple_New(2);
    if (!out) throw PythonError{};
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(k));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(v));
    return out;
}

// attention(cache, q, cu_q, kv_lens, block_table, max_q, max_len, scale, window, sinks, out, ws) -> out
PyObject* attention(PyObject* const* a) {
    const Held own(a[0]);
    const nf4_kv_cache* const c = &own.c;
    const char* const qw = "q: bf16 [total_q, q_heads, head_dim]";
    const at::Tensor& q = tensor(a[1], qw);
    need(q.dim() == 3 && q.size(1) <= INT32_MAX, qw);
    const int64_t q_stride = rows(q, q.size(0), q.size(1), c->head_dim, qw);
    const at::Tensor& table = tensor(a[4], "block_table: int32 [batch, width]");
    need(table.dim() == 2 && table.scalar_type() == at::kInt && table.is_contiguous() && table.size(0) <= INT32_MAX &&
             table.size(1) <= INT32_MAX,
         "block_table: int32 [batch, width]");
    const int64_t batch = table.size(0);
    const int32_t* cu = ints<int32_t>(a[2], batch + 1, "cu_q: int32 [batch + 1]");
    const int32_t* lens = ints<int32_t>(a[3], batch, "kv_lens: int32 [batch]");
    const int32_t max_q = int32(a[5], "max_q"), window = int32(a[8], "window"), sinks = int32(a[9], "sinks");
    const int64_t most = a[6] == Py_None ? table.size(1) * c->page_size : integer(a[6]);
    need(most <= INT32_MAX, "max_len");
    double scale = 1.0 / std::sqrt(double(c->head_dim));
    if (a[7] != Py_None) {
        scale = PyFloat_AsDouble(a[7]);
        if (scale == -1.0 && PyErr_Occurred()) throw PythonError{};
    }
    void* const stream = stream_for(own, {a[1], a[2], a[3], a[4], a[10], a[11]});
    const at::Tensor y = a[10] == Py_None ? made(q.sizes(), q.options()) : tensor(a[10], "out: as q");
    const int64_t y_stride = rows(y, q.size(0), q.size(1), c->head_dim, "out: as q");
    need(a[11] == Py_None || tensor(a[11], "ws: a contiguous tensor").is_contiguous(), "ws: a contiguous tensor");
    at::Tensor ws;
    size_t bytes = 0;
    if (a[11] == Py_None) {
        bytes = nf4_kv_attention_ws_bytes(int32_t(batch), int32_t(q.size(1)), c->n_heads, c->head_dim, max_q,
                                          int32_t(most), window, sinks);
        if (bytes) ws = made({int64_t(bytes)}, q.options().dtype(at::kByte));
    } else {
        ws = THPVariable_Unpack(a[11]);
        bytes = ws.numel() * ws.element_size();
    }
    // (a new output has zeros where the caller's own keeps what it has)
    const auto call = a[10] == Py_None ? nf4_kv_attention_padded : nf4_kv_attention;
    check(call(c, bf16(q), q_stride, q.size(0), int32_t(q.size(1)), cu, lens,
                           static_cast<const int32_t*>(table.data_ptr()), int32_t(table.size(1)), int32_t(batch),
                           max_q, int32_t(most), float(scale), window, sinks, bf16(y), y_stride,
                           ws.defined() ? ws.data_ptr() : nullptr, bytes, stream),
          "nf4_kv_attention");
    return THPVariable_Wrap(y);
}

// set_error(class)
PyObject* set_error(PyObject* const* a) {
    Py_INCREF(a[0]);
    Py_XDECREF(g_error);
    g_error = a[0];
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        // (the calls are no part of autograd: skip its dispatch layers)
        const at::AutoDispatchBelowADInplaceOrView below;
        return F(args);
    } catch (const PythonError&) {
    } catch (const Status& s) {
        PyObject* const e = g_error ? PyObject_CallFunction(g_error, "is", s.code, s.where) : nullptr;
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        } else if (!PyErr_Occurred()) {
            PyErr_Format(PyExc_RuntimeError, "%s: status %d", s.where, s.code);
        }
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<cache, 1>("cache"),     method<rope, 6>("rope"),
                           method<plan, 8>("plan"),       method<append, 9>("append"),
                           method<read, 2>("read"),       method<attention, 12>("attention"),
                           method<set_error, 1>("set_error"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_nf4kv", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit__nf4kv() {
    const char* const names[5] = {"k_codes", "k_scales", "v_codes", "v_scales", "quant_type"};
    for (int i = 0; i < 5; ++i)
        if (!(g_parts[i] = PyUnicode_InternFromString(names[i]))) return nullptr;
    return PyModule_Create(&g_module);
}
