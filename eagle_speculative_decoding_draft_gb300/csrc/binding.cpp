// binding.cpp - a short way from tensors to the calls that a step makes most often: eagle_rms_norm,
// eagle_quantize_rows, eagle_linear, eagle_kv4_append_rotary and eagle_kv4_read.
//
// Single tokens and small trees cost the GPU a few microseconds a call, less than Python takes to look at
// the arguments.  Each function here takes the arguments of its namesake in fp8.py or kv4.py, and where they are
// what they usually are (plain CUDA tensors of the right types, shapes and layouts on the current device) it
// allocates the outputs, makes the call on the current stream and returns them.  Anything else, an error of the
// call included, gives NotImplemented: the caller then takes the long way, which says what is wrong.
#include <Python.h>

#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/eagle_tree.h"

namespace {

decltype(&eagle_rms_norm) g_rms_norm;
decltype(&eagle_quantize_rows) g_quantize_rows;
decltype(&eagle_linear) g_linear;
decltype(&eagle_kv4_append_rotary) g_append_rotary;
decltype(&eagle_kv4_read) g_kv4_read;

constexpr auto kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kU8 = at::kByte;
constexpr auto kE4m3 = at::kFloat8_e4m3fn;

PyObject *not_here() { Py_RETURN_NOTIMPLEMENTED; }

// A plain tensor on device `index`, or null.
const at::Tensor *tensor(PyObject *o, int index) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    return t.is_cuda() && t.layout() == at::kStrided && t.get_device() == index ? &t : nullptr;
}

struct Matrix {
    void *p = nullptr;
    int64_t rows = 0, cols = 0, ld = 0;
};
bool matrix(PyObject *o, int index, at::ScalarType type, Matrix *m) {
    const at::Tensor *t = tensor(o, index);
    if (!t || t->scalar_type() != type || t->dim() != 2) return false;
    m->rows = t->size(0), m->cols = t->size(1), m->ld = t->stride(0);
    if ((m->cols > 1 && t->stride(1) != 1) || m->rows > INT32_MAX || m->cols > INT32_MAX) return false;
    if (m->rows < 2)
        m->ld = (m->cols + 15) / 16 * 16;  // whatever the strides of sizes of 1
    else if (m->ld < m->cols)
        return false;
    m->p = t->data_ptr();
    return true;
}
bool vector(PyObject *o, int index, at::ScalarType type, int64_t n, void **p) {
    const at::Tensor *t = tensor(o, index);
    if (!t || t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) return false;
    *p = t->data_ptr();
    return true;
}
at::Tensor new_rows(int index, int64_t rows, int64_t cols, at::ScalarType type, int64_t step, Matrix *m) {
    m->rows = rows, m->cols = cols, m->ld = (cols + step - 1) / step * step;
    at::Tensor t = at::empty_strided({rows, cols}, {m->ld, 1}, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(index)));
    m->p = t.data_ptr();
    return t;
}
eagle_stream_t stream(int index) {
    return reinterpret_cast<eagle_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream());
}

// (x)
PyObject *quantize_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    const int index = c10::cuda::current_device();
    Matrix x, y;
    if (n != 1 || !matrix(a[0], index, kBf16, &x)) return not_here();
    at::Tensor codes = new_rows(index, x.rows, x.cols, kE4m3, 16, &y);
    at::Tensor scale = at::empty_strided({x.rows}, {1}, codes.options().dtype(kF32));
    if (g_quantize_rows(x.p, x.ld, static_cast<int32_t>(x.rows), static_cast<int32_t>(x.cols), y.p, y.ld, scale.data_ptr<float>(),
                        stream(index)) != EAGLE_OK)
        return not_here();
    return Py_BuildValue("(NN)", THPVariable_Wrap(codes), THPVariable_Wrap(scale));
}

// (x, weight, eps, residual or None, whether y is 8-bit rows)
PyObject *rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    const int index = c10::cuda::current_device();
    Matrix x, r, y, s;
    void *w;
    if (n != 5 || !matrix(a[0], index, kBf16, &x) || !vector(a[1], index, kBf16, x.cols, &w) || !PyFloat_CheckExact(a[2])) return not_here();
    const bool residual = a[3] != Py_None, fp8 = a[4] == Py_True;
    if (residual && (!matrix(a[3], index, kBf16, &r) || r.rows != x.rows || r.cols != x.cols)) return not_here();
    at::Tensor out = new_rows(index, x.rows, x.cols, fp8 ? kE4m3 : kBf16, 16, &y), sum, scale;
    if (residual) sum = new_rows(index, x.rows, x.cols, kBf16, 8, &s);
    if (fp8) scale = at::empty_strided({x.rows}, {1}, out.options().dtype(kF32));
    if (g_rms_norm(x.p, x.ld, r.p, r.ld, w, static_cast<float>(PyFloat_AS_DOUBLE(a[2])), static_cast<int32_t>(x.rows),
                   static_cast<int32_t>(x.cols), s.p, s.ld, fp8 ? EAGLE_E4M3 : EAGLE_BF16, y.p, y.ld,
                   fp8 ? scale.data_ptr<float>() : nullptr, stream(index)) != EAGLE_OK)
        return not_here();
    PyObject *none = Py_None;
    PyObject *ps = fp8 ? THPVariable_Wrap(scale) : (Py_INCREF(none), none);
    PyObject *pt = residual ? THPVariable_Wrap(sum) : (Py_INCREF(none), none);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(out), ps, pt);
}

// (w, x, bias, act code, residual, w_scale, x_scale, whether y is fp32, out, workspace), None for what is not given
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    const int index = c10::cuda::current_device();
    if (n != 10 || !THPVariable_CheckExact(a[0])) return not_here();
    const at::ScalarType kind = THPVariable_Unpack(a[0]).scalar_type();
    const bool fp8 = kind == kE4m3;
    Matrix w, x, r, y;
    if ((!fp8 && kind != kBf16) || !matrix(a[0], index, kind, &w) || !matrix(a[1], index, kind, &x) || x.cols != w.cols) return not_here();
    const long act = PyLong_AsLong(a[3]);
    if (act < 0 || act > 3 || (act == EAGLE_ACT_SWIGLU && w.rows % 2)) return not_here();
    const int64_t width = act == EAGLE_ACT_SWIGLU ? w.rows / 2 : w.rows;
    void *bias = nullptr, *ws = nullptr, *xs = nullptr;
    if (fp8 ? !vector(a[5], index, kF32, w.rows, &ws) || !vector(a[6], index, kF32, x.rows, &xs) : a[5] != Py_None || a[6] != Py_None)
        return not_here();
    if (a[2] != Py_None && !vector(a[2], index, kBf16, w.rows, &bias)) return not_here();
    if (a[4] != Py_None && (!matrix(a[4], index, kBf16, &r) || r.rows != x.rows || r.cols != width)) return not_here();
    const at::ScalarType to = a[7] == Py_True ? kF32 : kBf16;
    void *scratch = nullptr;
    size_t bytes = 0;
    if (a[9] != Py_None) {
        const at::Tensor *t = tensor(a[9], index);
        if (!t || t->scalar_type() != kU8 || !t->is_contiguous()) return not_here();
        scratch = t->data_ptr(), bytes = static_cast<size_t>(t->numel());
    }
    at::Tensor made;
    if (a[8] == Py_None)
        made = new_rows(index, x.rows, width, to, 8, &y);
    else if (!matrix(a[8], index, to, &y) || y.rows != x.rows || y.cols != width)
        return not_here();
    eagle_linear_args l{};
    l.rows = static_cast<int32_t>(x.rows), l.out_features = static_cast<int32_t>(width), l.in_features = static_cast<int32_t>(w.cols);
    l.dtype = fp8 ? EAGLE_E4M3 : EAGLE_BF16, l.y_dtype = to == kF32 ? EAGLE_F32 : EAGLE_BF16, l.act = static_cast<eagle_activation>(act);
    l.w = w.p, l.x = x.p, l.ldw = w.ld, l.ldx = x.ld;
    l.w_scale = static_cast<const float *>(ws), l.x_scale = static_cast<const float *>(xs);
    l.bias = bias, l.residual = r.p, l.ldr = r.ld, l.y = y.p, l.ldy = y.ld;
    if (g_linear(&l, scratch, bytes, nullptr, stream(index)) != EAGLE_OK) return not_here();
    if (a[8] == Py_None) return THPVariable_Wrap(made);
    Py_INCREF(a[8]);
    return a[8];
}

// Rows of two bf16 tensors [B][n][heads][D] of one shape and layout, evenly spaced.
bool rows4(PyObject *o, PyObject *like, int index, int64_t B, int64_t heads, int64_t D, Matrix *m) {
    const at::Tensor *t = tensor(o, index), *u = o == like ? t : tensor(like, index);
    if (!t || !u || t->scalar_type() != kBf16 || u->scalar_type() != kBf16 || t->dim() != 4) return false;
    if (t != u && (t->sizes() != u->sizes() || t->strides() != u->strides())) return false;
    const int64_t n = t->size(1), step = t->stride(1);
    if (t->size(0) != B || t->size(3) != D || (heads && t->size(2) != heads) || t->size(2) < 1 || n < 1 || n > INT32_MAX) return false;
    if (t->stride(3) != 1 || t->stride(2) != D || t->stride(0) != n * step || step < t->size(2) * D || step % 8) return false;
    m->p = t->data_ptr(), m->rows = n, m->cols = t->size(2), m->ld = step;
    return true;
}
bool ints(PyObject *o, int index, int64_t B, int64_t n, const int32_t **p) {
    if (o == Py_None) return true;
    const at::Tensor *t = tensor(o, index);
    if (!t || t->scalar_type() != kI32 || !t->is_contiguous() || t->size(0) != B || t->dim() != (n < 0 ? 1 : 2)) return false;
    if (n >= 0 && t->size(1) != n) return false;
    *p = static_cast<const int32_t *>(t->data_ptr());
    return true;
}

// ((address of the cache's struct, batch, kv heads, head_dim, device, address of its status), k, v, q, theta, positions,
// select, count, start): the turned queries, or None without them
PyObject *append_rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9 || !PyTuple_CheckExact(a[0]) || PyTuple_GET_SIZE(a[0]) != 6 || !PyFloat_CheckExact(a[4])) return not_here();
    int64_t c[6];
    for (int i = 0; i < 6; ++i) c[i] = static_cast<int64_t>(PyLong_AsSsize_t(PyTuple_GET_ITEM(a[0], i)));
    const int index = c10::cuda::current_device();
    Matrix k, v, q;
    if (c[4] != index || !rows4(a[1], a[2], index, c[1], c[2], c[3], &k) || !rows4(a[2], a[2], index, c[1], c[2], c[3], &v)) return not_here();
    const bool queries = a[3] != Py_None;
    if (queries && (!rows4(a[3], a[3], index, c[1], 0, c[3], &q) || q.rows != k.rows)) return not_here();
    int64_t slots = k.rows;
    if (a[6] != Py_None) {
        const at::Tensor *s = tensor(a[6], index);
        if (!s || s->dim() != 2 || a[5] == Py_None || s->size(1) > INT32_MAX) return not_here();
        slots = s->size(1);
    }
    const int32_t *positions = nullptr, *select = nullptr, *count = nullptr, *start = nullptr;
    if (!ints(a[5], index, c[1], k.rows, &positions) || !ints(a[6], index, c[1], slots, &select) || !ints(a[7], index, c[1], -1, &count) ||
        !ints(a[8], index, c[1], -1, &start))
        return not_here();
    at::Tensor out;
    if (queries)
        out = at::empty_strided({c[1], q.rows, q.cols, c[3]}, {q.rows * q.cols * c[3], q.cols * c[3], c[3], 1},
                                at::TensorOptions().dtype(kBf16).device(at::kCUDA, static_cast<c10::DeviceIndex>(index)));
    if (g_append_rotary(reinterpret_cast<const eagle_kv4_cache *>(c[0]), static_cast<int32_t>(c[1]), static_cast<int32_t>(k.rows),
                        static_cast<int32_t>(slots), k.p, v.p, k.ld, positions, static_cast<float>(PyFloat_AS_DOUBLE(a[4])),
                        queries ? static_cast<int32_t>(q.cols) : 0, q.p, q.ld, queries ? out.data_ptr() : nullptr, select, count, start,
                        reinterpret_cast<int32_t *>(c[5]), stream(index)) != EAGLE_OK)
        return not_here();
    if (queries) return THPVariable_Wrap(out);
    Py_RETURN_NONE;
}

// (the same tuple, k, v, start): reads the cache back into k and v; True
PyObject *kv4_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 4 || !PyTuple_CheckExact(a[0]) || PyTuple_GET_SIZE(a[0]) != 6) return not_here();
    int64_t c[6];
    for (int i = 0; i < 6; ++i) c[i] = static_cast<int64_t>(PyLong_AsSsize_t(PyTuple_GET_ITEM(a[0], i)));
    const int index = c10::cuda::current_device();
    const at::Tensor *k = tensor(a[1], index), *v = tensor(a[2], index);
    if (c[4] != index || !k || !v || k->dim() != 4 || k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type()) return not_here();
    if (k->scalar_type() != kBf16 && k->scalar_type() != kF32) return not_here();
    if (!k->is_contiguous() || !v->is_contiguous() || k->size(0) != c[1] || k->size(2) != c[2] || k->size(3) != c[3] || k->size(1) > INT32_MAX)
        return not_here();
    const int32_t *start = nullptr;
    if (!ints(a[3], index, c[1], -1, &start)) return not_here();
    if (g_kv4_read(reinterpret_cast<const eagle_kv4_cache *>(c[0]), static_cast<int32_t>(c[1]), static_cast<int32_t>(k->size(1)), start,
                   k->data_ptr(), v->data_ptr(), k->scalar_type() == kF32 ? EAGLE_F32 : EAGLE_BF16, reinterpret_cast<int32_t *>(c[5]),
                   stream(index)) != EAGLE_OK)
        return not_here();
    Py_RETURN_TRUE;
}

// The library's entry points, by address: the library that is loaded, whichever build it is.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
        return nullptr;
    }
    g_rms_norm = reinterpret_cast<decltype(g_rms_norm)>(PyLong_AsVoidPtr(a[0]));
    g_quantize_rows = reinterpret_cast<decltype(g_quantize_rows)>(PyLong_AsVoidPtr(a[1]));
    g_linear = reinterpret_cast<decltype(g_linear)>(PyLong_AsVoidPtr(a[2]));
    g_append_rotary = reinterpret_cast<decltype(g_append_rotary)>(PyLong_AsVoidPtr(a[3]));
    g_kv4_read = reinterpret_cast<decltype(g_kv4_read)>(PyLong_AsVoidPtr(a[4]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

// No C++ exception reaches Python's frames: an allocation that fails, above all, is tried again the long way.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    try {
        PyObject *r = F(self, a, n);
        if (r == Py_NotImplemented) PyErr_Clear();
        return r;
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NOTIMPLEMENTED;
    }
}
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction method() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>));
}

PyMethodDef g_methods[] = {{"bind", method<bind>(), METH_FASTCALL, nullptr},
                           {"quantize_rows", method<quantize_rows>(), METH_FASTCALL, nullptr},
                           {"rms_norm", method<rms_norm>(), METH_FASTCALL, nullptr},
                           {"linear", method<linear>(), METH_FASTCALL, nullptr},
                           {"append_rotary", method<append_rotary>(), METH_FASTCALL, nullptr},
                           {"kv4_read", method<kv4_read>(), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
