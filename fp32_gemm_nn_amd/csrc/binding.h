// What the tensor forms' C++ halves share: arguments read through torch's C++
// interface, the stream and device of a call, outputs' versions.
#ifndef MISGEMM_BINDING_H
#define MISGEMM_BINDING_H

#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace misgemm_binding {

inline PyObject *raw_stream = nullptr;   // device index -> address of torch's current stream
inline PyObject *exchange = nullptr;     // makes a device index current, and returns the one before

constexpr int64_t kMost = 0x7fffffff;

inline int type_of(const at::Tensor &t) {
    switch (t.scalar_type()) {
        case at::kFloat: return 0;
        case at::kBFloat16: return 1;
        case at::kHalf: return 2;
        case at::kFloat8_e4m3fn: return 3;
        case at::kFloat8_e5m2: return 4;
        default: return -1;
    }
}
inline bool real(int type) { return type >= 0 && type <= 2; }

// A matrix (or, with `rows` 1 and a 1-D tensor, a vector) with contiguous rows.
struct Matrix {
    char *ptr = nullptr;
    char *end = nullptr;   // past its last byte; ptr where it is empty
    int rows = 0, cols = 0, ld = 1, type = -1, device = -1;

    bool same(const Matrix &o) const { return ptr == o.ptr && ld == o.ld; }
    bool apart(const Matrix &o) const { return end <= o.ptr || o.end <= ptr || ptr == end || o.ptr == o.end; }
};

inline bool given(PyObject *o) { return o != Py_None; }

inline bool read(PyObject *o, int dims, Matrix &m) {
    if (!THPVariable_Check(o)) return false;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided || t.dim() != dims || t.is_neg()) return false;
    const int64_t rows = dims == 2 ? t.size(0) : 1, cols = t.size(dims - 1);
    if (rows > kMost || cols > kMost) return false;
    if (cols > 1 && t.stride(dims - 1) != 1) return false;
    int64_t ld = rows > 1 ? t.stride(0) : cols;
    if (ld < cols || ld > kMost) return false;
    if (ld < 1) ld = 1;
    m.type = type_of(t);
    m.device = t.get_device();
    m.rows = (int)rows;
    m.cols = (int)cols;
    m.ld = (int)ld;
    m.ptr = static_cast<char *>(t.data_ptr());
    m.end = rows && cols ? m.ptr + ((rows - 1) * ld + cols) * (int64_t)t.element_size() : m.ptr;
    return true;
}
// The same, and of this shape and device.
inline bool read(PyObject *o, int rows, int cols, int device, Matrix &m) {
    return read(o, 2, m) && m.rows == rows && m.cols == cols && m.device == device;
}
inline bool read_vector(PyObject *o, int n, int device, Matrix &m) {
    return read(o, 1, m) && m.cols == n && m.device == device;
}
inline int blocks(int n) { return n / 128 + (n % 128 != 0); }
inline bool read_table(PyObject *o, int rows, int cols, bool tile, int device, Matrix &m) {
    return read(o, tile ? blocks(rows) : blocks(cols), tile ? blocks(cols) : rows, device, m) && m.type == 0;
}

// 0: "row", 1: "tile", -1: neither.
inline int kind(PyObject *o) {
    if (!PyUnicode_Check(o)) return -1;
    if (PyUnicode_CompareWithASCIIString(o, "tile") == 0) return 1;
    return PyUnicode_CompareWithASCIIString(o, "row") == 0 ? 0 : -1;
}
inline bool number(PyObject *o, float &f) {
    if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    f = static_cast<float>(d);
    return true;
}
// `f` of a device index.
inline PyObject *of_device(PyObject *f, int device) {
    PyObject *index = PyLong_FromLong(device);
    PyObject *value = index == nullptr ? nullptr : PyObject_CallOneArg(f, index);
    Py_XDECREF(index);
    return value;
}
inline bool stream_of(PyObject *o, int device, void **stream) {
    PyObject *value = o == Py_None ? of_device(raw_stream, device) : o;
    const bool ok = value != nullptr && PyLong_Check(value);
    if (ok) *stream = PyLong_AsVoidPtr(value);
    if (o == Py_None) Py_XDECREF(value);
    if (!ok || PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return true;
}

// The tensors' device is current while this lives: stream 0, torch's default
// one on every device, is the current device's.
struct OnDevice {
    int before = -1, device;
    explicit OnDevice(int device) : device(device) {
        PyObject *value = of_device(exchange, device);
        if (value != nullptr && PyLong_Check(value)) before = (int)PyLong_AsLong(value);
        Py_XDECREF(value);
        PyErr_Clear();
    }
    bool ok() const { return before >= 0; }
    ~OnDevice() {
        if (before < 0 || before == device) return;
        Py_XDECREF(of_device(exchange, before));
        PyErr_Clear();
    }
};

// For autograd: an output's values are new (an inference tensor has no version).
inline void written(PyObject *o) {
    if (!given(o)) return;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Runs `f`, which fills a status and says whether it made the call.
template <class F> PyObject *taken(F f) {
    int status = 0;
    bool ok = false;
    try {
        ok = f(status);
    } catch (...) {
        ok = false;   // a tensor without storage, for one: nothing was called
    }
    if (!ok) Py_RETURN_NONE;
    return PyLong_FromLong(status);
}

// Keeps what gives a device's current stream, and what makes a device current.
inline void bind_torch(PyObject *stream, PyObject *device) {
    Py_INCREF(stream);
    Py_XDECREF(raw_stream);
    raw_stream = stream;
    Py_INCREF(device);
    Py_XDECREF(exchange);
    exchange = device;
}
// `n` addresses of functions. False: a Python error is set.
inline bool addresses(PyObject *const *a, int n, void **at) {
    for (int i = 0; i < n; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return false;
    }
    return true;
}

// The feed-forward block's forms (binding_linear.cpp).
PyObject *bind_linear(PyObject *, PyObject *const *, Py_ssize_t);
PyObject *linear(PyObject *, PyObject *const *, Py_ssize_t);
PyObject *gated(PyObject *, PyObject *const *, Py_ssize_t);
PyObject *act_backward(PyObject *, PyObject *const *, Py_ssize_t);
PyObject *gated_backward(PyObject *, PyObject *const *, Py_ssize_t);

}  // namespace misgemm_binding

#endif  // MISGEMM_BINDING_H
