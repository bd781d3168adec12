// The tensor forms of the 8-bit linear layer, without the interpreter's time.
//
// A call for one token costs the GPU 3 to 6 us; with shapes, strides and
// pointers of five tensors read in Python and twenty arguments marshalled
// through ctypes it took the host 13 us. Read here through torch's C++ interface
// they take 0.4 us, and a call 3.4 to 3.9 us with its launch. Each function
// takes the Python form's arguments in order, and calls the C ABI where
// everything about them is plainly right: it returns the status. Otherwise it
// returns None and does nothing: fp8.py then checks argument by argument, and
// raises the error or makes the call itself.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

using Gemm = int (*)(int, int, int, int, int, int, int, float, const void *, int, const float *, int, const void *, int,
                     const float *, int, float, void *, int, void *);
using Quantize = int (*)(int, int, int, const void *, int, int, int, void *, int, float *, int, void *, int, float *,
                         int, void *);
using Norm = int (*)(int, int, int, int, const void *, int, const void *, int, const void *, float, void *, int, void *,
                     int, int, void *, int, float *, int, float *, void *);
using Backward = int (*)(int, int, int, int, const void *, int, const void *, int, const void *, const float *,
                         const void *, int, void *, int, float, float *, void *);

Gemm call_gemm = nullptr;
Quantize call_quantize = nullptr;
Norm call_norm = nullptr;
Backward call_backward = nullptr;
PyObject *raw_stream = nullptr;   // device index -> address of torch's current stream
PyObject *exchange = nullptr;     // makes a device index current, and returns the one before

constexpr int64_t kMost = 0x7fffffff;

int type_of(const at::Tensor &t) {
    switch (t.scalar_type()) {
        case at::kFloat: return 0;
        case at::kBFloat16: return 1;
        case at::kHalf: return 2;
        case at::kFloat8_e4m3fn: return 3;
        case at::kFloat8_e5m2: return 4;
        default: return -1;
    }
}
bool real(int type) { return type >= 0 && type <= 2; }

// A matrix (or, with `rows` 1 and a 1-D tensor, a vector) with contiguous rows.
struct Matrix {
    char *ptr = nullptr;
    char *end = nullptr;   // past its last byte; ptr where it is empty
    int rows = 0, cols = 0, ld = 1, type = -1, device = -1;

    bool same(const Matrix &o) const { return ptr == o.ptr && ld == o.ld; }
    bool apart(const Matrix &o) const { return end <= o.ptr || o.end <= ptr || ptr == end || o.ptr == o.end; }
};

bool given(PyObject *o) { return o != Py_None; }

bool read(PyObject *o, int dims, Matrix &m) {
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
bool read(PyObject *o, int rows, int cols, int device, Matrix &m) {
    return read(o, 2, m) && m.rows == rows && m.cols == cols && m.device == device;
}
bool read_vector(PyObject *o, int n, int device, Matrix &m) {
    return read(o, 1, m) && m.cols == n && m.device == device;
}
int blocks(int n) { return n / 128 + (n % 128 != 0); }
bool read_table(PyObject *o, int rows, int cols, bool tile, int device, Matrix &m) {
    return read(o, tile ? blocks(rows) : blocks(cols), tile ? blocks(cols) : rows, device, m) && m.type == 0;
}

// 0: "row", 1: "tile", -1: neither.
int kind(PyObject *o) {
    if (!PyUnicode_Check(o)) return -1;
    if (PyUnicode_CompareWithASCIIString(o, "tile") == 0) return 1;
    return PyUnicode_CompareWithASCIIString(o, "row") == 0 ? 0 : -1;
}
bool number(PyObject *o, float &f) {
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
PyObject *of_device(PyObject *f, int device) {
    PyObject *index = PyLong_FromLong(device);
    PyObject *value = index == nullptr ? nullptr : PyObject_CallOneArg(f, index);
    Py_XDECREF(index);
    return value;
}
bool stream_of(PyObject *o, int device, void **stream) {
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
void written(PyObject *o) {
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

// alpha, A, scale_a, B, scale_b, beta, C, block, stream
PyObject *gemm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9 || call_gemm == nullptr) Py_RETURN_NONE;
    return taken([&](int &status) {
        Matrix A, B, C, sa, sb;
        float alpha, beta;
        void *stream;
        const int block = kind(a[7]);
        if (block < 0 || !read(a[1], 2, A) || A.type < 3 || !read(a[3], 2, B) || B.type < 3) return false;
        if (B.cols != A.cols || B.device != A.device) return false;
        if (!read(a[6], A.rows, B.rows, A.device, C) || !real(C.type)) return false;
        if (!read_table(a[2], A.rows, A.cols, false, A.device, sa)) return false;
        if (!read_table(a[4], B.rows, B.cols, block == 1, A.device, sb)) return false;
        if (!C.apart(A) || !C.apart(B) || !C.apart(sa) || !C.apart(sb)) return false;
        if (!number(a[0], alpha) || !number(a[5], beta) || !stream_of(a[8], A.device, &stream)) return false;
        const OnDevice on(A.device);
        if (!on.ok()) return false;
        Py_BEGIN_ALLOW_THREADS
        status = call_gemm(A.type, B.type, block, C.type, A.rows, B.rows, A.cols, alpha, A.ptr, A.ld,
                           reinterpret_cast<const float *>(sa.ptr), sa.ld, B.ptr, B.ld,
                           reinterpret_cast<const float *>(sb.ptr), sb.ld, beta, C.ptr, C.ld, stream);
        Py_END_ALLOW_THREADS
        written(a[6]);
        return true;
    });
}

// x, q, scale, qt, scale_t, block, stream
PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 7 || call_quantize == nullptr) Py_RETURN_NONE;
    return taken([&](int &status) {
        Matrix x, q, s, qt, st;
        void *stream;
        const int block = kind(a[5]);
        const bool one = given(a[1]), other = given(a[3]);
        if (block < 0 || (!one && !other) || one != given(a[2]) || other != given(a[4])) return false;
        if (!read(a[0], 2, x) || !real(x.type)) return false;
        if (one) {
            if (!read(a[1], x.rows, x.cols, x.device, q) || q.type < 3) return false;
            if (!read_table(a[2], x.rows, x.cols, block == 1, x.device, s)) return false;
            if (!q.apart(x) || !s.apart(x) || !s.apart(q)) return false;
        }
        if (other) {
            if (!read(a[3], x.cols, x.rows, x.device, qt) || qt.type < 3 || (one && qt.type != q.type)) return false;
            if (!read_table(a[4], x.cols, x.rows, block == 1, x.device, st)) return false;
            if (!qt.apart(x) || !st.apart(x) || !st.apart(qt)) return false;
            if (one && (!qt.apart(q) || !qt.apart(s) || !st.apart(q) || !st.apart(s))) return false;
        }
        if (!stream_of(a[6], x.device, &stream)) return false;
        const OnDevice on(x.device);
        if (!on.ok()) return false;
        Py_BEGIN_ALLOW_THREADS
        status = call_quantize(x.type, x.rows, x.cols, x.ptr, x.ld, one ? q.type : qt.type, block, q.ptr, q.ld,
                               reinterpret_cast<float *>(s.ptr), s.ld, qt.ptr, qt.ld,
                               reinterpret_cast<float *>(st.ptr), st.ld, stream);
        Py_END_ALLOW_THREADS
        for (int i : {1, 2, 3, 4}) written(a[i]);
        return true;
    });
}

// x, weight, eps, residual, h, y, q, scale, rstd, stream
PyObject *rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 10 || call_norm == nullptr) Py_RETURN_NONE;
    return taken([&](int &status) {
        Matrix x, w, r, out[5];   // out: h, y, q, scale, rstd
        float eps;
        void *stream;
        if (!read(a[0], 2, x) || !real(x.type)) return false;
        if (!read_vector(a[1], x.cols, x.device, w) || (w.type != x.type && w.type != 0)) return false;
        if (given(a[3]) && (!read(a[3], x.rows, x.cols, x.device, r) || r.type != x.type)) return false;
        for (int i = 0; i < 2; ++i)
            if (given(a[4 + i]) && (!read(a[4 + i], x.rows, x.cols, x.device, out[i]) || out[i].type != x.type))
                return false;
        if ((!given(a[5]) && !given(a[6])) || given(a[6]) != given(a[7])) return false;
        if (given(a[6])) {
            if (!read(a[6], x.rows, x.cols, x.device, out[2]) || out[2].type < 3) return false;
            if (!read_table(a[7], x.rows, x.cols, false, x.device, out[3])) return false;
        }
        if (given(a[8]) && (!read_vector(a[8], x.rows, x.device, out[4]) || out[4].type != 0)) return false;
        for (int i = 0; i < 5; ++i) {
            if (out[i].ptr == out[i].end) continue;
            if (!out[i].apart(w)) return false;
            if (!out[i].apart(x) && !(i == 0 && out[i].same(x))) return false;
            if (!out[i].apart(r) && !(i == 0 && out[i].same(r))) return false;
            for (int j = 0; j < i; ++j)
                if (!out[i].apart(out[j])) return false;
        }
        if (!number(a[2], eps) || !stream_of(a[9], x.device, &stream)) return false;
        const OnDevice on(x.device);
        if (!on.ok()) return false;
        Py_BEGIN_ALLOW_THREADS
        status = call_norm(x.type, w.type, x.rows, x.cols, x.ptr, x.ld, r.ptr, r.ld, w.ptr, eps, out[0].ptr, out[0].ld,
                           out[1].ptr, out[1].ld, given(a[6]) ? out[2].type : 3, out[2].ptr, out[2].ld,
                           reinterpret_cast<float *>(out[3].ptr), out[3].ld, reinterpret_cast<float *>(out[4].ptr),
                           stream);
        Py_END_ALLOW_THREADS
        for (int i : {4, 5, 6, 7, 8}) written(a[i]);
        return true;
    });
}

// dy, h, weight, rstd, dx, dweight, dh, beta, stream
PyObject *rmsnorm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9 || call_backward == nullptr) Py_RETURN_NONE;
    return taken([&](int &status) {
        Matrix dy, h, w, rstd, dx, dw, dh;
        float beta;
        void *stream;
        if (!read(a[0], 2, dy) || !real(dy.type)) return false;
        if (!read(a[1], dy.rows, dy.cols, dy.device, h) || h.type != dy.type) return false;
        if (!read_vector(a[2], dy.cols, dy.device, w) || (w.type != dy.type && w.type != 0)) return false;
        if (!read_vector(a[3], dy.rows, dy.device, rstd) || rstd.type != 0) return false;
        if (!read(a[4], dy.rows, dy.cols, dy.device, dx) || dx.type != dy.type) return false;
        if (given(a[5]) && (!read_vector(a[5], dy.cols, dy.device, dw) || dw.type != 0)) return false;
        if (given(a[6]) && (!read(a[6], dy.rows, dy.cols, dy.device, dh) || dh.type != dy.type)) return false;
        if (!dx.apart(h) || !dx.apart(w) || !dx.apart(rstd) || !dx.apart(dw)) return false;
        if ((!dx.apart(dy) && !dx.same(dy)) || (!dx.apart(dh) && !dx.same(dh))) return false;
        if (!dw.apart(dy) || !dw.apart(h) || !dw.apart(w) || !dw.apart(rstd) || !dw.apart(dh)) return false;
        if (!number(a[7], beta) || !stream_of(a[8], dy.device, &stream)) return false;
        const OnDevice on(dy.device);
        if (!on.ok()) return false;
        Py_BEGIN_ALLOW_THREADS
        status = call_backward(dy.type, w.type, dy.rows, dy.cols, dy.ptr, dy.ld, h.ptr, h.ld, w.ptr,
                               reinterpret_cast<const float *>(rstd.ptr), dh.ptr, dh.ld, dx.ptr, dx.ld, beta,
                               reinterpret_cast<float *>(dw.ptr), stream);
        Py_END_ALLOW_THREADS
        for (int i : {4, 5}) written(a[i]);
        return true;
    });
}

// The addresses of mi_fp8_gemm, mi_fp8_quantize, mi_rmsnorm and
// mi_rmsnorm_backward, what gives a device's current stream, and what makes a
// device current.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *at[4];
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind takes four addresses and two functions");
        return nullptr;
    }
    for (int i = 0; i < 4; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    call_gemm = reinterpret_cast<Gemm>(at[0]);
    call_quantize = reinterpret_cast<Quantize>(at[1]);
    call_norm = reinterpret_cast<Norm>(at[2]);
    call_backward = reinterpret_cast<Backward>(at[3]);
    Py_INCREF(a[4]);
    Py_XDECREF(raw_stream);
    raw_stream = a[4];
    Py_INCREF(a[5]);
    Py_XDECREF(exchange);
    exchange = a[5];
    Py_RETURN_NONE;
}

#define FORM(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FORM(bind), FORM(gemm), FORM(quantize), FORM(rmsnorm), FORM(rmsnorm_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
