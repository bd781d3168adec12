// The tensor forms of the feed-forward block in 16 bits, as binding.cpp has the
// 8-bit layer's: each function takes the Python form's arguments in order, calls
// the C ABI where everything about them is plainly right and returns the status;
// otherwise it returns None and does nothing, and feedforward.py checks argument by
// argument.
#include "binding.h"

#include <initializer_list>

namespace misgemm_binding {
namespace {

using Linear = int (*)(char, char, int, int, int, int, float, const void *, int, const void *, int, int, const void *,
                       int, int, float, const void *, int, void *, int, int, void *, int, float *, int, void *);
using Gated = int (*)(int, int, int, int, const void *, int, const void *, int, const void *, int, int, const void *,
                      const void *, int, int, void *, int, int, void *, int, float *, int, void *, int, float *, int,
                      void *);
using ActBackward = int (*)(int, int, int, const void *, int, int, int, const void *, int, const float *, int, void *,
                            int, void *, int, float, float *, void *);
using GatedBackward = int (*)(int, int, int, const void *, int, int, int, const void *, int, const float *, int,
                              const void *, int, const float *, int, void *, int, void *, int, void *, int, float,
                              float *, float *, void *);

Linear call_linear = nullptr;
Gated call_gated = nullptr;
ActBackward call_act_backward = nullptr;
GatedBackward call_gated_backward = nullptr;

bool half(int type) { return type == 1 || type == 2; }

// 0: 'N', 1: 'T' or 'C', -1: neither.
int trans(PyObject *o) {
    if (!PyUnicode_Check(o) || PyUnicode_GetLength(o) != 1) return -1;
    switch (PyUnicode_ReadChar(o, 0)) {
        case 'N': case 'n': return 0;
        case 'T': case 't': case 'C': case 'c': return 1;
        default: return -1;
    }
}
// The activation's number, -1: none of them.
int act_of(PyObject *o) {
    if (!PyUnicode_Check(o)) return -1;
    const char *names[] = {"none", "relu", "silu", "gelu", "gelu_tanh"};
    for (int i = 0; i < 5; ++i)
        if (PyUnicode_CompareWithASCIIString(o, names[i]) == 0) return i;
    return -1;
}
// A checkpoint: of type `type` without a table, or of 8 bits with one. Not given: true, and left empty.
bool read_kept(PyObject *o, PyObject *table, int rows, int cols, int device, int type, Matrix &z, Matrix &s) {
    if (!given(o)) return !given(table);
    if (!read(o, rows, cols, device, z)) return false;
    if (z.type < 3) return z.type == type && !given(table);
    return given(table) && read_table(table, rows, cols, false, device, s);
}
bool read_bias(PyObject *o, int cols, int device, int type, Matrix &b) {
    return !given(o) || (read_vector(o, cols, device, b) && (b.type == type || b.type == 0));
}
bool all_apart(std::initializer_list<const Matrix *> outs, std::initializer_list<const Matrix *> ins) {
    for (const Matrix *o : outs)
        for (const Matrix *i : ins)
            if (!o->apart(*i)) return false;
    return true;
}
bool distinct(std::initializer_list<const Matrix *> outs) {
    for (const Matrix *const *a = outs.begin(); a != outs.end(); ++a)
        for (const Matrix *const *b = outs.begin(); b != a; ++b)
            if (!(*a)->apart(**b)) return false;
    return true;
}
float *floats(const Matrix &m) { return reinterpret_cast<float *>(m.ptr); }

}  // namespace

// transA, transB, alpha, A, B, beta, C, bias, act, residual, z, scale, stream
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13 || call_linear == nullptr) Py_RETURN_NONE;
    return taken([&](int &status) {
        Matrix A, B, C, bias, R, z, s;
        float alpha, beta;
        void *stream;
        const int ta = trans(a[0]), tb = trans(a[1]), act = act_of(a[8]);
        if (ta < 0 || tb < 0 || act < 0 || !read(a[3], 2, A) || !half(A.type) || !read(a[4], 2, B)) return false;
        const int M = ta ? A.cols : A.rows, K = ta ? A.rows : A.cols, N = tb ? B.rows : B.cols;
        if (B.type != A.type || B.device != A.device || (tb ? B.cols : B.rows) != K) return false;
        if (!read(a[6], M, N, A.device, C) || (C.type != A.type && C.type != 0)) return false;
        if (!read_bias(a[7], N, A.device, A.type, bias)) return false;
        if (given(a[9]) && (!read(a[9], M, N, A.device, R) || R.type != C.type)) return false;
        if (!read_kept(a[10], a[11], M, N, A.device, C.type, z, s)) return false;
        if (!all_apart({&C, &z, &s}, {&A, &B, &bias}) || !distinct({&C, &z, &s})) return false;
        if (!all_apart({&z, &s}, {&R}) || (!C.apart(R) && !C.same(R))) return false;
        if (!number(a[2], alpha) || !number(a[5], beta) || !stream_of(a[12], A.device, &stream)) return false;
        const OnDevice on(A.device);
        if (!on.ok()) return false;
        Py_BEGIN_ALLOW_THREADS
        status = call_linear(ta ? 'T' : 'N', tb ? 'T' : 'N', A.type, M, N, K, alpha, A.ptr, A.ld, B.ptr, B.ld,
                             given(a[7]) ? bias.type : 0, given(a[7]) ? bias.ptr : nullptr, act, C.type, beta,
                             given(a[9]) ? R.ptr : nullptr, R.ld, C.ptr, C.ld, given(a[10]) ? z.type : 0,
                             given(a[10]) ? z.ptr : nullptr, z.ld, floats(s), s.ld, stream);
        Py_END_ALLOW_THREADS
        for (int i : {6, 10, 11}) written(a[i]);
        return true;
    });
}

// A, G, U, h, act, bias_g, bias_u, g, scale_g, u, scale_u, stream
PyObject *gated(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 12 || call_gated == nullptr) Py_RETURN_NONE;
    return taken([&](int &status) {
        Matrix A, G, U, h, bg, bu, g, sg, u, su;
        void *stream;
        const int act = act_of(a[4]);
        if (act < 0 || !read(a[0], 2, A) || !half(A.type) || !read(a[1], 2, G)) return false;
        const int M = A.rows, K = A.cols, N = G.rows;
        if (G.cols != K || G.type != A.type || G.device != A.device) return false;
        if (!read(a[2], N, K, A.device, U) || U.type != A.type) return false;
        if (!read(a[3], M, N, A.device, h) || (h.type != A.type && h.type != 0)) return false;
        if (!read_bias(a[5], N, A.device, A.type, bg) || !read_bias(a[6], N, A.device, A.type, bu)) return false;
        if (given(a[5]) && given(a[6]) && bg.type != bu.type) return false;
        if (given(a[7]) != given(a[9])) return false;
        if (!read_kept(a[7], a[8], M, N, A.device, h.type, g, sg)) return false;
        if (!read_kept(a[9], a[10], M, N, A.device, h.type, u, su) || u.type != g.type) return false;
        if (!all_apart({&h, &g, &sg, &u, &su}, {&A, &G, &U, &bg, &bu}) || !distinct({&h, &g, &sg, &u, &su})) return false;
        if (!stream_of(a[11], A.device, &stream)) return false;
        const OnDevice on(A.device);
        if (!on.ok()) return false;
        Py_BEGIN_ALLOW_THREADS
        status = call_gated(A.type, M, N, K, A.ptr, A.ld, G.ptr, G.ld, U.ptr, U.ld,
                            given(a[5]) ? bg.type : given(a[6]) ? bu.type : 0, given(a[5]) ? bg.ptr : nullptr,
                            given(a[6]) ? bu.ptr : nullptr, act, h.type, h.ptr, h.ld, given(a[7]) ? g.type : 0,
                            given(a[7]) ? g.ptr : nullptr, g.ld, floats(sg), sg.ld, given(a[9]) ? u.ptr : nullptr, u.ld,
                            floats(su), su.ld, stream);
        Py_END_ALLOW_THREADS
        for (int i : {3, 7, 8, 9, 10}) written(a[i]);
        return true;
    });
}

// dy, z, dz, scale, act, y, dbias, beta, stream
PyObject *act_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 9 || call_act_backward == nullptr) Py_RETURN_NONE;
    return taken([&](int &status) {
        Matrix dy, z, dz, s, y, db;
        float beta;
        void *stream;
        const int act = act_of(a[4]);
        if (act < 0 || !read(a[0], 2, dy) || !real(dy.type) || !given(a[1])) return false;
        if (!read_kept(a[1], a[3], dy.rows, dy.cols, dy.device, dy.type, z, s)) return false;
        if (!read(a[2], dy.rows, dy.cols, dy.device, dz) || dz.type != dy.type) return false;
        if (given(a[5]) && (!read(a[5], dy.rows, dy.cols, dy.device, y) || y.type != dy.type)) return false;
        if (given(a[6]) && (!read_vector(a[6], dy.cols, dy.device, db) || db.type != 0)) return false;
        if (!all_apart({&dz, &y}, {&s}) || !all_apart({&db}, {&dy, &z, &s}) || !distinct({&dz, &y, &db})) return false;
        for (const Matrix *o : {&dz, &y})
            for (const Matrix *i : {&dy, &z})
                if (!o->apart(*i) && !(o->same(*i) && o->type == i->type)) return false;
        if (!number(a[7], beta) || !stream_of(a[8], dy.device, &stream)) return false;
        const OnDevice on(dy.device);
        if (!on.ok()) return false;
        Py_BEGIN_ALLOW_THREADS
        status = call_act_backward(dy.type, dy.rows, dy.cols, dy.ptr, dy.ld, act, z.type, z.ptr, z.ld, floats(s), s.ld,
                                   dz.ptr, dz.ld, given(a[5]) ? y.ptr : nullptr, y.ld, beta,
                                   given(a[6]) ? floats(db) : nullptr, stream);
        Py_END_ALLOW_THREADS
        for (int i : {2, 5, 6}) written(a[i]);
        return true;
    });
}

// dh, g, u, dg, du, scale_g, scale_u, act, h, dbias_g, dbias_u, beta, stream
PyObject *gated_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13 || call_gated_backward == nullptr) Py_RETURN_NONE;
    return taken([&](int &status) {
        Matrix dh, g, u, dg, du, sg, su, h, bg, bu;
        float beta;
        void *stream;
        const int act = act_of(a[7]);
        if (act < 0 || !read(a[0], 2, dh) || !real(dh.type) || !given(a[1]) || !given(a[2])) return false;
        const int rows = dh.rows, cols = dh.cols, device = dh.device;
        if (!read_kept(a[1], a[5], rows, cols, device, dh.type, g, sg)) return false;
        if (!read_kept(a[2], a[6], rows, cols, device, dh.type, u, su) || u.type != g.type) return false;
        if (!read(a[3], rows, cols, device, dg) || dg.type != dh.type) return false;
        if (!read(a[4], rows, cols, device, du) || du.type != dh.type) return false;
        if (given(a[8]) && (!read(a[8], rows, cols, device, h) || h.type != dh.type)) return false;
        if (given(a[9]) && (!read_vector(a[9], cols, device, bg) || bg.type != 0)) return false;
        if (given(a[10]) && (!read_vector(a[10], cols, device, bu) || bu.type != 0)) return false;
        if (!all_apart({&dg, &du, &h}, {&sg, &su}) || !all_apart({&bg, &bu}, {&dh, &g, &u, &sg, &su})) return false;
        if (!distinct({&dg, &du, &h, &bg, &bu})) return false;
        for (const Matrix *o : {&dg, &du, &h})
            for (const Matrix *i : {&dh, &g, &u})
                if (!o->apart(*i) && !(o->same(*i) && o->type == i->type)) return false;
        if (!number(a[11], beta) || !stream_of(a[12], device, &stream)) return false;
        const OnDevice on(device);
        if (!on.ok()) return false;
        Py_BEGIN_ALLOW_THREADS
        status = call_gated_backward(dh.type, rows, cols, dh.ptr, dh.ld, act, g.type, g.ptr, g.ld, floats(sg), sg.ld,
                                     u.ptr, u.ld, floats(su), su.ld, dg.ptr, dg.ld, du.ptr, du.ld,
                                     given(a[8]) ? h.ptr : nullptr, h.ld, beta, given(a[9]) ? floats(bg) : nullptr,
                                     given(a[10]) ? floats(bu) : nullptr, stream);
        Py_END_ALLOW_THREADS
        for (int i : {3, 4, 8, 9, 10}) written(a[i]);
        return true;
    });
}

// The addresses of mi_linear, mi_gated, mi_act_backward and mi_gated_backward,
// what gives a device's current stream, and what makes a device current.
PyObject *bind_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *at[4];
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind_linear takes four addresses and two functions");
        return nullptr;
    }
    if (!addresses(a, 4, at)) return nullptr;
    call_linear = reinterpret_cast<Linear>(at[0]);
    call_gated = reinterpret_cast<Gated>(at[1]);
    call_act_backward = reinterpret_cast<ActBackward>(at[2]);
    call_gated_backward = reinterpret_cast<GatedBackward>(at[3]);
    bind_torch(a[4], a[5]);
    Py_RETURN_NONE;
}

}  // namespace misgemm_binding
