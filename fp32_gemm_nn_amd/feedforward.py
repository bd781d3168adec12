"""The feed-forward block in 16 bits: products with their epilogue, the gated block, and the backward pass of both.

Functions with the C names (``include/misgemm_linear.h``) take raw device
pointers (ints) and return the C status code. The tensor forms beside them are
as those of the 8-bit layer (``fp8``): they check shapes, types, devices and
overlap, enqueue on ``stream`` (default: the current torch stream of the
tensors' device, which is current for the call), write outputs of the caller's
in place and raise on an error. Autograd records none of these calls; outputs'
version counters move.

What the forward pass keeps for the backward pass is a matrix, or an 8-bit pair
(q, scale) with a scale for each row and 128 columns (``fp8_empty(rows, cols)``).

Activations: "none", "relu", "silu" (z / (1 + e^-z)), "gelu" (with erf) and
"gelu_tanh" (its approximation).
"""
from __future__ import annotations

import torch

from . import load_library, mi_act_backward, mi_gated, mi_gated_backward, mi_linear
from .fp8 import _F8, _REAL, _Arg, _apart, _enqueue, _load_native as _load_fp8, _matrix, _on_device, _raise, _same, _table, _written

_HALF = {torch.bfloat16: 1, torch.float16: 2}
_ACT = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

_native = None


def _load_native():
    """The tensor forms' C++ half (csrc/binding_linear.cpp), bound to the library; raise if it is not built."""
    global _native
    import ctypes

    module, lib = _load_fp8(), load_library()
    address = [ctypes.cast(f, ctypes.c_void_p).value
               for f in (lib.mi_linear, lib.mi_gated, lib.mi_act_backward, lib.mi_gated_backward)]
    module.bind_linear(*address, getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: None),
                       getattr(torch._C, "_cuda_exchangeDevice", lambda index: None))
    _native = module
    return module


def _act(act):
    if act not in _ACT:
        raise ValueError(f"act must be one of {', '.join(map(repr, _ACT))}, not {act!r}")
    return _ACT[act]


def _trans(name, t):
    if t not in ("N", "n", "T", "t", "C", "c"):
        raise ValueError(f"{name} must be 'N' or 'T', not {t!r}")
    return t not in ("N", "n")


def _kept(name, sname, t, scale, shape, type, dev):
    """Checks of a checkpoint: (number of its type, [(name, arg, element size), ...], C arguments)."""
    if t is None:
        if scale is not None:
            raise ValueError(f"{sname} goes with {name}")
        return 0, [], [0, 0, 0, 0]
    a = _Arg(name, t, shape, (type, *_F8), dev)
    if t.dtype not in _F8:
        if scale is not None:
            raise ValueError(f"{sname} goes with {name} in 8 bits")
        return _REAL[type], [(name, a, t.element_size())], [a.ptr, a.ld, 0, 0]
    if scale is None:
        raise ValueError(f"{name} in 8 bits and {sname} go together")
    s = _Arg(sname, scale, _table(*shape, "row"), (torch.float32,), dev)
    return _F8[t.dtype], [(name, a, 1), (sname, s, 4)], [a.ptr, a.ld, s.ptr, s.ld]


def _bias(name, t, n, type, dev):
    if t is None:
        return None, []
    a = _Arg(name, t, (n,), (type, torch.float32), dev)
    return a, [(name, a, t.element_size())]


def _sums(name, t, n, dev):
    if t is None:
        return 0, []
    a = _Arg(name, t, (n,), (torch.float32,), dev)
    return a.ptr, [(name, a, 4)]


def linear(transA: str, transB: str, alpha: float, A, B, beta: float, C, bias=None, act: str = "none", residual=None,
           z=None, scale=None, stream=None):
    """C <- act(alpha * op(A) @ op(B) + bias) + beta * residual (or beta * C without one); returns C.

    A and B are bfloat16 or float16 matrices as they are stored (with op 'T', transposes of them are multiplied: a layer
    whose weight is outputs x inputs takes 'N', 'T'). C and residual have that type or float32, as bias does. residual may be C.
    z: where the activation's argument goes, for ``act_backward``: a matrix of C's type, or an 8-bit one with ``scale``.
    """
    rc = (_native or _load_native()).linear(transA, transB, alpha, A, B, beta, C, bias, act, residual, z, scale, stream)
    if rc is not None:
        _raise(rc, "mi_linear")
        return C
    ta, tb, f = _trans("transA", transA), _trans("transB", transB), _act(act)
    M, K = _matrix("A", A)[::-1] if ta else _matrix("A", A)
    N = _matrix("B", B)[0 if tb else 1]
    dev = _on_device("A", A)
    a = _Arg("A", A, A.shape, _HALF, dev)
    b = _Arg("B", B, (N, K) if tb else (K, N), (A.dtype,), dev)
    c = _Arg("C", C, (M, N), (A.dtype, torch.float32), dev)
    v, ins = _bias("bias", bias, N, A.dtype, dev)
    ins += [("A", a, 2), ("B", b, 2)]
    size = C.element_size()
    ztype, kept, zargs = _kept("z", "scale", z, scale, (M, N), C.dtype, dev)
    outs = [("C", c, size), *kept]
    _apart(outs, ins)
    r = None
    if residual is not None:
        r = _Arg("residual", residual, (M, N), (C.dtype,), dev)
        _apart(kept, [("residual", r, size)])
        if not _same(c, r):
            _apart(outs[:1], [("residual", r, size)])
    _raise(_enqueue(mi_linear, dev, stream, "T" if ta else "N", "T" if tb else "N", _HALF[A.dtype], M, N, K, alpha,
                    a.ptr, a.ld, b.ptr, b.ld, 0 if v is None else _REAL[bias.dtype], 0 if v is None else v.ptr, f,
                    _REAL[C.dtype], beta, 0 if r is None else r.ptr, 0 if r is None else max(r.ld, N), c.ptr, max(c.ld, N),
                    ztype, *zargs), "mi_linear")
    _written(C, z, scale)
    return C


def gated(A, G, U, h, act: str = "silu", bias_g=None, bias_u=None, g=None, scale_g=None, u=None, scale_u=None, stream=None):
    """h <- act(A @ G^T + bias_g) * (A @ U^T + bias_u), in one kernel; returns h.

    A (M x K), G and U (N x K each, outputs x inputs; they may be parts of one matrix) are bfloat16 or float16, h (M x N) and the biases
    that or float32. g and u: where the two projections go, for ``gated_backward``: matrices of h's type, or 8-bit ones with scales.
    """
    rc = (_native or _load_native()).gated(A, G, U, h, act, bias_g, bias_u, g, scale_g, u, scale_u, stream)
    if rc is not None:
        _raise(rc, "mi_gated")
        return h
    f = _act(act)
    M, K = _matrix("A", A)
    N = _matrix("G", G)[0]
    dev = _on_device("A", A)
    a = _Arg("A", A, A.shape, _HALF, dev)
    w = [_Arg(n, t, (N, K), (A.dtype,), dev) for n, t in (("G", G), ("U", U))]
    c = _Arg("h", h, (M, N), (A.dtype, torch.float32), dev)
    bg, ins = _bias("bias_g", bias_g, N, A.dtype, dev)
    bu, more = _bias("bias_u", bias_u, N, A.dtype, dev)
    if bg is not None and bu is not None and bias_g.dtype != bias_u.dtype:
        raise TypeError(f"bias_g and bias_u must have one type, not {bias_g.dtype} and {bias_u.dtype}")
    ins += [*more, ("A", a, 2), ("G", w[0], 2), ("U", w[1], 2)]
    if (g is None) != (u is None):
        raise ValueError("g and u go together")
    if g is not None and g.dtype != u.dtype:
        raise TypeError(f"g and u must have one type, not {g.dtype} and {u.dtype}")
    ztype, kept, gargs = _kept("g", "scale_g", g, scale_g, (M, N), h.dtype, dev)
    _, also, uargs = _kept("u", "scale_u", u, scale_u, (M, N), h.dtype, dev)
    _apart([("h", c, h.element_size()), *kept, *also], ins)
    biastype = _REAL[(bias_g if bg is not None else bias_u).dtype] if bg is not None or bu is not None else 0
    _raise(_enqueue(mi_gated, dev, stream, _HALF[A.dtype], M, N, K, a.ptr, a.ld, w[0].ptr, w[0].ld, w[1].ptr, w[1].ld, biastype,
                    0 if bg is None else bg.ptr, 0 if bu is None else bu.ptr, f, _REAL[h.dtype], c.ptr, max(c.ld, N), ztype,
                    *gargs, *uargs), "mi_gated")
    _written(h, g, scale_g, u, scale_u)
    return h


def _in_place(outs, ins):
    """Outputs that are not an input itself (and of its type) are apart from it."""
    for o in outs:
        _apart([o], [i for i in ins if not (_same(o[1], i[1]) and o[2] == i[2])])


def act_backward(dy, z, dz, scale=None, act: str = "none", y=None, dbias=None, beta: float = 0.0, stream=None):
    """dz <- dy * act'(z), y <- act(z), dbias <- the sum of dz over the rows, plus beta * dbias; returns dz.

    z is what ``linear`` kept: a matrix of dy's type (float32, bfloat16 or float16), or an 8-bit one with ``scale``. dz, and
    y where it is wanted, have dy's type; dbias is float32. dz or y may be dy or z itself.
    """
    rc = (_native or _load_native()).act_backward(dy, z, dz, scale, act, y, dbias, beta, stream)
    if rc is not None:
        _raise(rc, "mi_act_backward")
        return dz
    f = _act(act)
    rows, cols = _matrix("dy", dy)
    dev = _on_device("dy", dy)
    size = dy.element_size()
    a = _Arg("dy", dy, dy.shape, _REAL, dev)
    if z is None:
        raise ValueError("z must be given")
    ztype, kept, zargs = _kept("z", "scale", z, scale, (rows, cols), dy.dtype, dev)
    d = _Arg("dz", dz, (rows, cols), (dy.dtype,), dev)
    outs, yargs = [("dz", d, size)], [0, 0]
    if y is not None:
        o = _Arg("y", y, (rows, cols), (dy.dtype,), dev)
        outs.append(("y", o, size))
        yargs = [o.ptr, max(o.ld, cols)]
    b, sums = _sums("dbias", dbias, cols, dev)
    _in_place(outs, [("dy", a, size), *kept])
    _apart(sums, [("dy", a, size), *kept])
    _apart([*outs, *sums], [])
    _raise(_enqueue(mi_act_backward, dev, stream, _REAL[dy.dtype], rows, cols, a.ptr, max(a.ld, cols), f, ztype, zargs[0], max(zargs[1], cols),
                    *zargs[2:], d.ptr, max(d.ld, cols), *yargs, beta, b), "mi_act_backward")
    _written(dz, y, dbias)
    return dz


def gated_backward(dh, g, u, dg, du, scale_g=None, scale_u=None, act: str = "silu", h=None, dbias_g=None, dbias_u=None,
                   beta: float = 0.0, stream=None):
    """dg <- dh * u * act'(g), du <- dh * act(g), h <- act(g) * u; returns (dg, du).

    dbias_g and dbias_u <- the sums of dg and du over the rows, plus beta times what they were. g and u are what ``gated`` kept:
    matrices of dh's type (float32, bfloat16 or float16), or 8-bit ones with scales. dg, du and h have dh's type, and may each be
    dh, g or u itself; the sums are float32.
    """
    rc = (_native or _load_native()).gated_backward(dh, g, u, dg, du, scale_g, scale_u, act, h, dbias_g, dbias_u, beta, stream)
    if rc is not None:
        _raise(rc, "mi_gated_backward")
        return dg, du
    f = _act(act)
    rows, cols = _matrix("dh", dh)
    dev = _on_device("dh", dh)
    size = dh.element_size()
    a = _Arg("dh", dh, dh.shape, _REAL, dev)
    if g is None or u is None:
        raise ValueError("g and u must be given")
    if g.dtype != u.dtype:
        raise TypeError(f"g and u must have one type, not {g.dtype} and {u.dtype}")
    ztype, kept, gargs = _kept("g", "scale_g", g, scale_g, (rows, cols), dh.dtype, dev)
    _, also, uargs = _kept("u", "scale_u", u, scale_u, (rows, cols), dh.dtype, dev)
    ins = [("dh", a, size), *kept, *also]
    outs, args = [], []
    for name, t in (("dg", dg), ("du", du), ("h", h)):
        if t is None and name == "h":
            args += [0, 0]
            continue
        o = _Arg(name, t, (rows, cols), (dh.dtype,), dev)
        outs.append((name, o, size))
        args += [o.ptr, max(o.ld, cols)]
    bg, sums = _sums("dbias_g", dbias_g, cols, dev)
    bu, more = _sums("dbias_u", dbias_u, cols, dev)
    sums += more
    _in_place(outs, ins)
    _apart(sums, ins)
    _apart([*outs, *sums], [])
    for x in (gargs, uargs):
        x[1] = max(x[1], cols)
    _raise(_enqueue(mi_gated_backward, dev, stream, _REAL[dh.dtype], rows, cols, a.ptr, max(a.ld, cols), f, ztype, *gargs, *uargs, *args,
                    beta, bg, bu), "mi_gated_backward")
    _written(dg, du, h, dbias_g, dbias_u)
    return dg, du
