"""The 8-bit linear layer: quantisation, block-scaled products, RMS norm.

Functions with the C names (``include/misgemm_fp8.h``) take raw device
pointers (ints) and return the C status code. The tensor forms beside them
check shapes, types, devices and overlap, enqueue on ``stream`` (default: the
current torch stream of the tensors' device, which is current for the call:
stream 0 is its default stream) and raise on an error. Outputs are tensors of
the caller's, written in place; nothing is computed here.
Autograd records none of these calls: use them in a torch.autograd.Function or
with gradients of your own. Outputs' version counters move, as with torch's
in-place operators, so that a backward pass that saved one of them raises.
What is plainly right goes through a C++ binding, which reads the arguments in
0.4 us (a call takes the host 3.4 to 3.9 us with its launch); the checks below
name what is not, and decide the rest (memory that interleaves).

An 8-bit matrix is a pair (q, scale): q of torch.float8_e4m3fn or
torch.float8_e5m2 with contiguous rows, and a float32 table with a scale for

* ``block="row"``: each row and 128 columns, kept as (ceil(cols/128), rows);
* ``block="tile"``: each 128 x 128 block, kept as (ceil(rows/128), ceil(cols/128)).

``fp8_empty`` makes such a pair with rows 16 bytes aligned, as the product
reads them fastest.
"""
from __future__ import annotations

import torch

from . import MisgemmError, load_library, mi_fp8_gemm, mi_fp8_quantize, mi_rmsnorm, mi_rmsnorm_backward

_REAL = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_F8 = {torch.float8_e4m3fn: 3, torch.float8_e5m2: 4}
_BLOCK = {"row": 0, "tile": 1}


_native = None


def _load_native():
    """The tensor forms' C++ half (csrc/binding.cpp), bound to the library; raise if it is not built."""
    global _native
    import ctypes
    import importlib.machinery
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")
    lib = load_library()
    if not os.path.exists(path):
        raise RuntimeError(f"binding not built: {path} is missing. "
                           "Run `python -m fp32_gemm_nn_amd.build` (or __graft_entry__.build()).")
    loader = importlib.machinery.ExtensionFileLoader("_binding", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_binding", loader))
    loader.exec_module(module)
    address = [ctypes.cast(f, ctypes.c_void_p).value
               for f in (lib.mi_fp8_gemm, lib.mi_fp8_quantize, lib.mi_rmsnorm, lib.mi_rmsnorm_backward)]
    module.bind(*address, getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: None),
                getattr(torch._C, "_cuda_exchangeDevice", lambda index: None))
    _native = module
    return module


class _Arg:
    """A checked matrix: its address, leading dimension, and the bytes it spans."""
    __slots__ = ("ptr", "ld", "end", "row", "rows")

    def __init__(self, name, t, shape, types, device):
        if t.dtype not in types:
            raise TypeError(f"{name} must be {' or '.join(str(d) for d in types)}, not {t.dtype}")
        if t.device != device:
            if t.device.type != "cuda":
                raise ValueError(f"{name} must be a device tensor")
            raise ValueError(f"{name} must be on {device}, not {t.device}")
        if t.shape != shape:
            raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")
        if t.is_neg():
            raise ValueError(f"{name} stands for the negative of its memory: pass {name}.resolve_neg()")
        size = t.element_size()
        if len(shape) == 1:
            n = shape[0]
            if n > 1 and t.stride(0) != 1:
                raise ValueError(f"{name} must be contiguous")
            self.rows, self.ld = (1, n)
        else:
            self.rows, n = shape
            step, one = t.stride()
            if n > 1 and one != 1:
                raise ValueError(f"{name} must have contiguous rows (stride(1) == 1)")
            self.ld = step if self.rows > 1 else n
            if self.ld < n:
                raise ValueError(f"{name} must have distinct rows: its row stride {step} is less than their length {n}")
        self.ptr = t.data_ptr()
        self.ld = max(self.ld, 1)
        self.row = n * size
        self.end = self.ptr + ((self.rows - 1) * self.ld + n) * size if self.rows and n else self.ptr


def _share(x: _Arg, y: _Arg, x_size: int, y_size: int) -> bool:
    """Whether two matrices have a byte in common. Their spans mostly do not;
    where they do, columns of one buffer side by side are told from overlap
    row by row, as sgemm does."""
    if x.end <= y.ptr or y.end <= x.ptr or x.ptr == x.end or y.ptr == y.end:
        return False
    import numpy as np

    start = x.ptr + x.ld * x_size * np.arange(x.rows, dtype=np.int64)
    step = y.ld * y_size
    hi = np.minimum((start + x.row - y.ptr - 1) // step, y.rows - 1)
    lo = np.maximum((start - y.ptr - y.row) // step + 1, 0)
    return bool(np.any(lo <= hi))


def _apart(outs, ins):
    """Raise where an output shares memory with an input or another output. Each is (name, arg, element size)."""
    for k, (name, x, xs) in enumerate(outs):
        for other, y, ys in ins:
            if x.ptr < y.end and y.ptr < x.end and _share(x, y, xs, ys):
                raise ValueError(f"{name} must not overlap {other}")
        for other, y, ys in outs[:k]:
            if x.ptr < y.end and y.ptr < x.end and _share(x, y, xs, ys):
                raise ValueError(f"{name} must not overlap {other}")


def _enqueue(entry, device, stream, *args) -> int:
    """Call a C function on a stream with its device current: stream 0 (torch's default) is the current device's."""
    with torch.cuda.device(device):
        return entry(*args, torch.cuda.current_stream(device).cuda_stream if stream is None else stream)


def _on_device(name, t):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    return t.device


def _matrix(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    return t.shape


def _table(rows, cols, block):
    if block not in _BLOCK:
        raise ValueError(f"block must be 'row' or 'tile', not {block!r}")
    b = (cols + 127) // 128
    return torch.Size((b, rows)) if block == "row" else torch.Size(((rows + 127) // 128, b))


def _raise(rc, where):
    if rc != 0:
        raise MisgemmError(rc, where)


def _written(*outs):
    """For autograd: these tensors' values are new (an inference tensor has no version)."""
    for t in outs:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def fp8_empty(rows: int, cols: int, block: str = "row", dtype=torch.float8_e4m3fn, device="cuda"):
    """An uninitialised 8-bit matrix (q, scale), its rows a multiple of 16 bytes apart."""
    q = torch.empty(rows, cols + -cols % 16, dtype=dtype, device=device)[:, :cols]
    return q, torch.empty(_table(rows, cols, block), dtype=torch.float32, device=device)


def fp8_quantize(x, q=None, scale=None, qt=None, scale_t=None, block: str = "row", stream=None):
    """(q, scale) <- x in 8 bits, and/or (qt, scale_t) <- its transpose in 8 bits, from one pass over x.

    x is float32, bfloat16 or float16. Of each block, a = max(max|x|, 2^-100), scale = a / T and
    q = rn(x * (T / a)), with T = 448 (E4M3) or 57344 (E5M2). qt's row blocks run along x's rows.
    Returns the tensors that were given, in that order.
    """
    rc = (_native or _load_native()).quantize(x, q, scale, qt, scale_t, block, stream)
    if rc is not None:
        _raise(rc, "mi_fp8_quantize")
        return (q, scale) if qt is None else (qt, scale_t) if q is None else (q, scale, qt, scale_t)
    rows, cols = _matrix("x", x)
    dev = _on_device("x", x)
    a = _Arg("x", x, x.shape, _REAL, dev)
    ins = [("x", a, x.element_size())]
    if q is None and qt is None:
        raise ValueError("one of q and qt must be given")
    if q is not None and qt is not None and q.dtype != qt.dtype:
        raise TypeError(f"q and qt must have one type, not {q.dtype} and {qt.dtype}")
    outs, args, given = [], [], []
    for name, t, s, r, c in (("q", q, scale, rows, cols), ("qt", qt, scale_t, cols, rows)):
        sname = "scale" if name == "q" else "scale_t"
        if (t is None) != (s is None):
            raise ValueError(f"{name} and {sname} go together")
        if t is None:
            args += [0, 0, 0, 0]
            continue
        o = _Arg(name, t, (r, c), _F8, dev)
        z = _Arg(sname, s, _table(r, c, block), (torch.float32,), dev)
        outs += [(name, o, 1), (sname, z, 4)]
        args += [o.ptr, o.ld, z.ptr, z.ld]
        given += [t, s]
    _apart(outs, ins)
    _raise(_enqueue(mi_fp8_quantize, dev, stream, _REAL[x.dtype], rows, cols, a.ptr, max(a.ld, cols),
                    _F8[given[0].dtype], _BLOCK[block], *args), "mi_fp8_quantize")
    _written(*given)
    return tuple(given)


def fp8_gemm(alpha: float, A, scale_a, B, scale_b, beta: float, C, block: str = "tile", stream=None):
    """C <- alpha * A @ B^T + beta * C on 8-bit matrices A (M x K) and B (N x K); returns C.

    scale_a has a scale for each row and 128 of k; scale_b is a table of kind ``block``. C is M x N in
    float32, bfloat16 or float16; blocks are scaled and added in FP32. beta == 0: C is not read.
    A block's two scales are multiplied first: their product has to lie between 2^-126 and 2^128.
    """
    rc = (_native or _load_native()).gemm(alpha, A, scale_a, B, scale_b, beta, C, block, stream)
    if rc is not None:
        _raise(rc, "mi_fp8_gemm")
        return C
    M, K = _matrix("A", A)
    N = _matrix("B", B)[0]
    dev = _on_device("A", A)
    a = _Arg("A", A, A.shape, _F8, dev)
    sa = _Arg("scale_a", scale_a, _table(M, K, "row"), (torch.float32,), dev)
    b = _Arg("B", B, (N, K), _F8, dev)
    sb = _Arg("scale_b", scale_b, _table(N, K, block), (torch.float32,), dev)
    c = _Arg("C", C, (M, N), _REAL, dev)
    _apart([("C", c, C.element_size())], [("A", a, 1), ("scale_a", sa, 4), ("B", b, 1), ("scale_b", sb, 4)])
    _raise(_enqueue(mi_fp8_gemm, dev, stream, _F8[A.dtype], _F8[B.dtype], _BLOCK[block], _REAL[C.dtype], M, N, K, alpha,
                    a.ptr, a.ld, sa.ptr, sa.ld, b.ptr, b.ld, sb.ptr, sb.ld, beta, c.ptr, c.ld), "mi_fp8_gemm")
    _written(C)
    return C


def _same(x: _Arg, y: _Arg) -> bool:
    return x.ptr == y.ptr and x.ld == y.ld


def rmsnorm(x, weight, eps: float, residual=None, h=None, y=None, q=None, scale=None, rstd=None, stream=None):
    """h <- x + residual, y <- h / sqrt(mean(h^2) + eps) * weight by rows, (q, scale) <- y in 8 bits.

    x, residual, h and y share a type (float32, bfloat16 or float16); weight has that type or float32.
    h, y, (q, scale) and rstd are written where given (y or q must be). h may be x or residual itself.
    q is quantised from y in FP32, with scales of kind "row". rstd is for ``rmsnorm_backward``.
    """
    rc = (_native or _load_native()).rmsnorm(x, weight, eps, residual, h, y, q, scale, rstd, stream)
    if rc is not None:
        return _raise(rc, "mi_rmsnorm")
    rows, cols = _matrix("x", x)
    dev = _on_device("x", x)
    size, types = x.element_size(), (x.dtype,)
    ax = _Arg("x", x, x.shape, _REAL, dev)
    ins = [("x", ax, size)]
    aw = _Arg("weight", weight, (cols,), (x.dtype, torch.float32), dev)
    ins.append(("weight", aw, weight.element_size()))
    ptr, ld, outs = {}, {}, []
    for name, t in (("residual", residual), ("h", h), ("y", y)):
        ptr[name], ld[name] = 0, 0
        if t is not None:
            a = _Arg(name, t, (rows, cols), types, dev)
            ptr[name], ld[name] = a.ptr, a.ld
            (ins if name == "residual" else outs).append((name, a, size))
    if y is None and q is None:
        raise ValueError("one of y and q must be given")
    if (q is None) != (scale is None):
        raise ValueError("q and scale go together")
    qa = [3, 0, 0, 0, 0]
    if q is not None:
        aq = _Arg("q", q, (rows, cols), _F8, dev)
        az = _Arg("scale", scale, _table(rows, cols, "row"), (torch.float32,), dev)
        outs += [("q", aq, 1), ("scale", az, 4)]
        qa = [_F8[q.dtype], aq.ptr, aq.ld, az.ptr, az.ld]
    if rstd is not None:
        outs.append(("rstd", _Arg("rstd", rstd, (rows,), (torch.float32,), dev), 4))
    for name, o, s in outs:
        _apart([(name, o, s)], [i for i in ins if not (name == "h" and i[0] != "weight" and _same(o, i[1]))])
    _apart(outs, [])
    _raise(_enqueue(mi_rmsnorm, dev, stream, _REAL[x.dtype], _REAL[weight.dtype], rows, cols, ax.ptr, max(ax.ld, cols),
                    ptr["residual"], ld["residual"], aw.ptr, eps, ptr["h"], ld["h"], ptr["y"], ld["y"], *qa,
                    0 if rstd is None else rstd.data_ptr()), "mi_rmsnorm")
    _written(h, y, q, scale, rstd)


def rmsnorm_backward(dy, h, weight, rstd, dx, dweight=None, dh=None, beta: float = 0.0, stream=None):
    """dx <- gradient of h through ``rmsnorm``'s y, plus dh; dweight <- the weight's, plus beta * dweight.

    dy, h, dx and dh share a type; h and rstd are as ``rmsnorm`` wrote them. dx may be dy or dh itself.
    dweight is float32, or None where it is not wanted.
    """
    rc = (_native or _load_native()).rmsnorm_backward(dy, h, weight, rstd, dx, dweight, dh, beta, stream)
    if rc is not None:
        return _raise(rc, "mi_rmsnorm_backward")
    rows, cols = _matrix("dy", dy)
    dev = _on_device("dy", dy)
    size, types = dy.element_size(), (dy.dtype,)
    ady = _Arg("dy", dy, dy.shape, _REAL, dev)
    ah = _Arg("h", h, (rows, cols), types, dev)
    aw = _Arg("weight", weight, (cols,), (dy.dtype, torch.float32), dev)
    ar = _Arg("rstd", rstd, (rows,), (torch.float32,), dev)
    ins = [("dy", ady, size), ("h", ah, size), ("weight", aw, weight.element_size()), ("rstd", ar, 4)]
    adh = None
    if dh is not None:
        adh = _Arg("dh", dh, (rows, cols), types, dev)
        ins.append(("dh", adh, size))
    adx = _Arg("dx", dx, (rows, cols), types, dev)
    outs = [("dx", adx, size)]
    if dweight is not None:
        outs.append(("dweight", _Arg("dweight", dweight, (cols,), (torch.float32,), dev), 4))
    _apart(outs[:1], [i for i in ins if not (i[0] in ("dy", "dh") and _same(adx, i[1]))])
    _apart(outs[1:], ins)
    _apart(outs, [])
    _raise(_enqueue(mi_rmsnorm_backward, dev, stream, _REAL[dy.dtype], _REAL[weight.dtype], rows, cols, ady.ptr,
                    max(ady.ld, cols), ah.ptr, max(ah.ld, cols), aw.ptr, ar.ptr, 0 if adh is None else adh.ptr,
                    0 if adh is None else adh.ld, adx.ptr, max(adx.ld, cols), beta,
                    0 if dweight is None else dweight.data_ptr()), "mi_rmsnorm_backward")
    _written(dx, dweight)
