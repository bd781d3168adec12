"""The 8-bit linear layer's entry points on the host: what they refuse.

Nothing here launches a kernel: every C call below fails validation or takes
a quick return, both of which happen before any HIP call, and the tensor
forms are given tensors that they refuse.
"""
import pytest

import fp32_gemm_nn_amd as mg
from fp32_gemm_nn_amd import fp8

torch = pytest.importorskip("torch")

P = 0x10000   # never dereferenced

QUANT = dict(xtype=1, rows=300, cols=200, x=P, ldx=200, ftype=3, block=0, q=P, ldq=200, scale=P, lds=300, qt=P,
             ldqt=300, scale_t=P, lds_t=200)
GEMM = dict(atype=3, btype=4, block=1, ctype=1, M=8, N=300, K=200, alpha=1.0, A=P, lda=200, scaleA=P, ldsa=8, B=P,
            ldb=200, scaleB=P, ldsb=2, beta=0.0, C=P, ldc=300)
NORM = dict(type=1, wtype=0, rows=3, cols=200, x=P, ldx=200, residual=P, ldr=200, weight=P, eps=1e-5, h=P, ldh=200,
            y=P, ldy=200, ftype=3, q=P, ldq=200, scale=P, lds=3, rstd=P)
BACK = dict(type=1, wtype=1, rows=3, cols=200, dy=P, lddy=200, h=P, ldh=200, weight=P, rstd=P, dh=P, lddh=200, dx=P,
            lddx=200, beta=0.0, dweight=P)


@pytest.mark.parametrize("kw,code", [
    (dict(xtype=3), -30), (dict(xtype=-1), -30), (dict(rows=-1), -32), (dict(cols=-1), -33), (dict(x=0), -34),
    (dict(ldx=199), -37), (dict(ftype=1), -30), (dict(block=2), -31), (dict(q=0, qt=0), -35), (dict(ldq=199), -37),
    (dict(scale=0), -36), (dict(lds=299), -38), (dict(block=1, lds=1), -38), (dict(ldqt=299), -37),
    (dict(scale_t=0), -36), (dict(lds_t=199), -38), (dict(block=1, lds_t=2), -38),
    (dict(rows=65536 * 128, lds=2**30, ldqt=2**30), -21),
    # The first bad argument wins, and nothing is refused of what is not wanted.
    (dict(rows=-1, x=0), -32), (dict(q=0, ldq=0, scale=0, lds=0, lds_t=0), -38),
])
def test_quantize_refuses(kw, code):
    assert fp8.mi_fp8_quantize(**{**QUANT, **kw}) == code
    assert mg.mi_sgemm_status_string(code) not in ("", "unknown status")


@pytest.mark.parametrize("kw,code", [
    (dict(atype=0), -30), (dict(btype=2), -30), (dict(block=-1), -31), (dict(ctype=3), -30), (dict(M=-1), -3),
    (dict(N=-1), -4), (dict(K=-1), -5), (dict(A=0), -7), (dict(lda=199), -8), (dict(scaleA=0), -36),
    (dict(ldsa=7), -38), (dict(B=0), -9), (dict(ldb=199), -10), (dict(scaleB=0), -36), (dict(ldsb=1), -38),
    (dict(block=0, ldsb=299), -38), (dict(C=0), -12), (dict(ldc=299), -13), (dict(alpha=0.0, A=0, ldc=0), -13),
    (dict(N=2**31 - 1, ldc=2**31 - 1), -21), (dict(K=2**31 - 1, lda=2**31 - 1, ldb=2**31 - 1, ldsb=2**30), -21),
    (dict(M=2**20, N=2**20, ldsa=2**20, ldc=2**20, ldsb=2**20), -21),
])
def test_gemm_refuses(kw, code):
    assert fp8.mi_fp8_gemm(**{**GEMM, **kw}) == code
    assert mg.mi_sgemm_status_string(code) not in ("", "unknown status")


@pytest.mark.parametrize("kw,code", [
    (dict(type=4), -30), (dict(wtype=2), -30), (dict(rows=-1), -32), (dict(cols=-1), -33), (dict(x=0), -34),
    (dict(ldx=199), -37), (dict(ldr=199), -37), (dict(weight=0), -34), (dict(ldh=1), -37), (dict(ldy=1), -37),
    (dict(y=0, q=0), -35), (dict(ftype=0), -30), (dict(ldq=199), -37), (dict(scale=0), -36), (dict(lds=2), -38),
])
def test_norm_refuses(kw, code):
    assert fp8.mi_rmsnorm(**{**NORM, **kw}) == code


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), -30), (dict(wtype=2), -30), (dict(rows=-1), -32), (dict(cols=-1), -33), (dict(dy=0), -34),
    (dict(lddy=199), -37), (dict(h=0), -34), (dict(ldh=199), -37), (dict(weight=0), -34), (dict(rstd=0), -34),
    (dict(lddh=199), -37), (dict(dx=0), -35), (dict(lddx=199), -37),
])
def test_backward_refuses(kw, code):
    assert fp8.mi_rmsnorm_backward(**{**BACK, **kw}) == code


def test_quick_returns_touch_nothing():
    null = dict.fromkeys(("x", "q", "scale", "qt", "scale_t"), 0)
    assert fp8.mi_fp8_quantize(**{**QUANT, **null, "rows": 0}) == 0
    assert fp8.mi_fp8_quantize(**{**QUANT, **null, "cols": 0}) == 0
    null = dict.fromkeys(("A", "scaleA", "B", "scaleB", "C"), 0)
    assert fp8.mi_fp8_gemm(**{**GEMM, **null, "M": 0}) == 0
    assert fp8.mi_fp8_gemm(**{**GEMM, **null, "N": 0}) == 0
    # Nothing is added, and C keeps its values.
    for kw in (dict(K=0), dict(alpha=0.0)):
        assert fp8.mi_fp8_gemm(**{**GEMM, **null, "C": P, "beta": 1.0, **kw}) == 0
    assert fp8.mi_rmsnorm(**{**NORM, "rows": 0, "x": 0, "weight": 0, "y": 0, "q": 0}) == 0
    assert fp8.mi_rmsnorm(**{**NORM, "cols": 0}) == 0
    assert fp8.mi_rmsnorm_backward(**{**BACK, "cols": 0}) == 0
    assert fp8.mi_rmsnorm_backward(**{**BACK, "rows": 0, "dy": 0, "dx": 0, "beta": 1.0}) == 0


def test_host_tensors_are_refused():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    q, s = fp8.fp8_empty(4, 8, device="cpu")
    with pytest.raises(ValueError, match="device tensor"):
        mg.fp8_quantize(x, q, s)
    with pytest.raises(ValueError, match="device tensor"):
        mg.fp8_gemm(1.0, q, s, q, s, 0.0, x)
    with pytest.raises(ValueError, match="device tensor"):
        mg.rmsnorm(x, x[0], 1e-5, q=q, scale=s)
    with pytest.raises(ValueError, match="device tensor"):
        mg.rmsnorm_backward(x, x, x[0], s[0], x)


@pytest.mark.parametrize("rows,cols,block,table", [(1, 1, "row", (1, 1)), (5, 128, "row", (1, 5)),
                                                   (5, 129, "row", (2, 5)), (129, 300, "tile", (2, 3)),
                                                   (0, 16, "row", (1, 0)), (0, 0, "tile", (0, 0))])
def test_empty_pair(rows, cols, block, table):
    q, s = fp8.fp8_empty(rows, cols, block, torch.float8_e5m2, device="cpu")
    assert tuple(q.shape) == (rows, cols) and q.dtype == torch.float8_e5m2
    assert tuple(s.shape) == table and s.dtype == torch.float32
    if rows > 1:
        assert q.stride(0) % 16 == 0 and q.stride(0) >= cols
    with pytest.raises(ValueError, match="block"):
        fp8.fp8_empty(rows, cols, "col", device="cpu")


def test_argument_checks():
    cpu = torch.device("cpu")
    real = fp8._REAL
    a = fp8._Arg("x", torch.zeros(4, 8)[:, :5], (4, 5), real, cpu)
    assert a.ld == 8 and a.end - a.ptr == (3 * 8 + 5) * 4
    assert fp8._Arg("x", torch.zeros(0, 8), (0, 8), real, cpu).ld == 8
    assert fp8._Arg("x", torch.zeros(3, 0), (3, 0), real, cpu).ld >= 1
    assert fp8._Arg("x", torch.zeros(8, 8)[:1, :5], (1, 5), real, cpu).ld == 5
    assert fp8._Arg("x", torch.zeros(4, 8)[:, :1], (4, 1), real, cpu).ld == 8
    for t, kind in ((torch.zeros(8, 4).T, ValueError), (torch.zeros(1, 8).expand(4, 8), ValueError),
                    (torch.zeros(5, 8), ValueError), (torch.zeros(4, 8, dtype=torch.float64), TypeError)):
        with pytest.raises(kind):
            fp8._Arg("x", t, (4, 8), real, cpu)
    with pytest.raises(ValueError, match="contiguous"):
        fp8._Arg("w", torch.zeros(16)[::2], (8,), real, cpu)


def test_overlap():
    cpu, buf = torch.device("cpu"), torch.zeros(64, 64)
    arg = lambda t: ("t", fp8._Arg("t", t, tuple(t.shape), fp8._REAL, cpu), 4)  # noqa: E731
    left, right, mid = arg(buf[:, :32]), arg(buf[:, 32:]), arg(buf[10:20, 30:40])
    fp8._apart([left], [right])                       # side by side in one buffer
    fp8._apart([arg(buf[:32])], [arg(buf[32:])])
    for other in (left, right):
        with pytest.raises(ValueError, match="overlap"):
            fp8._apart([mid], [other])
    with pytest.raises(ValueError, match="overlap"):  # two outputs
        fp8._apart([left, mid], [])
    with pytest.raises(ValueError, match="overlap"):  # a vector within a matrix
        fp8._apart([arg(buf[5, 3:9])], [left])
    fp8._apart([arg(buf[5, 40:50])], [left])
    fp8._apart([arg(buf[:0])], [arg(buf)])


def test_binding_leaves_host_tensors():
    """What is not on a device is not taken by the binding; the tensor form names the argument."""
    torch = pytest.importorskip("torch")
    from fp32_gemm_nn_amd import fp8

    native = fp8._load_native()
    q, s = torch.zeros(4, 128).to(torch.float8_e4m3fn), torch.ones(1, 4)
    assert native.gemm(1.0, q, s, q, s, 0.0, torch.zeros(4, 4), "row", None) is None
    assert native.quantize(torch.zeros(4, 128), q, s, None, None, "row", None) is None
    assert native.gemm() is None and native.rmsnorm(1) is None and native.rmsnorm_backward(*[None] * 9) is None
    with pytest.raises(ValueError, match="A must be a device tensor"):
        mg.fp8_gemm(1.0, q, s, q, s, 0.0, torch.zeros(4, 4), block="row")
