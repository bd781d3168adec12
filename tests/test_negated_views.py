"""A tensor that torch keeps as the negative of its memory (the imaginary part of a conjugate, for one) is refused:
the tensor forms pass addresses, and the kernels would read the memory as it is."""
import pytest

import fp32_gemm_nn_amd as mg
from fp32_gemm_nn_amd import fp8

torch = pytest.importorskip("torch")

from test_devices import forms, machine  # noqa: E402,F401


def test_checks_in_python():
    cpu = torch.device("cpu")
    x = torch.ones(4, 8)
    fp8._Arg("x", x, (4, 8), fp8._REAL, cpu)
    with pytest.raises(ValueError, match="x .*resolve_neg"):
        fp8._Arg("x", torch._neg_view(x), (4, 8), fp8._REAL, cpu)
    z = torch.ones(4, 1, dtype=torch.complex64)
    assert z.conj().imag.is_neg()
    with pytest.raises(ValueError, match="resolve_neg"):
        fp8._Arg("x", z.conj().imag, (4, 1), fp8._REAL, cpu)


def test_8_bit_layer(forms, monkeypatch):  # noqa: F811
    x, w, y, dx, rstd = (forms.tensor(*s) for s in ((4, 128), (128,), (4, 128), (4, 128), (4,)))
    q, s = forms.tensor(4, 128, dtype=torch.float8_e4m3fn), forms.tensor(1, 4)
    c = forms.tensor(4, 4)
    neg = torch._neg_view
    for call in (lambda: mg.fp8_quantize(neg(x), q, s), lambda: mg.fp8_gemm(1.0, q, neg(s), q, s, 0.0, c, block="row"),
                 lambda: mg.fp8_gemm(1.0, q, s, q, s, 0.0, neg(c), block="row"),
                 lambda: mg.rmsnorm(x, neg(w), 1e-5, y=y), lambda: mg.rmsnorm(x, w, 1e-5, y=neg(y)),
                 lambda: mg.rmsnorm_backward(neg(y), x, w, rstd, dx), lambda: mg.rmsnorm_backward(y, x, w, neg(rstd), dx)):
        with pytest.raises(ValueError, match="resolve_neg"):
            call()
    assert not forms.calls


def test_sgemm(machine, monkeypatch):  # noqa: F811
    monkeypatch.setattr(mg, "mi_sgemm", machine.entry("sgemm"))
    A, B, C = (machine.tensor(4, 4) for _ in range(3))
    for at in range(3):
        args = [torch._neg_view(t) if i == at else t for i, t in enumerate((A, B, C))]
        with pytest.raises(ValueError, match="resolve_neg"):
            mg.sgemm("N", "N", 1.0, args[0], args[1], 0.0, args[2])
    assert not machine.calls
