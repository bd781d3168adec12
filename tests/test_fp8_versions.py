"""What the 8-bit layer's tensor forms write is new to autograd: the outputs' version counters move, so that a
backward pass that saved one of them before says so, and the inputs' stay."""
import pytest

import fp32_gemm_nn_amd as mg

torch = pytest.importorskip("torch")

from test_devices import forms, machine  # noqa: E402,F401


def test_outputs_and_inputs(forms):  # noqa: F811
    f8 = torch.float8_e4m3fn
    t = lambda *shape, dtype=torch.float32: forms.tensor(*shape, dtype=dtype)  # noqa: E731
    q, s, qt, st = t(4, 128, dtype=f8), t(1, 4), t(128, 4, dtype=f8), t(1, 128)
    W, sW, c = t(8, 128, dtype=f8), t(1, 1), t(4, 8)
    x, r, h, y, dx, w, rstd, dw = t(4, 128), t(4, 128), t(4, 128), t(4, 128), t(4, 128), t(128), t(4), t(128)
    every = [q, s, qt, st, W, sW, c, x, r, h, y, dx, w, rstd, dw]
    for call, written in (
            (lambda: mg.fp8_gemm(1.0, q, s, W, sW, 0.0, c), [c]),
            (lambda: mg.fp8_quantize(x, q, s), [q, s]),
            (lambda: mg.fp8_quantize(x, qt=qt, scale_t=st), [qt, st]),
            (lambda: mg.fp8_quantize(x, q, s, qt, st), [q, s, qt, st]),
            (lambda: mg.rmsnorm(x, w, 1e-5, y=y), [y]),
            (lambda: mg.rmsnorm(x, w, 1e-5, residual=r, h=h, y=y, q=q, scale=s, rstd=rstd), [h, y, q, s, rstd]),
            (lambda: mg.rmsnorm(x, w, 1e-5, residual=r, h=x, q=q, scale=s), [x, q, s]),
            (lambda: mg.rmsnorm_backward(y, h, w, rstd, dx), [dx]),
            (lambda: mg.rmsnorm_backward(y, h, w, rstd, y, dw, dh=dx), [y, dw])):
        before = [v._version for v in every]
        call()
        for v, n in zip(every, before):
            assert (v._version > n) == any(v is o for o in written)


def test_views_share_it(forms):  # noqa: F811
    x, w, whole = forms.tensor(4, 128), forms.tensor(128), forms.tensor(4, 128)
    before = whole._version
    mg.rmsnorm(x, w, 1e-5, y=whole.detach())
    assert whole._version > before


def test_a_refused_call_writes_nothing(forms, monkeypatch):  # noqa: F811
    x, w, y = forms.tensor(4, 128), forms.tensor(100), forms.tensor(4, 128)
    with pytest.raises((ValueError, AssertionError)):
        mg.rmsnorm(x, w, 1e-5, y=y)
    assert y._version == 0


def test_inference_tensors(forms):  # noqa: F811
    """They have no version, and are written all the same."""
    with torch.inference_mode():
        x, w, y = forms.tensor(4, 128), forms.tensor(128), forms.tensor(4, 128)
        assert y.is_inference()
    mg.rmsnorm(x, w, 1e-5, y=y)
    assert forms.calls[-1][0] == "mi_rmsnorm"


@pytest.mark.gpu
def test_backward_of_an_overwritten_value():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = torch.ones(4, 128, device="cuda", requires_grad=True)
    for overwrite in (False, True):
        y = x * 2
        z = (y * y).sum()                    # keeps y
        out = y.detach() if overwrite else torch.empty_like(y)
        mg.rmsnorm(torch.ones(4, 128, device="cuda"), torch.ones(128, device="cuda"), 1e-5, y=out)
        if overwrite:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                z.backward()
        else:
            z.backward()
    torch.cuda.synchronize()
