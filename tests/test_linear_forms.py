"""The feed-forward block's tensor forms on the host, with two devices and the library stood in for: the device that is
current for a call, the arguments that reach the C entry point, outputs' version counters, and refusals, through the C++
half and through the checks in Python alike."""
import ctypes

import pytest

import fp32_gemm_nn_amd as mg
from fp32_gemm_nn_amd import feedforward, fp8

torch = pytest.importorskip("torch")

import test_devices  # noqa: E402
from test_devices import machine  # noqa: E402,F401

test_devices.SIZE.setdefault(torch.float16, 2)
test_devices.SIZE.setdefault(torch.float8_e5m2, 1)
C_TYPES = {"mi_linear": "cciiiifpipiipiifpipiipipip", "mi_gated": "iiiipipipiippiipiipipipipip",
           "mi_act_backward": "iiipiiipipipipifpp", "mi_gated_backward": "iiipiiipipipipipipipifppp"}
C_KIND = {**test_devices.C_KIND, "c": ctypes.c_char}
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(params=["binding", "python"])
def forms(request, machine, monkeypatch):  # noqa: F811
    machine.got = []

    def entry(name):
        def call(*args):
            machine.got.append(args)
            return machine.entry(name)(*args)
        return call
    if request.param == "binding":
        class Library:
            pass

        for name, types in {**test_devices.C_TYPES, **C_TYPES}.items():
            setattr(Library, name, ctypes.CFUNCTYPE(ctypes.c_int, *(C_KIND[t] for t in types))(entry(name)))
        with monkeypatch.context() as patch:
            patch.setattr(fp8, "load_library", lambda: Library)
            patch.setattr(feedforward, "load_library", lambda: Library)
            feedforward._load_native()

        def left(*args, **kw):
            raise AssertionError("left to the checks in Python")
        for name in C_TYPES:
            monkeypatch.setattr(feedforward, name, left)
        yield machine
        monkeypatch.undo()
        fp8._native = feedforward._native = None
        if mg._lib is not None:
            feedforward._load_native()
    else:
        class Declines:
            def __getattr__(self, name):
                return lambda *args: None

        monkeypatch.setattr(feedforward, "_native", Declines())
        for name in C_TYPES:
            monkeypatch.setattr(feedforward, name, entry(name))
        yield machine


def strided(at, shape, stride, device=1):
    """A BF16 tensor of that device at an address, which is not read."""
    where = torch.device("cuda", device)
    storage = torch._C._construct_storage_from_data_pointer(at, where, 1 << 16)
    return torch._C._construct_CUDA_Tensor_From_Storage_And_Metadata(
        {"dtype": BF, "size": shape, "stride": stride, "storage_offset": 0, "device": where}, storage)


def plain(args):
    """Arguments as the library sees them: a null pointer is 0, a letter a text."""
    return [0 if a is None else a.decode() if isinstance(a, bytes) else a for a in args]


def calls(m, device=1):
    t = lambda *shape, dtype=BF: m.tensor(*shape, dtype=dtype, device=device)  # noqa: E731
    x, W, U, y, r, b = t(4, 128), t(256, 128), t(256, 128), t(4, 256), t(4, 256), t(256, dtype=F32)
    q, s, q2, s2 = t(4, 256, dtype=F8), t(2, 4, dtype=F32), t(4, 256, dtype=F8), t(2, 4, dtype=F32)
    z, dz, du, db, db2 = t(4, 256), t(4, 256), t(4, 256), t(256, dtype=F32), t(256, dtype=F32)
    every = [x, W, U, y, r, b, q, s, q2, s2, z, dz, du, db, db2]
    p = lambda v: v.data_ptr()  # noqa: E731
    return every, [
        (lambda **kw: mg.linear("N", "T", 2.0, x, W, 0.5, y, bias=b, act="gelu", residual=r, z=q, scale=s, **kw), "mi_linear", [y, q, s],
         ["N", "T", 1, 4, 256, 128, 2.0, p(x), 128, p(W), 128, 0, p(b), 3, 1, 0.5, p(r), 256, p(y), 256, 3, p(q), 256, p(s), 4]),
        (lambda **kw: mg.linear("N", "T", 1.0, x, W, 1.0, y, residual=y, z=z, **kw), "mi_linear", [y, z],
         ["N", "T", 1, 4, 256, 128, 1.0, p(x), 128, p(W), 128, 0, 0, 0, 1, 1.0, p(y), 256, p(y), 256, 1, p(z), 256, 0]),
        (lambda **kw: mg.linear("T", "N", 1.0, y, z, 0.0, t(256, 256, dtype=F32), **kw), "mi_linear", [], None),
        (lambda **kw: mg.gated(x, W, U, y, act="gelu_tanh", bias_u=b, g=q, scale_g=s, u=q2, scale_u=s2, **kw), "mi_gated", [y, q, s, q2, s2],
         [1, 4, 256, 128, p(x), 128, p(W), 128, p(U), 128, 0, 0, p(b), 4, 1, p(y), 256, 3, p(q), 256, p(s), 4, p(q2), 256, p(s2), 4]),
        (lambda **kw: mg.gated(x, W, W, y, **kw), "mi_gated", [y], None),
        (lambda **kw: mg.act_backward(r, q, dz, scale=s, act="silu", y=y, dbias=db, beta=1.0, **kw), "mi_act_backward", [dz, y, db],
         [1, 4, 256, p(r), 256, 2, 3, p(q), 256, p(s), 4, p(dz), 256, p(y), 256, 1.0, p(db)]),
        (lambda **kw: mg.act_backward(r, z, r, act="relu", **kw), "mi_act_backward", [r],
         [1, 4, 256, p(r), 256, 1, 1, p(z), 256, 0, None, p(r), 256, 0, None, 0.0, 0]),
        (lambda **kw: mg.gated_backward(r, q, q2, dz, du, scale_g=s, scale_u=s2, act="silu", h=y, dbias_g=db, dbias_u=db2, **kw),
         "mi_gated_backward", [dz, du, y, db, db2],
         [1, 4, 256, p(r), 256, 2, 3, p(q), 256, p(s), 4, p(q2), 256, p(s2), 4, p(dz), 256, p(du), 256, p(y), 256, 0.0, p(db), p(db2)]),
        (lambda **kw: mg.gated_backward(r, z, dz, z, dz, h=r, **kw), "mi_gated_backward", [z, dz, r], None),
    ]


@pytest.mark.parametrize("device", [0, 1])
def test_device_stream_and_arguments(forms, device):
    for call, name, _, args in calls(forms, device)[1]:
        for kw, stream in (({}, 0x100 * device), (dict(stream=0), 0), (dict(stream=0x700), 0x700)):
            forms.current = 0
            forms.calls.clear()
            forms.got.clear()
            call(**kw)
            assert forms.calls == [(name, device, stream)]
            assert forms.current == 0, "the caller's device"
            if args is not None:
                got = plain(forms.got[0])[:len(args)]
                assert all(a is None or a == b for a, b in zip(args, got)), (args, got)


def test_outputs_versions(forms):
    every, listed = calls(forms)
    for call, _, written, _ in listed:
        before = [v._version for v in every]
        call()
        for v, n in zip(every, before):
            assert (v._version > n) == any(v is o for o in written)


def test_refusals(forms):
    t = lambda *shape, dtype=BF, device=1: forms.tensor(*shape, dtype=dtype, device=device)  # noqa: E731
    x, W, U, y, b = t(4, 128), t(256, 128), t(256, 128), t(4, 256), t(256)
    q, s, r, z = t(4, 256, dtype=F8), t(2, 4, dtype=F32), t(4, 256), t(4, 256)
    neg = torch._neg_view
    lin, gat, act, back = mg.linear, mg.gated, mg.act_backward, mg.gated_backward
    for call, kind in [
        (lambda: lin("X", "T", 1.0, x, W, 0.0, y), ValueError), (lambda: lin("N", "", 1.0, x, W, 0.0, y), ValueError),
        (lambda: lin("N", "T", 1.0, x, W, 0.0, y, act="tanh"), ValueError), (lambda: lin("N", "N", 1.0, x, W, 0.0, y), ValueError),
        (lambda: lin("N", "T", 1.0, x, t(256, 128, dtype=torch.float16), 0.0, y), TypeError),
        (lambda: lin("N", "T", 1.0, t(4, 128, dtype=F32), t(256, 128, dtype=F32), 0.0, y), TypeError),
        (lambda: lin("N", "T", 1.0, x, W, 0.0, t(4, 256, dtype=torch.float16)), TypeError),
        (lambda: lin("N", "T", 1.0, x, W, 0.0, t(4, 255)), ValueError),
        (lambda: lin("N", "T", 1.0, x, t(256, 128, device=0), 0.0, y), ValueError),
        (lambda: lin("N", "T", 1.0, x, W, 0.0, y, bias=t(255)), ValueError),
        (lambda: lin("N", "T", 1.0, x, W, 0.0, y, bias=t(256, dtype=torch.float16)), TypeError),
        (lambda: lin("N", "T", 1.0, x, W, 1.0, y, residual=t(4, 256, dtype=F32)), TypeError),
        (lambda: lin("N", "T", 1.0, x, W, 1.0, y, residual=t(5, 256)), ValueError),
        (lambda: lin("N", "T", 1.0, x, W, 0.0, y, z=q), ValueError), (lambda: lin("N", "T", 1.0, x, W, 0.0, y, scale=s), ValueError),
        (lambda: lin("N", "T", 1.0, x, W, 0.0, y, z=z, scale=s), ValueError), (lambda: lin("N", "T", 1.0, x, W, 0.0, y, z=q, scale=t(4, 2, dtype=F32)), ValueError),
        (lambda: lin("N", "T", 1.0, x, W, 0.0, y, z=y), ValueError), (lambda: lin("N", "T", 1.0, x, W, 1.0, y, residual=r, z=r), ValueError),
        (lambda: lin("T", "N", 1.0, y, y, 0.0, t(256, 256), z=t(256, 256, dtype=F32)), TypeError),
        (lambda: lin("N", "T", 1.0, neg(x), W, 0.0, y), ValueError), (lambda: lin("N", "T", 1.0, x, W, 0.0, neg(y)), ValueError),
        (lambda: lin("N", "T", 1.0, t(128), W, 0.0, y), ValueError), (lambda: lin("N", "T", 1.0, strided(0x900000, (4, 128), (256, 2)), W, 0.0, y), ValueError),
        (lambda: gat(x, W, t(255, 128), y), ValueError), (lambda: gat(x, W, U, y, act=None), ValueError),
        (lambda: gat(x, W, U, y, g=q, scale_g=s), ValueError), (lambda: gat(x, W, U, y, g=z, u=q, scale_u=s), TypeError),
        (lambda: gat(x, W, U, y, bias_g=b, bias_u=t(256, dtype=F32)), TypeError), (lambda: gat(x, W, U, y, g=z, u=z), ValueError),
        (lambda: gat(x, W, U, y, g=z, u=y), ValueError), (lambda: gat(x, W, U, strided(W.data_ptr(), (4, 256), (256, 1))), ValueError),
        (lambda: act(y, z, t(4, 256, dtype=F32)), TypeError), (lambda: act(y, None, r), ValueError), (lambda: act(y, q, r), ValueError),
        (lambda: act(y, z, r, y=r), ValueError), (lambda: act(y, z, r, dbias=t(256)), TypeError), (lambda: act(y, t(4, 256, dtype=F32), r), TypeError),
        (lambda: act(y, z, t(4, 256), dbias=t(255, dtype=F32)), ValueError),
        (lambda: back(y, z, q, r, t(4, 256), scale_u=s), TypeError), (lambda: back(y, z, r, z, z), ValueError),
        (lambda: back(y, z, None, r, t(4, 256)), ValueError), (lambda: back(y, z, r, neg(t(4, 256)), t(4, 256)), ValueError),
    ]:
        forms.got.clear()
        with pytest.raises((kind, AssertionError)) as e:
            call()
        assert not forms.got
        if e.type is AssertionError:
            assert "left to the checks" in str(e.value)


def test_overlap_by_rows(forms):
    """Columns of one buffer side by side are apart; shifted ones are not."""
    at = lambda first: strided(0x900000 + 2 * first, (4, 128), (512, 1))  # noqa: E731
    dy, z = at(0), at(128)
    try:
        mg.act_backward(dy, z, at(256), act="silu", y=at(384))
        mg.act_backward(dy, z, dy, act="silu", y=z)
    except AssertionError as e:      # the binding leaves memory that interleaves to the checks in Python
        assert "left to the checks" in str(e)
    forms.got.clear()
    for kw in (dict(dz=at(64)), dict(dz=at(256), y=at(300))):
        with pytest.raises((ValueError, AssertionError)):
            mg.act_backward(dy, z, act="silu", **kw)
    assert not forms.got
