"""The tensor forms make the tensors' device current for the call, and leave the caller's device as it was.

Stream 0 is torch's default stream on every device, and work enqueued on it goes to the current one. Two devices
and the library are stood in for, so nothing is launched: the calls below say which device was current.
"""
import contextlib
import ctypes

import pytest

import fp32_gemm_nn_amd as mg
from fp32_gemm_nn_amd import fp8

torch = pytest.importorskip("torch")

SIZE = {torch.float32: 4, torch.bfloat16: 2, torch.float8_e4m3fn: 1}


class Machine:
    """Two devices, of which one is current, and entry points that note it."""

    def __init__(self):
        self.current, self.calls, self.at = 0, [], 0x10000

    def exchange(self, index):
        before, self.current = self.current, index
        return before

    @contextlib.contextmanager
    def device(self, device):
        before = self.exchange(device.index)
        try:
            yield
        finally:
            self.exchange(before)

    def entry(self, name, status=0):
        def call(*args):
            self.calls.append((name, self.current, args[-1] or 0))
            return status
        return call

    def tensor(self, *shape, dtype=torch.float32, device=1):
        """A tensor of that device at an address of its own, which is not read."""
        size = SIZE[dtype]
        bytes_ = max(1, int(torch.Size(shape).numel())) * size
        where = torch.device("cuda", device)
        storage = torch._C._construct_storage_from_data_pointer(self.at, where, bytes_)
        self.at += bytes_ + -bytes_ % 256
        stride = (shape[1], 1) if len(shape) == 2 else (1,)
        return torch._C._construct_CUDA_Tensor_From_Storage_And_Metadata(
            {"dtype": dtype, "size": shape, "stride": stride, "storage_offset": 0, "device": where}, storage)


class Stream:
    def __init__(self, index):
        self.cuda_stream = 0x100 * index


C_TYPES = {"mi_fp8_gemm": "iiiiiiifpipipipifpip", "mi_fp8_quantize": "iiipiiipipipipip",
           "mi_rmsnorm": "iiiipipipfpipiipipipp", "mi_rmsnorm_backward": "iiiipipippipipfpp"}
C_KIND = {"i": ctypes.c_int, "f": ctypes.c_float, "p": ctypes.c_void_p}


@pytest.fixture
def machine(monkeypatch):
    if not hasattr(torch._C, "_cuda_exchangeDevice"):
        pytest.skip("torch without devices")
    m = Machine()
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x100 * index)
    monkeypatch.setattr(torch._C, "_cuda_exchangeDevice", m.exchange)
    monkeypatch.setattr(torch.cuda, "device", m.device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: m.current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(device.index))
    return m


@pytest.fixture(params=["binding", "python"])
def forms(request, machine, monkeypatch):
    """The forms of the 8-bit layer through their C++ half, or through the checks in Python."""
    if request.param == "binding":
        class Library:
            pass

        for name, types in C_TYPES.items():
            setattr(Library, name, ctypes.CFUNCTYPE(ctypes.c_int, *(C_KIND[t] for t in types))(machine.entry(name)))
        with monkeypatch.context() as patch:
            patch.setattr(fp8, "load_library", lambda: Library)
            fp8._load_native()

        def left(*args, **kw):
            raise AssertionError("left to the checks in Python")
        for name in C_TYPES:
            monkeypatch.setattr(fp8, name, left)
        yield machine
        monkeypatch.undo()
        fp8._native = None
        if mg._lib is not None:
            fp8._load_native()
    else:
        class Declines:
            def __getattr__(self, name):
                return lambda *args: None

        monkeypatch.setattr(fp8, "_native", Declines())
        for name in C_TYPES:
            monkeypatch.setattr(fp8, name, machine.entry(name))
        yield machine


def layer_calls(m, device):
    f8 = torch.float8_e4m3fn
    t = lambda *shape, dtype=torch.float32: m.tensor(*shape, dtype=dtype, device=device)  # noqa: E731
    q, s, W, sW, c = t(4, 128, dtype=f8), t(1, 4), t(8, 128, dtype=f8), t(1, 1), t(4, 8)
    x, y, dx, w, rstd = t(4, 128), t(4, 128), t(4, 128), t(128), t(4)
    return [("mi_fp8_gemm", lambda **kw: mg.fp8_gemm(1.0, q, s, W, sW, 0.0, c, **kw)),
            ("mi_fp8_quantize", lambda **kw: mg.fp8_quantize(x, q, s, **kw)),
            ("mi_rmsnorm", lambda **kw: mg.rmsnorm(x, w, 1e-5, y=y, **kw)),
            ("mi_rmsnorm_backward", lambda **kw: mg.rmsnorm_backward(y, x, w, rstd, dx, **kw))]


@pytest.mark.parametrize("device", [0, 1])
def test_8_bit_layer(forms, device):
    for name, call in layer_calls(forms, device):
        for kw, stream in (({}, 0x100 * device), (dict(stream=0), 0), (dict(stream=0x700), 0x700)):
            forms.current = 0
            forms.calls.clear()
            call(**kw)
            assert forms.calls == [(name, device, stream)]
            assert forms.current == 0, "the caller's device"


def test_after_an_error(forms, monkeypatch):
    """The caller's device also comes back where the call is left to the other half, or does not return."""
    def fails(*args):
        assert forms.current == 1
        raise RuntimeError("no stream")
    for name, call in layer_calls(forms, 1):
        monkeypatch.setattr(fp8, name, fails)
        with pytest.raises(RuntimeError):
            call(stream="none such")
        assert forms.current == 0


def test_sgemm(machine, monkeypatch):
    monkeypatch.setattr(mg, "mi_sgemm", machine.entry("sgemm"))
    monkeypatch.setattr(mg, "mi_sgemm_with_config", machine.entry("with_config"))
    for device in (0, 1):
        A, B, C = (machine.tensor(4, 4, device=device) for _ in range(3))
        for kw, name, stream in (({}, "sgemm", 0x100 * device), (dict(stream=0), "sgemm", 0),
                                 (dict(config=0), "with_config", 0x100 * device)):
            machine.calls.clear()
            mg.sgemm("N", "N", 1.0, A, B, 0.0, C, **kw)
            assert machine.calls == [(name, device, stream)]
            assert machine.current == 0
