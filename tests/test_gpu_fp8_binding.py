"""The tensor forms' C++ half: what it takes, what it leaves to the checks in Python, and that both give one result."""
import pytest

import fp32_gemm_nn_amd as mg
from fp32_gemm_nn_amd import fp8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


class Declines:
    """Stands in for the binding and takes nothing."""

    def __getattr__(self, name):
        return lambda *args: None


@pytest.fixture
def data():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device="cuda").manual_seed(3)
    d = {"native": fp8._load_native()}
    for name, r, c in (("x", 70, 300), ("r", 70, 300), ("dy", 70, 300)):
        d[name] = torch.randn(r, c, generator=g, device="cuda").bfloat16()
    d["w"] = torch.randn(300, generator=g, device="cuda")
    d["W"], d["sW"] = mg.fp8_empty(200, 300, "tile")
    mg.fp8_quantize(torch.randn(200, 300, generator=g, device="cuda"), d["W"], d["sW"], block="tile")
    return d


def layer(d):
    """One pass through every form; all that it writes."""
    q, s = mg.fp8_empty(70, 300)
    qt, st = mg.fp8_empty(300, 70)
    h, y, dx = (torch.empty_like(d["x"]) for _ in range(3))
    rstd, dw = torch.empty(70, device="cuda"), torch.empty(300, device="cuda")
    c = torch.empty(70, 200, dtype=torch.float16, device="cuda")
    assert mg.rmsnorm(d["x"], d["w"], 1e-5, residual=d["r"], h=h, y=y, q=q, scale=s, rstd=rstd) is None
    assert mg.fp8_gemm(2, q, s, d["W"], d["sW"], 0.0, c) is c
    got = mg.fp8_quantize(d["dy"], qt=qt, scale_t=st)
    assert got[0] is qt and got[1] is st and len(got) == 2
    assert mg.rmsnorm_backward(d["dy"], h, d["w"], rstd, dx, dw, dh=y) is None
    torch.cuda.synchronize()
    return [t.contiguous().view(torch.uint8).cpu() for t in (q, s, h, y, rstd, c, qt, st, dx, dw)]


def test_both_ways_give_the_same(data, monkeypatch):
    quick = layer(data)
    monkeypatch.setattr(fp8, "_native", Declines())
    for a, b in zip(quick, layer(data)):
        assert torch.equal(a, b)


def test_plain_calls_are_taken(data):
    n, x, w = data["native"], data["x"], data["w"]
    q, s = mg.fp8_empty(70, 300)
    c = torch.empty(70, 200, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    rstd, dw = torch.ones(70, device="cuda"), torch.empty(300, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert n.quantize(x, q, s, None, None, "row", None) == 0
    assert n.gemm(1.0, q, s, data["W"], data["sW"], 0, c, "tile", stream) == 0
    assert n.rmsnorm(x, w, 1e-5, None, None, y, None, None, rstd, None) == 0
    assert n.rmsnorm_backward(x, y, w, rstd, dx, dw, dx, 0.0, None) == 0     # dx may be dh
    h = x.clone()
    assert n.rmsnorm(h, w, 1e-5, None, h, y, None, None, None, None) == 0    # h may be x
    torch.cuda.synchronize()


def test_the_rest_is_left(data):
    n, x, w = data["native"], data["x"], data["w"]
    q, s = mg.fp8_empty(70, 300)
    c = torch.empty(70, 200, device="cuda")
    W, sW = data["W"], data["sW"]
    good = [1.0, q, s, W, sW, 0.0, c, "tile", None]
    for at, bad in ((0, None), (0, "1"), (1, q.cpu()), (1, x), (1, q[:69]), (1, q[0]), (1, None), (2, s.double()),
                    (2, s.T), (2, s[:2]), (3, W[:, :299]), (4, sW[:1]), (4, sW.half()), (5, [0.0]), (6, c.T),
                    (6, c.double()), (6, c.int()), (6, c[:1].expand(70, 200)), (7, "col"), (7, 0), (8, "s"), (8, 1.5),
                    (6, None)):
        args = list(good)
        args[at] = bad
        assert n.gemm(*args) is None, at
    assert n.gemm(*good[:8]) is None
    # C inside A's memory.
    raw = torch.zeros(70 * 400, dtype=torch.uint8, device="cuda")
    inside = raw.view(torch.float32)[:70 * 100].view(70, 100)
    a = raw.view(F8).view(70, 400)[:, :300]
    assert n.gemm(1.0, a, s, W[:100], sW[:1], 0.0, inside, "tile", None) is None
    y = torch.empty_like(x)
    assert n.rmsnorm(x, w, 1e-5, None, None, None, None, None, None, None) is None
    assert n.rmsnorm(x, w, 1e-5, None, None, x, None, None, None, None) is None            # y is x
    assert n.rmsnorm(x, w.half(), 1e-5, None, None, y, None, None, None, None) is None
    assert n.rmsnorm(x, w, 1e-5, x.float(), None, y, None, None, None, None) is None
    assert n.rmsnorm(x, w, 1e-5, None, None, y, q, None, None, None) is None
    assert n.rmsnorm_backward(x, y, w, torch.ones(71, device="cuda"), y.clone(), None, None, 0.0, None) is None
    assert n.rmsnorm_backward(x, y, w, torch.ones(70, device="cuda"), y, None, None, 0.0, None) is None    # dx is h
    assert n.quantize(x, None, None, None, None, "row", None) is None
    assert n.quantize(x, q, None, None, None, "row", None) is None
    assert n.quantize(x, q, s, torch.empty(300, 70, device="cuda").to(torch.float8_e5m2), s, "row", None) is None


def test_columns_of_one_buffer(data):
    """x and q side by side in rows of one buffer: their spans cross, their bytes do not. The checks in Python tell."""
    raw = torch.zeros(40, 3 * 256, dtype=torch.uint8, device="cuda")
    x = raw[:, :512].view(torch.bfloat16)
    x.copy_(data["x"][:40, :256])
    q = raw[:, 512:].view(F8)
    s = torch.empty(2, 40, device="cuda")
    assert data["native"].quantize(x, q, s, None, None, "row", None) is None
    mg.fp8_quantize(x, q, s)
    want, ws = mg.fp8_empty(40, 256)
    mg.fp8_quantize(x.contiguous(), want, ws)
    torch.cuda.synchronize()
    assert torch.equal(q.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8)) and torch.equal(s, ws)
    with pytest.raises(ValueError, match="overlap"):
        mg.fp8_quantize(x, raw[:, 500:756].view(F8), s)
