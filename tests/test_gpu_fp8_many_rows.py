"""The norm over more rows than there are places for workgroups: each takes several, the next one's operands read
while one is written, also where the outputs take the inputs' places."""
import pytest

import fp32_gemm_nn_amd as mg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_fp8 import (DTYPE, EPS, U32, _device, _named, check_backward, check_quantized, gen, half,  # noqa: E402,F401
                          values)

# Every number of waves to a row, lengths that are multiples of 8 and not; rows that leave the last turn uneven.
SHAPES = [(20011, 64), (16384, 100), (9001, 512), (7000, 700), (6151, 1024), (5003, 1300), (3077, 2048), (2500, 2500),
          (2049, 4096), (1100, 5000), (777, 8192), (600, 9000), (520, 16384)]


@pytest.mark.parametrize("type,weight", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_many_rows(rows, cols, type, weight):
    dtype, g = DTYPE[type], gen(rows)
    x, r, dy, dh = (values(g, rows, cols, dtype) for _ in range(4))
    w = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(DTYPE[weight])
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    q, s = mg.fp8_empty(rows, cols)
    h = x.clone()
    mg.rmsnorm(h, w, EPS, residual=r, h=h, y=y, q=q, scale=s, rstd=rstd)
    torch.cuda.synchronize()
    assert torch.equal(h, (x.float() + r.float()).to(dtype))
    rstd64 = (h.double().square().mean(1) + EPS) ** -0.5
    y64 = h.double() * rstd64[:, None] * w.double()
    # The sum of squares passes at most 64 roundings, whose root halves them; eight more for the rest.
    rel = 40 * U32
    assert ((rstd.double() - rstd64).abs() <= rstd64 * rel).all()
    limit = y64.abs() * (rel + half(dtype)) + torch.finfo(dtype).tiny * half(dtype) * 2
    assert ((y.double() - y64).abs() <= limit).all()
    check_quantized(y64, q, s, "row", rel)
    dx, dw = dh.clone(), torch.empty(cols, device="cuda")
    mg.rmsnorm_backward(dy, h, w, rstd, dx, dw, dh=dx)
    again, dw1 = dy.clone(), torch.empty(cols, device="cuda")
    mg.rmsnorm_backward(again, h, w, rstd, again, dw1, dh=dh)
    torch.cuda.synchronize()
    check_backward(dy, h, w, rstd, dh, dx, dw, None, 0.0, dtype)
    assert torch.equal(dx, again) and torch.equal(dw, dw1)
