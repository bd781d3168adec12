"""Rows of as many values as a 32-bit length holds: launches stay within what a grid takes, and no column passes 2^31."""
import sys

import pytest

import fp32_gemm_nn_amd as mg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U32 = 2.0**-24


@pytest.mark.parametrize("cols", [2**28, 2**31 - 1])
def test_weight_gradient(cols):
    """One row, so that the weight's gradient is dy * (h * rstd), each rounded once; most weights are zero, so that
    the mean has few terms and dx is known in 64 bits."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 40 * cols:
        pytest.skip("not enough memory")
    sys.__stderr__.write(f"[gpu] weight gradient of {cols} columns\n")
    sys.__stderr__.flush()
    dy, h = (torch.empty(1, cols, dtype=torch.bfloat16, device="cuda").uniform_(-2, 2) for _ in range(2))
    w = torch.zeros(cols, dtype=torch.bfloat16, device="cuda")
    used = torch.tensor([0, 7, 8, 4095, 2**26 + 1, cols // 2, cols - 9, cols - 8, cols - 1], device="cuda")
    w[used] = torch.tensor([1.0, -2, 3, 0.5, 4, -1, 2, 1, -3], dtype=torch.bfloat16, device="cuda")
    rstd = torch.full((1,), 0.75, device="cuda")
    dx = torch.full_like(dy, float("nan"))
    dw = torch.full((cols,), float("nan"), device="cuda")
    mg.rmsnorm_backward(dy, h, w, rstd, dx, dw)
    torch.cuda.synchronize()
    for at in range(0, cols, 2**27):
        part = slice(at, min(cols, at + 2**27))
        u = h[0, part].float() * 0.75
        assert torch.equal(dw[part], dy[0, part].float() * u), at
    g, u = dy[0, used].double() * w[used].double(), h[0, used].double() * 0.75
    mean = (g * u).sum() / cols
    want = 0.75 * (g - u * mean)
    # g * u: two roundings, nine terms of a sum; four more for dx and one to BF16.
    limit = 16 * U32 * 0.75 * (g.abs() + u.abs() * (g * u).abs().sum() / cols) + want.abs() * 2.0**-8
    assert ((dx[0, used].double() - want).abs() <= limit).all()
    for at in range(0, cols, 2**27):
        assert torch.isfinite(dx[0, at:at + 2**27]).all(), at


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [5, 300, 4096, 20000])
def test_sum_of_squares_at_its_limit(cols, dtype):
    """Squares are summed in 32 bits: up to 2^128 rstd is right, past it it is 0, and y with it."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = torch.zeros(2, cols, dtype=dtype, device="cuda")
    x[0, cols // 2], x[1, cols // 2] = 2.0**63, 2.0**64
    y, rstd = torch.empty_like(x), torch.empty(2, device="cuda")
    mg.rmsnorm(x, torch.ones(cols, device="cuda"), 1e-5, y=y, rstd=rstd)
    torch.cuda.synchronize()
    want = (2.0**126 / cols) ** -0.5
    # A division, a root and a reciprocal, each a step off at most; y rounds twice more, once to its type.
    assert abs(float(rstd[0]) - want) <= 4 * 2 * U32 * want
    want *= 2.0**63
    assert abs(float(y[0, cols // 2]) - want) <= want * (10 * U32 + torch.finfo(dtype).eps / 2)
    assert float(rstd[1]) == 0 and (y[1] == 0).all()
