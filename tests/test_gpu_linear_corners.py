"""Corners of the feed-forward block's operators on the GPU: products of nothing whatever alpha is."""
import math
import sys

import pytest

import fp32_gemm_nn_amd as mg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_fp8 import Framed, gen, values  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _named(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.__stderr__.write(f"[gpu] {request.node.name}\n")
    sys.__stderr__.flush()
    mg.load_library()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("alpha", [math.inf, -math.inf, math.nan, 0.0, 3.0])
@pytest.mark.parametrize("M,N", [(1, 70), (33, 1000), (300, 264)])
def test_no_k_whatever_alpha(M, N, alpha):
    """K == 0: z is the bias, also where alpha times nothing would be NaN."""
    g = gen(M)
    a, b = torch.empty(M, 0, dtype=BF, device="cuda"), torch.empty(N, 0, dtype=BF, device="cuda")
    bias, r = torch.randn(N, generator=g, device="cuda"), values(g, M, N)
    for v in (None, bias):
        want = (torch.zeros(N, device="cuda") if v is None else v).expand(M, N)
        for ta, tb in ("NT", "TN"):
            c, z = Framed(M, N, F32, N + 3, 1), Framed(M, N, F32, N + 5, 2)
            mg.linear(ta, tb, alpha, a.T.contiguous() if ta == "T" else a, b.T.contiguous() if tb == "N" else b, 2.0, c.t, bias=v, act="relu",
                      residual=r, z=z.t)
            torch.cuda.synchronize()
            assert torch.equal(z.t, want) and torch.equal(c.t, want.clamp(min=0) + 2 * r) and c.whole() and z.whole()
        q, s = mg.fp8_empty(M, N)
        q2, s2 = mg.fp8_empty(M, N)
        mg.linear("N", "T", alpha, a, b, 0.0, c.t, bias=v, z=q, scale=s)
        mg.fp8_quantize(want.contiguous(), q2, s2)
        torch.cuda.synchronize()
        assert torch.equal(c.t, want) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
