"""Corners of the feed-forward block's operators on the GPU: products of nothing whatever alpha is, 8-bit checkpoints from
the largest tiles, and activations' derivatives where they are small.

Tolerances count roundings of 2^-24 in FP32.
"""
import math
import sys

import pytest

import fp32_gemm_nn_amd as mg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_fp8 import F8, U32, Framed, blocks, gen, values  # noqa: E402

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


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("ta,tb", ["NT", "NN", "TN", "TT"])
def test_kept_in_8_bits_from_the_largest_tiles(ta, tb, out, kind):
    """Enough outputs for tiles of 256 x 256 (of whole 16 bytes) or 256 x 128 (others), inside the matrix and over both of its
    edges, blocks of k that end early; rows and blocks of columns whose scales differ. The checkpoint is bit for bit what quantising
    z in FP32 gives, z as the same call keeps it in 32 bits, at any alignment."""
    for M, N, K, pad in ((2552, 4088, 136, 0), (4088, 3048, 136, 0), (2040, 3001, 520, 1)):
        g = gen(M)
        rows = torch.exp2(torch.randint(-8, 9, (M, 1), generator=g, device="cuda").float())
        a = torch.randint(-3, 4, (M, K), generator=g, device="cuda") * rows
        b = torch.randint(-3, 4, (N, K), generator=g, device="cuda").float()
        b[128:256] *= 2.0**20                   # a block of columns whose scale is another
        a, b = (Framed(*t.shape, BF, t.shape[1] + pad, pad).fill(t).t for t in (a.T if ta == "T" else a, b if tb == "T" else b.T))
        bias = torch.randint(-9, 10, (N,), generator=g, device="cuda") / 2
        x, y = (t.double().T.contiguous() if f == "T" else t.double() for t, f in ((a, ta), (b, tb)))
        z = Framed(M, N, F32, N + 1, 1)
        mg.linear(ta, tb, 1.0, a, b, 0.0, torch.empty(M, N, device="cuda"), bias=bias, act="relu", z=z.t)
        # At most K + 64 additions, each off by a whole step inside the matrix cores.
        assert ((z.t.double() - x @ y - bias.double()).abs() <= (x.abs() @ y.abs() + bias.double().abs()) * ((K + 64) * 2 * U32)).all()
        q, s = Framed(M, N, F8[kind], N + 5, 3), Framed(blocks(N), M, F32, M + 3, 1)
        c, r = Framed(M, N, out, N + 3, 1), values(g, M, N, out)
        mg.linear(ta, tb, 1.0, a, b, 1.0, c.t, bias=bias, act="relu", residual=r, z=q.t, scale=s.t)
        q2, s2 = Framed(M, N, F8[kind]), Framed(blocks(N), M, F32)
        mg.fp8_quantize(z.t, q2.t, s2.t)
        torch.cuda.synchronize()
        assert torch.equal(s.t, s2.t), (M, N, K)
        off = q.t.view(torch.uint8) != q2.t.view(torch.uint8)
        assert not off.any(), (M, N, K, int(off.sum()), off.nonzero()[:4].tolist())
        # The residual is added in FP32 (one rounding), and the sum rounded to its type.
        want = z.t.clamp(min=0) + r.float()
        assert torch.equal(c.t, want.to(out)), (M, N, K)
        assert q.whole() and s.whole() and c.whole() and z.whole()


def slope64(z, act):
    """f'(z), and how far FP32 may be off. u = 2^-24 is a rounding; v_exp_f32 and v_rcp_f32 are off by 2 u of their result.

    With s = 1 / (1 + e^-p), of which the exponent takes `arg` |p| u (its roundings) and the rest 5: s is off by
    s ((1 - s) (arg |p| + 2) + 3) u, and exact (1) where e^-p < 2^-25, so that 1 + e^-p is 1.
    """
    z, u = z.double(), U32
    if act == "gelu":
        # Phi(-|z|): the polynomial (21 u by its coefficients' sum, 1 u of approximation), its argument (3 u times at most
        # 2.4), e^(-z^2/2) (1.5 z^2 + 2) u, two products. The other part: a product and a constant, and that e again.
        h = torch.erfc(z.abs() / math.sqrt(2)) / 2
        b = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        df = torch.where(z > 0, 1 - h, h) + b
        return df, h * (34 + 1.5 * z * z) * u + (z > 0) * u + b.abs() * (6 + 1.5 * z * z) * u + df.abs() * u
    k1, k3 = math.sqrt(8 / math.pi), 0.044715 * math.sqrt(8 / math.pi)
    p, dp, arg = (z, torch.ones_like(z), 2) if act == "silu" else (k1 * z + k3 * z**3, k1 + 3 * k3 * z * z, 6)
    e = torch.exp(-p.clamp(-700, 700))
    s, w = 1 / (1 + e), e / (1 + e)             # w = 1 - s
    one = p > 25 * math.log(2) + 0.1
    n = w * (arg * p.abs() + 2) + 3
    es, ew = torch.where(one, w, s * n * u), torch.where(one, w, (s * n + w) * u)
    b = z * dp * s * w
    df = s + b
    if act == "silu":       # s (1 + z w)
        return df, s * (z.abs() * ew + (1 + z * w).abs() * u) + (1 + z * w).abs() * es + df.abs() * u
    # dp is off by 4 u; three products.
    return df, es + (z * dp).abs() * (s * ew + es * w) + b.abs() * 7 * u + df.abs() * u


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes_where_they_are_small(act):
    """f' relative to its parts, down to 2^-118, where v_exp_f32 and v_rcp_f32 may have given 0 for one below 2^-126."""
    z = torch.cat([torch.linspace(-110, 20, 130001), torch.linspace(-14, 8, 220001), torch.linspace(-1.5, -0.5, 20001),
                   10.0 ** torch.linspace(-38, 2, 1001), -(10.0 ** torch.linspace(-38, 2, 1001))]).cuda()[None]
    one, dz, dg, du, h = torch.ones_like(z), *(torch.empty_like(z) for _ in range(4))
    mg.act_backward(one, z, dz, act=act)
    mg.gated_backward(one, z, one, dg, du, act=act, h=h)
    torch.cuda.synchronize()
    want, limit = slope64(z, act)
    over = (dz.double() - want).abs() / (limit + 2.0**-118)
    assert over.max() <= 1, (float(over.max()), float(z.flatten()[over.argmax()]))
    assert torch.equal(dg, dz) and torch.equal(du, h)


@pytest.mark.parametrize("type", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(100003, 64), (70000, 136), (40001, 384), (70001, 9)])
def test_backward_of_narrow_matrices(rows, cols, type):
    """Many rows of few columns, cut into more parts than others: whole numbers, exact whatever the order."""
    g = gen(rows)
    dy, z, u = (torch.randint(-2, 3, (rows, cols), generator=g, device="cuda").to(type) for _ in range(3))
    out = [Framed(rows, cols, type, cols + 3, 1) for _ in range(3)]
    sums = torch.full((3, cols), 2.0, device="cuda")
    d64, u64, f64 = dy.double(), u.double(), z.double().clamp(min=0)
    on = (z > 0).double()
    for b in (None, sums[0]):
        mg.act_backward(dy, z, out[0].t, act="relu", y=out[1].t, dbias=b, beta=0.5)
        torch.cuda.synchronize()
        assert torch.equal(out[0].t.double(), d64 * on) and torch.equal(out[1].t.double(), f64)
    for b, b2 in ((None, None), (sums[1], sums[2])):
        mg.gated_backward(dy, z, u, out[0].t, out[1].t, act="relu", h=out[2].t, dbias_g=b, dbias_u=b2, beta=0.5)
        torch.cuda.synchronize()
        assert all(torch.equal(o.t.double(), w) for o, w in zip(out, (d64 * u64 * on, d64 * f64, f64 * u64)))
    for got, want in zip(sums, (d64 * on, d64 * u64 * on, d64 * f64)):
        assert torch.equal(got.double(), want.sum(0) + 1)
    assert all(o.whole() for o in out)
