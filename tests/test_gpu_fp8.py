"""The 8-bit linear layer on the GPU against its definitions in 64 bits.

Tolerances count roundings: half a step each, 2^-24 of a value in FP32 (2^-23
for an addition inside the matrix cores, whose rounding is taken to be off by
a whole step), 2^-8 in bfloat16, 2^-11 in float16, 2^-4 in E4M3, 2^-3 in E5M2.
Products with a 16-bit result use the 8-bit matrix instruction, which drops
bits below 2^-13 of the largest of eight neighbouring products: seven of them
are off by that each, at most.
"""
import sys

import pytest

import fp32_gemm_nn_amd as mg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
# Half a step of an 8-bit value: relative, and at least (a subnormal's).
HALF = {torch.float8_e4m3fn: (2.0**-4, 2.0**-10), torch.float8_e5m2: (2.0**-3, 2.0**-17)}
U32 = 2.0**-24
EPS = 1e-5


def note(msg):
    sys.__stderr__.write(f"[gpu] {msg}\n")
    sys.__stderr__.flush()


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.load_library()
    yield
    torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def _named(request):
    note(request.node.name)


def half(dtype):
    return torch.finfo(dtype).eps / 2


def blocks(n):
    return (n + 127) // 128


class Framed:
    """A matrix inside a buffer that holds a pattern: `off` elements in, rows `ld` apart. `whole()` checks the rest."""

    def __init__(self, rows, cols, dtype, ld=None, off=0):
        self.ld, self.off, self.rows, self.cols = ld or max(cols, 1), off, rows, cols
        n = off + rows * self.ld + 64
        self.size = torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((n * self.size,), 0x5B, dtype=torch.uint8, device="cuda")
        self.t = self.raw.view(dtype)[off:off + rows * self.ld].view(rows, self.ld)[:, :cols]

    def fill(self, v):
        self.t.copy_(v)
        return self

    def whole(self):
        mask = torch.zeros(self.raw.numel() // self.size, dtype=torch.bool, device="cuda")
        mask[self.off:self.off + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = True
        outside = self.raw.view(-1, self.size)[~mask]
        return bool((outside == 0x5B).all())


def values(g, rows, cols, dtype=torch.float32):
    spread = torch.exp(torch.randn(cols, generator=g, device="cuda"))
    return (torch.randn(rows, cols, generator=g, device="cuda") * spread).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def each(scale, rows, cols, block):
    """A scale for each element, in 64 bits."""
    s = scale.double()
    if block == "row":
        return s.T.repeat_interleave(128, 1)[:rows, :cols]
    return s.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def block_max(x, block):
    rows, cols = x.shape
    p = torch.nn.functional.pad(x.abs().nan_to_num(nan=0.0, posinf=float("inf")), (0, -cols % 128, 0, -rows % 128))
    if block == "row":
        return p.view(p.shape[0], -1, 128).amax(2)[:rows].T
    return p.view(-1, 128, p.shape[1] // 128, 128).amax((1, 3))


def factor(a, f8):
    """T / a, rounded once (torch takes a number over a tensor as a reciprocal and a product)."""
    return torch.full_like(a, TOP[f8]) / a


def check_quantized(x64, q, scale, block, rel=0.0):
    """q and scale stand for x64 (known to `rel` of itself) as the definition says."""
    rows, cols = x64.shape
    a = block_max(x64, block).clamp(min=2.0**-100) / TOP[q.dtype]
    assert ((scale.double() - a).abs() <= a * (rel + U32)).all()
    s = each(scale, rows, cols, block)
    r, least = HALF[q.dtype]
    # x * (T / a) is off by two roundings, and the table's scale by one, before the rounding to 8 bits.
    limit = torch.maximum(x64.abs() * r, s * least) * (1 + 16 * U32) + x64.abs() * (rel + 4 * U32)
    off = (q.double() * s - x64).abs()
    assert (off <= limit).all(), float((off - limit).max())


# ---- quantisation


SHAPES = [(1, 1), (1, 128), (3, 5), (7, 129), (128, 128), (129, 127), (130, 16), (200, 300), (257, 1000), (1, 4096)]


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("type", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(rows, cols, type, fmt, block):
    f8 = F8[fmt]
    for k, (ld, off, ldq, offq) in enumerate([(cols, 0, cols + -cols % 16, 0), (cols + 3, 1, cols + 5, 3)]):
        x = Framed(rows, cols, DTYPE[type], ld, off).fill(values(gen(k), rows, cols, DTYPE[type]))
        q, qt = Framed(rows, cols, f8, ldq, offq), Framed(cols, rows, f8, rows + (5 if k else -rows % 16), offq)
        table = (blocks(cols), rows) if block == "row" else (blocks(rows), blocks(cols))
        table_t = (blocks(rows), cols) if block == "row" else (blocks(cols), blocks(rows))
        s, st = (Framed(*t, torch.float32, t[1] + 2 * k, k) for t in (table, table_t))
        mg.fp8_quantize(x.t, q.t, s.t, qt.t, st.t, block=block)
        torch.cuda.synchronize()
        x64 = x.t.double()
        check_quantized(x64, q.t, s.t, block)
        check_quantized(x64.T, qt.t, st.t, block)
        # The definition in 32 bits on the host, bit for bit.
        a = block_max(x.t.float().cpu(), block).clamp(min=2.0**-100)
        f = each(factor(a, f8), rows, cols, block).float()
        assert torch.equal((x.t.float().cpu() * f).to(f8).view(torch.uint8), q.t.cpu().contiguous().view(torch.uint8))
        assert torch.equal(s.t.cpu(), a / TOP[f8])
        # Either alone gives the same bits.
        q1, s1 = mg.fp8_empty(rows, cols, block, f8)
        mg.fp8_quantize(x.t, q1, s1, block=block)
        qt1, st1 = mg.fp8_empty(cols, rows, block, f8)
        mg.fp8_quantize(x.t, qt=qt1, scale_t=st1, block=block)
        torch.cuda.synchronize()
        for u, v in ((q1, q.t), (qt1, qt.t)):
            assert torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8))
        assert torch.equal(s1, s.t) and torch.equal(st1, st.t)
        assert all(t.whole() for t in (x, q, qt, s, st))


@pytest.mark.parametrize("block", ["row", "tile"])
def test_quantize_special_values(block):
    x = torch.zeros(260, 300, device="cuda")
    x[:, 128:] = 1e-37                      # below the least maximum
    x[128:, :] = values(gen(1), 132, 300)
    x[130, 5], x[131, 140], x[200, 299] = float("nan"), float("inf"), float("-inf")
    x[140, :128] = float("nan")
    q, s = mg.fp8_empty(260, 300, block)
    qt, st = mg.fp8_empty(300, 260, block)
    mg.fp8_quantize(x, q, s, qt, st, block=block)
    torch.cuda.synchronize()
    for x_, q_, s_ in ((x.cpu(), q.cpu(), s.cpu()), (x.T.cpu(), qt.cpu(), st.cpu())):
        a = block_max(x_, block).clamp(min=2.0**-100)
        assert torch.equal(s_, a / 448.0)
        f = each(factor(a, F8["e4m3"]), *x_.shape, block).float()
        want = (x_ * f).to(F8["e4m3"]).float()
        got = q_.float()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
    assert (q[:128, :128].float() == 0).all()


def test_quantize_far_rows():
    """Rows whose offsets pass 32 bits."""
    rows, cols, ld = 5, 200, 2**30
    x = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)[:, :cols]
    q = torch.empty(rows * ld, dtype=torch.uint8, device="cuda").view(F8["e4m3"]).view(rows, ld)[:, :cols]
    x.copy_(values(gen(3), rows, cols))
    s = torch.empty(2, rows, device="cuda")
    mg.fp8_quantize(x, q, s)
    torch.cuda.synchronize()
    check_quantized(x.double(), q, s, "row")


# ---- products


def operand(g, rows, cols, fmt, block, pad=0, off=0):
    f8 = F8[fmt]
    x = values(g, rows, cols)
    a = block_max(x, block).clamp(min=2.0**-100)
    f = each(factor(a, f8), rows, cols, block).float()
    table = Framed(*a.shape, torch.float32, a.shape[1] + (pad % 4), off % 3).fill(a / TOP[f8])
    return Framed(rows, cols, f8, cols + -cols % 16 + pad, off).fill((x * f).to(f8)), table


def check_product(a, sa, b, sb, block, alpha, beta, c0, c, out):
    M, K = a.t.shape
    N = b.t.shape[0]
    x = a.t.double() * each(sa.t, M, K, "row")
    y = b.t.double() * each(sb.t, N, K, block)
    want = alpha * (x @ y.T.contiguous())
    mass = abs(alpha) * (x.abs() @ y.abs().T.contiguous())
    if beta:
        want = want + beta * c0.double()
        mass = mass + abs(beta) * c0.double().abs()
    # 128 additions inside a block, a scaled one for each block and split, the scales, alpha and beta.
    limit = mass * (128 + 2 * blocks(K) + 8) * 2 * U32 + want.abs() * half(out)
    if out != torch.float32:
        limit = limit + mass * 7 * 2.0**-13 + torch.finfo(out).smallest_normal * half(out) * 2
    off = (c.double() - want).abs()
    assert (off <= limit).all(), (float((off - limit).max()), float((off / limit.clamp(min=1e-300)).max()))


PRODUCTS = [(1, 64, 128), (1, 1, 1), (2, 3, 5), (16, 128, 128), (17, 130, 129), (1, 4096, 4096), (5, 300, 1000),
            (33, 257, 640), (64, 512, 2048), (100, 100, 100), (128, 128, 128), (129, 255, 257), (200, 1000, 384),
            (300, 130, 4096), (513, 700, 144), (1000, 1300, 700)]


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_gemm(M, N, K, block):
    kinds = [("e4m3", "e4m3", "bf16", 1.0, 0.0, 0, 0), ("e4m3", "e4m3", "fp32", 1.0, 0.0, 3, 1),
             ("e5m2", "e4m3", "fp16", 0.25, 0.5, 16, 16), ("e4m3", "e5m2", "bf16", -1.5, 1.0, 0, 5),
             ("e5m2", "e5m2", "fp32", 2.0, -1.0, 32, 0)]
    for k, (fa, fb, out, alpha, beta, pad, off) in enumerate(kinds):
        note(f"{fa} {fb} {out} alpha {alpha} beta {beta} pad {pad} off {off}")
        g = gen(17 * k + M)
        a, sa = operand(g, M, K, fa, "row", pad, off)
        b, sb = operand(g, N, K, fb, block, pad, off)
        c = Framed(M, N, DTYPE[out], N + (pad % 7), off % 2)
        c0 = values(g, M, N).to(DTYPE[out]) if beta else torch.full((M, N), float("nan"), device="cuda")
        c.fill(c0)
        mg.fp8_gemm(alpha, a.t, sa.t, b.t, sb.t, beta, c.t, block=block)
        torch.cuda.synchronize()
        check_product(a, sa, b, sb, block, alpha, beta, c0, c.t, DTYPE[out])
        assert all(t.whole() for t in (a, sa, b, sb, c))
        again = Framed(M, N, DTYPE[out]).fill(c0)
        mg.fp8_gemm(alpha, a.t, sa.t, b.t, sb.t, beta, again.t, block=block)
        torch.cuda.synchronize()
        assert torch.equal(again.t, c.t), "two calls differ"


LARGE = [(2048, 4096, 1024), (4096, 2048, 512), (4100, 4090, 400), (256, 8192, 2048), (700, 7000, 1500)]


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", LARGE)
def test_gemm_large(M, N, K, block):
    for fa, fb, out, beta in (("e4m3", "e4m3", "bf16", 0.0), ("e5m2", "e4m3", "fp32", 1.0)):
        g = gen(M)
        a, sa = operand(g, M, K, fa, "row")
        b, sb = operand(g, N, K, fb, block)
        c0 = values(g, M, N).to(DTYPE[out])
        c = Framed(M, N, DTYPE[out]).fill(c0)
        mg.fp8_gemm(1.0, a.t, sa.t, b.t, sb.t, beta, c.t, block=block)
        torch.cuda.synchronize()
        check_product(a, sa, b, sb, block, 1.0, beta, c0, c.t, DTYPE[out])
        assert c.whole()


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", [(1, 200, 4096), (24, 384, 4096), (130, 260, 900), (1024, 1024, 1024)])
def test_gemm_whole_numbers(M, N, K, block):
    """Small whole numbers and scales that are powers of two have one exact result, whatever the order."""
    g = gen(5)
    a = torch.randint(-4, 5, (M, K), generator=g, device="cuda").float()
    b = torch.randint(-4, 5, (N, K), generator=g, device="cuda").float()
    sa = torch.exp2(torch.randint(-1, 2, (blocks(K), M), generator=g, device="cuda").float())
    table = (blocks(K), N) if block == "row" else (blocks(N), blocks(K))
    sb = torch.exp2(torch.randint(-1, 2, table, generator=g, device="cuda").float())
    c = torch.empty(M, N, device="cuda")
    mg.fp8_gemm(1.0, a.to(F8["e4m3"]), sa, b.to(F8["e4m3"]), sb, 0.0, c, block=block)
    torch.cuda.synchronize()
    want = (a.double() * each(sa, M, K, "row")) @ (b.double() * each(sb, N, K, block)).T.contiguous()
    assert torch.equal(c.double(), want)


def test_gemm_every_value():
    """Every finite 8-bit value, subnormals among them, times one: what the matrix cores read is what it stands for."""
    for fmt in F8:
        v = torch.arange(256, dtype=torch.uint8, device="cuda").view(F8[fmt])
        fine = torch.isfinite(v.float())
        a = torch.zeros(256, 128, dtype=F8[fmt], device="cuda")
        a[:, 3] = torch.where(fine, v.float(), 0.0).to(F8[fmt])
        one = torch.zeros(16, 128, device="cuda")
        one[:, 3] = 1.0
        for fb in F8:
            c = torch.empty(256, 16, device="cuda")
            mg.fp8_gemm(1.0, a, torch.ones(1, 256, device="cuda"), one.to(F8[fb]), torch.ones(1, 1, device="cuda"),
                        0.0, c)
            d = torch.empty(16, 256, device="cuda")
            mg.fp8_gemm(1.0, one.to(F8[fb]), torch.ones(1, 16, device="cuda"), a, torch.ones(2, 1, device="cuda"),
                        0.0, d)
            torch.cuda.synchronize()
            want = torch.where(fine, v.float(), 0.0)
            assert torch.equal(c, want[:, None].expand(256, 16)) and torch.equal(d.T, c)


def test_gemm_nan_and_infinite_scales_stay_in_their_rows():
    g = gen(9)
    a, sa = operand(g, 70, 500, "e4m3", "row")
    b, sb = operand(g, 300, 500, "e4m3", "row")
    a.t.view(torch.uint8)[7, 450] = 0x7F          # NaN
    sa.t[1, 20] = float("inf")
    sb.t[3, 11] = float("nan")
    c = torch.empty(70, 300, device="cuda")
    mg.fp8_gemm(1.0, a.t, sa.t, b.t, sb.t, 0.0, c, block="row")
    torch.cuda.synchronize()
    bad = torch.zeros(70, 300, dtype=torch.bool, device="cuda")
    bad[7], bad[20], bad[:, 11] = True, True, True
    assert torch.isfinite(c[~bad]).all()
    assert torch.isnan(c[7]).all() and torch.isnan(c[:, 11]).all() and not torch.isfinite(c[20]).any()


def test_gemm_nothing_to_add():
    c0 = values(gen(2), 33, 1000)
    for K, alpha in ((0, 1.0), (64, 0.0)):
        for beta in (0.0, 1.0, -0.5):
            c = Framed(33, 1000, torch.float32, 1003, 1).fill(c0 if beta else torch.full_like(c0, float("nan")))
            a, sa = mg.fp8_empty(33, K)
            b, sb = mg.fp8_empty(1000, K, "tile")
            mg.fp8_gemm(alpha, a, sa, b, sb, beta, c.t)
            torch.cuda.synchronize()
            assert torch.equal(c.t, c0 * beta if beta else torch.zeros_like(c0)) and c.whole()


def test_gemm_far_rows():
    """Rows whose offsets pass 32 bits, of both operands and of C."""
    M, N, K, ld = 6, 7, 300, 2**30
    g = gen(4)
    mats = []
    for rows in (M, N):
        x, s = operand(g, rows, K, "e4m3", "row")
        far = torch.empty(rows * ld, dtype=torch.uint8, device="cuda").view(F8["e4m3"]).view(rows, ld)[:, :K]
        far.copy_(x.t)
        x.t = far
        mats += [x, s]
    c = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda").view(M, ld)[:, :N]
    mg.fp8_gemm(1.0, mats[0].t, mats[1].t, mats[2].t, mats[3].t, 0.0, c, block="row")
    torch.cuda.synchronize()
    check_product(*mats, "row", 1.0, 0.0, None, c, torch.bfloat16)


# ---- the norm


COLS = [1, 7, 8, 100, 128, 512, 513, 1300, 2048, 4096, 4100, 8192, 8200, 16384, 16500, 40000]


@pytest.mark.parametrize("type,weight", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                         ("fp32", "fp32")])
@pytest.mark.parametrize("cols", COLS)
def test_norm(cols, type, weight):
    dtype = DTYPE[type]
    for rows, off, fmt in ((1, 0, "e4m3"), (5, 1, "e4m3"), (130, 0, "e5m2")):
        g = gen(cols + rows)
        x = Framed(rows, cols, dtype, cols + off * 3, off).fill(values(g, rows, cols))
        r = Framed(rows, cols, dtype, cols + off * 5, off).fill(values(g, rows, cols))
        w = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(DTYPE[weight])
        h, y = Framed(rows, cols, dtype, cols + off, off), Framed(rows, cols, dtype, cols + off * 2, off)
        q = Framed(rows, cols, F8[fmt], cols + -cols % 16 + 3 * off, off)
        s, rstd = Framed(blocks(cols), rows, torch.float32, rows + off, off), Framed(1, rows, torch.float32)
        mg.rmsnorm(x.t, w, EPS, residual=r.t, h=h.t, y=y.t, q=q.t, scale=s.t, rstd=rstd.t[0])
        torch.cuda.synchronize()
        assert torch.equal(h.t, (x.t.float() + r.t.float()).to(dtype))
        h64 = h.t.double()
        rstd64 = (h64.square().mean(1) + EPS) ** -0.5
        y64 = h64 * rstd64[:, None] * w.double()
        # The sum of squares passes at most 64 roundings, whose root halves them; eight more for the rest of rstd and y.
        rel = 40 * U32
        assert ((rstd.t[0].double() - rstd64).abs() <= rstd64 * rel).all()
        assert ((y.t.double() - y64).abs() <= y64.abs() * (rel + half(dtype)) + torch.finfo(dtype).tiny * half(dtype) * 2).all()
        check_quantized(y64, q.t, s.t, "row", rel)
        assert all(t.whole() for t in (x, r, h, y, q, s, rstd))
        # Without the residual; q alone, and y alone; the sum in x's or the residual's place.
        q1, s1 = mg.fp8_empty(rows, cols, dtype=F8[fmt])
        mg.rmsnorm(h.t, w, EPS, q=q1, scale=s1)
        y1 = torch.empty(rows, cols, dtype=dtype, device="cuda")
        mg.rmsnorm(h.t, w, EPS, y=y1)
        x1, r1, y2 = x.t.clone(), r.t.clone(), torch.empty_like(y1)
        mg.rmsnorm(x1, w, EPS, residual=r.t, h=x1, y=y2)
        mg.rmsnorm(x.t, w, EPS, residual=r1, h=r1, y=y2)
        torch.cuda.synchronize()
        assert torch.equal(q1.contiguous().view(torch.uint8), q.t.contiguous().view(torch.uint8))
        assert torch.equal(s1, s.t) and torch.equal(y1, y.t) and torch.equal(y2, y.t)
        assert torch.equal(x1, h.t) and torch.equal(r1, h.t)


def test_norm_rows_of_nothing_and_not_finite():
    x = values(gen(1), 6, 300)
    x[0] = 0.0
    x[1, 7], x[2, 9], x[3] = float("nan"), float("inf"), 1e-30
    w = torch.ones(300, device="cuda")
    y, (q, s) = torch.empty_like(x), mg.fp8_empty(6, 300)
    mg.rmsnorm(x, w, EPS, y=y, q=q, scale=s)
    torch.cuda.synchronize()
    assert (y[0] == 0).all() and (q[0].float() == 0).all() and (s[:, 0] == 2.0**-100 / 448).all()
    assert torch.isnan(y[1]).all() and torch.isnan(q[1].float()).all()
    assert torch.isnan(y[2, 9]) and (y[2, :9] == 0).all()
    assert torch.isfinite(y[3:]).all() and torch.isfinite(q[3:].float()).all()


# ---- the norm's gradients


def check_backward(dy, h, w, rstd, dh, dx, dw, dw0, beta, dtype):
    rows, cols = dy.shape
    dy, h, w, r = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    g, u = dy * w, h * r
    want = r * (g - u * (g * u).mean(1, keepdim=True))
    mass = r * (g.abs() + u.abs() * (g * u).abs().mean(1, keepdim=True))
    if dh is not None:
        want, mass = want + dh.double(), mass + dh.double().abs()
    # A sum over a row passes at most 64 roundings.
    limit = mass * 72 * U32 + want.abs() * half(dtype) + torch.finfo(dtype).tiny * half(dtype) * 2
    assert ((dx.double() - want).abs() <= limit).all()
    if dw is not None:
        want, mass = (dy * u).sum(0), (dy * u).abs().sum(0)
        if beta:
            want, mass = want + beta * dw0.double(), mass + abs(beta) * dw0.double().abs()
        # No sum over the rows adds more than a quarter of them one by one and then a hundred partial ones.
        limit = mass * (rows / 4 + 110) * U32
        assert ((dw.double() - want).abs() <= limit).all()


@pytest.mark.parametrize("type,weight", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("cols", COLS)
def test_backward(cols, type, weight):
    dtype = DTYPE[type]
    for rows, off, beta in ((1, 0, 0.0), (7, 1, 1.0), (600, 0, -0.5)):
        g = gen(cols + rows)
        dy, h, dh = (Framed(rows, cols, dtype, cols + off * k, off).fill(values(g, rows, cols)) for k in (1, 2, 3))
        w = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(DTYPE[weight])
        rstd = torch.rsqrt(h.t.float().square().mean(1) + EPS)
        dx, dw = Framed(rows, cols, dtype, cols + off * 4, off), Framed(1, cols, torch.float32, None, off)
        dw0 = torch.randn(cols, generator=g, device="cuda") if beta else torch.full((cols,), float("nan"), device="cuda")
        dw.t[0].copy_(dw0)
        mg.rmsnorm_backward(dy.t, h.t, w, rstd, dx.t, dw.t[0], dh=dh.t, beta=beta)
        torch.cuda.synchronize()
        check_backward(dy.t, h.t, w, rstd, dh.t, dx.t, dw.t[0], dw0, beta, dtype)
        assert all(t.whole() for t in (dy, h, dh, dx, dw))
        # Without dh; in the place of dh, and of dy, with the same weight's gradient.
        alone = torch.empty(rows, cols, dtype=dtype, device="cuda")
        mg.rmsnorm_backward(dy.t, h.t, w, rstd, alone)
        dh1, dy1, dw1 = dh.t.clone(), dy.t.clone(), dw0.clone()
        mg.rmsnorm_backward(dy.t, h.t, w, rstd, dh1, dh=dh1)
        mg.rmsnorm_backward(dy1, h.t, w, rstd, dy1, dw1, dh=dh.t, beta=beta)
        torch.cuda.synchronize()
        check_backward(dy.t, h.t, w, rstd, None, alone, None, None, 0.0, dtype)
        assert torch.equal(dh1, dx.t) and torch.equal(dy1, dx.t) and torch.equal(dw1, dw.t[0])


def test_backward_against_differences():
    rows, cols, step = 3, 37, 1e-6
    g = gen(11)
    h, dy, dh = (values(g, rows, cols) for _ in range(3))
    w = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    y, rstd = torch.empty_like(h), torch.empty(rows, device="cuda")
    mg.rmsnorm(h, w, EPS, y=y, rstd=rstd)
    dx, dw = torch.empty_like(h), torch.empty_like(w)
    mg.rmsnorm_backward(dy, h, w, rstd, dx, dw, dh=dh)
    torch.cuda.synchronize()
    h, dy, dh, w, dx, dw = (t.double().cpu() for t in (h, dy, dh, w, dx, dw))

    def loss(h, w):
        y = h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * w
        return (dy * y).sum() + (dh * h).sum()

    scale = float(dx.abs().max()), float(dw.abs().max())
    for i in range(rows):
        for j in range(cols):
            e = torch.zeros_like(h)
            e[i, j] = step
            d = (loss(h + e, w) - loss(h - e, w)) / (2 * step)
            # 32-bit sums of 37 terms, and differences good to about 1e-16 / step of the loss.
            assert abs(d - dx[i, j]) <= 1e-5 * scale[0]
    for j in range(cols):
        e = torch.zeros_like(w)
        e[j] = step
        d = (loss(h, w + e) - loss(h, w - e)) / (2 * step)
        assert abs(d - dw[j]) <= 1e-5 * scale[1]


def test_backward_without_rows():
    h, w = torch.empty(0, 40, device="cuda"), torch.ones(40, device="cuda")
    dw = torch.ones(40, device="cuda")
    mg.rmsnorm_backward(h, h, w, torch.empty(0, device="cuda"), torch.empty_like(h), dw, beta=0.5)
    torch.cuda.synchronize()
    assert (dw == 0.5).all()


# ---- streams, graphs, refusals


def _layer(stream=None):
    """Norm, product and their backward pass as one layer's step: (calls, outputs to compare)."""
    g = gen(21)
    rows, cols, out = 200, 1000, 520
    x, r, dz = values(g, rows, cols, torch.bfloat16), values(g, rows, cols, torch.bfloat16), values(g, rows, out, torch.bfloat16)
    w, W = torch.ones(cols, device="cuda"), values(g, out, cols)
    h, y, z = torch.empty_like(x), torch.empty_like(x), torch.empty_like(dz)
    rstd, dw = torch.empty(rows, device="cuda"), torch.empty(cols, device="cuda")
    q, s = mg.fp8_empty(rows, cols)
    qt, st = mg.fp8_empty(cols, rows)
    Wq, Ws = mg.fp8_empty(out, cols, "tile")
    Wt, Wts = mg.fp8_empty(cols, out, "tile")
    dq, ds = mg.fp8_empty(rows, out)
    dt, dts = mg.fp8_empty(out, rows)
    dy, dx, dW = torch.empty_like(x), torch.empty_like(x), torch.empty(out, cols, device="cuda")

    def step():
        mg.fp8_quantize(W, Wq, Ws, Wt, Wts, block="tile", stream=stream)
        mg.rmsnorm(x, w, EPS, residual=r, h=h, y=y, q=q, scale=s, rstd=rstd, stream=stream)
        mg.fp8_gemm(1.0, q, s, Wq, Ws, 0.0, z, stream=stream)
        mg.fp8_quantize(y, qt=qt, scale_t=st, stream=stream)
        mg.fp8_quantize(dz, dq, ds, dt, dts, stream=stream)
        mg.fp8_gemm(1.0, dq, ds, Wt, Wts, 0.0, dy, stream=stream)
        mg.fp8_gemm(1.0, dt, dts, qt, st, 0.0, dW, block="row", stream=stream)
        mg.rmsnorm_backward(dy, h, w, rstd, dx, dw, dh=r, stream=stream)

    return step, (x, dz, W), (h, z, dx, dw, dW)


def test_layer_on_another_stream_and_in_a_graph():
    stream = torch.cuda.Stream()
    step, ins, outs = _layer(stream.cuda_stream)
    torch.cuda.synchronize()
    saved = [t.clone() for t in ins]
    other = [t.flip(0).contiguous() for t in ins]
    want = []
    for source in (saved, other):
        for t, v in zip(ins, source):
            t.copy_(v)
        torch.cuda.synchronize()
        step()
        stream.synchronize()
        want.append([t.clone() for t in outs])
    plain, ins2, outs2 = _layer()
    plain()
    torch.cuda.synchronize()
    for a, b in zip(outs2, want[0]):
        assert torch.equal(a, b), "the current stream's result differs"
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for rep in range(6):
        for t, v in zip(ins, (saved, other)[rep % 2]):
            t.copy_(v)
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want[rep % 2]):
            assert torch.equal(a, b), f"replay {rep}"
    del graph


def test_captured_without_a_workspace():
    """Captured on a stream that has none: the product runs unsplit, the weight's gradient sums whole columns."""
    a = torch.randint(-3, 4, (24, 4096), generator=gen(1), device="cuda").float().to(F8["e4m3"])
    b = torch.randint(-3, 4, (300, 4096), generator=gen(2), device="cuda").float().to(F8["e4m3"])
    sa, sb = torch.ones(32, 24, device="cuda"), torch.ones(3, 32, device="cuda")
    h, dy = values(gen(3), 900, 300), values(gen(4), 900, 300)
    w, rstd = torch.ones(300, device="cuda"), torch.rsqrt(h.square().mean(1) + EPS)
    c, dx, dw = torch.empty(24, 300, device="cuda"), torch.empty_like(h), torch.empty(300, device="cuda")
    dyx = dy.clone()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        mg.fp8_gemm(1.0, a, sa, b, sb, 0.0, c, stream=stream.cuda_stream)
        mg.rmsnorm_backward(dyx, h, w, rstd, dyx, dw, stream=stream.cuda_stream)   # dx in dy's place
    for rep in range(3):
        c.fill_(float("nan"))
        dyx.copy_(dy)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.double(), a.double() @ b.double().T.contiguous())
        check_backward(dy, h, w, rstd, None, dyx, dw, None, 0.0, torch.float32)
    del graph


def test_refusals():
    q, s = mg.fp8_empty(40, 300)
    c = torch.empty(40, 40, device="cuda")
    x = torch.empty(40, 300, device="cuda")
    for call, kind in [
        (lambda: mg.fp8_gemm(1.0, q, s, q, s, 0.0, c, block="tile"), ValueError),           # a table of the other kind
        (lambda: mg.fp8_gemm(1.0, q, s, q, s.T.contiguous(), 0.0, c, block="row"), ValueError),
        (lambda: mg.fp8_gemm(1.0, q, s, q[:, :299], s, 0.0, c, block="row"), ValueError),
        (lambda: mg.fp8_gemm(1.0, x, s, q, s, 0.0, c, block="row"), TypeError),
        (lambda: mg.fp8_gemm(1.0, q, s, q, s, 0.0, c[:, ::2], block="row"), ValueError),
        (lambda: mg.fp8_gemm(1.0, q, s, q, s, 0.0, c.double(), block="row"), TypeError),
        (lambda: mg.fp8_gemm(1.0, q, s, q, s, 0.0, c.cpu(), block="row"), ValueError),
        (lambda: mg.fp8_gemm(1.0, q, s, q, s, 0.0, c, block="col"), ValueError),
        (lambda: mg.fp8_quantize(x), ValueError),
        (lambda: mg.fp8_quantize(x, q), ValueError),
        (lambda: mg.fp8_quantize(x, q, s[:2]), ValueError),
        (lambda: mg.fp8_quantize(x, q, s, *mg.fp8_empty(300, 40, dtype=F8["e5m2"])), TypeError),
        (lambda: mg.fp8_quantize(x, q, x.view(-1)[:120].view(3, 40)), ValueError),           # the table lies in x
        (lambda: mg.rmsnorm(x, x[0], EPS), ValueError),
        (lambda: mg.rmsnorm(x, x[0], EPS, y=x), ValueError),
        (lambda: mg.rmsnorm(x, x[0].bfloat16(), EPS, y=torch.empty_like(x)), TypeError),
        (lambda: mg.rmsnorm(x, x[0, :299], EPS, y=torch.empty_like(x)), ValueError),
        (lambda: mg.rmsnorm(x[:, :200], x[0, :200].clone(), EPS, residual=x[:, 100:], h=x[:, :200], y=torch.empty(40, 200, device="cuda")), ValueError),
        (lambda: mg.rmsnorm_backward(x, x, x[0], x[:, 0], torch.empty_like(x)), ValueError),
        (lambda: mg.rmsnorm_backward(x, x, torch.ones(300, device="cuda"), torch.ones(40, device="cuda"), x[:, :299]), ValueError),
        (lambda: mg.rmsnorm_backward(torch.empty_like(x), x, torch.ones(300, device="cuda"), torch.ones(40, device="cuda"), x), ValueError),
    ]:
        with pytest.raises(kind):
            call()
