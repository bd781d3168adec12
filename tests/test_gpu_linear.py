"""The feed-forward block's operators on the GPU against their definitions in 64 bits.

Tolerances count roundings: half a step each, 2^-24 of a value in FP32 (2^-23 for an addition inside the matrix cores,
whose rounding is taken to be off by a whole step), 2^-8 in bfloat16, 2^-11 in float16, 2^-4 in E4M3, 2^-3 in E5M2.
Products of two 16-bit values are exact in FP32.
"""
import math
import sys

import pytest

import fp32_gemm_nn_amd as mg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_fp8 import F8, U32, Framed, blocks, check_quantized, each, gen, half, values  # noqa: E402

DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# v_rcp_f32 and v_exp_f32 give 0 for results below 2^-126, and z times them is at most 104 as much.
LOST = 104 * 2.0**-126
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(autouse=True)
def _named(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.__stderr__.write(f"[gpu] {request.node.name}\n")
    sys.__stderr__.flush()
    mg.load_library()
    yield
    torch.cuda.synchronize()


def act64(z, act):
    """f(z), f'(z) and how many steps of 2^-24 of f a value in FP32 may be off by: the argument's roundings times the
    function's condition, a step for v_exp and v_rcp each, and those of the rest."""
    z = z.double()
    if act == "none":
        return z, torch.ones_like(z), torch.zeros_like(z)
    if act == "relu":
        return torch.where(z <= 0, 0 * z.nan_to_num(posinf=0, neginf=0), z), torch.where(z > 0, 1.0, 0 * z.nan_to_num(posinf=0, neginf=0)), torch.zeros_like(z)
    zc = z.clamp(-200, 200)
    if act == "gelu":
        s = torch.erfc(-zc / math.sqrt(2)) / 2
        f = torch.where(z > 200, z, zc * s)
        # The argument z / sqrt 2 is off by two roundings, erfc by 16 steps.
        return f, s + zc * torch.exp(-zc * zc / 2) / math.sqrt(2 * math.pi), 24 + 4 * zc * zc
    p, dp = zc, torch.ones_like(z)
    if act == "gelu_tanh":
        c = math.sqrt(8 / math.pi)
        p, dp = c * (zc + 0.044715 * zc**3), c * (1 + 3 * 0.044715 * zc**2)
    s = 1 / (1 + torch.exp(-p.clamp(-700, 700)))
    return torch.where(z > 200, z, zc * s), s + zc * s * (1 - s) * dp, 16 + 6 * p.abs()


def act_limit(z, err, act, steps=1.0):
    """How far f(z) in FP32 may be off where z is off by `err`: |f'| <= 1.13."""
    f, _, n = act64(z, act)
    return 1.13 * err + f.abs() * n * U32 * steps + LOST


def rounded(want, limit, dtype):
    """`limit` and the rounding to dtype."""
    return limit + (want.abs() + limit) * half(dtype) + (0 if dtype == torch.float32 else torch.finfo(dtype).smallest_normal * half(dtype) * 2)


def near(got, want, limit):
    off = (got.double() - want).abs()
    assert (off <= limit).all(), (float((off - limit).max()), float((off / limit.clamp(min=1e-300)).max()))


def stored(g, rows, cols, dtype, pad=0, off=0):
    return Framed(rows, cols, dtype, cols + pad, off).fill(values(g, rows, cols))


def check_kept(z64, err, q, scale):
    """A checkpoint of z, which is known to `err`: 8 bits and a table, or a matrix."""
    if scale is None:
        return near(q.t, z64, rounded(z64, err, q.t.dtype))
    rows, cols = z64.shape
    a = torch.nn.functional.pad(z64.abs(), (0, -cols % 128)).view(rows, -1, 128).amax(2).T
    e = torch.nn.functional.pad(err, (0, -cols % 128)).view(rows, -1, 128).amax(2).T
    top = 448.0 if q.t.dtype == F8["e4m3"] else 57344.0
    a = a.clamp(min=2.0**-100)
    assert ((scale.t.double() * top - a).abs() <= e + a * 4 * U32).all()
    s = each(scale.t, rows, cols, "row")
    r, least = (2.0**-4, 2.0**-10) if top == 448.0 else (2.0**-3, 2.0**-17)
    off = (q.t.double() * s - z64).abs()
    limit = torch.maximum((z64.abs() + err) * r, s * least) * (1 + 16 * U32) + z64.abs() * 8 * U32 + 2 * err
    assert (off <= limit).all(), float((off - limit).max())


def room(kind, rows, cols, dtype, pad, off):
    """Where a checkpoint goes: (matrix, table or None)."""
    if kind in F8:
        return Framed(rows, cols, F8[kind], cols + -cols % 16 + pad, off), Framed(blocks(cols), rows, torch.float32, rows + pad % 4, off % 3)
    return Framed(rows, cols, dtype, cols + pad, off), None


# ---- products


SHAPES = [(1, 1, 1), (1, 4096, 512), (2, 3, 5), (7, 9, 8), (16, 128, 64), (17, 130, 129), (33, 257, 640), (100, 100, 100),
          (64, 512, 1024), (128, 128, 128), (129, 255, 257), (200, 1000, 384), (300, 130, 2048), (513, 700, 144), (1000, 1300, 700)]
KINDS = [  # type, out, bias, act, beta, residual, keep, pad, off
    ("bf16", "bf16", "bf16", "silu", 1.0, "own", "e4m3", 0, 0),
    ("fp16", "fp32", "fp32", "gelu", -0.5, "c", "e5m2", 8, 8),
    ("bf16", "fp32", None, "none", 0.0, None, "same", 3, 1),
    ("fp16", "fp16", "fp16", "gelu_tanh", 0.0, None, None, 16, 0),
    ("bf16", "bf16", "fp32", "relu", 2.0, "own", "same", 5, 3),
]


def product64(a, b, ta, tb, alpha, bias):
    """z and how far FP32 sums may be off."""
    x, y = a.double(), b.double()
    x, y = x.T.contiguous() if ta == "T" else x, y.T.contiguous() if tb == "T" else y
    z, mass = alpha * (x @ y), abs(alpha) * (x.abs() @ y.abs())
    if bias is not None:
        z, mass = z + bias.double(), mass + bias.double().abs()
    # Every addition of products, of parts of k, of the bias; alpha's product.
    return z, mass * (x.shape[1] + 64) * 2 * U32


def run_linear(M, N, K, ta, tb, kind, seed, alpha=1.0):
    type, out, bias, act, beta, residual, keep, pad, off = kind
    g, dtype, ctype = gen(seed), DTYPE[type], DTYPE[out]
    a = stored(g, *((K, M) if ta == "T" else (M, K)), dtype, pad, off)
    b = stored(g, *((N, K) if tb == "T" else (K, N)), dtype, pad, off)
    for t in (a, b):
        t.t.mul_(K**-0.25)
    v = None if bias is None else torch.randn(N, generator=g, device="cuda").to(DTYPE[bias])
    c0 = values(g, M, N).to(ctype) if residual == "c" else torch.full((M, N), float("nan"), device="cuda")
    c = Framed(M, N, ctype, N + pad, off).fill(c0)
    r = stored(g, M, N, ctype, pad, off) if residual == "own" else None
    z, zs = room(keep, M, N, ctype, pad, off) if keep else (None, None)

    def call(c):
        mg.linear(ta, tb, alpha, a.t, b.t, beta, c.t, bias=v, act=act, residual=None if r is None else r.t,
                  z=None if z is None else z.t, scale=None if zs is None else zs.t)
        torch.cuda.synchronize()
    call(c)
    z64, err = product64(a.t, b.t, ta, tb, alpha, v)
    want = act64(z64, act)[0]
    limit = act_limit(z64, err, act)
    if beta:
        add = beta * (r.t if residual == "own" else c0).double()
        want = want + add
        limit = limit + (want.abs() + add.abs()) * U32
    near(c.t, want, rounded(want, limit, ctype))
    if z is not None:
        check_kept(z64, err, z, zs)
    assert all(t.whole() for t in (a, b, c, r, z, zs) if t is not None)
    again = Framed(M, N, ctype).fill(c0)
    call(again)
    assert torch.equal(again.t, c.t), "two calls differ"
    if residual == "own":
        # The residual's place is C's.
        mg.linear(ta, tb, alpha, a.t, b.t, beta, r.t, bias=v, act=act)
        torch.cuda.synchronize()
        near(r.t, want, rounded(want, limit, ctype))


@pytest.mark.parametrize("ta,tb", ["NT", "NN", "TN", "TT"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, ta, tb):
    for n, kind in enumerate(KINDS):
        run_linear(M, N, K, ta, tb, kind, 17 * n + M, alpha=(1.0, 0.5, -2.0)[n % 3])


LARGE = [(2048, 4096, 1024), (4100, 4090, 400), (256, 8192, 2048), (700, 7000, 1500), (1, 8192, 8192), (40, 4096, 4096), (3000, 3000, 8)]


@pytest.mark.parametrize("ta,tb", ["NT", "NN", "TN", "TT"])
@pytest.mark.parametrize("M,N,K", LARGE)
def test_linear_large(M, N, K, ta, tb):
    for n in (0, 2, 4):
        run_linear(M, N, K, ta, tb, KINDS[n], M + n)


@pytest.mark.parametrize("type", ["bf16", "fp16"])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("ta,tb", ["NT", "NN", "TN", "TT"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (24, 384, 4096), (130, 260, 900), (256, 256, 64), (300, 520, 192), (1024, 1024, 1024),
                                   (520, 2056, 2056), (2048, 2304, 320), (64, 64, 16384), (257, 4097, 129)])
def test_linear_whole_numbers(M, N, K, ta, tb, pad, type):
    """Small whole numbers have one sum whatever the order: a value read before it landed, a block counted twice or a
    row of another shows as a difference."""
    g = gen(M + K)
    a, b = (Framed(*((c, r) if t else (r, c)), DTYPE[type], (r if t else c) + pad, pad).fill(
        torch.randint(-4, 5, (c, r) if t else (r, c), generator=g, device="cuda").float()) for r, c, t in ((M, K, ta == "T"), (K, N, tb == "T")))
    bias = torch.randint(-9, 10, (N,), generator=g, device="cuda").float()
    c0 = torch.randint(-9, 10, (M, N), generator=g, device="cuda").float()
    c, z = c0.clone(), torch.empty_like(c0)
    mg.linear(ta, tb, 2.0, a.t, b.t, -1.0, c, bias=bias, act="relu", z=z)
    torch.cuda.synchronize()
    x, y = (t.t.double().T.contiguous() if f == "T" else t.t.double() for t, f in ((a, ta), (b, tb)))
    want = 2 * (x @ y) + bias.double()
    assert torch.equal(z.double(), want), int((z.double() != want).sum())
    assert torch.equal(c.double(), want.clamp(min=0) - c0.double())


@pytest.mark.parametrize("type", ["bf16", "fp16"])
def test_every_value(type):
    """Every finite value, subnormals among them, times one, through each of the layouts."""
    dtype = DTYPE[type]
    v = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
    v = torch.where(torch.isfinite(v), v, torch.zeros_like(v)).view(512, 128)
    one = torch.eye(128, device="cuda").to(dtype)
    for ta, tb in ("NT", "NN", "TN", "TT"):
        c = torch.empty(512, 128, device="cuda")
        mg.linear(ta, tb, 1.0, v.T.contiguous() if ta == "T" else v, one, 0.0, c)
        torch.cuda.synchronize()
        assert torch.equal(c, v.float())
        d = torch.empty(128, 512, device="cuda")
        mg.linear(ta, tb, 1.0, one, v if tb == "T" else v.T.contiguous(), 0.0, d)
        torch.cuda.synchronize()
        assert torch.equal(d.T, v.float())


def test_linear_not_finite_stays_in_its_rows():
    g = gen(9)
    a, b = values(g, 70, 500, torch.bfloat16), values(g, 300, 500, torch.bfloat16)
    a[7, 450], a[20, 3], b[11, 499] = float("nan"), float("inf"), float("-inf")
    c = torch.empty(70, 300, device="cuda")
    mg.linear("N", "T", 1.0, a, b, 0.0, c)
    torch.cuda.synchronize()
    bad = torch.zeros(70, 300, dtype=torch.bool, device="cuda")
    bad[7], bad[20], bad[:, 11] = True, True, True
    assert torch.isfinite(c[~bad]).all()
    assert torch.isnan(c[7]).all() and not torch.isfinite(c[20]).any() and not torch.isfinite(c[:, 11]).any()


@pytest.mark.parametrize("ta,tb", ["NT", "NN", "TN", "TT"])
def test_linear_what_lies_behind_a_matrix_does_not_count(ta, tb):
    """NaN between rows, before and behind: short last blocks in either direction take none of it."""
    for M, N, K in ((130, 70, 70), (5, 200, 33), (300, 264, 136)):
        for pad in (8, 5):
            g = gen(K)
            mats = []
            for r, c, t in ((M, K, ta == "T"), (K, N, tb == "T")):
                r, c = (c, r) if t else (r, c)
                raw = torch.full(((r + 2) * (c + pad),), float("nan"), dtype=torch.bfloat16, device="cuda")
                m = raw[pad:pad + r * (c + pad)].view(r, c + pad)[:, :c]
                m.copy_(torch.randint(-3, 4, (r, c), generator=g, device="cuda"))
                mats.append(m)
            out = torch.empty(M, N, device="cuda")
            mg.linear(ta, tb, 1.0, *mats, 0.0, out)
            torch.cuda.synchronize()
            x, y = (m.double().T.contiguous() if f == "T" else m.double() for m, f in zip(mats, (ta, tb)))
            assert torch.equal(out.double(), x @ y)


@pytest.mark.parametrize("alpha,K", [(0.0, 64), (1.0, 0)])
def test_linear_nothing_to_add(alpha, K):
    g = gen(2)
    a, b = (torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in ((33, K), (1000, K)))
    bias, c0 = torch.randn(1000, generator=g, device="cuda"), values(g, 33, 1000)
    for beta in (0.0, 1.0, -0.5):
        for v in (None, bias):
            c = Framed(33, 1000, torch.float32, 1003, 1).fill(c0 if beta else torch.full_like(c0, float("nan")))
            mg.linear("N", "T", alpha, a, b, beta, c.t, bias=v, act="relu")
            torch.cuda.synchronize()
            want = (torch.zeros(1000, device="cuda") if v is None else v).clamp(min=0).expand(33, 1000)
            assert torch.equal(c.t, want + beta * c0 if beta else want) and c.whole()


@pytest.mark.parametrize("act", ACTS)
def test_activations(act):
    """f over FP32's range, through a product of nothing: z is the bias. Limits at infinity; NaN stays."""
    z = torch.cat([torch.linspace(-12, 12, 20001), torch.linspace(-110, 110, 4001), 10.0 ** torch.linspace(-38, 38, 1001),
                   -(10.0 ** torch.linspace(-38, 38, 1001)), torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan])]).cuda()
    n = z.numel()
    a, b = torch.empty(1, 0, dtype=torch.bfloat16, device="cuda"), torch.empty(n, 0, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(1, n, device="cuda")
    mg.linear("N", "T", 1.0, a, b, 0.0, y, bias=z, act=act)
    dz, y2 = torch.empty(1, n, device="cuda"), torch.empty(1, n, device="cuda")
    mg.act_backward(torch.ones(1, n, device="cuda"), z[None], dz, act=act, y=y2)
    torch.cuda.synchronize()
    f, df, steps = act64(z, act)
    fine = torch.isfinite(z)
    near(y[0][fine], f[fine], f[fine].abs() * (steps[fine] + 1) * U32 + LOST)
    assert torch.equal(y2[0][fine], y[0][fine])
    # f' is a sum of two parts, each off by its own steps; the second is at most 1.13 and no larger than |z| of the first.
    near(dz[0][fine], df[fine], (steps[fine].clamp(max=400) * 2 + 16) * U32 * (df[fine].abs() + 0.2))
    for got, ends in ((y[0], (math.inf, -math.inf if act == "none" else 0.0)), (dz[0], (1.0, 1.0 if act == "none" else 0.0))):
        assert got[-3] == ends[0] and got[-2] == ends[1] and (torch.isnan(got[-1]) or (act == "none" and got is dz[0]) or (act == "none" and got[-1] == 1))


@pytest.mark.parametrize("ta,tb", ["NT", "NN", "TN"])
def test_linear_far_rows(ta, tb):
    """Rows whose offsets pass 32 bits, of both operands, of C, the residual and z."""
    M, N, K, ld = 6, 7, 9, 2**29 + 8
    g = gen(4)

    def far(rows, cols):
        t = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)[:, :cols]
        return t.copy_(torch.randint(-3, 4, (rows, cols), generator=g, device="cuda"))
    a, b = far(*((K, M) if ta == "T" else (M, K))), far(*((N, K) if tb == "T" else (K, N)))
    c, r, z = far(M, N), far(M, N), far(M, N)
    mg.linear(ta, tb, 1.0, a, b, 1.0, c, residual=r, z=z)
    torch.cuda.synchronize()
    x, y = (m.double().T.contiguous() if f == "T" else m.double() for m, f in ((a, ta), (b, tb)))
    assert torch.equal(z.double(), x @ y) and torch.equal(c.double(), x @ y + r.double())


# ---- the gated block


def run_gated(M, N, K, kind, seed):
    type, out, bias, act, _, _, keep, pad, off = kind
    g, dtype, ctype = gen(seed), DTYPE[type], DTYPE[out]
    a, G, U = stored(g, M, K, dtype, pad, off), stored(g, N, K, dtype, pad, off), stored(g, N, K, dtype, pad + 8, off)
    for t in (a, G, U):
        t.t.mul_(K**-0.25)
    bg, bu = (None, None) if bias is None else (torch.randn(N, generator=g, device="cuda").to(DTYPE[bias]) for _ in range(2))
    if seed % 2:
        bu = None
    h = Framed(M, N, ctype, N + pad, off)
    (zg, sg), (zu, su) = (room(keep, M, N, ctype, pad, off) if keep else (None, None) for _ in range(2))
    t = lambda x: None if x is None else x.t  # noqa: E731
    mg.gated(a.t, G.t, U.t, h.t, act=act, bias_g=bg, bias_u=bu, g=t(zg), scale_g=t(sg), u=t(zu), scale_u=t(su))
    torch.cuda.synchronize()
    g64, eg = product64(a.t, G.t, "N", "T", 1.0, bg)
    u64, eu = product64(a.t, U.t, "N", "T", 1.0, bu)
    f = act64(g64, act)[0]
    ef = act_limit(g64, eg, act)
    limit = ef * (u64.abs() + eu) + f.abs() * eu + (f * u64).abs() * U32
    near(h.t, f * u64, rounded(f * u64, limit, ctype))
    if zg is not None:
        check_kept(g64, eg, zg, sg)
        check_kept(u64, eu, zu, su)
    assert all(x.whole() for x in (a, G, U, h, zg, sg, zu, su) if x is not None)
    again = Framed(M, N, ctype)
    mg.gated(a.t, G.t, U.t, again.t, act=act, bias_g=bg, bias_u=bu, g=t(zg), scale_g=t(sg), u=t(zu), scale_u=t(su))
    torch.cuda.synchronize()
    assert torch.equal(again.t, h.t), "two calls differ"


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gated(M, N, K):
    for n, kind in enumerate(KINDS):
        run_gated(M, N, K, kind, 17 * n + M)


@pytest.mark.parametrize("M,N,K", LARGE)
def test_gated_large(M, N, K):
    for n in (0, 1, 3):
        run_gated(M, N, K, KINDS[n], M + n)


@pytest.mark.parametrize("type", ["bf16", "fp16"])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (24, 384, 4096), (130, 260, 900), (256, 128, 64), (300, 520, 192), (1024, 1024, 1024),
                                   (2048, 2304, 320), (64, 64, 16384), (257, 2049, 129)])
def test_gated_whole_numbers(M, N, K, pad, type):
    g = gen(M + K)
    a, G, U = (Framed(r, K, DTYPE[type], K + pad, pad).fill(torch.randint(-1, 2, (r, K), generator=g, device="cuda").float()) for r in (M, N, N))
    h, zg, zu = (torch.empty(M, N, device="cuda") for _ in range(3))
    mg.gated(a.t, G.t, U.t, h, act="relu", g=zg, u=zu)
    torch.cuda.synchronize()
    g64, u64 = (a.t.double() @ w.t.double().T.contiguous() for w in (G, U))
    assert torch.equal(zg.double(), g64) and torch.equal(zu.double(), u64)
    assert torch.equal(h.double(), g64.clamp(min=0) * u64)
    # Both projections as parts of one matrix, and as the same one.
    W = torch.cat([G.t, U.t])
    h2 = torch.empty_like(h)
    mg.gated(a.t, W[:N], W[N:], h2, act="relu")
    torch.cuda.synchronize()
    assert torch.equal(h2, h)
    mg.gated(a.t, W[N:], W[N:], h2, act="none")
    torch.cuda.synchronize()
    assert torch.equal(h2.double(), u64 * u64)


def test_kept_rows_of_nothing_and_not_finite():
    """8-bit checkpoints of zeros, NaN and infinities are what quantising z gives."""
    K, N = 64, 300
    a = torch.zeros(6, K, dtype=torch.bfloat16, device="cuda")
    a[1, 0], a[2, 0], a[3, 0], a[4, 0], a[5, 1] = 1.0, float("nan"), float("inf"), 1e-38, 1.0
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = (values(gen(1), 1, N)[0].abs() + 0.1).bfloat16()
    w[140, 1], w[7, 1] = float("nan"), float("inf")
    w[140, 0] = w[7, 0] = 0.0
    z, c = torch.empty(6, N, device="cuda"), torch.empty(6, N, device="cuda")
    q, s = mg.fp8_empty(6, N)
    mg.linear("N", "T", 1.0, a[:5], w, 0.0, c[:5], z=z[:5])
    mg.linear("N", "T", 1.0, a, w, 0.0, c, z=q, scale=s)
    mg.linear("N", "T", 1.0, a, w, 0.0, c, z=z)
    q2, s2 = mg.fp8_empty(6, N)
    mg.fp8_quantize(z, q2, s2)
    torch.cuda.synchronize()
    same = q.float().nan_to_num(nan=-1.0) == q2.float().nan_to_num(nan=-1.0)
    assert same.all() and torch.equal(s.nan_to_num(posinf=-1.0), s2.nan_to_num(posinf=-1.0))


# ---- the backward pass


def kept64(z, s):
    rows, cols = z.t.shape
    # As the kernel reads it: the product of a value and its scale, rounded once.
    return (z.t.float() * each(s.t, rows, cols, "row").float()).double() if s is not None else z.t.double()


def checkpoint(g, kind, rows, cols, dtype, pad, off):
    z, s = room(kind, rows, cols, dtype, pad, off)
    v = values(g, rows, cols)
    if s is None:
        z.fill(v)
    else:
        mg.fp8_quantize(v, z.t, s.t)
    return z, s


def sums_limit(terms, err, rows):
    """A sum over the rows in FP32: at most rows + 70 additions, of terms off by err."""
    return terms.abs().sum(0) * (rows + 70) * U32 + err.sum(0)


BACK = [(1, 1), (1, 4096), (3, 5), (7, 129), (64, 128), (65, 127), (130, 16), (200, 300), (1000, 260), (4, 9000), (2100, 136)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("type,keep", [("bf16", "e4m3"), ("bf16", "same"), ("fp16", "e5m2"), ("fp32", "e4m3"), ("fp32", "same")])
@pytest.mark.parametrize("rows,cols", BACK)
def test_act_backward(rows, cols, type, keep, act):
    dtype = DTYPE[type]
    for pad, off, beta in ((0, 0, 0.0), (3, 1, -0.5)):
        g = gen(rows + cols)
        dy, (z, s) = stored(g, rows, cols, dtype, pad, off), checkpoint(g, keep, rows, cols, dtype, pad, off)
        dz, y, db = Framed(rows, cols, dtype, cols + pad, off), Framed(rows, cols, dtype, cols + pad, off), Framed(1, cols, torch.float32, None, off)
        db0 = torch.randn(cols, generator=g, device="cuda") if beta else torch.full((cols,), float("nan"), device="cuda")
        db.t[0].copy_(db0)
        mg.act_backward(dy.t, z.t, dz.t, scale=None if s is None else s.t, act=act, y=y.t, dbias=db.t[0], beta=beta)
        torch.cuda.synchronize()
        z64 = kept64(z, s)
        f, df, steps = act64(z64, act)
        near(y.t, f, rounded(f, f.abs() * (steps + 2) * U32 + LOST, dtype))
        want = dy.t.double() * df
        err = dy.t.double().abs() * ((steps.clamp(max=400) * 2 + 16) * U32 * (df.abs() + 0.2)) + want.abs() * U32
        near(dz.t, want, rounded(want, err, dtype))
        total, limit = want.sum(0), sums_limit(want, err, rows)
        if beta:
            total, limit = total + beta * db0.double(), limit + db0.double().abs() * 2 * U32 + total.abs() * 2 * U32
        near(db.t[0], total, limit)
        assert all(t.whole() for t in (dy, z, s, dz, y, db) if t is not None)
        # dz alone; in dy's place, and in z's.
        alone = torch.empty(rows, cols, dtype=dtype, device="cuda")
        mg.act_backward(dy.t, z.t, alone, scale=None if s is None else s.t, act=act)
        here = dy.t.clone()
        mg.act_backward(here, z.t, here, scale=None if s is None else s.t, act=act)
        assert torch.equal(alone, dz.t) and torch.equal(here, dz.t)
        if s is None:
            here = z.t.clone()
            mg.act_backward(dy.t, here, here, act=act)
            y2, there = z.t.clone(), dy.t.clone()
            mg.act_backward(there, y2, there, act=act, y=y2)
            assert torch.equal(here, dz.t) and torch.equal(there, dz.t) and torch.equal(y2, y.t)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("type,keep", [("bf16", "e4m3"), ("bf16", "same"), ("fp16", "e5m2"), ("fp32", "e4m3"), ("fp32", "same")])
@pytest.mark.parametrize("rows,cols", BACK)
def test_gated_backward(rows, cols, type, keep, act):
    dtype = DTYPE[type]
    for pad, off, beta in ((0, 0, 0.0), (3, 1, 1.5)):
        g = gen(rows + cols)
        dh = stored(g, rows, cols, dtype, pad, off).fill(0.1 * torch.randn(rows, cols, generator=g, device="cuda"))
        (zg, sg), (zu, su) = (checkpoint(g, keep, rows, cols, dtype, pad, off) for _ in range(2))
        dg, du, h = (Framed(rows, cols, dtype, cols + pad, off) for _ in range(3))
        sums0 = torch.randn(2, cols, generator=g, device="cuda") if beta else torch.full((2, cols), float("nan"), device="cuda")
        bg, bu = sums0.clone()
        t = lambda x: None if x is None else x.t  # noqa: E731
        mg.gated_backward(dh.t, zg.t, zu.t, dg.t, du.t, scale_g=t(sg), scale_u=t(su), act=act, h=h.t, dbias_g=bg, dbias_u=bu, beta=beta)
        torch.cuda.synchronize()
        d, u, (f, df, steps) = dh.t.double(), kept64(zu, su), act64(kept64(zg, sg), act)
        ef = f.abs() * (steps + 2) * U32 + LOST
        edf = (steps.clamp(max=400) * 2 + 16) * U32 * (df.abs() + 0.2)
        wants = [(dg, d * u * df, (d * u).abs() * edf + (d * u * df).abs() * 3 * U32), (du, d * f, d.abs() * ef + (d * f).abs() * U32),
                 (h, f * u, u.abs() * ef + (f * u).abs() * U32)]
        for out, want, err in wants:
            near(out.t, want, rounded(want, err, dtype))
        for got, first, (_, want, err) in zip((bg, bu), sums0, wants):
            total, limit = want.sum(0), sums_limit(want, err, rows)
            if beta:
                total, limit = total + beta * first.double(), limit + first.double().abs() * 4 * U32 + total.abs() * 2 * U32
            near(got, total, limit)
        assert all(x.whole() for x in (dh, zg, sg, zu, su, dg, du, h) if x is not None)
        # Without h and the sums; one sum alone; in the places of what was read.
        p, q, b1 = torch.empty(rows, cols, dtype=dtype, device="cuda"), dh.t.clone(), sums0[1].clone()
        mg.gated_backward(q, zg.t, zu.t, p, q, scale_g=t(sg), scale_u=t(su), act=act, dbias_u=b1, beta=beta)
        assert torch.equal(p, dg.t) and torch.equal(q, du.t) and torch.equal(b1, bu)
        if sg is None:
            p, q, r = zg.t.clone(), zu.t.clone(), dh.t.clone()
            mg.gated_backward(r, p, q, p, q, act=act, h=r)
            assert torch.equal(p, dg.t) and torch.equal(q, du.t) and torch.equal(r, h.t)


def test_gradients_against_differences():
    rows, cols, step = 3, 40, 1e-6
    for act in ACTS[2:]:
        g = gen(11)
        z, u, dy = (torch.randn(rows, cols, generator=g, device="cuda") for _ in range(3))
        dz, dg, du = (torch.empty_like(z) for _ in range(3))
        mg.act_backward(dy, z, dz, act=act)
        mg.gated_backward(dy, z, u, dg, du, act=act)
        torch.cuda.synchronize()
        z, u, dy = (t.double() for t in (z, u, dy))
        f = lambda z, u: act64(z, act)[0] * u  # noqa: E731
        one = torch.ones_like(u)
        for got, up, down in ((dz, f(z + step, one), f(z - step, one)), (dg, f(z + step, u), f(z - step, u)),
                              (du, f(z, u + step), f(z, u - step))):
            # Elementwise, so all differences at once; they are good to about 1e-16 / step and step^2.
            assert (got.double() - dy * (up - down) / (2 * step)).abs().max() <= 1e-6 * max(1.0, float(got.abs().max()))


def test_backward_without_rows():
    e = torch.empty(0, 40, device="cuda")
    for beta, want in ((0.5, 0.5), (0.0, 0.0), (1.0, 1.0)):
        b, b2 = torch.ones(40, device="cuda"), torch.ones(40, device="cuda")
        mg.act_backward(e, e.clone(), torch.empty_like(e), act="silu", dbias=b, beta=beta)
        mg.gated_backward(e, e.clone(), e.clone(), torch.empty_like(e), torch.empty_like(e), dbias_g=b2, beta=beta)
        torch.cuda.synchronize()
        assert (b == want).all() and (b2 == want).all()


def test_backward_far_rows():
    rows, cols, ld = 5, 200, 2**30
    far = lambda: torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)[:, :cols]  # noqa: E731
    dy, z, dz = far(), far(), far()
    v = values(gen(3), rows, cols, torch.bfloat16), values(gen(4), rows, cols, torch.bfloat16)
    dy.copy_(v[0]), z.copy_(v[1])
    near_, db, db2 = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda"), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    mg.act_backward(dy, z, dz, act="silu", dbias=db)
    mg.act_backward(*v, near_, act="silu", dbias=db2)
    torch.cuda.synchronize()
    assert torch.equal(dz, near_) and torch.equal(db, db2)
