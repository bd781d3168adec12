"""The feed-forward block's operators together, as a step uses them: norm, gated block with 8-bit checkpoints, the way
back down, and the backward pass; on other streams, in graphs, and without a workspace."""
import sys

import pytest

import fp32_gemm_nn_amd as mg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 1e-5
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _named(request):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.__stderr__.write(f"[gpu] {request.node.name}\n")
    sys.__stderr__.flush()
    mg.load_library()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Block:
    """y = x + W_d (silu(W_g n) * (W_u n)), n = norm(x), in BF16, and its gradients. rows x width, `inner` between."""

    def __init__(self, rows, width, inner, keep=True, seed=3):
        g = gen(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.x, self.dy = r(rows, width).to(BF), r(rows, width).to(BF)
        self.norm = 1 + 0.1 * r(width)
        self.wg, self.wu = ((r(inner, width) / width**0.5).to(BF) for _ in range(2))
        self.wd = (r(width, inner) / inner**0.5).to(BF)
        e = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.n, self.y, self.dn, self.dx = (e(rows, width) for _ in range(4))
        self.rstd = e(rows, dtype=torch.float32)
        self.h, self.dh, self.dg, self.du = (e(rows, inner) for _ in range(4))
        self.keep = (mg.fp8_empty(rows, inner) + mg.fp8_empty(rows, inner)) if keep else (e(rows, inner), None, e(rows, inner), None)
        self.dwg, self.dwu = (torch.zeros(inner, width, device="cuda") for _ in range(2))
        self.dwd, self.dnorm = torch.zeros(width, inner, device="cuda"), e(width, dtype=torch.float32)

    def step(self, stream=None):
        g, sg, u, su = self.keep
        kw = dict(stream=stream)
        mg.rmsnorm(self.x, self.norm, EPS, y=self.n, rstd=self.rstd, **kw)
        mg.gated(self.n, self.wg, self.wu, self.h, g=g, scale_g=sg, u=u, scale_u=su, **kw)
        mg.linear("N", "T", 1.0, self.h, self.wd, 1.0, self.y, residual=self.x, **kw)
        # The backward pass: h again, from the checkpoints.
        mg.linear("N", "N", 1.0, self.dy, self.wd, 0.0, self.dh, **kw)
        mg.gated_backward(self.dh, g, u, self.dg, self.du, scale_g=sg, scale_u=su, h=self.h, **kw)
        mg.linear("T", "N", 1.0, self.dy, self.h, 0.0, self.dwd, **kw)
        mg.linear("T", "N", 1.0, self.dg, self.n, 0.0, self.dwg, **kw)
        mg.linear("T", "N", 1.0, self.du, self.n, 0.0, self.dwu, **kw)
        mg.linear("N", "N", 1.0, self.dg, self.wg, 0.0, self.dn, **kw)
        mg.linear("N", "N", 1.0, self.du, self.wu, 1.0, self.dn, **kw)
        mg.rmsnorm_backward(self.dn, self.x, self.norm, self.rstd, self.dx, self.dnorm, dh=self.dy, **kw)

    outs = ("y", "dx", "dwg", "dwu", "dwd", "dnorm")

    def results(self):
        return [getattr(self, n) for n in self.outs]

    def plain(self):
        """The same by autograd, in 64 bits."""
        x, norm, wg, wu, wd = (t.double().detach().requires_grad_() for t in (self.x, self.norm, self.wg, self.wu, self.wd))
        n = x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * norm
        g, u = n @ wg.T, n @ wu.T
        y = x + (g * torch.sigmoid(g) * u) @ wd.T
        y.backward(self.dy.double())
        return y.detach(), x.grad, wg.grad, wu.grad, wd.grad, norm.grad


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("rows,width,inner", [(1, 64, 128), (37, 100, 260), (300, 512, 1024), (1030, 520, 700)])
def test_step(rows, width, inner, keep):
    b = Block(rows, width, inner, keep)
    b.step()
    torch.cuda.synchronize()
    # Roundings to nearest, relative: 2^-8 for each of the BF16 matrices on the way (n, h, y; dh, dg or du, dn, dx, and
    # n and h again), each of which enters its product once and linearly; 2^-4 each for g and u in 8 bits, of which the
    # gradients are at most quadratic (dg = dh u f'(g): u once, and g through f', whose slope is at most 1 of its size).
    # A sum of products whose factors are off by independent roundings is off by no more than that of its size.
    eight = 3 * 2.0**-4 if keep else 0.0
    limits = dict(y=3 * 2.0**-8, dx=9 * 2.0**-8 + eight, dwg=6 * 2.0**-8 + eight, dwu=6 * 2.0**-8 + eight, dwd=4 * 2.0**-8 + eight,
                  dnorm=9 * 2.0**-8 + eight)
    for name, got, want in zip(b.outs, b.results(), b.plain()):
        off = float((got.double() - want).norm() / want.norm())
        sys.__stderr__.write(f"[gpu] {name} {off:.2e}\n")
        assert off <= limits[name], name


def test_gradients_of_small_values_against_differences():
    """A loss's slope along a direction, from the block's gradients in 64-bit differences of the plain form."""
    b = Block(5, 48, 96, keep=False)
    b.step()
    torch.cuda.synchronize()
    x, norm, wg, wu, wd, dy = (t.double() for t in (b.x, b.norm, b.wg, b.wu, b.wd, b.dy))

    def loss(x, wg, wu, wd):
        n = x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * norm
        g, u = n @ wg.T, n @ wu.T
        return float(((x + (g * torch.sigmoid(g) * u) @ wd.T) * dy).sum())
    g = gen(8)
    for at, grad in ((0, b.dx), (1, b.dwg), (2, b.dwu), (3, b.dwd)):
        args = [x, wg, wu, wd]
        d = torch.randn(args[at].shape, generator=g, device="cuda", dtype=torch.float64)
        d = d * (grad.double().abs() > 0)
        d = torch.where(grad.double() * d >= 0, d, -d)          # a direction in which every part adds
        ends = []
        for e in (1e-6, -1e-6):
            moved = list(args)
            moved[at] = args[at] + e * d
            ends.append(loss(*moved))
        slope, want = (ends[0] - ends[1]) / 2e-6, float((grad.double() * d).sum())
        # Nine BF16 roundings of either sign; the parts have one sign, so their sum is off by at most that share, and
        # small parts whose sign the roundings may turn weigh little.
        assert abs(slope - want) <= 9 * 2.0**-8 * want


def test_another_stream_and_a_graph():
    stream = torch.cuda.Stream()
    b, other = Block(200, 264, 520), Block(200, 264, 520)
    ins = (b.x, b.dy, b.wg)
    torch.cuda.synchronize()
    saved = [t.clone() for t in ins]
    turned = [t.flip(0).contiguous() for t in ins]
    want = []
    for source in (saved, turned):
        for t, v in zip(ins, source):
            t.copy_(v)
        torch.cuda.synchronize()
        b.step(stream.cuda_stream)
        stream.synchronize()
        want.append([t.clone() for t in b.results()])
    other.step()
    torch.cuda.synchronize()
    for x, y in zip(other.results(), want[0]):
        assert torch.equal(x, y), "the current stream's result differs"
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        b.step(torch.cuda.current_stream().cuda_stream)
    for rep in range(6):
        for t, v in zip(ins, (saved, turned)[rep % 2]):
            t.copy_(v)
        for t in b.results():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(b.results(), want[rep % 2]):
            assert torch.equal(x, y), f"replay {rep}"
        other.step()
    del graph


def test_captured_without_a_workspace():
    """Captured on a stream that has none: products whose k is shared otherwise, and sums over many rows, run whole."""
    g = gen(1)
    whole = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").to(BF)  # noqa: E731
    a, w, u = whole(70, 8192), whole(264, 8192), whole(264, 8192)
    c, h = torch.empty(70, 264, device="cuda"), torch.empty(70, 264, device="cuda")
    q, s = mg.fp8_empty(70, 264)
    dy, z = torch.randint(-3, 4, (3000, 264), generator=g, device="cuda").float(), torch.randn(3000, 264, generator=g, device="cuda")
    dz, db, db2 = torch.empty_like(z), torch.empty(264, device="cuda"), torch.empty(264, device="cuda")
    eager = torch.empty(70, 264, device="cuda")
    mg.linear("N", "T", 1.0, a, w, 0.0, eager)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        on = dict(stream=torch.cuda.current_stream().cuda_stream)
        mg.linear("N", "T", 1.0, a, w, 0.0, c, z=q, scale=s, **on)
        mg.gated(a, w, u, h, act="none", **on)
        mg.act_backward(dy, z, dz, act="relu", dbias=db, **on)
        mg.gated_backward(dy, z, z, dz, torch.empty_like(z), act="relu", dbias_u=db2, **on)
    g64, u64 = (a.double() @ t.double().T.contiguous() for t in (w, u))
    for rep in range(3):
        for t in (c, h, db, db2):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.double(), g64) and torch.equal(c, eager)
        want = g64 * u64
        assert ((h.double() - want).abs() <= want.abs() * 2.0**-24).all()
        assert torch.equal(db.double(), (dy.double() * (z > 0)).sum(0))
        total = (dy.double() * z.double().clamp(min=0))
        assert ((db2.double() - total.sum(0)).abs() <= total.abs().sum(0) * 3070 * 2.0**-24).all()
    del graph


def test_two_streams_at_once():
    """Two streams have workspaces of their own; calls in turn on both, nothing waiting between."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    g = gen(5)
    sets = []
    for _ in streams:
        a = torch.randint(-3, 4, (120, 4096), generator=g, device="cuda").to(BF)
        w = torch.randint(-3, 4, (300, 4096), generator=g, device="cuda").to(BF)
        dy = torch.randint(-3, 4, (4000, 300), generator=g, device="cuda").float()
        sets.append((a, w, torch.empty(120, 300, device="cuda"), mg.fp8_empty(120, 300), dy, torch.empty_like(dy), torch.empty(300, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (a, w, c, (q, s), dy, dz, db) in zip(streams, sets):
            mg.linear("N", "T", 1.0, a, w, 0.0, c, z=q, scale=s, stream=st.cuda_stream)
            mg.act_backward(dy, dy, dz, act="none", dbias=db, stream=st.cuda_stream)
    torch.cuda.synchronize()
    for a, w, c, _, dy, dz, db in sets:
        assert torch.equal(c.double(), a.double() @ w.double().T.contiguous())
        assert torch.equal(dz, dy) and torch.equal(db.double(), dy.double().sum(0))


def test_weights_and_norm_of_the_8_bit_layer_beside_it():
    """h in BF16 goes on in 8 bits: quantised for the 8-bit product, as a layer with 8-bit weights takes it."""
    b = Block(130, 256, 384)
    b.step()
    q, s = mg.fp8_empty(130, 384)
    W, Ws = mg.fp8_empty(256, 384, "tile")
    y = torch.empty(130, 256, dtype=BF, device="cuda")
    mg.fp8_quantize(b.h, q, s)
    mg.fp8_quantize(b.wd, W, Ws, block="tile")
    mg.fp8_gemm(1.0, q, s, W, Ws, 0.0, y)
    torch.cuda.synchronize()
    want = b.h.double() @ b.wd.double().T.contiguous()
    # Two E4M3 operands and a BF16 result.
    assert float((y.double() - want).norm() / want.norm()) <= 2 * 2.0**-4 + 2.0**-8


@pytest.mark.parametrize("ta,tb", ["NT", "NN", "TN", "TT"])
def test_sizes_that_end_everywhere(ta, tb):
    """Each remainder of rows, columns and k around a tile's and a chunk's size, against 64 bits, whole numbers."""
    g = gen(6)
    for M, N, K in ((63, 65, 63), (64, 127, 65), (65, 128, 127), (127, 129, 129), (128, 255, 7), (129, 256, 9), (255, 257, 191), (257, 8, 193),
                    (8, 264, 72), (7, 15, 1), (9, 1, 17), (512, 640, 8), (320, 384, 56)):
        a, b = (torch.randint(-4, 5, (c, r) if t == "T" else (r, c), generator=g, device="cuda").to(BF) for r, c, t in ((M, K, ta), (K, N, tb)))
        c = torch.empty(M, N, device="cuda")
        mg.linear(ta, tb, 1.0, a, b, 0.0, c)
        torch.cuda.synchronize()
        x, y = (t.double().T.contiguous() if f == "T" else t.double() for t, f in ((a, ta), (b, tb)))
        assert torch.equal(c.double(), x @ y), (M, N, K)


@pytest.mark.parametrize("out", [BF, torch.float32])
@pytest.mark.parametrize("M,N,K", [(4096, 4096, 1024), (1030, 2060, 512), (300, 500, 200), (130, 130, 2048), (40, 500, 200), (1, 500, 200)])
def test_outputs_at_any_alignment(M, N, K, out):
    """Aligned operands, and outputs and a residual whose rows lie anywhere: nothing beside them is written."""
    g = gen(7)
    a, w, u = (torch.randint(-1, 2, (r, K), generator=g, device="cuda") * (torch.arange(K, device="cuda") % max(1, K // 200) == 0) for r in (M, N, N))
    a, w, u = (t.to(BF) for t in (a, w, u))          # sums of at most 200: whole numbers that BF16 holds

    def place(dtype):
        raw = torch.full((M * (N + 1) + 9,), 77.0, dtype=dtype, device="cuda")
        return raw, raw[1:1 + M * (N + 1)].view(M, N + 1)[:, :N]

    def beside(raw, t):
        v = raw.clone()
        v[1:1 + M * (N + 1)].view(M, N + 1)[:, :N] = 77.0
        return bool((v == 77.0).all())
    (rc, c), (rz, z), (rr, r) = place(out), place(out), place(out)
    r.copy_(torch.randint(-9, 10, (M, N), generator=g, device="cuda"))
    x, y = (a.double() @ t.double().T.contiguous() for t in (w, u))
    mg.linear("N", "T", 1.0, a, w, 1.0, c, residual=r, z=z, act="relu")
    torch.cuda.synchronize()
    assert torch.equal(z.double(), x) and torch.equal(c.double(), (x.clamp(min=0) + r.double()).to(out).double())
    assert all(beside(*p) for p in ((rc, c), (rz, z), (rr, r)))
    mg.gated(a, w, u, c, act="relu", g=z, u=r)
    torch.cuda.synchronize()
    assert torch.equal(z.double(), x) and torch.equal(r.double(), y) and torch.equal(c.double(), (x.clamp(min=0) * y).to(out).double())
    assert all(beside(*p) for p in ((rc, c), (rz, z), (rr, r)))
    q = [torch.full((M * (N + 3) + 9,), 0x5B, dtype=torch.uint8, device="cuda") for _ in range(2)]
    p, p2 = (t[5:5 + M * (N + 3)].view(M, N + 3)[:, :N].view(torch.float8_e4m3fn) for t in q)
    s, s2, want, ws = *(torch.empty((N + 127) // 128, M, device="cuda") for _ in range(2)), *mg.fp8_empty(M, N)
    mg.gated(a, w, u, c, act="none", g=p, scale_g=s, u=p2, scale_u=s2)
    mg.fp8_quantize(x.float(), want, ws)
    torch.cuda.synchronize()
    assert torch.equal(p.view(torch.uint8), want.view(torch.uint8)) and torch.equal(s, ws)
    mg.fp8_quantize(y.float(), want, ws)
    torch.cuda.synchronize()
    assert torch.equal(p2.view(torch.uint8), want.view(torch.uint8)) and torch.equal(s2, ws)
    for t in q:
        t[5:5 + M * (N + 3)].view(M, N + 3)[:, :N] = 0x5B
        assert (t == 0x5B).all()


@pytest.mark.parametrize("type", [BF, torch.float16])
@pytest.mark.parametrize("ta,tb", ["NT", "NN", "TN", "TT"])
def test_sizes_of_every_tile(ta, tb, type):
    """From outputs that few workgroups share to those that fill the card, k whole and shared: each tile size in turn.
    Whole numbers, K not a whole number of blocks; outputs in FP32 (exact) and in the operands' type (rounded once)."""
    g = gen(8)
    for M, N, K in ((104, 4208, 544), (112, 4176, 1616), (3440, 4752, 328), (2960, 2600, 328), (4216, 416, 328), (4792, 200, 2544), (4304, 136, 3032),
                    (4272, 904, 328), (3344, 2328, 328), (1752, 4640, 328)):
        a, b = (torch.randint(-4, 5, (c, r) if t == "T" else (r, c), generator=g, device="cuda").to(type) for r, c, t in ((M, K, ta), (K, N, tb)))
        x, y = (t.double().T.contiguous() if f == "T" else t.double() for t, f in ((a, ta), (b, tb)))
        want = x @ y
        for out in (torch.float32, type):
            c = torch.full((M, N), float("nan"), dtype=out, device="cuda")
            mg.linear(ta, tb, 1.0, a, b, 0.0, c)
            torch.cuda.synchronize()
            assert torch.equal(c, want.to(out)), (M, N, K, out)


@pytest.mark.parametrize("type", [BF, torch.float16])
def test_gated_sizes_of_every_tile(type):
    g = gen(9)
    for M, N, K in ((400, 4240, 344), (40, 4216, 3152), (72, 4392, 520), (104, 2080, 2280), (2624, 248, 336), (608, 3272, 328), (904, 4264, 328)):
        a, w, u = (torch.randint(-4, 5, (r, K), generator=g, device="cuda").to(type) for r in (M, N, N))
        x, y = (a.double() @ t.double().T.contiguous() for t in (w, u))
        c, z, z2 = (torch.full((M, N), float("nan"), device="cuda") for _ in range(3))
        mg.gated(a, w, u, c, act="relu", g=z, u=z2)
        torch.cuda.synchronize()
        assert torch.equal(z.double(), x) and torch.equal(z2.double(), y) and torch.equal(c, (x.clamp(min=0) * y).float()), (M, N, K)
