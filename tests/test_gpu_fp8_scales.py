"""Every kernel of the 8-bit product with scales that differ from row to row and block to block, in steady state.

The choice of a kernel rests on the size, C's width, the kind of scales and the alignment; each size below names the
tile it is made for. Operands of -1, 0 and 1 (so that the matrix cores drop nothing) and scales that are powers of two
have one exact result, whatever the order: each output has some 200 products that are not zero, spread over all of k,
of which FP16 holds the sum in quarters up to 512.
"""
import ctypes
import sys

import pytest

import fp32_gemm_nn_amd as mg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


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


def blocks(n):
    return (n + 127) // 128


def rows_apart(t, ld):
    """t's values in rows `ld` elements apart; what lies between is not set."""
    far = torch.empty(t.shape[0] * ld, dtype=torch.uint8, device="cuda").view(t.dtype).view(t.shape[0], ld)[:, :t.shape[1]]
    far.copy_(t)
    return far


def powers(g, *shape):
    return torch.exp2(torch.randint(-1, 2, shape, generator=g, device="cuda").float())


def tables(g, M, N, K, block):
    return powers(g, blocks(K), M), powers(g, *((blocks(K), N) if block == "row" else (blocks(N), blocks(K))))


def each(s, rows, K, block):
    i, k = torch.arange(rows, device="cuda"), torch.arange(K, device="cuda") // 128
    return s.double()[k][:, i].T if block == "row" else s.double()[i // 128][:, k]


def signs(g, rows, K, dtype, share=1.0):
    v = torch.randint(0, 2, (rows, K), generator=g, device="cuda").float() * 2 - 1
    if share < 1:
        v *= torch.rand(rows, K, generator=g, device="cuda") < share
    return v.to(dtype)


def wanted(a, sa, b, sb, block):
    K = a.shape[1]
    return (a.double() * each(sa, a.shape[0], K, "row")) @ (b.double() * each(sb, b.shape[0], K, block)).T.contiguous()


# 256 x 256 with five blocks of k and more (each buffer is filled again and again), whole and short last blocks, odd
# edges; 128 x 128 alone and with k shared; 64 x 128; then 64 x 64 to 16 x 16 without barriers. Rows three bytes
# further apart take the 128 x 128 and 64 x 128 tiles that read at any address instead of the first three kinds.
SIZES = [(4096, 4096, 700), (4001, 4005, 1500), (2999, 3003, 1100), (4096, 3840, 640), (2048, 4096, 1024),
         (2607, 502, 7188), (1024, 2048, 8192), (1000, 1300, 700), (512, 2048, 2048), (500, 2040, 1000),
         (130, 4100, 1300), (460, 1900, 2500), (300, 1000, 1030), (100, 3000, 1000), (250, 2040, 900),
         (36, 3600, 1100), (300, 700, 2000), (40, 2000, 3000), (9, 3001, 900), (1, 700, 8192)]


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_scales(M, N, K, block, pad):
    ld = K + -K % 16 + pad
    for k, (fa, fb, out) in enumerate(((E4M3, E5M2, torch.float16), (E5M2, E4M3, torch.float16),
                                       (E4M3, E4M3, torch.float32))):
        g = gen(M + N + K + k)
        a = rows_apart(signs(g, M, K, fa), ld)
        b = rows_apart(signs(g, N, K, fb, 200 / K), ld)
        sa, sb = tables(g, M, N, K, block)
        c = torch.full((M, N), float("nan"), dtype=out, device="cuda")
        mg.fp8_gemm(1.0, a, sa, b, sb, 0.0, c, block=block)
        torch.cuda.synchronize()
        want = wanted(a, sa, b, sb, block)
        assert want.abs().max() <= 512
        assert torch.equal(c.double(), want), (fa, fb, out, int((c.double() != want).sum()))


# Rows so far apart that 32-bit offsets inside a tile end: 2^24 where tiles go through LDS, 2^26 elsewhere.
@pytest.mark.parametrize("ld", [2**24 - 16, 2**24, 2**26 - 16, 2**26 + 3])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", [(70, 150, 300), (130, 140, 5000)])
def test_far_rows(M, N, K, block, ld):
    if torch.cuda.mem_get_info()[0] < 2 * (M + N) * ld:
        pytest.skip("not enough memory")
    for k, (fa, fb, out) in enumerate(((E4M3, E4M3, torch.float16), (E5M2, E4M3, torch.float32))):
        g = gen(M + k)
        a = rows_apart(signs(g, M, K, fa), ld)
        b = rows_apart(signs(g, N, K, fb, 200 / K), ld)
        sa, sb = tables(g, M, N, K, block)
        c = torch.full((M, N), float("nan"), dtype=out, device="cuda")
        mg.fp8_gemm(1.0, a, sa, b, sb, 0.0, c, block=block)
        torch.cuda.synchronize()
        want = wanted(a, sa, b, sb, block)
        assert want.abs().max() <= 512
        assert torch.equal(c.double(), want), (out, int((c.double() != want).sum()))
        del a, b
    torch.cuda.empty_cache()


# Products that share k: the tile of 128 x 128 for C of 16 and of 32 bits, rows aligned and not.
SHARED = [(2607, 502, 7188, 0, torch.bfloat16), (2607, 502, 7188, 0, torch.float32), (1024, 2048, 8192, 0, torch.float32),
          (1024, 2048, 8192, 3, torch.float16), (1024, 2048, 8192, 3, torch.float32)]


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K,pad,out", SHARED)
def test_shared_k_gives_the_same_bits_each_time(M, N, K, pad, out, block):
    """With values whose sums round: the order of the partial sums does not depend on which workgroup ends last."""
    g, ld = gen(3), K + -K % 16 + pad
    a, b = (rows_apart(torch.randn(n, K, generator=g, device="cuda").to(E4M3), ld) for n in (M, N))
    sa = torch.rand(blocks(K), M, generator=g, device="cuda")
    sb = torch.rand((blocks(K), N) if block == "row" else (blocks(N), blocks(K)), generator=g, device="cuda")
    first = None
    for _ in range(6):
        c = torch.full((M, N), float("nan"), dtype=out, device="cuda")
        mg.fp8_gemm(1.0, a, sa, b, sb, 0.0, c, block=block)
        torch.cuda.synchronize()
        first = c if first is None else first
        assert torch.equal(c, first)


@pytest.fixture(scope="module")
def streams():
    """Two streams of their own, never destroyed: torch hands its own out again, and a graph keeps the workspace of
    the stream that it was captured on. The first never has a workspace, since nothing but captures runs on it."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.init()
    create = mg.load_library().hipStreamCreate       # of the HIP runtime that the library is linked against
    create.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
    made = []
    for _ in range(2):
        handle = ctypes.c_void_p()
        assert create(ctypes.byref(handle)) == 0
        made.append(torch.cuda.ExternalStream(handle.value))
    return made


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K,pad,out", SHARED)
def test_shared_k_captured_with_and_without_a_workspace(M, N, K, pad, out, block, streams):
    """A stream that is captured before it has a workspace gets a graph that does not share k, with the same exact
    result; one that has a workspace gets one that shares it."""
    g, ld = gen(4), K + -K % 16 + pad
    a, b = rows_apart(signs(g, M, K, E4M3), ld), rows_apart(signs(g, N, K, E4M3, 50 / K), ld)
    sa, sb = torch.ones(blocks(K), M, device="cuda"), tables(g, M, N, K, block)[1]
    want = wanted(a, sa, b, sb, block)
    assert want.abs().max() <= 128          # in halves: BF16 holds them up to that
    c = torch.empty(M, N, dtype=out, device="cuda")
    for warm, stream in zip((False, True), streams):
        call = lambda: mg.fp8_gemm(1.0, a, sa, b, sb, 0.0, c, block=block, stream=stream.cuda_stream)  # noqa: E731
        torch.cuda.synchronize()
        if warm:
            call()
            stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
        for rep in range(3):
            c.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.double(), want), (warm, rep)
        del graph


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", [(5, 9, 8), (1, 700, 2048), (64, 1024, 2048), (512, 2048, 2048), (1000, 1300, 700),
                                   (2048, 4096, 1024), (4096, 4096, 700)])
def test_scales_whose_product_is_at_the_edge(M, N, K, block):
    """The least and the largest products of two scales that FP32 holds, shared out between them in different ways."""
    g = gen(M)
    for total, many in ((-126, 60), (127, 1)):
        a = signs(g, M, K, E4M3)
        b = signs(g, N, K, E5M2, min(1.0, many / K)) if many > 1 else torch.zeros(N, K, device="cuda").to(E5M2)
        if many == 1:
            at = torch.randint(0, K, (N,), generator=g, device="cuda")
            b = b.float().scatter_(1, at[:, None], -1.0).to(E5M2)
        a, b = (rows_apart(t, K + -K % 16) for t in (a, b))
        for ea in (-110, -63, -16) if total < 0 else (110, 63, 16):
            sa = torch.full((blocks(K), M), 2.0**ea, device="cuda")
            sb = torch.full((blocks(K), N) if block == "row" else (blocks(N), blocks(K)), 2.0 ** (total - ea), device="cuda")
            want = a.double() @ b.double().T.contiguous()
            assert want.abs().max() <= (1 if many == 1 else 256)
            for out in (torch.float32, torch.bfloat16):
                c = torch.full((M, N), float("nan"), dtype=out, device="cuda")
                mg.fp8_gemm(1.0, a, sa, b, sb, 0.0, c, block=block)
                torch.cuda.synchronize()
                assert torch.equal(c.double(), want * 2.0**total), (total, ea, out)
