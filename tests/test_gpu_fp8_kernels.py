"""Sizes that reach every kernel of the 8-bit product, in both alignments, with exact results.

Small whole numbers have one sum whatever the order, so a value read before it landed, a block counted twice or
a scale of another row shows as a difference. Results with 16 bits keep sums below 2048, where FP16 holds every
whole number; their products are of one size, so the matrix cores drop nothing.
"""
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


def blocks(n):
    return (n + 127) // 128


def matrix(g, rows, cols, dtype, most, pad):
    """Whole numbers up to `most` in 8 bits, rows `pad` bytes further apart than the next multiple of 16."""
    t = torch.full((rows, cols + -cols % 16 + pad), float("nan"), device="cuda").to(dtype)[:, :cols]
    t.copy_(torch.randint(-most, most + 1, (rows, cols), generator=g, device="cuda").float())
    return t


def powers(g, *shape):
    return torch.exp2(torch.randint(-1, 2, shape, generator=g, device="cuda").float())


# Every tile shape (16 x 16 to 256 x 256), k shared by workgroups and not, whole blocks of k and not.
SIZES = [(1, 700, 8192), (16, 900, 130), (20, 4100, 300), (64, 1024, 2048), (100, 3000, 1000), (300, 1000, 1030),
         (500, 2050, 900), (700, 1400, 640), (1000, 1300, 700), (1500, 1500, 1600), (600, 3000, 3000),
         (2500, 2600, 400), (3000, 3000, 300), (2100, 4100, 260), (4096, 4096, 256), (1024, 2048, 8192),
         (257, 8000, 4100), (3001, 2999, 16), (2048, 2048, 2048), (331, 5752, 352), (136, 7840, 2048),
         (418, 3648, 2580)]


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_whole_numbers(M, N, K, block, pad):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    table = (blocks(K), N) if block == "row" else (blocks(N), blocks(K))
    i, j, k = (torch.arange(n, device="cuda") for n in (M, N, K))
    for fa, fb, out, most, beta in ((E4M3, E5M2, torch.float32, 3, 1.0), (E5M2, E4M3, torch.float16, 1, 0.0)):
        a, b = matrix(g, M, K, fa, most, pad), matrix(g, N, K, fb, most, pad)
        if out == torch.float32:
            sa, sb = powers(g, blocks(K), M), powers(g, *table)
        else:
            # Half of the products are zero, so that sums of any length stay small.
            b.copy_(torch.where(k[None] % max(1, K // 1000) == 0, b.float(), 0.0))
            sa, sb = torch.ones(blocks(K), M, device="cuda"), torch.ones(table, device="cuda")
        c0 = torch.randint(-9, 10, (M, N), generator=g, device="cuda").to(out)
        c = c0.clone()
        mg.fp8_gemm(1.0, a, sa, b, sb, beta, c, block=block)
        torch.cuda.synchronize()
        x = a.double() * sa.double()[k // 128][:, i].T
        y = b.double() * (sb.double()[k // 128][:, j].T if block == "row" else sb.double()[j // 128][:, k // 128])
        want = x @ y.T.contiguous() + beta * c0.double()
        assert out == torch.float32 or want.abs().max() <= 2048
        assert torch.equal(c.double(), want), int((c.double() != want).sum())


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (40, 2000, 3000), (700, 1400, 640), (1024, 2048, 8192),
                                   (3000, 3000, 300)])
def test_the_same_bits_each_time(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(7)
    a, sa = torch.randn(M, K, generator=g, device="cuda").to(E4M3), torch.rand(blocks(K), M, device="cuda")
    b, sb = torch.randn(N, K, generator=g, device="cuda").to(E4M3), torch.rand(blocks(N), blocks(K), device="cuda")
    first = None
    for _ in range(5):
        c = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        mg.fp8_gemm(1.0, a, sa, b, sb, 0.0, c)
        torch.cuda.synchronize()
        first = c if first is None else first
        assert torch.equal(c, first)
