"""The feed-forward block's entry points on the host: what they refuse.

Nothing here launches a kernel: every C call below fails validation or takes
a quick return, both of which happen before any HIP call, and the tensor
forms are given tensors that they refuse.
"""
import pytest

import fp32_gemm_nn_amd as mg

torch = pytest.importorskip("torch")

P, MOST = 0x10000, 2**31 - 1   # never dereferenced

LINEAR = dict(transA="N", transB="T", type=1, M=8, N=300, K=200, alpha=1.0, A=P, lda=200, B=P, ldb=200, biastype=0, bias=P, act=2,
              ctype=0, beta=1.0, R=P, ldr=300, C=P, ldc=300, ztype=3, z=P, ldz=300, zscale=P, lds=8)
GATED = dict(type=2, M=8, N=300, K=200, A=P, lda=200, G=P, ldg=200, U=P, ldu=200, biastype=2, biasG=P, biasU=P, act=2, htype=2, h=P,
             ldh=300, ztype=4, g=P, ldg_=300, gscale=P, ldsg=8, u=P, ldu_=300, uscale=P, ldsu=8)
ACT = dict(type=1, rows=3, cols=200, dy=P, lddy=200, act=3, ztype=3, z=P, ldz=200, zscale=P, lds=3, dz=P, lddz=200, y=P, ldy=200, beta=0.0,
           dbias=P)
BACK = dict(type=0, rows=3, cols=200, dh=P, lddh=200, act=4, ztype=4, g=P, ldg=200, gscale=P, ldsg=3, u=P, ldu=200, uscale=P, ldsu=3,
            dg=P, lddg=200, du=P, lddu=200, h=P, ldh=200, beta=0.0, dbiasG=P, dbiasU=P)


@pytest.mark.parametrize("kw,code", [
    (dict(transA="X"), -1), (dict(transB="Q"), -2), (dict(type=0), -30), (dict(type=3), -30), (dict(M=-1), -3), (dict(N=-1), -4),
    (dict(K=-1), -5), (dict(A=0), -7), (dict(lda=199), -8), (dict(transA="T", lda=7), -8), (dict(lda=0, K=0), -8), (dict(B=0), -9),
    (dict(ldb=199), -10), (dict(transB="N", ldb=299), -10), (dict(biastype=2), -30), (dict(act=5), -39), (dict(act=-1), -39),
    (dict(ctype=2), -30), (dict(ctype=3), -30), (dict(ldr=299), -37), (dict(C=0), -12), (dict(ldc=299), -13), (dict(ztype=1), -30),
    (dict(ldz=299), -37), (dict(zscale=0), -36), (dict(lds=7), -38), (dict(N=MOST, ldb=MOST, ldc=MOST, ldr=MOST, ldz=MOST), -21),
    (dict(K=MOST, lda=MOST, ldb=MOST), -21), (dict(M=MOST, lds=MOST), -21), (dict(M=64 * 2**12, N=128 * 2**11, ldc=MOST, ldr=MOST, ldz=MOST, lds=MOST), -21),
    # The first bad argument wins; nothing is refused of what is not read or wanted.
    (dict(M=-1, A=0, act=9), -3), (dict(alpha=0.0, A=0, B=0, C=0), -12), (dict(bias=0, biastype=7, ldc=0), -13),
    (dict(beta=0.0, ldr=0, ldc=0), -13), (dict(R=0, ldr=0, ldc=0), -13),
])
def test_linear_refuses(kw, code):
    assert mg.mi_linear(**{**LINEAR, **kw}) == code
    assert mg.mi_sgemm_status_string(code) not in ("", "unknown status")


@pytest.mark.parametrize("kw,code", [
    (dict(type=0), -30), (dict(M=-1), -3), (dict(N=-1), -4), (dict(K=-1), -5), (dict(A=0), -7), (dict(lda=199), -8), (dict(G=0), -9),
    (dict(ldg=199), -10), (dict(U=0), -9), (dict(ldu=199), -10), (dict(biastype=1), -30), (dict(biasG=0, biastype=1), -30), (dict(act=5), -39),
    (dict(htype=1), -30), (dict(h=0), -12), (dict(ldh=299), -13), (dict(ztype=1), -30), (dict(g=0), -35), (dict(u=0), -35), (dict(ldg_=299), -37),
    (dict(ldu_=299), -37), (dict(gscale=0), -36), (dict(uscale=0), -36), (dict(ldsg=7), -38), (dict(ldsu=7), -38),
    (dict(N=MOST, ldh=MOST, ldg_=MOST, ldu_=MOST), -21), (dict(g=0, u=0, ztype=9, ldh=0), -13), (dict(biasG=0, biasU=0, biastype=9, ldh=0), -13),
])
def test_gated_refuses(kw, code):
    assert mg.mi_gated(**{**GATED, **kw}) == code


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), -30), (dict(rows=-1), -32), (dict(cols=-1), -33), (dict(dy=0), -34), (dict(lddy=199), -37), (dict(act=5), -39),
    (dict(ztype=2), -30), (dict(z=0), -34), (dict(ldz=199), -37), (dict(zscale=0), -36), (dict(lds=2), -38), (dict(dz=0), -35),
    (dict(lddz=199), -37), (dict(ldy=199), -37), (dict(ztype=1, zscale=0, lds=0, lddz=1), -37),
    (dict(cols=2**31 - 128, lddy=MOST, ldz=MOST, lddz=MOST, ldy=MOST), -21),
])
def test_act_backward_refuses(kw, code):
    assert mg.mi_act_backward(**{**ACT, **kw}) == code


@pytest.mark.parametrize("kw,code", [
    (dict(type=4), -30), (dict(rows=-1), -32), (dict(cols=-1), -33), (dict(dh=0), -34), (dict(lddh=199), -37), (dict(act=-1), -39),
    (dict(ztype=1), -30), (dict(g=0), -34), (dict(ldg=199), -37), (dict(gscale=0), -36), (dict(ldsg=2), -38), (dict(u=0), -34),
    (dict(ldu=199), -37), (dict(uscale=0), -36), (dict(ldsu=2), -38), (dict(dg=0), -35), (dict(lddg=199), -37), (dict(du=0), -35),
    (dict(lddu=199), -37), (dict(ldh=199), -37),
    (dict(cols=2**31 - 128, lddh=MOST, ldg=MOST, ldu=MOST, lddg=MOST, lddu=MOST, ldh=MOST), -21),
])
def test_gated_backward_refuses(kw, code):
    assert mg.mi_gated_backward(**{**BACK, **kw}) == code


def test_quick_returns_touch_nothing():
    null = dict.fromkeys(("A", "B", "bias", "R", "C", "z"), 0)
    for kw in (dict(M=0), dict(N=0)):
        assert mg.mi_linear(**{**LINEAR, **null, **kw}) == 0
        assert mg.mi_linear(**{**LINEAR, **kw, "zscale": 0}) == 0
    null = dict.fromkeys(("A", "G", "U", "h", "g", "u"), 0)
    for kw in (dict(M=0), dict(N=0)):
        assert mg.mi_gated(**{**GATED, **null, **kw}) == 0
    for call, args, null in ((mg.mi_act_backward, ACT, ("dy", "z", "zscale", "dz", "y", "dbias")),
                             (mg.mi_gated_backward, BACK, ("dh", "g", "u", "gscale", "uscale", "dg", "du", "h", "dbiasG", "dbiasU"))):
        for kw in (dict(rows=0), dict(cols=0)):
            assert call(**{**args, **dict.fromkeys(null, 0), **kw}) == 0
        assert call(**{**args, "rows": 0, "beta": 1.0}) == 0      # sums that stay as they are


def test_host_tensors_are_refused():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16)
    y = torch.zeros(4, 6, dtype=torch.bfloat16)
    for call in (lambda: mg.linear("N", "T", 1.0, x, w, 0.0, y), lambda: mg.gated(x, w, w, y),
                 lambda: mg.act_backward(y, y, y), lambda: mg.gated_backward(y, y, y, y, y)):
        with pytest.raises(ValueError, match="device tensor"):
            call()


def test_binding_leaves_what_it_does_not_know():
    from fp32_gemm_nn_amd import feedforward

    native = feedforward._load_native()
    y = torch.zeros(4, 6, dtype=torch.bfloat16)
    assert native.linear() is None and native.gated(1) is None
    assert native.act_backward(*[None] * 9) is None and native.gated_backward(*[None] * 13) is None
    assert native.act_backward(y, y, y, None, "silu", None, None, 0.0, None) is None
