"""The largest sizes that the 8-bit layer's entry points take, as their header states them: one more is refused,
before any HIP call."""
import os
import re

import pytest

from fp32_gemm_nn_amd import fp8
from test_fp8_abi import GEMM, QUANT

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "misgemm_fp8.h")
TOO_LARGE, MOST = -21, 2**31 - 1


def comment(entry):
    """The comment above an entry point, its words one space apart."""
    text = open(HEADER).read()
    text = text[:text.index(f"int {entry}(")]
    return re.sub(r"\s+", " ", re.sub(r"\n \* ?", " ", text[text.rindex("/*"):]))


@pytest.mark.parametrize("kw", [dict(rows=65535 * 128 + 1, ldqt=MOST), dict(cols=2**31 - 127, ldx=MOST, ldq=MOST)])
def test_quantize(kw):
    for block in (0, 1):
        assert fp8.mi_fp8_quantize(**{**QUANT, "block": block, "lds": MOST, "lds_t": MOST, **kw}) == TOO_LARGE
    said = comment("mi_fp8_quantize")
    assert "65,535 * 128 rows" in said and "2^31 - 128 columns: MISGEMM_TOO_LARGE" in said


@pytest.mark.parametrize("kw", [dict(M=2**31 - 256, ldsa=MOST, ldsb=MOST), dict(N=2**31 - 256, ldc=MOST, ldsb=MOST),
                                dict(K=2**31 - 256, lda=MOST, ldb=MOST, ldsb=MOST),
                                dict(M=128 * 2**12, N=128 * 2**11, ldsa=MOST, ldsb=MOST, ldc=MOST)])
def test_gemm(kw):
    for block in (0, 1):
        assert fp8.mi_fp8_gemm(**{**GEMM, "block": block, **kw}) == TOO_LARGE
    said = comment("mi_fp8_gemm")
    assert "From 2^23 blocks of 128 x 128 outputs on" in said and "2^31 - 257: MISGEMM_TOO_LARGE" in said
