"""The example layer, small and odd-sized: a training step and a token, against the same in FP32."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens,inner,outer", [(64, 256, 128), (300, 520, 700)])
def test_layer(tokens, inner, outer):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_layer

    off = fp8_layer.main(["--tokens", str(tokens), "--inner", str(inner), "--outer", str(outer), "--steps", "2"])
    # Roundings to nearest, at most 2^-4 of a value in E4M3 and 2^-3 in E5M2, and 2^-8 in BF16 for a result: a sum of
    # products of two such operands is off by at most the sum of these for each product, and as far as their signs
    # are independent of the values by that of its size (both operands' sums are of values of either sign).
    assert off["y"] <= 2 * 2**-4 + 2**-8
    assert off["dweight"] <= 2**-4 + 2**-3
    assert off["dx"] <= 2**-4 + 2**-3 + 2**-7 and off["dnorm"] <= 2**-4 + 2**-3 + 2**-7
    # The same 8-bit operands, summed in another order and rounded to BF16.
    assert off["token"] <= 2**-7
