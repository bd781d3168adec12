"""The example block, small and odd-sized: a training step and a token, against the same in FP32."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens,width,inner,act", [(64, 256, 128, "silu"), (300, 520, 700, "gelu_tanh"), (33, 100, 60, "gelu")])
def test_block(tokens, width, inner, act):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import feed_forward

    off = feed_forward.main(["--tokens", str(tokens), "--width", str(width), "--inner", str(inner), "--steps", "2", "--act", act])
    # Roundings to nearest, 2^-8 of a value for each BF16 matrix on the way (n, h, y; dh, dg or du, dn, dx, and n and h
    # again), 2^-4 for each projection in E4M3, on which the gradients depend at most threefold (dg on u once, on g through
    # f'). Sums of products whose factors are off by independent roundings are off by no more than that of their size.
    eight = 3 * 2**-4
    assert off["y"] <= 3 * 2**-8
    assert max(off[k] for k in ("dwg", "dwu", "dwd")) <= 6 * 2**-8 + eight
    assert max(off["dx"], off["dnorm"]) <= 9 * 2**-8 + eight
    # The same values, summed in another order and rounded to BF16 at n, h and y.
    assert off["token"] <= 3 * 2**-8
