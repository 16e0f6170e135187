"""The probabilities' exponent has one rounding: temperatures whose log2(e) / T
lies between two fp32 numbers, and logits far below the largest."""
import math

import pytest
import torch

from iq4_xs_quantized_gb300 import binding as B

pytestmark = pytest.mark.gpu

U = 2.0**-24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from iq4_xs_quantized_gb300 import build
    build.build()
    B.load()
    B.iq4xs_last_device_error()
    yield
    assert B.iq4xs_last_device_error() == 0


@pytest.mark.parametrize("rows,vocab", ((1, 1000), (50, 131073), (3, 20001)))
@pytest.mark.parametrize("t", (0.3479994, 1.3929858, 1.4119856, 2.8779667, 1.0))
def test_probs_of_small_weights(rows, vocab, t):
    """Logits are multiples of 2^-6 below 0, which every thousandth is: the
    differences are exact.  Then z = d log2(e) / T is rounded once (half a step of
    z, times ln 2, of the weight), the power is off by two units (4 2^-24), the
    sum by one rounding an addition (50 of them one behind another at most: a
    thread's, a warp's, the warps', the CTAs'), the quotient and the product by one each.
    And the sum is made of weights that are off themselves: by 4 2^-24, and by half a
    step of z below 8, ln 2 2^-22, for those behind have below e^-5.5 of it (above: 3 more)."""
    t = float(torch.tensor(t, dtype=torch.float32))
    g = torch.Generator(device="cuda").manual_seed(vocab)
    most = int(84 * t * 64)
    x = -torch.randint(0, most, (rows, vocab), generator=g, device="cuda").float() / 64
    x[:, ::1000] = 0.0
    out = torch.empty_like(x)
    B.iq4xs_token_probs(x, out, temperature=torch.full((rows,), t, device="cuda"))
    want = torch.softmax(x.double() / t, -1)
    z = (x.double() / t * math.log2(math.e)).abs().clamp(min=2.0**-20)
    half_step = torch.exp2(torch.floor(torch.log2(z)) - 24)
    tol = want * (math.log(2) * half_step + (4 + 50 + 2 + 4 + 3) * U)
    off = ((out.double() - want).abs() / tol).max().item()
    assert off <= 1, off
