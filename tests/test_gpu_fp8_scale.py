"""A block's scale and its reciprocal against the correctly rounded quotient and reciprocal."""

import pytest
import torch

from gpu_util import device, lib
from test_gpu_fp8 import done

pytestmark = pytest.mark.gpu

MIN_SCALE = 2.0 ** -126


# amax's exponents: ordinary, the smallest whose scales are all normal and the next, across the floor of the scale,
# subnormal, the largest
@pytest.mark.parametrize("exponent", [127, 128, 9, 10, 8, 1, 0, 254])
def test_scale_and_reciprocal_of_every_mantissa(exponent):
    """In 64 bits a quotient's second rounding is harmless: 53 >= 2 * 24 + 2 bits."""
    device()
    ap = lib()
    n = 1 << 23
    amax = (torch.arange(n, dtype=torch.int32, device="cuda") + (exponent << 23)).view(torch.float32)
    scale, inv = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    ap.ap_debug_block_scale(amax, scale, inv, n)
    done(ap)
    want = (amax.double() / 448).float()
    want = torch.where(want < MIN_SCALE, torch.full_like(want, MIN_SCALE), want)
    assert torch.equal(scale, want)
    assert torch.equal(inv, (1 / want.double()).float())


def test_scale_of_no_number():
    device()
    ap = lib()
    amax = torch.tensor([0.0, float("inf"), float("nan"), 448.0], device="cuda")
    scale, inv = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    ap.ap_debug_block_scale(amax, scale, inv, 4)
    done(ap)
    assert scale[0] == MIN_SCALE and inv[0] == 2.0 ** 126
    assert torch.isposinf(scale[1]) and inv[1] == 0
    assert torch.isnan(scale[2]) and torch.isnan(inv[2])
    assert scale[3] == 1 and inv[3] == 1
