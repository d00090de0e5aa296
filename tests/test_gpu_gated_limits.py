"""The gated block's operators at their limits: values that are not finite, and where their documentation promises more
than a size or a type."""

import numpy as np
import pytest
import torch

import gated_util as gu
from fp8_util import TYPES, U, f64
from gpu_util import device, lib, reset_debug
from test_gpu_gated_backward import Outputs, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture
def ap():
    device()
    ap = lib()
    reset_debug(ap)
    yield ap
    reset_debug(ap)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", [1, 7, 129, 290, 300, 381])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_zeros_between_the_halves_beside_a_block_that_is_not_finite(ap, kind, cols, bad):
    """q's columns between dg's last and du's first are zeros, whatever dg's last block holds."""
    rows, first = 140, -(-cols // 128) * 128
    dy, gate, up = inputs(rows, cols, TYPES[kind], cols)
    clean = Outputs(rows, cols, TYPES[kind], "codes")
    ap.ap_gated_backward(dy, gate, up, 0, **clean.named)
    spots = ((0, cols - 1), (77, max(0, cols - 5)), (139, first - 128))
    for row, col in spots:
        dy[row, col] = float(bad)
    for pad, shift in ((0, 0), (3, 1)):
        out = Outputs(rows, cols, TYPES[kind], "codes", pad, shift)
        ap.ap_gated_backward(dy, gate, up, 0, **out.named)
        assert ap.ap_check() == 0
        for row, col in spots:
            assert not torch.isfinite(out.scales[row, [col // 128, (first + col) // 128]]).any()
        assert (out.q[:, cols:first] == 0).all()
        keep = [r for r in range(rows) if r not in (0, 77, 139)]
        assert torch.equal(out.q[keep], clean.q[keep]) and torch.equal(out.scales[keep], clean.scales[keep])
        assert out.intact()


@pytest.mark.parametrize("act,lo,hi", [("silu", -130.0, -60.0), ("gelu", -14.0, -7.0)])
def test_where_the_logistic_function_becomes_zero(ap, act, lo, hi):
    """act and its slope near the least s that is a normal number: within the bound of s above it, 0 and off by no more
    than the header says below it."""
    g = torch.linspace(lo, hi, 5001, device="cuda")[None].contiguous()
    one, slope, value = torch.ones_like(g), torch.empty_like(g), torch.empty_like(g)
    ap.ap_gated_backward(one, g, one, gu.ACTS[act], dgate=slope, dup=value)
    assert ap.ap_check() == 0
    x = f64(g)
    w = gu.argument(act, x)
    s = np.exp(w) / (1 + np.exp(w))
    dw = 1.0 if act == "silu" else 2 * gu.ROOT * (1 + 3 * 0.044715 * x ** 2)
    normal = s >= 2.0 ** -126 * 1.001  # U's of s on either side of the border
    gone = s < 2.0 ** -126 * 0.999
    assert normal.any() and gone.any()
    v, d = gu.value(act, x), gu.slope(act, x)
    off, off_slope = np.abs(f64(value) - v), np.abs(f64(slope) - d)
    assert np.all(off[normal] <= (np.abs(v) * (10 + 3 * np.abs(w)) * U)[normal])
    assert np.all(off <= np.maximum(np.abs(v) * (10 + 3 * np.abs(w)) * U, np.abs(x) * 2.0 ** -126))
    near = ((8 + 3 * np.abs(w)) * s + (39 + 9 * np.abs(w)) * np.abs(d - s) + 3 * np.abs(d)) * U
    assert np.all(off_slope[normal] <= near[normal])
    assert np.all(off_slope <= np.maximum(near, (1 + np.abs(x) * dw) * 2.0 ** -126))
    assert (f64(value)[gone] == 0).all() and (f64(slope)[gone] == 0).all()
