"""The gated block's operators at their limits: values that are not finite, and where their documentation promises more
than a size or a type."""

import pytest
import torch

from fp8_util import TYPES
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
