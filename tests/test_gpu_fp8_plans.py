"""The 8-bit operators under plans that the device at hand does not ask for by itself."""

import pytest
import torch

from gpu_util import device, lib, reset_debug
from test_gpu_fp8 import check_grad, done, grad_case, randn

pytestmark = pytest.mark.gpu


@pytest.fixture
def ap():
    device()
    ap = lib()
    reset_debug(ap)
    yield ap
    reset_debug(ap)


@pytest.mark.parametrize("ctas", [1, 20, 148])
@pytest.mark.parametrize("rows,cols", [(3000, 264), (2000, 1001), (1000, 8192)])
def test_norm_backward_on_fewer_ctas(ap, ctas, rows, cols):
    """dweight sums the rows of partials that this call's CTAs wrote, however many they are."""
    dy, h, w, r, d = grad_case(rows, cols, torch.bfloat16, torch.float32, True)
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.full((ap.ap_rms_norm_backward_workspace(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
    ap.ap_debug_set(ap.AP_DBG_GRID, ctas)
    ap.ap_rms_norm_backward(dy, h, w, r, dx, dw, ws, dresidual=d)
    done(ap)
    assert ap.ap_debug_get(ap.AP_DBG_LAST_GRID) == ctas and ap.ap_debug_get(ap.AP_DBG_LAST_FLAGS) & 4
    check_grad(dx, dw, dy, h, w, r, d)


@pytest.mark.parametrize("ctas", [1, 20])
def test_norm_on_fewer_ctas(ap, ctas):
    x, w = randn(3000, 4096).bfloat16(), randn(4096, seed=1)
    res = randn(3000, 4096, seed=2)
    got = []
    for cap in (0, ctas):
        y, out = torch.empty_like(x), torch.empty_like(res)
        ap.ap_debug_set(ap.AP_DBG_GRID, cap)
        ap.ap_rms_norm(x, w, 1e-6, y=y, residual=res, residual_out=out)
        done(ap)
        got.append((y, out, ap.ap_debug_get(ap.AP_DBG_LAST_GRID)))
    assert got[1][2] == ctas < got[0][2]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
