"""Waits of the 8-bit operators that run out: the call ends, the error is reported once, and the next call works."""

import pytest
import torch

from gpu_util import device, lib, reset_debug
from test_gpu_fp8 import done, grad_case, randn

pytestmark = pytest.mark.gpu

SITE_ROWS_CONSUMER = 21


@pytest.fixture
def ap():
    device()
    ap = lib()
    reset_debug(ap)
    yield ap
    reset_debug(ap)


# teams of one warp and of several, in the ring's forms for rows on and off the 16-byte boundaries
ROWS = [(2000, 512), (1300, 2048), (1300, 2047), (900, 5000), (700, 8192), (700, 8191)]


def ring_calls(ap, rows, cols):
    """The norm and its gradient through the ring, each with a tensor that shows what it wrote."""
    ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, 1)
    dy, h, w, r, d = grad_case(rows, cols, torch.bfloat16, torch.bfloat16, True)
    y, out = torch.empty_like(dy), torch.empty_like(h)
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.empty(ap.ap_rms_norm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    return [(lambda: ap.ap_rms_norm(dy, w, 1e-6, y=y, residual=h, residual_out=out), (y, out)),
            (lambda: ap.ap_rms_norm_backward(dy, h, w, r, dx, dw, ws, dresidual=d), (dx, dw))]


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("fault", ["nothing arrives", 1, 2, 16])
def test_ring_of_rows_gives_up(ap, rows, cols, fault):
    """No stage ever fills; or one warp of a CTA (the first, the second, the last) gives up alone, its team mates not:
    they must not wait for it at the barriers of their rows' sums."""
    for call, outputs in ring_calls(ap, rows, cols):
        call()
        done(ap)
        assert ap.ap_debug_get(ap.AP_DBG_LAST_FLAGS) & 4
        want = [t.clone() for t in outputs]
        ap.ap_debug_set(ap.AP_DBG_TIMEOUT_NS, 2_000_000)
        if fault == "nothing arrives":
            ap.ap_debug_set(ap.AP_DBG_EXPECT_TX_EXTRA, 16)
        else:
            ap.ap_debug_set(ap.AP_DBG_GIVE_UP, fault)
        call()
        status = ap.ap_check()
        if fault == 16 and status == ap.AP_OK:
            pass  # a warp of no team
        else:
            assert status == ap.AP_ERR_DEVICE_TIMEOUT
        if fault in (1, 2):
            assert ap.ap_debug_get(ap.AP_DBG_LAST_SITE) == SITE_ROWS_CONSUMER
        assert ap.ap_check() == ap.AP_OK
        reset_debug(ap)
        ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, 1)
        call()
        done(ap)
        assert all(torch.equal(a, b) for a, b in zip(outputs, want))


def test_rows_of_a_warp_that_gave_up_are_not_passed_off_as_results(ap):
    """What a team makes of a row without one of its warps' part is NaN."""
    rows, cols = 1300, 2048
    x, w, y = randn(rows, cols), torch.ones(cols, device="cuda"), torch.zeros(rows, cols, device="cuda")
    ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, 1)
    ap.ap_debug_set(ap.AP_DBG_GIVE_UP, 1)
    ap.ap_rms_norm(x, w, 1e-6, y=y)
    assert ap.ap_check() == ap.AP_ERR_DEVICE_TIMEOUT
    reset_debug(ap)
    want = torch.empty_like(y)
    ap.ap_rms_norm(x, w, 1e-6, y=want)
    done(ap)
    right = torch.isclose(y, want, rtol=1e-5, atol=0)
    assert (right | torch.isnan(y) | (y == 0)).all()
