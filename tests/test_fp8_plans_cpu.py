"""What the 8-bit operators plan on the host, without a GPU."""

import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ap():
    from async_global_shared_gb300 import build

    build.build()
    import async_global_shared_gb300 as ap

    ap.load()
    return ap


@pytest.mark.parametrize("sms", [1, 20, 148, 152, 160, 304, 400])
def test_norm_backward_writes_and_sums_the_same_rows(ap, sms):
    """The first kernel writes one row of the workspace a CTA and the second adds up as many: whatever the device's SM
    count, no more than the workspace holds, and, in the ring (which these calls take), one CTA an SM."""
    for rows, cols in ((20000, 256), (8192, 4096), (6062, 2694), (3000, 8192), (700, 16384)):
        for t, rt in ((ap.AP_F32, ap.AP_F32), (ap.AP_BF16, ap.AP_BF16), (ap.AP_F16, ap.AP_F32)):
            for dres in (False, True):
                ctas = ap.ap_debug_norm_grad_ctas(rows, cols, t, rt, dres, sms)
                held = ap.ap_rms_norm_backward_workspace(rows, cols) // (4 * cols)
                assert 1 <= ctas <= held
                if cols <= 8192:
                    assert ctas == min(sms, held)


def test_norm_backward_plan_of_few_rows_and_refusals(ap):
    f = ap.ap_debug_norm_grad_ctas
    assert f(0, 100, ap.AP_F32, ap.AP_F32, False, 20) == 0
    assert f(1, 100, ap.AP_F32, ap.AP_F32, False, 20) == 1
    assert f(100, 100, ap.AP_F32, ap.AP_F32, True, 20) == 100  # in registers: a row a CTA, on any device
    for bad in ((-1, 4, 0, 0, False, 20), (4, 0, 0, 0, False, 20), (4, 4, 7, 0, False, 20), (4, 4, ap.AP_F16, ap.AP_BF16, False, 20),
                (4, 4, 0, 0, False, 0), (1 << 30, 1 << 30, 0, 0, False, 20)):
        assert f(*bad) == -1


def test_norm_backward_plan_under_the_cap(ap):
    try:
        ap.ap_debug_set(ap.AP_DBG_GRID, 20)
        assert ap.ap_debug_norm_grad_ctas(8192, 4096, ap.AP_BF16, ap.AP_BF16, True, 152) == 20
    finally:
        ap.ap_debug_set(ap.AP_DBG_GRID, 0)


def test_give_up_setting(ap):
    lib = ap.load()
    assert lib.ap_debug_set(ap.AP_DBG_GIVE_UP, 17) == ap.AP_ERR_ARG and lib.ap_debug_set(ap.AP_DBG_GIVE_UP, -1) == ap.AP_ERR_ARG
    for value in (16, 0):
        ap.ap_debug_set(ap.AP_DBG_GIVE_UP, value)
        assert ap.ap_debug_get(ap.AP_DBG_GIVE_UP) == value


def test_block_scale_refusals(ap):
    f = ap.load().ap_debug_block_scale
    assert f(None, None, None, -1, None) == ap.AP_ERR_SHAPE and f(None, None, None, 0, None) == ap.AP_OK
    assert f(None, 4096, 8192, 4, None) == ap.AP_ERR_NULL
    assert f(2, 4096, 8192, 4, None) == ap.AP_ERR_ALIGN
    assert f(4096, 4100, 8192, 4, None) == ap.AP_ERR_ALIAS


def test_no_device_behind_made_up_addresses(ap, request):
    """Sessions without the GPU tests see no device, whatever the machine has."""
    import os

    import torch

    assert not torch.cuda.is_available()
    assert ap.load().ap_check(None) != ap.AP_OK
    if request.config.option.markexpr.replace(" ", "") == "notgpu":
        assert os.environ["CUDA_VISIBLE_DEVICES"] == ""
