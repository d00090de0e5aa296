"""The norm and its gradient: which form ran, and matrices past 2^31 elements."""

import numpy as np
import pytest
import torch

import fp8_util as fu
from fp8_util import TYPES, U, f64
from gpu_util import device, lib, reset_debug
from test_gpu_fp8 import E4M3, check_grad, done, empty8, grad_case, randn

pytestmark = pytest.mark.gpu


@pytest.fixture
def ap():
    device()
    ap = lib()
    reset_debug(ap)
    yield ap
    reset_debug(ap)


def flags(ap):
    return ap.ap_debug_get(ap.AP_DBG_LAST_FLAGS)


@pytest.mark.parametrize("rows,cols,forms", [(700, 1000, (4, 0)), (333, 2048, (4, 0)), (460, 8192, (4, 0)), (700, 1001, (12, 8)),
                                             (311, 2057, (12, 8)), (5, 20000, (2, 2)), (5, 20001, (2, 2))])
@pytest.mark.parametrize("kind,res,dres", [("f32", "f32", True), ("bf16", "f32", True), ("f16", "f16", False)])
def test_norm_backward_takes_the_form_asked_for(ap, rows, cols, forms, kind, res, dres):
    """Path 1 the ring where it takes the rows, 2 the registers; rows too wide for both take the two passes."""
    dy, h, w, r, d = grad_case(rows, cols, TYPES[kind], TYPES[res], dres, seed=cols)
    ws = torch.empty(ap.ap_rms_norm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    for path, form in zip((1, 2), forms):
        ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, path)
        dx, dw = torch.full_like(h, float("nan")), torch.empty(cols, device="cuda")
        ap.ap_rms_norm_backward(dy, h, w, r, dx, dw, ws, dresidual=d)
        done(ap)
        assert flags(ap) == form
        check_grad(dx, dw, dy, h, w, r, d)


def repeated(rows, cols, kind, seed, scale=1.0):
    """A matrix whose rows repeat 16 rows but for the last three."""
    some = randn(16, cols, seed=seed, scale=scale).to(kind)
    x = torch.empty(rows, cols, dtype=kind, device="cuda")
    whole = rows // 16 * 16
    x[:whole].view(-1, 16, cols).copy_(some[None].expand(whole // 16, 16, cols))
    x[whole:] = some[: rows - whole]
    x[-3:] = randn(3, cols, seed=seed + 1, scale=scale).to(kind)
    return x


@pytest.mark.parametrize("path,form", [(1, 4), (2, 0)])
def test_norm_forms_past_2_31_elements(ap, path, form):
    rows, cols = 270001, 8192
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x, res = repeated(rows, cols, torch.bfloat16, 1), repeated(rows, cols, torch.bfloat16, 3)
    want_out = (x[-3:].float() + res[-3:].float()).bfloat16()
    w = 1 + 0.1 * randn(cols, seed=5)
    _, rr, yy = fu.norm(f64(x[-3:]), f64(res[-3:]), f64(w), 1e-6)
    y, q = torch.empty_like(x), torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    s, r = torch.empty(rows, cols // 128, device="cuda"), torch.empty(rows, device="cuda")
    ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, path)
    ap.ap_rms_norm(x, w, 1e-6, y=y, q=q, q_scales=s, residual=res, residual_out=res, rstd=r)
    done(ap)
    assert flags(ap) == form
    rel = (fu.DEPTH / 2 + 8) * U
    assert np.all(np.abs(f64(r[-3:]) - rr) <= rel * rr)
    assert np.all(np.abs(f64(y[-3:]) - yy) <= fu.rounding(yy, torch.bfloat16) * (1 + rel) + rel * np.abs(yy))
    assert torch.equal(res[-3:], want_out)
    fu.check_codes(q[-3:].view(E4M3), s[-3:], yy, 1, rel, "last rows")
    whole = (rows - 3) // 16 * 16
    for t in (y, q, s, res):
        v = t[:whole].view(-1, 16, t.shape[1])
        assert all(bool((part == v[:1]).all().item()) for part in v.split(2048))


@pytest.mark.parametrize("path,form", [(1, 4), (2, 0)])
def test_norm_backward_forms_past_2_31_elements(ap, path, form):
    rows, cols = 270001, 8192
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    dy, h = repeated(rows, cols, torch.bfloat16, 1, 1e-2), repeated(rows, cols, torch.bfloat16, 3)
    w, dx, dw = 1 + 0.1 * randn(cols, seed=5), torch.empty_like(h), torch.empty(cols, device="cuda")
    r = torch.cat([1 / torch.sqrt(part.float().square().mean(1) + 1e-6) for part in h.split(1 << 14)])
    ws = torch.empty(ap.ap_rms_norm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, path)
    ap.ap_rms_norm_backward(dy, h, w, r, dx, dw, ws)
    done(ap)
    assert flags(ap) == form
    tail = slice(rows - 3, rows)
    want, near, _, _ = fu.norm_backward(f64(dy[tail]), f64(h[tail]), f64(w), f64(r[tail]), None)
    assert np.all(np.abs(f64(dx[tail]) - want) <= fu.rounding(want, torch.bfloat16) * (1 + U) + near)
    whole = (rows - 3) // 16 * 16
    v = dx[:whole].view(-1, 16, cols)
    assert all(bool((part == v[:1]).all().item()) for part in v.split(2048))
    sums, terms = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 1 << 14):
        p = dy[i:i + (1 << 14)].double() * h[i:i + (1 << 14)].double() * r[i:i + (1 << 14)].double()[:, None]
        sums += p.sum(0)
        terms += p.abs().sum(0)
    # a CTA adds at most ceil(rows / 152) rows one after another, the partials' sum 304 more
    assert bool(((dw.double() - sums).abs() <= (rows // 152 + 320) * U * terms).all().item())


@pytest.mark.parametrize("rows,cols", [(3, 200), (2, 1000), (2, 5000), (2, 40001), (3, 4099), (700, 1024), (700, 1023)])
@pytest.mark.parametrize("size,weight", [(1e16, 1e-25), (1e-15, 1e25), (1e-17, 1e30), (1e15, 1e-30)])
def test_norm_of_large_rows_with_small_weights(ap, rows, cols, size, weight):
    """h r is of the order of 1; r times the weight is subnormal or past the largest float."""
    x, w = size * randn(rows, cols), weight * (1 + 0.1 * randn(cols, seed=1))
    _, rr, yy = fu.norm(f64(x), None, f64(w), 0.0)
    rel = (fu.DEPTH / 2 + 8) * U
    for path in (1, 2):
        ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, path)
        y, q, s = torch.empty_like(x), empty8(rows, cols), torch.empty(rows, fu.blocks(cols), device="cuda")
        ap.ap_rms_norm(x, w, 0.0, y=y, q=q, q_scales=s)
        done(ap)
        assert np.all(np.abs(f64(y) - yy) <= rel * np.abs(yy) + U * np.abs(yy))
        fu.check_codes(q, s, yy, 1, rel, "norm")


@pytest.mark.parametrize("rows,cols", [(3, 7), (3, 200), (2, 1000), (2, 5000), (2, 40001), (3, 4099), (700, 1032), (700, 1023)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_norm_of_rows_whose_squares_vanish(ap, rows, cols, kind):
    """No eps and squares below the smallest float: r is infinite and so is every y; the last block of a row, which may be
    short, is one of infinities like the others."""
    x = (1e-25 * (1 + torch.rand(rows, cols, device="cuda"))).to(TYPES[kind])
    w = torch.ones(cols, device="cuda")
    for path in (1, 2):
        ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, path)
        y, q = torch.empty_like(x), empty8(rows, cols)
        s, r = torch.zeros(rows, fu.blocks(cols), device="cuda"), torch.empty(rows, device="cuda")
        ap.ap_rms_norm(x, w, 0.0, y=y, q=q, q_scales=s, rstd=r)
        done(ap)
        assert torch.isposinf(r).all() and torch.isposinf(y).all() and torch.isposinf(s).all()
        assert torch.isnan(q.float()).all()
