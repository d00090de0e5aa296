"""The 8-bit block-scaled operators on a GPU against plain forms in 64 bits:
types, sizes from one element up, odd widths, strides and offsets, blocks with
zeros, infinities and NaN, in-place calls, streams and graphs."""

import numpy as np
import pytest
import torch

import fp8_util as fu
from fp8_util import TYPES, Strided, U, f64
from gpu_util import device, lib, reset_debug

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture
def ap():
    device()
    ap = lib()
    reset_debug(ap)
    yield ap
    reset_debug(ap)


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(1000 + seed)
    return (torch.randn(*shape, generator=g) * scale).cuda()


def empty8(rows, cols, ld=None):
    ld = -(-cols // 16) * 16 if ld is None else ld
    return torch.zeros(rows, ld, dtype=torch.uint8, device="cuda").view(E4M3)[:, :cols]


def done(ap):
    assert ap.ap_check() == ap.AP_OK


# ------------------------------------------------------------------ norm

NORM_SIZES = [(1, 1), (1, 128), (3, 7), (9, 129), (5, 250), (17, 512), (8, 1000), (2, 1025), (3, 4096), (2, 5000), (2, 8192),
              (1, 8200), (2, 16384), (1, 32768), (2, 40001)]


@pytest.mark.parametrize("rows,cols", NORM_SIZES)
@pytest.mark.parametrize("kind,res", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"),
                                      ("bf16", None)])
def test_norm(ap, rows, cols, kind, res):
    t = TYPES[kind]
    x = randn(rows, cols, seed=cols).to(t)
    residual = None if res is None else (2 * randn(rows, cols, seed=cols + 1)).to(TYPES[res])
    weight = (1 + 0.1 * randn(cols, seed=2)).to(t if (rows + cols) % 2 else torch.float32)
    out = None if res is None else torch.empty_like(residual)
    y, q = torch.empty_like(x), empty8(rows, cols)
    s = torch.empty(rows, fu.blocks(cols), device="cuda")
    r = torch.empty(rows, device="cuda")
    ap.ap_rms_norm(x, weight, 1e-5, y=y, q=q, q_scales=s, residual=residual, residual_out=out, rstd=r)
    done(ap)
    assert ap.ap_debug_get(ap.AP_DBG_LAST_PATH) == 7
    h, rr, yy = fu.norm(f64(x), None if res is None else f64(residual), f64(weight), 1e-5)
    # the sum's error halves under the root; four more roundings
    rel = (fu.DEPTH / 2 + 4) * U
    assert np.all(np.abs(f64(r) - rr) <= rel * rr)
    rel += 4 * U
    assert np.all(np.abs(f64(y) - yy) <= fu.rounding(yy, t) * (1 + rel) + rel * np.abs(yy))
    # h carries one 32-bit rounding, which a sum near zero makes relatively large: absolute, by its terms
    if res is not None:
        assert np.all(np.abs(f64(out) - h) <= fu.rounding(h, out.dtype) * (1 + U) + U * np.abs(h))
    fu.check_codes(q, s, yy, 1, rel, f"norm {rows}x{cols}")


def test_norm_q_only_and_y_only_agree(ap):
    x, w = randn(33, 1536).bfloat16(), randn(1536, seed=1)
    y1, y2, q1, q2 = torch.empty_like(x), torch.empty_like(x), empty8(33, 1536), empty8(33, 1536)
    s1, s2 = torch.empty(33, 12, device="cuda"), torch.empty(33, 12, device="cuda")
    ap.ap_rms_norm(x, w, 1e-6, y=y1, q=q1, q_scales=s1)
    ap.ap_rms_norm(x, w, 1e-6, y=y2)
    ap.ap_rms_norm(x, w, 1e-6, q=q2, q_scales=s2)
    done(ap)
    assert torch.equal(y1, y2) and torch.equal(q1.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s1, s2)


@pytest.mark.parametrize("cols", [64, 257, 1000, 4100, 9001, 33000])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 3), (4, 5)])
def test_norm_strided_rows_stay_inside(ap, cols, shift, pad):
    rows, t = 5, torch.float16
    x = Strided(rows, cols, t, cols + pad, shift, randn(rows, cols).to(t))
    res = Strided(rows, cols, torch.float32, cols + pad + 1, shift, randn(rows, cols, seed=1))
    y = Strided(rows, cols, t, cols + pad + 2, shift)
    q = Strided(rows, cols, torch.uint8, cols + pad + 3, shift)
    s, r, w = torch.empty(rows, fu.blocks(cols), device="cuda"), torch.empty(rows, device="cuda"), randn(cols + 1)[1:]
    h, rr, yy = fu.norm(f64(x.view), f64(res.view), f64(w), 0.0)
    ap.ap_rms_norm(x.view, w, 0.0, y=y.view, q=q.view, q_scales=s, residual=res.view, residual_out=res.view, rstd=r)
    done(ap)
    assert all(b.intact() for b in (x, res, y, q))
    rel = (fu.DEPTH / 2 + 8) * U
    assert np.all(np.abs(f64(y.view) - yy) <= fu.rounding(yy, t) * (1 + rel) + rel * np.abs(yy))
    assert np.all(np.abs(f64(res.view) - h) <= fu.rounding(h, torch.float32) + U * np.abs(h))
    # cloned: a strided view of float8 is not indexed by every torch release
    fu.check_codes(q.view.clone().view(E4M3), s, yy, 1, rel, "strided norm")


@pytest.mark.parametrize("cols", [200, 2048, 40000])
def test_norm_in_place(ap, cols):
    x, res, w = randn(7, cols).bfloat16(), randn(7, cols, seed=1).bfloat16(), randn(cols, seed=2)
    y, out = torch.empty_like(x), torch.empty_like(res)
    ap.ap_rms_norm(x, w, 1e-6, y=y, residual=res, residual_out=out)
    ap.ap_rms_norm(x, w, 1e-6, y=x, residual=res, residual_out=res)
    done(ap)
    assert torch.equal(x, y) and torch.equal(res, out)


def test_norm_between_column_slices_of_one_matrix(ap):
    wide = torch.cat([randn(5, 256), torch.full((5, 256), 7.0, device="cuda")], 1).bfloat16()
    w, want = randn(256, seed=1), torch.empty(5, 256, dtype=torch.bfloat16, device="cuda")
    ap.ap_rms_norm(wide[:, :256], w, 1e-6, y=want)
    ap.ap_rms_norm(wide[:, :256], w, 1e-6, y=wide[:, 256:])
    done(ap)
    assert torch.equal(wide[:, 256:], want)
    ap.ap_rms_norm(wide[:, 256:], w, 1e-6, y=wide[:, :256])
    done(ap)
    with pytest.raises(ap.APError) as e:
        ap.ap_rms_norm(wide[:, :256], w, 1e-6, y=wide[:, 255:511])
    assert e.value.status == ap.AP_ERR_ALIAS


@pytest.mark.parametrize("cols", [300, 2048, 40000])
def test_norm_zeros_infinities_nan(ap, cols):
    x = randn(6, cols)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 200] = float("nan")
    x[4] *= 1e-20  # squares vanish: eps rules
    x[5, : min(cols, 128)] = 0
    w = torch.ones(cols, device="cuda")
    y, q, s, r = torch.empty_like(x), empty8(6, cols), torch.empty(6, fu.blocks(cols), device="cuda"), torch.empty(6, device="cuda")
    ap.ap_rms_norm(x, w, 1e-6, y=y, q=q, q_scales=s, rstd=r)
    done(ap)
    y, q, s, r = y.cpu(), q.float().cpu(), s.cpu(), r.cpu()
    assert (y[1] == 0).all() and (q[1] == 0).all() and (s[1] == fu.MIN_SCALE).all()
    assert r[2] == 0 and torch.isnan(y[2, 5]) and (y[2, :5] == 0).all()  # inf * 0 and x * 0, as the formula has them
    assert torch.isnan(q[2, :128]).all() and torch.isnan(s[2, 0]) and (s[2, 1:] == fu.MIN_SCALE).all()
    assert torch.isnan(y[3]).all() and torch.isnan(q[3]).all() and torch.isnan(r[3])
    assert torch.isfinite(y[4]).all() and torch.isfinite(s[4]).all()
    assert (q[5, : min(cols, 128)] == 0).all() and s[5, 0] == fu.MIN_SCALE


def test_norm_past_2_31_elements(ap):
    rows, cols = 65600, 32768 + 128
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.arange(cols, device="cuda") % 7 - 3)
    x[-1] *= 2
    q, s, r = torch.empty(rows, cols, dtype=torch.uint8, device="cuda"), torch.empty(rows, cols // 128, device="cuda"), torch.empty(rows, device="cuda")
    w = torch.ones(cols, device="cuda")
    ap.ap_rms_norm(x, w, 0.0, q=q, q_scales=s, rstd=r)
    done(ap)
    _, rr, yy = fu.norm(f64(x[-2:]), None, f64(w), 0.0)
    assert np.all(np.abs(f64(r[-2:]) - rr) <= (fu.DEPTH / 2 + 4) * U * rr)
    fu.check_codes(q[-2:].view(E4M3), s[-2:], yy, 1, (fu.DEPTH / 2 + 8) * U, "norm past 2^31")
    assert bool((q[:-1] == q[0]).all().item()) and bool((s[:-1] == s[0]).all().item())


# ------------------------------------------------------------------ norm gradient

GRAD_SIZES = [(1, 1), (1, 128), (3, 7), (700, 129), (1300, 264), (50, 1000), (333, 2048), (9, 4100), (40, 8192), (5, 16384),
              (4, 20001)]


def grad_case(rows, cols, t, rt, dres, seed=0):
    dy = (1e-2 * randn(rows, cols, seed=seed)).to(t)
    h = randn(rows, cols, seed=seed + 1).to(rt)
    w = 1 + 0.1 * randn(cols, seed=seed + 2)
    r = (1 / torch.sqrt(h.float().square().mean(1) + 1e-6))
    d = (1e-2 * randn(rows, cols, seed=seed + 3)).to(rt) if dres else None
    return dy, h, w, r, d


def check_grad(dx, dw, dy, h, w, r, d):
    rows = dy.shape[0]
    want, near, wdw, terms = fu.norm_backward(f64(dy), f64(h), f64(w), f64(r), None if d is None else f64(d))
    assert np.all(np.abs(f64(dx) - want) <= fu.rounding(want, dx.dtype) * (1 + U) + near)
    # each product carries two roundings; a column's rows are added at worst one after another
    assert np.all(np.abs(f64(dw) - wdw) <= (rows + 16) * U * terms)


@pytest.mark.parametrize("rows,cols", GRAD_SIZES)
@pytest.mark.parametrize("kind,res,dres", [("f32", "f32", True), ("bf16", "bf16", True), ("bf16", "f32", False),
                                           ("f16", "f32", True), ("f16", "f16", False)])
def test_norm_backward(ap, rows, cols, kind, res, dres):
    t, rt = TYPES[kind], TYPES[res]
    dy, h, w, r, d = grad_case(rows, cols, t, rt, dres, seed=rows)
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.empty(ap.ap_rms_norm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    ap.ap_rms_norm_backward(dy, h, w, r, dx, dw, ws, dresidual=d)
    done(ap)
    assert ap.ap_debug_get(ap.AP_DBG_LAST_PATH) == 8
    check_grad(dx, dw, dy, h, w, r, d)
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    ws.fill_(0xFF)  # its contents do not matter
    ap.ap_rms_norm_backward(dy, h, w, r, dx2, dw2, ws, dresidual=d)
    dx3 = torch.empty_like(dx)
    ap.ap_rms_norm_backward(dy, h, w, r, dx3, dresidual=d)
    done(ap)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(dx, dx3)


@pytest.mark.parametrize("cols", [130, 1001, 5000, 17000])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 3)])
def test_norm_backward_strided_in_place(ap, cols, shift, pad):
    rows = 300 if cols < 2000 else 6
    dy, h, w, r, d = grad_case(rows, cols, torch.bfloat16, torch.bfloat16, True)
    w = torch.cat([w[:1], w])[1:]  # a weight off the 16-byte boundary
    bufs = [Strided(rows, cols, torch.bfloat16, cols + pad + i, shift, v) for i, v in enumerate((dy, h, d))]
    dw = torch.empty(cols + 1, device="cuda")[1:]
    ws = torch.empty(ap.ap_rms_norm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    ap.ap_rms_norm_backward(bufs[0].view, bufs[1].view, w, r, bufs[2].view, dw, ws, dresidual=bufs[2].view)
    done(ap)
    assert all(b.intact() for b in bufs)
    check_grad(bufs[2].view, dw, dy, h, w, r, d)


def test_norm_backward_no_rows(ap):
    e, dw = torch.empty(0, 70, device="cuda"), torch.full((70,), 7.0, device="cuda")
    ap.ap_rms_norm_backward(e, e, torch.ones(70, device="cuda"), torch.empty(0, device="cuda"), e, dw,
                            torch.empty(0, dtype=torch.uint8, device="cuda"))
    done(ap)
    assert (dw == 0).all()


def test_norm_backward_against_differences(ap):
    """dx and dweight against central differences of the definition in 64 bits along random directions."""
    rows, cols, eps = 4, 384, 1e-4
    h, w, dy = randn(rows, cols), 1 + 0.1 * randn(cols, seed=1), randn(rows, cols, seed=2)
    y, r = torch.empty_like(h), torch.empty(rows, device="cuda")
    ap.ap_rms_norm(h, w, eps, y=y, rstd=r)
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.empty(ap.ap_rms_norm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    ap.ap_rms_norm_backward(dy, h, w, r, dx, dw, ws)
    done(ap)
    H, W, D = f64(h), f64(w), f64(dy)
    rng = np.random.default_rng(0)
    step = 1e-5
    for _ in range(8):
        u, v = rng.standard_normal(H.shape), rng.standard_normal(W.shape)
        f = lambda a, b: float((D * fu.norm(a, None, b, eps)[2]).sum())  # noqa: E731
        along_h = (f(H + step * u, W) - f(H - step * u, W)) / (2 * step)
        along_w = (f(H, W + step * v) - f(H, W - step * v)) / (2 * step)
        # a difference is off by step^2 times a third derivative, the gradient by DEPTH U of its terms
        for got, g, along in ((along_h, f64(dx), u), (along_w, f64(dw), v)):
            assert abs(got - (g * along).sum()) <= 1e-7 + fu.DEPTH * U * np.abs(g * along).sum() * 4


# ------------------------------------------------------------------ quantiser

QUANT_SIZES = [(1, 1), (1, 128), (3, 127), (16, 130), (128, 128), (129, 257), (200, 1000), (5, 4099), (1030, 140)]


def quant_buffers(rows, cols, tile, q=True, qt=True):
    f = dict(device="cuda", dtype=torch.float32)
    st = [None] * 4
    if q:
        st[0], st[1] = empty8(rows, cols), torch.empty(-(-rows // tile), fu.blocks(cols), **f)
    if qt:
        st[2], st[3] = empty8(cols, rows), torch.empty(-(-cols // tile), fu.blocks(rows), **f)
    return st


@pytest.mark.parametrize("rows,cols", QUANT_SIZES)
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_quantize(ap, rows, cols, tile, kind):
    x = (randn(rows, cols, seed=cols) * torch.exp(2 * randn(cols, seed=1))).to(TYPES[kind])
    both = quant_buffers(rows, cols, tile)
    one, other = quant_buffers(rows, cols, tile, qt=False), quant_buffers(rows, cols, tile, q=False)
    ap.ap_quantize(x, tile, *both)
    ap.ap_quantize(x, tile, *one)
    ap.ap_quantize(x, tile, *other)
    done(ap)
    assert ap.ap_debug_get(ap.AP_DBG_LAST_PATH) == 9
    v = x.float().cpu()
    for (q, s), m, alone in ((both[:2], v, one[:2]), (both[2:], v.t().contiguous(), other[2:])):
        fu.check_codes(q, s, m.double().numpy(), tile, 0.0, f"quantize {rows}x{cols}")
        # and bit for bit by the definition's own 32-bit steps
        wq, ws = fu.codes_32(m, tile)
        assert torch.equal(s.cpu(), ws) and torch.equal(q.cpu().view(torch.uint8), wq.view(torch.uint8))
        assert torch.equal(alone[1], s) and torch.equal(alone[0].float(), q.float())


@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("shift,pad", [(0, 16), (1, 3), (8, 8)])
def test_quantize_strided(ap, tile, shift, pad):
    rows, cols = 150, 300
    x = Strided(rows, cols, torch.bfloat16, cols + pad, shift, randn(rows, cols).bfloat16())
    q = Strided(rows, cols, torch.uint8, cols + pad, shift)
    qt = Strided(cols, rows, torch.uint8, rows + pad, shift)
    _, s, _, st = quant_buffers(rows, cols, tile)
    ap.ap_quantize(x.view, tile, q.view, s, qt.view, st)
    done(ap)
    assert x.intact() and q.intact() and qt.intact()
    v = x.view.float().cpu()
    for got, scales, m in ((q, s, v), (qt, st, v.t().contiguous())):
        wq, ws = fu.codes_32(m, tile)
        assert torch.equal(scales.cpu(), ws) and torch.equal(got.view.cpu(), wq.view(torch.uint8))


@pytest.mark.parametrize("shift", range(8))
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out", ["rows", "cols"])
def test_quantize_rows_at_every_place_of_a_unit(ap, shift, kind, out):
    rows, cols = 40, 411
    x = Strided(rows, cols, TYPES[kind], cols + 2 * (shift % 2), shift, randn(rows, cols, seed=shift).to(TYPES[kind]))
    q, s, qt, st = quant_buffers(rows, cols, 1)
    v = x.view.float().cpu()
    if out == "rows":
        ap.ap_quantize(x.view, 1, q, s)
    else:
        ap.ap_quantize(x.view, 1, None, None, qt, st)
        q, s, v = qt, st, v.t().contiguous()
    done(ap)
    wq, ws = fu.codes_32(v, 1)
    assert torch.equal(s.cpu(), ws) and torch.equal(q.cpu().view(torch.uint8), wq.view(torch.uint8))


@pytest.mark.parametrize("tile", [1, 128])
def test_quantize_extremes(ap, tile):
    """Zeros, subnormals, the largest floats, infinities and NaN, each in a block of its own."""
    rows, cols = 256, 1024
    x = randn(rows, cols).cpu()
    x[:128, :128] = 0
    x[:128, 128:256] *= 1e-44
    x[:128, 256:384] *= 1e37
    x[:128, 384:512] = torch.finfo(torch.float32).max
    x[5, 512 + 9] = float("inf")
    x[7, 640 + 3] = float("-inf")
    x[9, 768] = float("nan")
    x[128:, 900:] = -0.0
    both = quant_buffers(rows, cols, tile)
    ap.ap_quantize(x.cuda(), tile, *both)
    done(ap)
    for (q, s), m in ((both[:2], x), (both[2:], x.t().contiguous())):
        fu.check_codes(q, s, m.double().numpy(), tile, 0.0, "extremes")


def test_quantize_past_2_32_elements(ap):
    rows, cols = 33000, 131072 + 64
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.arange(cols, device="cuda") % 251 - 125)
    x[-100:] *= 3
    q, s = torch.empty(rows, cols, dtype=torch.uint8, device="cuda"), torch.empty(rows, fu.blocks(cols), device="cuda")
    qt = torch.empty(cols, -(-rows // 16) * 16, dtype=torch.uint8, device="cuda")[:, :rows]
    st = torch.empty(cols, fu.blocks(rows), device="cuda")
    ap.ap_quantize(x, 1, q, s, qt, st)
    done(ap)
    fu.check_codes(q[-3:].view(E4M3), s[-3:], f64(x[-3:]), 1, 0.0, "rows past 2^32")
    fu.check_codes(qt[-3:].clone().view(E4M3), st[-3:], f64(x[:, -3:].t()), 1, 0.0, "columns past 2^32")
    assert bool((q[1000:-100] == q[0]).all().item())


# ------------------------------------------------------------------ matrix product

MM_SIZES = [(1, 1, 1), (1, 128, 128), (1, 1000, 4096), (2, 257, 130), (7, 129, 1000), (16, 640, 2048), (17, 4100, 300),
            (33, 136, 5000), (64, 2000, 640), (65, 300, 777), (100, 1030, 1280), (128, 256, 128), (129, 257, 129),
            (200, 520, 2100), (333, 1000, 384), (512, 768, 4096), (1000, 2050, 520)]


# many blocks of k a CTA in every form: the rings and the scales' slots go round several times
LONG_SIZES = [(1, 8192, 8192), (12, 20000, 1900), (30, 20000, 1900), (24, 8192, 8192), (48, 8192, 4096), (64, 8192, 8192),
              (100, 9000, 2600), (600, 5000, 4000)]


def operand(rows, cols, tile, seed):
    """Random codes (every finite e4m3 value) and scales."""
    g = torch.Generator().manual_seed(seed)
    code = torch.randint(0, 256, (rows, cols), generator=g, dtype=torch.uint8)
    code[(code & 0x7F) == 0x7F] = 0
    q = empty8(rows, cols)
    q.view(torch.uint8).copy_(code.cuda())
    s = torch.exp(torch.randn(-(-rows // tile), fu.blocks(cols), generator=g)).cuda()
    return q, s


def check_matmul(ap, m, n, k, tile, t, c=None, seed=0):
    a, sa = operand(m, k, 1, seed + 1)
    b, sb = operand(n, k, tile, seed + 2)
    c = torch.full((m, n), float("nan"), dtype=t, device="cuda") if c is None else c
    ap.ap_matmul_fp8(a, sa, b, sb, c, tile)
    done(ap)
    want, terms = fu.matmul(f64(a), f64(sa), f64(b), f64(sb), tile)
    if t == torch.float16:
        over = np.abs(want) > 60000  # past float16's largest value
        want[over], terms[over] = 0, 0
        c = c.clone()
        c[torch.from_numpy(over).cuda()] = 0
    err, near = np.abs(f64(c) - want), fu.matmul_bound(want, terms, k, t)
    assert np.all(err <= near), f"{m}x{n}x{k}: worst {np.nanmax(err / near)} of the bound"


@pytest.mark.parametrize("m,n,k", LONG_SIZES)
@pytest.mark.parametrize("tile", [1, 128])
def test_matmul_long_runs(ap, m, n, k, tile):
    for seed in range(2):
        check_matmul(ap, m, n, k, tile, torch.bfloat16, seed=seed)


def test_matmul_calls_one_behind_another(ap):
    """Calls that start early behind the ones before, through every form: each gives what it gives alone."""
    cases, alone = [], []
    for m, n, k in ((1, 4096, 4096), (16, 8192, 2048), (32, 8192, 4096), (64, 4096, 4096), (333, 2000, 2000), (2048, 2048, 2048)):
        a, sa = operand(m, k, 1, m)
        b, sb = operand(n, k, 128, n)
        cases.append((a, sa, b, sb, torch.empty(m, n, device="cuda")))
    for a, sa, b, sb, c in cases:
        ap.ap_matmul_fp8(a, sa, b, sb, c)
        done(ap)
        alone.append(c.clone())
        c.fill_(float("nan"))
    for _ in range(200):
        for a, sa, b, sb, c in cases:
            ap.ap_matmul_fp8(a, sa, b, sb, c)
    done(ap)
    assert all(torch.equal(case[4], want) for case, want in zip(cases, alone))


@pytest.mark.parametrize("m,n,k", MM_SIZES)
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_matmul(ap, m, n, k, tile, kind):
    check_matmul(ap, m, n, k, tile, TYPES[kind], seed=m + n + k)
    assert ap.ap_debug_get(ap.AP_DBG_LAST_PATH) == 10


@pytest.mark.parametrize("m,n,k", [(3, 300, 500), (40, 1000, 700), (150, 333, 260)])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 3)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_matmul_strided_output_stays_inside(ap, m, n, k, shift, pad, kind):
    c = Strided(m, n, TYPES[kind], n + pad, shift)
    check_matmul(ap, m, n, k, 128, TYPES[kind], c=c.view)
    assert c.intact()


@pytest.mark.parametrize("m,n,k", [(5, 200, 100), (150, 300, 200)])
def test_matmul_reads_only_k_columns(ap, m, n, k):
    """What lies past k in a row (here NaN codes) is not part of the product."""
    a, sa = operand(m, k, 1, 1)
    b, sb = operand(n, k, 1, 2)
    wide_a = torch.full((m, 512), 0x7F, dtype=torch.uint8, device="cuda")
    wide_b = torch.full((n, 512), 0x7F, dtype=torch.uint8, device="cuda")
    wide_a[:, 16:16 + k].copy_(a.view(torch.uint8))
    wide_b[:, 32:32 + k].copy_(b.view(torch.uint8))
    c, d = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    ap.ap_matmul_fp8(a, sa, b, sb, c, 1)
    ap.ap_matmul_fp8(wide_a[:, 16:16 + k], sa, wide_b[:, 32:32 + k], sb, d, 1)
    done(ap)
    assert torch.equal(c, d)


@pytest.mark.parametrize("m", [2, 150])
@pytest.mark.parametrize("tile", [1, 128])
def test_matmul_nan_stays_in_its_row_and_column(ap, m, tile):
    n, k = 300, 700
    a, sa = operand(m, k, 1, 1)
    b, sb = operand(n, k, tile, 2)
    a.view(torch.uint8)[1, 600] = 0x7F
    if tile == 1:
        sb[7, 2] = float("inf")
    c = torch.empty(m, n, device="cuda")
    ap.ap_matmul_fp8(a, sa, b, sb, c, tile)
    done(ap)
    bad = ~torch.isfinite(c)
    assert torch.isnan(c[1]).all()
    rest = torch.cat([bad[:1], bad[2:]])
    if tile == 1:
        assert rest[:, 7].all()
        rest[:, 7] = False
    assert not rest.any()


def test_matmul_no_k_and_empty(ap):
    c = torch.full((5, 9), 3.0, device="cuda")
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    ap.ap_matmul_fp8(e(5, 0).to(torch.uint8), e(5, 0), e(9, 0).to(torch.uint8), e(9, 0), c[:, :], 1)
    done(ap)
    assert (c == 0).all()
    ap.ap_matmul_fp8(empty8(0, 64), e(0, 1), empty8(9, 64), e(9, 1), e(0, 9), 1)
    done(ap)


@pytest.mark.parametrize("m,n,k", [(2, 500, 3000), (300, 600, 1500)])
def test_matmul_same_bits_every_time(ap, m, n, k):
    a, sa = operand(m, k, 1, 1)
    b, sb = operand(n, k, 128, 2)
    c = [torch.empty(m, n, device="cuda") for _ in range(6)]
    for x in c:
        ap.ap_matmul_fp8(a, sa, b, sb, x)
    done(ap)
    assert all(torch.equal(c[0], x) for x in c[1:])


def test_matmul_past_2_32_bytes(ap):
    m, n, k = 140000, 130, 32768
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB of device memory")
    a = torch.zeros(m, k, dtype=torch.uint8, device="cuda")
    tail, st = operand(3, k, 1, 1)
    a[-3:] = tail.view(torch.uint8)
    sa = torch.ones(m, k // 128, device="cuda")
    sa[-3:] = st
    b, sb = operand(n, k, 128, 2)
    c = torch.empty(m, n, device="cuda")
    d = torch.empty(n, m, device="cuda")
    ap.ap_matmul_fp8(a, sa, b, sb, c)
    one = torch.ones(n, k // 128, device="cuda")
    ap.ap_matmul_fp8(b, one, a, sa, d, 1)  # the long matrix as the second operand
    done(ap)
    want, terms = fu.matmul(f64(tail), f64(st), f64(b), f64(sb), 128)
    assert np.all(np.abs(f64(c[-3:]) - want) <= fu.matmul_bound(want, terms, k, torch.float32))
    want, terms = fu.matmul(f64(tail), f64(st), f64(b), f64(one), 1)
    assert np.all(np.abs(f64(d[:, -3:].t()) - want) <= fu.matmul_bound(want, terms, k, torch.float32))
    assert (c[:-3] == 0).all() and (d[:, :-3] == 0).all()


@pytest.mark.parametrize("m", [3, 200])
def test_matmul_bounded_wait(ap, m):
    """A stage that never fills: the waits give up, the call ends, the error is reported once, and the next call works."""
    a, sa = operand(m, 1000, 1, 1)
    b, sb = operand(300, 1000, 128, 2)
    c = torch.empty(m, 300, device="cuda")
    ap.ap_matmul_fp8(a, sa, b, sb, c)
    done(ap)
    ap.ap_debug_set(ap.AP_DBG_TIMEOUT_NS, 2_000_000)
    ap.ap_debug_set(ap.AP_DBG_EXPECT_TX_EXTRA, 16)
    ap.ap_matmul_fp8(a, sa, b, sb, c)
    assert ap.ap_check() == ap.AP_ERR_DEVICE_TIMEOUT
    reset_debug(ap)
    check_matmul(ap, m, 300, 1000, 128, torch.float32)


# ------------------------------------------------------------------ streams and graphs


def layer(ap, x, res, w, out, q, s, b, sb, c, stream=None):
    ap.ap_rms_norm(x, w, 1e-6, q=q, q_scales=s, residual=res, residual_out=out, stream=stream)
    ap.ap_matmul_fp8(q, s, b, sb, c, stream=stream)


def layer_state(m=40, n=300, k=1000):
    x, res, w = randn(m, k).bfloat16(), randn(m, k, seed=1), randn(k, seed=2)
    b, sb = operand(n, k, 128, 5)
    return [x, res, w, torch.empty_like(res), empty8(m, k), torch.empty(m, fu.blocks(k), device="cuda"), b, sb,
            torch.empty(m, n, device="cuda")]


def test_side_stream_and_graph(ap):
    state = layer_state()
    layer(ap, *state)
    done(ap)
    want = state[-1].clone()
    state[-1].zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layer(ap, *state, stream=side)
    side.synchronize()
    assert torch.equal(state[-1], want)
    state[-1].zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(ap, *state)
    for _ in range(3):
        state[-1].zero_()
        g.replay()
        done(ap)
        assert torch.equal(state[-1], want)


def test_quantize_scale_of_every_mantissa(ap):
    """s = max(amax / 448, 2^-126) is the correctly rounded quotient for all 2^23 mantissas, at a middle exponent and where
    the quotient becomes subnormal. (In 64 bits the quotient's second rounding is harmless: 53 >= 2 * 24 + 2 bits.)"""
    for exponent in (0x3F800000, 0x04800000, 0x04000000):
        x = (torch.arange(1 << 23, dtype=torch.int32, device="cuda") + exponent).view(torch.float32)[:, None]
        q, s = torch.empty(1 << 23, 1, dtype=torch.uint8, device="cuda"), torch.empty(1 << 23, 1, device="cuda")
        ap.ap_quantize(x, 1, q, s)
        done(ap)
        want = (x.double() / 448).float()
        assert torch.equal(s, torch.where(want < fu.MIN_SCALE, torch.full_like(want, fu.MIN_SCALE), want))


RING_SIZES = [(1, 8), (2, 200), (17, 512), (1500, 8), (999, 264), (400, 520), (700, 1000), (333, 2048), (311, 2056), (600, 5000),
              (460, 8192), (307, 8200), (308, 16384)]


@pytest.mark.parametrize("rows,cols", RING_SIZES)
@pytest.mark.parametrize("kind,res", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", None)])
def test_norm_ring_and_registers(ap, rows, cols, kind, res):
    """Both forms of the norm on the same rows (1: the ring wherever it takes them, 2: the register form)."""
    t = TYPES[kind]
    x = randn(rows, cols, seed=cols).to(t)
    residual = None if res is None else (2 * randn(rows, cols, seed=cols + 1)).to(TYPES[res])
    weight = 1 + 0.1 * randn(cols, seed=2)
    h, rr, yy = fu.norm(f64(x), None if res is None else f64(residual), f64(weight), 1e-5)
    rel = (fu.DEPTH / 2 + 8) * U
    for path in (1, 2):
        ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, path)
        out = None if res is None else torch.full_like(residual, float("nan"))
        y, q = torch.full_like(x, float("nan")), empty8(rows, cols)
        s, r = torch.empty(rows, fu.blocks(cols), device="cuda"), torch.empty(rows, device="cuda")
        ap.ap_rms_norm(x, weight, 1e-5, y=y, q=q, q_scales=s, residual=residual, residual_out=out, rstd=r)
        done(ap)
        # (past 8192 columns two stages of a row of both types may not fit)
        assert ap.ap_debug_get(ap.AP_DBG_LAST_FLAGS) == 4 or path == 2 or cols > 8192
        assert np.all(np.abs(f64(r) - rr) <= rel * rr)
        assert np.all(np.abs(f64(y) - yy) <= fu.rounding(yy, t) * (1 + rel) + rel * np.abs(yy))
        if res is not None:
            assert np.all(np.abs(f64(out) - h) <= fu.rounding(h, out.dtype) * (1 + U) + U * np.abs(h))
        fu.check_codes(q, s, yy, 1, rel, f"norm {rows}x{cols} path {path}")


@pytest.mark.parametrize("shift,pad", [(0, 8), (8, 24)])
def test_norm_ring_strided_rows_stay_inside(ap, shift, pad):
    rows, cols, t = 700, 1032, torch.bfloat16
    ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, 1)
    x = Strided(rows, cols, t, cols + pad, shift, randn(rows, cols).to(t))
    res = Strided(rows, cols, torch.float32, cols + 2 * pad, shift, randn(rows, cols, seed=1))
    q = Strided(rows, cols, torch.uint8, cols + pad, shift)
    s, w = torch.empty(rows, fu.blocks(cols), device="cuda"), randn(cols, seed=2)
    h, rr, yy = fu.norm(f64(x.view), f64(res.view), f64(w), 0.0)
    ap.ap_rms_norm(x.view, w, 0.0, y=x.view, q=q.view, q_scales=s, residual=res.view, residual_out=res.view)
    done(ap)
    assert ap.ap_debug_get(ap.AP_DBG_LAST_FLAGS) == 4 and all(b.intact() for b in (x, res, q))
    rel = (fu.DEPTH / 2 + 8) * U
    assert np.all(np.abs(f64(x.view) - yy) <= fu.rounding(yy, t) * (1 + rel) + rel * np.abs(yy))
    assert np.all(np.abs(f64(res.view) - h) <= fu.rounding(h, torch.float32) + U * np.abs(h))
    fu.check_codes(q.view.clone().view(E4M3), s, yy, 1, rel, "strided ring norm")


ODD_SIZES = [(1, 1), (1, 7), (2, 199), (17, 513), (1500, 9), (999, 263), (700, 1001), (311, 2057), (500, 4999), (307, 8201),
             (40, 16383)]


@pytest.mark.parametrize("rows,cols", ODD_SIZES)
@pytest.mark.parametrize("kind,res,shift,pad", [("f32", "f32", 0, 0), ("bf16", "bf16", 1, 0), ("bf16", "f32", 3, 5), ("f16", None, 0, 0),
                                                ("f16", "f32", 0, 1)])
def test_norm_rows_off_the_boundaries(ap, rows, cols, kind, res, shift, pad):
    """Rows that start and end anywhere, in both forms: what lies around them is neither read into results nor written."""
    t = TYPES[kind]
    data = randn(rows, cols, seed=cols).to(t)
    rdata = None if res is None else (2 * randn(rows, cols, seed=cols + 1)).to(TYPES[res])
    weight = torch.cat([torch.ones(1, device="cuda"), 1 + 0.1 * randn(cols, seed=2)])[1:]
    h, rr, yy = fu.norm(f64(data), None if res is None else f64(rdata), f64(weight), 1e-5)
    rel = (fu.DEPTH / 2 + 8) * U
    for path in (1, 2):
        ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, path)
        x = Strided(rows, cols, t, cols + pad, shift, data)
        y, q = Strided(rows, cols, t, cols + 2 * pad, 1), Strided(rows, cols, torch.uint8, cols + pad, shift)
        stream = None if res is None else Strided(rows, cols, TYPES[res], cols + pad, shift, rdata)
        s, r = torch.empty(rows, fu.blocks(cols), device="cuda"), torch.empty(rows, device="cuda")
        at = None if res is None else stream.view
        ap.ap_rms_norm(x.view, weight, 1e-5, y=y.view, q=q.view, q_scales=s, residual=at, residual_out=at, rstd=r)
        done(ap)
        assert ap.ap_debug_get(ap.AP_DBG_LAST_FLAGS) in ((12,) if path == 1 and cols <= 8192 else (8, 9, 12))
        assert all(b.intact() for b in (x, y, q) + (() if res is None else (stream,)))
        assert torch.equal(x.view, data)
        assert np.all(np.abs(f64(r) - rr) <= rel * rr)
        assert np.all(np.abs(f64(y.view) - yy) <= fu.rounding(yy, t) * (1 + rel) + rel * np.abs(yy))
        if res is not None:
            assert np.all(np.abs(f64(stream.view) - h) <= fu.rounding(h, TYPES[res]) * (1 + U) + U * np.abs(h))
        fu.check_codes(q.view.clone().view(E4M3), s, yy, 1, rel, f"norm {rows}x{cols} path {path}")
        ap.ap_rms_norm(x.view, weight, 1e-5, y=x.view)  # in place
        done(ap)
        assert x.intact()
        if res is None:
            assert torch.equal(x.view, y.view)


@pytest.mark.parametrize("rows,cols", ODD_SIZES)
@pytest.mark.parametrize("kind,res,dres,shift,pad", [("f32", "f32", True, 0, 0), ("bf16", "f32", True, 1, 0), ("f16", "f16", False, 3, 5),
                                                     ("bf16", "bf16", True, 0, 1), ("f16", "f32", False, 1, 3)])
def test_norm_backward_rows_off_the_boundaries(ap, rows, cols, kind, res, dres, shift, pad):
    t, rt = TYPES[kind], TYPES[res]
    dy, h, w, r, d = grad_case(rows, cols, t, rt, dres, seed=rows)
    for path in (1, 2):
        ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, path)
        bufs = [Strided(rows, cols, t, cols + pad, shift, dy), Strided(rows, cols, rt, cols + pad, shift, h)]
        more = Strided(rows, cols, rt, cols + 2 * pad, shift + 1, d) if dres else None
        at = more.view if dres else None
        dx, dw = Strided(rows, cols, rt, cols + pad, 1), torch.empty(cols, device="cuda")
        ws = torch.empty(ap.ap_rms_norm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
        ap.ap_rms_norm_backward(bufs[0].view, bufs[1].view, w, r, dx.view, dw, ws, dresidual=at)
        done(ap)
        assert dx.intact() and torch.equal(bufs[0].view, dy) and torch.equal(bufs[1].view, h)
        check_grad(dx.view, dw, dy, h, w, r, d)
        ap.ap_rms_norm_backward(bufs[0].view, bufs[1].view, w, r, bufs[1].view, dresidual=at)  # in place
        done(ap)
        assert bufs[1].intact() and torch.equal(bufs[1].view, dx.view)


@pytest.mark.parametrize("rows,cols", RING_SIZES)
@pytest.mark.parametrize("kind,res,dres", [("f32", "f32", True), ("bf16", "f32", True), ("f16", "f16", False)])
def test_norm_backward_ring_and_registers(ap, rows, cols, kind, res, dres):
    dy, h, w, r, d = grad_case(rows, cols, TYPES[kind], TYPES[res], dres, seed=cols)
    ws = torch.empty(ap.ap_rms_norm_backward_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    for path in (1, 2):
        ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, path)
        dx, dw = torch.full_like(h, float("nan")), torch.empty(cols, device="cuda")
        ap.ap_rms_norm_backward(dy, h, w, r, dx, dw, ws, dresidual=d)
        done(ap)
        check_grad(dx, dw, dy, h, w, r, d)


def test_norm_ring_first_and_last_unit(ap):
    """Rows at the very start and end of what the caller owns, beside NaN: nothing of the neighbours gets in."""
    rows, cols = 300, 1029
    flat = torch.full((rows * cols + 16,), float("nan"), dtype=torch.float16, device="cuda")
    x = flat[3:3 + rows * cols].view(rows, cols)
    x.copy_(randn(rows, cols).half())
    w, y, r = torch.ones(cols, device="cuda"), torch.empty(rows, cols, dtype=torch.float16, device="cuda"), torch.empty(rows, device="cuda")
    ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, 1)
    ap.ap_rms_norm(x, w, 1e-5, y=y, rstd=r)
    done(ap)
    assert ap.ap_debug_get(ap.AP_DBG_LAST_FLAGS) == 12
    rr = fu.norm(f64(x), None, f64(w), 1e-5)[1]
    assert np.all(np.abs(f64(r) - rr) <= (fu.DEPTH / 2 + 8) * U * rr) and bool(y.isfinite().all().item())


def test_norm_ring_bounded_wait(ap):
    """Rows that never arrive: both ring kernels give up, the error is reported once, and the next calls work."""
    x, w = randn(2000, 512), torch.ones(512, device="cuda")
    y, r = torch.empty_like(x), torch.empty(2000, device="cuda")
    ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, 1)
    ap.ap_rms_norm(x, w, 1e-6, y=y, rstd=r)
    done(ap)
    want, dx = y.clone(), torch.empty_like(x)
    for call in (lambda: ap.ap_rms_norm(x, w, 1e-6, y=y), lambda: ap.ap_rms_norm_backward(x, x, w, r, dx)):
        ap.ap_debug_set(ap.AP_DBG_TIMEOUT_NS, 2_000_000)
        ap.ap_debug_set(ap.AP_DBG_EXPECT_TX_EXTRA, 16)
        call()
        assert ap.ap_check() == ap.AP_ERR_DEVICE_TIMEOUT
        reset_debug(ap)
        ap.ap_debug_set(ap.AP_DBG_FORCE_PATH, 1)
        call()
        done(ap)
    assert torch.equal(y, want)
