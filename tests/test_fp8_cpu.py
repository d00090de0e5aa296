"""The 8-bit block-scaled operators without a GPU: what the entry points refuse
before any CUDA call, the workspace's size, and the plain forms' own pins.
The addresses are made up, so no call here may pass its checks: on a machine
with a GPU it would launch."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import fp8_util as fu  # noqa: E402

A, B, C, D, E, F, G = (0x7F0000000000 + (i << 36) for i in range(7))


@pytest.fixture(scope="module")
def ap():
    from async_global_shared_gb300 import build

    build.build()
    import async_global_shared_gb300 as ap

    ap.load()
    return ap


def norm(ap, **kw):
    d = dict(x=A, ldx=256, type=ap.AP_BF16, residual=B, out=C, ldr=256, rtype=ap.AP_F32, w=D, wtype=ap.AP_F32, eps=1e-6,
             rows=4, cols=256, y=E, ldy=256, q=F, ldq=256, s=G, r=G + 4096)
    assert set(kw) <= set(d)
    d.update(kw)
    return ap.load().ap_rms_norm(*d.values(), None)


def test_norm_refusals(ap):
    assert norm(ap, type=7) == ap.AP_ERR_ARG
    assert norm(ap, type=ap.AP_F16, wtype=ap.AP_BF16) == ap.AP_ERR_ARG
    assert norm(ap, type=ap.AP_F16, rtype=ap.AP_BF16) == ap.AP_ERR_ARG
    assert norm(ap, eps=-1.0) == ap.AP_ERR_ARG
    assert norm(ap, eps=float("nan")) == ap.AP_ERR_ARG
    assert norm(ap, rows=-1) == ap.AP_ERR_SHAPE
    assert norm(ap, cols=1 << 41) == ap.AP_ERR_SHAPE
    for ld in ("ldx", "ldr", "ldy", "ldq"):
        assert norm(ap, **{ld: 255}) == ap.AP_ERR_SHAPE
    for p in ("x", "w", "residual", "out", "q", "s"):
        assert norm(ap, **{p: None}) == ap.AP_ERR_NULL
    assert norm(ap, y=None, q=None, s=None) == ap.AP_ERR_NULL
    for p, off in (("x", 1), ("residual", 2), ("out", 2), ("w", 2), ("y", 1), ("s", 2), ("r", 2)):
        assert norm(ap, **{p: (A if p == "x" else G) + off}) == ap.AP_ERR_ALIGN
    assert norm(ap, out=B + 4) == ap.AP_ERR_ALIAS
    assert norm(ap, y=A + 2) == ap.AP_ERR_ALIAS
    assert norm(ap, y=A, ldy=512) == ap.AP_ERR_ALIAS  # in place needs the same pitch
    assert norm(ap, q=E) == ap.AP_ERR_ALIAS
    assert norm(ap, s=D) == ap.AP_ERR_ALIAS
    assert norm(ap, r=G + 4) == ap.AP_ERR_ALIAS
    assert norm(ap, rows=0, x=None, w=None) == ap.AP_OK
    assert norm(ap, cols=0, x=None, w=None) == ap.AP_OK


def test_column_slices_that_touch_are_refused(ap):
    # one byte column past the halves of a 4 x 512 matrix; every call here is
    # refused (the halves themselves are accepted: tests/test_gpu_fp8.py)
    assert norm(ap, ldx=512, y=A + 2 * 255, ldy=512) == ap.AP_ERR_ALIAS
    assert norm(ap, ldx=512, y=A - 2 * 255, ldy=512) == ap.AP_ERR_ALIAS


def grad(ap, **kw):
    d = dict(dy=A, lddy=256, type=ap.AP_BF16, h=B, ldh=256, rtype=ap.AP_F32, w=C, wtype=ap.AP_F32, r=C + 4096, dres=D,
             lddr=256, rows=4, cols=256, dx=E, lddx=256, dw=F, ws=G)
    assert set(kw) <= set(d)
    d.update(kw)
    return ap.load().ap_rms_norm_backward(*d.values(), None)


def test_norm_backward_refusals(ap):
    assert grad(ap, rtype=ap.AP_F16) == ap.AP_ERR_ARG
    assert grad(ap, wtype=9) == ap.AP_ERR_ARG
    assert grad(ap, rows=-1) == ap.AP_ERR_SHAPE
    for ld in ("lddy", "ldh", "lddr", "lddx"):
        assert grad(ap, **{ld: 255}) == ap.AP_ERR_SHAPE
    for p in ("dy", "h", "w", "r", "dx", "ws"):
        assert grad(ap, **{p: None}) == ap.AP_ERR_NULL
    assert grad(ap, ws=G + 8) == ap.AP_ERR_ALIGN
    assert grad(ap, dw=F + 2) == ap.AP_ERR_ALIGN
    assert grad(ap, dx=B + 4) == ap.AP_ERR_ALIAS
    assert grad(ap, dx=A) == ap.AP_ERR_ALIAS  # other element size
    assert grad(ap, dw=C) == ap.AP_ERR_ALIAS
    assert grad(ap, ws=E) == ap.AP_ERR_ALIAS
    assert grad(ap, cols=0) == ap.AP_OK
    assert grad(ap, rows=0, dw=None, dy=None) == ap.AP_OK


def test_norm_backward_workspace(ap):
    f = ap.load().ap_rms_norm_backward_workspace
    assert f(0, 100) == 0 and f(100, 0) == 0
    assert f(-1, 4) == -1 and f(4, -1) == -1 and f(1 << 30, 1 << 30) == -1
    assert f(1, 100) == 400
    for cols in (1, 1000, 4096, 8192, 100000):
        assert f(1 << 20, cols) % (4 * cols) == 0 and f(1 << 20, cols) <= 16 * 152 * 4 * cols
    with pytest.raises(ap.APError):
        ap.ap_rms_norm_backward_workspace(-1, 4)


def quant(ap, **kw):
    d = dict(x=A, ldx=300, type=ap.AP_F32, rows=200, cols=300, block=1, q=B, ldq=300, s=C, qt=D, ldqt=200, st=E)
    assert set(kw) <= set(d)
    d.update(kw)
    return ap.load().ap_quantize(*d.values(), None)


def test_quantize_refusals(ap):
    assert quant(ap, type=-1) == ap.AP_ERR_ARG
    assert quant(ap, block=64) == ap.AP_ERR_ARG
    assert quant(ap, rows=-1) == ap.AP_ERR_SHAPE
    for ld, v in (("ldx", 299), ("ldq", 299), ("ldqt", 199)):
        assert quant(ap, **{ld: v}) == ap.AP_ERR_SHAPE
    assert quant(ap, x=None) == ap.AP_ERR_NULL
    assert quant(ap, q=None) == ap.AP_ERR_NULL
    assert quant(ap, st=None) == ap.AP_ERR_NULL
    assert quant(ap, q=None, s=None, qt=None, st=None) == ap.AP_ERR_NULL
    assert quant(ap, x=A + 2) == ap.AP_ERR_ALIGN
    assert quant(ap, s=C + 2) == ap.AP_ERR_ALIGN
    assert quant(ap, q=A) == ap.AP_ERR_ALIAS
    assert quant(ap, qt=B + 100) == ap.AP_ERR_ALIAS
    assert quant(ap, st=C) == ap.AP_ERR_ALIAS
    assert quant(ap, rows=0, x=None) == ap.AP_OK


def mm(ap, **kw):
    d = dict(a=A, lda=512, sa=B, b=C, ldb=512, sb=D, block=128, c=E, ldc=300, type=ap.AP_BF16, m=40, n=300, k=500)
    assert set(kw) <= set(d)
    d.update(kw)
    return ap.load().ap_matmul_fp8(*d.values(), None)


def test_matmul_refusals(ap):
    assert mm(ap, type=3) == ap.AP_ERR_ARG
    assert mm(ap, block=32) == ap.AP_ERR_ARG
    assert mm(ap, m=-1) == ap.AP_ERR_SHAPE
    assert mm(ap, k=1 << 31) == ap.AP_ERR_SHAPE
    for ld, v in (("lda", 496), ("ldb", 496), ("ldc", 299)):
        assert mm(ap, **{ld: v}) == ap.AP_ERR_SHAPE
    for p in ("a", "sa", "b", "sb", "c"):
        assert mm(ap, **{p: None}) == ap.AP_ERR_NULL
    assert mm(ap, a=A + 8) == ap.AP_ERR_ALIGN
    assert mm(ap, b=C + 1) == ap.AP_ERR_ALIGN
    assert mm(ap, lda=520) == ap.AP_ERR_ALIGN
    assert mm(ap, ldb=520) == ap.AP_ERR_ALIGN
    assert mm(ap, c=E + 1) == ap.AP_ERR_ALIGN
    assert mm(ap, sa=B + 2) == ap.AP_ERR_ALIGN
    for p in (A, B, C, D):
        assert mm(ap, c=p) == ap.AP_ERR_ALIAS
    assert mm(ap, m=0, a=None, c=None) == ap.AP_OK
    assert mm(ap, n=0) == ap.AP_OK


def test_tensors_are_checked(ap):
    x = torch.zeros(4, 128)
    with pytest.raises(TypeError):
        ap.ap_rms_norm(x, torch.ones(128), 1e-6, y=torch.zeros(4, 128))  # not on a device
    with pytest.raises(TypeError):
        ap.ap_matmul_fp8(x, x, x, x, x)  # not 8-bit codes
    with pytest.raises(TypeError):
        ap.ap_quantize(x, 1, q=torch.zeros(4, 128, dtype=torch.uint8), scales=torch.zeros(4, 1))


def test_plain_codes_pin():
    """The plain quantiser on values whose codes are known: 448 s, halves, ties to even and the zero block."""
    v = torch.zeros(2, 256)
    v[0, :6] = torch.tensor([448.0, -448.0, 1.0, 17.0, 19.0, 2.0 ** -9])  # scale 1: 17 and 19 are ties between 16, 18, 20
    q, s = fu.codes_32(v, 1)
    assert s.tolist() == [[1.0, 2.0 ** -126], [2.0 ** -126, 2.0 ** -126]]
    assert q[0, :6].float().tolist() == [448.0, -448.0, 1.0, 16.0, 20.0, 2.0 ** -9]
    assert q[0, :6].view(torch.uint8).tolist() == [0x7E, 0xFE, 0x38, 0x58, 0x5A, 0x01]
    fu.check_codes(q, s, v.double().numpy(), 1, 0.0, "pin")
    with pytest.raises(AssertionError):
        w = q.clone()
        w.view(torch.uint8)[0, 2] += 1  # one code off by one
        fu.check_codes(w, s, v.double().numpy(), 1, 0.0, "planted")


def test_plain_matmul_pin():
    a, b = np.array([[2.0, 3.0]]), np.array([[5.0, 7.0], [1.0, -1.0]])
    c, terms = fu.matmul(a, np.array([[0.5]]), b, np.array([[2.0]]), 128)
    assert c.tolist() == [[31.0, -1.0]] and terms.tolist() == [[31.0, 5.0]]
