"""The gated block's products with very many rows of x or of the weights: the most tiles, row tiles and passes. The 64-bit
forms are torch's on the device."""

import pytest
import torch

import gated_util as gu
from fp8_util import TYPES, U, blocks
from gpu_util import device, lib, reset_debug
from test_gpu_fp8 import operand

pytestmark = pytest.mark.gpu


@pytest.fixture
def ap():
    device()
    ap = lib()
    reset_debug(ap)
    yield ap
    reset_debug(ap)


@pytest.mark.parametrize("m,n,k", [(1 << 20, 17, 33), (5, 300000, 70), (20, 100003, 32)])
@pytest.mark.parametrize("gated", [False, True])
def test_w4(ap, m, n, k, gated):
    """Whole numbers: a sum of |x| <= 3 times |code - 8| <= 8 is exact, and its product with the other sum too."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randint(-3, 4, (m, k), generator=g, device="cuda").to(torch.bfloat16)
    room = torch.randint(0, 256, (n, -(-k // 32) * 16), generator=g, device="cuda", dtype=torch.uint8)
    codes, scales = room[:, : (k + 1) // 2], torch.ones(n, -(-k // 64), dtype=torch.bfloat16, device="cuda")
    w = torch.stack([codes & 15, codes >> 4], 2).view(n, -1)[:, :k].double() - 8
    c = torch.empty(m, n, device="cuda")
    if gated:
        ap.ap_gated_matmul_w4(x, codes, scales, codes, scales, gu.ACTS["silu"], c, 64)
    else:
        ap.ap_matmul_w4(x, codes, scales, c, 64)
    assert ap.ap_check() == 0
    for rows in torch.arange(m, device="cuda").split(1 << 17):
        want = x[rows].double() @ w.t()
        if gated:  # 13 + 3 |g| roundings of the activation and the product, |g| below 128 where they matter
            near = (13 + 3 * want.abs().clamp(max=128)) * U * want.square() + 1e-30
            assert ((c[rows].double() - want * want * torch.sigmoid(want)).abs() <= near).all()
        else:
            assert torch.equal(c[rows].double(), want)


@pytest.mark.parametrize("m,n,k", [(200001, 24, 40), (3, 300001, 48), (100, 200003, 32), (60000, 130, 16)])
def test_gated(ap, m, n, k):
    a, sa = operand(m, k, 1, 1)
    g, sg = operand(n, k, 128, 2)
    u, su = operand(n, k, 128, 3)
    a, g, u = (t.float().clamp(-8, 8).to(torch.float8_e4m3fn) for t in (a, g, u))
    out = [torch.empty(m, n, device="cuda") for _ in range(3)]
    q, s = torch.empty(m, n, dtype=torch.uint8, device="cuda"), torch.empty(m, blocks(n), device="cuda")
    pad = lambda t: torch.nn.functional.pad(t.view(torch.uint8), (0, -k % 16))[:, :k]
    ap.ap_gated_matmul_fp8(pad(a), sa, pad(g), sg, pad(u), su, gu.ACTS["silu"], gate=out[0], up=out[1], y=out[2], q=q, q_scales=s)
    assert ap.ap_check() == 0
    for rows in torch.arange(m, device="cuda").split(max(1, (1 << 24) // n)):
        x = a[rows].double()
        for w, sw, got in ((g, sg, out[0]), (u, su, out[1])):
            by = sa[rows].double() * sw[:, 0].double().repeat_interleave(128)[:n]
            want, terms = (x @ w.double().t()) * by, (x.abs() @ w.double().abs().t()) * by
            assert ((got[rows].double() - want).abs() <= 84 * U * terms + 1e-30).all()
        v, f, y = out[0][rows].double(), out[1][rows].double(), out[2][rows].double()
        act = v * torch.sigmoid(v)
        assert ((y - act * f).abs() <= (13 + 3 * v.abs().clamp(max=128)) * U * (act * f).abs() + (v * f).abs() * 2.0 ** -125).all()
        top = torch.nn.functional.pad(out[2][rows].abs(), (0, -n % 128)).view(len(rows), -1, 128).amax(2)
        assert ((s[rows] - top / 448).abs() <= 2 * U * top / 448 + 2.0 ** -126).all()
        held = q[rows].view(torch.float8_e4m3fn).double() * s[rows].double().repeat_interleave(128, 1)[:, :n]
        step = s[rows].double().repeat_interleave(128, 1)[:, :n]
        # half a step of e4m3; v / s is known to 3 U, which of a subnormal number, below 2^-6, is 48 U of half a step of 2^-9
        assert ((held - y).abs() <= torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * step) * (1 + 64 * U)).all()
