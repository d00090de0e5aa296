"""Sums of the products with 4-bit weights, which are of x and code - zero themselves: whole numbers come out exactly, a
column whose code is its zero point takes no part however large its x, every zero point a byte holds, infinities."""

import numpy as np
import pytest
import torch

import gated_util as gu
from fp8_util import TYPES, f64
from gpu_util import device, lib, reset_debug

pytestmark = pytest.mark.gpu

FORMS = [1, 7, 12, 20, 40]  # rows of x: 8, 16 and 32 a pass, and more than one pass


@pytest.fixture
def ap():
    device()
    ap = lib()
    reset_debug(ap)
    yield ap
    reset_debug(ap)


def packed(codes):
    """Codes (n x k, whole numbers) two a byte in rows of whole 16-byte units."""
    n, k = codes.shape
    c = torch.nn.functional.pad(codes.to(torch.uint8), (0, k % 2))
    room = torch.full((n, -(-c.shape[1] // 32) * 16), 0xA5, dtype=torch.uint8)
    room[:, : c.shape[1] // 2] = c[:, 0::2] | c[:, 1::2] << 4
    return room.cuda()[:, : c.shape[1] // 2]


def products(ap, x, codes, scales, zeros, group):
    """c in 32 bits, and y of the gated form with this weight twice, silu."""
    c, y = (torch.full((x.shape[0], codes.shape[0]), float("nan"), device="cuda") for _ in range(2))
    ap.ap_matmul_w4(x, codes, scales, c, group, zeros=zeros)
    ap.ap_gated_matmul_w4(x, codes, scales, codes, scales, gu.ACTS["silu"], y, group, gate_zeros=zeros, up_zeros=zeros)
    assert ap.ap_check() == 0
    return c, y


def check(ap, x, codes, zeros, group, kind, scale=1.0):
    """Whole numbers below 2^24 in every partial sum: c is exact, y what the activation makes of it."""
    (n, k), groups = codes.shape, -(-codes.shape[1] // group)
    scales = torch.full((n, groups), scale, dtype=TYPES[kind], device="cuda")
    c, y = products(ap, x, packed(codes), scales, None if zeros is None else zeros.to(torch.uint8).cuda(), group)
    z = np.full((n, k), 8.0) if zeros is None else np.repeat(f64(zeros), group, 1)[:, :k]
    w = f64(codes) - z
    want = np.stack([(np.where(w == 0, 0.0, f64(x)[i]) * w).sum(1) for i in range(x.shape[0])]) * scale
    assert np.array_equal(f64(c), want)
    assert np.all(np.abs(f64(y) - gu.value("silu", want) * want) <= gu.gated_bound("silu", want, 0, want, 0, torch.float32))


@pytest.mark.parametrize("m", FORMS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind,huge", [("bf16", 2.0 ** 100), ("f16", 65504.0)])
def test_a_weight_of_zero_keeps_a_huge_x_out(ap, m, group, kind, huge):
    """A few channels of x many times larger than the rest, where every code is its zero point."""
    n, k = 50, 1001
    g = torch.Generator().manual_seed(m + group)
    for given in (False, True):
        x = torch.randint(-8, 9, (m, k), generator=g).to(TYPES[kind])
        codes = torch.randint(0, 16, (n, k), generator=g)
        zeros = torch.randint(0, 16, (n, -(-k // group)), generator=g) if given else None
        at = torch.arange(3, k, 37)
        codes[:, at] = zeros[:, at // group] if given else 8
        x[:, at] = torch.where(torch.rand(m, len(at), generator=g) < 0.5, huge, -huge).to(x.dtype)
        check(ap, x.cuda(), codes, zeros, group, kind)


@pytest.mark.parametrize("m", FORMS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_every_zero_point(ap, m, group, kind):
    """0 to 255, in one weight, in weights of small ones only, and of 255 only; x of one sign. Partial sums stay below
    8 * 255 * 700 < 2^24 in the scale's units."""
    n, k = 256, 700
    g = torch.Generator().manual_seed(m)
    x = torch.randint(0, 9, (m, k), generator=g).to(TYPES[kind]).cuda()
    codes = torch.randint(0, 16, (n, k), generator=g)
    each = torch.arange(n)[:, None].expand(n, -(-k // group)).contiguous()
    for zeros in (each, each.roll(17, 0) % 16, torch.full_like(each, 128), torch.full_like(each, 129), torch.full_like(each, 255)):
        check(ap, x, codes, zeros, group, kind, 0.125)


@pytest.mark.parametrize("m", FORMS)
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_an_infinity_in_x(ap, m, group, kind):
    """Infinite where the weight is not 0, with its sign; NaN only where it is, as 0 times infinity is."""
    n, k = 32, 300
    codes = torch.arange(n)[:, None].expand(n, k) % 16
    scales = torch.full((n, -(-k // group)), 0.5, dtype=TYPES[kind], device="cuda")
    for zeros in (None, 3, 255):
        z = None if zeros is None else torch.full(scales.shape, zeros, dtype=torch.uint8, device="cuda")
        w = (torch.arange(n) % 16 - (8 if zeros is None else zeros)).double()
        for sign in (1, -1):
            x = torch.ones(m, k, dtype=TYPES[kind], device="cuda")
            x[:, 5] = sign * float("inf")
            c, _ = products(ap, x, packed(codes), scales, z, group)
            want = (w * sign * float("inf")).float().cuda().expand(m, n)
            assert torch.equal(torch.isnan(c), torch.isnan(want))
            assert torch.equal(torch.nan_to_num(c, nan=0.0), torch.nan_to_num(want, nan=0.0))


@pytest.mark.parametrize("m", FORMS)
def test_products_near_the_largest_float(ap, m):
    """x of 2^124 times weights of -4 to 4, with a scale that brings them back: nothing passes the largest float."""
    n, k = 40, 256
    codes = torch.full((n, k), 8)
    at = torch.arange(n) * 6
    codes[torch.arange(n), at] = 8 + torch.arange(n) % 9 - 4
    x = torch.full((m, k), 2.0 ** 124, dtype=torch.bfloat16)
    c, _ = products(ap, x.cuda(), packed(codes), torch.full((n, 2), 2.0 ** -100, dtype=torch.bfloat16, device="cuda"), None, 128)
    assert torch.equal(c.cpu(), ((torch.arange(n) % 9 - 4) * 2.0 ** 24).expand(m, n))
