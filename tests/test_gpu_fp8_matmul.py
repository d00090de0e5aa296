"""The 8-bit matrix product where its forms can go wrong: see each test."""

import numpy as np
import pytest
import torch

import fp8_util as fu
from fp8_util import f64
from gpu_util import device, lib, reset_debug
from test_gpu_fp8 import check_matmul, done, operand

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


@pytest.mark.parametrize("m,n,k", [(1, 130, 4096), (3, 1000, 2048), (7, 129, 8192), (13, 333, 6000), (31, 100, 4096), (17, 257, 1500),
                                   (45, 250, 2000), (127, 131, 4000)])
def test_shares_of_uneven_length(ap, m, n, k):
    """k split over a cluster whose CTAs' parts of a tile are no multiples of a warp: lanes add up different numbers of
    values, and none of a warp may leave a barrier of the cluster before the others."""
    for tile in (1, 128):
        check_matmul(ap, m, n, k, tile, torch.float32)
        assert flags(ap) >> 4 > 1
    a, sa = operand(m, k, 1, 1)
    b, sb = operand(n, k, 128, 2)
    c = [torch.empty(m, n, device="cuda") for _ in range(50)]
    for out in c:
        ap.ap_matmul_fp8(a, sa, b, sb, out)
    done(ap)
    assert all(torch.equal(c[0], out) for out in c[1:])


# one case for each form: a's rows on 16 and 32 columns, 128 x 128 tiles, pairs of CTAs on 256 x 256
FORMS = [(5, 300, 700), (30, 200, 1000), (100, 333, 900), (1100, 2400, 520)]


def form(m):
    return 1 if m <= 32 else (0 if m < 1000 else 2)


def scaled_operand(rows, k, tile, exponent, seed):
    q, s = operand(rows, k, tile, seed)
    return q, s.clamp(0.25, 4) * 2.0 ** exponent


def by_definition(a, sa, b, sb, tile):
    """c with each block's two scales multiplied first, in 32 bits, and the sum of its terms' magnitudes."""
    (m, k), n = a.shape, b.shape[0]
    a, b = np.pad(f64(a), ((0, 0), (0, -k % 128))), np.pad(f64(b), ((0, 0), (0, -k % 128)))
    sa, sb = sa.cpu().numpy(), np.repeat(sb.cpu().numpy(), tile, 0)[:n]
    c, terms = np.zeros((m, n)), np.zeros((m, n))
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        for kb in range(fu.blocks(k)):
            at = slice(128 * kb, 128 * kb + 128)
            both = np.outer(sa[:, kb], sb[:, kb]).astype(np.float64)  # a float32 product of float32 scales
            c += both * (a[:, at] @ b[:, at].T)
            terms += np.abs(both) * (np.abs(a[:, at]) @ np.abs(b[:, at]).T)
    return c, terms


@pytest.mark.parametrize("m,n,k", FORMS)
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("ea,eb", [(-124, -3), (-3, -124), (-68, -66), (-40, -95), (110, -105), (-110, 105), (124, -124), (-124, 124),
                                   (60, 30), (0, 0)])
def test_scales_are_multiplied_first(ap, m, n, k, tile, ea, eb):
    """Very small scales with very large ones keep every bit; where the product is subnormal the term is that product's."""
    a, sa = scaled_operand(m, k, 1, ea, 1)
    b, sb = scaled_operand(n, k, tile, eb, 2)
    c = torch.empty(m, n, device="cuda")
    ap.ap_matmul_fp8(a, sa, b, sb, c, tile)
    done(ap)
    assert flags(ap) & 3 == form(m)
    want, terms = by_definition(a, sa, b, sb, tile)
    # sums of subnormal values: half of 2^-149 for each addition and for the result
    near = fu.matmul_bound(want, terms, k, torch.float32) + (fu.blocks(k) + 1) * 2.0 ** -150
    assert np.all(np.abs(f64(c) - want) <= near)


@pytest.mark.parametrize("m,n,k", FORMS)
@pytest.mark.parametrize("tile", [1, 128])
def test_scales_whose_product_is_no_float(ap, m, n, k, tile):
    """Two scales past 2^64: the term is an infinity, NaN where the block's sum is 0; rows without them are not touched."""
    a, sa = operand(m, k, 1, 1)
    b, sb = operand(n, k, tile, 2)
    sb[:, 1] = 2.0 ** 70
    sa[1, 1] = 2.0 ** 70
    c = torch.empty(m, n, device="cuda")
    ap.ap_matmul_fp8(a, sa, b, sb, c, tile)
    done(ap)
    assert not torch.isfinite(c[1]).any() and torch.isfinite(c[2:]).all() and torch.isfinite(c[0]).all()
    a.view(torch.uint8)[1, 128:256] = 0
    ap.ap_matmul_fp8(a, sa, b, sb, c, tile)
    done(ap)
    assert torch.isnan(c[1]).all() and torch.isfinite(c[2:]).all() and torch.isfinite(c[0]).all()
