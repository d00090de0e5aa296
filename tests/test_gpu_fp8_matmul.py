"""The 8-bit matrix product where its forms can go wrong: see each test."""

import numpy as np
import pytest
import torch

import fp8_util as fu
from fp8_util import TYPES, Strided, f64
from gpu_util import device, lib, reset_debug
from test_gpu_fp8 import check_matmul, done, operand, randn

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


# ------------------------------------------------------------------ pairs of CTAs
#
# More than 128 rows and at least 38 tiles of 256 x 256. A pair whose second CTA has no rows at all, tiles that end
# everywhere, k of one block and of many, more tiles than pairs.
PAIRS = [(129, 9800, 1000), (300, 5000, 384), (1100, 2400, 520), (2048, 2048, 128), (700, 3300, 2600), (2500, 5200, 300), (257, 4900, 1)]


@pytest.mark.parametrize("m,n,k", PAIRS)
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_pairs(ap, m, n, k, tile, kind):
    check_matmul(ap, m, n, k, tile, TYPES[kind], seed=m + k)
    assert flags(ap) & 3 == 2


@pytest.mark.parametrize("m,n,k", [(1100, 2400, 520), (300, 5001, 384), (2500, 5203, 300)])
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 3), (8, 24)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_pairs_strided_output_stays_inside(ap, m, n, k, tile, shift, pad, kind):
    """Rows of c on and off the 16-byte boundaries, with guards between and around them."""
    c = Strided(m, n, TYPES[kind], n + pad, shift)
    check_matmul(ap, m, n, k, tile, TYPES[kind], c=c.view)
    assert c.intact() and flags(ap) & 3 == 2


@pytest.mark.parametrize("tile", [1, 128])
def test_pairs_nan_stays_in_its_row_and_column(ap, tile):
    m, n, k = 1100, 2400, 700
    a, sa = operand(m, k, 1, 1)
    b, sb = operand(n, k, tile, 2)
    rows, cols = [1, 127, 128, 300, 1099], [7, 300, 2399]
    for r in rows:  # either CTA of a pair, the last rows
        a.view(torch.uint8)[r, 600] = 0x7F
    if tile == 1:
        for j in cols:
            sb[j, 2] = float("inf")
    c = torch.empty(m, n, device="cuda")
    ap.ap_matmul_fp8(a, sa, b, sb, c, tile)
    done(ap)
    bad = ~torch.isfinite(c)
    assert flags(ap) & 3 == 2 and torch.isnan(c[rows]).all()
    bad[rows] = False
    if tile == 1:
        assert not torch.isfinite(c[:, cols]).any()
        bad[:, cols] = False
    assert not bad.any()


@pytest.mark.parametrize("tile", [1, 128])
def test_pairs_read_only_k_columns(ap, tile):
    m, n, k = 1100, 2400, 200
    a, sa = operand(m, k, 1, 1)
    b, sb = operand(n, k, tile, 2)
    wide_a = torch.full((m, 512), 0x7F, dtype=torch.uint8, device="cuda")
    wide_b = torch.full((n, 512), 0x7F, dtype=torch.uint8, device="cuda")
    wide_a[:, 16:16 + k].copy_(a.view(torch.uint8))
    wide_b[:, 32:32 + k].copy_(b.view(torch.uint8))
    c = [torch.empty(m, n, device="cuda") for _ in range(4)]
    for out in c[1:]:
        ap.ap_matmul_fp8(wide_a[:, 16:16 + k], sa, wide_b[:, 32:32 + k], sb, out, tile)
    ap.ap_matmul_fp8(a, sa, b, sb, c[0], tile)
    done(ap)
    assert flags(ap) & 3 == 2 and all(torch.equal(c[0], out) for out in c[1:])


@pytest.mark.parametrize("tile", [1, 128])
def test_pairs_bounded_wait(ap, tile):
    """A stage that never fills: both CTAs' waits give up, the error is reported once, and the next call works."""
    m, n, k = 1100, 2400, 1000
    a, sa = operand(m, k, 1, 1)
    b, sb = operand(n, k, tile, 2)
    c = torch.empty(m, n, device="cuda")
    ap.ap_matmul_fp8(a, sa, b, sb, c, tile)
    done(ap)
    assert flags(ap) & 3 == 2
    ap.ap_debug_set(ap.AP_DBG_TIMEOUT_NS, 2_000_000)
    ap.ap_debug_set(ap.AP_DBG_EXPECT_TX_EXTRA, 16)
    ap.ap_matmul_fp8(a, sa, b, sb, c, tile)
    assert ap.ap_check() == ap.AP_ERR_DEVICE_TIMEOUT
    assert ap.ap_check() == ap.AP_OK
    reset_debug(ap)
    check_matmul(ap, m, n, k, tile, torch.float32)


def test_products_between_the_library_s(ap):
    """Kernels that hold tensor memory, this library's and torch's, one behind another in a stream: each product is what it
    is alone, and none keeps another from starting."""
    x, y = randn(512, 2048).bfloat16(), randn(2048, 512, seed=1).bfloat16()
    big = randn(2048, 2048, seed=2).bfloat16()
    cases, alone = [], []
    for m, n, k in ((1, 8192, 4096), (16, 8192, 2048), (32, 8192, 4096), (64, 4096, 4096), (2048, 2560, 1024)):
        cases.append((*operand(m, k, 1, m), *operand(n, k, 128, n), torch.empty(m, n, device="cuda")))
        ap.ap_matmul_fp8(*cases[-1])
        done(ap)
        alone.append(cases[-1][-1].clone())
    want = [x @ y, big @ big]
    got = None
    for _ in range(100):
        for case in cases:
            case[-1].fill_(float("nan"))
            ap.ap_matmul_fp8(*case)
            got = [x @ y, big @ big]
            ap.ap_matmul_fp8(*case)
    done(ap)
    assert all(torch.equal(case[-1], c) for case, c in zip(cases, alone))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
