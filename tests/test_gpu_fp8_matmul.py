"""The 8-bit matrix product where its forms can go wrong: see each test."""

import pytest
import torch

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
