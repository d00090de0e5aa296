"""The gated product beside the two plain products it stands for, bit for bit where both share k alike."""

import pytest
import torch

import gated_util as gu
from gpu_util import device, lib, reset_debug
from test_gpu_gated_matmul import FORMS, done, flags, operands

pytestmark = pytest.mark.gpu


@pytest.fixture
def ap():
    device()
    ap = lib()
    reset_debug(ap)
    yield ap
    reset_debug(ap)


def test_equal_where_both_share_k_alike(ap):
    """g and u add up the same blocks' products in the same order as ap_matmul_fp8's c, wherever the same number of CTAs
    shares k: whatever the tiles' sizes, each number is the same. Every form has such a case here."""
    equal = set()
    for m, n, k in FORMS + [(1, 130, 128), (16, 200, 2000), (32, 129, 4000), (64, 100, 1000), (1100, 1200, 1000), (2048, 2560, 300)]:
        a, sa, wg, sg, wu, su = operands(m, n, k)
        g, u, y, c = (torch.empty(m, n, device="cuda") for _ in range(4))
        ap.ap_gated_matmul_fp8(a, sa, wg, sg, wu, su, gu.ACTS["silu"], y=y, gate=g, up=u)
        form, split = flags(ap) & 3, flags(ap) >> 4
        for w, s, got in ((wg, sg, g), (wu, su, u)):
            ap.ap_matmul_fp8(a, sa, w, s, c)
            if flags(ap) >> 4 == split:
                done(ap)
                assert torch.equal(c, got), (m, n, k)
                equal.add((form, split > 1))
    done(ap)
    # few rows and a CTA a tile, both with k in one piece and shared; pairs, which never share it
    assert {form for form, _ in equal} == {0, 1, 2} and any(shared for _, shared in equal)
