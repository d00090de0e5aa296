"""Products with 4-bit weights for more rows of x than one pass takes, with k shared by a cluster or whole."""

import pytest
import torch

from gpu_util import device, lib, reset_debug
from test_gpu_gated_w4 import check

pytestmark = pytest.mark.gpu


@pytest.fixture
def ap():
    device()
    ap = lib()
    reset_debug(ap)
    yield ap
    reset_debug(ap)


# last passes of 1, 6, 8, 1, 1, 8 and 1 rows; few columns and long sums, whose k a cluster shares, and many columns
@pytest.mark.parametrize("m,n,k,shared", [(33, 24, 20000, True), (70, 100, 9000, True), (40, 700, 4104, True), (65, 5000, 2048, None),
                                          (257, 1000, 4104, True), (1000, 130, 1300, True), (65, 8192, 512, False)])
@pytest.mark.parametrize("act", [None, "gelu"])
@pytest.mark.parametrize("kind,group,zeros", [("bf16", 32, True), ("f16", 64, False), ("bf16", 128, True)])
def test_more_rows_than_one_pass(ap, m, n, k, shared, act, kind, group, zeros):
    check(ap, m, n, k, group, zeros, kind, "f32" if group == 64 else kind, act, seed=m)
    if shared is not None and torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert (ap.ap_debug_get(ap.AP_DBG_LAST_FLAGS) >> 4 > 1) == shared
