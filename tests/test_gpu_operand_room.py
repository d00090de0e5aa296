"""Shared memory of the 8-bit products' forms: the matrix instructions' operands of a CTA end at least 20 KiB before the
CTA's own end, so that they lie below 208 KiB of an SM's 228 wherever the CTA starts, beside whatever other CTAs."""

import pytest
import torch

from gpu_util import device, lib, reset_debug
from test_gpu_fp8 import check_matmul, done, operand, randn

pytestmark = pytest.mark.gpu

ROOM = (228 - 208) * 1024
BOX = 128 * 128  # bytes of 128 rows of an operand in a stage


@pytest.fixture
def ap():
    device()
    ap = lib()
    reset_debug(ap)
    yield ap
    reset_debug(ap)


def room(ap, stage_bytes):
    """Bytes of a CTA behind its ring, whose first 1024-byte boundary may be 1023 bytes in."""
    return ap.ap_debug_get(ap.AP_DBG_LAST_SMEM) - 1024 - ap.ap_debug_get(ap.AP_DBG_LAST_STAGES) * stage_bytes


# rows of a and, for one CTA, of its operands in a stage: 128 of the weight and 16 or 32; 128 and 128; a pair's halves
@pytest.mark.parametrize("m,n,k,stage", [(1, 8192, 2048, BOX + 16 * 128), (16, 300, 640, BOX + 16 * 128), (17, 8192, 1024, BOX + 32 * 128),
                                         (32, 300, 640, BOX + 32 * 128), (100, 300, 640, 2 * BOX), (1024, 2560, 512, 2 * BOX)])
def test_plain_product(ap, m, n, k, stage):
    check_matmul(ap, m, n, k, 128, torch.float32)
    assert room(ap, stage) >= ROOM


@pytest.mark.parametrize("m,stage", [(1, 2 * BOX + 16 * 128), (32, 2 * BOX + 32 * 128), (100, 3 * BOX), (1100, 2 * BOX)])
def test_gated_product(ap, m, stage):
    n, k = 1200, 512
    a, sa = operand(m, k, 1, 1)
    g, sg = operand(n, k, 128, 2)
    y = torch.empty(m, n, device="cuda")
    ap.ap_gated_matmul_fp8(a, sa, g, sg, g, sg, 0, y=y)
    done(ap)
    assert room(ap, stage) >= ROOM


def test_few_rows_beside_the_library_s_other_kernels(ap):
    """Products of few rows behind the quantiser, norms and products with 4-bit weights, whose CTAs may share an SM with
    theirs, on three streams at once: each is what it is alone."""
    cases = []
    for m in (1, 8, 32):
        x = randn(m, 4096, seed=m).bfloat16()
        a, sa = operand(m, 4096, 1, m)
        w, sw = operand(4096, 4096, 128, 50 + m)
        c = torch.empty(m, 4096, device="cuda")
        ap.ap_matmul_fp8(a, sa, w, sw, c)
        done(ap)
        cases.append((x, a, sa, w, sw, c))
    big, weight = randn(1024, 4096, seed=9).bfloat16(), torch.ones(4096, device="cuda")
    codes = torch.randint(0, 256, (4096, 2048), dtype=torch.uint8, device="cuda")
    scales = torch.ones(4096, 32, dtype=torch.bfloat16, device="cuda")
    streams, made = [torch.cuda.Stream() for _ in range(3)], []
    torch.cuda.synchronize()
    for i in range(30):
        with torch.cuda.stream(streams[i % 3]):
            for x, a, sa, w, sw, c in cases:
                q, s = torch.empty_like(big, dtype=torch.uint8), torch.empty(1024, 32, device="cuda")
                got = torch.empty_like(c)
                if i % 2:
                    ap.ap_quantize(big, 1, q, s)
                else:
                    ap.ap_rms_norm(big, weight, 1e-6, q=q, q_scales=s)
                ap.ap_matmul_fp8(a, sa, w, sw, got)
                ap.ap_matmul_w4(x, codes, scales, torch.empty_like(c))
                made.append((got, c))
    done(ap)
    assert all(torch.equal(a, b) for a, b in made)
