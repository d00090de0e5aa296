"""Plain forms of the 8-bit block-scaled operators in 64 bits, and the error
bounds their tests use. Nothing here calls the library.

Bounds. u is half the spacing at 1 of the type a result is rounded to, U = 2^-24
that of float32. A sum of N terms taken in d sequential additions is off by at
most d * U * sum(|terms|); the kernels add at most 80 terms in sequence per
thread before their trees (a row of 70000 over 1024 threads is 72)."""

import numpy as np
import torch

U = 2.0 ** -24
DEPTH = 96  # sequential additions of a row's sum, trees and the few roundings around it
MIN_SCALE = 2.0 ** -126
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_SPACING = {t: torch.finfo(t).eps / 2 for t in TYPES.values()}
SMALLEST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def blocks(n):
    return -(-n // 128)


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def rounding(v, dtype):
    """How far |v| may be off by its one rounding to dtype."""
    return HALF_SPACING[dtype] * np.abs(v) + SMALLEST[dtype] / 2


def amax_blocks(v, tile):
    """amax of row blocks (tile 1) or tiles (128) of a 64-bit matrix, with NaN where a block has one."""
    rows, cols = v.shape
    w = np.zeros((-(-rows // tile) * tile, blocks(cols) * 128))
    w[:rows, :cols] = np.abs(v)
    return w.reshape(-1, tile, blocks(cols), 128).max(axis=(1, 3))


def spread_scales(s, rows, cols, tile):
    return np.repeat(np.repeat(s, tile, 0)[:rows], 128, 1)[:, :cols]


def check_codes(q, s, v, tile, rel, what):
    """q and s hold the 64-bit matrix v, which the kernel knew to a relative `rel`."""
    rows, cols = v.shape
    q, s = f64(q), f64(s)
    with np.errstate(invalid="ignore"):
        want = np.maximum(amax_blocks(v, tile) / 448, MIN_SCALE)
    finite = np.isfinite(want)
    assert np.array_equal(np.isnan(s), np.isnan(want)) and np.array_equal(np.isinf(s), np.isinf(want)), what
    assert np.all(np.abs(s[finite] - want[finite]) <= (rel + 4 * U) * want[finite]), f"{what}: scales"
    at = spread_scales(s, rows, cols, tile)
    ok = np.isfinite(at)
    assert np.array_equal(np.isnan(q[~ok]), ~np.isfinite(v[~ok]) | np.isnan(at[~ok])), f"{what}: not finite"
    assert np.all(q[~ok & np.isfinite(v) & np.isinf(at)] == 0), f"{what}: beside an infinity"
    x = v[ok] / at[ok]
    # e4m3: three mantissa bits (half spacing 2^-4 of the value), subnormals of 2^-9
    near = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10) * (1 + 8 * U) + (rel + 8 * U) * np.abs(x)
    bad = np.abs(q[ok] - x) > near
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off, worst {np.max(np.abs(q[ok] - x) / near)} of the bound"


def codes_32(v, tile):
    """Codes and scales by the definition's own 32-bit operations (torch on the CPU), for a float32 matrix."""
    rows, cols = v.shape
    s = torch.from_numpy(amax_blocks(v.double().numpy(), tile)).float() / 448
    s = torch.where(s < MIN_SCALE, torch.full_like(s, MIN_SCALE), s)
    inv = 1 / s
    at = inv.repeat_interleave(tile, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return (v * at).to(torch.float8_e4m3fn), s


def norm(x, residual, weight, eps):
    h = x if residual is None else x + residual
    r = 1 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h, r, h * r[:, None] * weight


def norm_backward(dy, h, weight, r, dresidual):
    n, g = h * r[:, None], dy * weight
    dx = r[:, None] * (g - n * np.mean(g * n, axis=1)[:, None])
    near = r[:, None] * (np.abs(g) + np.abs(n) * np.mean(np.abs(g * n), axis=1)[:, None]) * DEPTH * U
    if dresidual is not None:
        dx = dx + dresidual
        near = near + 2 * U * np.abs(dresidual)
    return dx, near, (dy * n).sum(0), np.abs(dy * n).sum(0)


def matmul(a, sa, b, sb, tile):
    """c and the sum of its terms' magnitudes, in 64 bits."""
    a = a * np.repeat(sa, 128, 1)[:, : a.shape[1]]
    b = b * spread_scales(sb, *b.shape, tile)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def matmul_bound(c, terms, k, dtype):
    """The products are exact. A block's 128 products are added in the tensor core: at worst each of four
    instructions truncates 32 aligned terms, 64 U of the terms in all; then one scaled addition a block
    (2 U for the two scales)."""
    return rounding(c, dtype) + (blocks(k) + 80) * U * terms


class Strided:
    """A rows x cols device matrix inside a larger buffer: leading dimension ld, starting `shift` elements past a
    256-byte boundary, everything around it filled with a pattern that intact() looks for."""

    def __init__(self, rows, cols, dtype, ld=None, shift=0, fill=None, dev="cuda:0"):
        self.rows, self.cols, self.ld, self.lo = rows, cols, cols if ld is None else ld, 256 + shift
        size = torch.empty(0, dtype=dtype).element_size()
        n = self.lo + rows * self.ld + 256
        self.bytes = torch.full((n * size,), 0xA5, dtype=torch.uint8, device=dev)
        flat = self.bytes.view(dtype)
        self.view = flat.as_strided((rows, cols), (self.ld, 1), self.lo)
        if fill is not None:
            self.view.copy_(fill)
        inside = torch.zeros(n, dtype=torch.bool, device=dev)
        inside.as_strided((rows, cols), (self.ld, 1), self.lo).fill_(True)
        self.outside = ~inside.repeat_interleave(size)

    def intact(self):
        return bool((self.bytes[self.outside] == 0xA5).all().item())
