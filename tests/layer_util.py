"""Shared helpers of the linear-layer operators' tests: operands whose row
padding is poisoned, outputs with guard values around every row, and the error
bounds of one fp32 product."""
from __future__ import annotations

import numpy as np
import torch

from oracle import layers as L

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# Unit roundoff (half a unit in the last place, relative) and the absolute half
# step of the subnormal range of the output formats.
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
GUARD = -96.0  # exactly representable in every format used


def normal(shape, dtype, seed, std=1.0, pad=0, unit=1, poison=float("nan")):
    """A CUDA matrix of normal values, rows padded to a multiple of `unit` plus
    `pad` elements; the padding holds `poison`."""
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(shape, generator=g) * std).to(dtype)
    rows, cols = shape
    ld = -(-cols // unit) * unit + pad
    buf = torch.full((max(rows, 1), max(ld, 1)), poison, dtype=torch.float32).to(dtype)
    buf[:rows, :cols] = v
    return buf.cuda()[:rows, :cols]


def e4m3(rows, cols, seed, std=1.0):
    """Normal values as e4m3 with a scale per row; row padding holds NaN."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, cols, generator=g) * std
    scale = v.abs().amax(1) / 448 if cols else torch.ones(rows)
    ld = -(-cols // 16) * 16 + 16
    buf = torch.full((max(rows, 1), ld), 0x7f, dtype=torch.uint8)
    buf[:rows, :cols] = (v / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(
        torch.uint8)
    return buf.cuda().view(torch.float8_e4m3fn)[:rows, :cols], scale.cuda()


class Out:
    """An output matrix inside a buffer of guard values: `pad` extra elements per
    row, `shift` elements off the buffer's 256-byte alignment."""

    def __init__(self, rows, cols, dtype, pad=0, shift=0):
        ld = cols + pad
        self.flat = torch.full((64 + shift + rows * ld + 64,), GUARD, device="cuda").to(dtype)
        self.start, self.rows, self.cols, self.ld = 64 + shift, rows, cols, ld
        self.t = self.flat[self.start:self.start + rows * ld].view(rows, ld)[:, :cols]

    def check_guards(self):
        f = self.flat.to(torch.float32).cpu()
        f[self.start:self.start + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] \
            = GUARD
        assert bool((f == GUARD).all()), "a kernel wrote outside its output"


def product_bound(A, B, alpha=1.0, scale_a=None, scale_b=None):
    """Worst-case error of an fp32 sum of K exact products: K additions, each off
    by at most 2^-23 of the running sum of magnitudes (the tensor cores truncate),
    and four roundings of the scaling."""
    s = abs(alpha) * (np.abs(A) @ np.abs(B))
    if scale_a is not None:
        s = s * scale_a[:, None]
    if scale_b is not None:
        s = s * scale_b[None, :]
    return (A.shape[1] + 4) * 2.0 ** -23 * s


def act_error(z, name):
    """Bound of the activations' own evaluation error: 2^-16 of the value (the
    exponential's argument carries a relative 2^-24, times |x| < 90) plus 2^-22
    |z| for cancellation."""
    if name in (None, "none", "relu"):
        return np.zeros_like(z)
    return 2.0 ** -16 * np.abs(L.act(z, name)) + 2.0 ** -22 * np.abs(z)


def assert_close(got, ref, bound, what):
    got = np.asarray(got, dtype=np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    err = np.where(np.isnan(ref), 0.0, np.abs(got - ref))
    bad = err > np.where(np.isnan(ref), np.inf, bound)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, err / np.maximum(bound, 1e-300), 0)),
                              err.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.size} out of bounds; worst at "
                             f"{at}: got {got[at]!r}, exact {ref[at]!r}, bound {bound[at]:.3e}")


def rounded_bound(ref, bound, dtype):
    """The bound of an fp32 result within `bound` of `ref` after one rounding."""
    u = UNIT[dtype]
    return bound * (1 + u) + u * np.abs(ref) + TINY[dtype]
