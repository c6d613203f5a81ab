"""rms_norm and rms_norm_grad on matrices that are not aligned alike: one operand at
a time one value off the others' 16-byte alignment, or in rows of another stride,
for widths and row counts that would take each of the faster forms otherwise.
Bounds as in tests/test_rms_norm_gpu.py."""
import numpy as np
import pytest
import torch

from oracle import layers as L
from tests.layer_util import DTYPES, Out, assert_close, normal, rounded_bound

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(autouse=True)
def clean_error_word(gemm_mod):
    gemm_mod.check_device_error()
    yield
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0


def vector(n, dtype, seed, shift=0):
    v = 1 + 0.3 * torch.randn(n, generator=torch.Generator().manual_seed(seed))
    out = torch.full((n + shift + 8,), float("nan"), dtype=dtype, device="cuda")[shift:shift + n]
    out.copy_(v)
    return out


def placed(values, shift=0, pad=0):
    """A copy of a matrix in an Out: `shift` values off, rows `pad` longer."""
    m, n = values.shape
    out = Out(m, n, values.dtype, pad=pad, shift=shift)
    out.t.copy_(values)
    return out


WIDTHS = [(5, 64), (4000, 64), (33, 255), (3000, 255), (7, 500), (2500, 500), (6, 1001),
          (1700, 1001), (9, 5000)]
# Which matrix is placed differently, and how.
UNLIKE = [("H", 1, 0), ("H", 0, 3), ("dH", 5, 0), ("dH", 0, 1), ("dX", 1, 0), ("dX", 0, 4),
          ("dY", 2, 7)]


@pytest.mark.parametrize("shape", WIDTHS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("which,shift,pad", UNLIKE)
def test_grad(gemm_mod, shape, which, shift, pad):
    m, n = shape
    dtype = DTYPES["f16" if (m + pad) % 2 else "bf16"]
    at = {name: (shift, pad) if name == which else (0, 0) for name in ("dY", "H", "dH", "dX")}
    Y, H, B = (placed(normal(shape, dtype, n + i, std), *at[name])
               for i, (name, std) in enumerate((("dY", 1.0), ("H", 2.0), ("dH", 1.0))))
    W = vector(n, dtype, n)
    X = Out(m, n, dtype, *reversed(at["dX"]))
    h64, y64, d64, w64 = L.to64(H.t), L.to64(Y.t), L.to64(B.t), L.to64(W)
    rstd = torch.from_numpy(1 / np.sqrt((h64 * h64).mean(1) + EPS)).float().cuda()
    s64 = L.to64(rstd)
    D, D2 = Out(1, n, dtype), Out(1, n, dtype)
    gemm_mod.rms_norm_grad(Y.t, H.t, rstd, X.t, weight=W, dh=B.t, dweight=D.t[0])
    torch.cuda.synchronize()
    dx, dw = L.rms_norm_grad(y64, h64, s64, w64, d64)
    nrm, g = h64 * s64[:, None], np.abs(y64 * w64)
    terms = s64[:, None] * (g + np.abs(nrm) * (g * np.abs(nrm)).mean(1, keepdims=True)) \
        + np.abs(d64)
    bound = rounded_bound(dx, 2.0 ** -17 * terms, dtype)
    assert_close(L.to64(X.t), dx, bound, "dX")
    ew = rounded_bound(dw, (m + 20) * 2.0 ** -24 * np.abs(y64 * nrm).sum(0), dtype)
    assert_close(L.to64(D.t[0]), dw, ew, "dW")
    # The same with dX in place of dY, then of dH.
    for out, dh in ((Y, B.t), (B, B.t)):
        if out is B:
            Y.t.copy_(torch.from_numpy(y64))
        gemm_mod.rms_norm_grad(Y.t, H.t, rstd, out.t, weight=W, dh=dh, dweight=D2.t[0])
        torch.cuda.synchronize()
        assert_close(L.to64(out.t), dx, bound, "dX in place")
        assert_close(L.to64(D2.t[0]), dw, ew, "dW in place")
    for o in (X, D, D2, Y, H, B):
        o.check_guards()


@pytest.mark.parametrize("out8", [False, True], ids=["out16", "e4m3"])
@pytest.mark.parametrize("shape", WIDTHS + [(400, 2500), (200, 9000)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("which,shift,pad", [("R", 1, 0), ("R", 0, 3), ("X", 3, 0), ("H", 1, 0),
                                             ("Y", 1, 2), ("W", 1, 0)])
def test_norm(gemm_mod, shape, which, shift, pad, out8):
    m, n = shape
    dtype = DTYPES["bf16" if (m + pad) % 2 else "f16"]
    at = {name: (shift, pad) if name == which else (0, 0) for name in ("X", "R", "H", "Y")}
    X, R = placed(normal(shape, dtype, n), *at["X"]), placed(normal(shape, dtype, n + 1, 2.0),
                                                             *at["R"])
    W = vector(n, dtype, n, shift if which == "W" else 0)
    H = Out(m, n, dtype, *reversed(at["H"]))
    Y = Out(m, n, torch.float8_e4m3fn if out8 else dtype, *reversed(at["Y"]))
    rstd = torch.empty(m, device="cuda")
    scale = torch.empty(m, device="cuda") if out8 else None
    gemm_mod.rms_norm(X.t, Y.t, weight=W, residual=R.t, h=H.t, scale=scale, rstd=rstd, eps=EPS)
    torch.cuda.synchronize()
    y, _, s = L.rms_norm(L.to64(X.t), L.to64(W), L.to64(R.t), EPS)
    assert_close(L.to64(rstd), s, 2.0 ** -18 * s, "rstd")
    assert torch.equal(H.t, (X.t.float() + R.t.float()).to(dtype))
    if out8:
        q, qs = L.quantise_e4m3(y)
        assert_close(L.to64(scale), qs, 2.0 ** -17 * qs, "scale")
        step = qs[:, None] * 2.0 ** -10
        assert_close(L.to64(Y.t) * L.to64(scale)[:, None], y,
                     (2.0 ** -4 + 2.0 ** -16) * np.abs(y) + step * (1 + 2.0 ** -16), "Y")
        assert (L.to64(Y.t) == q).mean() >= 0.99
    else:
        bound = rounded_bound(y, 2.0 ** -17 * np.abs(y), dtype)
        assert_close(L.to64(Y.t), y, bound, "Y")
        gemm_mod.rms_norm(X.t, R.t, weight=W, residual=R.t, eps=EPS)  # Y in place of R
        assert_close(L.to64(R.t), y, bound, "Y in place")
    for o in (X, R, H, Y):
        o.check_guards()
