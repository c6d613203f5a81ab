"""GPU parity of rms_norm and rms_norm_grad against the float64 oracle.

Tolerances: the sum of squares has positive terms and is added in short chains,
so the statistic is within 2^-18 relative; y and dx carry that and a few fp32
roundings (2^-17 of their terms), then one rounding to 16 bits. The 8-bit values
are within one rounding of the e4m3 grid of y / scale (2^-4 relative, or half the
subnormal step 2^-10), and at least 99 % of them are the oracle's own: a value
changes sides only within 2^-17 of a boundary, and boundaries are 2^-4 apart.
"""
import numpy as np
import pytest
import torch

from oracle import layers as L
from tests.layer_util import DTYPES, Out, assert_close, normal, rounded_bound

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 4096), (3, 8), (5, 64), (33, 250), (7, 255), (130, 256), (9, 1000), (4, 1001),
          (300, 1024), (17, 2048), (20, 4096), (5, 5120), (3, 8192), (2, 8200), (2, 16384), (3, 7777),
          (2, 20001), (2, 40000), (2500, 128)]
EPS = 1e-5


@pytest.fixture(autouse=True)
def clean_error_word(gemm_mod):
    gemm_mod.check_device_error()
    yield
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0


def vector(n, dtype, seed):
    return (1 + 0.3 * torch.randn(n, generator=torch.Generator().manual_seed(seed))).to(
        dtype).cuda()


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("out8", [False, True], ids=["out16", "e4m3"])
def test_norm(gemm_mod, shape, dtype, out8):
    m, n = shape
    i = SHAPES.index(shape)
    pad = [0, 8, 1][i % 3]
    X = normal(shape, dtype, i, pad=pad)
    R = normal(shape, dtype, i + 1, 2.0, pad=pad) if i % 4 != 3 else None
    W = vector(n, dtype, i) if i % 5 != 4 else None
    H = Out(m, n, dtype, pad=pad, shift=pad % 2) if i % 2 == 0 else None
    Y = Out(m, n, torch.float8_e4m3fn if out8 else dtype, pad=pad)
    rstd = torch.empty(m, device="cuda")
    scale = torch.empty(m, device="cuda") if out8 else None
    gemm_mod.rms_norm(X, Y.t, weight=W, residual=R, h=H.t if H else None, scale=scale, rstd=rstd,
                      eps=EPS)
    torch.cuda.synchronize()
    y, h, s = L.rms_norm(L.to64(X), None if W is None else L.to64(W),
                         None if R is None else L.to64(R), EPS)
    assert_close(L.to64(rstd), s, 2.0 ** -18 * s, "rstd")
    if H:
        want = X.float() if R is None else X.float() + R.float()
        assert torch.equal(H.t, want.to(dtype))
        H.check_guards()
    if out8:
        q, qs = L.quantise_e4m3(y)
        assert_close(L.to64(scale), qs, 2.0 ** -17 * qs, "scale")
        got = L.to64(Y.t)
        step = qs[:, None] * 2.0 ** -10
        assert_close(got * L.to64(scale)[:, None], y,
                     (2.0 ** -4 + 2.0 ** -16) * np.abs(y) + step * (1 + 2.0 ** -16), "Y")
        assert (got == q).mean() >= 0.99
    else:
        assert_close(L.to64(Y.t), y, rounded_bound(y, 2.0 ** -17 * np.abs(y), dtype), "Y")
    Y.check_guards()


@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("out8", [False, True], ids=["out16", "e4m3"])
@pytest.mark.parametrize("shape", [(2600, 1000), (1601, 1031), (1000, 2047), (700, 2500), (500, 4095),
                                   (400, 5280), (250, 8191), (200, 10001), (160, 16384)],
                         ids=lambda s: "x".join(map(str, s)))
def test_norm_of_many_rows(gemm_mod, shape, out8, residual):
    """Rows enough for blocks that walk over several; X one value off a 16-byte
    boundary, 8-bit rows padded, 16-bit Y in place of X."""
    m, n = shape
    dtype = DTYPES["f16" if residual == out8 else "bf16"]
    buf = torch.full((m * n + 16,), float("nan"), device="cuda", dtype=dtype)
    X = torch.as_strided(buf, (m, n), (n, 1), 1)
    X.copy_(normal(shape, dtype, n))
    R, H = None, None
    if residual:  # aligned as X is
        R = torch.as_strided(torch.empty_like(buf), (m, n), (n, 1), 1)
        R.copy_(normal(shape, dtype, n + 1, 2.0))
        H = Out(m, n, dtype, pad=3)
    W = vector(n, dtype, n)
    x64, r64 = L.to64(X), L.to64(R) if residual else None
    want = X.float() + R.float() if residual else None
    Y = Out(m, n, torch.float8_e4m3fn, pad=-n % 16) if out8 else None
    rstd = torch.empty(m, device="cuda")
    scale = torch.empty(m, device="cuda") if out8 else None
    gemm_mod.rms_norm(X, Y.t if out8 else X, weight=W, residual=R, h=H.t if H else None,
                      scale=scale, rstd=rstd, eps=EPS)
    torch.cuda.synchronize()
    y, _, s = L.rms_norm(x64, L.to64(W), r64, EPS)
    assert_close(L.to64(rstd), s, 2.0 ** -18 * s, "rstd")
    if residual:
        assert torch.equal(H.t, want.to(dtype))
        H.check_guards()
    if out8:
        q, qs = L.quantise_e4m3(y)
        assert_close(L.to64(scale), qs, 2.0 ** -17 * qs, "scale")
        step = qs[:, None] * 2.0 ** -10
        assert_close(L.to64(Y.t) * L.to64(scale)[:, None], y,
                     (2.0 ** -4 + 2.0 ** -16) * np.abs(y) + step * (1 + 2.0 ** -16), "Y")
        assert (L.to64(Y.t) == q).mean() >= 0.99
        Y.check_guards()
    else:
        assert_close(L.to64(X), y, rounded_bound(y, 2.0 ** -17 * np.abs(y), dtype), "Y")
    assert torch.isnan(buf[0]) and torch.isnan(buf[m * n + 1:]).all()


@pytest.mark.parametrize("n", [1, 3, 7, 9, 13, 101, 1001, 2049, 2056, 4095, 6001, 7777, 16383])
def test_8_bit_rows_padded_for_the_product(gemm_mod, n):
    """Y in rows of whole 16-byte units, X in packed rows: the two are aligned
    differently in most rows. Every value, and nothing else, is written."""
    m = 19
    X, R = normal((m, n), torch.bfloat16, n), normal((m, n), torch.bfloat16, n + 1)
    W = vector(n, torch.bfloat16, n)
    Y = Out(m, n, torch.float8_e4m3fn, pad=-n % 16)
    scale = torch.empty(m, device="cuda")
    gemm_mod.rms_norm(X, Y.t, weight=W, residual=R, scale=scale, eps=EPS)
    torch.cuda.synchronize()
    y, _, _ = L.rms_norm(L.to64(X), L.to64(W), L.to64(R), EPS)
    q, qs = L.quantise_e4m3(y)
    step = qs[:, None] * 2.0 ** -10
    assert_close(L.to64(Y.t) * L.to64(scale)[:, None], y,
                 (2.0 ** -4 + 2.0 ** -16) * np.abs(y) + step * (1 + 2.0 ** -16), "Y")
    assert (L.to64(Y.t) == q).mean() >= 0.99
    Y.check_guards()


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_grad(gemm_mod, shape, dtype):
    m, n = shape
    i = SHAPES.index(shape)
    pad = [0, 8, 1][i % 3]
    H, dY = normal(shape, dtype, i, 2.0, pad=pad), normal(shape, dtype, i + 1, pad=pad)
    dH = normal(shape, dtype, i + 2, pad=pad) if i % 3 else None
    W = vector(n, dtype, i) if i % 5 != 4 else None
    h64 = L.to64(H)
    rstd = torch.from_numpy(1 / np.sqrt((h64 * h64).mean(1) + EPS)).float().cuda()
    dX, dW = Out(m, n, dtype, pad=pad), Out(1, n, dtype)
    gemm_mod.rms_norm_grad(dY, H, rstd, dX.t, weight=W, dh=dH, dweight=dW.t[0])
    torch.cuda.synchronize()
    y64, s64 = L.to64(dY), L.to64(rstd)
    w64 = None if W is None else L.to64(W)
    d64 = None if dH is None else L.to64(dH)
    dx, dw = L.rms_norm_grad(y64, h64, s64, w64, d64)
    nrm = h64 * s64[:, None]
    g = np.abs(y64 if W is None else y64 * w64)
    terms = s64[:, None] * (g + np.abs(nrm) * (g * np.abs(nrm)).mean(1, keepdims=True))
    if dH is not None:
        terms = terms + np.abs(d64)
    assert_close(L.to64(dX.t), dx, rounded_bound(dx, 2.0 ** -17 * terms, dtype), "dX")
    ew = (m + 20) * 2.0 ** -24 * np.abs(y64 * nrm).sum(0)
    assert_close(L.to64(dW.t[0]), dw, rounded_bound(dw, ew, dtype), "dW")
    dX.check_guards()
    dW.check_guards()


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("shape", [(6001, 64), (4864, 255), (2433, 500), (4864, 519), (305, 1001),
                                   (2600, 1000), (4864, 1024), (1521, 1500), (2432, 2047),
                                   (1530, 2055)], ids=lambda s: "x".join(map(str, s)))
def test_grad_of_several_rows_per_warp(gemm_mod, shape, dtype):
    """Rows enough that a warp walks over several, with rings shorter and longer
    than its rows; dX in place of dY, as dY's and dh's rows are walked ahead."""
    m, n = shape
    W, D = vector(n, dtype, n), Out(1, n, dtype)
    H, dH = normal(shape, dtype, m, 2.0), normal(shape, dtype, m + 1)
    X = Out(m, n, dtype)
    X.t.copy_(normal(shape, dtype, m + 2))
    y64, h64, d64, w64 = L.to64(X.t), L.to64(H), L.to64(dH), L.to64(W)
    rstd = torch.from_numpy(1 / np.sqrt((h64 * h64).mean(1) + EPS)).float().cuda()
    s64 = L.to64(rstd)
    gemm_mod.rms_norm_grad(X.t, H, rstd, X.t, weight=W, dh=dH, dweight=D.t[0])
    torch.cuda.synchronize()
    dx, dw = L.rms_norm_grad(y64, h64, s64, w64, d64)
    nrm, g = h64 * s64[:, None], np.abs(y64 * w64)
    terms = s64[:, None] * (g + np.abs(nrm) * (g * np.abs(nrm)).mean(1, keepdims=True)) + np.abs(d64)
    assert_close(L.to64(X.t), dx, rounded_bound(dx, 2.0 ** -17 * terms, dtype), "dX")
    ew = (m + 20) * 2.0 ** -24 * np.abs(y64 * nrm).sum(0)
    assert_close(L.to64(D.t[0]), dw, rounded_bound(dw, ew, dtype), "dW")
    X.check_guards()
    D.check_guards()


def test_in_place(gemm_mod):
    for n in (1000, 1001, 20000):
        X, R = normal((6, n), torch.bfloat16, 1), normal((6, n), torch.bfloat16, 2)
        W = vector(n, torch.bfloat16, 3)
        H, Y = torch.empty_like(X), torch.empty_like(X)
        gemm_mod.rms_norm(X, Y, weight=W, residual=R, h=H)
        x, r = X.clone(), R.clone()
        gemm_mod.rms_norm(x, x, weight=W, residual=r, h=r)
        assert torch.equal(x, Y) and torch.equal(r, H)
        dY, dH = normal((6, n), torch.bfloat16, 4), normal((6, n), torch.bfloat16, 5)
        rstd = torch.rsqrt(H.float().square().mean(1))
        dX = torch.empty_like(X)
        gemm_mod.rms_norm_grad(dY, H, rstd, dX, weight=W, dh=dH)
        a, b = dY.clone(), dH.clone()
        gemm_mod.rms_norm_grad(a, H, rstd, a, weight=W, dh=dH)
        gemm_mod.rms_norm_grad(dY, H, rstd, b, weight=W, dh=b)
        torch.cuda.synchronize()
        assert torch.equal(a, dX) and torch.equal(b, dX)


@pytest.mark.parametrize("n", [64, 4096, 4097, 40000])
def test_special_rows(gemm_mod, n):
    """Rows of zeros, with a NaN, with an infinity: no other row is touched."""
    X = normal((6, n), torch.bfloat16, 1)
    clean = X.clone()
    X[1] = 0
    X[2, n // 2] = float("nan")
    X[4, n - 1] = float("inf")
    Y, ref = torch.empty_like(X), torch.empty_like(X)
    gemm_mod.rms_norm(X, Y)
    gemm_mod.rms_norm(clean, ref)
    assert not Y[1].any() and bool(Y[2].isnan().all()) and bool(Y[4, n - 1].isnan())
    for r in (0, 3, 5):
        assert torch.equal(Y[r], ref[r])
    Q = torch.empty(6, n, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(6, device="cuda")
    gemm_mod.rms_norm(X, Q, scale=s)
    assert s[1].item() == 0 and not Q[1].float().any()
    assert not s[2].isfinite() and not s[4].isfinite()
    assert bool(s[[0, 3, 5]].isfinite().all())
    gemm_mod.rms_norm(X, Y, eps=0.0)
    assert bool(Y[1].isnan().all())  # 0 / 0, as the formula says


def test_tiny_rows_count_as_zeros_in_8_bits(gemm_mod):
    X = torch.ones(2, 64, dtype=torch.bfloat16, device="cuda")
    W = torch.full((64,), 1e-33, dtype=torch.bfloat16, device="cuda")
    Q = torch.empty(2, 64, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(2, device="cuda")
    gemm_mod.rms_norm(X, Q, weight=W, scale=s)
    assert not s.any() and not Q.float().any()


def test_no_rows(gemm_mod):
    z = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    gemm_mod.rms_norm(z, z)
    dw = torch.ones(32, dtype=torch.bfloat16, device="cuda")
    gemm_mod.rms_norm_grad(z, z, torch.empty(0, device="cuda"), z, dweight=dw)
    assert not dw.any()


def test_same_bits_on_another_stream(gemm_mod):
    H, dY = normal((700, 1024), torch.float16, 1), normal((700, 1024), torch.float16, 2)
    rstd = torch.rsqrt(H.float().square().mean(1))
    out = []
    for s in (None, torch.cuda.Stream()):
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        dX, dW = torch.empty_like(H), torch.empty(1024, dtype=torch.float16, device="cuda")
        Y = torch.empty_like(H)
        torch.cuda.synchronize()
        gemm_mod.rms_norm(H, Y, stream=s)
        gemm_mod.rms_norm_grad(dY, H, rstd, dX, dweight=dW, stream=s)
        torch.cuda.synchronize()
        out.append((Y, dX, dW))
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_more_than_2_to_31_elements(gemm_mod):
    """Row offsets pass 32 bits: the last row of a matrix with a wide row stride."""
    rows, n, ld = 3, 256, 1 << 30
    buf = torch.empty((rows - 1) * ld + n, dtype=torch.bfloat16, device="cuda")
    X = buf.as_strided((rows, n), (ld, 1))
    src = normal((rows, n), torch.bfloat16, 1)
    X.copy_(src)
    Y, ref = torch.empty_like(src), torch.empty_like(src)
    gemm_mod.rms_norm(X, Y)
    gemm_mod.rms_norm(src, ref)
    assert torch.equal(Y, ref)
    gemm_mod.rms_norm(src, X)
    assert torch.equal(X, ref)


def test_refusals_of_the_binding(gemm_mod):
    X = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    Y = torch.zeros_like(X)
    s = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        gemm_mod.rms_norm(X.float(), Y)
    with pytest.raises(TypeError):
        gemm_mod.rms_norm(X, Y.half())
    with pytest.raises(ValueError):
        gemm_mod.rms_norm(X, Y, scale=s)
    with pytest.raises(ValueError):
        gemm_mod.rms_norm(X, Y.to(torch.float8_e4m3fn))
    with pytest.raises(ValueError):
        gemm_mod.rms_norm(X, Y, rstd=s[:3])
    with pytest.raises(ValueError):
        gemm_mod.rms_norm(X.cpu(), Y)
    with pytest.raises(ValueError):
        gemm_mod.rms_norm(X, Y, weight=X[0, ::2])
    with pytest.raises(gemm_mod.GemmError) as e:
        gemm_mod.rms_norm(X, Y, eps=-1.0)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        gemm_mod.rms_norm_grad(X, Y[:2], s, X)
