"""GPU parity of layer_norm and layer_norm_grad against the float64 oracle.

Tolerances. A sum of n terms is added in chains of fewer than 64 additions (a
thread's values, its warp, the block's warps), so it is within 2^-18 of the sum of
magnitudes. The mean carries that of mean |h|. h - mean carries the mean's error and
the roundings of h and of the difference. The sum of its squares is stationary in
the mean's error, which adds its square only; the roundings of h enter to first
order. y adds a few fp32 roundings of its terms, then one to 16 bits. The gradient's
terms are sums as above (2^-17 of their magnitudes); dw and db are chains over rows.
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
# Rows enough for blocks and warps that walk over several, with rings shorter and
# longer than that.
MANY = [(6001, 64), (4864, 255), (2433, 500), (2600, 1000), (1601, 1031), (1521, 1500),
        (1000, 2047), (1530, 2055), (700, 2500), (500, 4095), (400, 5280), (250, 8191),
        (200, 10001), (160, 16384)]
EPS = 1e-5


@pytest.fixture(autouse=True)
def clean_error_word(gemm_mod):
    gemm_mod.check_device_error()
    yield
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0


def vector(n, dtype, seed, mean=1.0):
    g = torch.Generator().manual_seed(seed)
    return (mean + 0.3 * torch.randn(n, generator=g)).to(dtype).cuda()


def placed(values, shift=0, pad=0):
    """A copy of a matrix in an Out: `shift` values off, rows `pad` longer."""
    out = Out(*values.shape, values.dtype, pad=pad, shift=shift)
    out.t.copy_(values)
    return out


def opt64(t):
    return None if t is None else L.to64(t)


def check_forward(x64, r64, w64, b64, eps, dtype, Y, mean, rstd):
    y, h, m, s = L.layer_norm(x64, w64, b64, r64, eps)
    n = h.shape[1]
    c, w = h - m[:, None], 1.0 if w64 is None else np.abs(w64)
    dm = 2.0 ** -18 * np.abs(h).mean(1)
    ec = dm[:, None] + 2.0 ** -23 * (np.abs(h) + np.abs(c))
    rel = 2.0 ** -17 + 2.0 ** -23 * (np.abs(c) * np.abs(h)).sum(1) * s * s / n + (dm * s) ** 2
    if mean is not None:
        assert_close(L.to64(mean), m, dm, "mean")
        assert_close(L.to64(rstd), s, rel * s, "rstd")
    term = np.abs(c) * s[:, None] * w
    ey = w * s[:, None] * ec + (1.01 * rel[:, None] + 2.0 ** -22) * term
    if b64 is not None:
        ey = ey + 2.0 ** -22 * np.abs(b64)
    assert_close(L.to64(Y), y, rounded_bound(y, ey, dtype), "Y")


def check_grad(y64, h64, m64, s64, w64, d64, dtype, dX, dW, db):
    rows = len(y64)
    dx, dw, b = L.layer_norm_grad(y64, h64, m64, s64, w64, d64)
    nrm = np.abs((h64 - m64[:, None]) * s64[:, None])
    g = np.abs(y64 if w64 is None else y64 * w64)
    terms = s64[:, None] * (g + g.mean(1, keepdims=True) + nrm * (g * nrm).mean(1, keepdims=True))
    if d64 is not None:
        terms = terms + np.abs(d64)
    assert_close(L.to64(dX), dx, rounded_bound(dx, 2.0 ** -17 * terms, dtype), "dX")
    for got, ref, parts, what in ((dW, dw, np.abs(y64) * nrm, "dW"), (db, b, np.abs(y64), "db")):
        if got is not None:
            e = (rows + 20) * 2.0 ** -24 * parts.sum(0)
            assert_close(L.to64(got), ref, rounded_bound(ref, e, dtype), what)


def statistics(H, eps=EPS):
    """mean and rstd as a forward call leaves them, in fp32."""
    h = L.to64(H)
    m = h.mean(1)
    s = 1 / np.sqrt(((h - m[:, None]) ** 2).mean(1) + eps)
    return torch.from_numpy(m).float().cuda(), torch.from_numpy(s).float().cuda()


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norm(gemm_mod, shape, dtype):
    m, n = shape
    i = SHAPES.index(shape)
    pad = [0, 8, 1][i % 3]
    X = normal(shape, dtype, i, pad=pad)
    R = normal(shape, dtype, i + 1, 2.0, pad=pad) if i % 4 != 3 else None
    W = vector(n, dtype, i) if i % 5 != 4 else None
    B = vector(n, dtype, i + 9, 0.0) if i % 5 != 3 else None
    H = Out(m, n, dtype, pad=pad, shift=pad % 2) if i % 2 == 0 else None
    Y = Out(m, n, dtype, pad=pad)
    mean, rstd = (torch.empty(m, device="cuda") for _ in range(2))
    gemm_mod.layer_norm(X, Y.t, weight=W, bias=B, residual=R, h=H.t if H else None, mean=mean,
                        rstd=rstd, eps=EPS)
    torch.cuda.synchronize()
    check_forward(L.to64(X), opt64(R), opt64(W), opt64(B), EPS, dtype, Y.t, mean, rstd)
    if H:
        want = X.float() if R is None else X.float() + R.float()
        assert torch.equal(H.t, want.to(dtype))
        H.check_guards()
    Y.check_guards()
    # Without the statistics, and in place of X: the same bits.
    Z = placed(X, 0, pad)
    gemm_mod.layer_norm(Z.t, Z.t, weight=W, bias=B, residual=R, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(Z.t, Y.t)
    Z.check_guards()


@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("shape", MANY, ids=lambda s: "x".join(map(str, s)))
def test_norm_of_many_rows(gemm_mod, shape, residual):
    """X one value off a 16-byte boundary, Y in place of X."""
    m, n = shape
    dtype = DTYPES["f16" if residual == bool(n % 2) else "bf16"]
    buf = torch.full((m * n + 16,), float("nan"), device="cuda", dtype=dtype)
    X = torch.as_strided(buf, (m, n), (n, 1), 1)
    X.copy_(normal(shape, dtype, n))
    R, H = None, None
    if residual:  # aligned as X is
        R = torch.as_strided(torch.empty_like(buf), (m, n), (n, 1), 1)
        R.copy_(normal(shape, dtype, n + 1, 2.0))
        H = Out(m, n, dtype, pad=3)
    W, B = vector(n, dtype, n), vector(n, dtype, n + 5, 0.0)
    x64, want = L.to64(X), X.float() + R.float() if residual else None
    mean, rstd = (torch.empty(m, device="cuda") for _ in range(2))
    gemm_mod.layer_norm(X, X, weight=W, bias=B, residual=R, h=H.t if H else None, mean=mean,
                        rstd=rstd, eps=EPS)
    torch.cuda.synchronize()
    check_forward(x64, opt64(R), L.to64(W), L.to64(B), EPS, dtype, X, mean, rstd)
    if residual:
        assert torch.equal(H.t, want.to(dtype))
        H.check_guards()
    assert torch.isnan(buf[0]) and torch.isnan(buf[m * n + 1:]).all()


@pytest.mark.parametrize("shape", [(5, 64), (4000, 64), (33, 255), (7, 500), (6, 1001), (1700, 1001),
                                   (9, 5000), (400, 2500), (200, 9000)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("which,shift,pad", [("R", 1, 0), ("R", 0, 3), ("X", 3, 0), ("H", 1, 0),
                                             ("Y", 1, 2), ("W", 1, 0), ("B", 3, 0)])
def test_norm_of_matrices_not_aligned_alike(gemm_mod, shape, which, shift, pad):
    m, n = shape
    dtype = DTYPES["bf16" if (m + pad) % 2 else "f16"]
    at = {k: (shift, pad) if k == which else (0, 0) for k in "XRHYWB"}
    X = placed(normal(shape, dtype, n), *at["X"])
    R = placed(normal(shape, dtype, n + 1, 2.0), *at["R"])
    W = placed(vector(n, dtype, n).view(1, n), at["W"][0])
    B = placed(vector(n, dtype, n + 1, 0.0).view(1, n), at["B"][0])
    H, Y = (Out(m, n, dtype, *reversed(at[k])) for k in "HY")
    mean, rstd = (torch.empty(m, device="cuda") for _ in range(2))
    gemm_mod.layer_norm(X.t, Y.t, weight=W.t[0], bias=B.t[0], residual=R.t, h=H.t, mean=mean,
                        rstd=rstd, eps=EPS)
    torch.cuda.synchronize()
    check_forward(L.to64(X.t), L.to64(R.t), L.to64(W.t[0]), L.to64(B.t[0]), EPS, dtype, Y.t, mean,
                  rstd)
    assert torch.equal(H.t, (X.t.float() + R.t.float()).to(dtype))
    for o in (X, R, W, B, H, Y):
        o.check_guards()


@pytest.mark.parametrize("shape", [(3, 64), (2, 4097), (700, 2500), (2, 40000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_large_mean(gemm_mod, shape):
    """A mean of 200 standard deviations: the squares are summed about the mean."""
    X = (normal(shape, torch.float16, 3, 0.25).float() + 50).half()
    Y = Out(*shape, torch.float16)
    mean, rstd = (torch.empty(shape[0], device="cuda") for _ in range(2))
    gemm_mod.layer_norm(X, Y.t, mean=mean, rstd=rstd, eps=0.0)
    torch.cuda.synchronize()
    check_forward(L.to64(X), None, None, None, 0.0, torch.float16, Y.t, mean, rstd)
    want = 1 / np.sqrt(L.to64(X).var(1))
    assert (np.abs(L.to64(rstd) / want - 1) < 1e-4).all()


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES + MANY, ids=lambda s: "x".join(map(str, s)))
def test_grad(gemm_mod, shape, dtype):
    m, n = shape
    i = (SHAPES + MANY).index(shape)
    pad = [0, 8, 1][i % 3]
    H, dY = normal(shape, dtype, i, 2.0, pad=pad), normal(shape, dtype, i + 1, pad=pad)
    H += 1
    dH = normal(shape, dtype, i + 2, pad=pad) if i % 3 else None
    W = vector(n, dtype, i) if i % 5 != 4 else None
    mean, rstd = statistics(H)
    dX, dW, db = Out(m, n, dtype, pad=pad), Out(1, n, dtype), Out(1, n, dtype)
    gemm_mod.layer_norm_grad(dY, H, mean, rstd, dX.t, weight=W, dh=dH, dweight=dW.t[0],
                             dbias=db.t[0])
    torch.cuda.synchronize()
    args = (L.to64(dY), L.to64(H), L.to64(mean), L.to64(rstd), opt64(W), opt64(dH), dtype)
    check_grad(*args, dX.t, dW.t[0], db.t[0])
    # Each parameter's gradient alone, or none, and dX in place of dY: the same bits.
    only_w, only_b, place = Out(1, n, dtype), Out(1, n, dtype), placed(dY, 0, pad)
    other = torch.empty_like(dX.t)
    gemm_mod.layer_norm_grad(dY, H, mean, rstd, other, weight=W, dh=dH, dweight=only_w.t[0])
    assert torch.equal(other, dX.t) or pad  # (rows placed otherwise go another way)
    gemm_mod.layer_norm_grad(dY, H, mean, rstd, other, weight=W, dh=dH, dbias=only_b.t[0])
    gemm_mod.layer_norm_grad(place.t, H, mean, rstd, place.t, weight=W, dh=dH)
    torch.cuda.synchronize()
    assert torch.equal(place.t, dX.t)
    check_grad(*args, other, only_w.t[0], only_b.t[0])
    for o in (dX, dW, db, only_w, only_b, place):
        o.check_guards()


@pytest.mark.parametrize("shape", [(5, 64), (4000, 64), (3000, 255), (7, 500), (2500, 500), (6, 1001),
                                   (1700, 1001), (9, 5000)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("which,shift,pad", [("H", 1, 0), ("H", 0, 3), ("dH", 5, 0), ("dH", 0, 1),
                                             ("dX", 1, 0), ("dX", 0, 4), ("dY", 2, 7)])
def test_grad_of_matrices_not_aligned_alike(gemm_mod, shape, which, shift, pad):
    m, n = shape
    dtype = DTYPES["f16" if (m + pad) % 2 else "bf16"]
    at = {name: (shift, pad) if name == which else (0, 0) for name in ("dY", "H", "dH", "dX")}
    Y, H, B = (placed(normal(shape, dtype, n + i, std), *at[name])
               for i, (name, std) in enumerate((("dY", 1.0), ("H", 2.0), ("dH", 1.0))))
    W, X = vector(n, dtype, n), Out(m, n, dtype, *reversed(at["dX"]))
    mean, rstd = statistics(H.t)
    dW, db = Out(1, n, dtype), Out(1, n, dtype)
    args = (L.to64(Y.t), L.to64(H.t), L.to64(mean), L.to64(rstd), L.to64(W), L.to64(B.t), dtype)
    gemm_mod.layer_norm_grad(Y.t, H.t, mean, rstd, X.t, weight=W, dh=B.t, dweight=dW.t[0],
                             dbias=db.t[0])
    torch.cuda.synchronize()
    check_grad(*args, X.t, dW.t[0], db.t[0])
    gemm_mod.layer_norm_grad(Y.t, H.t, mean, rstd, B.t, weight=W, dh=B.t)  # in place of dH
    torch.cuda.synchronize()
    check_grad(*args, B.t, None, None)
    for o in (X, dW, db, Y, H, B):
        o.check_guards()


def test_in_place(gemm_mod):
    for n in (1000, 1001, 20000):
        X, R = normal((6, n), torch.bfloat16, 1), normal((6, n), torch.bfloat16, 2)
        H, Y = torch.empty_like(X), torch.empty_like(X)
        gemm_mod.layer_norm(X, Y, residual=R, h=H)
        x, r = X.clone(), R.clone()
        gemm_mod.layer_norm(x, x, residual=r, h=r)
        assert torch.equal(x, Y) and torch.equal(r, H)
        x, r = X.clone(), R.clone()
        gemm_mod.layer_norm(x, r, residual=r, h=x)
        assert torch.equal(r, Y) and torch.equal(x, H)


@pytest.mark.parametrize("n", [64, 4096, 4097, 40000])
def test_special_rows(gemm_mod, n):
    """Rows of equal values, with a NaN, with an infinity: no other row is touched."""
    X = normal((6, n), torch.bfloat16, 1)
    clean = X.clone()
    X[1] = 3
    X[2, n // 2] = float("nan")
    X[4, n - 1] = float("inf")
    Y, ref = torch.empty_like(X), torch.empty_like(X)
    gemm_mod.layer_norm(X, Y)
    gemm_mod.layer_norm(clean, ref)
    assert bool((Y[1].abs() < 1e-3).all()) and bool(Y[2].isnan().all()) and bool(Y[4].isnan().all())
    for r in (0, 3, 5):
        assert torch.equal(Y[r], ref[r])
    X.fill_(2.0)  # a power of two times 64 ... 4096 sums exactly
    if n in (64, 4096):
        gemm_mod.layer_norm(X, Y, eps=0.0)
        assert bool(Y.isnan().all())  # 0 / 0, as the formula says


def test_no_rows(gemm_mod):
    z, e = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), torch.empty(0, device="cuda")
    gemm_mod.layer_norm(z, z)
    dw, db = (torch.ones(32, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gemm_mod.layer_norm_grad(z, z, e, e, z, dweight=dw, dbias=db)
    assert not dw.any() and not db.any()
    db.fill_(1)
    gemm_mod.layer_norm_grad(z, z, e, e, z, dbias=db)
    assert not db.any()


def test_captured_calls_on_another_stream(gemm_mod):
    """The forward and backward call captured together and replayed on new inputs,
    beside a second capture with sums of its own: the bits of eager calls."""
    shapes = [(700, 1024), (333, 1001)]
    graphs = []
    for m, n in shapes:
        X, dY = (torch.zeros(m, n, dtype=torch.float16, device="cuda") for _ in range(2))
        W, B = vector(n, torch.float16, 1), vector(n, torch.float16, 2, 0.0)

        def step(X=X, dY=dY, W=W, B=B):
            Y, dX = torch.empty_like(X), torch.empty_like(X)
            mean, rstd = (torch.empty(len(X), device="cuda") for _ in range(2))
            dW, db = torch.empty_like(W), torch.empty_like(W)
            gemm_mod.layer_norm(X, Y, weight=W, bias=B, mean=mean, rstd=rstd)
            gemm_mod.layer_norm_grad(dY, X, mean, rstd, dX, weight=W, dweight=dW, dbias=db)
            return Y, mean, rstd, dX, dW, db

        step()
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            out = step()
        graphs.append((graph, X, dY, out, step))
    for seed in (1, 2):
        for (graph, X, dY, _, _), (m, n) in zip(graphs, shapes):
            X.copy_(normal((m, n), torch.float16, seed))
            dY.copy_(normal((m, n), torch.float16, seed + 7))
        torch.cuda.synchronize()
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g[0].replay()
        torch.cuda.synchronize()
        for _, _, _, out, step in graphs:
            want = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_more_than_2_to_31_elements(gemm_mod):
    """Row offsets pass 32 bits: the last row of a matrix with a wide row stride."""
    rows, n, ld = 3, 256, 1 << 30
    buf = torch.empty((rows - 1) * ld + n, dtype=torch.bfloat16, device="cuda")
    X = buf.as_strided((rows, n), (ld, 1))
    src = normal((rows, n), torch.bfloat16, 1)
    X.copy_(src)
    Y, ref = torch.empty_like(src), torch.empty_like(src)
    gemm_mod.layer_norm(X, Y)
    gemm_mod.layer_norm(src, ref)
    assert torch.equal(Y, ref)
    mean, rstd = statistics(src)
    gemm_mod.layer_norm_grad(src, X, mean, rstd, Y)
    gemm_mod.layer_norm_grad(src, src, mean, rstd, ref)
    gemm_mod.layer_norm_grad(src, src, mean, rstd, X)
    torch.cuda.synchronize()
    for got in (Y, X):  # other forms: another order of the sums
        assert torch.allclose(got.float(), ref.float(), rtol=2 ** -7, atol=1e-3)


def test_refusals_of_the_binding(gemm_mod):
    X = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    Y, s = torch.zeros_like(X), torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        gemm_mod.layer_norm(X.float(), Y)
    with pytest.raises(TypeError):
        gemm_mod.layer_norm(X, Y.to(torch.float8_e4m3fn))
    with pytest.raises(TypeError):
        gemm_mod.layer_norm(X, Y, bias=Y[0].float())
    with pytest.raises(TypeError):
        gemm_mod.layer_norm(X, Y, mean=s.double())
    for kw in ({"mean": s[:3]}, {"rstd": s[:3]}, {"weight": X[0, ::2]}, {"bias": X[0, :3]},
               {"residual": Y[:3]}, {"h": Y.t()}):
        with pytest.raises(ValueError):
            gemm_mod.layer_norm(X, Y, **kw)
    with pytest.raises(ValueError):
        gemm_mod.layer_norm(X, Y.cpu())
    with pytest.raises(gemm_mod.GemmError) as e:
        gemm_mod.layer_norm(X, Y, eps=float("nan"))
    assert e.value.status == 1
    for bad in ((X, Y[:2], s, s, X), (X, Y, s[:2], s, X), (X, Y, s, s[:2], X)):
        with pytest.raises(ValueError):
            gemm_mod.layer_norm_grad(*bad)
    with pytest.raises(TypeError):
        gemm_mod.layer_norm_grad(X, Y, None, s, X)
    with pytest.raises(ValueError):
        gemm_mod.layer_norm_grad(X, Y, s, s, X, dbias=X[0, :32])
