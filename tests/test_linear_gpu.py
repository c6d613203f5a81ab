"""GPU parity of the product with an epilogue (gemm_epilogue) and of its gradient
(gemm_dact, act_grad) against the float64 oracle.

Tolerances (tests/layer_util.py), each from the arithmetic that is promised:

* every output element is the fp32 result rounded once: within one unit roundoff
  of the exact value plus the fp32 error carried through the activation, whose
  slope is at most 1.13;
* a stored pre-activation the same without the activation;
* dbias: the elements' errors before rounding, added up, M fp32 additions and
  one rounding;
* in the mean, outputs are within the rounding of their format: relative
  Frobenius error at most the unit roundoff plus the product's fp32 error (this
  is what a dropped k-block or a lost scale would break).
"""
import numpy as np
import pytest
import torch

from oracle import layers as L
from tests.layer_util import (DTYPES, UNIT, Out, act_error, assert_close, e4m3, normal,
                              product_bound, rounded_bound)

pytestmark = pytest.mark.gpu

MAX_SLOPE = 1.13
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(autouse=True)
def clean_error_word(gemm_mod):
    gemm_mod.check_device_error()
    yield
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0


def frobenius(got, ref):
    return np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300)


def run_linear(g, m, n, k, dtype, act="none", bias=True, residual=True, preact=True, trans_a=False,
               trans_b=False, alpha=1.0, pad=0, shift=0, eight_bit=False, inplace=False, seed=0):
    std = max(k, 1) ** -0.5
    sa = sb = None
    if eight_bit:
        A, sa = e4m3(m, k, seed + 1)
        B, sb = e4m3(n, k, seed + 2, std)
        trans_b = True
    else:
        A = normal((k, m) if trans_a else (m, k), dtype, seed + 1, unit=8)
        B = normal((n, k) if trans_b else (k, n), dtype, seed + 2, std, unit=8)
    b = normal((1, n), dtype, seed + 3)[0] if bias else None
    out = Out(m, n, dtype, pad, shift)
    R = None
    if residual:
        R = normal((m, n), dtype, seed + 4, pad=pad)
        if inplace:
            out.t.copy_(R)
            R64 = L.to64(R)
            R = out.t
    pre = Out(m, n, dtype, pad, shift) if preact else None
    g.gemm_epilogue(A, B, out.t, alpha=alpha, bias=b, act=act, residual=R,
                    preact=pre.t if pre else None, trans_a=trans_a, trans_b=trans_b, scale_a=sa,
                    scale_b=sb)
    torch.cuda.synchronize()
    A64 = L.to64(A).T if trans_a else L.to64(A)
    B64 = L.to64(B).T if trans_b else L.to64(B)
    s64 = [None if s is None else L.to64(s) for s in (sa, sb)]
    b64 = None if b is None else L.to64(b)
    if R is not None and not inplace:
        R64 = L.to64(R)
    D, Z = L.linear(A64, B64, alpha, b64, act, R64 if residual else None, *s64)
    ez = product_bound(A64, B64, alpha, *s64) + 2.0 ** -23 * np.abs(Z)
    ed = MAX_SLOPE * ez + act_error(Z, act) + 2.0 ** -23 * np.abs(D)
    got = L.to64(out.t)
    assert_close(got, D, rounded_bound(D, ed, dtype), "D")
    if m * n:
        assert frobenius(got, D) <= UNIT[dtype] + 2e-5
    out.check_guards()
    if pre:
        assert_close(L.to64(pre.t), Z, rounded_bound(Z, ez, dtype), "Z")
        pre.check_guards()


# Sizes around the tiles' and the few-rows kernel's edges, one row to several
# tiles, k from one element over one k-block to many, and odd everything.
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 4096, 512), (2, 129, 65), (5, 250, 1000), (16, 1024, 2048),
          (17, 2048, 136), (33, 520, 200), (64, 640, 2048), (65, 130, 72), (100, 1111, 513),
          (128, 256, 64), (129, 257, 127), (200, 384, 4096), (255, 1023, 520), (256, 512, 1024),
          (257, 255, 63), (384, 4096, 128), (513, 777, 1023), (1000, 300, 2000)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3-bf16", "e4m3-f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(gemm_mod, shape, kind):
    m, n, k = shape
    i = SHAPES.index(shape)
    run_linear(gemm_mod, m, n, k, DTYPES[kind.split("-")[-1]], ACTS[i % 5], bias=i % 3 != 0,
               residual=i % 2 == 0, preact=i % 4 != 1, trans_a=False, trans_b=i % 2 == 1,
               eight_bit=kind.startswith("e4m3"), seed=i)


@pytest.mark.parametrize("trans_a", [False, True], ids=["an", "at"])
@pytest.mark.parametrize("trans_b", [False, True], ids=["bn", "bt"])
@pytest.mark.parametrize("shape", [(3, 140, 260), (40, 300, 100), (130, 200, 264),
                                   (300, 520, 1000)], ids=lambda s: "x".join(map(str, s)))
def test_operand_forms(gemm_mod, shape, trans_a, trans_b):
    run_linear(gemm_mod, *shape, torch.bfloat16, "silu", trans_a=trans_a, trans_b=trans_b,
               alpha=-0.75, seed=31)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [7, 150, 600])
def test_activations(gemm_mod, act, m):
    for dtype in DTYPES.values():
        run_linear(gemm_mod, m, 264, 128, dtype, act, alpha=3.0, seed=m)


@pytest.mark.parametrize("shift,pad", [(0, 0), (0, 8), (0, 3), (1, 0), (8, 1), (3, 5)])
@pytest.mark.parametrize("m", [9, 140, 520])
def test_output_layouts(gemm_mod, m, shift, pad):
    run_linear(gemm_mod, m, 272, 96, torch.float16, "gelu", pad=pad, shift=shift, trans_b=True)
    run_linear(gemm_mod, m, 272, 96, torch.bfloat16, "relu", pad=pad, shift=shift, inplace=True)


@pytest.mark.parametrize("m", [4, 200, 1030])
def test_every_combination_of_terms(gemm_mod, m):
    for mask in range(8):
        run_linear(gemm_mod, m, 136, 80, torch.bfloat16, "gelu_tanh", bias=bool(mask & 1),
                   residual=bool(mask & 2), preact=bool(mask & 4), trans_b=True)


@pytest.mark.parametrize("m", [12, 144, 700])
def test_scales_may_be_left_out(gemm_mod, m):
    A, sa = e4m3(m, 160, 1)
    B, sb = e4m3(96, 160, 2)
    for qa, qb in ((None, None), (sa, None), (None, sb)):
        D = torch.empty(m, 96, dtype=torch.bfloat16, device="cuda")
        alpha = 1.0 if qa is not None or qb is not None else 2.0 ** -12
        gemm_mod.gemm_epilogue(A, B, D, alpha=alpha, trans_b=True, scale_a=qa, scale_b=qb)
        torch.cuda.synchronize()
        s = [None if q is None else L.to64(q) for q in (qa, qb)]
        ref, _ = L.linear(L.to64(A), L.to64(B).T, alpha, None, None, None, *s)
        e = product_bound(L.to64(A), L.to64(B).T, alpha, *s)
        assert_close(L.to64(D), ref, rounded_bound(ref, e, torch.bfloat16), "D")


@pytest.mark.parametrize("m", [3, 300])
def test_empty_inner_dimension(gemm_mod, m):
    for dtype in DTYPES.values():
        run_linear(gemm_mod, m, 70, 0, dtype, "silu")
    run_linear(gemm_mod, m, 70, 0, torch.bfloat16, "gelu", eight_bit=True)


@pytest.mark.parametrize("m", [6, 260])
def test_integers_are_exact(gemm_mod, m):
    """Small integers: every sum is exact in fp32, so D is the rounded integer."""
    r = torch.Generator().manual_seed(m)
    A = torch.randint(-8, 9, (m, 520), generator=r).to(torch.float32)
    B = torch.randint(-8, 9, (144, 520), generator=r).to(torch.float32)
    ref = (A.double() @ B.double().t())
    for dtype in DTYPES.values():
        D = torch.empty(m, 144, dtype=dtype, device="cuda")
        gemm_mod.gemm_epilogue(A.to(dtype).cuda(), B.to(dtype).cuda(), D, trans_b=True)
        assert torch.equal(D.cpu(), ref.to(dtype))
    A8 = torch.zeros(m, 528, dtype=torch.float8_e4m3fn, device="cuda")[:, :520]
    B8 = torch.zeros(144, 528, dtype=torch.float8_e4m3fn, device="cuda")[:, :520]
    A8.copy_(A.to(torch.float8_e4m3fn))
    B8.copy_(B.to(torch.float8_e4m3fn))
    D = torch.empty(m, 144, dtype=torch.bfloat16, device="cuda")
    gemm_mod.gemm_epilogue(A8, B8, D, trans_b=True)
    assert torch.equal(D.cpu(), ref.to(torch.bfloat16))


@pytest.mark.parametrize("m", [5, 270])
def test_special_values_stay_in_their_row_and_column(gemm_mod, m):
    """A NaN in row 1 of A and an infinity in column 2 of B reach the outputs that
    use them and no others; relu keeps NaN; +-infinite pre-activations."""
    A = normal((m, 72), torch.bfloat16, 1)
    B = normal((40, 72), torch.bfloat16, 2)
    A[1, 3] = float("nan")
    B[2, 5] = float("inf")
    A[:, 5] = A[:, 5].abs() + 0.5
    D = torch.empty(m, 40, dtype=torch.bfloat16, device="cuda")
    gemm_mod.gemm_epilogue(A, B, D, act="relu", trans_b=True)
    got = D.float().cpu()
    assert bool(got[1].isnan().all())
    rest = torch.cat([got[:1], got[2:]])
    assert bool((rest[:, 2] == float("inf")).all())
    rest[:, 2] = 0
    assert bool(rest.isfinite().all())


@pytest.mark.parametrize("m", [8, 190, 1500])
def test_same_bits_every_call_and_on_another_stream(gemm_mod, m):
    A = normal((m, 1000), torch.bfloat16, 1)
    B = normal((520, 1000), torch.bfloat16, 2)
    D = [torch.empty(m, 520, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    gemm_mod.gemm_epilogue(A, B, D[0], act="silu", trans_b=True)
    gemm_mod.gemm_epilogue(A, B, D[1], act="silu", trans_b=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gemm_mod.gemm_epilogue(A, B, D[2], act="silu", trans_b=True, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(D[0], D[1]) and torch.equal(D[0], D[2])


def test_output_past_2_to_31_elements(gemm_mod):
    """Offsets of D, Z and R pass 32 bits: the last rows of a tall output, against
    the same rows computed alone."""
    m, n, k = 70000, 32768, 64
    A = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    A[-300:] = normal((300, k), torch.bfloat16, 1)
    B = normal((n, k), torch.bfloat16, 2)
    D, R = (torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    R[:-300].zero_()
    R[-300:] = normal((300, n), torch.bfloat16, 3)
    gemm_mod.gemm_epilogue(A, B, D, residual=R, act="silu", trans_b=True)
    tail = torch.empty(300, n, dtype=torch.bfloat16, device="cuda")
    gemm_mod.gemm_epilogue(A[-300:], B, tail, residual=R[-300:], act="silu", trans_b=True)
    assert torch.equal(D[-300:], tail)
    assert not D[:-300].any()
    gemm_mod.act_grad(D, R, D, act="relu")
    want = torch.empty_like(tail)
    gemm_mod.act_grad(tail, R[-300:], want, act="relu")
    assert torch.equal(D[-300:], want)


def test_captured_in_a_graph(gemm_mod):
    A = normal((24, 512), torch.bfloat16, 1)
    B = normal((768, 512), torch.bfloat16, 2)
    W = normal((768, 512), torch.bfloat16, 3)
    H = torch.empty(24, 768, dtype=torch.bfloat16, device="cuda")
    Y = torch.empty(24, 512, dtype=torch.bfloat16, device="cuda")

    def layers():
        gemm_mod.gemm_epilogue(A, B, H, act="relu", trans_b=True)
        gemm_mod.gemm_epilogue(H, W, Y, residual=A)

    layers()
    torch.cuda.synchronize()
    ref = Y.clone()
    Y.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, ref)


# ------------------------------------------------------------------- gradient

def check_grad(d64, ed, Z, act, dz, db, dtype, m):
    """dz, db against the exact gradient of d64 (within ed) at Z."""
    Z64 = L.to64(Z) if Z is not None else np.zeros_like(d64)
    ref, ref_b = L.linear_grad(d64, Z64, act)
    slope_error = 0.0 if act in ("none", "relu") else 2.0 ** -18 * (1 + np.abs(Z64))
    e = MAX_SLOPE * ed + np.abs(d64) * slope_error + 2.0 ** -23 * np.abs(ref)
    if dz is not None:
        assert_close(L.to64(dz), ref, rounded_bound(ref, e, dtype), "dZ")
    if db is not None:
        eb = e.sum(0) + m * 2.0 ** -24 * np.abs(ref).sum(0)
        assert_close(L.to64(db), ref_b, rounded_bound(ref_b, eb, dtype), "dbias")


GRAD_SHAPES = [(1, 1, 1), (1, 320, 200), (7, 129, 65), (60, 1000, 264), (128, 256, 64),
               (129, 130, 1000), (300, 1000, 520), (520, 257, 96), (1030, 640, 128)]


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("shape", GRAD_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_dact(gemm_mod, shape, dtype):
    m, n, k = shape
    i = GRAD_SHAPES.index(shape)
    act, trans_b = ACTS[i % 5], i % 2 == 0
    A = normal((m, k), dtype, i, unit=8)
    B = normal((n, k) if trans_b else (k, n), dtype, i + 1, k ** -0.5, unit=8)
    Z = normal((m, n), dtype, i + 2, 1.5, pad=i % 3)
    out = Out(m, n, dtype, pad=i % 4, shift=i % 2)
    db = Out(1, n, dtype)
    gemm_mod.gemm_dact(A, B, Z if act != "none" else None, out.t, act=act, alpha=0.5,
                       dbias=db.t[0], trans_b=trans_b)
    torch.cuda.synchronize()
    A64, B64 = L.to64(A), L.to64(B).T if trans_b else L.to64(B)
    check_grad(0.5 * (A64 @ B64), product_bound(A64, B64, 0.5), Z, act, out.t, db.t[0], dtype, m)
    out.check_guards()
    db.check_guards()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [10, 310])
def test_dact_activations_in_place_and_without_sums(gemm_mod, act, m):
    A = normal((m, 96), torch.bfloat16, 1)
    B = normal((96, 264), torch.bfloat16, 2, 0.1)
    Z = normal((m, 264), torch.bfloat16, 3, 2.0)
    ref, out = torch.empty_like(Z), Z.clone()
    gemm_mod.gemm_dact(A, B, Z, ref, act=act)
    gemm_mod.gemm_dact(A, B, out, out, act=act)
    torch.cuda.synchronize()
    A64, B64 = L.to64(A), L.to64(B)
    check_grad(A64 @ B64, product_bound(A64, B64), Z, act, ref, None, torch.bfloat16, m)
    assert torch.equal(ref, out)


@pytest.mark.parametrize("trans_a", [False, True], ids=["an", "at"])
@pytest.mark.parametrize("trans_b", [False, True], ids=["bn", "bt"])
def test_dact_operand_forms(gemm_mod, trans_a, trans_b):
    m, n, k = 150, 280, 200
    A = normal((k, m) if trans_a else (m, k), torch.float16, 1, unit=8)
    B = normal((n, k) if trans_b else (k, n), torch.float16, 2, 0.1, unit=8)
    Z = normal((m, n), torch.float16, 3)
    out, db = torch.empty_like(Z), torch.empty(n, dtype=torch.float16, device="cuda")
    gemm_mod.gemm_dact(A, B, Z, out, act="gelu", dbias=db, trans_a=trans_a, trans_b=trans_b)
    torch.cuda.synchronize()
    A64 = L.to64(A).T if trans_a else L.to64(A)
    B64 = L.to64(B).T if trans_b else L.to64(B)
    check_grad(A64 @ B64, product_bound(A64, B64), Z, "gelu", out, db, torch.float16, m)


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", [(1, 1), (1, 4096), (9, 255), (300, 256), (1000, 264),
                                   (4100, 24), (37, 1001)], ids=lambda s: "x".join(map(str, s)))
def test_act_grad(gemm_mod, shape, act, dtype):
    m, n = shape
    pad = 8 if m % 2 else 3 * (n % 2)
    dD = normal(shape, dtype, m, pad=pad)
    Z = normal(shape, dtype, n, 2.0, pad=pad)
    out, db = Out(m, n, dtype, pad=pad), Out(1, n, dtype)
    gemm_mod.act_grad(dD, Z, out.t, act=act, dbias=db.t[0])
    torch.cuda.synchronize()
    d64 = L.to64(dD)
    check_grad(d64, np.zeros_like(d64), Z, act, out.t, db.t[0], dtype, m)
    out.check_guards()
    db.check_guards()


def test_act_grad_sums_only_and_in_place(gemm_mod):
    dD = normal((333, 520), torch.bfloat16, 1)
    db = torch.empty(520, dtype=torch.bfloat16, device="cuda")
    gemm_mod.act_grad(dD, None, None, dbias=db)
    torch.cuda.synchronize()
    d64 = L.to64(dD)
    check_grad(d64, np.zeros_like(d64), None, "none", None, db, torch.bfloat16, 333)
    Z = normal((333, 520), torch.bfloat16, 2)
    a, b, c = torch.empty_like(dD), dD.clone(), Z.clone()
    gemm_mod.act_grad(dD, Z, a, act="silu")
    gemm_mod.act_grad(b, Z, b, act="silu")
    gemm_mod.act_grad(dD, c, c, act="silu")
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


def test_act_grad_far_values(gemm_mod):
    """Slopes far out are 0 and 1, also where the polynomials overflow."""
    z = torch.tensor([[-3e38, -1e30, -1e19, -200.0, -90.0, 90.0, 200.0, 1e19, 1e30, 3e38]])
    Z = z.bfloat16().cuda()
    dD = torch.ones_like(Z)
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        out = torch.empty_like(Z)
        gemm_mod.act_grad(dD, Z, out, act=act)
        assert out.float().cpu().tolist() == [[0.0] * 5 + [1.0] * 5], act


@pytest.mark.parametrize("k", [0, 64])
def test_gradient_of_nothing(gemm_mod, k):
    """No rows, or no inner dimension: the sums are zero."""
    m = 0 if k else 9
    A = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    B = torch.empty(k, 40, dtype=torch.bfloat16, device="cuda").fill_(1)
    Z = torch.ones(m, 40, dtype=torch.bfloat16, device="cuda")
    dZ = torch.full_like(Z, 5)
    db = torch.full((40,), 5.0, dtype=torch.bfloat16, device="cuda")
    gemm_mod.gemm_dact(A, B, Z, dZ, act="silu", dbias=db)
    assert not db.any() and not dZ.any()
    db.fill_(5)
    gemm_mod.act_grad(Z[:0], Z[:0], dZ[:0], act="silu", dbias=db)
    assert not db.any()


def test_gradient_against_differences_of_the_kernel(gemm_mod):
    """d(sum(G * D)) of the GPU forward call by bias and along random directions
    of A and B, against the GPU gradients. Steps of 2^-3 in fp16 at k = 8: the
    forward outputs round to 2^-11 relative, so a difference over 2^-2 carries
    at most (sum |G| |D|) 2^-11 / 2^-2, plus a curvature error h^2 / 6 * |f'''|
    with |f'''| <= 1.2 for silu."""
    m, n, k, h = 24, 40, 8, 2.0 ** -3
    f16 = torch.float16
    A, B = normal((m, k), f16, 1), normal((k, n), f16, 2, 0.5)
    bias, G = normal((1, n), f16, 3)[0].contiguous(), normal((m, n), f16, 4)
    dD, Z = torch.empty_like(G), torch.empty_like(G)

    def forward(bias, keep=None):
        D = torch.empty_like(G)
        gemm_mod.gemm_epilogue(A, B, D, bias=bias, act="silu", preact=keep)
        return D.double()

    D0 = forward(bias, Z)
    dD.copy_(G)
    dZ, db = torch.empty_like(G), torch.empty_like(bias)
    gemm_mod.act_grad(dD, Z, dZ, act="silu", dbias=db)
    up, down = forward(bias + h), forward(bias - h)
    fd = (G.double() * (up - down)).sum(0) / (2 * h)
    g = G.double().abs()
    tol = (g * (up.abs() + down.abs())).sum(0) * 2.0 ** -11 / (2 * h) + g.sum(0) * h * h / 6 * 1.2
    tol += 2.0 ** -10 * (g * (1.2 + D0.abs())).sum(0)  # rounded Z, db and bias +- h
    assert bool(((fd - db.double()).abs() <= tol).all())
    # dA = dZ B^T through the product itself
    dA = torch.empty_like(A)
    gemm_mod.gemm_epilogue(dZ, B, dA, trans_b=True)
    ref = L.to64(dZ) @ L.to64(B).T
    e = product_bound(L.to64(dZ), L.to64(B).T)
    assert_close(L.to64(dA), ref, rounded_bound(ref, e, f16), "dA")


def test_refusals_of_the_binding(gemm_mod):
    A = torch.zeros(16, 32, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(32, 24, dtype=torch.bfloat16, device="cuda")
    D = torch.zeros(16, 24, dtype=torch.bfloat16, device="cuda")
    ok = dict(act="relu")
    with pytest.raises(ValueError):
        gemm_mod.gemm_epilogue(A, B, D[:8], **ok)
    with pytest.raises(TypeError):
        gemm_mod.gemm_epilogue(A, B, D.float(), **ok)
    with pytest.raises(TypeError):
        gemm_mod.gemm_epilogue(A, B.half(), D, **ok)
    with pytest.raises(ValueError):
        gemm_mod.gemm_epilogue(A, B, D, act="tanh")
    with pytest.raises(ValueError):
        gemm_mod.gemm_epilogue(A, B, D, residual=D[:1].expand(16, 24))
    with pytest.raises(ValueError):
        gemm_mod.gemm_epilogue(A, B, D, residual=D.cpu())
    with pytest.raises(ValueError):
        gemm_mod.gemm_epilogue(A.cpu(), B, D)
    with pytest.raises(ValueError):
        gemm_mod.gemm_epilogue(A, B, D, bias=torch.zeros(16, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        gemm_mod.gemm_epilogue(A, B, D, scale_a=torch.zeros(16, device="cuda"))
    f8 = torch.float8_e4m3fn
    with pytest.raises(ValueError):
        gemm_mod.gemm_epilogue(A.to(f8), B.to(f8), D)  # B has to be N x K
    with pytest.raises(gemm_mod.GemmError) as e:
        gemm_mod.gemm_epilogue(A[:, 1:], B[1:], D)
    assert e.value.status == 2
    with pytest.raises(gemm_mod.GemmError) as e:
        gemm_mod.gemm_dact(A, B, None, D, act="silu")
    assert e.value.status == 1
