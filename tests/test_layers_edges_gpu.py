"""Edges of the linear-layer operators on the GPU: few rows spread unevenly over a
warp's lanes, sizes and alignments that pick the rarer kernels, special values in
gradients, captured gradients. Bounds come from tests/layer_util.py; results that
are exact by construction are compared exactly."""
import numpy as np
import pytest
import torch

from oracle import layers as L
from tests.layer_util import (DTYPES, Out, act_error, assert_close, normal, product_bound,
                              rounded_bound)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word(gemm_mod):
    gemm_mod.check_device_error()
    yield
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0


@pytest.mark.parametrize("m", [1, 3, 17, 33, 100])
def test_lanes_with_different_numbers_of_rows_over_many_calls(gemm_mod, m):
    """The finishing lanes of the few-rows kernel have different numbers of rows, and
    of the last column tile's lanes some have none (N = 1000 in tiles of 128): calls
    back to back, on operands that change, against a call alone."""
    A = [normal((m, 2048), torch.bfloat16, i) for i in range(4)]
    B = normal((1000, 2048), torch.bfloat16, 9, 0.02)
    R = normal((m, 1000), torch.bfloat16, 10)
    ref = []
    for a in A:
        D = torch.empty_like(R)
        gemm_mod.gemm_epilogue(a, B, D, act="silu", residual=R, trans_b=True)
        torch.cuda.synchronize()
        ref.append(D)
    out = [torch.empty_like(R) for _ in range(400)]
    for i, D in enumerate(out):
        gemm_mod.gemm_epilogue(A[i % 4], B, D, act="silu", residual=R, trans_b=True)
    torch.cuda.synchronize()
    assert all(torch.equal(D, ref[i % 4]) for i, D in enumerate(out))


@pytest.mark.parametrize("preact", [False, True])
def test_stores_of_several_units_per_warp_over_many_calls(gemm_mod, preact):
    """256-row tiles, several units per warp and several tiles per CTA pair, with the
    last tile cut in both directions: every call the same bits."""
    m, n, k = 2100, 2440, 192
    A, B = normal((m, k), torch.bfloat16, 1), normal((n, k), torch.bfloat16, 2)
    ref = None
    for _ in range(20):
        D = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        Z = torch.empty_like(D) if preact else None
        gemm_mod.gemm_epilogue(A, B, D, act="gelu_tanh", preact=Z, trans_b=True)
        ref = ref or (D, Z)
        assert torch.equal(D, ref[0]) and (Z is None or torch.equal(Z, ref[1]))


@pytest.mark.parametrize("m", [16, 100, 128, 200])
def test_bias_gradient_of_few_rows_with_a_long_inner_dimension(gemm_mod, m):
    """Few-rows gradients whose k range is split over a cluster, at every tile height:
    the sums are those of the stored dZ's unrounded values, the same on every call."""
    n, k = 1000, 4096
    A = normal((m, k), torch.bfloat16, 1)
    B = normal((n, k), torch.bfloat16, 2, k ** -0.5)
    Z = normal((m, n), torch.bfloat16, 3)
    ref = None
    for _ in range(50):
        dZ, db = torch.empty_like(Z), torch.empty(n, dtype=torch.bfloat16, device="cuda")
        gemm_mod.gemm_dact(A, B, Z, dZ, act="silu", dbias=db, trans_b=True)
        ref = ref or (dZ, db)
        assert torch.equal(dZ, ref[0]) and torch.equal(db, ref[1])
    A64, B64 = L.to64(A), L.to64(B).T
    dz, want = L.linear_grad(A64 @ B64, L.to64(Z), "silu")
    e = 1.13 * product_bound(A64, B64) + np.abs(A64 @ B64) * 2.0 ** -18 * (1 + np.abs(L.to64(Z)))
    assert_close(L.to64(dZ), dz, rounded_bound(dz, e, torch.bfloat16), "dZ")
    eb = e.sum(0) + m * 2.0 ** -24 * np.abs(dz).sum(0)
    assert_close(L.to64(db), want, rounded_bound(want, eb, torch.bfloat16), "dbias")


@pytest.mark.parametrize("op", ["linear", "gradient"])
@pytest.mark.parametrize("n", [600, 777])
def test_rows_read_by_copies_and_written_by_plain_stores(gemm_mod, op, n):
    """R (Zin) in whole 16-byte units, D off them: the tile kernel's staging buffer is
    in turn filled by an asynchronous copy and by ordinary stores, over several units
    per warp and several tiles per CTA pair. Against the same call with D aligned."""
    m, k = 2600, 128
    A, B = normal((m, k), torch.bfloat16, 1), normal((n, k), torch.bfloat16, 2, 0.1)
    R = normal((m, n), torch.bfloat16, 3, unit=8)
    ref = torch.empty(m, 784, dtype=torch.bfloat16, device="cuda")[:, :n]
    for i in range(10):
        flat = torch.empty(m * n + 1, dtype=torch.bfloat16, device="cuda")
        D = flat[1:].view(m, n)
        for out in (ref, D) if i == 0 else (D,):
            if op == "linear":
                gemm_mod.gemm_epilogue(A, B, out, act="gelu", residual=R, trans_b=True)
            else:
                gemm_mod.gemm_dact(A, B, R, out, act="silu", trans_b=True)
        assert torch.equal(D, ref)
    A64, B64 = L.to64(A), L.to64(B).T
    if op == "linear":
        want, z = L.linear(A64, B64, 1.0, None, "gelu", L.to64(R))
        e = 1.13 * product_bound(A64, B64) + act_error(z, "gelu") + 2.0 ** -23 * np.abs(want)
    else:
        d = A64 @ B64
        want, _ = L.linear_grad(d, L.to64(R), "silu")
        e = 1.13 * product_bound(A64, B64) + np.abs(d) * 2.0 ** -18 * (1 + np.abs(L.to64(R)))
    assert_close(L.to64(ref), want, rounded_bound(want, e, torch.bfloat16), "D")


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("m", [5, 65, 300, 352, 513])
def test_bias_gradient_of_an_infinite_column(gemm_mod, m, value, act):
    """An infinity in column 2 of B makes that column of dZ infinite, of one sign: so
    is its sum, whatever M is modulo 32, and no other column changes."""
    A = normal((m, 72), torch.bfloat16, 1)
    A[:, 5] = A[:, 5].abs() + 0.5
    B = normal((72, 96), torch.bfloat16, 2)
    Z = torch.ones(m, 96, dtype=torch.bfloat16, device="cuda")
    out = []
    for v in (0.0, value):
        B[5, 2] = v
        dZ, db = torch.empty_like(Z), torch.empty(96, dtype=torch.bfloat16, device="cuda")
        gemm_mod.gemm_dact(A, B, Z, dZ, act=act, dbias=db)
        out.append((dZ, db))
    (dZ0, db0), (dZ, db) = out
    assert bool((dZ[:, 2] == value).all()) and db[2].item() == value
    dZ[:, 2], db[2] = dZ0[:, 2], db0[2]
    assert torch.equal(dZ, dZ0) and torch.equal(db, db0)


@pytest.mark.parametrize("m,n", [(9, 64), (700, 500), (40, 1001), (5, 4096), (2, 20001)])
@pytest.mark.parametrize("shift", [0, 1])
def test_gradient_of_tiny_rows(gemm_mod, m, n, shift):
    """Rows whose rstd squared is past fp32's largest value, dX itself is not."""
    H = normal((m, n), torch.bfloat16, n, 2e-20)
    dY, W = normal((m, n), torch.bfloat16, n + 1), normal((1, n), torch.bfloat16, n + 2)[0]
    h64, y64, w64 = L.to64(H), L.to64(dY), L.to64(W)
    rstd = torch.from_numpy((h64 * h64).mean(1) ** -0.5).float().cuda()
    s64 = L.to64(rstd)
    assert s64.min() > 2.0 ** 64
    dX, dW = Out(m, n, torch.bfloat16, shift=shift), Out(1, n, torch.bfloat16)
    gemm_mod.rms_norm_grad(dY, H, rstd, dX.t, weight=W, dweight=dW.t[0])
    torch.cuda.synchronize()
    dx, dw = L.rms_norm_grad(y64, h64, s64, w64)
    nrm, g = h64 * s64[:, None], np.abs(y64 * w64)
    terms = s64[:, None] * (g + np.abs(nrm) * (g * np.abs(nrm)).mean(1, keepdims=True))
    assert_close(L.to64(dX.t), dx, rounded_bound(dx, 2.0 ** -17 * terms, torch.bfloat16), "dX")
    ew = (m + 20) * 2.0 ** -24 * np.abs(y64 * nrm).sum(0)
    assert_close(L.to64(dW.t[0]), dw, rounded_bound(dw, ew, torch.bfloat16), "dW")


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m", [5, 300])
@pytest.mark.parametrize("k", [0, 8])
def test_infinite_preactivations(gemm_mod, m, act, k):
    """+inf stays +inf; -inf is 0 for relu and NaN where the formula has -inf * 0."""
    inf = float("inf")
    for dtype in DTYPES.values():
        A, B = torch.zeros(m, k, dtype=dtype, device="cuda"), torch.zeros(
            k, 40, dtype=dtype, device="cuda")
        bias = torch.zeros(40, dtype=dtype, device="cuda")
        bias[3], bias[4] = inf, -inf
        if k:
            B[0] = 1
            A[1, 0] = inf
            A[2, 0] = -inf
        D = torch.empty(m, 40, dtype=dtype, device="cuda")
        gemm_mod.gemm_epilogue(A, B, D, act=act, bias=bias)
        z = np.zeros((m, 40))
        z[:, 3] += inf
        z[:, 4] -= inf
        if k:
            with np.errstate(invalid="ignore"):
                z[1] += inf
                z[2] -= inf
        with np.errstate(invalid="ignore"):
            ref = L.act(z, act)
        assert np.array_equal(L.to64(D), ref, equal_nan=True), act


@pytest.mark.parametrize("m,n", [(40, 264), (300, 1000), (2000, 512), (700, 2048)])
def test_gradients_captured_in_a_graph(gemm_mod, m, n):
    """A layer's gradients, whose column sums allocate from the library's pool inside
    the calls, captured once and replayed on new inputs: the bits of plain calls."""
    dt = torch.bfloat16
    inputs = [torch.empty(m, n, dtype=dt, device="cuda") for _ in range(4)]
    dD, Z, H, dH = inputs
    Wt, gain = normal((n, n), dt, 1, n ** -0.5), normal((1, n), dt, 2)[0]
    rstd = torch.empty(m, device="cuda")

    def draw(seed):
        for i, t in enumerate(inputs):
            t.copy_(normal((m, n), dt, 10 * seed + i))
        rstd.copy_(torch.rsqrt(H.float().square().mean(1)))

    def layer():
        out = [torch.empty_like(dD) for _ in range(3)]
        sums = [torch.empty(n, dtype=dt, device="cuda") for _ in range(3)]
        gemm_mod.act_grad(dD, Z, out[0], act="gelu", dbias=sums[0])
        gemm_mod.gemm_dact(out[0], Wt, Z, out[1], act="silu", dbias=sums[1])
        gemm_mod.rms_norm_grad(out[1], H, rstd, out[2], weight=gain, dh=dH, dweight=sums[2])
        return out + sums

    draw(1)
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer()
    for seed in (2, 3, 3):
        draw(seed)
        for t in captured:
            t.fill_(7)
        graph.replay()
        want = layer()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m", [7, 300])
def test_tails_keep_their_relative_accuracy(gemm_mod, act, m):
    """z from -12 to -3 (a product of one value and one, exact): within 2^-15 relative,
    then rounded. The exponential's argument in base 2 is at most 126, where the factor
    underflows, and carries at most three roundings of 2^-24; the rest (the polynomial's
    2^-19, the one-instruction exponential and reciprocal, products) adds less than
    2^-18: 126 * 3 * 2^-24 * ln 2 + 2^-18 < 2^-15.6. A factor below 2^-126 counts as
    zero: 2^-126 |z| absolute."""
    n = 288
    bf = torch.bfloat16
    z = torch.linspace(-12, -3, m).to(bf)
    A = torch.zeros(m, 8, dtype=bf)
    A[:, 0] = z
    B = torch.zeros(8, n, dtype=bf)
    B[0] = 1
    D = torch.empty(m, n, dtype=bf, device="cuda")
    gemm_mod.gemm_epilogue(A.cuda(), B.cuda(), D, act=act)
    z64 = L.to64(z)
    want = L.act(z64, act) if act != "gelu_tanh" else z64 / (
        1 + np.exp(-2 * np.sqrt(2 / np.pi) * (z64 + 0.044715 * z64 ** 3)))
    bound = rounded_bound(want, 2.0 ** -15 * np.abs(want) + 2.0 ** -126 * np.abs(z64), bf)
    assert_close(L.to64(D), np.repeat(want[:, None], n, 1), np.repeat(bound[:, None], n, 1), "D")
