"""Rows of the layer norm whose result is known exactly, or whose sums are long."""
import pytest
import torch

from tests.layer_util import DTYPES, Out

pytestmark = pytest.mark.gpu

VALUES = {torch.float16: [1.0, -3.0, 0.1, 1000.0, 60000.0],
          torch.bfloat16: [1.0, -3.0, 0.1, 1e6, 1e30]}


@pytest.fixture(autouse=True)
def clean_error_word(gemm_mod):
    gemm_mod.check_device_error()
    yield
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0


# Every form of the kernel: few rows and many, each width. The sum of n equal values of
# p significant bits (fp16 11, bf16 8), and every part of it, has at most p + log2 n bits
# and is exact in fp32 up to 24 of them: 8192 and 65536 columns.
@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("n", [1, 41, 82, 121, 500, 1000, 1022, 2000, 2055, 4095, 5000, 7168, 8192,
                               12000, 20001, 65536])
def test_rows_of_equal_values(gemm_mod, n, dtype):
    """h - mean is 0 in each of them: y = b, the mean is the value, and with eps = 0 y is
    0 / 0, NaN, as the formula says."""
    if dtype == torch.float16 and n > 8192:
        n = 8192 - n % 1000
    values = VALUES[dtype]
    for rows in (len(values), 8 * (1600000 // n // 8 + 1)):
        v = torch.tensor(values, device="cuda").to(dtype).repeat(-(-rows // len(values)))[:rows]
        X = v[:, None].expand(rows, n).contiguous()
        b = (torch.arange(n, device="cuda") % 7 - 3).to(dtype)
        mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
        for residual in (None, X):  # twice the value
            Y = Out(rows, n, dtype)
            gemm_mod.layer_norm(X, Y.t, weight=b, bias=b, residual=residual, mean=mean, rstd=rstd,
                                eps=1e-5)
            assert torch.equal(mean, v.float() * (1 if residual is None else 2))
            assert bool((rstd * 1e-5 ** 0.5 - 1).abs().max() < 1e-6)
            assert torch.equal(Y.t, b.expand(rows, n))
            Y.check_guards()
        Y = torch.zeros_like(X)
        gemm_mod.layer_norm(X, Y, eps=0.0)
        assert bool(Y.isnan().all())


@pytest.mark.parametrize("n", [3, 41, 333, 1000, 1031, 2055, 4095, 7168, 16000, 20001])
def test_mean_of_exact_sums(gemm_mod, n):
    """Integers up to 31, whose sums fp32 holds: the mean is the rounded quotient. An
    infinity makes it infinite."""
    for rows in (3, 1600000 // n + 8):
        X = torch.randint(-31, 32, (rows, n), device="cuda",
                          generator=torch.Generator(device="cuda").manual_seed(n)).half()
        mean, Y = torch.empty(rows, device="cuda"), torch.empty_like(X)
        gemm_mod.layer_norm(X, Y, mean=mean)
        assert torch.equal(mean, (X.double().sum(1) / n).float())
        X[1, n // 2] = float("-inf")
        gemm_mod.layer_norm(X, Y, mean=mean)
        assert mean[1] == float("-inf") and bool(mean[[0, 2]].isfinite().all())
        assert bool(Y[1].isnan().all())


# Bounds for long rows. A thread adds 8 values at a time in fp32; those sums are added
# with compensation, so that their number does not matter (2 roundings); then 5 steps in
# the warp and 32 warps: fewer than 64 additions in turn, 2^-18 of the sum of magnitudes.
LONG = [(1, 1 << 26), (2, 20001 * 64 + 5), (3, 16400)]


@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s)))
def test_long_rows_of_equal_values(gemm_mod, shape):
    """1 + 2^-10: added one at a time, sums beyond 2^14 lose the 2^-10 each time."""
    X = torch.full(shape, 1 + 2.0 ** -10, dtype=torch.float16, device="cuda")
    mean, rstd = (torch.empty(shape[0], device="cuda") for _ in range(2))
    Y = torch.empty_like(X)
    gemm_mod.layer_norm(X, Y, mean=mean, rstd=rstd, eps=1.0)
    off = (1 + 2.0 ** -10) * 2.0 ** -18
    assert bool(((mean.double() - (1 + 2.0 ** -10)).abs() <= off).all())
    assert bool((rstd.double() - 1).abs().max() <= 2.0 ** -22)
    assert float(Y.abs().max()) <= off * 1.01
    # the variance: 1 + 2^-10 and its negative in turn, mean 0, rstd = 1 / (1 + 2^-10)
    X[:, 1::2] *= -1
    if shape[1] % 2 == 0:
        gemm_mod.layer_norm(X, Y, mean=mean, rstd=rstd, eps=0.0)
        assert not mean.any()
        assert bool((rstd.double() * (1 + 2.0 ** -10) - 1).abs().max() <= 2.0 ** -18)


@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s)))
def test_gradient_of_long_rows(gemm_mod, shape):
    """g = c and n in turn 1 and -1 but for a level: mean(g) = c and mean(g n) = 0 leave
    dX = 0; with g = c n they leave c n - n c = 0. (c = 1 + 2^-10.)"""
    rows, n = shape
    c = 1 + 2.0 ** -10
    H = torch.ones(rows, n, dtype=torch.float16, device="cuda")
    H[:, 1::2] = -1
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dX = torch.empty_like(H)
    for dY in (torch.full_like(H, c), H * c):
        g, h = dY.double(), H.double()
        want = g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True)
        gemm_mod.layer_norm_grad(dY, H, mean, rstd, dX)
        # terms of c: g, mean(g) and n mean(g n); then one rounding to 16 bits
        bound = 2.0 ** -17 * 3 * c + want.abs() * 2.0 ** -11 + 2.0 ** -25
        assert bool(((dX.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s)))
def test_root_mean_square_of_long_rows(gemm_mod, shape):
    rows, n = shape
    c = 1 + 2.0 ** -10
    X = torch.full(shape, c, dtype=torch.float16, device="cuda")
    rstd, Y = torch.empty(rows, device="cuda"), torch.empty_like(X)
    gemm_mod.rms_norm(X, Y, rstd=rstd, eps=0.0)
    # half the sum of squares' 2^-18, and rsqrt's and the quotient's roundings
    assert bool((rstd.double() * c - 1).abs().max() <= 2.0 ** -19 + 2.0 ** -22)
    dX = torch.empty_like(X)
    rstd.fill_(1 / c)
    gemm_mod.rms_norm_grad(X, X, rstd, dX)  # g = c, n = 1: dX = (c - mean(c)) / c
    assert float(dX.abs().max()) <= 2.0 ** -17 * 2 + 2.0 ** -22
