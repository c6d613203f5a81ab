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
