"""The linear-layer operators at the largest sizes that their entry points accept,
2^31 - 1 in each direction: round-ups of sizes must not leave 32 bits. Operands are
zeros with a few ones, so every result is known exactly."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BIG = 2 ** 31 - 1
PLACES = [0, 63, 64, 12345678, 2 ** 30 + 7, BIG - 130, BIG - 65, BIG - 2, BIG - 1]


@pytest.fixture(autouse=True)
def clean_error_word(gemm_mod):
    gemm_mod.check_device_error()
    yield
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0
    torch.cuda.empty_cache()


def zeros(n, dtype=torch.bfloat16):
    return torch.zeros(n, dtype=dtype, device="cuda")


def ones_at(n, dtype=torch.bfloat16):
    v = zeros(n, dtype)
    for p in PLACES:
        v[p] = 1
    return v


def check(v, value=1.0):
    """v holds `value` at PLACES and zeros elsewhere."""
    assert v[PLACES].tolist() == [value] * len(PLACES)
    for p in PLACES:
        v[p] = 0
    assert not any(bool(c.any()) for c in v.split(1 << 28))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "e4m3"])
def test_longest_inner_dimension(gemm_mod, dtype):
    if dtype is torch.bfloat16:
        a = ones_at(BIG)
    else:
        a = zeros(BIG, torch.uint8)
        for p in PLACES:
            a[p] = 0x38  # 1.0
        a = a.view(dtype)
    D = torch.full((1, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    gemm_mod.gemm_epilogue(a.view(1, BIG), a.view(1, BIG), D, trans_b=True)
    assert D.item() == len(PLACES)


def test_most_columns(gemm_mod):
    b, D = ones_at(BIG).view(1, BIG), torch.full((1, BIG), 7.0, dtype=torch.bfloat16, device="cuda")
    a = torch.full((1, 1), 3.0, dtype=torch.bfloat16, device="cuda")
    gemm_mod.gemm_epilogue(a, b, D)
    check(D[0], 3.0)


def test_most_rows(gemm_mod):
    a, D = ones_at(BIG).view(1, BIG), torch.full((BIG, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    b = torch.full((1, 1), 3.0, dtype=torch.bfloat16, device="cuda")
    gemm_mod.gemm_epilogue(a, b, D, trans_a=True)
    check(D[:, 0], 3.0)


def test_most_rows_of_a_gradient(gemm_mod):
    a, D = ones_at(BIG).view(1, BIG), torch.full((BIG, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    b, db = torch.full((1, 1), 3.0, dtype=torch.bfloat16, device="cuda"), zeros(1)
    gemm_mod.gemm_dact(a, b, None, D, dbias=db, trans_a=True)
    assert db.item() == 3 * len(PLACES)
    check(D[:, 0], 3.0)


@pytest.mark.parametrize("tall", [False, True])
def test_pointwise_gradient(gemm_mod, tall):
    d = ones_at(BIG).view(BIG, 1) if tall else ones_at(BIG).view(1, BIG)
    db = torch.full((d.shape[1],), 7.0, dtype=torch.bfloat16, device="cuda")
    gemm_mod.act_grad(d, d, d, act="relu", dbias=db)
    if tall:
        assert db.item() == len(PLACES)
    else:
        check(db)
    check(d.view(-1))
