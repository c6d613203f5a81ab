"""Main loops that take longer than the kernels' bound on a single wait (2 s): the result
is right and no wait is recorded as given up."""
import pytest
import torch

pytestmark = pytest.mark.gpu

LONG = 5 << 27  # 2^20 * 10 k-blocks of 64 by one pair of CTAs, 0.27 us each: 2.8 s
MOST = 2 ** 31 - 1  # 9 s
PLACES = [0, 63, 64, 12345678, 2 ** 29 + 7, LONG - 65, LONG - 1]


@pytest.fixture(autouse=True)
def clean_error_word(gemm_mod):
    gemm_mod.check_device_error()
    yield
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0
    torch.cuda.empty_cache()


def column(k):
    """A k x 1 matrix of zeros, ones at PLACES, in rows of 16 bytes. Used transposed it has
    one row, which the few-rows kernels do not take."""
    t = torch.zeros(8 * (k - 1) + 1, dtype=torch.bfloat16, device="cuda").as_strided((k, 1), (8, 1))
    for p in PLACES:
        t[p] = 1
    return t


def value(x):
    return torch.full((1, 1), x, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("k", [LONG, MOST])
def test_gated(gemm_mod, k):
    a, D, G, U = column(k), value(5), value(5), value(5)
    gemm_mod.gemm_gated(a, a, a, D, act="none", gate=G, up=U, trans_a=True)
    assert (D.item(), G.item(), U.item()) == (49, 7, 7)


def test_gradients(gemm_mod):
    a, D, dG, dU, s, t = column(LONG), value(5), value(5), value(5), value(5), value(5)
    gemm_mod.gemm_gated_dact(a, a, value(2), value(3), dG, dU, act="none", dbias_gate=s[0],
                             dbias_up=t[0], trans_a=True)
    assert (dG.item(), dU.item(), s.item(), t.item()) == (21, 14, 21, 14)
    gemm_mod.gemm_dact(a, a, None, D, dbias=s[0], trans_a=True)
    assert (D.item(), s.item()) == (7, 7)
