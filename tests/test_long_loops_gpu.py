"""Main loops that take longer than the kernels' bound on a single wait (2 s): the result
is right, the calls behind it are, and no wait is recorded as given up."""
import pytest
import torch

from oracle import layers as L
from tests.layer_util import normal

pytestmark = pytest.mark.gpu

LONG = 3 << 28  # by one pair of CTAs 2.9 s
MOST = 2 ** 31 - 1  # 8 s
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


def quantised(g, rows, cols, block_rows, seed):
    q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(-(-rows // block_rows), cols // 128, device="cuda")
    g.quantise_blocks(normal((rows, cols), torch.bfloat16, seed), q, s, rows=block_rows)
    return q, s


@pytest.mark.parametrize("m", [20, 700], ids=["few rows", "tiles"])
@pytest.mark.parametrize("kind", ["plain", "block"])
def test_the_call_behind_a_long_one(gemm_mod, kind, m):
    """It starts while the long call still runs, on the other SMs, and waits for it."""
    g, n, k = gemm_mod, 512, 1024
    D, want = (torch.zeros(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    if kind == "plain":
        A, B = normal((m, k), torch.bfloat16, 1), normal((n, k), torch.bfloat16, 2)

        def call(D):
            g.gemm_epilogue(A, B, D, trans_b=True)
    else:
        (A, sa), (B, sb) = quantised(g, m, k, 1, 1), quantised(g, n, k, 128, 2)

        def call(D):
            g.gemm_epilogue(A, B, D, trans_b=True, scale_a=sa, scale_b=sb)
    a, one = column(LONG), value(5)
    call(want)
    torch.cuda.synchronize()
    g.gemm_epilogue(a, a, one, trans_a=True)
    call(D)
    torch.cuda.synchronize()
    assert one.item() == 7 and torch.equal(D, want) and L.to64(want).any()
