"""The feed-forward block's 8-bit weights: rows that hold no values, weights that
change between calls. The bound of the 8-bit forward pass is that of the block's
other tests: 0.08 of the second product's norm plus the 16-bit roundings."""
import numpy as np
import pytest
import torch

from dense_gemm_row_gb300.feed_forward import FeedForward
from oracle import layers as L
from tests.layer_util import UNIT

pytestmark = pytest.mark.gpu


def near(ff, x, r, out):
    y, h, _ = L.rms_norm(L.to64(x), L.to64(ff.gain), L.to64(r), ff.eps)
    u, _ = L.linear(y, L.to64(ff.w1).T, 1.0, L.to64(ff.b1), ff.act)
    ref, _ = L.linear(u, L.to64(ff.w2).T, 1.0, L.to64(ff.b2), None, h)
    product = u @ L.to64(ff.w2).T
    return np.linalg.norm(L.to64(out) - ref) <= 0.08 * np.linalg.norm(product) \
        + 4 * UNIT[ff.dtype] * np.linalg.norm(ref)


@pytest.mark.parametrize("tokens", [3, 300])
@pytest.mark.parametrize("tiny", [0.0, 1e-36])
def test_rows_of_zeros(gemm_mod, tokens, tiny):
    ff = FeedForward(128, 264, "silu", seed=3)
    x, r = (torch.randn(tokens, 128, device="cuda").bfloat16() for _ in range(2))
    ff.w1[7] = tiny
    ff.w1[200:] = tiny
    assert near(ff, x, r, ff.forward8(x, r))


def test_weights_that_change_between_calls(gemm_mod):
    """forward8 works on the weights of the call: after a change in place, as a
    training step makes, and after new ones; weights quantised by the caller stay."""
    ff, other = FeedForward(128, 264, "silu", seed=3), FeedForward(128, 264, "silu", seed=3)
    x, r = (torch.randn(40, 128, device="cuda").bfloat16() for _ in range(2))
    kept, first = ff.quantise(), ff.forward8(x, r)
    ff.w1.neg_()
    other.w1.neg_()
    second = ff.forward8(x, r)
    assert near(ff, x, r, second) and torch.equal(second, other.forward8(x, r))
    ff.w1 = torch.randn_like(ff.w1) * 0.1
    assert near(ff, x, r, ff.forward8(x, r))
    assert torch.equal(ff.forward8(x, r, kept), first)
