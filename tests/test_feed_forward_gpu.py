"""The feed-forward block that runs the linear-layer operators together, against
the same block in float64.

The block rounds to 16 bits after every operator, so its results are compared in
norm. Forward: y, u and out are each rounded (unit roundoff u, errors add in
quadrature at most linearly: 4 u with the operators' slopes). The gradients are
those at the saved values (what the backward pass is a function of: at the exact
pre-activations relu's slope would be another one wherever rounding crossed its
step) and carry the roundings of dz and dy: 8 u. 8-bit inference adds
one e4m3 rounding (2^-4 relative at most, 2^-5.3 in the mean) of both operands of
the widening product: 0.08 of the product's own norm, while out also contains the
exact residual.
"""
import numpy as np
import pytest
import torch

from dense_gemm_row_gb300.feed_forward import FeedForward, main
from oracle import layers as L
from tests.layer_util import DTYPES, UNIT

pytestmark = pytest.mark.gpu


def block64(ff, x, r, dout, saved):
    x, r, dout = L.to64(x), L.to64(r), L.to64(dout)
    gain, w1, b1, w2, b2 = (L.to64(getattr(ff, n)) for n in ("gain", "w1", "b1", "w2", "b2"))
    y, h, rstd = L.rms_norm(x, gain, r, ff.eps)
    u, z = L.linear(y, w1.T, 1.0, b1, ff.act)
    out, _ = L.linear(u, w2.T, 1.0, b2, None, h)
    product = u @ w2.T
    h, rstd, y, z, u = (L.to64(t) for t in saved)
    dz, db1 = L.linear_grad(dout @ w2, z, ff.act)
    dx, dgain = L.rms_norm_grad(dz @ w1, h, rstd, gain, dout)
    return out, {"b2": dout.sum(0), "w2": dout.T @ u, "b1": db1, "w1": dz.T @ y, "gain": dgain,
                 "x": dx}, product


def off(got, ref):
    return np.linalg.norm(L.to64(got) - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("tokens,model,hidden,act", [(1, 256, 1024, "silu"), (48, 128, 520, "relu"),
                                                     (333, 264, 1000, "gelu"),
                                                     (700, 512, 2048, "gelu_tanh")])
def test_block(gemm_mod, tokens, model, hidden, act, dtype):
    ff = FeedForward(model, hidden, act, dtype, seed=tokens)
    x, r, dout = (torch.randn(tokens, model, device="cuda").to(dtype) for _ in range(3))
    out, saved = ff.forward(x, r)
    grads = ff.backward(dout, saved)
    out8 = ff.forward8(x, r)
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0
    ref, ref_grads, product = block64(ff, x, r, dout, saved)
    u = UNIT[dtype]
    assert off(out, ref) <= 4 * u
    for name, want in ref_grads.items():
        assert off(grads[name], want) <= 8 * u, name
    assert np.linalg.norm(L.to64(out8) - ref) <= 0.08 * np.linalg.norm(product) \
        + 4 * u * np.linalg.norm(ref)


def test_command_prints_a_line(gemm_mod, capsys):
    main(["--tokens", "128", "--model", "256", "--hidden", "512"])
    assert '"step_tflops"' in capsys.readouterr().out
