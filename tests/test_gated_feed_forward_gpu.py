"""The gated feed-forward block that runs its operators together (layer norm, gated
product and its gradient, quantisation, block-scaled products), against the same block
in float64.

Compared in norm, as the block rounds to 16 bits after every operator. Forward: y, u
and out are rounded (4 u with the operators' slopes). Gradients are those at the saved
values and carry the roundings of dgate, dup and twice of dy: 8 u. 8-bit inference:
an e4m3 rounding is at most 2^-4 relative, 0.036 in the mean square (uniform within
it), so a product of two rounded operands is off by 0.051 of its norm; act(G) U by
0.051 from U and at most 0.051 * 1.13 |G| / |act(G)|, 0.1, from G; the last product
adds 0.051: 0.12 in quadrature, bounded by 0.15 of the product's norm.
"""
import numpy as np
import pytest
import torch

from dense_gemm_row_gb300.feed_forward import GatedFeedForward, main
from oracle import layers as L
from tests.layer_util import DTYPES, UNIT

pytestmark = pytest.mark.gpu

CASES = [(1, 256, 1024, "silu"), (48, 128, 520, "relu"), (333, 264, 1000, "gelu"),
         (700, 512, 2048, "gelu_tanh")]


def block64(ff, x, r, dout=None, saved=None):
    x, r = L.to64(x), L.to64(r)
    gain, shift, wg, wu, wd = (L.to64(getattr(ff, n)) for n in ("gain", "shift", "wg", "wu", "wd"))
    y, h, _, _ = L.layer_norm(x, gain, shift, r, ff.eps)
    product = L.gated(y, wg.T, wu.T, act_name=ff.act)[0] @ wd.T
    if saved is None:
        return product + h, product
    dout = L.to64(dout)
    h, mean, rstd, y, gate, up, u = (L.to64(t) for t in saved)
    dg, du, _, _ = L.gated_grad(dout @ wd, gate, up, ff.act)
    dx, dgain, dshift = L.layer_norm_grad(dg @ wg + du @ wu, h, mean, rstd, gain, dout)
    return {"wd": dout.T @ u, "wg": dg.T @ y, "wu": du.T @ y, "gain": dgain, "shift": dshift,
            "x": dx}


def off(got, ref):
    return np.linalg.norm(L.to64(got) - ref) / np.linalg.norm(ref)


def near8(ff, x, r, out):
    ref, product = block64(ff, x, r)
    return np.linalg.norm(L.to64(out) - ref) <= 0.15 * np.linalg.norm(product) \
        + 4 * UNIT[ff.dtype] * np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("tokens,model,hidden,act", CASES)
def test_block(gemm_mod, tokens, model, hidden, act, dtype):
    ff = GatedFeedForward(model, hidden, act, dtype, seed=tokens)
    ff.gain += 0.1 * torch.randn_like(ff.gain)
    ff.shift += 0.1 * torch.randn_like(ff.shift)
    x, r, dout = (torch.randn(tokens, model, device="cuda").to(dtype) for _ in range(3))
    out, saved = ff.forward(x, r)
    grads = ff.backward(dout, saved)
    out8 = ff.forward8(x, r)
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0
    u = UNIT[dtype]
    assert off(out, block64(ff, x, r)[0]) <= 4 * u
    for name, want in block64(ff, x, r, dout, saved).items():
        assert off(grads[name], want) <= 8 * u, name
    assert near8(ff, x, r, out8)


@pytest.mark.parametrize("tokens", [3, 300])
def test_8_bit_weights_that_change_between_calls(gemm_mod, tokens):
    """forward8 works on the weights of the call; weights quantised by the caller stay.
    Blocks of zeros and rows of tiny values among them."""
    ff = GatedFeedForward(264, 400, seed=3)
    x, r = (torch.randn(tokens, 264, device="cuda").bfloat16() for _ in range(2))
    ff.wu[:128, :128] = 0
    ff.wg[200:] = 1e-36
    kept, first = ff.quantise(), ff.forward8(x, r)
    assert near8(ff, x, r, first)
    ff.wd.neg_()
    assert near8(ff, x, r, ff.forward8(x, r))
    assert torch.equal(ff.forward8(x, r, kept), first)


def test_a_captured_training_step(gemm_mod):
    """Forward, backward and 8-bit forward in one graph, replayed on new inputs while
    results of eager calls are alive: the same bits."""
    ff = GatedFeedForward(264, 520, seed=1)
    x, r, dout = (torch.zeros(300, 264, dtype=torch.bfloat16, device="cuda") for _ in range(3))

    def step():
        out, saved = ff.forward(x, r)
        return [out, ff.forward8(x, r), *ff.backward(dout, saved).values()]

    eager = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        captured = step()
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x, r, dout):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
        assert not torch.equal(eager[0], want[0])
    assert gemm_mod.check_device_error() == 0


def test_command_prints_a_line(gemm_mod, capsys):
    main(["--tokens", "128", "--model", "256", "--hidden", "512", "--gated", "--act", "silu"])
    line = capsys.readouterr().out
    assert '"step_tflops"' in line and '"gated": true' in line


def test_every_operator_on_a_stream_of_the_caller(gemm_mod):
    """stream=: the work runs there, behind what that stream holds and unordered with the
    current one; the bits of calls on the current stream."""
    g, bf = gemm_mod, torch.bfloat16
    x, w = (torch.randn(300, 256, device="cuda").to(bf) for _ in range(2))
    side = torch.cuda.Stream()

    def run(x, stream=None):
        new = lambda *shape, dtype=bf: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
        f32, e4 = torch.float32, torch.float8_e4m3fn
        y, mean, rstd = new(300, 256), new(300, dtype=f32), new(300, dtype=f32)
        D, G, U, dG, dU = (new(300, 300) for _ in range(5))
        dX, dw, db, sg, su = new(300, 256), new(256), new(256), new(300), new(300)
        y8, w8, sy, sw = new(300, 256, dtype=e4), new(300, 256, dtype=e4), new(300, 2, dtype=f32), \
            new(3, 2, dtype=f32)
        D8, Z8 = new(300, 300), new(300, 300)
        g.layer_norm(x, y, mean=mean, rstd=rstd, stream=stream)
        g.gemm_gated(y, w, w, D, gate=G, up=U, trans_b=True, stream=stream)
        g.gemm_gated_dact(x, w, G, U, dG, dU, dbias_gate=sg, dbias_up=su, trans_b=True,
                          stream=stream)
        g.layer_norm_grad(y, x, mean, rstd, dX, dweight=dw, dbias=db, stream=stream)
        g.quantise_blocks(y, y8, sy, stream=stream)
        g.quantise_blocks(w, w8, sw, rows=128, stream=stream)
        g.gemm_gated(y8, w8, w8, D8, trans_b=True, scale_a=sy, scale_gate=sw, scale_up=sw,
                     stream=stream)
        g.gemm_epilogue(y8, w8, Z8, trans_b=True, scale_a=sy, scale_b=sw, stream=stream)
        return [y, mean, rstd, D, G, U, dG, dU, sg, su, dX, dw, db, sy, sw, D8, Z8,
                y8.view(torch.uint8), w8.view(torch.uint8)]

    want = run(x)
    late = torch.zeros_like(x)  # holds x only once the side stream gets there
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(x)
    got = run(late, side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert g.check_device_error() == 0
