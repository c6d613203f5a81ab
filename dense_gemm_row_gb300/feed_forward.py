"""Pre-norm feed-forward blocks made of the linear-layer operators: a training
step (forward and backward) and 8-bit inference.

    h = x + r                      residual stream
    y = rms_norm(h) * gain
    u = act(y W1^T + b1)
    out = u W2^T + b2 + h

and the gated one, whose 8-bit form has a scale for each block of 128 values:

    y = layer_norm(h) * gain + shift
    u = act(y Wg^T) * (y Wu^T)
    out = u Wd^T + h

    python -m dense_gemm_row_gb300.feed_forward [--tokens 4096] [--model 4096] [--hidden 16384]
        [--act gelu_tanh] [--dtype bf16] [--gated]

runs a training step and an 8-bit forward pass on random data and prints one JSON
line with their times. Weights are stored as layers usually are, (outputs,
inputs): op T of the products.
"""
from __future__ import annotations

import argparse
import json

import torch

from . import binding as g


class FeedForward:
    """Weights of one block (gain, w1, b1, w2, b2); every call works on torch's current
    stream and allocates what it returns."""

    def __init__(self, model: int, hidden: int, act: str = "gelu_tanh",
                 dtype: torch.dtype = torch.bfloat16, eps: float = 1e-6, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def draw(*shape, std):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

        self.model, self.hidden, self.act, self.dtype, self.eps = model, hidden, act, dtype, eps
        self.gain = torch.ones(model, dtype=dtype, device="cuda")
        self.w1, self.b1 = draw(hidden, model, std=model ** -0.5), draw(hidden, std=0.02)
        self.w2, self.b2 = draw(model, hidden, std=hidden ** -0.5), draw(model, std=0.02)

    def _new(self, *shape, dtype=None):
        return torch.empty(*shape, dtype=dtype or self.dtype, device="cuda")

    def forward(self, x, r):
        """(out, saved) for x and r (tokens x model); saved is what backward needs."""
        m = x.shape[0]
        h, y = self._new(m, self.model), self._new(m, self.model)
        rstd = self._new(m, dtype=torch.float32)
        g.rms_norm(x, y, weight=self.gain, residual=r, h=h, rstd=rstd, eps=self.eps)
        z, u = self._new(m, self.hidden), self._new(m, self.hidden)
        g.gemm_epilogue(y, self.w1, u, bias=self.b1, act=self.act, preact=z, trans_b=True)
        out = self._new(m, self.model)
        g.gemm_epilogue(u, self.w2, out, bias=self.b2, residual=h, trans_b=True)
        return out, (h, rstd, y, z, u)

    def backward(self, dout, saved):
        """Gradients from dout: a dict of dx (of x and r alike) and each weight's."""
        h, rstd, y, z, u = saved
        m = dout.shape[0]
        grads = {n: torch.empty_like(getattr(self, n)) for n in ("gain", "w1", "b1", "w2", "b2")}
        # out = u W2^T + b2 + h
        g.act_grad(dout, None, None, dbias=grads["b2"])
        g.gemm_epilogue(dout, u, grads["w2"], trans_a=True)
        # u = act(z): the gradient comes back through W2 with act' in the epilogue
        dz = self._new(m, self.hidden)
        g.gemm_dact(dout, self.w2, z, dz, act=self.act, dbias=grads["b1"])
        g.gemm_epilogue(dz, y, grads["w1"], trans_a=True)
        dy = self._new(m, self.model)
        g.gemm_epilogue(dz, self.w1, dy)
        # the norm, plus the gradient that reaches h past it
        dx = self._new(m, self.model)
        g.rms_norm_grad(dy, h, rstd, dx, weight=self.gain, dh=dout, dweight=grads["gain"])
        grads["x"] = dx
        return grads

    def quantise(self):
        """W1 as e4m3 values and a scale per output (row), for forward8. As in the norm, a
        row whose largest value is below 1e-30 counts as zeros, with scale 0."""
        top = self.w1.float().abs().amax(1)
        scale = torch.where(top < 1e-30, torch.zeros_like(top), top / 448)
        inverse = torch.where(top < 1e-30, torch.zeros_like(top), 448 / top)
        ld = -(-self.model // 16) * 16  # rows in whole 16-byte units
        q = torch.zeros(self.hidden, ld, dtype=torch.float8_e4m3fn, device="cuda")[:, :self.model]
        q.copy_((self.w1.float() * inverse[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn))
        return q, scale

    def forward8(self, x, r, weights=None):
        """out with the widening layer in 8 bits: the norm writes e4m3 values and a
        scale per token, the product reads them as stored. weights: what quantise()
        returned, which a program whose weights no longer change keeps; None quantises
        W1 as it is now."""
        m = x.shape[0]
        q, scale = self.quantise() if weights is None else weights
        h = self._new(m, self.model)
        y8 = self._new(m, q.stride(0) if self.hidden > 1 else self.model,
                       dtype=torch.float8_e4m3fn)[:, :self.model]
        s = self._new(m, dtype=torch.float32)
        g.rms_norm(x, y8, weight=self.gain, residual=r, h=h, scale=s, eps=self.eps)
        u, out = self._new(m, self.hidden), self._new(m, self.model)
        g.gemm_epilogue(y8, q, u, bias=self.b1, act=self.act, scale_a=s, scale_b=scale,
                        trans_b=True)
        g.gemm_epilogue(u, self.w2, out, bias=self.b2, residual=h, trans_b=True)
        return out


class GatedFeedForward:
    """Weights of one gated block (gain, shift, wg, wu, wd); calls as FeedForward's."""

    def __init__(self, model: int, hidden: int, act: str = "silu",
                 dtype: torch.dtype = torch.bfloat16, eps: float = 1e-5, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def draw(rows, cols):
            return (torch.randn(rows, cols, generator=gen, device="cuda") * cols ** -0.5).to(dtype)

        self.model, self.hidden, self.act, self.dtype, self.eps = model, hidden, act, dtype, eps
        self.gain = torch.ones(model, dtype=dtype, device="cuda")
        self.shift = torch.zeros(model, dtype=dtype, device="cuda")
        self.wg, self.wu = draw(hidden, model), draw(hidden, model)
        self.wd = draw(model, hidden)

    def _new(self, *shape, dtype=None):
        return torch.empty(*shape, dtype=dtype or self.dtype, device="cuda")

    def forward(self, x, r):
        """(out, saved) for x and r (tokens x model); saved is what backward needs."""
        m = x.shape[0]
        h, y = self._new(m, self.model), self._new(m, self.model)
        mean, rstd = (self._new(m, dtype=torch.float32) for _ in range(2))
        g.layer_norm(x, y, weight=self.gain, bias=self.shift, residual=r, h=h, mean=mean,
                     rstd=rstd, eps=self.eps)
        gate, up, u = (self._new(m, self.hidden) for _ in range(3))
        g.gemm_gated(y, self.wg, self.wu, u, act=self.act, gate=gate, up=up, trans_b=True)
        out = self._new(m, self.model)
        g.gemm_epilogue(u, self.wd, out, residual=h, trans_b=True)
        return out, (h, mean, rstd, y, gate, up, u)

    def backward(self, dout, saved):
        """Gradients from dout: a dict of dx (of x and r alike) and each weight's."""
        h, mean, rstd, y, gate, up, u = saved
        m = dout.shape[0]
        grads = {n: torch.empty_like(getattr(self, n)) for n in ("gain", "shift", "wg", "wu", "wd")}
        g.gemm_epilogue(dout, u, grads["wd"], trans_a=True)
        # u = act(gate) * up: the gradient comes back through Wd, both factors' in the epilogue
        dgate, dup = self._new(m, self.hidden), self._new(m, self.hidden)
        g.gemm_gated_dact(dout, self.wd, gate, up, dgate, dup, act=self.act)
        g.gemm_epilogue(dgate, y, grads["wg"], trans_a=True)
        g.gemm_epilogue(dup, y, grads["wu"], trans_a=True)
        dy = self._new(m, self.model)
        g.gemm_epilogue(dgate, self.wg, dy)
        g.gemm_epilogue(dup, self.wu, dy, residual=dy)
        # the norm, plus the gradient that reaches h past it
        dx = self._new(m, self.model)
        g.layer_norm_grad(dy, h, mean, rstd, dx, weight=self.gain, dh=dout, dweight=grads["gain"],
                          dbias=grads["shift"])
        grads["x"] = dx
        return grads

    def _blocks(self, t, rows):
        """t in 8 bits with a scale per block of rows x 128, rows in whole 16-byte units."""
        m, n = t.shape
        q = self._new(m, -(-n // 16) * 16, dtype=torch.float8_e4m3fn)[:, :n]
        scale = self._new(-(-m // rows), -(-n // 128), dtype=torch.float32)
        g.quantise_blocks(t, q, scale, rows=rows)
        return q, scale

    def quantise(self):
        """The three weight matrices in 8 bits, (values, scales) each, for forward8."""
        return tuple(self._blocks(w, 128) for w in (self.wg, self.wu, self.wd))

    def forward8(self, x, r, weights=None):
        """out with all three products in 8 bits. weights: what quantise() returned, which
        a program whose weights no longer change keeps; None quantises them as they are
        now."""
        m = x.shape[0]
        (wg, sg), (wu, su), (wd, sd) = self.quantise() if weights is None else weights
        h, y = self._new(m, self.model), self._new(m, self.model)
        g.layer_norm(x, y, weight=self.gain, bias=self.shift, residual=r, h=h, eps=self.eps)
        y8, sy = self._blocks(y, 1)
        u, out = self._new(m, self.hidden), self._new(m, self.model)
        g.gemm_gated(y8, wg, wu, u, act=self.act, trans_b=True, scale_a=sy, scale_gate=sg,
                     scale_up=su)
        u8, s = self._blocks(u, 1)
        g.gemm_epilogue(u8, wd, out, residual=h, trans_b=True, scale_a=s, scale_b=sd)
        return out


def _time_us(f, iters=10):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    for _ in range(iters):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e3 / iters


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--model", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=16384)
    ap.add_argument("--act", default="gelu_tanh", choices=["none", "relu", "gelu", "gelu_tanh",
                                                           "silu"])
    ap.add_argument("--dtype", default="bf16", choices=["bf16", "f16"])
    ap.add_argument("--gated", action="store_true", help="the gated block")
    a = ap.parse_args(argv)
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float16
    ff = (GatedFeedForward if a.gated else FeedForward)(a.model, a.hidden, a.act, dtype)
    x, r, dout = (torch.randn(a.tokens, a.model, device="cuda").to(dtype) for _ in range(3))
    _, saved = ff.forward(x, r)
    flops = (3 if a.gated else 2) * a.tokens * a.model * a.hidden
    fwd, bwd = _time_us(lambda: ff.forward(x, r)), _time_us(lambda: ff.backward(dout, saved))
    weights = ff.quantise()
    fwd8 = _time_us(lambda: ff.forward8(x, r, weights))
    g.check_device_error()
    print(json.dumps({
        "tokens": a.tokens, "model": a.model, "hidden": a.hidden, "act": a.act, "dtype": a.dtype,
        "gated": a.gated,
        "forward_us": round(fwd, 1), "backward_us": round(bwd, 1), "forward8_us": round(fwd8, 1),
        "step_tflops": round(6 * flops / (fwd + bwd) / 1e6, 1)}))


if __name__ == "__main__":
    main()
