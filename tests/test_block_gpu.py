"""GPU parity of the block-scaled e4m3 products (gemm_epilogue and gemm_gated with
scales per block of 128) and of quantise_blocks against the float64 oracle.

Tolerances. A block's sum has at most 128 exact products, added by the tensor cores
(each addition off by at most 2^-23 of the running magnitudes), and the blocks are
added in fp32 with a rounding of the scale product and one per block: within
(min(K, 128) + blocks + 8) 2^-23 of the sum of scaled magnitudes. The epilogue as in
tests/test_linear_gpu.py and test_gated_gpu.py. quantise_blocks: the scale is one
division; a value is x times 448 / max, both rounded, so within one rounding of the
e4m3 grid (2^-4 relative, or half the subnormal step) and 2^-22 of x / scale, and it
differs from the oracle's only within that of a boundary.
"""
import numpy as np
import pytest
import torch

from oracle import layers as L
from tests.layer_util import DTYPES, Out, act_error, assert_close, normal, rounded_bound

pytestmark = pytest.mark.gpu

MAX_SLOPE = 1.13
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(autouse=True)
def clean_error_word(gemm_mod):
    gemm_mod.check_device_error()
    yield
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0


def operand(rows, cols, block_rows, seed, std=1.0, scale_pad=0):
    """(q, scale): e4m3 values whose rows differ in size, padding NaN; scales in rows
    `scale_pad` longer, padding NaN. No kernel of the library takes part."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * std
    x = x * torch.exp(0.5 * torch.randn(rows, 1, generator=g))
    q, s = L.quantise_blocks(x.double().numpy(), block_rows)
    buf = torch.full((max(rows, 1), -(-cols // 16) * 16 + 16), 0x7f, dtype=torch.uint8)
    buf[:rows, :cols] = torch.from_numpy(q).float().to(torch.float8_e4m3fn).view(torch.uint8)
    sbuf = torch.full((max(s.shape[0], 1), s.shape[1] + scale_pad), float("nan"))
    sbuf[:s.shape[0], :s.shape[1]] = torch.from_numpy(s).float()
    return (buf.cuda().view(torch.float8_e4m3fn)[:rows, :cols],
            sbuf.cuda()[:s.shape[0], :s.shape[1]])


def value(q, s, block_rows):
    return L.to64(q) * L.spread(L.to64(s), block_rows, q.shape)


def product(A64, B64, alpha):
    """(alpha A B^T, its bound)."""
    k = A64.shape[1]
    rel = (min(k, 128) + -(-k // 128) + 8) * 2.0 ** -23
    return alpha * (A64 @ B64.T), rel * abs(alpha) * (np.abs(A64) @ np.abs(B64).T)


def run_block(g, m, n, k, dtype, act="none", bias=True, residual=True, preact=True, alpha=1.0,
              pad=0, shift=0, inplace=False, scale_pad=0, seed=0):
    A, sa = operand(m, k, 1, seed + 1, scale_pad=scale_pad)
    B, sb = operand(n, k, 128, seed + 2, max(k, 1) ** -0.5, scale_pad)
    b = normal((1, n), dtype, seed + 3)[0] if bias else None
    R = normal((m, n), dtype, seed + 4, pad=pad) if residual else None
    r64 = L.to64(R) if residual else None
    D = Out(m, n, dtype, pad, shift)
    Z = Out(m, n, dtype, pad, shift) if preact else None
    if residual and inplace:
        D.t.copy_(R)
        R = D.t
    g.gemm_epilogue(A, B, D.t, alpha=alpha, bias=b, act=act, residual=R,
                    preact=Z.t if Z else None, trans_b=True, scale_a=sa, scale_b=sb)
    torch.cuda.synchronize()
    z, ez = product(value(A, sa, 1), value(B, sb, 128), alpha)
    if bias:
        z = z + L.to64(b)
    ez = ez + 2.0 ** -23 * np.abs(z)
    d = L.act(z, act) + (r64 if residual else 0)
    ed = MAX_SLOPE * ez + act_error(z, act) + 2.0 ** -23 * np.abs(d)
    assert_close(L.to64(D.t), d, rounded_bound(d, ed, dtype), "D")
    D.check_guards()
    if Z:
        assert_close(L.to64(Z.t), z, rounded_bound(z, ez, dtype), "Z")
        Z.check_guards()


def run_gated(g, m, n, k, dtype, act="silu", bias=(True, True), keep=(True, True), alpha=1.0, pad=0,
              shift=0, scale_pad=0, seed=0):
    A, sa = operand(m, k, 1, seed + 1, scale_pad=scale_pad)
    Bg, sg = operand(n, k, 128, seed + 2, max(k, 1) ** -0.5, scale_pad)
    Bu, su = operand(n, k, 128, seed + 3, max(k, 1) ** -0.5, scale_pad)
    bias = [normal((1, n), dtype, seed + 4 + i)[0] if b else None for i, b in enumerate(bias)]
    D = Out(m, n, dtype, pad, shift)
    kept = [Out(m, n, dtype, pad, shift) if want else None for want in keep]
    g.gemm_gated(A, Bg, Bu, D.t, act=act, alpha=alpha, bias_gate=bias[0], bias_up=bias[1],
                 gate=kept[0].t if kept[0] else None, up=kept[1].t if kept[1] else None,
                 trans_b=True, scale_a=sa, scale_gate=sg, scale_up=su)
    torch.cuda.synchronize()
    a64 = value(A, sa, 1)
    (gz, eg), (uz, eu) = (product(a64, value(B, s, 128), alpha) for B, s in ((Bg, sg), (Bu, su)))
    gz, uz = (z if b is None else z + L.to64(b) for z, b in zip((gz, uz), bias))
    eg, eu = eg + 2.0 ** -23 * np.abs(gz), eu + 2.0 ** -23 * np.abs(uz)
    a = L.act(gz, act)
    d = a * uz
    ed = (MAX_SLOPE * eg + act_error(gz, act)) * (np.abs(uz) + eu) + np.abs(a) * eu \
        + 2.0 ** -23 * np.abs(d)
    assert_close(L.to64(D.t), d, rounded_bound(d, ed, dtype), "D")
    D.check_guards()
    for o, z, e, what in zip(kept, (gz, uz), (eg, eu), "GU"):
        if o:
            assert_close(L.to64(o.t), z, rounded_bound(z, e, dtype), what)
            o.check_guards()


# Sizes around the tiles' and the few-rows kernel's edges, one k-block with and
# without a remainder, more k-blocks than accumulators and stages, odd everything.
SHAPES = [(1, 1, 1), (1, 64, 128), (1, 4096, 512), (2, 129, 130), (5, 250, 1000), (16, 1024, 2048),
          (17, 2048, 136), (33, 520, 1200), (64, 640, 4096), (65, 130, 72), (100, 1111, 513),
          (128, 256, 64), (129, 257, 127), (200, 384, 4096), (255, 1023, 520), (256, 512, 1024),
          (257, 255, 63), (384, 4096, 128), (513, 777, 1023), (1000, 300, 2000), (1500, 2700, 1280)]


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(gemm_mod, shape, dtype):
    i = SHAPES.index(shape)
    run_block(gemm_mod, *shape, dtype, ACTS[i % 5], bias=i % 3 != 0, residual=i % 2 == 0,
              preact=i % 4 != 1, scale_pad=i % 3, seed=i)
    run_gated(gemm_mod, *shape, dtype, ACTS[-i % 5], bias=(i % 3 != 0, i % 3 != 1),
              keep=(i % 4 != 1, i % 4 != 2), scale_pad=-i % 4, seed=i)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [7, 150, 600])
def test_activations(gemm_mod, act, m):
    for dtype in DTYPES.values():
        run_block(gemm_mod, m, 264, 400, dtype, act, alpha=3.0, seed=m)
        run_gated(gemm_mod, m, 264, 400, dtype, act, alpha=-3.0, seed=m)


@pytest.mark.parametrize("shift,pad", [(0, 0), (0, 8), (0, 3), (1, 0), (8, 1), (3, 5)])
@pytest.mark.parametrize("m", [9, 140, 520])
def test_output_layouts(gemm_mod, m, shift, pad):
    for mask in range(8):
        run_block(gemm_mod, m, 272, 300, torch.bfloat16, "relu", bias=False,
                  residual=bool(mask & 1), preact=bool(mask & 2), inplace=bool(mask & 4), pad=pad,
                  shift=shift, seed=mask)
        run_gated(gemm_mod, m, 272, 300, torch.float16, "gelu", keep=(bool(mask & 1), bool(mask & 2)),
                  bias=(bool(mask & 4), False), pad=pad, shift=shift, seed=mask)


@pytest.mark.parametrize("m", [5, 700])
def test_several_tiles_per_pair_with_everything(gemm_mod, m):
    run_block(gemm_mod, m, 9000, 260, torch.bfloat16, "gelu_tanh", seed=1)
    run_block(gemm_mod, m, 9000, 260, torch.float16, "none", preact=False, seed=2)
    run_gated(gemm_mod, m, 9000, 260, torch.bfloat16, seed=3)


@pytest.mark.parametrize("shape", [(0, 40, 16), (3, 0, 16), (3, 40, 0), (300, 136, 0)],
                         ids=lambda s: "x".join(map(str, s)))
def test_empty(gemm_mod, shape):
    run_block(gemm_mod, *shape, torch.bfloat16, "silu")
    run_gated(gemm_mod, *shape, torch.float16)


@pytest.mark.parametrize("m", [20, 400])
def test_scales_far_apart_and_special(gemm_mod, m):
    """Blocks whose scales differ by 2^40, a block with scale 0 (of zeros), and a row
    and a block of columns with a NaN scale: each stays where it belongs."""
    n, k, dtype = 300, 640, torch.bfloat16
    A, sa = operand(m, k, 1, 1)
    B, sb = operand(n, k, 128, 2, k ** -0.5)
    sa[:, 1] *= 2.0 ** -40
    sa[:, 3] *= 2.0 ** 20
    sb[1, 2] = 0
    A64, B64 = value(A, sa, 1), value(B, sb, 128)
    D = Out(m, n, dtype)
    gemm_mod.gemm_epilogue(A, B, D.t, trans_b=True, scale_a=sa, scale_b=sb)
    torch.cuda.synchronize()
    z, e = product(A64, B64, 1.0)
    assert_close(L.to64(D.t), z, rounded_bound(z, e, dtype), "D")
    clean = D.t.clone()
    sa[m // 2, 4] = float("nan")
    sb[2, 0] = float("inf")
    gemm_mod.gemm_epilogue(A, B, D.t, trans_b=True, scale_a=sa, scale_b=sb)
    torch.cuda.synchronize()
    rows = [i for i in range(m) if i != m // 2]
    assert bool(D.t[m // 2].isnan().all()) and not bool(D.t[:, 256:].isfinite().any())
    assert torch.equal(D.t[rows, :256], clean[rows, :256])
    D.check_guards()


QUANT = [(1, 1), (1, 128), (3, 129), (127, 4096), (128, 128), (129, 1000), (200, 255), (1000, 513),
         (1001, 4095), (2, 20001), (3000, 264)]


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("shape", QUANT, ids=lambda s: "x".join(map(str, s)))
def test_quantise(gemm_mod, shape, rows, dtype):
    m, n = shape
    i = QUANT.index(shape)
    for xpad, ypad, shift in ((0, 0, 0), (-n % 8, -n % 16, 0), (3, 5, 1), (8, 16, 8)):
        X = Out(m, n, dtype, xpad, shift)
        X.t.copy_(normal(shape, dtype, i, 3.0))
        if m > 2 and n > 128:
            X.t[1, :128] = 0
        Y = Out(m, n, torch.float8_e4m3fn, ypad, shift)
        scale = Out(-(-m // rows), -(-n // 128), torch.float32, xpad)
        gemm_mod.quantise_blocks(X.t, Y.t, scale.t, rows=rows)
        torch.cuda.synchronize()
        x = L.to64(X.t)
        q, s = L.quantise_blocks(x, rows)
        assert_close(L.to64(scale.t), s, 2.0 ** -24 * s, "scale")
        wide, got = L.spread(s, rows, shape), L.to64(Y.t)
        assert_close(got * wide, x, (2.0 ** -4 + 2.0 ** -21) * np.abs(x) + wide * 2.0 ** -10, "Y")
        ratio = x / np.where(wide == 0, 1, wide)
        far = np.abs(L.round_e4m3(ratio * (1 + 2.0 ** -22)) - L.round_e4m3(ratio * (1 - 2.0 ** -22)))
        assert_close(got, q, far, "Y against the oracle's rounding")
        for o in (X, Y, scale):
            o.check_guards()


@pytest.mark.parametrize("rows", [1, 128])
def test_quantise_special_values(gemm_mod, rows):
    """NaN and infinities show in their own block's scale, and no other block changes; a
    block of zeros, of the type's lowest value, of values too small to divide by."""
    X = normal((256, 512), torch.bfloat16, 1)
    clean, Y = (torch.empty(256, 512, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    s0, s = (torch.empty(256 // rows, 4, device="cuda") for _ in range(2))
    gemm_mod.quantise_blocks(X, clean, s0, rows=rows)
    at = 0 if rows == 128 else 7
    X[7, 5] = float("nan")
    X[7, 130] = float("-inf")
    block = slice(0, 128) if rows == 128 else slice(7, 8)
    X[block, 256:384] = torch.finfo(torch.bfloat16).min
    X[block, 384:] = 1e-31
    gemm_mod.quantise_blocks(X, Y, s, rows=rows)
    torch.cuda.synchronize()
    assert s[at, 0].isnan() and s[at, 1].isinf() and s[at, 3] == 0
    assert bool((Y[block, 256:384].float() == -448).all()) and not Y[block, 384:].float().any()
    other = [i for i in range(256) if not block.start <= i < block.stop]
    assert torch.equal(Y.view(torch.uint8)[other], clean.view(torch.uint8)[other])
    keep = [i for i in range(len(s)) if i != at]
    assert torch.equal(s[keep], s0[keep])


def test_quantised_operands_in_a_product_captured(gemm_mod):
    """quantise -> gated -> quantise -> product, as a layer uses them, in a graph
    replayed on new inputs: the bits of eager calls on another stream."""
    m, model, hidden, dtype = 70, 256, 400, torch.bfloat16
    X = torch.zeros(m, model, dtype=dtype, device="cuda")

    def empty(rows, cols, block_rows):
        ld = -(-cols // 16) * 16
        return (torch.empty(rows, ld, dtype=torch.float8_e4m3fn, device="cuda")[:, :cols],
                torch.empty(-(-rows // block_rows), -(-cols // 128), device="cuda"))

    weights = []
    for i, (rows, cols) in enumerate(((hidden, model), (hidden, model), (model, hidden))):
        w = normal((rows, cols), dtype, i, cols ** -0.5)
        weights.append(empty(rows, cols, 128))
        gemm_mod.quantise_blocks(w, *weights[-1], rows=128)
    (wg, sg), (wu, su), (wd, sd) = weights

    def step():
        (x8, sx), (h8, sh) = empty(m, model, 1), empty(m, hidden, 1)
        h, out = (torch.empty(m, c, dtype=dtype, device="cuda") for c in (hidden, model))
        gemm_mod.quantise_blocks(X, x8, sx)
        gemm_mod.gemm_gated(x8, wg, wu, h, trans_b=True, scale_a=sx, scale_gate=sg, scale_up=su)
        gemm_mod.quantise_blocks(h, h8, sh)
        gemm_mod.gemm_epilogue(h8, wd, out, residual=X, trans_b=True, scale_a=sh, scale_b=sd)
        return h, out

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        out = step()
    for seed in (1, 2):
        X.copy_(normal((m, model), dtype, seed))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_offsets_past_2_to_31_elements(gemm_mod):
    rows, n, ld, dtype = 3, 256, 1 << 30, torch.bfloat16
    buf = torch.empty((rows - 1) * ld + n, dtype=dtype, device="cuda")
    X = buf.as_strided((rows, n), (ld, 1))
    src = normal((rows, n), dtype, 1)
    X.copy_(src)
    Y, ref = (torch.empty(rows, n, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    wide = torch.empty((rows - 1) * ld + n, dtype=torch.float8_e4m3fn, device="cuda").as_strided(
        (rows, n), (ld, 1))
    for block_rows in (1, 128):
        s, t = (torch.empty(-(-rows // block_rows), 2, device="cuda") for _ in range(2))
        gemm_mod.quantise_blocks(src, ref, s, rows=block_rows)
        gemm_mod.quantise_blocks(X, Y, t, rows=block_rows)
        assert torch.equal(Y.view(torch.uint8), ref.view(torch.uint8)) and torch.equal(s, t)
        gemm_mod.quantise_blocks(src, wide, t, rows=block_rows)
        assert torch.equal(wide.contiguous().view(torch.uint8), ref.view(torch.uint8))


def test_refusals_of_the_binding(gemm_mod):
    g = gemm_mod
    A, sa = operand(64, 256, 1, 1)
    B, sb = operand(256, 256, 128, 2)
    D = torch.empty(64, 256, dtype=torch.bfloat16, device="cuda")
    good = dict(trans_b=True, scale_a=sa, scale_b=sb)
    g.gemm_epilogue(A, B, D, **good)
    for bad in (dict(scale_a=sa[:, :1]), dict(scale_a=sa[:3]), dict(scale_b=sb[:1]),
                dict(scale_b=sb[:, :1]), dict(scale_b=sb.cpu()), dict(trans_b=False)):
        with pytest.raises(ValueError):
            g.gemm_epilogue(A, B, D, **{**good, **bad})
    for bad in (dict(scale_a=None), dict(scale_b=None), dict(scale_a=sa.double())):
        with pytest.raises(TypeError):
            g.gemm_epilogue(A, B, D, **{**good, **bad})
    gated = dict(trans_b=True, scale_a=sa, scale_gate=sb, scale_up=sb)
    g.gemm_gated(A, B, B, D, **gated)
    for bad in (dict(scale_up=sb[:1]), dict(scale_a=sa[:3]), dict(trans_b=False)):
        with pytest.raises(ValueError):
            g.gemm_gated(A, B, B, D, **{**gated, **bad})
    with pytest.raises(TypeError):
        g.gemm_gated(A, B, B, D, trans_b=True)  # no scales
    with pytest.raises(ValueError):
        g.gemm_gated(D, D, D, D[:, :64], trans_b=True, scale_a=sa)  # scales, 16-bit operands
    X, Y = D, torch.empty(64, 256, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(64, 2, device="cuda")
    for bad in ((X, Y, s[:3]), (X, Y, s[:, :1]), (X, Y[:, :128], s), (X.cpu(), Y, s)):
        with pytest.raises(ValueError):
            g.quantise_blocks(*bad)
    for bad in ((X.float(), Y, s), (X, X, s), (X, Y, s.half()), (X, Y, None)):
        with pytest.raises(TypeError):
            g.quantise_blocks(*bad)
    with pytest.raises(ValueError):
        g.quantise_blocks(X, Y, s, rows=64)
