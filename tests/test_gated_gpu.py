"""GPU parity of the gated layer (gemm_gated) and its gradient (gemm_gated_dact)
against the float64 oracle.

Tolerances, from the arithmetic that is promised (tests/layer_util.py): a projection
is an fp32 product, off by its bound and one rounding of the bias's addition; the
activation carries that times its slope (at most 1.13) and its own evaluation error;
the product of the two carries both factors' errors; each output is rounded once.
Gradient: slopes are within 2^-18 (1 + |z|), values as above. Column sums: the
elements' errors before rounding, added up, and M fp32 additions.
"""
import numpy as np
import pytest
import torch

from oracle import layers as L
from tests.layer_util import (DTYPES, Out, act_error, assert_close, normal, product_bound,
                              rounded_bound)

pytestmark = pytest.mark.gpu

MAX_SLOPE = 1.13
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(autouse=True)
def clean_error_word(gemm_mod):
    gemm_mod.check_device_error()
    yield
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0


def stored(rows, cols, trans, dtype, seed, std=1.0):
    return normal((cols, rows) if trans else (rows, cols), dtype, seed, std, unit=8)


def logical(t, trans):
    return L.to64(t).T if trans else L.to64(t)


def check_gated(A64, Bg64, Bu64, alpha, bg, bu, act, dtype, D, G=None, U=None):
    d, g, u = L.gated(A64, Bg64, Bu64, alpha, bg, bu, act)
    eg, eu = (product_bound(A64, B, alpha) + 2.0 ** -23 * np.abs(z)
              for B, z in ((Bg64, g), (Bu64, u)))
    a = np.abs(L.act(g, act))
    ea = MAX_SLOPE * eg + act_error(g, act)
    ed = ea * (np.abs(u) + eu) + a * eu + 2.0 ** -23 * np.abs(d)
    assert_close(L.to64(D), d, rounded_bound(d, ed, dtype), "D")
    if G is not None:
        assert_close(L.to64(G), g, rounded_bound(g, eg, dtype), "G")
    if U is not None:
        assert_close(L.to64(U), u, rounded_bound(u, eu, dtype), "U")


def run_gated(g, m, n, k, dtype, act="silu", bias=(True, True), keep=(True, True), trans_a=False,
              trans_b=False, alpha=1.0, pad=0, shift=0, seed=0):
    A = stored(m, k, trans_a, dtype, seed + 1)
    Bg, Bu = (stored(k, n, trans_b, dtype, seed + i, max(k, 1) ** -0.5) for i in (2, 3))
    bias = [normal((1, n), dtype, seed + 4 + i)[0] if b else None for i, b in enumerate(bias)]
    D = Out(m, n, dtype, pad, shift)
    kept = [Out(m, n, dtype, pad, shift) if want else None for want in keep]
    g.gemm_gated(A, Bg, Bu, D.t, act=act, alpha=alpha, bias_gate=bias[0], bias_up=bias[1],
                 gate=kept[0].t if kept[0] else None, up=kept[1].t if kept[1] else None,
                 trans_a=trans_a, trans_b=trans_b)
    torch.cuda.synchronize()
    check_gated(logical(A, trans_a), logical(Bg, trans_b), logical(Bu, trans_b), alpha,
                *(None if b is None else L.to64(b) for b in bias), act, dtype, D.t,
                *(o.t if o else None for o in kept))
    for o in (D, *kept):
        if o:
            o.check_guards()


def check_grad(A64, B64, alpha, g64, u64, act, dtype, dG, dU, dbg=None, dbu=None):
    d = alpha * (A64 @ B64)
    dg, du, sg, su = L.gated_grad(d, g64, u64, act)
    ep = product_bound(A64, B64, alpha) + 2.0 ** -23 * np.abs(d)
    slope, value = np.abs(L.act_slope(g64, act)), np.abs(L.act(g64, act))
    es = 2.0 ** -18 * (1 + np.abs(g64)) if act not in ("none", "relu") else np.zeros_like(g64)
    eg = np.abs(u64) * (slope * ep + (np.abs(d) + ep) * es) + 2.0 ** -22 * np.abs(dg)
    eu = value * ep + (np.abs(d) + ep) * act_error(g64, act) + 2.0 ** -22 * np.abs(du)
    for got, ref, e, what in ((dG, dg, eg, "dG"), (dU, du, eu, "dU")):
        assert_close(L.to64(got), ref, rounded_bound(ref, e, dtype), what)
    for got, ref, each, e, what in ((dbg, sg, dg, eg, "dbias_gate"), (dbu, su, du, eu, "dbias_up")):
        if got is not None:
            bound = e.sum(0) + (len(d) + 20) * 2.0 ** -24 * np.abs(each).sum(0)
            assert_close(L.to64(got), ref, rounded_bound(ref, bound, dtype), what)


def run_grad(g, m, n, k, dtype, act="silu", sums=(True, True), trans_a=False, trans_b=False,
             alpha=1.0, pad=0, shift=0, inplace=False, seed=0):
    A = stored(m, k, trans_a, dtype, seed + 1)
    B = stored(k, n, trans_b, dtype, seed + 2, max(k, 1) ** -0.5)
    G, U = normal((m, n), dtype, seed + 3, 1.5, pad=pad), normal((m, n), dtype, seed + 4, pad=pad)
    g64, u64 = L.to64(G), L.to64(U)
    dG, dU = (Out(m, n, dtype, pad, shift) for _ in range(2))
    if inplace:
        dG.t.copy_(G), dU.t.copy_(U)
        G, U = dG.t, dU.t
    sums = [Out(1, n, dtype) if s else None for s in sums]
    g.gemm_gated_dact(A, B, G, U, dG.t, dU.t, act=act, alpha=alpha,
                      dbias_gate=sums[0].t[0] if sums[0] else None,
                      dbias_up=sums[1].t[0] if sums[1] else None, trans_a=trans_a, trans_b=trans_b)
    torch.cuda.synchronize()
    check_grad(logical(A, trans_a), logical(B, trans_b), alpha, g64, u64, act, dtype, dG.t, dU.t,
               *(s.t[0] if s else None for s in sums))
    for o in (dG, dU, *sums):
        if o:
            o.check_guards()


# Sizes around the tiles' and the few-rows kernel's edges, one row to several
# tiles, k from one element over one k-block to many, and odd everything.
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 4096, 512), (2, 129, 65), (5, 250, 1000), (16, 1024, 2048),
          (17, 2048, 136), (33, 520, 200), (64, 640, 2048), (65, 130, 72), (100, 1111, 513),
          (128, 256, 64), (129, 257, 127), (200, 384, 4096), (255, 1023, 520), (256, 512, 1024),
          (257, 255, 63), (384, 4096, 128), (513, 777, 1023), (1000, 300, 2000), (2000, 3000, 64)]


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes(gemm_mod, shape, dtype):
    i = SHAPES.index(shape)
    run_gated(gemm_mod, *shape, dtype, ACTS[i % 5], bias=(i % 3 != 0, i % 3 != 1),
              keep=(i % 4 != 1, i % 4 != 2), trans_b=i % 2 == 1, seed=i)
    run_grad(gemm_mod, *shape, dtype, ACTS[i % 5], sums=(i % 3 != 0, i % 3 != 1),
             trans_b=i % 2 == 0, seed=i)


@pytest.mark.parametrize("trans_a", [False, True], ids=["an", "at"])
@pytest.mark.parametrize("trans_b", [False, True], ids=["bn", "bt"])
@pytest.mark.parametrize("shape", [(3, 140, 260), (40, 300, 100), (130, 200, 264),
                                   (300, 520, 1000)], ids=lambda s: "x".join(map(str, s)))
def test_operand_forms(gemm_mod, shape, trans_a, trans_b):
    run_gated(gemm_mod, *shape, torch.bfloat16, trans_a=trans_a, trans_b=trans_b, alpha=-0.75,
              seed=31)
    run_grad(gemm_mod, *shape, torch.float16, trans_a=trans_a, trans_b=trans_b, alpha=-0.75,
             seed=31)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [7, 150, 600])
def test_activations(gemm_mod, act, m):
    for dtype in DTYPES.values():
        run_gated(gemm_mod, m, 264, 128, dtype, act, alpha=3.0, seed=m)
        run_grad(gemm_mod, m, 264, 128, dtype, act, alpha=3.0, seed=m)


@pytest.mark.parametrize("shift,pad", [(0, 0), (0, 8), (0, 3), (1, 0), (8, 1), (3, 5)])
@pytest.mark.parametrize("m", [9, 140, 520])
def test_output_layouts(gemm_mod, m, shift, pad):
    for keep in ((True, True), (False, True)):
        run_gated(gemm_mod, m, 272, 96, torch.float16, "gelu", keep=keep, pad=pad, shift=shift,
                  trans_b=True)
    for inplace in (False, True):
        run_grad(gemm_mod, m, 272, 96, torch.bfloat16, "relu", pad=pad, shift=shift,
                 inplace=inplace, sums=(inplace, True))


def test_outputs_of_unlike_layouts(gemm_mod):
    """dG by TMA with dU by plain stores and the other way round, G and U likewise; the
    128- and 256-column tiles."""
    dtype = torch.bfloat16
    for n, k in ((520, 64), (2560, 512)):
        A, B = normal((600, k), dtype, 1), normal((k, n), dtype, 2, k ** -0.5)
        A64, B64 = L.to64(A), L.to64(B)
        for odd in range(4):
            G = Out(600, n, dtype, pad=odd == 0)
            U = Out(600, n, dtype, pad=odd == 1)
            G.t.copy_(normal((600, n), dtype, 3)), U.t.copy_(normal((600, n), dtype, 4))
            g64, u64 = L.to64(G.t), L.to64(U.t)
            dG, dU = Out(600, n, dtype, pad=odd == 2), Out(600, n, dtype, shift=odd == 3)
            gemm_mod.gemm_gated_dact(A, B, G.t, U.t, dG.t, dU.t)
            torch.cuda.synchronize()
            check_grad(A64, B64, 1.0, g64, u64, "silu", dtype, dG.t, dU.t)
            gemm_mod.gemm_gated_dact(A, B, G.t, U.t, G.t, U.t)
            torch.cuda.synchronize()
            assert torch.equal(G.t, dG.t) and torch.equal(U.t, dU.t)
            for o in (G, U, dG, dU):
                o.check_guards()


def test_the_two_weights_as_parts_of_one_matrix(gemm_mod):
    dtype = torch.bfloat16
    A = normal((300, 256), dtype, 1)
    rows, cols = normal((1024, 256), dtype, 2, 1 / 16), normal((256, 1024), dtype, 3, 1 / 16)
    D = [Out(300, 512, dtype) for _ in range(2)]
    gemm_mod.gemm_gated(A, rows[:512], rows[512:], D[0].t, trans_b=True)
    gemm_mod.gemm_gated(A, cols[:, 512:], cols[:, :512], D[1].t)
    torch.cuda.synchronize()
    r, c = L.to64(rows), L.to64(cols)
    check_gated(L.to64(A), r[:512].T, r[512:].T, 1.0, None, None, "silu", dtype, D[0].t)
    check_gated(L.to64(A), c[:, 512:], c[:, :512], 1.0, None, None, "silu", dtype, D[1].t)
    for o in D:
        o.check_guards()


@pytest.mark.parametrize("shape", [(0, 40, 16), (3, 0, 16), (3, 40, 0), (300, 136, 0)],
                         ids=lambda s: "x".join(map(str, s)))
def test_empty(gemm_mod, shape):
    m, n, k = shape
    run_gated(gemm_mod, m, n, k, torch.bfloat16)
    run_gated(gemm_mod, m, n, k, torch.float16, bias=(False, True), keep=(False, False))
    run_grad(gemm_mod, m, n, k, torch.bfloat16)
    run_grad(gemm_mod, m, n, k, torch.float16, sums=(False, True))


@pytest.mark.parametrize("m", [5, 300])
def test_special_values_stay_in_their_rows_and_columns(gemm_mod, m):
    """A NaN in a row of A makes that row NaN, an infinity in a column of one weight
    that column infinite or NaN; nothing else changes. Rows of G and U with NaN and
    the type's lowest value leave other rows' gradients alone; the sums of a column
    with a NaN are NaN, the others finite."""
    n, k, dtype = 264, 128, torch.bfloat16
    A, Bg, Bu = normal((m, k), dtype, 1), normal((k, n), dtype, 2), normal((k, n), dtype, 3)
    clean, D = torch.empty(m, n, dtype=dtype, device="cuda"), Out(m, n, dtype)
    gemm_mod.gemm_gated(A, Bg, Bu, clean)
    A[m // 2, 3] = float("nan")
    Bu[5, 17] = float("inf")
    gemm_mod.gemm_gated(A, Bg, Bu, D.t)
    torch.cuda.synchronize()
    assert bool(D.t[m // 2].isnan().all()) and not bool(D.t[:, 17].isfinite().any())
    rows = [i for i in range(m) if i != m // 2]
    cols = [j for j in range(n) if j != 17]
    assert torch.equal(D.t[rows][:, cols], clean[rows][:, cols])
    A = normal((m, k), dtype, 1)
    G, U = normal((m, n), dtype, 4), normal((m, n), dtype, 5)
    out = []
    for dirty in (False, True):
        if dirty:
            G[m // 2, 9], U[m // 2, 11] = float("nan"), float("-inf")
            G[m // 2, 13] = torch.finfo(dtype).min
        dG, dU = Out(m, n, dtype), Out(m, n, dtype)
        sg, su = (torch.empty(n, dtype=dtype, device="cuda") for _ in range(2))
        gemm_mod.gemm_gated_dact(A, Bg, G, U, dG.t, dU.t, act="gelu_tanh", dbias_gate=sg,
                                 dbias_up=su)
        torch.cuda.synchronize()
        out.append((dG.t, dU.t, sg, su))
    clean, got = out
    assert bool(got[0][m // 2, 9].isnan()) and not bool(got[0][m // 2, 11].isfinite())
    assert bool(got[1][m // 2, 9].isnan()) and bool(got[1][m // 2, 11].isfinite())
    assert bool(got[0][m // 2, 13].isfinite()) and bool(got[1][m // 2, 13].isfinite())
    cols = [j for j in range(n) if j not in (9, 11, 13)]
    for a, b in zip(clean[:2], got[:2]):
        assert torch.equal(a[rows], b[rows]) and torch.equal(a[:, cols], b[:, cols])
    for a, b in zip(clean[2:], got[2:]):
        assert torch.equal(a[cols], b[cols])


def test_captured_steps_on_two_streams(gemm_mod):
    """Two captured steps (each with sums of its own from the library's pool) replayed
    on two streams at a time, on new inputs: the bits of eager calls."""
    dtype, graphs = torch.float16, []
    for m, n, k in ((40, 520, 256), (300, 1000, 520)):
        A, G, U = (torch.zeros(m, c, dtype=dtype, device="cuda") for c in (k, n, n))
        Bg, Bu = normal((k, n), dtype, 1, k ** -0.5), normal((k, n), dtype, 2, k ** -0.5)

        def step(A=A, G=G, U=U, Bg=Bg, Bu=Bu):
            D, dG, dU = (torch.empty_like(G) for _ in range(3))
            sg, su = (torch.empty(G.shape[1], dtype=dtype, device="cuda") for _ in range(2))
            gemm_mod.gemm_gated(A, Bg, Bu, D, gate=G, up=U)
            gemm_mod.gemm_gated_dact(A, Bg, G, U, dG, dU, dbias_gate=sg, dbias_up=su)
            return D, dG, dU, sg, su

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            out = step()
        graphs.append((graph, A, out, step))
    for seed in (1, 2):
        for _, A, _, _ in graphs:
            A.copy_(normal(tuple(A.shape), dtype, seed))
        torch.cuda.synchronize()
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g[0].replay()
        torch.cuda.synchronize()
        for _, _, out, step in graphs:
            got = [t.clone() for t in out]
            want = step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_outputs_past_2_to_31_elements(gemm_mod):
    m, n, k, ld, dtype = 70, 136, 64, 1 << 25, torch.bfloat16
    buf = torch.empty((m - 1) * ld + n, dtype=dtype, device="cuda")
    D = buf.as_strided((m, n), (ld, 1))
    A, Bg, Bu = normal((m, k), dtype, 1), normal((k, n), dtype, 2), normal((k, n), dtype, 3)
    ref = torch.empty(m, n, dtype=dtype, device="cuda")
    G, U = normal((m, n), dtype, 4), normal((m, n), dtype, 5)
    for rows in (20, m):
        gemm_mod.gemm_gated(A[:rows], Bg, Bu, ref[:rows])
        gemm_mod.gemm_gated(A[:rows], Bg, Bu, D[:rows])
        assert torch.equal(D[:rows], ref[:rows])
        other = torch.empty_like(ref)
        gemm_mod.gemm_gated_dact(A[:rows], Bg, G[:rows], U[:rows], ref[:rows], other[:rows])
        gemm_mod.gemm_gated_dact(A[:rows], Bg, G[:rows], U[:rows], other[:rows], D[:rows])
        assert torch.equal(other[:rows], ref[:rows])


def test_refusals_of_the_binding(gemm_mod):
    x = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    ok = (x, x, x, torch.empty_like(x))
    gemm_mod.gemm_gated(*ok)
    for at in range(4):
        with pytest.raises(TypeError):
            gemm_mod.gemm_gated(*[t.half() if i == at else t for i, t in enumerate(ok)])
        with pytest.raises(ValueError):
            gemm_mod.gemm_gated(*[t[:, :40] if i == at else t for i, t in enumerate(ok)])
        with pytest.raises(ValueError):
            gemm_mod.gemm_gated(*[t.cpu() if i == at else t for i, t in enumerate(ok)])
    for kw in ({"gate": x[:3]}, {"up": x[:, :8]}, {"bias_gate": x[0, :3]}, {"bias_up": x[0, ::2]},
               {"act": "swish"}):
        with pytest.raises(ValueError):
            gemm_mod.gemm_gated(*ok, **kw)
    with pytest.raises(gemm_mod.GemmError) as e:  # a second weight off a 16-byte boundary
        gemm_mod.gemm_gated(x[:, :32], x[:32, :32], x[:32, 1:33], torch.empty_like(x)[:, :32])
    assert e.value.status == 2
    good = (x, x, x, x, torch.empty_like(x), torch.empty_like(x))
    for at in range(2, 6):
        with pytest.raises(TypeError):
            gemm_mod.gemm_gated_dact(*[None if i == at else t for i, t in enumerate(good)])
        with pytest.raises(ValueError):
            gemm_mod.gemm_gated_dact(*[t[:, :40] if i == at else t for i, t in enumerate(good)])
    with pytest.raises(ValueError):
        gemm_mod.gemm_gated_dact(*good, dbias_up=x[0, :8])
