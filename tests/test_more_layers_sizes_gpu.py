"""The gated layer, the block-scaled products, their quantisation and the layer norm at
the largest sizes that their entry points accept, 2^31 - 1 in each direction: sums and
round-ups of sizes must not leave 32 bits. Results are known exactly, or to the few
roundings that are given."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BIG = 2 ** 31 - 1
PLACES = [0, 63, 64, 12345678, 2 ** 30 + 7, BIG - 130, BIG - 65, BIG - 2, BIG - 1]
GUARD = 7.0


@pytest.fixture(autouse=True)
def clean_error_word(gemm_mod):
    gemm_mod.check_device_error()
    yield
    torch.cuda.synchronize()
    assert gemm_mod.check_device_error() == 0
    torch.cuda.empty_cache()


def filled(n, value, dtype=torch.bfloat16):
    return torch.full((n,), value, dtype=dtype, device="cuda")


def ones_at(n):
    v = filled(n, 0)
    for p in PLACES:
        v[p] = 1
    return v


def check(v, value=1.0):
    """v holds `value` at PLACES and zeros elsewhere."""
    assert v[PLACES].float().tolist() == [value] * len(PLACES)
    for p in PLACES:
        v[p] = 0
    assert not any(bool(c.view(torch.uint8).any()) for c in v.split(1 << 28))


def test_gated_most_columns(gemm_mod):
    b = ones_at(BIG).view(1, BIG)
    a = torch.full((1, 1), 3.0, dtype=torch.bfloat16, device="cuda")
    buf = filled(BIG + 8, GUARD)
    D = buf[:BIG].view(1, BIG)
    gemm_mod.gemm_gated(a, b, b, D, act="none")  # (3 b)^2
    check(D[0], 9.0)
    assert (buf[BIG:] == GUARD).all()
    # dD = 3 b: dG = dD U = 3 b, dU = dD G = 3 b for G = U = b; no sums
    out = filled(BIG + 8, GUARD)
    gemm_mod.gemm_gated_dact(a, b, b, b, out[:BIG].view(1, BIG), D, act="none")
    check(out[:BIG], 3.0)
    check(D[0], 3.0)
    assert (out[BIG:] == GUARD).all() and (buf[BIG:] == GUARD).all()


def test_gated_most_rows(gemm_mod):
    flat = filled(8 * (BIG - 1) + 1, 0)
    A = flat.as_strided((BIG, 1), (8, 1))
    for p in PLACES:
        A[p] = 1
    b = torch.full((1, 1), 3.0, dtype=torch.bfloat16, device="cuda")
    buf = filled(BIG + 8, GUARD)
    D = buf[:BIG].view(BIG, 1)
    gemm_mod.gemm_gated(A, b, b, D, act="none")
    check(buf[:BIG], 9.0)
    assert (buf[BIG:] == GUARD).all()


@pytest.mark.parametrize("kind", ["gated", "block", "block gated"])
def test_longest_inner_dimension(gemm_mod, kind):
    D = torch.full((1, 1), GUARD, dtype=torch.bfloat16, device="cuda")
    if kind == "gated":
        a = ones_at(BIG).view(1, BIG)
        gemm_mod.gemm_gated(a, a, a, D, act="none", trans_b=True)
        assert D.item() == len(PLACES) ** 2
        return
    a = filled(BIG, 0, torch.uint8)
    for p in PLACES:
        a[p] = 0x38  # 1.0
    a = a.view(torch.float8_e4m3fn).view(1, BIG)
    scale = torch.full((1, -(-BIG // 128)), 0.5, device="cuda")
    if kind == "block":
        gemm_mod.gemm_epilogue(a, a, D, trans_b=True, scale_a=scale, scale_b=scale)
        assert D.item() == len(PLACES) / 4
    else:
        gemm_mod.gemm_gated(a, a, a, D, act="none", trans_b=True, scale_a=scale, scale_gate=scale,
                            scale_up=scale)
        assert D.item() == (len(PLACES) / 4) ** 2 or abs(D.item() - (len(PLACES) / 4) ** 2) <= 2 ** -6


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("shift", [0, 1])
def test_quantise_longest_row(gemm_mod, rows, shift):
    X = filled(BIG + shift, 0)[shift:]
    for p in PLACES:
        X[p] = 2
    buf = filled(BIG + 8, 0x55, torch.uint8)
    Y = buf[:BIG].view(torch.float8_e4m3fn)
    scale = filled(-(-BIG // 128) + 4, GUARD, torch.float32)
    gemm_mod.quantise_blocks(X.view(1, BIG), Y.view(1, BIG), scale[:-4].view(1, -1), rows=rows)
    torch.cuda.synchronize()
    assert (buf[BIG:] == 0x55).all() and (scale[-4:] == GUARD).all()
    blocks = sorted({p // 128 for p in PLACES})
    want = torch.zeros(len(scale) - 4, device="cuda")
    want[blocks] = 2 / torch.tensor(448.0).item()
    assert torch.equal(scale[:-4], want)
    check(Y, 448.0)


def test_quantise_most_rows(gemm_mod):
    X = filled(BIG, 0)
    for p in PLACES:
        X[p] = 2
    for rows in (1, 128):
        Y = filled(BIG, 0x55, torch.uint8).view(torch.float8_e4m3fn)
        scale = filled(-(-BIG // rows), GUARD, torch.float32)
        gemm_mod.quantise_blocks(X.view(BIG, 1), Y.view(BIG, 1), scale.view(-1, 1), rows=rows)
        check(Y, 448.0)
        assert int((scale != 0).sum()) == len({p // rows for p in PLACES})


def test_layer_norm_longest_row(gemm_mod):
    X = filled(BIG, 3)
    buf = filled(BIG + 8, GUARD)
    mean, rstd = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    gemm_mod.layer_norm(X.view(1, BIG), buf[:BIG].view(1, BIG), mean=mean, rstd=rstd, eps=1.0)
    assert abs(mean.item() - 3) < 1e-5 and abs(rstd.item() - 1) < 1e-5
    assert all(float(c.abs().max()) < 1e-4 for c in buf[:BIG].split(1 << 28))
    assert (buf[BIG:] == GUARD).all()
    mean.fill_(3), rstd.fill_(1)
    dw, db = filled(BIG + 8, GUARD), filled(BIG + 8, GUARD)
    dY = ones_at(BIG)
    gemm_mod.layer_norm_grad(dY.view(1, BIG), X.view(1, BIG), mean, rstd, X.view(1, BIG),
                             dweight=dw[:BIG], dbias=db[:BIG])
    check(db[:BIG])
    assert not any(bool(c.any()) for c in dw[:BIG].split(1 << 28))
    assert (dw[BIG:] == GUARD).all() and (db[BIG:] == GUARD).all()
    # dX = dY - mean(dY), 9 / 2^31 below
    for p in PLACES:
        assert abs(X[p].item() - 1) < 1e-2
        X[p] = 0
    assert all(float(c.abs().max()) < 1e-8 for c in X.split(1 << 28))


def test_layer_norm_most_rows(gemm_mod):
    X, Y = ones_at(BIG).view(BIG, 1), filled(BIG + 8, GUARD)
    b = torch.full((1,), 2.0, dtype=torch.bfloat16, device="cuda")
    gemm_mod.layer_norm(X, Y[:BIG].view(BIG, 1), bias=b)  # one column: h - mean = 0
    assert all(bool((c == 2).all()) for c in Y[:BIG].split(1 << 28)) and (Y[BIG:] == GUARD).all()
    stats = torch.ones(BIG, device="cuda")
    db = filled(1, GUARD)
    gemm_mod.layer_norm_grad(X, X, stats, stats, Y[:BIG].view(BIG, 1), dbias=db)
    assert db.item() == len(PLACES)
    assert not any(bool(c.any()) for c in Y[:BIG].split(1 << 28)) and (Y[BIG:] == GUARD).all()
