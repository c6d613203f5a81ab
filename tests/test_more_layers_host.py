"""Host-side refusals of the C entry points of the gated layer, the block-scaled
products, their quantisation and the layer norm: bad arguments return their status
before anything is enqueued (no GPU is needed), and empty problems are no-ops."""
import pytest

OK, INVALID, LAYOUT = 0, 1, 2
P = 1 << 20  # an aligned non-NULL address that is never dereferenced
BIG = 2 ** 31

# Arguments of a good call, in order, for each family.
FAMILIES = {
    "gemm_layer_norm_{}": dict(M=16, N=32, eps=0.0, X=P, ldx=32, R=P, ldr=32, W=P, b=P, H=P, ldh=32,
                               Y=P, ldy=32, mean=P, rstd=P, s=None),
    "gemm_layer_norm_grad_{}": dict(M=16, N=32, dY=P, lddy=32, H=P, ldh=32, mean=P, rstd=P, W=P,
                                    dH=P, lddh=32, dX=P, lddx=32, dW=P, db=P, s=None),
}
# What each refuses: changes of the good call and the status.
REFUSED = {
    "gemm_layer_norm_{}": [
        (INVALID, [dict(M=-1), dict(N=-1), dict(M=BIG), dict(N=BIG), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(X=None), dict(Y=None), dict(ldx=31),
                   dict(ldr=31), dict(ldh=31), dict(ldy=31)]),
        (LAYOUT, [{k: P + 1} for k in "XRWbHY"] + [dict(mean=P + 2), dict(rstd=P + 2)])],
    "gemm_layer_norm_grad_{}": [
        (INVALID, [dict(M=-1), dict(N=-1), dict(M=BIG), dict(N=BIG), dict(dY=None), dict(H=None),
                   dict(mean=None), dict(rstd=None), dict(dX=None), dict(lddy=31), dict(ldh=31),
                   dict(lddh=31), dict(lddx=31)]),
        (LAYOUT, [{k: P + 1} for k in ("dY", "H", "W", "dH", "dX", "dW", "db")]
         + [dict(mean=P + 2), dict(rstd=P + 2)])],
}
# Empty problems: nothing is read, written or enqueued.
EMPTY = {
    "gemm_layer_norm_{}": [dict(M=0), dict(N=0), dict(M=0, X=None, Y=None)],
    "gemm_layer_norm_grad_{}": [dict(N=0), dict(M=0, dW=None, db=None),
                                dict(M=0, dW=None, db=None, dY=None, H=None, dX=None, mean=None)],
}


def call(lib, family, dtype, change):
    args = FAMILIES[family]
    assert not set(change) - set(args), change
    return getattr(lib, family.format(dtype))(*{**args, **change}.values())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("family", FAMILIES)
def test_refusals(gemm_mod, family, dtype):
    for status, changes in REFUSED[family]:
        for change in changes:
            assert call(gemm_mod.lib, family, dtype, change) == status, change


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("family", FAMILIES)
def test_empty_problems_are_no_ops(gemm_mod, family, dtype):
    for change in EMPTY[family]:
        assert call(gemm_mod.lib, family, dtype, change) == OK, change


def test_cpu_tensors_are_refused(gemm_mod):
    import torch
    x, s = torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(8)
    for f in (lambda: gemm_mod.layer_norm(x, x), lambda: gemm_mod.layer_norm_grad(x, x, s, s, x)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
