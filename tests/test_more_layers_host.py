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
    "gemm_{}_gated": dict(opA=0, opB=0, M=16, N=32, K=64, alpha=1.0, A=P, lda=64, Bg=P, ldbg=32,
                          Bu=P, ldbu=32, act=4, bias_g=P, bias_u=P, G=P, ldg=32, U=P, ldu=32, D=P,
                          ldd=32, s=None),
    "gemm_{}_gated_dact": dict(opA=0, opB=0, M=16, N=32, K=64, alpha=1.0, A=P, lda=64, B=P, ldb=32,
                               act=4, G=P, ldg=32, U=P, ldu=32, dG=P, lddg=32, dU=P, lddu=32,
                               dbias_g=P, dbias_u=P, s=None),
    "gemm_e4m3_{}_gated": dict(M=16, N=32, K=256, alpha=1.0, A=P, lda=256, sa=P, ldsa=2, Bg=P,
                               ldbg=256, sg=P, ldsg=2, Bu=P, ldbu=256, su=P, ldsu=2, act=4,
                               bias_g=P, bias_u=P, G=P, ldg=32, U=P, ldu=32, D=P, ldd=32, s=None),
    "gemm_e4m3_block_{}_epi": dict(M=16, N=32, K=256, alpha=1.0, A=P, lda=256, sa=P, ldsa=2, B=P,
                                   ldb=256, sb=P, ldsb=2, act=4, bias=P, R=P, ldr=32, Z=P, ldz=32,
                                   D=P, ldd=32, s=None),
    "gemm_quantise_{}_e4m3": dict(M=16, N=256, rows=1, X=P, ldx=256, Y=P, ldy=256, scale=P, lds=2,
                                  s=None),
}
PRODUCT = [dict(M=-1), dict(N=-1), dict(K=-1), dict(M=BIG), dict(N=BIG), dict(K=BIG),
           dict(A=None), dict(lda=56), dict(act=5), dict(act=-1)]
FORMS = [dict(opA=2), dict(opB=-1), dict(opA=1, M=128)]
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
    "gemm_{}_gated": [
        (INVALID, PRODUCT + FORMS + [dict(Bg=None), dict(Bu=None), dict(D=None), dict(ldbg=24),
                                     dict(ldbu=24), dict(opB=1), dict(opB=1, ldbg=64),
                                     dict(ldd=31), dict(ldg=31), dict(ldu=31)]),
        (LAYOUT, [{k: P + 1} for k in ("bias_g", "bias_u", "G", "U", "D")]
         + [{k: P + 8} for k in ("A", "Bg", "Bu")] + [dict(lda=68), dict(ldbg=36), dict(ldbu=36)])],
    "gemm_{}_gated_dact": [
        (INVALID, PRODUCT + FORMS + [dict(B=None), dict(ldb=24), dict(opB=1)]
         + [{k: None} for k in ("G", "U", "dG", "dU")] + [dict(act=0, G=None)]
         + [{k: 31} for k in ("ldg", "ldu", "lddg", "lddu")]),
        (LAYOUT, [{k: P + 1} for k in ("G", "U", "dG", "dU", "dbias_g", "dbias_u")]
         + [dict(A=P + 8), dict(B=P + 8), dict(lda=68), dict(ldb=36)])],
    "gemm_e4m3_{}_gated": [
        (INVALID, PRODUCT + [{k: None} for k in ("Bg", "Bu", "D", "sa", "sg", "su")]
         + [{k: 240} for k in ("ldbg", "ldbu")] + [{k: 1} for k in ("ldsa", "ldsg", "ldsu")]
         + [{k: 31} for k in ("ldd", "ldg", "ldu")]),
        (LAYOUT, [{k: P + 1} for k in ("bias_g", "bias_u", "G", "U", "D")]
         + [{k: P + 8} for k in ("A", "Bg", "Bu")] + [{k: P + 2} for k in ("sa", "sg", "su")]
         + [{k: 264} for k in ("lda", "ldbg", "ldbu")])],
    "gemm_e4m3_block_{}_epi": [
        (INVALID, PRODUCT + [{k: None} for k in ("B", "D", "sa", "sb")]
         + [{k: 1} for k in ("ldsa", "ldsb")] + [{k: 31} for k in ("ldd", "ldz", "ldr")]
         + [dict(ldb=240)]),
        (LAYOUT, [{k: P + 1} for k in ("bias", "R", "Z", "D")] + [{k: P + 8} for k in "AB"]
         + [{k: P + 2} for k in ("sa", "sb")] + [{k: 264} for k in ("lda", "ldb")])],
    "gemm_quantise_{}_e4m3": [
        (INVALID, [dict(M=-1), dict(N=-1), dict(M=BIG), dict(N=BIG), dict(rows=0), dict(rows=64),
                   dict(X=None), dict(Y=None), dict(scale=None), dict(ldx=255), dict(ldy=255),
                   dict(lds=1)]),
        (LAYOUT, [dict(X=P + 1), dict(scale=P + 2)])],
}
# Empty problems: nothing is read, written or enqueued.
EMPTY = {
    "gemm_layer_norm_{}": [dict(M=0), dict(N=0), dict(M=0, X=None, Y=None)],
    "gemm_layer_norm_grad_{}": [dict(N=0), dict(M=0, dW=None, db=None),
                                dict(M=0, dW=None, db=None, dY=None, H=None, dX=None, mean=None)],
    "gemm_{}_gated": [dict(M=0), dict(N=0), dict(M=0, A=None, D=None, G=None)],
    "gemm_{}_gated_dact": [dict(N=0), dict(M=0, dbias_g=None, dbias_u=None),
                           dict(M=0, dbias_g=None, dbias_u=None, G=None, dU=None)],
    "gemm_e4m3_{}_gated": [dict(M=0), dict(N=0), dict(M=0, A=None, sa=None, D=None)],
    "gemm_e4m3_block_{}_epi": [dict(M=0), dict(N=0), dict(N=0, B=None, sb=None)],
    "gemm_quantise_{}_e4m3": [dict(M=0), dict(N=0), dict(M=0, X=None, Y=None, scale=None)],
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
    for f in (lambda: gemm_mod.gemm_gated(x, x, x, x[:, :8], trans_b=True),
              lambda: gemm_mod.gemm_gated_dact(x, x, *[x[:, :8]] * 4, trans_b=True),
              lambda: gemm_mod.quantise_blocks(x, x.to(torch.float8_e4m3fn), s.view(8, 1)),
              lambda: gemm_mod.layer_norm(x, x), lambda: gemm_mod.layer_norm_grad(x, x, s, s, x)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
