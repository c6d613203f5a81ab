"""Host-side refusals of the linear-layer C entry points: bad arguments return
their status before anything is enqueued (no GPU is needed), and empty problems
are no-ops."""
import pytest

OK, INVALID, LAYOUT = 0, 1, 2
P = 1 << 20  # an aligned non-NULL address that is never dereferenced
BIG = 2 ** 31


def call(lib, name, **kw):
    f = getattr(lib, name)
    if name.startswith("gemm_e4m3"):
        v = dict(M=16, N=32, K=64, alpha=1.0, A=P, lda=64, sa=P, B=P, ldb=64, sb=P, act=1, bias=P,
                 R=P, ldr=32, Z=P, ldz=32, D=P, ldd=32, s=None)
    elif name.endswith("_epi"):
        v = dict(opA=0, opB=0, M=16, N=32, K=64, alpha=1.0, A=P, lda=64, B=P, ldb=32, act=1,
                 bias=P, R=P, ldr=32, Z=P, ldz=32, D=P, ldd=32, s=None)
    elif name.endswith("_dact"):
        v = dict(opA=0, opB=0, M=16, N=32, K=64, alpha=1.0, A=P, lda=64, B=P, ldb=32, act=1, Z=P,
                 ldz=32, D=P, ldd=32, dbias=P, s=None)
    elif "act_grad" in name:
        v = dict(M=16, N=32, act=1, A=P, lda=32, Z=P, ldz=32, D=P, ldd=32, dbias=P, s=None)
    elif "norm_grad" in name:
        v = dict(M=16, N=32, A=P, lda=32, H=P, ldh=32, rstd=P, W=P, dH=P, lddh=32, D=P, ldd=32,
                 dW=P, s=None)
    elif name.endswith("_e4m3"):
        v = dict(M=16, N=32, eps=0.0, A=P, lda=32, R=P, ldr=32, W=P, H=P, ldh=32, D=P, ldd=32,
                 scale=P, rstd=P, s=None)
    else:
        v = dict(M=16, N=32, eps=0.0, A=P, lda=32, R=P, ldr=32, W=P, H=P, ldh=32, D=P, ldd=32,
                 rstd=P, s=None)
    assert not set(kw) - set(v), kw
    v.update(kw)
    return f(*v.values())


EPI = ["gemm_bf16_epi", "gemm_f16_epi"]
EPI8 = ["gemm_e4m3_bf16_epi", "gemm_e4m3_f16_epi"]
DACT = ["gemm_bf16_dact", "gemm_f16_dact"]
POINT = ["gemm_act_grad_bf16", "gemm_act_grad_f16"]
NORM = ["gemm_rms_norm_bf16", "gemm_rms_norm_f16"]
NORM8 = ["gemm_rms_norm_bf16_e4m3", "gemm_rms_norm_f16_e4m3"]
NORM_GRAD = ["gemm_rms_norm_grad_bf16", "gemm_rms_norm_grad_f16"]
ALL = EPI + EPI8 + DACT + POINT + NORM + NORM8 + NORM_GRAD


@pytest.mark.parametrize("name", ALL)
def test_sizes_strides_and_null_operands(gemm_mod, name):
    lib = gemm_mod.lib
    for size in ("M", "N"):
        assert call(lib, name, **{size: -1}) == INVALID
        assert call(lib, name, **{size: BIG}) == INVALID
    for operand in ("A", "D"):
        assert call(lib, name, **{operand: None}) == INVALID
    for ld in ("lda", "ldd"):
        assert call(lib, name, **{ld: 16}) == INVALID


@pytest.mark.parametrize("name", EPI + EPI8 + DACT)
def test_products(gemm_mod, name):
    lib = gemm_mod.lib
    assert call(lib, name, K=-1) == INVALID
    assert call(lib, name, K=BIG) == INVALID
    assert call(lib, name, B=None) == INVALID
    assert call(lib, name, ldb=16) == INVALID
    assert call(lib, name, ldz=31) == INVALID
    assert call(lib, name, act=5) == INVALID and call(lib, name, act=-1) == INVALID
    assert call(lib, name, A=P + 8) == LAYOUT and call(lib, name, B=P + 2) == LAYOUT
    assert call(lib, name, lda=68) == LAYOUT and call(lib, name, ldb=68) == LAYOUT
    assert call(lib, name, D=P + 1) == LAYOUT and call(lib, name, Z=P + 1) == LAYOUT
    if name in EPI8:
        assert call(lib, name, lda=72) == LAYOUT  # whole 16-byte units of bytes
        assert call(lib, name, sa=P + 2) == LAYOUT and call(lib, name, sb=P + 1) == LAYOUT
    else:
        assert call(lib, name, opA=2) == INVALID and call(lib, name, opB=-1) == INVALID
        assert call(lib, name, opB=1, ldb=32) == INVALID  # rows of a stored N x K hold K
        assert call(lib, name, opA=1, M=128, lda=64) == INVALID
    if name in DACT:
        assert call(lib, name, Z=None) == INVALID  # an activation's slope needs Z
        assert call(lib, name, dbias=P + 1) == LAYOUT
    else:
        assert call(lib, name, ldr=31) == INVALID
        assert call(lib, name, bias=P + 1) == LAYOUT and call(lib, name, R=P + 1) == LAYOUT


@pytest.mark.parametrize("name", POINT)
def test_pointwise_gradient(gemm_mod, name):
    lib = gemm_mod.lib
    assert call(lib, name, act=5) == INVALID
    assert call(lib, name, Z=None) == INVALID
    assert call(lib, name, ldz=31) == INVALID
    assert call(lib, name, act=0, A=P + 1) == LAYOUT
    assert call(lib, name, act=0, D=None, dbias=None) == OK  # nothing is wanted
    assert call(lib, name, Z=P + 1) == LAYOUT and call(lib, name, dbias=P + 1) == LAYOUT


@pytest.mark.parametrize("name", NORM + NORM8 + NORM_GRAD)
def test_norms(gemm_mod, name):
    lib = gemm_mod.lib
    assert call(lib, name, W=P + 1) == LAYOUT and call(lib, name, rstd=P + 2) == LAYOUT
    assert call(lib, name, H=P + 1) == LAYOUT and call(lib, name, ldh=31) == INVALID
    if name in NORM_GRAD:
        assert call(lib, name, rstd=None) == INVALID and call(lib, name, H=None) == INVALID
        assert call(lib, name, lddh=31) == INVALID and call(lib, name, dH=P + 1) == LAYOUT
        assert call(lib, name, dW=P + 1) == LAYOUT
    else:
        assert call(lib, name, eps=-1.0) == INVALID
        assert call(lib, name, eps=float("nan")) == INVALID
        assert call(lib, name, ldr=31) == INVALID and call(lib, name, R=P + 1) == LAYOUT
        if name in NORM8:
            assert call(lib, name, scale=None) == INVALID
            assert call(lib, name, scale=P + 2) == LAYOUT


@pytest.mark.parametrize("name", ALL)
def test_empty_problems_are_no_ops(gemm_mod, name):
    lib = gemm_mod.lib
    assert call(lib, name, N=0) == OK
    none = {"dbias": None} if name in DACT + POINT else {"dW": None} if name in NORM_GRAD else {}
    assert call(lib, name, M=0, A=None, D=None, **none) == OK


def test_wrong_arguments_of_the_marshalling_module(gemm_mod):
    mod = gemm_mod._load_layers()
    with pytest.raises(TypeError):
        mod.rms_norm(1, 2)                      # too few
    with pytest.raises(TypeError):
        mod.act_grad(1, None, None, None, None, None)  # not a tensor
    with pytest.raises(KeyError):
        mod.bind("gemm_f32", 0)


def test_cpu_tensors_are_refused(gemm_mod):
    import torch
    x = torch.zeros(8, 16, dtype=torch.bfloat16)
    for f in (lambda: gemm_mod.gemm_epilogue(x, x, x[:, :8], trans_b=True),
              lambda: gemm_mod.gemm_dact(x, x, None, x[:, :8], trans_b=True),
              lambda: gemm_mod.act_grad(x, None, x), lambda: gemm_mod.rms_norm(x, x),
              lambda: gemm_mod.rms_norm_grad(x, x, torch.zeros(8), x)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
