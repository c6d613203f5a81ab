"""layer_norm_grad with each choice of outputs: every call's dX has the layout of the
first one's, so that the same kernel runs, and the same bits; each result is also checked
against the float64 oracle before the next call writes its own."""
import pytest
import torch

from oracle import layers as L
from tests.layer_util import DTYPES, Out, normal
from tests.test_layer_norm_gpu import MANY, SHAPES, check_grad, opt64, statistics, vector

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES.values(), ids=list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES + MANY, ids=lambda s: "x".join(map(str, s)))
def test_each_choice_of_outputs(gemm_mod, shape, dtype):
    m, n = shape
    i = (SHAPES + MANY).index(shape)
    pad = [1, 0, 8][i % 3]
    H, dY = normal(shape, dtype, i, 2.0, pad=pad), normal(shape, dtype, i + 1, pad=pad)
    dH = normal(shape, dtype, i + 2, pad=pad) if i % 2 else None
    W = vector(n, dtype, i) if i % 4 != 3 else None
    mean, rstd = statistics(H)
    args = (L.to64(dY), L.to64(H), L.to64(mean), L.to64(rstd), opt64(W), opt64(dH), dtype)
    first = None
    for layout in (pad, pad, 2):  # rows 2 longer: another form where the others are not
        for want_w, want_b in ((True, True), (True, False), (False, True), (False, False)):
            dX = Out(m, n, dtype, pad=layout)
            dW, db = (Out(1, n, dtype) if want else None for want in (want_w, want_b))
            gemm_mod.layer_norm_grad(dY, H, mean, rstd, dX.t, weight=W, dh=dH,
                                     dweight=dW.t[0] if dW else None,
                                     dbias=db.t[0] if db else None)
            torch.cuda.synchronize()
            check_grad(*args, dX.t, dW.t[0] if dW else None, db.t[0] if db else None)
            if first is None:
                first = dX, dW, db
            if layout == pad:
                for got, same in zip((dX, dW, db), first):
                    assert got is None or torch.equal(got.t, same.t)
            for o in (dX, dW, db):
                if o:
                    o.check_guards()
    assert gemm_mod.check_device_error() == 0
