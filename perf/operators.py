"""The linear-layer and normalisation operators as measured cases.

Four operators of a transformer block's feed-forward half, each in a plain form
(elementary torch operations in fp32, rounded once at the end) and, with
``own`` set, through this library's binding:

* ``linear``: D = act(alpha * op(A) * op(B) * scales + bias) + R, optionally
  with the pre-activation Z written too; bf16 and fp16, and e4m3 operands with
  a scale per row of A and per column of B.
* ``linear_grad``: the gradient at the pre-activation, dZ = act'(Z) * dD with
  the bias gradient (its column sums), where dD is either the product
  alpha * op(A) * op(B) of the next layer's gradient and weights ("product")
  or a matrix in hand ("pointwise").
* ``rms_norm``: h = x + r, y = h * rsqrt(mean(h^2) + eps) * w per row, y in 16
  bits or as e4m3 values with one scale per row.
* ``rms_norm_grad``: dx (added to the gradient that bypasses the norm) and dw.

Matrices are row-major. Row lengths that are not whole 16-byte units are kept
in rows padded up to one, the layout rule of the library's tensor-core entry
points; outputs have no padding.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # One new token through an attention output projection: the weights'
        # bytes and the call's latency are the cost.
        {"name": "decode bf16 1 token", "op": "linear", "dtype": "bf16", "m": 1, "n": 4096,
         "k": 4096, "trans_b": True, "act": "none", "bias": True, "residual": True,
         "preact": False},
        # A small batch of decoding sequences through the widening layer with
        # 8-bit weights and activations.
        {"name": "decode e4m3 24 tokens", "op": "linear", "dtype": "e4m3", "out": "bf16", "m": 24,
         "n": 16384, "k": 4096, "trans_b": True, "act": "gelu_tanh", "bias": True,
         "residual": False, "preact": False},
        # A short fp16 batch with odd sizes, weights stored input-major.
        {"name": "ragged f16 777x1023x513", "op": "linear", "dtype": "f16", "m": 777, "n": 1023,
         "k": 513, "trans_b": False, "act": "silu", "bias": True, "residual": True,
         "preact": False},
        # The widening layer of a training step: the pre-activation is kept for
        # the backward pass.
        {"name": "train up bf16 4096x16384x4096", "op": "linear", "dtype": "bf16", "m": 4096,
         "n": 16384, "k": 4096, "trans_b": True, "act": "gelu_tanh", "bias": True,
         "residual": False, "preact": True},
        # The narrowing layer of a long prefill in 8 bits, added to the
        # residual stream.
        {"name": "prefill e4m3 8192x8192x8192", "op": "linear", "dtype": "e4m3", "out": "bf16",
         "m": 8192, "n": 8192, "k": 8192, "trans_b": True, "act": "none", "bias": False,
         "residual": True, "preact": False},
        # Backward of the widening layer's activation, fused into the product
        # that brings the gradient back through the narrowing layer.
        {"name": "grad product bf16 8192x8192x4096", "op": "linear_grad", "form": "product",
         "dtype": "bf16", "m": 8192, "n": 8192, "k": 4096, "trans_b": False, "act": "gelu_tanh"},
        # The same for a short fp16 batch with odd sizes.
        {"name": "grad product f16 300x1000x520", "op": "linear_grad", "form": "product",
         "dtype": "f16", "m": 300, "n": 1000, "k": 520, "trans_b": True, "act": "silu"},
        # The gradient of a layer whose output gradient is already there.
        {"name": "grad pointwise bf16 8192x4096", "op": "linear_grad", "form": "pointwise",
         "dtype": "bf16", "m": 8192, "n": 4096, "k": 0, "trans_b": False, "act": "gelu"},
        # One token's norm before an 8-bit product: latency.
        {"name": "norm e4m3 1x4096", "op": "rms_norm", "dtype": "bf16", "out": "e4m3", "m": 1,
         "n": 4096, "residual": True, "rstd": False},
        # A training batch's norm: the residual stream and the statistic are kept.
        {"name": "norm bf16 16384x4096", "op": "rms_norm", "dtype": "bf16", "out": "same",
         "m": 16384, "n": 4096, "residual": True, "rstd": True},
        # Its backward pass at a wide model.
        {"name": "norm grad bf16 8192x8192", "op": "rms_norm_grad", "dtype": "bf16", "m": 8192,
         "n": 8192, "bypass": True},
        # A short fp16 batch with an odd width.
        {"name": "norm grad f16 333x1001", "op": "rms_norm_grad", "dtype": "f16", "m": 333,
         "n": 1001, "bypass": False},
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]; half of the draws become a multiple of 160 (when
    large enough: whole 16-byte units, not a power of two), the others are odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = v // 160 * 160 if v >= 160 and rng.random() < 0.5 else v | 1
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "rms_norm", "rms_norm_grad"])
    if op == "linear":
        dtype = rng.choice(["bf16", "f16", "e4m3"])
        case = {"op": op, "dtype": dtype, "m": _size(rng, 1, 8192), "n": _size(rng, 64, 16384),
                "k": _size(rng, 64, 8192),
                "trans_b": True if dtype == "e4m3" else rng.random() < 0.5,
                "act": rng.choice(ACTS), "bias": rng.random() < 0.7,
                "residual": rng.random() < 0.5, "preact": rng.random() < 0.3}
        if dtype == "e4m3":
            case["out"] = rng.choice(["bf16", "f16"])
    elif op == "linear_grad":
        form = rng.choice(["product", "product", "pointwise"])
        case = {"op": op, "form": form, "dtype": rng.choice(["bf16", "f16"]),
                "m": _size(rng, 1, 8192), "n": _size(rng, 64, 16384),
                "k": _size(rng, 64, 8192) if form == "product" else 0,
                "trans_b": form == "product" and rng.random() < 0.5, "act": rng.choice(ACTS[1:])}
    elif op == "rms_norm":
        case = {"op": op, "dtype": rng.choice(["bf16", "f16"]),
                "out": rng.choice(["same", "e4m3"]), "m": _size(rng, 1, 16384),
                "n": _size(rng, 64, 8192), "residual": rng.random() < 0.7,
                "rstd": rng.random() < 0.5}
    else:
        case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "m": _size(rng, 1, 8192),
                "n": _size(rng, 64, 8192), "bypass": rng.random() < 0.7}
    # No more work than the largest listed case.
    while case.get("k") and case["m"] * case["n"] * case["k"] > 8192 ** 3:
        case["m"] = case["m"] // 2 | 1
    return case


def _rows(shape, dtype, unit):
    """An empty rows x cols CUDA matrix whose rows are padded to a multiple of
    `unit` elements."""
    rows, cols = shape
    ld = -(-cols // unit) * unit
    return torch.empty(rows, ld, dtype=dtype, device="cuda")[:, :cols]


def _normal(shape, dtype, gen, std=1.0, unit=8):
    t = _rows(shape, dtype, unit)
    t.copy_(torch.randn(shape, generator=gen, device="cuda") * std)
    return t


def _quantised(shape, gen, std=1.0):
    """Normal values as e4m3 with one scale per row (the largest magnitude of a
    row maps to the format's largest value)."""
    v = torch.randn(shape, generator=gen, device="cuda") * std
    scale = v.abs().amax(1) / E4M3_MAX
    q = _rows(shape, torch.float8_e4m3fn, 16)
    q.copy_((v / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn))
    return q, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, m, n = case["op"], case["m"], case["n"]
    s = dict(case)
    if own:
        from dense_gemm_row_gb300 import binding
        s["lib"] = binding
    if op == "linear":
        k, e4m3 = case["k"], case["dtype"] == "e4m3"
        out = DTYPES[case["out"] if e4m3 else case["dtype"]]
        if e4m3:
            s["A"], s["scale_a"] = _quantised((m, k), gen)
            s["B"], s["scale_b"] = _quantised((n, k), gen, k ** -0.5)
        else:
            s["A"] = _normal((m, k), out, gen)
            s["B"] = _normal((n, k) if case["trans_b"] else (k, n), out, gen, k ** -0.5)
            s["scale_a"] = s["scale_b"] = None
        s["bias"] = torch.randn(n, generator=gen, device="cuda").to(out) if case["bias"] else None
        s["R"] = _normal((m, n), out, gen, unit=1) if case["residual"] else None
        s["D"] = torch.empty(m, n, dtype=out, device="cuda")
        s["Z"] = torch.empty(m, n, dtype=out, device="cuda") if case["preact"] else None
    elif op == "linear_grad":
        dt = DTYPES[case["dtype"]]
        if case["form"] == "product":
            k = case["k"]
            s["A"] = _normal((m, k), dt, gen)
            s["B"] = _normal((n, k) if case["trans_b"] else (k, n), dt, gen, k ** -0.5)
        else:
            s["dD"] = _normal((m, n), dt, gen, unit=1)
        s["Z"] = _normal((m, n), dt, gen, 1.5, unit=1)
        s["dZ"] = torch.empty(m, n, dtype=dt, device="cuda")
        s["dbias"] = torch.empty(n, dtype=dt, device="cuda")
    elif op == "rms_norm":
        dt = DTYPES[case["dtype"]]
        s["X"] = _normal((m, n), dt, gen, unit=1)
        s["R"] = _normal((m, n), dt, gen, 2.0, unit=1) if case["residual"] else None
        s["W"] = (1 + 0.2 * torch.randn(n, generator=gen, device="cuda")).to(dt)
        s["H"] = torch.empty(m, n, dtype=dt, device="cuda") if case["residual"] else None
        s["rstd_out"] = torch.empty(m, device="cuda") if case["rstd"] else None
        if case["out"] == "e4m3":
            s["Y"] = _rows((m, n), torch.float8_e4m3fn, 16)
            s["scale"] = torch.empty(m, device="cuda")
        else:
            s["Y"] = torch.empty(m, n, dtype=dt, device="cuda")
            s["scale"] = None
    else:
        dt = DTYPES[case["dtype"]]
        s["dY"] = _normal((m, n), dt, gen, unit=1)
        s["H"] = _normal((m, n), dt, gen, 2.0, unit=1)
        s["W"] = (1 + 0.2 * torch.randn(n, generator=gen, device="cuda")).to(dt)
        s["rstd"] = torch.rsqrt(s["H"].float().square().mean(1) + EPS)
        s["dH"] = _normal((m, n), dt, gen, unit=1) if case["bypass"] else None
        s["dX"] = torch.empty(m, n, dtype=dt, device="cuda")
        s["dW"] = torch.empty(n, dtype=dt, device="cuda")
    return s


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
        return z / (1 + torch.exp(-2 * u))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = 1 / (1 + torch.exp(-2 * c * (z + 0.044715 * z * z * z)))
        return t + z * t * (1 - t) * 2 * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        t = 1 / (1 + torch.exp(-z))
        return t + z * t * (1 - t)
    return torch.ones_like(z)


def _plain(s):
    op = s["op"]
    if op == "linear":
        B = s["B"].float()
        z = s["A"].float() @ (B.t() if s["trans_b"] else B)
        if s["scale_a"] is not None:
            z = z * s["scale_a"][:, None] * s["scale_b"][None, :]
        if s["bias"] is not None:
            z = z + s["bias"].float()
        d = _act(z, s["act"])
        if s["R"] is not None:
            d = d + s["R"].float()
        out = {"D": d.to(s["D"].dtype)}
        if s["Z"] is not None:
            out["Z"] = z.to(s["D"].dtype)
        return out
    if op == "linear_grad":
        if s["form"] == "product":
            B = s["B"].float()
            g = s["A"].float() @ (B.t() if s["trans_b"] else B)
        else:
            g = s["dD"].float()
        dz = g * _act_grad(s["Z"].float(), s["act"])
        return {"dZ": dz.to(s["dZ"].dtype), "dbias": dz.sum(0).to(s["dZ"].dtype)}
    if op == "rms_norm":
        h = s["X"].float()
        out = {}
        if s["R"] is not None:
            h = h + s["R"].float()
            out["H"] = h.to(s["X"].dtype)
        rstd = torch.rsqrt((h * h).mean(1) + EPS)
        y = h * rstd[:, None] * s["W"].float()
        if s["out"] == "e4m3":
            out["scale"] = y.abs().amax(1) / E4M3_MAX
            q = (y / out["scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            out["Y"] = q.to(torch.float8_e4m3fn)
        else:
            out["Y"] = y.to(s["X"].dtype)
        if s["rstd"]:
            out["rstd"] = rstd
        return out
    dy, w = s["dY"].float(), s["W"].float()
    norm = s["H"].float() * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - norm * (g * norm).mean(1, keepdim=True))
    if s["dH"] is not None:
        dx = dx + s["dH"].float()
    return {"dX": dx.to(s["dX"].dtype), "dW": (dy * norm).sum(0).to(s["dX"].dtype)}


def run(s):
    if not own:
        return _plain(s)
    lib, op = s["lib"], s["op"]
    if op == "linear":
        lib.gemm_epilogue(s["A"], s["B"], s["D"], bias=s["bias"], act=s["act"], residual=s["R"],
                          preact=s["Z"], trans_b=s["trans_b"], scale_a=s["scale_a"],
                          scale_b=s["scale_b"])
        return {"D": s["D"]} if s["Z"] is None else {"D": s["D"], "Z": s["Z"]}
    if op == "linear_grad":
        if s["form"] == "product":
            lib.gemm_dact(s["A"], s["B"], s["Z"], s["dZ"], act=s["act"], dbias=s["dbias"],
                          trans_b=s["trans_b"])
        else:
            lib.act_grad(s["dD"], s["Z"], s["dZ"], act=s["act"], dbias=s["dbias"])
        return {"dZ": s["dZ"], "dbias": s["dbias"]}
    if op == "rms_norm":
        lib.rms_norm(s["X"], s["Y"], weight=s["W"], residual=s["R"], h=s["H"], scale=s["scale"],
                     rstd=s["rstd_out"], eps=EPS)
        out = {"Y": s["Y"]}
        if s["R"] is not None:
            out["H"] = s["H"]
        if s["scale"] is not None:
            out["scale"] = s["scale"]
        if s["rstd"]:
            out["rstd"] = s["rstd_out"]
        return out
    lib.rms_norm_grad(s["dY"], s["H"], s["rstd"], s["dX"], weight=s["W"], dh=s["dH"],
                      dweight=s["dW"])
    return {"dX": s["dX"], "dW": s["dW"]}


def work(case):
    op, m, n = case["op"], case["m"], case["n"]
    if op == "linear":
        k, e4m3 = case["k"], case["dtype"] == "e4m3"
        b = (1 if e4m3 else 2) * (m * k + k * n) + 2 * m * n
        b += 4 * (m + n) if e4m3 else 0
        b += 2 * n if case["bias"] else 0
        b += 2 * m * n * (int(case["residual"]) + int(case["preact"]))
        return {"bytes": b, "flops": 2 * m * n * k}
    if op == "linear_grad":
        b = 2 * (2 * m * n + n)
        if case["form"] == "product":
            return {"bytes": b + 2 * (m + n) * case["k"], "flops": 2 * m * n * case["k"]}
        return {"bytes": b + 2 * m * n, "flops": 2 * m * n}
    if op == "rms_norm":
        b = 2 * m * n + 2 * n + (4 * m * n if case["residual"] else 0)
        b += m * n + 4 * m if case["out"] == "e4m3" else 2 * m * n
        return {"bytes": b + (4 * m if case["rstd"] else 0), "flops": 4 * m * n}
    return {"bytes": 2 * m * n * (4 if case["bypass"] else 3) + 4 * n + 4 * m, "flops": 9 * m * n}


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    n = case["n"]
    if case["op"] == "linear":
        z = torch.einsum("ik,jk->ij" if case["trans_b"] else "ik,kj->ij", wide["A"], wide["B"])
        if "scale_a" in wide:
            z *= torch.outer(wide["scale_a"], wide["scale_b"])
        if "bias" in wide:
            z += wide["bias"]
        out = {"D": _exact_act(z, case["act"])[0]}
        if "R" in wide:
            out["D"] = out["D"] + wide["R"]
        if case["preact"]:
            out["Z"] = z
        return out
    if case["op"] == "linear_grad":
        if case["form"] == "product":
            d = torch.einsum("ik,jk->ij" if case["trans_b"] else "ik,kj->ij", wide["A"], wide["B"])
        else:
            d = wide["dD"]
        d = d * _exact_act(wide["Z"], case["act"])[1]
        return {"dZ": d, "dbias": torch.ones(d.shape[0], dtype=d.dtype, device=d.device) @ d}
    if case["op"] == "rms_norm":
        h = wide["X"] + wide["R"] if "R" in wide else wide["X"]
        rstd = ((torch.linalg.vector_norm(h, dim=1) ** 2) / n + EPS) ** -0.5
        y = torch.einsum("ij,i,j->ij", h, rstd, wide["W"])
        out = {"Y": y}
        if case["out"] == "e4m3":  # the quotients that the 8-bit values round
            out["scale"] = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / E4M3_MAX
            out["Y"] = y / out["scale"].unsqueeze(1)
        if "R" in wide:
            out["H"] = h
        if case["rstd"]:
            out["rstd"] = rstd
        return out
    # y_j = w_j h_j r with r = (|h|^2 / n + eps)^(-1/2): dr/dh_i = -r^3 h_i / n
    r, h, dy = wide["rstd"], wide["H"], wide["dY"]
    along = torch.einsum("ij,ij,j->i", dy, h, wide["W"])
    dx = torch.einsum("ij,i,j->ij", dy, r, wide["W"]) - h * (along * r ** 3 / n).unsqueeze(1)
    if "dH" in wide:
        dx += wide["dH"]
    return {"dX": dx, "dW": torch.einsum("ij,ij,i->j", dy, h, r)}


def _exact_act(z, act):
    """(act(z), act'(z)) in 64 bits."""
    if act == "relu":
        on = (z > 0).double()
        return z * on, on
    if act == "gelu":  # z * Phi(z)
        cdf = 0.5 * torch.special.erfc(-z / 2 ** 0.5)
        return z * cdf, cdf + z * torch.exp(-z ** 2 / 2) / (2 * math.pi) ** 0.5
    if act == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return (0.5 * z * (1 + t),
                0.5 * (1 + t) + 0.5 * z * (1 - t ** 2) * c * (1 + 0.134145 * z ** 2))
    if act == "silu":
        t = torch.sigmoid(z)
        return z * t, t * (1 + z * (1 - t))
    return z, torch.ones_like(z)
