"""The gated feed-forward block, its block-scaled 8-bit form and layer norm as
measured cases.

Six operators, each in a plain form (elementary torch operations in fp32, rounded
once at the end) and, with ``own`` set, through this library's binding:

* ``gated``: D = act(G) * U with the two projections G = A op(Bg) + bg and
  U = A op(Bu) + bu of one input, optionally with G and U written too for the
  backward pass; bf16 and fp16.
* ``gated_grad``: its gradient at the projections, fused into the product
  dD = A op(B) that brings the gradient back through the next layer:
  dG = dD * U * act'(G), dU = dD * act(G), and their column sums.
* ``block``: e4m3 products with a scale for each block of 128: A (tokens) in
  blocks of 1 x 128 along k, B (weights, N x K) in blocks of 128 x 128. Either
  D = act(A B^T + bias) + R or the gated pair of projections.
* ``quantise``: what makes those operands: a scale per block of 128 columns of a
  row, or of 128 rows x 128 columns, and the values divided by it in e4m3.
* ``layer_norm``: h = x + r, y = (h - mean) * rstd * w + b per row.
* ``layer_norm_grad``: dx (added to the gradient that bypasses the norm), dw, db.

Matrices are row-major. Row lengths of products' operands that are not whole
16-byte units are kept in rows padded up to one, the layout rule of the library's
tensor-core entry points; outputs have no padding.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 128
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # One new token through both projections of a gated block: the weights'
        # bytes and the call's latency are the cost.
        {"name": "gated decode bf16 1 token", "op": "gated", "dtype": "bf16", "m": 1, "n": 16384,
         "k": 4096, "trans_b": True, "act": "silu", "bias": False, "keep": False},
        # A training batch: both projections are kept for the backward pass.
        {"name": "gated train bf16 4096x8192x4096", "op": "gated", "dtype": "bf16", "m": 4096,
         "n": 8192, "k": 4096, "trans_b": True, "act": "silu", "bias": False, "keep": True},
        # The backward pass of a training batch through the narrowing layer.
        {"name": "gated grad bf16 8192x8192x4096", "op": "gated_grad", "dtype": "bf16", "m": 8192,
         "n": 8192, "k": 4096, "trans_b": False, "act": "silu", "bias": False},
        # The same for a short fp16 batch with odd sizes and biases.
        {"name": "gated grad f16 300x1000x520", "op": "gated_grad", "dtype": "f16", "m": 300,
         "n": 1000, "k": 520, "trans_b": True, "act": "gelu_tanh", "bias": True},
        # A small batch of decoding sequences through both 8-bit projections.
        {"name": "block gated decode 24 tokens", "op": "block", "gated": True, "out": "bf16",
         "m": 24, "n": 16384, "k": 4096, "act": "silu", "bias": False, "residual": False},
        # The narrowing layer of a long prefill, added to the residual stream.
        {"name": "block prefill 8192x8192x8192", "op": "block", "gated": False, "out": "bf16",
         "m": 8192, "n": 8192, "k": 8192, "act": "none", "bias": False, "residual": True},
        # A prefill's activations on their way into an 8-bit product.
        {"name": "quantise tokens bf16 8192x8192", "op": "quantise", "dtype": "bf16", "m": 8192,
         "n": 8192, "rows": 1},
        # A layer's weights, of an odd size.
        {"name": "quantise weights f16 1001x4095", "op": "quantise", "dtype": "f16", "m": 1001,
         "n": 4095, "rows": 128},
        # One token's norm: latency.
        {"name": "layer norm bf16 1x4096", "op": "layer_norm", "dtype": "bf16", "m": 1, "n": 4096,
         "residual": True, "keep": False},
        # A training batch's norm: the residual stream and the statistics are kept.
        {"name": "layer norm bf16 16384x4096", "op": "layer_norm", "dtype": "bf16", "m": 16384,
         "n": 4096, "residual": True, "keep": True},
        # Its backward pass at a wide model.
        {"name": "layer norm grad bf16 8192x8192", "op": "layer_norm_grad", "dtype": "bf16",
         "m": 8192, "n": 8192, "bypass": True},
        # A short fp16 batch with an odd width.
        {"name": "layer norm grad f16 333x1001", "op": "layer_norm_grad", "dtype": "f16",
         "m": 333, "n": 1001, "bypass": False},
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]; half of the draws become a multiple of 160 (when
    large enough: whole 16-byte units, not a power of two), the others are odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = v // 160 * 160 if v >= 160 and rng.random() < 0.5 else v | 1
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_grad", "block", "block", "quantise", "layer_norm",
                     "layer_norm_grad"])
    if op == "gated":
        case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "m": _size(rng, 1, 8192),
                "n": _size(rng, 64, 16384), "k": _size(rng, 64, 8192),
                "trans_b": rng.random() < 0.6, "act": rng.choice(ACTS[1:]),
                "bias": rng.random() < 0.4, "keep": rng.random() < 0.5}
    elif op == "gated_grad":
        case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "m": _size(rng, 1, 8192),
                "n": _size(rng, 64, 16384), "k": _size(rng, 64, 8192),
                "trans_b": rng.random() < 0.5, "act": rng.choice(ACTS[1:]),
                "bias": rng.random() < 0.5}
    elif op == "block":
        gated = rng.random() < 0.5
        case = {"op": op, "gated": gated, "out": rng.choice(["bf16", "f16"]),
                "m": _size(rng, 1, 8192), "n": _size(rng, 64, 16384), "k": _size(rng, 64, 16384),
                "act": rng.choice(ACTS[1:] if gated else ACTS), "bias": rng.random() < 0.4,
                "residual": not gated and rng.random() < 0.5}
    elif op == "quantise":
        case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "m": _size(rng, 1, 16384),
                "n": _size(rng, 64, 8192), "rows": rng.choice([1, 1, 128])}
    elif op == "layer_norm":
        case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "m": _size(rng, 1, 16384),
                "n": _size(rng, 64, 8192), "residual": rng.random() < 0.7,
                "keep": rng.random() < 0.5}
    else:
        case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "m": _size(rng, 1, 8192),
                "n": _size(rng, 64, 8192), "bypass": rng.random() < 0.7}
    # No more work than the largest listed case.
    pair = 2 if op == "gated" or case.get("gated") else 1
    while case.get("k") and pair * case["m"] * case["n"] * case["k"] > 8192 ** 3:
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


def _spread(scale, rows, shape):
    """A value per block -> a value per element."""
    return (scale.repeat_interleave(rows, 0)[:shape[0]]
            .repeat_interleave(BLOCK, 1)[:, :shape[1]])


def _block_max(x, rows):
    """The largest magnitude of each block of `rows` rows x 128 columns."""
    m, n = x.shape
    mb, nb = -(-m // rows), -(-n // BLOCK)
    full = torch.zeros(mb * rows, nb * BLOCK, dtype=x.dtype, device=x.device)
    full[:m, :n] = x.abs()
    return full.view(mb, rows, nb, BLOCK).amax(3).amax(1)


def _blocks(x, rows):
    """(q, scale) of an fp32 matrix: e4m3 values and a scale per block."""
    scale = _block_max(x, rows) / E4M3_MAX
    wide = _spread(scale, rows, x.shape)
    return (x / wide).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _quantised(shape, rows, gen, std=1.0):
    """Normal values as a product's e4m3 operand. Rows differ in size, as tokens
    and outputs do."""
    x = torch.randn(shape, generator=gen, device="cuda") * std
    x = x * torch.exp(0.5 * torch.randn(shape[0], 1, generator=gen, device="cuda"))
    q = _rows(shape, torch.float8_e4m3fn, 16)
    v, scale = _blocks(x, rows)
    q.copy_(v)
    return q, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, m, n = case["op"], case["m"], case["n"]
    s = dict(case)
    if own:
        from dense_gemm_row_gb300 import binding
        s["lib"] = binding

    def bias(dt):
        return torch.randn(n, generator=gen, device="cuda").to(dt) if case["bias"] else None

    if op == "gated":
        dt, k = DTYPES[case["dtype"]], case["k"]
        weights = (n, k) if case["trans_b"] else (k, n)
        s["A"] = _normal((m, k), dt, gen)
        s["Bg"], s["Bu"] = (_normal(weights, dt, gen, k ** -0.5) for _ in range(2))
        s["bg"], s["bu"] = bias(dt), bias(dt)
        s["D"] = torch.empty(m, n, dtype=dt, device="cuda")
        s["G"], s["U"] = (torch.empty(m, n, dtype=dt, device="cuda") if case["keep"] else None
                          for _ in range(2))
    elif op == "gated_grad":
        dt, k = DTYPES[case["dtype"]], case["k"]
        s["A"] = _normal((m, k), dt, gen)
        s["B"] = _normal((n, k) if case["trans_b"] else (k, n), dt, gen, k ** -0.5)
        s["G"], s["U"] = _normal((m, n), dt, gen, 1.5, unit=1), _normal((m, n), dt, gen, unit=1)
        s["dG"], s["dU"] = (torch.empty(m, n, dtype=dt, device="cuda") for _ in range(2))
        s["dbg"], s["dbu"] = (torch.empty(n, dtype=dt, device="cuda") if case["bias"] else None
                              for _ in range(2))
    elif op == "block":
        dt, k = DTYPES[case["out"]], case["k"]
        s["A"], s["sa"] = _quantised((m, k), 1, gen)
        s["B"], s["sb"] = _quantised((n, k), BLOCK, gen, k ** -0.5)
        s["bias"] = bias(dt)
        s["D"] = torch.empty(m, n, dtype=dt, device="cuda")
        if case["gated"]:
            s["Bu"], s["su"] = _quantised((n, k), BLOCK, gen, k ** -0.5)
            s["bu"] = bias(dt)
        s["R"] = _normal((m, n), dt, gen, unit=1) if case["residual"] else None
    elif op == "quantise":
        dt = DTYPES[case["dtype"]]
        size = torch.exp(torch.randn(m, 1, generator=gen, device="cuda"))
        s["X"] = (torch.randn((m, n), generator=gen, device="cuda") * size).to(dt)
        s["Y"] = _rows((m, n), torch.float8_e4m3fn, 16)
        s["scale"] = torch.empty(-(-m // case["rows"]), -(-n // BLOCK), device="cuda")
    elif op == "layer_norm":
        dt = DTYPES[case["dtype"]]
        s["X"] = _normal((m, n), dt, gen, unit=1)
        s["R"] = _normal((m, n), dt, gen, 2.0, unit=1) if case["residual"] else None
        s["W"] = (1 + 0.2 * torch.randn(n, generator=gen, device="cuda")).to(dt)
        s["b"] = (0.2 * torch.randn(n, generator=gen, device="cuda")).to(dt)
        s["H"] = torch.empty(m, n, dtype=dt, device="cuda") if case["residual"] else None
        s["Y"] = torch.empty(m, n, dtype=dt, device="cuda")
        s["mean"], s["rstd"] = (torch.empty(m, device="cuda") if case["keep"] else None
                                for _ in range(2))
    else:
        dt = DTYPES[case["dtype"]]
        s["dY"] = _normal((m, n), dt, gen, unit=1)
        s["H"] = _normal((m, n), dt, gen, 2.0, unit=1)
        s["W"] = (1 + 0.2 * torch.randn(n, generator=gen, device="cuda")).to(dt)
        h = s["H"].double()
        mean = h.mean(1)
        s["mean"] = mean.float()
        s["rstd"] = torch.rsqrt((h - mean[:, None]).square().mean(1) + EPS).float()
        s["dH"] = _normal((m, n), dt, gen, unit=1) if case["bypass"] else None
        s["dX"] = torch.empty(m, n, dtype=dt, device="cuda")
        s["dW"], s["db"] = (torch.empty(n, dtype=dt, device="cuda") for _ in range(2))
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


def _project(a, b, trans_b, bias):
    z = a @ (b.t() if trans_b else b)
    return z if bias is None else z + bias.float()


def _plain(s):
    op = s["op"]
    if op == "gated":
        a, dt = s["A"].float(), s["D"].dtype
        g = _project(a, s["Bg"].float(), s["trans_b"], s["bg"])
        u = _project(a, s["Bu"].float(), s["trans_b"], s["bu"])
        out = {"D": (_act(g, s["act"]) * u).to(dt)}
        if s["keep"]:
            out["G"], out["U"] = g.to(dt), u.to(dt)
        return out
    if op == "gated_grad":
        d = _project(s["A"].float(), s["B"].float(), s["trans_b"], None)
        g, u, dt = s["G"].float(), s["U"].float(), s["dG"].dtype
        dg, du = d * u * _act_grad(g, s["act"]), d * _act(g, s["act"])
        out = {"dG": dg.to(dt), "dU": du.to(dt)}
        if s["bias"]:
            out["dbg"], out["dbu"] = dg.sum(0).to(dt), du.sum(0).to(dt)
        return out
    if op == "block":
        a = s["A"].float() * _spread(s["sa"], 1, s["A"].shape)
        z = _project(a, s["B"].float() * _spread(s["sb"], BLOCK, s["B"].shape), True, s["bias"])
        d = _act(z, s["act"])
        if s["gated"]:
            d = d * _project(a, s["Bu"].float() * _spread(s["su"], BLOCK, s["Bu"].shape), True,
                             s["bu"])
        if s["R"] is not None:
            d = d + s["R"].float()
        return {"D": d.to(s["D"].dtype)}
    if op == "quantise":
        q, scale = _blocks(s["X"].float(), s["rows"])
        return {"Y": q, "scale": scale}
    if op == "layer_norm":
        h, out = s["X"].float(), {}
        if s["R"] is not None:
            h = h + s["R"].float()
            out["H"] = h.to(s["X"].dtype)
        mean = h.mean(1)
        c = h - mean[:, None]
        rstd = torch.rsqrt((c * c).mean(1) + EPS)
        out["Y"] = (c * rstd[:, None] * s["W"].float() + s["b"].float()).to(s["X"].dtype)
        if s["keep"]:
            out["mean"], out["rstd"] = mean, rstd
        return out
    dy, w = s["dY"].float(), s["W"].float()
    norm = (s["H"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True)
                               - norm * (g * norm).mean(1, keepdim=True))
    if s["dH"] is not None:
        dx = dx + s["dH"].float()
    dt = s["dX"].dtype
    return {"dX": dx.to(dt), "dW": (dy * norm).sum(0).to(dt), "db": dy.sum(0).to(dt)}


def run(s):
    if not own:
        return _plain(s)
    lib, op = s["lib"], s["op"]
    if op == "gated":
        lib.gemm_gated(s["A"], s["Bg"], s["Bu"], s["D"], act=s["act"], bias_gate=s["bg"],
                       bias_up=s["bu"], gate=s["G"], up=s["U"], trans_b=s["trans_b"])
        return {"D": s["D"], "G": s["G"], "U": s["U"]} if s["keep"] else {"D": s["D"]}
    if op == "gated_grad":
        lib.gemm_gated_dact(s["A"], s["B"], s["G"], s["U"], s["dG"], s["dU"], act=s["act"],
                            dbias_gate=s["dbg"], dbias_up=s["dbu"], trans_b=s["trans_b"])
        out = {"dG": s["dG"], "dU": s["dU"]}
        if s["bias"]:
            out["dbg"], out["dbu"] = s["dbg"], s["dbu"]
        return out
    if op == "block":
        if s["gated"]:
            lib.gemm_gated(s["A"], s["B"], s["Bu"], s["D"], act=s["act"], bias_gate=s["bias"],
                           bias_up=s["bu"], trans_b=True, scale_a=s["sa"], scale_gate=s["sb"],
                           scale_up=s["su"])
        else:
            lib.gemm_epilogue(s["A"], s["B"], s["D"], bias=s["bias"], act=s["act"],
                              residual=s["R"], trans_b=True, scale_a=s["sa"], scale_b=s["sb"])
        return {"D": s["D"]}
    if op == "quantise":
        lib.quantise_blocks(s["X"], s["Y"], s["scale"], rows=s["rows"])
        return {"Y": s["Y"], "scale": s["scale"]}
    if op == "layer_norm":
        lib.layer_norm(s["X"], s["Y"], weight=s["W"], bias=s["b"], residual=s["R"], h=s["H"],
                       mean=s["mean"], rstd=s["rstd"], eps=EPS)
        out = {"Y": s["Y"]}
        if s["R"] is not None:
            out["H"] = s["H"]
        if s["keep"]:
            out["mean"], out["rstd"] = s["mean"], s["rstd"]
        return out
    lib.layer_norm_grad(s["dY"], s["H"], s["mean"], s["rstd"], s["dX"], weight=s["W"],
                        dh=s["dH"], dweight=s["dW"], dbias=s["db"])
    return {"dX": s["dX"], "dW": s["dW"], "db": s["db"]}


def work(case):
    op, m, n = case["op"], case["m"], case["n"]
    if op == "gated":
        b = 2 * (m * case["k"] + 2 * n * case["k"] + m * n * (3 if case["keep"] else 1))
        return {"bytes": b + (4 * n if case["bias"] else 0), "flops": 4 * m * n * case["k"]}
    if op == "gated_grad":
        b = 2 * ((m + n) * case["k"] + 4 * m * n) + (4 * n if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * m * n * case["k"]}
    if op == "block":
        k, pair = case["k"], 2 if case["gated"] else 1
        kb, nb = -(-k // BLOCK), -(-n // BLOCK)
        b = m * k + pair * n * k + 4 * kb * (m + pair * nb) + 2 * m * n
        b += (2 * pair * n if case["bias"] else 0) + (2 * m * n if case["residual"] else 0)
        return {"bytes": b, "flops": 2 * pair * m * n * k}
    if op == "quantise":
        blocks = -(-m // case["rows"]) * -(-n // BLOCK)
        return {"bytes": 3 * m * n + 4 * blocks, "flops": 2 * m * n}
    if op == "layer_norm":
        b = 2 * m * n * (4 if case["residual"] else 2) + 4 * n + (8 * m if case["keep"] else 0)
        return {"bytes": b, "flops": 8 * m * n}
    return {"bytes": 2 * m * n * (4 if case["bypass"] else 3) + 6 * n + 8 * m, "flops": 12 * m * n}


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op, n = case["op"], case["n"]
    if op == "gated":
        form = "ik,jk->ij" if case["trans_b"] else "ik,kj->ij"
        g, u = (torch.einsum(form, wide["A"], wide[b]) for b in ("Bg", "Bu"))
        if case["bias"]:
            g, u = g.add_(wide["bg"]), u.add_(wide["bu"])
        out = {"D": torch.einsum("ij,ij->ij", _exact_act(g, case["act"])[0], u)}
        if case["keep"]:
            out["G"], out["U"] = g, u
        return out
    if op == "gated_grad":
        form = "ik,jk->ij" if case["trans_b"] else "ik,kj->ij"
        d = torch.einsum(form, wide["A"], wide["B"])
        value, slope = _exact_act(wide["G"], case["act"])
        out = {"dG": torch.einsum("ij,ij,ij->ij", d, wide["U"], slope),
               "dU": torch.einsum("ij,ij->ij", d, value)}
        if case["bias"]:
            ones = torch.ones(d.shape[0], dtype=d.dtype, device=d.device)
            out["dbg"], out["dbu"] = ones @ out["dG"], ones @ out["dU"]
        return out
    if op == "block":
        # The sum over blocks of the products' sums within a block.
        def product(b, scale):
            z = 0
            for kb in range(scale.shape[1]):
                cols = slice(kb * BLOCK, (kb + 1) * BLOCK)
                part = torch.einsum("ik,jk->ij", wide["A"][:, cols], wide[b][:, cols])
                side = torch.repeat_interleave(scale[:, kb], BLOCK)[:n]
                z = z + part.mul_(wide["sa"][:, kb].unsqueeze(1)).mul_(side)
            return z
        z = product("B", wide["sb"])
        if case["bias"]:
            z = z + wide["bias"]
        d = _exact_act(z, case["act"])[0]
        if case["gated"]:
            u = product("Bu", wide["su"])
            d = d * (u + wide["bu"] if case["bias"] else u)
        return {"D": d + wide["R"] if case["residual"] else d}
    if op == "quantise":  # the quotients that the 8-bit values round
        rows, x = case["rows"], wide["X"]
        scale = torch.empty_like(wide["scale"])
        y = torch.empty_like(x)
        for j in range(scale.shape[1]):
            part = x[:, j * BLOCK:(j + 1) * BLOCK]
            top = torch.linalg.vector_norm(part, ord=math.inf, dim=1)
            for lo in range(0, x.shape[0], rows) if rows > 1 else ():
                top[lo:lo + rows] = torch.linalg.vector_norm(top[lo:lo + rows], ord=math.inf)
            scale[:, j] = top[::rows] / E4M3_MAX
            y[:, j * BLOCK:(j + 1) * BLOCK] = part * (E4M3_MAX / top).unsqueeze(1)
        return {"Y": y, "scale": scale}
    if op == "layer_norm":
        h = wide["X"] + wide["R"] if case["residual"] else wide["X"]
        var, mean = torch.var_mean(h, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.einsum("ij,i,j->ij", h, rstd, wide["W"])
        y = y + wide["b"] - torch.outer(mean * rstd, wide["W"])
        out = {"Y": y}
        if case["residual"]:
            out["H"] = h
        if case["keep"]:
            out["mean"], out["rstd"] = mean, rstd
        return out
    # n_j = (h_j - mean) r: its Jacobian is r (I - 1 1^T / N - n n^T / N)
    r, dy = wide["rstd"], wide["dY"]
    norm = torch.einsum("ij,i->ij", wide["H"] - wide["mean"].unsqueeze(1), r)
    g = torch.einsum("ij,j->ij", dy, wide["W"])
    along, level = torch.einsum("ij,ij->i", g, norm) / n, torch.einsum("ij->i", g) / n
    dx = torch.einsum("ij,i->ij", g - level.unsqueeze(1), r)
    dx -= torch.einsum("ij,i,i->ij", norm, along, r)
    if case["bypass"]:
        dx += wide["dH"]
    return {"dX": dx, "dW": torch.einsum("ij,ij->j", dy, norm), "db": torch.einsum("ij->j", dy)}


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
