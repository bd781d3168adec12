"""The 8-bit linear layer's operators, as they are measured: cases, inputs, plain forms and exact values.

Four operators that a layer with 8-bit weights and activations is made of:

``gemm``      C = alpha A B^T + beta C. A (m x k) and B (n x k) are in 8-bit floating point, with k running fastest;
              A has a scale for each row and 128 elements of k, B for each 128 x 128 block ("tile") or like A ("row").
``quantize``  x in 8 bits with such scales, and on request x^T in 8 bits with its own (the operand of the product that
              sums over x's rows).
``norm``      h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight, and y in 8 bits with a scale for each row and 128 columns.
``backward``  the norm's gradients: of h (and so of x and the residual), and of the weight.

Where ``own`` is false, ``run`` computes them in elementary torch operations in 32 bits; where it is true, it calls the library.
"""
import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}      # the largest finite value of each 8-bit type
DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
TINY = 2.0 ** -100                          # the least |x| maximum that a scale is made for
EPS = 1e-5
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


def _gemm(name, m, n, k, a="e4m3", b="e4m3", block="tile", out="bf16", beta=0.0, pad=0):
    return {"name": name, "op": "gemm", "m": m, "n": n, "k": k, "a": a, "b": b, "block": block, "out": out, "beta": beta, "pad": pad}


def _quantize(name, rows, cols, type="bf16", fmt="e4m3", block="row", both=False, pad=0):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "type": type, "fmt": fmt, "block": block, "both": both, "pad": pad}


def _norm(name, rows, cols, type="bf16", weight="bf16", residual=True, train=False):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "type": type, "weight": weight, "residual": residual, "train": train}


def _backward(name, rows, cols, type="bf16", weight="bf16", residual=True):
    return {"name": name, "op": "backward", "rows": rows, "cols": cols, "type": type, "weight": weight, "residual": residual}


def listed():
    return [
        # One token's product: the weight is read once, and nothing else counts.
        _gemm("gemm one token", 1, 4096, 4096),
        # A small batch of tokens being generated: the skinny layer shape.
        _gemm("gemm 16 tokens", 16, 4096, 4096),
        # A short prompt through a layer-shaped product.
        _gemm("gemm layer", 2048, 4096, 1024),
        # No size a multiple of a tile or of 128, with padded rows.
        _gemm("gemm ragged", 1000, 1300, 700, pad=20, out="fp32"),
        # A training batch's forward product.
        _gemm("gemm batch", 8192, 8192, 4096),
        # The weight's gradient of a layer, added to the one before: sums over the tokens, both operands scaled by rows.
        _gemm("gemm weight gradient", 4096, 4096, 8192, a="e5m2", block="row", out="fp32", beta=1.0),
        # A layer's fp32 weight, after an update, for the forward product and for the input's gradient.
        _quantize("quantize weight", 4096, 4096, type="fp32", block="tile", both=True),
        # A batch's output gradient, for both products of the backward pass.
        _quantize("quantize gradient", 8192, 4096, fmt="e5m2", both=True),
        # One token before a layer.
        _norm("norm one token", 1, 4096),
        # A training batch before a layer: y is kept for the weight's gradient.
        _norm("norm batch", 8192, 4096, train=True),
        _backward("backward batch", 8192, 4096),
        # Few rows of an odd length, no residual branch, in 32 bits.
        _backward("backward ragged", 333, 1300, type="fp32", weight="fp32", residual=False),
    ]


def _log(rng, lo, hi):
    """A whole number, spread evenly over its logarithm: one in two is a multiple of 16 where that leaves it in range."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 0.5 and v >= 16:
        v = v // 16 * 16
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "quantize", "norm", "backward"])
    if op == "gemm":
        while True:
            m, n, k = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 8192)
            if m * n * k <= 8192 * 8192 * 4096:
                break
        c = _gemm("", m, n, k, a=rng.choice(["e4m3", "e4m3", "e5m2"]), b=rng.choice(["e4m3", "e4m3", "e5m2"]), block=rng.choice(["tile", "tile", "row"]),
                  out=rng.choice(["bf16", "bf16", "fp16", "fp32"]), beta=rng.choice([0.0, 0.0, 1.0]), pad=rng.choice([0, 0, 16, 3]))
    else:
        while True:
            rows, cols = _log(rng, 1, 16384), _log(rng, 64, 16384)
            if rows * cols <= 8192 * 4096:
                break
        t = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if op == "quantize":
            c = _quantize("", rows, cols, type=t, fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), block=rng.choice(["row", "row", "tile"]), both=rng.random() < 0.6,
                          pad=rng.choice([0, 0, 8, 3]))
        elif op == "norm":
            c = _norm("", rows, cols, type=t, weight=rng.choice([t, "fp32"]), residual=rng.random() < 0.7, train=rng.random() < 0.5)
        else:
            c = _backward("", rows, cols, type=t, weight=rng.choice([t, "fp32"]), residual=rng.random() < 0.7)
    del c["name"]
    return c


# ---- the plain form


def _blocks(n):
    return (n + 127) // 128


def _amax(x, axis):
    """The largest |x| of each 128 along `axis` (0 or 1) of a matrix: (blocks, n) or (n, blocks)."""
    n = x.shape[axis]
    pad = _blocks(n) * 128 - n
    x = torch.nn.functional.pad(x.abs(), (0, 0, 0, pad) if axis == 0 else (0, pad))
    return x.view(-1, 128, x.shape[1]).amax(1) if axis == 0 else x.view(x.shape[0], -1, 128).amax(2)


def _spread(s, rows, cols, block):
    """A scale for each element of a (rows x cols) operand, from its table."""
    if block == "row":
        return s.repeat_interleave(128, 0)[:cols].T
    return s.repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def _quant(x, fmt, block):
    """(q, scale) of a float32 matrix. Scales by rows are kept as (blocks of columns) x (rows)."""
    a = _amax(x, 1)
    if block == "tile":
        a = _amax(a, 0)
    else:
        a = a.T.contiguous()
    a = a.clamp(min=TINY)
    f = torch.full_like(a, TOP[fmt]) / a     # not TOP / a, which torch computes as a reciprocal and a product
    q = (x * _spread(f, *x.shape, block)).to(F8[fmt])
    return q, a / TOP[fmt]


def _plain_gemm(s):
    c = s["case"]
    a = s["a"].float() * _spread(s["sa"], c["m"], c["k"], "row")
    b = s["b"].float() * _spread(s["sb"], c["n"], c["k"], c["block"])
    r = a @ b.T
    if c["beta"]:
        r = r + c["beta"] * s["c"].float()
    s["c"].copy_(r)
    return s["c"]


def _plain_quantize(s):
    c = s["case"]
    x = s["x"].float()
    got = list(_quant(x, c["fmt"], c["block"]))
    if c["both"]:
        got += _quant(x.T.contiguous(), c["fmt"], c["block"])
    return got


def _plain_norm(s):
    c = s["case"]
    h = s["x"]
    if c["residual"]:
        h = (h.float() + s["r"].float()).to(h.dtype)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(1) + EPS)
    y = f * rstd[:, None] * s["w"].float()
    q, scale = _quant(y, "e4m3", "row")
    got = {"q": q, "scale": scale}
    if c["residual"]:
        got["h"] = h
    if c["train"]:
        got |= {"y": y.to(h.dtype), "rstd": rstd}
    return got


def _plain_backward(s):
    dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    g, u = dy * s["w"].float(), h * rstd
    dx = (g - u * (g * u).mean(1, keepdim=True)) * rstd
    if s["case"]["residual"]:
        dx = dx + s["dh"].float()
    return dx.to(s["dy"].dtype), (dy * u).sum(0)


# ---- the library's calls


def _own_gemm(s):
    import fp32_gemm_nn_amd as mg
    return mg.fp8_gemm(1.0, s["a"], s["sa"], s["b"], s["sb"], s["case"]["beta"], s["c"], block=s["case"]["block"])


def _own_quantize(s):
    import fp32_gemm_nn_amd as mg
    mg.fp8_quantize(s["x"], s["q"], s["scale"], s.get("qt"), s.get("scale_t"), block=s["case"]["block"])
    return [s["q"], s["scale"]] + ([s["qt"], s["scale_t"]] if s["case"]["both"] else [])


def _own_norm(s):
    import fp32_gemm_nn_amd as mg
    mg.rmsnorm(s["x"], s["w"], EPS, residual=s.get("r"), h=s.get("h"), y=s.get("y"), q=s["q"], scale=s["scale"], rstd=s.get("rstd"))
    return {k: s[k] for k in ("q", "scale", "h", "y", "rstd") if k in s}


def _own_backward(s):
    import fp32_gemm_nn_amd as mg
    mg.rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], s["dx"], s["dw"], dh=s.get("dh"))
    return s["dx"], s["dw"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"gemm": _own_gemm, "quantize": _own_quantize, "norm": _own_norm, "backward": _own_backward}[op](state)
    return {"gemm": _plain_gemm, "quantize": _plain_quantize, "norm": _plain_norm, "backward": _plain_backward}[op](state)


# ---- inputs


def _rows(rows, cols, dtype, pad=0):
    """A matrix whose rows are `pad` elements apart."""
    return torch.empty(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]


def _values(g, rows, cols, type, pad=0):
    """Activations or gradients: normal, with the columns of different spread, as those of a network are."""
    spread = torch.exp(0.8 * torch.randn(cols, generator=g, device="cuda"))
    x = _rows(rows, cols, DTYPE[type], pad)
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda") * spread)
    return x


def _operand(g, rows, cols, fmt, block, pad):
    q, scale = _quant(_values(g, rows, cols, "fp32"), fmt, block)
    kept = _rows(rows, cols, F8[fmt], pad)
    kept.copy_(q)
    return kept, scale


def _weight(g, n, type):
    return (1 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(DTYPE[type])


def _out8(rows, cols, fmt, block):
    """Where an operand in 8 bits goes: rows a multiple of 16 bytes apart, as the product reads them fastest."""
    scale = (_blocks(cols), rows) if block == "row" else (_blocks(rows), _blocks(cols))
    return _rows(rows, cols, F8[fmt], -cols % 16), torch.empty(scale, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = _operand(g, m, k, case["a"], "row", -k % 16 + case["pad"])
        s["b"], s["sb"] = _operand(g, n, k, case["b"], case["block"], -k % 16 + case["pad"])
        s["c"] = _values(g, m, n, case["out"])
        return s
    rows, cols, t = case["rows"], case["cols"], case["type"]
    if case["op"] == "quantize":
        s["x"] = _values(g, rows, cols, t, case["pad"])
        s["q"], s["scale"] = _out8(rows, cols, case["fmt"], case["block"])
        if case["both"]:
            s["qt"], s["scale_t"] = _out8(cols, rows, case["fmt"], case["block"])
        return s
    s["w"] = _weight(g, cols, case["weight"])
    if case["op"] == "norm":
        s["x"] = _values(g, rows, cols, t)
        s["q"], s["scale"] = _out8(rows, cols, "e4m3", "row")
        if case["residual"]:
            s["r"], s["h"] = _values(g, rows, cols, t), _rows(rows, cols, DTYPE[t])
        if case["train"]:
            s["y"], s["rstd"] = _rows(rows, cols, DTYPE[t]), torch.empty(rows, device="cuda")
        return s
    s["h"], s["dy"] = _values(g, rows, cols, t), _values(g, rows, cols, t)
    s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
    if case["residual"]:
        s["dh"] = _values(g, rows, cols, t)
    s["dx"], s["dw"] = _rows(rows, cols, DTYPE[t]), torch.empty(cols, device="cuda")
    return s


def work(case):
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        scales = m * _blocks(k) + (n if case["block"] == "row" else _blocks(n)) * _blocks(k)
        c = m * n * SIZE[case["out"]] * (2 if case["beta"] else 1)
        return {"bytes": m * k + n * k + 4 * scales + c, "flops": 2 * m * n * k}
    rows, cols, size = case["rows"], case["cols"], SIZE[case["type"]]
    n = rows * cols
    if case["op"] == "quantize":
        per = lambda r, c: 4 * _blocks(c) * (r if case["block"] == "row" else _blocks(r))  # noqa: E731
        return {"bytes": n * (size + 1) + per(rows, cols) + (n + per(cols, rows) if case["both"] else 0), "flops": 3 * n}
    w = cols * SIZE[case["weight"]]
    if case["op"] == "norm":
        moved = size * (1 + 2 * case["residual"] + case["train"]) + 1
        return {"bytes": n * moved + w + 4 * rows * (_blocks(cols) + case["train"]), "flops": 7 * n}
    return {"bytes": n * size * (3 + case["residual"]) + w + 4 * rows + 4 * cols, "flops": 10 * n}


# ---- the definition, in 64 bits


def _each(s, rows, cols, block):
    i = torch.arange(rows, device=s.device)[:, None]
    j = torch.arange(cols, device=s.device)[None] // 128
    s = s.double()
    return s[j, i] if block == "row" else s[i // 128, j]


def _grid(x, fmt):
    """x rounded to the nearest value of an 8-bit type, ties to even, in 64 bits."""
    digits, least = (3, -6) if fmt == "e4m3" else (2, -14)
    e = (torch.frexp(x)[1] - 1).clamp(min=least)
    step = torch.ldexp(torch.ones_like(x), e - digits)
    return torch.round(x / step) * step


def _exact_quant(x, fmt, block):
    rows, cols = x.shape
    row = torch.arange(rows, device=x.device)[:, None].expand(rows, cols)
    col = torch.arange(cols, device=x.device)[None].expand(rows, cols) // 128
    shape = (_blocks(cols), rows) if block == "row" else (_blocks(rows), _blocks(cols))
    at = col * rows + row if block == "row" else row // 128 * _blocks(cols) + col
    a = torch.full((shape[0] * shape[1],), TINY, dtype=torch.float64, device=x.device)
    a = a.scatter_reduce(0, at.reshape(-1), x.abs().reshape(-1), "amax")
    s = a / TOP[fmt]
    return [_grid(x / s[at], fmt), s.view(shape)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        a = s["a"].double() * _each(s["sa"], case["m"], case["k"], "row")
        b = s["b"].double() * _each(s["sb"], case["n"], case["k"], case["block"])
        return torch.addmm(s["c"].double(), a, b.T.contiguous(), beta=case["beta"])
    if case["op"] == "quantize":
        x = s["x"].double()
        got = _exact_quant(x, case["fmt"], case["block"])
        return got + (_exact_quant(x.T.contiguous(), case["fmt"], case["block"]) if case["both"] else [])
    w = s["w"].double()
    if case["op"] == "norm":
        h = s["x"].double()
        if case["residual"]:
            h = (h + s["r"].double()).to(s["x"].dtype).double()      # the sum is kept, and used, in x's type
        rstd = (h.pow(2).sum(1) / case["cols"] + EPS).pow(-0.5)
        y = torch.einsum("ij,i,j->ij", h, rstd, w)
        # y in 8 bits has no one value here: next to a border of two, 32 bits of y may fall on either side.
        got = {"q": None, "scale": _exact_quant(y, "e4m3", "row")[1]}
        if case["residual"]:
            got["h"] = h
        if case["train"]:
            got |= {"y": y, "rstd": rstd}
        return got
    # The gradient of sum(dy * y), by the chain rule through r = (mean(h^2) + eps)^-1/2 as it was kept.
    h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double().unsqueeze(1)
    through = (dy * w * h).sum(1, keepdim=True)                      # d / d r
    dx = dy * w * r - through * r.pow(3) * h / case["cols"]
    if case["residual"]:
        dx = dx + s["dh"].double()
    return dx, torch.mv((h * r * dy).T, torch.ones(case["rows"], dtype=torch.float64, device=h.device))
