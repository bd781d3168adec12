"""The feed-forward block's operators in 16 bits, as they are measured: cases, inputs, plain forms and exact values.

Three operators that the block between two norms is made of, in BF16 or FP16:

``linear``    z = op(A) op(B) + bias, C = act(z) + beta R, with op N or T: the layer's product, and those of its gradients.
              z may be kept for the backward pass, in 16 bits or in 8 with a scale for each row and 128 columns.
``gated``     g = A G^T + bias, u = A U^T + bias, h = act(g) u, with g and u kept likewise.
``backward``  from the gradient of act(z) or of act(g) u, and the kept z, or g and u: their gradients, the value that
              the block went on with (an operand of the next weight's gradient), and the sums over rows that are the biases' gradients.

Where ``own`` is false, ``run`` computes them in elementary torch operations in 32 bits; where it is true, it calls the library.
"""
import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}      # the largest finite value of each 8-bit type
DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2, "e4m3": 1, "e5m2": 1}
TINY = 2.0 ** -100                          # the least |x| maximum that a scale is made for
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _linear(name, m, n, k, ta="N", tb="T", type="bf16", out="bf16", bias="", act="none", residual="", keep="", pad=0):
    """`bias`, `keep`: a type, or "" for none. `residual`: "" none, "own" a matrix of its own, "c" C as it was. `pad`: elements between rows."""
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "ta": ta, "tb": tb, "type": type, "out": out, "bias": bias, "act": act,
            "residual": residual, "keep": keep, "pad": pad}


def _gated(name, m, n, k, type="bf16", out="bf16", bias="", act="silu", keep="", pad=0):
    return {"name": name, "op": "gated", "m": m, "n": n, "k": k, "type": type, "out": out, "bias": bias, "act": act, "keep": keep, "pad": pad}


def _backward(name, rows, cols, gated, type="bf16", act="silu", keep="e4m3", value=True, bias=False, pad=0):
    return {"name": name, "op": "backward", "rows": rows, "cols": cols, "gated": gated, "type": type, "act": act, "keep": keep, "value": value, "bias": bias,
            "pad": pad}


def listed():
    return [
        # One token back down to the block's width, onto its residual: the weight is read once, and nothing else counts.
        _linear("linear one token", 1, 4096, 8192, residual="own"),
        # A small batch of tokens being generated through a layer with bias and activation; an odd number of them.
        _linear("linear 33 tokens", 33, 4096, 4096, bias="bf16", act="gelu"),
        # No size a multiple of a tile, rows that no wide read fits; results in 32 bits.
        _linear("linear ragged", 1000, 1300, 700, type="fp16", out="fp32", bias="fp32", act="silu", residual="own", pad=3),
        # A training batch's first layer: z is kept in 8 bits for the backward pass.
        _linear("linear batch", 8192, 8192, 4096, bias="bf16", act="gelu_tanh", keep="e4m3"),
        # The input's gradient, from the second of two projections: onto the first one's.
        _linear("linear input gradient", 8192, 4096, 8192, tb="N", residual="c"),
        # A weight's gradient: summed over the tokens, added in 32 bits to the one before.
        _linear("linear weight gradient", 4096, 4096, 8192, ta="T", tb="N", out="fp32", residual="c"),
        # One token into the gated block.
        _gated("gated one token", 1, 8192, 4096),
        # A short prompt through it; nothing is kept.
        _gated("gated prompt", 500, 4096, 2048, act="gelu_tanh"),
        # A training batch: g and u are kept in 8 bits.
        _gated("gated batch", 8192, 8192, 4096, keep="e4m3"),
        # That batch's gradients from the 8-bit checkpoints, and h again for the next weight's.
        _backward("backward batch", 8192, 8192, True),
        # One layer with a bias, odd sizes, its checkpoint in 16 bits.
        _backward("backward ragged", 777, 1300, False, type="fp16", act="gelu", keep="fp16", value=False, bias=True, pad=1),
        # Few rows, checkpoints in 8 bits with a wider range, biases for both projections.
        _backward("backward few rows", 64, 4096, True, act="gelu_tanh", keep="e5m2", bias=True),
    ]


def _log(rng, lo, hi):
    """A whole number, spread evenly over its logarithm: one in two is a multiple of 16 where that leaves it in range."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 0.5 and v >= 16:
        v = v // 16 * 16
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "gated", "gated", "backward"])
    t = rng.choice(["bf16", "bf16", "fp16"])
    if op == "backward":
        t = rng.choice([t, t, "fp32"])
        while True:
            rows, cols = _log(rng, 1, 16384), _log(rng, 16, 16384)
            if rows * cols <= 8192 * 8192:
                break
        c = _backward("", rows, cols, rng.random() < 0.6, type=t, act=rng.choice(ACTS), keep=rng.choice(["e4m3", "e4m3", "e5m2", t]), value=rng.random() < 0.6,
                      bias=rng.random() < 0.4, pad=rng.choice([0, 0, 8, 3]))
    else:
        while True:
            m, n, k = _log(rng, 1, 8192), _log(rng, 16, 8192), _log(rng, 16, 8192)
            if m * n * k <= 8192 * 8192 * 4096:
                break
        more = {"type": t, "out": rng.choice([t, t, "fp32"]), "bias": rng.choice(["", t, "fp32"]), "act": rng.choice(ACTS), "pad": rng.choice([0, 0, 8, 3])}
        more["keep"] = rng.choice(["", "", "e4m3", "e5m2", more["out"]])
        if op == "linear":
            c = _linear("", m, n, k, ta=rng.choice("NNT"), tb=rng.choice("TTN"), residual=rng.choice(["", "own", "c"]), **more)
        else:
            c = _gated("", m, n, k, **more)
    del c["name"]
    return c


# ---- the plain form


def _blocks(n):
    return (n + 127) // 128


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _slope(z, act):
    """The derivative of act at z."""
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _each(scale, cols):
    """A scale for each element, from its table of (blocks of columns) x (rows)."""
    return scale.repeat_interleave(128, 0)[:cols].T


def _quant(x, fmt):
    """(q, scale) of a float32 matrix, with a scale for each row and 128 columns."""
    rows, cols = x.shape
    a = torch.nn.functional.pad(x.abs(), (0, -cols % 128)).view(rows, -1, 128).amax(2).T.contiguous().clamp(min=TINY)
    f = torch.full_like(a, TOP[fmt]) / a     # not TOP / a, which torch computes as a reciprocal and a product
    return (x * _each(f, cols)).to(F8[fmt]), a / TOP[fmt]


def _keep(z, kind, out):
    """What is kept of z: a pair in 8 bits, or one matrix."""
    return list(_quant(z, kind)) if kind in F8 else [z.to(DTYPE[out])]


def _kept(s, name):
    """The same read back, in 32 bits."""
    z = s[name].float()
    return z * _each(s[name + "s"], z.shape[1]) if s["case"]["keep"] in F8 else z


def _plain_linear(s):
    c = s["case"]
    a, b = s["a"].float(), s["b"].float()
    z = (a.T if c["ta"] == "T" else a) @ (b.T if c["tb"] == "T" else b)
    if c["bias"]:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + s["r" if c["residual"] == "own" else "c"].float()
    s["c"].copy_(y)
    return [s["c"]] + (_keep(z, c["keep"], c["out"]) if c["keep"] else [])


def _plain_gated(s):
    c = s["case"]
    a = s["a"].float()
    g, u = a @ s["g"].float().T, a @ s["u"].float().T
    if c["bias"]:
        g, u = g + s["bg"].float(), u + s["bu"].float()
    got = [(_act(g, c["act"]) * u).to(DTYPE[c["out"]])]
    return got + (_keep(g, c["keep"], c["out"]) + _keep(u, c["keep"], c["out"]) if c["keep"] else [])


def _plain_backward(s):
    c, t, dy = s["case"], DTYPE[s["case"]["type"]], s["dy"].float()
    if not c["gated"]:
        z = _kept(s, "z")
        dz = dy * _slope(z, c["act"])
        return [dz.to(t)] + ([_act(z, c["act"]).to(t)] if c["value"] else []) + ([dz.sum(0)] if c["bias"] else [])
    g, u = _kept(s, "g"), _kept(s, "u")
    v = _act(g, c["act"])
    dg, du = dy * u * _slope(g, c["act"]), dy * v
    return [dg.to(t), du.to(t)] + ([(v * u).to(t)] if c["value"] else []) + ([dg.sum(0), du.sum(0)] if c["bias"] else [])


# ---- the library's calls


def _own_linear(s):
    import fp32_gemm_nn_amd as mg
    c = s["case"]
    mg.linear(c["ta"], c["tb"], 1.0, s["a"], s["b"], 1.0 if c["residual"] else 0.0, s["c"], bias=s.get("bias"), act=c["act"], residual=s.get("r"),
              z=s.get("z"), scale=s.get("zs"))
    return [s["c"]] + [s[k] for k in ("z", "zs") if k in s]


def _own_gated(s):
    import fp32_gemm_nn_amd as mg
    c = s["case"]
    mg.gated(s["a"], s["g"], s["u"], s["h"], act=c["act"], bias_g=s.get("bg"), bias_u=s.get("bu"), g=s.get("zg"), scale_g=s.get("zgs"), u=s.get("zu"),
             scale_u=s.get("zus"))
    return [s["h"]] + [s[k] for k in ("zg", "zgs", "zu", "zus") if k in s]


def _own_backward(s):
    import fp32_gemm_nn_amd as mg
    c = s["case"]
    if c["gated"]:
        mg.gated_backward(s["dy"], s["g"], s["u"], s["dg"], s["du"], scale_g=s.get("gs"), scale_u=s.get("us"), act=c["act"], h=s.get("y"),
                          dbias_g=s.get("dbg"), dbias_u=s.get("dbu"))
    else:
        mg.act_backward(s["dy"], s["z"], s["dz"], scale=s.get("zs"), act=c["act"], y=s.get("y"), dbias=s.get("db"))
    return [s[k] for k in ("dz", "dg", "du", "y", "db", "dbg", "dbu") if k in s]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "gated": _own_gated, "backward": _own_backward}[op](state)
    return {"linear": _plain_linear, "gated": _plain_gated, "backward": _plain_backward}[op](state)


# ---- inputs


def _rows(rows, cols, dtype, pad=0):
    """A matrix whose rows are `pad` elements apart."""
    return torch.empty(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]


def _values(g, rows, cols, type, pad=0, size=1.0):
    """Activations or gradients: normal, with the columns of different spread, as those of a network are."""
    spread = size * torch.exp(0.8 * torch.randn(cols, generator=g, device="cuda"))
    x = _rows(rows, cols, DTYPE[type], pad)
    x.copy_(torch.randn(rows, cols, generator=g, device="cuda") * spread)
    return x


def _weight(g, rows, cols, k, type, pad):
    """A projection's weight: normal, of the size that keeps its outputs as large as its inputs."""
    w = _rows(rows, cols, DTYPE[type], pad)
    w.copy_(torch.randn(rows, cols, generator=g, device="cuda") / math.sqrt(k))
    return w


def _bias(g, n, type):
    return (0.3 * torch.randn(n, generator=g, device="cuda")).to(DTYPE[type])


def _room(s, name, rows, cols, kind, out, pad):
    """Where z goes: an 8-bit pair, or a matrix of the result's type."""
    if kind in F8:
        s[name], s[name + "s"] = _rows(rows, cols, F8[kind], -cols % 16 + pad), torch.empty(_blocks(cols), rows, device="cuda")
    elif kind:
        s[name] = _rows(rows, cols, DTYPE[out], pad)


def _checkpoint(s, g, name, rows, cols, c):
    """A z as the forward pass left it."""
    z = _values(g, rows, cols, "fp32")
    _room(s, name, rows, cols, c["keep"], c["type"], c["pad"])
    if c["keep"] in F8:
        q, scale = _quant(z, c["keep"])
        s[name].copy_(q)
        s[name + "s"].copy_(scale)
    else:
        s[name].copy_(z)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s, c, pad = {"case": case}, case, case["pad"]
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        # A layer's product and its input's gradient have a weight as B; summed over the tokens both are activations, a gradient among them small.
        s["a"] = _values(g, *((k, m) if c["ta"] == "T" else (m, k)), c["type"], pad, size=0.02 if c["ta"] == "T" else 1.0)
        rows, cols = (n, k) if c["tb"] == "T" else (k, n)
        s["b"] = _values(g, rows, cols, c["type"], pad) if c["ta"] == "T" else _weight(g, rows, cols, k, c["type"], pad)
        s["c"] = _values(g, m, n, c["out"], pad)
        if c["bias"]:
            s["bias"] = _bias(g, n, c["bias"])
        if c["residual"] == "own":
            s["r"] = _values(g, m, n, c["out"], pad)
        _room(s, "z", m, n, c["keep"], c["out"], pad)
        return s
    if c["op"] == "gated":
        m, n, k = c["m"], c["n"], c["k"]
        s["a"] = _values(g, m, k, c["type"], pad)
        s["g"], s["u"] = _weight(g, n, k, k, c["type"], pad), _weight(g, n, k, k, c["type"], pad)
        s["h"] = _rows(m, n, DTYPE[c["out"]], pad)
        if c["bias"]:
            s["bg"], s["bu"] = _bias(g, n, c["bias"]), _bias(g, n, c["bias"])
        _room(s, "zg", m, n, c["keep"], c["out"], pad)
        _room(s, "zu", m, n, c["keep"], c["out"], pad)
        return s
    rows, cols, t = c["rows"], c["cols"], c["type"]
    s["dy"] = _values(g, rows, cols, t, pad)
    for name in ("g", "u") if c["gated"] else ("z",):
        _checkpoint(s, g, name, rows, cols, c)
        s["d" + name] = _rows(rows, cols, DTYPE[t], pad)
        if c["bias"]:
            s["db" + (name if c["gated"] else "")] = torch.empty(cols, device="cuda")
    if c["value"]:
        s["y"] = _rows(rows, cols, DTYPE[t], pad)
    return s


def work(case):
    c = case
    if c["op"] == "backward":
        n, z = c["rows"] * c["cols"], 1 + c["gated"]
        tables = 4 * c["rows"] * _blocks(c["cols"]) if c["keep"] in F8 else 0
        moved = SIZE[c["type"]] * (1 + z + c["value"]) + z * SIZE[c["keep"]]
        return {"bytes": n * moved + z * tables + (4 * z * c["cols"] if c["bias"] else 0), "flops": 12 * n}
    m, n, k = c["m"], c["n"], c["k"]
    weights = 2 if c["op"] == "gated" else 1
    moved = SIZE[c["type"]] * (m * k + weights * n * k) + SIZE[c["out"]] * m * n
    if c["keep"]:
        moved += weights * m * (n * SIZE[c["keep"]] + (4 * _blocks(n) if c["keep"] in F8 else 0))
    if c["bias"]:
        moved += weights * n * SIZE[c["bias"]]
    if c.get("residual"):
        moved += SIZE[c["out"]] * m * n
    return {"bytes": moved, "flops": 2 * weights * m * n * k}


# ---- the definition, in 64 bits


def _exact_act(z, act):
    """(value, derivative)."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if act == "gelu":
        phi = torch.erfc(-z / 2 ** 0.5) / 2
        return z * phi, phi + z * torch.exp(-z.pow(2) / 2) / (2 * math.pi) ** 0.5
    # The other two are z / (1 + e^-p): p = z, and p = 2 sqrt(2/pi) (z + 0.044715 z^3).
    c = (8 / math.pi) ** 0.5
    p, dp = (z, torch.ones_like(z)) if act == "silu" else (c * (z + 0.044715 * z.pow(3)), c * (1 + 0.134145 * z.pow(2)))
    e = torch.exp(-p)
    return z / (1 + e), 1 / (1 + e) + z * dp / ((1 + e) * (1 + 1 / e))


def _exact_keep(z, kind):
    """The table of scales; 8 bits themselves have no one value here: next to a border of two, 32 bits of z may fall on either side."""
    if kind not in F8:
        return [z]
    a = torch.stack([part.abs().max(1).values for part in z.split(128, 1)])
    return [None, torch.maximum(a, torch.full_like(a, TINY)) / TOP[kind]]


def _exact_kept(z, scale):
    if scale is None:
        return z.double()
    return torch.cat([part.double() * scale[b].double()[:, None] for b, part in enumerate(z.float().split(128, 1))], 1)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "linear":
        a, b = s["a"].double(), s["b"].double()
        a, b = a.T.contiguous() if c["ta"] == "T" else a, b.T.contiguous() if c["tb"] == "T" else b
        z = torch.mm(a, b)
        if "bias" in s:
            z += s["bias"].double()
        y = _exact_act(z, c["act"])[0]
        if c["residual"]:
            y = y + (s["r"] if "r" in s else s["c"]).double()
        return [y] + (_exact_keep(z, c["keep"]) if c["keep"] else [])
    if c["op"] == "gated":
        a = s["a"].double()
        both = []
        for w, bias in (("g", "bg"), ("u", "bu")):
            z = torch.mm(a, s[w].double().T.contiguous())
            both.append(z + s[bias].double() if bias in s else z)
        g, u = both
        return [u * _exact_act(g, c["act"])[0]] + (_exact_keep(g, c["keep"]) + _exact_keep(u, c["keep"]) if c["keep"] else [])
    dy = s["dy"].double()
    if c["gated"]:
        g, u = (_exact_kept(s[n], s.get(n + "s")) for n in "gu")
        v, slope = _exact_act(g, c["act"])
        grads, value = [u * slope * dy, v * dy], v * u
    else:
        v, slope = _exact_act(_exact_kept(s["z"], s.get("zs")), c["act"])
        grads, value = [slope * dy], v
    return grads + ([value] if c["value"] else []) + ([torch.mv(x.T, x.new_ones(c["rows"])) for x in grads] if c["bias"] else [])
