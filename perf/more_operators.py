"""Cases of the residual block's operators: inputs, plain forms, exact values and the work each call cannot do without.

What a deep network keeps and computes around each of its layers when it is trained:

* the norms after and before a block, fused with the block's gate, its residual scale and the addition to the
  residual stream, forward and backward:  v = norm(u) pw + pb,  r = alpha x + s a(g) v,  y = norm(r) w + b;
* activations kept in 8 bits for the backward pass: blocks of 32 elements of a row share a power of two;
* the backward pass from them: the fused norms' own, and the weight gradient of a linear layer,
  dw = dy^T x, whose input was kept so.

``run`` computes an operator in elementary torch operations in 32 bits, rounded once at the end, or, where ``own`` is
set, through the package's entry points.  ``exact`` computes the same from the definitions in 64 bits.
"""

import math

import torch

own = False

GROUP = 32  # elements of a row that share a scale
LEAST = 6  # least scale byte: no unit below 2^-127
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5


def _residual(name, mode, rows, cols, dtype, *, stream="same", norm="layer", post=True, gate="full", act="none", scale="vector",
              kept="plain"):
    return {"name": name, "op": "residual", "mode": mode, "rows": rows, "cols": cols, "dtype": dtype, "stream": stream,
            "norm": norm, "post": post, "gate": gate, "act": act, "scale": scale, "kept": kept}


def listed():
    return [
        # between two small layers: the call's latency is what counts
        _residual("residual forward 16x512 f32", "forward", 16, 512, "f32", gate="none"),
        # inference or the first half of a training step over a full batch, the stream kept wider than the block
        _residual("residual forward 16384x4096 bf16", "forward", 16384, 4096, "bf16", stream="f32", norm="rms", act="silu"),
        # backward alone, at a width that no vector load divides (a ragged feature count), a gate for each token
        _residual("residual backward 2999x1001 f32", "backward", 2999, 1001, "f32", gate="row"),
        # a training step of a large batch: forward leaves 8-bit copies, backward reads them
        _residual("residual step 16384x4096 bf16 8-bit", "step", 16384, 4096, "bf16", kept="8bit"),
        # backward of wide rows in half precision from 8-bit copies
        _residual("residual backward 4096x8192 f16 8-bit", "backward", 4096, 8192, "f16", norm="rms", act="sigmoid", kept="8bit"),
        # a small activation kept and read back: latency
        {"name": "kept 16x512 f32", "op": "kept", "mode": "round", "rows": 16, "cols": 512, "dtype": "f32"},
        # a large batch's activation kept and read back, bound by memory
        {"name": "kept 32768x4096 bf16", "op": "kept", "mode": "round", "rows": 32768, "cols": 4096, "dtype": "bf16"},
        # read back alone, at a ragged width whose last group is part-filled
        {"name": "values 40950x1001 f16", "op": "kept", "mode": "values", "rows": 40950, "cols": 1001, "dtype": "f16"},
        # the weight gradient of a toy layer: one tile, latency
        {"name": "weight grad 7x64x96 bf16", "op": "grad", "tokens": 7, "out": 64, "in": 96, "dtype": "bf16", "to": "same",
         "bias": True},
        # ragged in every direction, half precision, with the bias's gradient
        {"name": "weight grad 1021x2003x1000 f16", "op": "grad", "tokens": 1021, "out": 2003, "in": 1000, "dtype": "f16",
         "to": "same", "bias": True},
        # few tokens and a large layer, 32-bit gradients: bound by writing them
        {"name": "weight grad 64x16384x4096 bf16", "op": "grad", "tokens": 64, "out": 16384, "in": 4096, "dtype": "bf16",
         "to": "f32", "bias": False},
        # a training batch: bound by the products
        {"name": "weight grad 8192x8192x8192 bf16", "op": "grad", "tokens": 8192, "out": 8192, "in": 8192, "dtype": "bf16",
         "to": "same", "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["residual", "residual", "kept", "grad"])
    if op == "grad":
        while True:
            t, o, i = _log(rng, 1, 16384), _log(rng, 16, 16384), _log(rng, 16, 16384)
            if t * o * i <= 8192 ** 3 and o * i <= 1 << 27:
                return {"op": op, "tokens": t, "out": o, "in": i, "dtype": rng.choice(["bf16", "f16"]),
                        "to": rng.choice(["same", "f32"]), "bias": rng.random() < 0.5}
    while True:
        rows, cols = _log(rng, 1, 65536), _log(rng, 16, 16384)
        if rows * cols <= 16384 * 4096:
            break
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "kept":
        return {"op": op, "mode": rng.choice(["round", "values"]), "rows": rows, "cols": cols, "dtype": dtype}
    kept = rng.choice(["plain", "8bit"])
    modes = ["forward", "backward"] if kept == "8bit" and dtype == "f32" else ["forward", "backward", "step"]
    case = _residual("", rng.choice(modes), rows, cols, dtype, stream=rng.choice(["same", "f32"]), norm=rng.choice(["layer", "rms"]),
                     post=rng.random() < 0.75, gate=rng.choice(["none", "row", "full", "full"]),
                     act=rng.choice(["none", "sigmoid", "silu"]), scale=rng.choice(["number", "vector"]), kept=kept)
    if kept == "8bit" and case["mode"] == "step":
        case["stream"] = "same"
    del case["name"]
    return case


# ------------------------------------------------------------------ 8-bit copies, in 32 bits


def _pack(x):
    """Codes (in rows of whole groups of bytes) and scale bytes of a matrix: exact, since the units are powers of two."""
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    padded = torch.zeros(rows, groups * GROUP, device=x.device)
    padded[:, :cols] = x
    blocks = padded.view(rows, groups, GROUP)
    byte = ((blocks.abs().amax(2).view(torch.int32) >> 23) & 255).clamp(min=LEAST)
    codes = torch.round(blocks * _power(133 - byte)[..., None]).clamp(-127, 127)
    return codes.view(rows, -1).to(torch.int8)[:, :cols], byte.to(torch.uint8)


def _power(n):
    """2^n for whole n from -127 to 127, exactly."""
    half = torch.where(n < -126, 0.5, 1.0)
    return ((n.clamp(min=-126) + 127) << 23).to(torch.int32).view(torch.float32) * half


def _values(codes, scales):
    unit = _power(scales.to(torch.int32) - 133).repeat_interleave(GROUP, 1)
    return codes.float() * unit[:, :codes.shape[1]]


# ------------------------------------------------------------------ inputs


def _types(case):
    dt = DTYPES[case["dtype"]]
    return dt, torch.float32 if case["stream"] == "f32" else dt


def _options(case):
    return dict(gate_act=case["act"], post_norm=case["post"], norm=case["norm"], alpha=0.9)


def _prepare_residual(case, gen):
    rows, cols = case["rows"], case["cols"]
    dt, st = _types(case)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    spread = 0.5 + 1.5 * torch.rand(cols, generator=gen, device="cuda")  # features of unlike size
    s = {"x": (normal(rows, cols) * spread).to(st), "u": (normal(rows, cols) * spread + normal(rows, 1)).to(dt),
         "weight": (1 + 0.1 * normal(cols)).to(dt), "bias": None, "post_weight": None, "post_bias": None, "gate": None}
    if case["norm"] == "layer":
        s["bias"] = (0.1 * normal(cols)).to(dt)
    if case["post"]:
        s["post_weight"] = (1 + 0.1 * normal(cols)).to(dt)
        if case["norm"] == "layer":
            s["post_bias"] = (0.1 * normal(cols)).to(dt)
    if case["gate"] != "none":
        s["gate"] = normal(rows, cols if case["gate"] == "full" else 1).to(dt)
    s["scale"] = (0.3 + 0.05 * normal(cols)).to(dt) if case["scale"] == "vector" else 0.3
    if case["mode"] != "forward":
        s["dy"], s["dr"] = normal(rows, cols).to(dt), normal(rows, cols).to(st)
    if case["mode"] == "backward":  # what the forward call left behind
        _, r, s["stats"] = _residual_forward(s, case)
        s["r"] = r.to(st)
        del s["x"]
        if case["kept"] == "8bit":
            for k in ("u", "r") + (("gate",) if case["gate"] == "full" else ()):
                s[k] = _pack(s[k].float())
    return s


def _prepare_kept(case, gen):
    x = torch.randn(case["rows"], case["cols"], generator=gen, device="cuda")
    x *= torch.exp(torch.randn(case["cols"], generator=gen, device="cuda"))  # a few features much larger than the others
    x = x.to(DTYPES[case["dtype"]])
    return {"x": x} if case["mode"] == "round" else {"kept": _pack(x.float())}


def _prepare_grad(case, gen):
    t, o, i = case["tokens"], case["out"], case["in"]
    dt = DTYPES[case["dtype"]]
    x = torch.randn(t, i, generator=gen, device="cuda")
    x *= 0.5 + 1.5 * torch.rand(i, generator=gen, device="cuda")
    return {"kept": _pack(x.to(dt).float()), "dy": torch.randn(t, o, generator=gen, device="cuda").to(dt)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    make = {"residual": _prepare_residual, "kept": _prepare_kept, "grad": _prepare_grad}[case["op"]]
    return {"case": dict(case), **make(case, gen)}


# ------------------------------------------------------------------ plain forms, in 32 bits


def _stats(t, norm):
    mean = t.mean(1) if norm == "layer" else torch.zeros_like(t[:, 0])
    centred = t - mean[:, None]
    return mean, 1 / torch.sqrt((centred * centred).mean(1) + EPS)


def _affine(h, weight, bias):
    h = h if weight is None else h * weight.float()
    return h if bias is None else h + bias.float()


def _gate(g, act):
    """The gate's value and its derivative."""
    g = g.float()
    if act == "none":
        return g, torch.ones_like(g)
    sig = 1 / (1 + torch.exp(-g))
    return (sig, sig * (1 - sig)) if act == "sigmoid" else (g * sig, sig * (1 + g * (1 - sig)))


def _number(scale):
    return scale if isinstance(scale, float) else scale.float()


def _residual_forward(s, case):
    u = s["u"].float()
    pm, pr = torch.zeros_like(u[:, 0]), torch.ones_like(u[:, 0])
    v = u
    if case["post"]:
        pm, pr = _stats(u, case["norm"])
        v = _affine((u - pm[:, None]) * pr[:, None], s["post_weight"], s["post_bias"])
    v = v * _number(s["scale"])
    if s["gate"] is not None:
        v = v * _gate(s["gate"], case["act"])[0]
    r = 0.9 * s["x"].float() + v
    mean, rstd = _stats(r, case["norm"])
    y = _affine((r - mean[:, None]) * rstd[:, None], s["weight"], s["bias"])
    return y, r, torch.stack([pm, pr, mean, rstd])


def _float_of(t):
    return _values(*t) if isinstance(t, tuple) else t.float()


def _norm_back(e, h, rstd, norm):
    out = e - h * (e * h).mean(1, keepdim=True)
    if norm == "layer":
        out = out - e.mean(1, keepdim=True)
    return out * rstd[:, None]


def _residual_backward(s, case, r, u, gate, stats):
    r, u = _float_of(r), _float_of(u)
    pm, pr, mean, rstd = stats
    dy = s["dy"].float()
    h = (r - mean[:, None]) * rstd[:, None]
    d = s["dr"].float() + _norm_back(dy * s["weight"].float(), h, rstd, case["norm"])
    out = {"dx": 0.9 * d, "dweight": (dy * h).sum(0)}
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    uh = (u - pm[:, None]) * pr[:, None] if case["post"] else u
    v = _affine(uh, s["post_weight"], s["post_bias"])
    scale = _number(s["scale"])
    a = 1.0
    if gate is not None:
        a, slope = _gate(_float_of(gate), case["act"])
        dgate = d * scale * v * slope
        out["dgate"] = dgate if case["gate"] == "full" else dgate.sum(1, keepdim=True)
    if case["scale"] == "vector":
        out["dscale"] = (d * a * v).sum(0)
    dv = d * scale * a
    if case["post"]:
        out["dpost_weight"] = (dv * uh).sum(0)
        if s["post_bias"] is not None:
            out["dpost_bias"] = dv.sum(0)
        dv = _norm_back(dv * s["post_weight"].float(), uh, pr, case["norm"])
    out["du"] = dv
    return out


def _seen(kept, dt):
    """8-bit copies as the values they stand for: in 16 bits, which hold them."""
    return _values(*kept).to(torch.bfloat16 if dt == torch.float32 else dt)


def _residual_plain(s, case):
    (dt, st), out = _types(case), {}
    r, u, gate, stats = s.get("r"), s["u"], s["gate"], s.get("stats")
    if case["mode"] != "backward":
        y, r, stats = _residual_forward(s, case)
        r = r.to(st)
        out = {"y": y.to(dt), "r": r, "stats": stats}
        if case["kept"] == "8bit":
            r, u = _pack(r.float()), _pack(u.float())
            gate = _pack(gate.float()) if case["gate"] == "full" else gate
            out |= {"u8": _seen(u, dt), "r8": _seen(r, st)}
            if case["gate"] == "full":
                out["gate8"] = _seen(gate, dt)
    if case["mode"] != "forward":
        grads = _residual_backward(s, case, r, u, gate, stats)
        out |= {k: v.to(st if k == "dx" else dt) for k, v in grads.items()}
    return out


def _run_plain(s):
    case = s["case"]
    if case["op"] == "residual":
        return _residual_plain(s, case)
    dt = DTYPES[case["dtype"]]
    kept = s["kept"] if "kept" in s else _pack(s["x"].float())
    if case["op"] == "kept":
        return _values(*kept).to(dt)
    to = torch.float32 if case["to"] == "f32" else dt
    dy = s["dy"].float()
    out = {"dw": (dy.T @ _values(*kept).to(dt).float()).to(to)}  # (the values in dy's type: the product's operands)
    if case["bias"]:
        out["db"] = dy.sum(0).to(to)
    return out


# ------------------------------------------------------------------ the package's operators


def _residual_own(s, case):
    import einsum_device_side_gb300 as trop

    (dt, st), out, options = _types(case), {}, _options(case)
    r, u, gate, stats = s.get("r"), s["u"], s["gate"], s.get("stats")
    if case["mode"] != "backward":
        y, r, stats, kept = trop.residual_norm(s["x"], u, s["weight"], s["bias"], gate=gate, scale=s["scale"],
                                               post_weight=s["post_weight"], post_bias=s["post_bias"], eps=EPS,
                                               keep=case["kept"] == "8bit", **options)
        out = {"y": y, "r": r, "stats": stats}
        if case["kept"] == "8bit":
            u, gate, r = kept
            seen = lambda k, d: trop.activation_values(*k, torch.bfloat16 if d == torch.float32 else d)  # noqa: E731
            out |= {"u8": seen(u, dt), "r8": seen(r, st)}
            if case["gate"] == "full":
                out["gate8"] = seen(gate, dt)
    if case["mode"] != "forward":
        names = ("dx", "du", "dgate", "dscale", "dweight", "dbias", "dpost_weight", "dpost_bias")
        grads = trop.residual_norm_backward(s["dy"], s["dr"], r, u, stats, s["weight"], s["bias"], gate=gate, scale=s["scale"],
                                            post_weight=s["post_weight"], post_bias=s["post_bias"], **options)
        out |= {k: v for k, v in zip(names, grads) if v is not None}
    return out


def _run_own(s):
    import einsum_device_side_gb300 as trop

    case = s["case"]
    if case["op"] == "residual":
        return _residual_own(s, case)
    if case["op"] == "kept":
        kept = s["kept"] if "kept" in s else trop.activation_pack(s["x"])
        return trop.activation_values(*kept, DTYPES[case["dtype"]])
    dw, db = trop.activation_weight_grad(s["dy"], *s["kept"], out_dtype=torch.float32 if case["to"] == "f32" else None,
                                         want_bias=case["bias"])
    return {"dw": dw, "db": db} if case["bias"] else {"dw": dw}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    b = SIZE[case["dtype"]]
    if case["op"] == "grad":
        t, o, i = case["tokens"], case["out"], case["in"]
        to = 4 if case["to"] == "f32" else b
        return {"bytes": t * o * b + t * i + t * -(-i // GROUP) + (o * i + (o if case["bias"] else 0)) * to, "flops": 2 * t * o * i}
    rows, cols = case["rows"], case["cols"]
    n, codes = rows * cols, rows * cols + rows * -(-cols // GROUP)
    if case["op"] == "kept":  # the elements in (kept and read back: both ways), the values out
        return {"bytes": n * b * (2 if case["mode"] == "round" else 1) + codes, "flops": 4 * n}
    st = 4 if case["stream"] == "f32" else b
    gate = {"none": 0, "row": rows * b, "full": n * b}[case["gate"]]
    gate8 = codes if case["gate"] == "full" else gate
    vectors = cols * b * (1 + (case["norm"] == "layer") + (case["post"] + (case["post"] and case["norm"] == "layer")) +
                          (case["scale"] == "vector"))
    eight, moved, flops = case["kept"] == "8bit", 0, 0
    if case["mode"] != "backward":  # x, u and gate in; r, y and the statistics out; 8-bit copies out and seen as values
        moved += n * (2 * st + 2 * b) + gate + 16 * rows + vectors
        if eight:  # (the values in 16 bits)
            moved += (codes + 2 * n) * (3 if case["gate"] == "full" else 2)
        flops += 20 * n
    if case["mode"] != "forward":  # dy, dr, r, u and gate in; dx, du and the gate's gradient out; the vectors' gradients
        moved += n * (2 * st + 2 * b) + gate + 16 * rows + 2 * vectors
        moved += 2 * codes + gate8 if eight else n * (st + b) + gate
        flops += 40 * n
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------ 64 bits, from the definitions


def _exact_power(n):
    """2^n of whole n in 64 bits, by its exponent bits (a power function may be a last place off, which moves ties)."""
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_pack(x):
    """A matrix as its 8-bit copy stands for it, in 64 bits."""
    out = torch.empty_like(x, dtype=torch.float64)
    for c in range(0, x.shape[1], 8192):  # whole groups at a time, for room
        part = x[:, c:c + 8192].double()
        fill = -part.shape[1] % GROUP
        blocks = torch.nn.functional.pad(part, (0, fill)).unflatten(1, (-1, GROUP))
        _, power = torch.frexp(blocks.abs().amax(2, keepdim=True))  # the largest lies in [2^(power-1), 2^power)
        unit = _exact_power((power - 1).clamp(min=LEAST - 127) - 6)
        out[:, c:c + 8192] = (torch.round(blocks / unit).clamp(-127, 127) * unit).flatten(1)[:, :part.shape[1]]
    return out


def _exact_values(kept):
    codes, scales = kept
    group = torch.arange(codes.shape[1], device=codes.device) // GROUP
    return codes.double() * _exact_power(scales.to(torch.int64) - 133)[:, group]


def _exact_norm(t, norm):
    if norm == "layer":
        var, mu = torch.var_mean(t, dim=1, correction=0)
    else:
        mu, var = torch.zeros_like(t[:, 0]), torch.einsum("rc,rc->r", t, t) / t.shape[1]
    return mu, torch.rsqrt(var + EPS)


def _exact_residual(s):
    case = s["case"]
    wide = lambda t: t.double() if isinstance(t, torch.Tensor) else t  # noqa: E731
    _, st = _types(case)
    w, b, pw, pb, scale = (wide(s[k]) for k in ("weight", "bias", "post_weight", "post_bias", "scale"))
    out, eight = {}, case["kept"] == "8bit"
    at = {}  # what the backward pass reads
    if case["mode"] == "backward":
        at = {k: _exact_values(s[k]) if isinstance(s[k], tuple) else wide(s[k]) for k in ("r", "u", "gate")}
        stats = s["stats"].double()
    act = {"none": lambda g: g, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu}[case["act"]]

    def branch(u, g, mu, rs):
        v = (u - mu[:, None]) * rs[:, None] if case["post"] else u
        v = v if pw is None else v * pw
        v = v if pb is None else v + pb
        return v if g is None else v * act(g)

    if case["mode"] != "backward":
        at = {"u": wide(s["u"]), "gate": wide(s["gate"])}
        mu, rs = _exact_norm(at["u"], case["norm"]) if case["post"] else (torch.zeros_like(at["u"][:, 0]), torch.ones_like(at["u"][:, 0]))
        r = 0.9 * wide(s["x"]) + scale * branch(at["u"], at["gate"], mu, rs)
        m, q = _exact_norm(r, case["norm"])
        y = (r - m[:, None]) * q[:, None] * w
        stats = torch.stack([mu, rs, m, q])
        out = {"y": y if b is None else y + b, "r": r, "stats": stats}
        at["r"] = r.to(st).double()
        if eight:
            at["r"], at["u"] = _exact_pack(at["r"]), _exact_pack(at["u"])
            out |= {"u8": at["u"], "r8": at["r"]}
            if case["gate"] == "full":
                out["gate8"] = at["gate"] = _exact_pack(at["gate"])
    if case["mode"] == "forward":
        return out
    n, (mu, rs, m, q) = case["cols"], stats
    # y = w z + b with z = (r - m) q: the Jacobian of z with respect to r, applied to w dy
    ones = torch.ones(n, dtype=torch.float64, device="cuda")

    def jacobian(e, z, q):
        along = torch.einsum("rc,rc->r", e, z)[:, None] / n
        flat = (e @ ones)[:, None] / n if case["norm"] == "layer" else 0.0
        return (e - flat - z * along) * q[:, None]

    dy, z = wide(s["dy"]), (at["r"] - m[:, None]) * q[:, None]
    d = wide(s["dr"]) + jacobian(dy * w, z, q)
    out |= {"dx": 0.9 * d, "dweight": torch.einsum("rc,rc->c", dy, z)}
    if b is not None:
        out["dbias"] = torch.einsum("rc->c", dy)
    zu = (at["u"] - mu[:, None]) * rs[:, None] if case["post"] else at["u"]
    v = branch(at["u"], None, mu, rs)
    g = at["gate"]
    a = torch.ones_like(d[:, :1]) if g is None else act(g)
    if g is not None:
        sig = torch.sigmoid(g)
        slope = {"none": torch.ones_like(g), "sigmoid": sig * torch.sigmoid(-g), "silu": sig + g * sig * torch.sigmoid(-g)}[case["act"]]
        dg = d * scale * v * slope
        out["dgate"] = dg if case["gate"] == "full" else torch.einsum("rc->r", dg)[:, None]
    da = d * a
    if case["scale"] == "vector":
        out["dscale"] = torch.einsum("rc,rc->c", da, v)
    dv = da * scale
    if case["post"]:
        out["dpost_weight"] = torch.einsum("rc,rc->c", dv, zu)
        if pb is not None:
            out["dpost_bias"] = torch.einsum("rc->c", dv)
        dv = jacobian(dv * pw, zu, rs)
    out["du"] = dv
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "residual":
        return _exact_residual(s)
    if case["op"] == "kept":
        return _exact_values(s["kept"]) if "kept" in s else _exact_pack(s["x"])
    if 2 * case["tokens"] * case["out"] * case["in"] > 12e12:
        return None
    dy, x = s["dy"].double(), _exact_values(s["kept"]).to(DTYPES[case["dtype"]]).double()
    out = {"dw": torch.einsum("to,ti->oi", dy, x)}
    if case["bias"]:
        out["db"] = torch.einsum("to->o", dy)
    return out
