"""The training operators' cases: inputs, plain forms, exact values and the work each call cannot do without.

Three operators that turn the tropical product and its gradient into something a user trains:

* layer norm, forward and backward, with the reduction of the weight's and the bias's gradients;
* the softmax cross entropy of a linear head over a large vocabulary, forward and backward, without the logits
  being kept;
* an AdamW step over many tensors at once, with 32-bit states or with 8-bit states in blocks of 256.

``run`` computes an operator in elementary torch operations in 32 bits, rounded once at the end, or, where ``own`` is
set, through the package's entry points.  ``exact`` computes the same from the definitions in 64 bits.
"""

import itertools
import math

import torch

own = False

BLOCK = 256  # elements that share one scale of an 8-bit state
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5  # layer norm
HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01}
IGNORE = -100


def listed():
    return [
        # layer norm: a few rows between two small layers, where the call's latency is what counts
        {"name": "norm forward 16x512 f32", "op": "norm", "mode": "forward", "rows": 16, "cols": 512, "dtype": "f32"},
        # backward alone, at a width that no vector load divides (a ragged feature count)
        {"name": "norm backward 2999x1001 f32", "op": "norm", "mode": "backward", "rows": 2999, "cols": 1001,
         "dtype": "f32"},
        # both directions over a full training batch, bound by memory
        {"name": "norm step 16384x4096 bf16", "op": "norm", "mode": "step", "rows": 16384, "cols": 4096,
         "dtype": "bf16"},
        # the loss of a toy model: everything fits one tile, latency counts
        {"name": "loss forward 4x64x256 bf16", "op": "loss", "mode": "forward", "tokens": 4, "dim": 64, "vocab": 256,
         "dtype": "bf16", "reduction": "mean"},
        # scoring a few tokens against a large vocabulary: the weights are read once and bound it
        {"name": "loss forward 16x4096x131072 bf16", "op": "loss", "mode": "forward", "tokens": 16, "dim": 4096,
         "vocab": 131072, "dtype": "bf16", "reduction": "none"},
        # evaluation of a whole batch: bound by the products
        {"name": "loss forward 8192x2048x65536 bf16", "op": "loss", "mode": "forward", "tokens": 8192, "dim": 2048,
         "vocab": 65536, "dtype": "bf16", "reduction": "mean"},
        # forward and backward at ragged sizes in half precision, a gradient of its own for each token
        {"name": "loss step 1021x1000x32003 f16", "op": "loss", "mode": "step", "tokens": 1021, "dim": 1000,
         "vocab": 32003, "dtype": "f16", "reduction": "none"},
        # backward of a training batch, the logits computed again in pieces of the vocabulary
        {"name": "loss backward 8192x2048x65536 bf16", "op": "loss", "mode": "backward", "tokens": 8192, "dim": 2048,
         "vocab": 65536, "dtype": "bf16", "reduction": "mean"},
        # the optimiser of a small model: a dozen tensors, latency counts
        {"name": "adamw 12 tensors 2e5 f32", "op": "adamw", "tensors": 12, "total": 200000, "dtype": "f32",
         "state": "f32"},
        # a training step's update of a large model with 32-bit states
        {"name": "adamw 96 tensors 1.3e8 f32", "op": "adamw", "tensors": 96, "total": 1 << 27, "dtype": "f32",
         "state": "f32"},
        # 8-bit states on many small odd tensors: every last block is part-filled
        {"name": "adamw 151 tensors 7e5 bf16 8-bit", "op": "adamw", "tensors": 151, "total": 700000, "dtype": "bf16",
         "state": "8bit"},
        # 8-bit states of a large model
        {"name": "adamw 96 tensors 1.3e8 f32 8-bit", "op": "adamw", "tensors": 96, "total": 1 << 27, "dtype": "f32",
         "state": "8bit"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "loss", "adamw"])
    if op == "norm":
        while True:
            rows, cols = _log(rng, 1, 65536), _log(rng, 32, 16384)
            if rows * cols <= 16384 * 4096:
                return {"op": op, "mode": rng.choice(["forward", "backward", "step"]), "rows": rows, "cols": cols,
                        "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op == "loss":
        while True:
            tokens, dim, vocab = _log(rng, 1, 8192), _log(rng, 32, 4096), _log(rng, 128, 131072)
            if tokens * dim * vocab <= 8192 * 2048 * 65536 and tokens * vocab <= 8192 * 65536:
                return {"op": op, "mode": rng.choice(["forward", "backward", "step"]), "tokens": tokens, "dim": dim,
                        "vocab": vocab, "dtype": rng.choice(["bf16", "f16"]),
                        "reduction": rng.choice(["none", "mean"])}
    tensors = _log(rng, 1, 192)
    return {"op": op, "tensors": tensors, "total": tensors * _log(rng, 300, (1 << 27) / tensors),
            "dtype": rng.choice(["f32", "bf16"]), "state": rng.choice(["f32", "8bit"])}


# ------------------------------------------------------------------ inputs


def _sizes(case):
    """The tensors' element counts: unequal, most of them no multiple of anything, their sum near `total`."""
    n, total = case["tensors"], case["total"]
    share = [1.0 + (7 * i % 11) for i in range(n)]  # one to eleven parts
    return [max(1, int(total * s / sum(share)) - (i % 3)) for i, s in enumerate(share)]


def _prepare_norm(case, gen):
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    x = (normal(rows, cols) * (0.5 + torch.rand(rows, 1, generator=gen, device="cuda")) + normal(rows, 1)).to(dt)
    s = {"x": x, "weight": (1 + 0.1 * normal(cols)).to(dt), "bias": (0.1 * normal(cols)).to(dt)}
    if case["mode"] != "forward":
        s["dy"] = normal(rows, cols).to(dt)
    if case["mode"] == "backward":  # what the forward call left behind
        xf = x.float()
        s["mean"] = xf.mean(1)
        s["rstd"] = 1 / torch.sqrt((xf - s["mean"][:, None]).square().mean(1) + EPS)
    return s


def _prepare_loss(case, gen):
    n, d, v, dt = case["tokens"], case["dim"], case["vocab"], DTYPES[case["dtype"]]
    s = {"x": torch.randn(n, d, generator=gen, device="cuda").to(dt),
         "w": torch.empty(v, d, device="cuda", dtype=dt)}
    step = max(1, (1 << 27) // d)
    for r in range(0, v, step):  # logits with a spread of about two
        part = s["w"][r:r + step]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * (2 / math.sqrt(d)))
    s["target"] = torch.randint(0, v, (n,), generator=gen, device="cuda")
    drop = torch.rand(n, generator=gen, device="cuda") < 0.05  # padding
    drop[0] = False
    s["target"][drop] = IGNORE
    if case["mode"] != "forward":
        if case["reduction"] == "none":
            s["dloss"] = torch.rand(n, generator=gen, device="cuda")
        else:  # half precision trains with its loss scaled up
            s["dloss"] = torch.full((), 1024.0 if dt == torch.float16 else 1.0, device="cuda")
    if case["mode"] == "backward":  # what the forward call left behind
        s["lse"] = torch.empty(n, device="cuda")
        step = max(1, (1 << 28) // v)
        for r in range(0, n, step):  # in pieces, for room
            s["lse"][r:r + step] = torch.logsumexp(s["x"][r:r + step].float() @ s["w"].float().T, 1)
        s["kept"] = (s["target"] != IGNORE).sum().float()
    return s


def _views(flat, sizes, block=1):
    """Views of the tensors in a flat buffer: each starts on a multiple of BLOCK elements (of one scale for scales)."""
    starts = [0, *itertools.accumulate(-(-n // BLOCK) for n in sizes)]
    if block == 1:
        return [flat[BLOCK * a:BLOCK * a + n] for a, n in zip(starts, sizes)]
    return [flat[a:b] for a, b in zip(starts, starts[1:])]


def _prepare_adamw(case, gen):
    """Every kind of buffer is one flat allocation with the tensors as views of it, as a program keeps them that saves
    and clears its parameters, gradients and states in one go; what lies between two tensors is zero."""
    dt, sizes = DTYPES[case["dtype"]], _sizes(case)
    count = sum(-(-n // BLOCK) for n in sizes) * BLOCK
    live, spread = torch.zeros(count, device="cuda"), torch.zeros(count, device="cuda")
    for i, (a, b) in enumerate(zip(_views(live, sizes), _views(spread, sizes))):
        a.fill_(1)
        b.fill_(10.0 ** (-2 - i % 3))  # gradients of unlike size
    normal = lambda: torch.randn(count, generator=gen, device="cuda")  # noqa: E731
    s = {"flat_p": (0.02 * normal() * live).to(dt), "flat_g": (normal() * spread).to(dt), "step": 1000}
    m = 0.3 * normal() * spread
    v = (0.5 + torch.rand(count, generator=gen, device="cuda")) * spread * spread
    if case["state"] == "f32":
        s |= {"flat_m": m, "flat_v": v}
    else:
        (cm, ms), (cv, vs) = _encode_m(m.reshape(-1, BLOCK)), _encode_r(v.sqrt().reshape(-1, BLOCK))
        s |= {"flat_m": cm.reshape(-1).to(torch.int8), "flat_v": cv.reshape(-1).to(torch.uint8),
              "flat_ms": ms.reshape(-1).clone(), "flat_vs": vs.reshape(-1).clone(),
              "flat_mval": torch.zeros_like(m), "flat_vval": torch.zeros_like(m)}
    for k in [k[5:] for k in s if k.startswith("flat_")]:
        s[k] = _views(s["flat_" + k], sizes, BLOCK if k in ("ms", "vs") else 1)
    if own:  # the handle that a program keeps which steps the same tensors again and again
        import einsum_device_side_gb300 as trop
        values = (s["mval"], s["vval"]) if "ms" in s else None
        s["plan"] = trop.AdamWPlan(s["p"], s["g"], s["m"], s["v"], s.get("ms"), s.get("vs"), values=values)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    make = {"norm": _prepare_norm, "loss": _prepare_loss, "adamw": _prepare_adamw}[case["op"]]
    return {"case": dict(case), **make(case, gen)}


# ------------------------------------------------------------------ plain forms, in 32 bits


def _norm_forward(x, weight, bias):
    x = x.float()
    mean = x.mean(1)
    centred = x - mean[:, None]
    rstd = 1 / torch.sqrt((centred * centred).mean(1) + EPS)
    return centred * rstd[:, None] * weight.float() + bias.float(), mean, rstd


def _norm_backward(dy, x, mean, rstd, weight):
    dy, xhat = dy.float(), (x.float() - mean[:, None]) * rstd[:, None]
    dxhat = dy * weight.float()
    along, flat = (dxhat * xhat).mean(1, keepdim=True), dxhat.mean(1, keepdim=True)
    return rstd[:, None] * (dxhat - flat - xhat * along), (dy * xhat).sum(0), dy.sum(0)


def _loss_forward(x, w, target, reduction):
    logits = x.float() @ w.float().T
    top = logits.amax(1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(1))
    kept = target != IGNORE
    at = torch.gather(logits, 1, torch.where(kept, target, 0)[:, None])[:, 0]
    loss, count = torch.where(kept, lse - at, 0.0), kept.sum().float()
    return loss.sum() / count if reduction == "mean" else loss, lse, count


def _loss_backward(dloss, x, w, target, lse, count):
    xf, wf = x.float(), w.float()
    kept = target != IGNORE
    scale = dloss / count if count is not None else dloss
    scale = torch.where(kept, scale, 0.0)[:, None]
    p = torch.exp(xf @ wf.T - lse[:, None])
    at = torch.where(kept, target, 0)[:, None]
    p.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    p = p * scale
    return p @ wf, p.T @ xf


def _inverse(top):
    return torch.where(top > 0, 1 / top, 0.0)


def _encode_m(m):
    """Signed codes c of a block's values, c |c| / 127^2 times the block's largest magnitude; and the scales."""
    top = m.abs().amax(1, keepdim=True)
    c = torch.round(torch.sqrt((m.abs() * _inverse(top)).clamp(max=1)) * 127)
    return torch.copysign(c, m), top / 16129


def _encode_r(r):
    """Codes c of a block's square-rooted second moments, c^2 / 255^2 times the largest; none but zero gets zero."""
    top = r.amax(1, keepdim=True)
    c = torch.round(torch.sqrt((r * _inverse(top)).clamp(max=1)) * 255)
    return torch.where(r > 0, c.clamp(min=1), c), top / 65025


def _adamw(p, g, m, v, step):
    h = HYPER
    first, second = 1 - h["beta1"] ** step, 1 - h["beta2"] ** step
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + (g * g) * (1 - h["beta2"])
    r = torch.sqrt(v)
    p = p * (1 - h["lr"] * h["weight_decay"]) - (m / (r * (1 / math.sqrt(second)) + h["eps"])) * (h["lr"] / first)
    return p, m, v, r


def _adamw_plain(s, step):
    """All tensors in one chain of elementary operations over the flat buffers; zeros between them stay zeros."""
    p, g, m, v = (s["flat_" + k].float() for k in "pgmv")
    if s["case"]["state"] == "f32":
        p, m, v, _ = _adamw(p, g, m, v, step)
        s["flat_p"].copy_(p)
        return {"p": s["flat_p"], "m": s["flat_m"].copy_(m), "v": s["flat_v"].copy_(v)}
    m = (m * m.abs()).reshape(-1, BLOCK) * s["flat_ms"][:, None]
    r = (v * v).reshape(-1, BLOCK) * s["flat_vs"][:, None]
    p, m, v, r = _adamw(p, g, m.reshape(-1), (r * r).reshape(-1), step)
    (cm, ms), (cv, vs) = _encode_m(m.reshape(-1, BLOCK)), _encode_r(r.reshape(-1, BLOCK))
    s["flat_p"].copy_(p)
    s["flat_m"].copy_(cm.reshape(-1))
    s["flat_v"].copy_(cv.reshape(-1))
    s["flat_ms"].copy_(ms.reshape(-1))
    s["flat_vs"].copy_(vs.reshape(-1))
    r = cv * cv * vs
    return {"p": s["flat_p"], "m": (cm * cm.abs() * ms).reshape(-1), "v": (r * r).reshape(-1)}


def _run_plain(s):
    case = s["case"]
    if case["op"] == "norm":
        dt, out = DTYPES[case["dtype"]], {}
        mean, rstd = s.get("mean"), s.get("rstd")
        if case["mode"] != "backward":
            y, mean, rstd = _norm_forward(s["x"], s["weight"], s["bias"])
            out = {"y": y.to(dt), "mean": mean, "rstd": rstd}
        if case["mode"] != "forward":
            dx, dweight, dbias = _norm_backward(s["dy"], s["x"], mean, rstd, s["weight"])
            out |= {"dx": dx.to(dt), "dweight": dweight.to(dt), "dbias": dbias.to(dt)}
        return out
    if case["op"] == "loss":
        dt, out = DTYPES[case["dtype"]], {}
        lse, kept = s.get("lse"), s.get("kept")
        if case["mode"] != "backward":
            loss, lse, kept = _loss_forward(s["x"], s["w"], s["target"], case["reduction"])
            out = {"loss": loss, "lse": lse}
        if case["mode"] != "forward":
            dx, dw = _loss_backward(s["dloss"], s["x"], s["w"], s["target"], lse,
                                    kept if case["reduction"] == "mean" else None)
            out |= {"dx": dx.to(dt), "dw": dw.to(dt)}
        return out
    out = _adamw_plain(s, s["step"])
    s["step"] += 1
    return out


# ------------------------------------------------------------------ the package's operators


def _run_own(s):
    import einsum_device_side_gb300 as trop

    case = s["case"]
    if case["op"] == "norm":
        out, mean, rstd = {}, s.get("mean"), s.get("rstd")
        if case["mode"] != "backward":
            y, mean, rstd = trop.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
            out = {"y": y, "mean": mean, "rstd": rstd}
        if case["mode"] != "forward":
            dx, dweight, dbias = trop.layer_norm_backward(s["dy"], s["x"], mean, rstd, s["weight"])
            out |= {"dx": dx, "dweight": dweight, "dbias": dbias}
        return out
    if case["op"] == "loss":
        out, lse, kept = {}, s.get("lse"), s.get("kept")
        if case["mode"] != "backward":
            loss, lse, kept = trop.linear_cross_entropy(s["x"], s["w"], s["target"], reduction=case["reduction"],
                                                        ignore_index=IGNORE)
            out = {"loss": loss, "lse": lse}
        if case["mode"] != "forward":
            dx, dw = trop.linear_cross_entropy_backward(s["dloss"], s["x"], s["w"], s["target"], lse,
                                                        kept if case["reduction"] == "mean" else None,
                                                        ignore_index=IGNORE)
            out |= {"dx": dx, "dw": dw}
        return out
    s["plan"].step(s["step"], **HYPER)
    if case["state"] == "f32":
        out = {"p": s["flat_p"], "m": s["flat_m"], "v": s["flat_v"]}
    else:
        s["plan"].state_values()
        out = {"p": s["flat_p"], "m": s["flat_mval"], "v": s["flat_vval"]}
    s["step"] += 1
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    if case["op"] == "norm":
        rows, cols, b = case["rows"], case["cols"], SIZE[case["dtype"]]
        n, stats, small = rows * cols * b, 8 * rows, cols * b
        forward, backward = case["mode"] != "backward", case["mode"] != "forward"
        # x in; y, mean and rstd out; dy in, dx out; weight and bias in, their gradients out
        moved = n + stats + small + forward * (n + small) + backward * (2 * n + 2 * small)
        return {"bytes": moved, "flops": rows * cols * (8 * forward + 12 * backward)}
    if case["op"] == "loss":
        n, d, v, b = case["tokens"], case["dim"], case["vocab"], SIZE[case["dtype"]]
        read, product = (n + v) * d * b + 8 * n, 2 * n * d * v
        if case["mode"] == "forward":
            return {"bytes": read + 8 * n, "flops": product}
        # x, w and the targets in, both gradients out; the logits' product and the two gradients'
        return {"bytes": 2 * read, "flops": 3 * product}
    n, b = sum(_sizes(case)), SIZE[case["dtype"]]
    # the parameters and states in and out, the gradients in; 8-bit states are answered as 32-bit values besides
    return {"bytes": n * (3 * b + (16 if case["state"] == "f32" else 4 + 16 / BLOCK + 8)),
            "flops": n * (16 if case["state"] == "f32" else 32)}


# ------------------------------------------------------------------ 64 bits, from the definitions


def _exact_norm(s):
    mode = s["case"]["mode"]
    x, w, b = (s[k].double() for k in ("x", "weight", "bias"))
    var, mu = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    sd = torch.sqrt(var + EPS)
    out = {}
    if mode != "backward":
        out = {"y": (x - mu) / sd * w + b, "mean": mu[:, 0], "rstd": 1 / sd[:, 0]}
    else:  # the statistics are inputs
        mu, sd = s["mean"].double()[:, None], 1 / s["rstd"].double()[:, None]
    if mode != "forward":
        # y = w z + b with z = (x - mu) / sd: the Jacobian of z with respect to x, applied to u = w dy
        z, dy = (x - mu) / sd, s["dy"].double()
        u, n = w * dy, x.shape[1]
        out["dx"] = (u - (u @ torch.ones_like(u[0]))[:, None] / n - z * torch.einsum("rc,rc->r", u, z)[:, None] / n) / sd
        out["dweight"] = torch.einsum("rc,rc->c", dy, z)
        out["dbias"] = torch.einsum("rc->c", dy)
    return out


def _exact_loss(s):
    case = s["case"]
    n, d, v = case["tokens"], case["dim"], case["vocab"]
    if (2 if case["mode"] == "forward" else 8) * n * d * v > 12e12:
        return None
    x, w, t = s["x"].double(), s["w"].double(), s["target"]
    rows = torch.nonzero(t != IGNORE)[:, 0]
    out, lse = {}, s["lse"].double() if "lse" in s else None
    step = max(1, (1 << 28) // v)
    if lse is None:
        lse = torch.cat([torch.logsumexp(x[r:r + step] @ w.T, 1) for r in range(0, n, step)])
        loss = torch.zeros(n, dtype=torch.float64, device="cuda")
        loss[rows] = lse[rows] - torch.einsum("rd,rd->r", x[rows], w[t[rows]])
        out = {"loss": loss.sum() / rows.numel() if case["reduction"] == "mean" else loss, "lse": lse}
    if case["mode"] != "forward":
        weight = s["dloss"].double().expand(n) / (rows.numel() if case["reduction"] == "mean" else 1)
        dx, dw = torch.zeros_like(x), torch.zeros_like(w)
        for a in range(0, rows.numel(), step):  # sum over the tokens of weight (softmax - one at the target)
            r = rows[a:a + step]
            soft = torch.exp(x[r] @ w.T - lse[r, None]) * weight[r, None]
            dx[r] = soft @ w - weight[r, None] * w[t[r]]
            dw += soft.T @ x[r]
        dw.index_add_(0, t[rows], -weight[rows, None] * x[rows])
        out |= {"dx": dx, "dw": dw}
    return out


def _exact_adamw(s):
    h, k, sizes = HYPER, s["step"], _sizes(s["case"])
    out = {key: torch.zeros(s["flat_p"].numel(), dtype=torch.float64, device="cuda") for key in "pmv"}
    at = {key: _views(out[key], sizes) for key in "pmv"}
    for i, n in enumerate(sizes):
        p, g, m, v = (s[key][i].double() for key in "pgmv")
        blocks = torch.arange(n, device="cuda") // BLOCK
        if s["case"]["state"] != "f32":
            m = m * m.abs() * s["ms"][i].double()[blocks]
            v = (v * v * s["vs"][i].double()[blocks]) ** 2
        m = h["beta1"] * m + (1 - h["beta1"]) * g
        v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
        hat = (m / (1 - h["beta1"] ** k)) / (torch.sqrt(v / (1 - h["beta2"] ** k)) + h["eps"])
        at["p"][i].copy_(p - h["lr"] * (hat + h["weight_decay"] * p))
        if s["case"]["state"] != "f32":
            none = torch.zeros(s["ms"][i].numel(), dtype=torch.float64, device="cuda")
            top = none.scatter_reduce(0, blocks, m.abs(), "amax")[blocks]
            c = torch.round(127 * torch.sqrt(m.abs() / top.clamp(min=1e-300)))
            m, r = torch.sign(m) * top * (c / 127) ** 2, torch.sqrt(v)
            top = none.scatter_reduce(0, blocks, r, "amax")[blocks]
            c = torch.round(255 * torch.sqrt(r / top.clamp(min=1e-300)))
            v = (top * (torch.where(r > 0, c.clamp(min=1), c) / 255) ** 2) ** 2
        at["m"][i].copy_(m)
        at["v"][i].copy_(v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "loss": _exact_loss, "adamw": _exact_adamw}[case["op"]](s)
