"""The residual block's operators in 64 bits, from their definitions, for the tests."""

import torch

ACTS = {"none": lambda g: g, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu}


def wide(t):
    return t.double() if isinstance(t, torch.Tensor) else t


def stats_of(t, norm, eps):
    mean = t.mean(1) if norm == "layer" else torch.zeros_like(t[:, 0])
    return mean, 1 / torch.sqrt((t - mean[:, None]).square().mean(1) + eps)


def forward(x, u, weight=None, bias=None, gate=None, gate_act="none", scale=None, post_weight=None, post_bias=None,
            post_norm=True, norm="layer", alpha=1.0, eps=1e-5):
    """(y, r, stats) of matrices."""
    x, u, weight, bias, gate, scale, post_weight, post_bias = map(wide, (x, u, weight, bias, gate, scale, post_weight, post_bias))
    um, ur = torch.zeros_like(u[:, 0]), torch.ones_like(u[:, 0])
    v = u
    if post_norm:
        um, ur = stats_of(u, norm, eps)
        v = (u - um[:, None]) * ur[:, None]
        v = v if post_weight is None else v * post_weight
        v = v if post_bias is None else v + post_bias
    v = v if scale is None else v * scale
    v = v if gate is None else v * ACTS[gate_act](gate)
    r = alpha * x + v
    mean, rstd = stats_of(r, norm, eps)
    y = (r - mean[:, None]) * rstd[:, None]
    y = y if weight is None else y * weight
    y = y if bias is None else y + bias
    return y, r, torch.stack([um, ur, mean, rstd])


def backward(dy, dr, r, u, stats, weight=None, bias=None, gate=None, gate_act="none", scale=None, post_weight=None,
             post_bias=None, post_norm=True, norm="layer", alpha=1.0):
    """The gradients by name, of r, u, gate and statistics as they are given; and by name the same with every sum taken over
    magnitudes: what roundings on the way to a result that cancels are relative to."""
    dy, dr, r, u, stats, weight, bias, gate, scale, post_weight, post_bias = map(
        wide, (dy, dr, r, u, stats, weight, bias, gate, scale, post_weight, post_bias))
    um, ur, mean, rstd = (s[:, None] for s in stats)

    def jacobian(e, h, k):
        flat = e.mean(1, keepdim=True) if norm == "layer" else 0.0
        return k * (e - flat - h * (e * h).mean(1, keepdim=True))

    def terms(e, h, k):
        e, h = e.abs(), h.abs()
        return k * (e + e.mean(1, keepdim=True) + h * (e * h).mean(1, keepdim=True))

    h = (r - mean) * rstd
    e = dy if weight is None else dy * weight
    d = jacobian(e, h, rstd) + (0.0 if dr is None else dr)
    size = terms(e, h, rstd) + (0.0 if dr is None else dr.abs())
    out, sizes = {"x": alpha * d}, {"x": abs(alpha) * size}
    if weight is not None:
        out["weight"], sizes["weight"] = (dy * h).sum(0), (dy * h).abs().sum(0)
    if bias is not None:
        out["bias"], sizes["bias"] = dy.sum(0), dy.abs().sum(0)
    uh = (u - um) * ur if post_norm else u
    v = uh if post_weight is None else uh * post_weight
    vs = v.abs() if post_bias is None else v.abs() + post_bias.abs()
    v = v if post_bias is None else v + post_bias
    k = 1.0 if scale is None else scale
    a = torch.ones_like(d)
    if gate is not None:
        with torch.enable_grad():
            g = gate.detach().requires_grad_()
            a = ACTS[gate_act](g)
            slope, = torch.autograd.grad(a.sum(), g)
        a = a.detach()
        out["gate"], sizes["gate"] = d * k * v * slope, size * vs * abs(k * slope)
        if gate.shape[1] == 1 and d.shape[1] > 1:
            out["gate"], sizes["gate"] = (t.sum(1, keepdim=True) for t in (out["gate"], sizes["gate"]))
        a = a.expand_as(d)
    if isinstance(scale, torch.Tensor):
        out["scale"], sizes["scale"] = (d * a * v).sum(0), (size * a.abs() * vs).sum(0)
    dv, size = d * k * a, size * abs(k * a)
    if post_norm:
        if post_weight is not None:
            out["post_weight"], sizes["post_weight"] = (dv * uh).sum(0), (size * uh.abs()).sum(0)
        if post_bias is not None:
            out["post_bias"], sizes["post_bias"] = dv.sum(0), size.sum(0)
        w = 1.0 if post_weight is None else post_weight
        dv, size = jacobian(dv * w, uh, ur), terms(size * abs(w), uh, ur)
    out["u"], sizes["u"] = dv, size
    return out, sizes
