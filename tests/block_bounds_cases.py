"""The residual block's kernels on the bounds-checked build of the library: run as a script in a process of its own
with TROP_LIBRARY=debug.  Every kernel and every route of it runs on small ragged shapes, strides and offsets; the
library's violation record is read at the end.  Prints one JSON line: {"library", "cases", "wrong": [...],
"report": {...}}."""

from __future__ import annotations

import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for path in (ROOT, os.path.join(ROOT, "tests")):
    if path not in sys.path:
        sys.path.insert(0, path)


def main() -> int:
    import torch

    import einsum_device_side_gb300 as trop
    import residual_reference as ref

    trop.load()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    F, B, H = torch.float32, torch.bfloat16, torch.float16
    cases, wrong = 0, []

    # 1 % for results of bf16, 0.2 % otherwise: far above any rounding, far below what a misread element does
    def near(name, got, want):
        nonlocal cases
        cases += 1
        err = float((got.double() - want.double()).norm() / want.double().norm().clamp(min=1e-30))
        if not err <= (1e-2 if got.dtype == B else 2e-3):
            wrong.append(f"{name}: {err:.3g}")

    def rows(n, c, dt, pad=0, shift=0):
        return torch.randn(n, c + pad + shift, generator=gen, device="cuda").to(dt)[:, shift:shift + c]

    def residual(n, c, S, U, Y, gate="full", keep=False, W=None, pad=0, shift=0, norm="layer", post=True):
        x, u, dy, dr = rows(n, c, S, pad, shift), rows(n, c, U, pad, shift), rows(n, c, Y, pad, shift), rows(n, c, S, pad, shift)
        g = None if gate == "none" else rows(n, c, U, pad, shift) if gate == "full" else rows(n, 1, U)
        w, b, pw, pb, s = (m + 0.2 * torch.randn(c, generator=gen, device="cuda") for m in (1, 0, 1, 0, 0.4))
        w, b, pw, pb, s = (v.to(W or Y) for v in (w, b, pw, pb, s))
        if not post:
            pw = pb = None
        o = dict(gate_act="silu", post_norm=post, norm=norm, alpha=0.8)
        v = dict(scale=s, post_weight=pw, post_bias=pb)
        y, r, stats, kept = trop.residual_norm(x, u, w, b, gate=g, out_dtype=Y if Y != U else None, keep=keep, **v, **o)
        wy, wr, _ = ref.forward(x, u, w, b, g, scale=s, post_weight=pw, post_bias=pb, **o)
        name = f"residual {n}x{c} {S} {U} {Y} {gate} keep={keep}"
        near(name + " y", y, wy)
        near(name + " r", r, wr)
        ku, kg, kr = kept if keep else (u, g, r)
        got = trop.residual_norm_backward(dy, dr, kr, ku, stats, w, b, gate=kg, x_dtype=S, u_dtype=U, **v, **o)
        value = lambda t: trop.activation_values(*t, F) if isinstance(t, tuple) else t  # noqa: E731
        want, _ = ref.backward(dy, dr, value(kr), value(ku), stats, w, b, value(kg), scale=s, post_weight=pw, post_bias=pb, **o)
        for k, t in zip(("x", "u", "gate", "scale", "weight", "bias", "post_weight", "post_bias"), got):
            if t is not None:
                near(f"{name} d{k}", t, want[k])

    for S, U, Y in ((F, F, F), (B, B, B), (H, H, H), (F, B, B), (F, H, H), (F, F, B), (F, F, H)):
        for n, c in ((1, 8), (5, 33), (7, 256), (9, 1001), (3, 4096), (3, 8192), (2, 16384), (2, 20001)):
            residual(n, c, S, U, Y)
            residual(n, c, S, U, Y, keep=True, gate="row" if c == 256 else "full")
    for keep in (False, True):
        for S, U, Y in ((F, F, F), (B, B, B), (F, B, B)):
            residual(2500, 64, S, U, Y, keep=keep)      # short rows, several a block
            residual(700, 2048, S, U, Y, keep=keep)     # rows through the ring
            residual(330, 8192, S, U, Y, keep=keep, gate="none", norm="rms")
            residual(620, 1001, S, U, Y, keep=keep, gate="row")
            residual(70, 40, S, U, Y, keep=keep, pad=3, shift=1)
            residual(70, 40, S, U, Y, keep=keep, pad=8, post=False)
            residual(70, 24, S, U, Y, keep=keep, W=F)
    for dt in (F, B, H):
        for n, c, pad, shift in ((1, 1, 0, 0), (5, 33, 0, 0), (40, 96, 0, 0), (300, 1001, 0, 0), (64, 200, 3, 1), (3, 20001, 0, 0)):
            x = rows(n, c, dt, pad, shift)
            codes, scales = trop.activation_pack(x)
            v = trop.activation_values(codes, scales, dt)
            cases += 1  # half a unit is 1/128 of the group's largest magnitude at most, and the largest may lose a whole one
            if not bool(((v.float() - x.float()).abs() <= x.float().abs().max() / 64).all()):
                wrong.append(f"kept {n}x{c} {dt}")
    for dt in (B, H):
        for t, o, c in ((1, 1, 1), (7, 64, 96), (65, 257, 255), (129, 1000, 31), (1021, 203, 700), (4100, 96, 64), (300, 520, 1030)):
            dy, x = rows(t, o, dt), rows(t, c, dt)
            codes, scales = trop.activation_pack(x)
            for to in (None, F):
                dw, db = trop.activation_weight_grad(dy, codes, scales, out_dtype=to, want_bias=True)
                near(f"weight grad {t}x{o}x{c} {dt} {to}", dw, dy.double().T @ trop.activation_values(codes, scales, F).double())
                near(f"bias grad {t}x{o}x{c} {dt} {to}", db, dy.double().sum(0))
    torch.cuda.synchronize()
    print(json.dumps({"library": trop.LIB_DEBUG_PATH if os.environ.get("TROP_LIBRARY") == "debug" else trop.LIB_PATH, "cases": cases, "wrong": wrong, "report": trop.debug_bounds_report()}))
    return 0


if __name__ == "__main__":
    sys.exit(main())
