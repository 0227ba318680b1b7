"""The training operators' kernels on the bounds-checked build of the library: run as a script in a process
of its own with TROP_LIBRARY=debug.  Every kernel and every route of it runs on small ragged shapes, strides
and offsets; the library's violation record is read at the end.  Prints one JSON line: {"library", "cases",
"wrong": [...], "report": {...}}."""

from __future__ import annotations

import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def main() -> int:
    import torch

    import einsum_device_side_gb300 as trop

    trop.load()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    F, B, H = torch.float32, torch.bfloat16, torch.float16
    cases, wrong = 0, []

    def near(name, got, want, limit):
        nonlocal cases
        cases += 1
        err = float((got.double() - want.double()).norm() / want.double().norm().clamp(min=1e-30))
        if not err <= limit:
            wrong.append(f"{name}: {err:.3g}")

    def norm(rows, cols, dt, pad=0, shift=0):
        buf = normal(rows, cols + pad + shift).to(dt)
        x = buf[:, shift:shift + cols]
        w, b, dy = normal(cols).to(dt), normal(cols).to(dt), normal(rows, cols).to(dt)
        y, mean, rstd = trop.layer_norm(x, w, b)
        dx, dw, db = trop.layer_norm_backward(dy, x, mean, rstd, w)
        xr = x.double().requires_grad_()
        wr, br = w.double().requires_grad_(), b.double().requires_grad_()
        yr = torch.nn.functional.layer_norm(xr, (cols,), wr, br)
        yr.backward(dy.double())
        limit = {F: 1e-5, B: 1e-2, H: 2e-3}[dt]
        for n, g, e in (("y", y, yr.detach()), ("dx", dx, xr.grad), ("dw", dw, wr.grad), ("db", db, br.grad)):
            near(f"norm {rows}x{cols} {dt} {n}", g, e, limit)

    for dt in (F, B, H):
        for rows, cols in ((1, 8), (5, 33), (7, 256), (40, 1000), (9, 1001), (3, 4099), (2, 16384), (2, 20001)):
            norm(rows, cols, dt)
        norm(2500, 64, dt)       # short rows, several at a time
        norm(2600, 512, dt)
        norm(700, 2048, dt)      # rows through the ring
        for cols in (7, 33, 257, 1001, 2047, 4085, 8191):  # many rows off the 16-byte granules
            norm(2440, cols, dt)
        norm(60, 128, dt, pad=8)
        norm(60, 100, dt, pad=3, shift=1)

    def loss(n, d, v, dt, shift=0):
        x = normal(n, d + shift).to(dt)[:, shift:]
        w = (normal(v, d) * 2 / d ** 0.5).to(dt)
        t = torch.randint(0, v, (n,), generator=gen, device="cuda")
        t[::7] = -100
        for red in ("none", "mean"):
            val, lse, kept = trop.linear_cross_entropy(x, w, t, red)
            g = torch.ones((), device="cuda") if red == "mean" else normal(n).abs()
            dx, dw = trop.linear_cross_entropy_backward(g, x, w, t, lse, kept if red == "mean" else None)
            xr, wr = x.double().requires_grad_(), w.double().requires_grad_()
            each = torch.nn.functional.cross_entropy(xr @ wr.T, t, reduction="none")
            total = each.sum() / kept.double() if red == "mean" else (each * g.double()).sum()
            total.backward()
            near(f"loss {n}x{d}x{v} {dt} {red}", val, each.detach() if red == "none" else total.detach(), 1e-4)
            near(f"dx {n}x{d}x{v} {dt} {red}", dx, xr.grad, 2e-2)
            near(f"dw {n}x{d}x{v} {dt} {red}", dw, wr.grad, 2e-2)

    for dt in (B, H):
        for n, d, v in ((2, 8, 3), (5, 64, 300), (128, 72, 1000), (129, 65, 257), (300, 512, 2050), (70, 2100, 700), (260, 2100, 300),
                        (37, 1031, 300)):
            loss(n, d, v, dt)
        loss(20, 64, 100, dt, shift=3)

    def adamw(sizes, pdt, gdt, bits, shift, copies=False):
        mk = lambda dt, f=1.0: [(f * normal(n + shift)).to(dt)[shift:] for n in sizes]  # noqa: E731
        p, g = mk(pdt), mk(gdt, 0.1)
        cp = [torch.empty(n, dtype=B, device="cuda") for n in sizes] if copies else None
        want = [q.double() for q in p]
        opt = trop.AdamW(p, g, state_bits=bits, weight_decay=0.0, copies=cp)
        opt.step()
        for i, q in enumerate(want):
            e = g[i].double()
            near(f"adamw {pdt} {gdt} {bits} {shift} {sizes[i]}", p[i], q - 1e-3 * e / (e.abs() + 1e-8), 1e-2 if pdt != F else 1e-5)
        if bits == 8:
            trop.adamw_state_values(opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale)

    for bits in (32, 8):
        for pdt, gdt in ((F, F), (F, B), (B, B), (H, F)):
            adamw([1, 255, 256, 257, 4095, 4096, 9001], pdt, gdt, bits, 0)
            adamw([300, 5000], pdt, gdt, bits, 1)
        adamw([100 + i for i in range(400)], F, F, bits, 0)
        adamw([4096, 333], F, B, bits, 0, copies=True)

    torch.cuda.synchronize()
    print(json.dumps({"library": trop.LIB_DEBUG_PATH if os.environ.get("TROP_LIBRARY") == "debug" else trop.LIB_PATH,
                      "cases": cases, "wrong": wrong, "report": trop.debug_bounds_report()}))
    return 0


if __name__ == "__main__":
    sys.exit(main())
