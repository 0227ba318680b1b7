"""The norms around a block against 64 bits: every type, norm, gate and layout, the forward pass's 8-bit copies bit for
bit, gradients against the formula, against autograd and against differences.

Limits: a stored value is off by at most half a step of its type, eps / 2 relative to itself, so the norm of a result's
errors is at most eps / 2 of the result's norm, plus what f32 sums and products lose before: rows of up to 20001
columns summed in trees of depth 32 at most, a dozen operations an element, each 2^-24 (6e-8) of what it adds or
multiplies: under 1e-5 of the terms that a result is the sum of.  Where those cancel (of one column a norm's gradient is
k e (1 - h^2), with h^2 = 1 - O(eps)) the result is smaller than they, so the second part is taken of the terms' norm."""

import itertools

import pytest
import torch

import residual_reference as ref

pytestmark = pytest.mark.gpu

F, B, H = torch.float32, torch.bfloat16, torch.float16
NAMES = ("x", "u", "gate", "scale", "weight", "bias", "post_weight", "post_bias")


@pytest.fixture(scope="module")
def trop():
    import einsum_device_side_gb300 as t
    t.load()
    return t


LOST = 1e-5


def near(name, got, want, dt=F, terms=None, lost=LOST):
    """got, stored as dt (None: compared as it is), against want, a sum of terms of that size."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, name
    assert bool(got.isfinite().all()), name
    size = max(float(want.norm()), 0.0 if terms is None else float(terms.norm()))
    most = (torch.finfo(dt).eps / 2 * float(want.norm()) if dt else 0.0) + lost * size + 1e-30
    err = float((got - want).norm())
    assert err <= most, f"{name}: {err:.3g} > {most:.3g}"


def make(rows, cols, S=F, U=F, Y=F, W=None, *, gate="full", gate_act="none", scale="vector", post_norm=True, norm="layer",
         affine=True, seed=0, pad=0, shift=0):
    """Inputs of one call and its options."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = W or Y

    def normal(n, c, dt):
        return torch.randn(n, c + pad + shift, generator=g, device="cuda").to(dt)[:, shift:shift + c]

    vec = lambda m, k: (m + k * torch.randn(cols, generator=g, device="cuda")).to(W)  # noqa: E731
    t = {"x": normal(rows, cols, S), "u": (2 * normal(rows, cols, F) + 1).to(U), "gate": None, "weight": None, "bias": None,
         "post_weight": None, "post_bias": None, "scale": 0.4}
    if pad or shift:
        t["u"] = normal(rows, cols, U)
    if gate != "none":
        t["gate"] = normal(rows, cols, U) if gate == "full" else torch.randn(rows, 1, generator=g, device="cuda").to(U)
    if scale == "vector":
        t["scale"] = vec(0.3, 0.1)
    if affine:
        t["weight"], t["bias"] = vec(1, 0.2), vec(0, 0.2)
        if post_norm:
            t["post_weight"], t["post_bias"] = vec(1, 0.2), vec(0, 0.2)
    t["dy"], t["dr"] = normal(rows, cols, Y), normal(rows, cols, S)
    options = dict(gate_act=gate_act, post_norm=post_norm, norm=norm, alpha=0.7)
    return t, options


def values(trop, t):
    return trop.activation_values(*t, F) if isinstance(t, tuple) else t


def check(trop, t, options, S=F, U=F, Y=F, keep=False, names=NAMES, dr=True, lost=LOST):
    tensors = {k: t[k] for k in ("gate", "scale", "post_weight", "post_bias")}
    y, r, stats, kept = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], **tensors, **options, eps=1e-5,
                                           out_dtype=Y if Y != U else None, keep=keep)
    wy, wr, ws = ref.forward(t["x"], t["u"], t["weight"], t["bias"], **tensors, **options)
    assert (y.dtype, r.dtype) == (Y, S)
    near("y", y, wy, Y, lost=lost)
    near("r", r, wr, S, lost=lost)
    near("stats", stats[1::2], ws[1::2], lost=lost)
    near("means", stats[::2] + 1, ws[::2] + 1, lost=lost)
    u, gate = t["u"], t["gate"]
    if keep:
        full = gate is not None and gate.shape[1] == u.shape[1] and isinstance(kept[1], tuple)
        for name, pair, of in (("u", kept[0], u), ("r", kept[2], r)) + ((("gate", kept[1], gate),) if full else ()):
            codes, scales = trop.activation_pack(of)
            assert torch.equal(pair[0], codes) and torch.equal(pair[1], scales), name
        u, gate, r = kept
        assert full or gate is t["gate"]
        tensors["gate"] = gate
    g = trop.residual_norm_backward(t["dy"], t["dr"] if dr else None, r, u, stats, t["weight"], t["bias"], **tensors, **options,
                                    want=names, x_dtype=S, u_dtype=U)
    got = dict(zip(NAMES, g))
    tensors["gate"] = values(trop, gate)
    want, sizes = ref.backward(t["dy"], t["dr"] if dr else None, values(trop, r), values(trop, u), stats, t["weight"], t["bias"], **tensors,
                        **options)
    for name in NAMES:
        if name in want and name in names:
            dt = {"x": S, "u": U, "gate": U}.get(name, got[name].dtype)
            assert got[name].dtype == dt, name
            near("d" + name, got[name], want[name], dt, sizes[name], lost)
        else:
            assert got[name] is None, name
    return got


TYPES = [(F, F, F), (B, B, B), (H, H, H), (F, B, B), (F, H, H), (F, F, B), (F, F, H)]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("S, U, Y", TYPES)
@pytest.mark.parametrize("rows, cols", [(1, 1), (3, 7), (5, 33), (2, 256), (9, 1001), (40, 1000), (3, 4096), (2, 8192), (2, 16384),
                                        (3, 20001)])
def test_sizes_and_types(trop, rows, cols, S, U, Y, keep):
    if cols == 1:  # (a norm over one element is zero: only the bias is left, and gradients that cancel)
        t, o = make(rows, cols, S, U, Y, norm="rms")
    else:
        t, o = make(rows, cols, S, U, Y)
    check(trop, t, o, S, U, Y, keep)


@pytest.mark.parametrize("norm, gate, act, scale, post, affine", [
    c for i, c in enumerate(itertools.product(("layer", "rms"), ("none", "row", "full"), ("none", "sigmoid", "silu"),
                                              ("number", "vector"), (True, False), (True, False))) if c[1] != "none" or c[2] == "none"])
def test_variants(trop, norm, gate, act, scale, post, affine):
    kw = dict(norm=norm, gate=gate, gate_act=act, scale=scale, post_norm=post, affine=affine)
    for S, U, Y, keep, rows, cols in ((F, F, F, False, 13, 100), (F, B, B, True, 13, 512), (B, B, B, False, 300, 96)):
        t, o = make(rows, cols, S, U, Y, seed=3, **kw)
        check(trop, t, o, S, U, Y, keep, dr=affine)


@pytest.mark.parametrize("S, U, Y, keep", [(F, F, F, False), (B, B, B, False), (B, B, B, True), (F, H, H, True)])
@pytest.mark.parametrize("rows, cols", [(2500, 64), (2600, 512), (700, 2048), (1300, 1001), (620, 4096), (400, 8192), (200, 16384)])
def test_many_rows(trop, rows, cols, S, U, Y, keep):
    t, o = make(rows, cols, S, U, Y, seed=5)
    check(trop, t, o, S, U, Y, keep)


@pytest.mark.parametrize("pad, shift", [(8, 0), (3, 1), (5, 0)])
@pytest.mark.parametrize("dt", [F, B])
def test_strided_rows(trop, dt, pad, shift):
    for cols in (64, 100):
        t, o = make(37, cols, dt, dt, dt, pad=pad, shift=shift)
        for keep in (False, True):
            check(trop, t, o, dt, dt, dt, keep)


def test_wide_vectors(trop):
    for W in (F, B):
        t, o = make(70, 320, B, B, B, W)
        assert check(trop, t, o, B, B, B)["weight"].dtype == W


@pytest.mark.parametrize("names", [(), ("x",), ("u",), ("gate",), ("bias",), ("scale",), ("post_weight",), ("post_bias", "weight"),
                                   ("x", "post_bias")])
def test_wanted_gradients_alone(trop, names):
    for cols in (40, 20001):
        t, o = make(11, cols)
        check(trop, t, o, names=names)


def test_a_row_depends_on_itself_alone(trop):
    """A row gives the same bits whatever rows stand beside it, and the kept copies' gradients too."""
    t, o = make(2500, 512, B, B, B)
    tensors = {k: t[k] for k in ("gate", "scale", "post_weight", "post_bias")}
    y, r, stats, _ = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], **tensors, **o)
    again = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], **tensors, **o)
    assert all(torch.equal(a, b) for a, b in zip((y, r, stats), again))
    g = trop.residual_norm_backward(t["dy"], t["dr"], r, t["u"], stats, t["weight"], t["bias"], **tensors, **o)
    h = trop.residual_norm_backward(t["dy"], t["dr"], r, t["u"], stats, t["weight"], t["bias"], **tensors, **o)
    assert all(torch.equal(a, b) for a, b in zip(g, h))


def test_rows_with_infinities_and_nan_spoil_no_others(trop):
    for cols in (64, 1001, 4096):
        t, o = make(40, cols, B, B, B)
        tensors = {k: t[k] for k in ("gate", "scale", "post_weight", "post_bias")}
        good = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], **tensors, **o, keep=True)
        t["x"][3, 5], t["u"][7, 1], t["gate"][11, 2] = float("inf"), float("nan"), float("-inf")
        y, r, stats, kept = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], **tensors, **o, keep=True)
        rows = torch.ones(40, dtype=torch.bool, device="cuda")
        rows[[3, 7, 11]] = False
        assert torch.equal(y[rows], good[0][rows]) and torch.equal(r[rows], good[1][rows])
        assert not bool(y[~rows].isfinite().any())
        for pair, before in zip(kept, good[3]):
            assert torch.equal(pair[0][rows], before[0][rows]) and torch.equal(pair[1][rows], before[1][rows])


def test_large_means_and_constant_rows(trop):
    """A constant row's norm is its bias, exactly.  A mean far above the deviation: of 1e4 the f32 mean is off by up to half
    a step, 2^-11, which is 2.5e-4 of a deviation of 2: under 1e-3 with what the results add up from it."""
    for cols in (48, 1001, 4096):
        u = torch.full((5, cols), 1000.3, device="cuda")
        x = torch.full((5, cols), 77.7, device="cuda")
        pb = torch.randn(cols, device="cuda")
        y, r, stats, _ = trop.residual_norm(x, u, post_bias=pb * 0)
        assert bool((y == 0).all()) and torch.equal(r, x)
        y, r, stats, _ = trop.residual_norm(x, u, post_bias=pb)
        near("r", r, x + pb.double())
        t, o = make(6, cols)
        t["u"] = 1e4 + t["u"]
        check(trop, t, o, lost=1e-3)


@pytest.mark.parametrize("shape", [(0, 40), (3, 0, 8)])
def test_no_rows(trop, shape):
    x = torch.empty(shape, device="cuda")
    c = shape[-1]
    w = torch.ones(c, device="cuda")
    y, r, stats, kept = trop.residual_norm(x, x, w, w, scale=w, post_weight=w, post_bias=w, keep=True)
    assert y.shape == r.shape == x.shape and stats.shape == (4, *shape[:-1])
    for a in (dict(r=r, u=x), dict(r=kept[2], u=kept[0])):
        g = trop.residual_norm_backward(y, r, a["r"], a["u"], stats, w, w, scale=w, post_weight=w, post_bias=w)
        assert g[0].shape == x.shape and all(torch.equal(v, torch.zeros_like(w)) for v in g[3:])


def test_leading_axes(trop):
    t, o = make(24, 96, B, B, B, gate="row")
    tensors = {k: t[k] for k in ("scale", "post_weight", "post_bias")}
    y, r, stats, kept = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], gate=t["gate"], **tensors, **o, keep=True)
    v = lambda a: a.view(2, 3, 4, -1)  # noqa: E731
    other = trop.residual_norm(v(t["x"]).transpose(0, 1), v(t["u"]).transpose(0, 1), t["weight"], t["bias"],
                               gate=v(t["gate"]).transpose(0, 1), **tensors, **o, keep=True)
    assert torch.equal(other[0].transpose(0, 1).reshape(24, 96), y) and torch.equal(other[1].transpose(0, 1).reshape(24, 96), r)
    assert other[2].shape == (4, 3, 2, 4)
    g = trop.residual_norm_backward(t["dy"], t["dr"], kept[2], kept[0], stats, t["weight"], t["bias"], gate=t["gate"], **tensors, **o)
    h = trop.residual_norm_backward(v(t["dy"]).transpose(0, 1), v(t["dr"]).transpose(0, 1), other[3][2], other[3][0], other[2],
                                    t["weight"], t["bias"], gate=v(t["gate"]).transpose(0, 1), **tensors, **o)
    for a, b in zip(g[:3], h[:3]):
        assert torch.equal(b.transpose(0, 1).reshape(a.shape), a)


@pytest.mark.parametrize("gate, act, norm", [("full", "silu", "layer"), ("row", "sigmoid", "rms"), ("none", "none", "layer")])
def test_autograd(trop, gate, act, norm):
    """Against autograd of the definition in 64 bits, and a difference along a direction."""
    t, o = make(19, 130, gate=gate, gate_act=act, norm=norm)
    keys = [k for k in ("x", "u", "weight", "bias", "gate", "scale", "post_weight", "post_bias") if t[k] is not None]
    leaves = {k: t[k].clone().requires_grad_() for k in keys}
    args = lambda d: (d["x"], d["u"], d["weight"], d["bias"], d.get("gate"), act, d["scale"], d["post_weight"], d["post_bias"],  # noqa: E731
                      True, norm, 0.7, 1e-5)
    y, r = trop.ResidualNorm.apply(*args(leaves))
    ((y * t["dy"]).sum() + (r * t["dr"]).sum()).backward()
    wide = {k: t[k].double().requires_grad_() for k in keys}
    f = lambda d: ref.forward(d["x"], d["u"], d["weight"], d["bias"], d.get("gate"), act, d["scale"], d["post_weight"],  # noqa: E731
                              d["post_bias"], True, norm, 0.7, 1e-5)
    total = lambda d: (f(d)[0] * t["dy"]).sum() + (f(d)[1] * t["dr"]).sum()  # noqa: E731
    total(wide).backward()
    for k in keys:
        near(k, leaves[k].grad, wide[k].grad)
    with torch.no_grad():
        way = {k: torch.randn_like(wide[k]) for k in keys}
        step = 1e-6
        up, down = ({k: wide[k] + s * way[k] for k in keys} for s in (step, -step))
        slope = float(total(up) - total(down)) / (2 * step)
    mine = sum(float((leaves[k].grad.double() * way[k]).sum()) for k in keys)
    size = sum(float(leaves[k].grad.double().norm() * way[k].norm()) for k in keys)
    assert abs(mine - slope) <= 1e-5 * size


def test_autograd_parts(trop):
    """One of the two results unused, few arguments, 8-bit copies, no gradient wanted, second derivatives."""
    t, o = make(23, 96, B, B, B)
    x, u = t["x"].clone().requires_grad_(), t["u"].clone().requires_grad_()
    y, r = trop.ResidualNorm.apply(x, u)
    y.float().square().sum().backward()
    assert x.grad.dtype == u.grad.dtype == B and bool(u.grad.isfinite().all())
    y, r = trop.ResidualNorm.apply(t["x"], u)
    u.grad = None
    r.sum().backward()
    want, sizes = ref.backward(torch.zeros_like(y), torch.ones_like(r), r.detach(), u.detach(), ref.forward(t["x"], u.detach())[2])
    near("du", u.grad, want["u"], B, sizes["u"])  # (a sum over a norm: its gradient cancels)
    y, r = trop.ResidualNorm.apply(x, u, t["weight"], t["bias"], t["gate"].requires_grad_(), "silu", t["scale"], t["post_weight"],
                                   t["post_bias"], True, "layer", 1.0, 1e-5, None, True)
    held = sum(v.numel() * v.element_size() for v in y.grad_fn.saved_tensors if v is not None)
    assert held < 3 * x.numel() * 1.1 + 16 * 23 + 6 * 2 * 96 + 23 * 3 * 64
    (y.sum() + r.sum()).backward()
    assert t["gate"].grad.shape == t["gate"].shape
    y, _ = trop.ResidualNorm.apply(x, u)
    g, = torch.autograd.grad(y.sum(), u, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_streams_graphs_and_threads(trop):
    t, o = make(300, 1001, B, B, B)
    tensors = {k: t[k] for k in ("gate", "scale", "post_weight", "post_bias")}

    def step(stream=None):
        y, r, stats, kept = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], **tensors, **o, keep=True, stream=stream)
        g = trop.residual_norm_backward(t["dy"], t["dr"], kept[2], kept[0], stats, t["weight"], t["bias"], stream=stream,
                                        **{**tensors, "gate": kept[1]}, **o)
        return (y, r, stats, *g)

    want = [v.clone() for v in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    t["x"].mul_(2)
    want = [v.clone() for v in step()]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):  # two graphs at once, and eager calls beside them
        for (g, _), side in zip(graphs, sides):
            with torch.cuda.stream(side):
                g.replay()
        eager = step()
        torch.cuda.synchronize()
        for out in (*[out for _, out in graphs], eager):
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals(trop):
    t, o = make(6, 64, B, B, B)

    def name(f, *a, **k):
        with pytest.raises(trop.TropicalError) as e:
            f(*a, **k)
        return e.value.name

    fw, x, u, w = trop.residual_norm, t["x"], t["u"], t["weight"]
    assert name(fw, x, u[:5]) == "SHAPE"
    assert name(fw, x, u.float()) == "DTYPE"
    assert name(fw, x, u.half()) == "DTYPE"
    assert name(fw, x.float(), u, out_dtype=F) == "DTYPE"
    assert name(fw, x, u, w.half()) == "DTYPE"
    assert name(fw, x, u, w[:63]) == "SHAPE"
    assert name(fw, x, u, w.cpu()) == "DEVICE_MISMATCH"
    assert name(fw, x, u.cpu()) == "DEVICE_MISMATCH"
    assert name(fw, x, u, gate=t["gate"][:, :2]) == "SHAPE"
    assert name(fw, x, u, gate=t["gate"].float()) == "DTYPE"
    assert name(fw, x, u, norm="group") == "INVALID_ARG"
    assert name(fw, x, u, gate_act="tanh") == "INVALID_ARG"
    assert name(fw, x, u, eps=-1.0) == "INVALID_ARG"
    assert name(fw, x, u, alpha=float("nan")) == "INVALID_ARG"
    assert name(fw, x, u, post_norm=False, post_weight=w) == "INVALID_ARG"
    assert name(fw, x[:, :0], u[:, :0]) == "SHAPE"
    assert name(fw, x.t(), u.t()) == "UNSUPPORTED"
    y, r, stats, kept = fw(x, u, w, keep=True)
    bw = trop.residual_norm_backward
    assert name(bw, t["dy"], t["dr"], kept[2], u, stats) == "INVALID_ARG"
    assert name(bw, t["dy"], t["dr"], r, u, stats, gate=kept[0]) == "INVALID_ARG"
    assert name(bw, t["dy"], t["dr"], kept[2], kept[0], stats, gate=t["gate"]) == "INVALID_ARG"
    assert name(bw, t["dy"], t["dr"].float(), r, u, stats) == "DTYPE"
    assert name(bw, t["dy"], t["dr"], r, u, stats[:3]) == "SHAPE"
    assert name(bw, t["dy"], t["dr"][:5], r, u, stats) == "SHAPE"
    assert name(bw, t["dy"].float(), t["dr"], r, u, stats) == "DTYPE"
    assert name(bw, t["dy"], t["dr"], (kept[2][0], kept[2][1][:, :1]), kept[0], stats) == "SHAPE"
