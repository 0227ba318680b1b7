"""The residual block's operators where their routes change: rows on 8 bytes but not on 16, copies that a user cut out of
others, many rows of few columns, offsets past 32 bits, clusters under capture, one tensor given twice; and a small deep
network that uses them all.

Limits as in test_gpu_residual_norm.py: a stored value is off by at most eps / 2 of its type relative to itself, sums in
32 bits lose less than 1e-5 of the terms that a result is the sum of."""

import pytest
import torch

import residual_reference as ref
from test_gpu_residual_norm import check, make, near

pytestmark = pytest.mark.gpu

F, B, H = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def trop():
    import einsum_device_side_gb300 as t
    t.load()
    return t


@pytest.mark.parametrize("S, U, Y, keep", [(F, F, F, False), (F, F, B, False), (F, F, H, True), (B, B, B, True), (F, B, B, True), (H, H, H, False)])
@pytest.mark.parametrize("rows, cols", [(7, 4), (33, 12), (130, 24), (1500, 40), (3000, 104), (400, 4104), (330, 5000), (300, 12296)])
def test_columns_that_divide_by_8_alone(trop, rows, cols, S, U, Y, keep):
    t, o = make(rows, cols, S, U, Y, gate="full" if cols % 16 else "row", gate_act="silu", seed=rows)
    check(trop, t, o, S, U, Y, keep)


@pytest.mark.parametrize("S, U, Y", [(F, F, F), (B, B, B), (F, F, B)])
@pytest.mark.parametrize("pad, shift", [(4, 0), (4, 4), (8, 8), (12, 4)])
def test_rows_between_16_bytes(trop, S, U, Y, pad, shift):
    t, o = make(500, 256, S, U, Y, gate_act="sigmoid", pad=pad, shift=shift)
    check(trop, t, o, S, U, Y)


@pytest.mark.parametrize("cut, width", [(0, 256), (32, 224), (64, 160), (96, 100)])
def test_copies_cut_out_of_wider_ones(trop, cut, width):
    """Copies from column `cut` on (whole groups), with the wide copies' strides; and with codes one byte further on."""
    t, o = make(90, width, B, B, B, gate_act="silu")
    y, r, stats, kept = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], gate=t["gate"], scale=t["scale"],
                                           post_weight=t["post_weight"], post_bias=t["post_bias"], **o, keep=True)
    kw = dict(scale=t["scale"], post_weight=t["post_weight"], post_bias=t["post_bias"], **o)
    want = trop.residual_norm_backward(t["dy"], t["dr"], kept[2], kept[0], stats, t["weight"], t["bias"], gate=kept[1], **kw)

    def inside(pair, off):
        codes = torch.full((90, cut + width + 70), 77, dtype=torch.int8, device="cuda")
        scales = torch.full((90, (cut + width + 70) // 32 + 2), 200, dtype=torch.uint8, device="cuda")
        groups = pair[1].shape[1]
        c, s = codes[:, cut + off:cut + off + width], scales[:, cut // 32:cut // 32 + groups]
        c.copy_(pair[0])
        s.copy_(pair[1])
        return c, s

    for off in (0, 1, 8):
        ku, kg, kr = (inside(p, off) for p in kept)
        got = trop.residual_norm_backward(t["dy"], t["dr"], kr, ku, stats, t["weight"], t["bias"], gate=kg, **kw)
        for name, a, b in zip("dx du dgate dscale dweight dbias dpost_weight dpost_bias".split(), got, want):
            near(name, a, b, B, b.double().abs())  # (another route adds up in another order)
        dy = t["dy"]
        near("dw", trop.activation_weight_grad(dy, *ku)[0], dy.double().T @ trop.activation_values(*ku, F).double(), B)


@pytest.mark.parametrize("cols, dt", [(32, B), (100, F), (64, H), (513, B)])
def test_rows_in_excess_of_every_block(trop, cols, dt):
    t, o = make(70001, cols, dt, dt, dt, gate="row", gate_act="sigmoid", norm="rms")
    # column sums over 70001 rows, 152 blocks' at a time, in f32: chains of up to 500 additions a thread, 3e-5 of the terms
    check(trop, t, o, dt, dt, dt, lost=5e-5)


@pytest.mark.parametrize("stride", [(1 << 31) + 8, (1 << 32) + 64])
def test_rows_far_apart(trop, stride):
    """Rows whose distance 32 bits of bytes do not hold."""
    t, o = make(2, 96, B, B, B, gate_act="silu")
    far = torch.empty(stride + 96, dtype=B, device="cuda")
    x = far.as_strided((2, 96), (stride, 1))
    x.copy_(t["x"])
    want = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], gate=t["gate"], **o)
    got = trop.residual_norm(x, t["u"], t["weight"], t["bias"], gate=t["gate"], **o)
    for name, a, b, dt in zip(("y", "r", "stats"), got, want, (B, B, F)):
        near(name, a, b, dt, b.double().abs())
    g = trop.residual_norm_backward(t["dy"], x, got[1], t["u"], got[2], t["weight"], t["bias"], gate=t["gate"], **o)
    w = trop.residual_norm_backward(t["dy"], t["x"], got[1], t["u"], got[2], t["weight"], t["bias"], gate=t["gate"], **o)
    for a, b in zip(g, w):
        if b is not None:
            near("gradient", a, b, a.dtype, b.double().abs())


def test_offsets_past_32_bits(trop):
    """More elements than 31 bits count: the last rows as if they stood alone."""
    rows, cols, tail = (1 << 31) // 1024 + 1003, 1024, 900
    x = torch.randn(rows, cols, device="cuda", dtype=B)
    u = x.roll(1, 0)
    w = torch.randn(cols, device="cuda").to(B)
    y, r, stats, kept = trop.residual_norm(x, u, w, keep=True)
    y1, r1, stats1, kept1 = trop.residual_norm(x[-tail:], u[-tail:], w, keep=True)
    assert torch.equal(y[-tail:], y1) and torch.equal(r[-tail:], r1) and torch.equal(stats[:, -tail:], stats1)
    assert all(torch.equal(a[-tail:], b) for p, q in ((kept[0], kept1[0]), (kept[2], kept1[2])) for a, b in zip(p, q))
    del r
    dx, du, *_ = trop.residual_norm_backward(y, x, kept[2], kept[0], stats, w, want=("x", "u"))
    dx1, du1, *_ = trop.residual_norm_backward(y1, x[-tail:], kept1[2], kept1[0], stats1, w, want=("x", "u"))
    assert torch.equal(dx[-tail:], dx1) and torch.equal(du[-tail:], du1)
    values = trop.activation_values(*kept[0], B)
    assert torch.equal(values[-tail:], trop.activation_values(*kept1[0], B))


def test_wide_rows_repeat_and_can_be_captured(trop):
    """Rows shared by a cluster: bit for bit the same again, on two streams at once, and from a graph with other inputs."""
    t, o = make(333, 8192, B, B, B, gate_act="silu")

    def step():
        y, r, stats, kept = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], gate=t["gate"], scale=t["scale"], **o, keep=True)
        return (y, r, *trop.residual_norm_backward(t["dy"], t["dr"], kept[2], kept[0], stats, t["weight"], t["bias"], gate=kept[1],
                                                   scale=t["scale"], **o))

    same = lambda p, q: all(a is b if b is None else torch.equal(a, b) for a, b in zip(p, q))  # noqa: E731
    want = step()
    assert same(step(), want)
    sides = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            results.append([step() for _ in range(3)])
    torch.cuda.synchronize()
    assert all(same(r, want) for rs in results for r in rs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    t["u"].mul_(-0.5)
    g.replay()
    torch.cuda.synchronize()
    assert same(out, step())


@pytest.mark.parametrize("keep", [False, True])
def test_one_tensor_given_twice(trop, keep):
    t, o = make(70, 300, B, B, B)
    args = dict(gate=t["x"], scale=t["scale"], **o, keep=keep)
    one = trop.residual_norm(t["x"], t["x"], t["weight"], t["weight"], **args)
    two = trop.residual_norm(t["x"], t["x"].clone(), t["weight"], t["weight"].clone(), **{**args, "gate": t["x"].clone()})
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    ku, kg, kr = one[3] if keep else (t["x"], t["x"], one[1])
    a = trop.residual_norm_backward(t["dy"], t["dy"], kr, ku, one[2], t["weight"], t["weight"], gate=kg, scale=t["scale"], **o)
    b = trop.residual_norm_backward(t["dy"], t["dy"].clone(), kr, ku, one[2], t["weight"], t["weight"].clone(), gate=kg,
                                    scale=t["scale"].clone(), **o)
    assert all(p is q or torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("capture", [False, True])
def test_a_deep_network(trop, capture):
    """Two blocks, each a linear layer that keeps its input in 8 bits and the fused norms around it with 8-bit copies, then the
    head's cross entropy: as a user trains it, eagerly and captured, against 64 bits with the same copies."""
    n, c, vocab, dt = 192, 160, 500, B
    g = torch.Generator(device="cuda").manual_seed(5)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    params = {"x": normal(n, c), "head": normal(vocab, c) / c ** 0.5}
    for i in range(2):
        params |= {f"w{i}": normal(c, c) / c ** 0.5, f"g{i}": normal(c, c) / c ** 0.5, f"s{i}": 0.5 + 0.1 * normal(c), f"n{i}": 1 + 0.1 * normal(c),
                   f"p{i}": 1 + 0.1 * normal(c)}
    params = {k: v.to(dt).requires_grad_() for k, v in params.items()}
    target = torch.randint(0, vocab, (n,), generator=g, device="cuda")

    def loss():
        p = params
        r = y = p["x"]
        for i in range(2):
            u, gate = trop.Linear8.apply(y, p[f"w{i}"]), trop.Linear8.apply(y, p[f"g{i}"])
            y, r = trop.ResidualNorm.apply(r, u, p[f"n{i}"], None, gate, "silu", p[f"s{i}"], p[f"p{i}"], None, True, "rms", 1.0, 1e-5, None, True)
        return trop.LinearCrossEntropy.apply(y, p["head"], target)

    def exact():
        p = {k: v.detach().double().requires_grad_() for k, v in params.items()}
        r = y = p["x"]
        for i in range(2):
            u, gate = y @ p[f"w{i}"].T, y @ p[f"g{i}"].T
            y, r, _ = ref.forward(r, u, p[f"n{i}"], None, gate, "silu", p[f"s{i}"], p[f"p{i}"], None, True, "rms", 1.0, 1e-5)
        total = torch.nn.functional.cross_entropy(y @ p["head"].T, target)
        return total.detach(), dict(zip(p, torch.autograd.grad(total, list(p.values()))))

    def grads():
        return dict(zip(params, torch.autograd.grad(loss(), list(params.values()))))

    got = grads()
    if capture:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            grads()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = grads()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], got[k]) for k in got)
        return
    total, want = exact()
    assert abs(float(loss().detach()) - float(total)) <= 0.05 * float(total)
    # An 8-bit element is off by 1/128 of its group's largest, about 1/60 of the group's size; half a dozen such roundings and a
    # dozen of bf16 (2^-9 each on average) in a chain of two blocks: a few per cent of a gradient's norm.
    for k in want:
        err, size = float((got[k].double() - want[k]).norm()), float(want[k].norm())
        assert err <= 0.1 * size, (k, err / size)


@pytest.mark.parametrize("S, U, Y, keep", [(F, F, B, False), (F, F, H, True), (F, B, B, False), (F, B, B, True), (B, B, B, False), (H, H, H, True)])
@pytest.mark.parametrize("rows, cols", [(20, 1000), (300, 4096), (160, 8192), (40, 9001)])
def test_32_bit_vectors_beside_16_bit_results(trop, rows, cols, S, U, Y, keep):
    t, o = make(rows, cols, S, U, Y, W=F, gate_act="silu", seed=cols)
    check(trop, t, o, S, U, Y, keep)


def test_vectors_of_a_call_over_no_rows(trop):
    """They are read for the sums' products: on the host they are refused there too."""
    import ctypes

    from einsum_device_side_gb300 import block, train
    x = torch.empty(0, 8, device="cuda")
    host, grad = torch.ones(8), torch.empty(8, device="cuda")
    o = block._Options(0, 1, 0, 0, 1.0, 1.0, 0.0, None, None, host.data_ptr(), None, None)
    g = block._Grads(None, None, None, None, None, None, grad.data_ptr(), None)
    rc = trop._lib.tropical_residual_norm_backward(ctypes.byref(o), train._desc(x), None, train._desc(x), train._desc(x), None, None, None, 0,
                                                   0, ctypes.byref(g), None)
    assert trop.ERRORS.get(rc) == "HOST_POINTER"
