"""The weight gradient from an 8-bit copy against 64 bits: sizes that end inside a stage, a tile and a group, splits of
the tokens, strides, empty sums, types.

Limits: products are exact (8 bits times 8 or 11), a sum of n of them in f32 loses at most a last place of the
accumulator for every 16 products, so n / 16 2^-24 of the sum of magnitudes; a stored value half a step besides."""

import pytest
import torch

pytestmark = pytest.mark.gpu

F, B, H = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def trop():
    import einsum_device_side_gb300 as t
    t.load()
    return t


def make(trop, t, o, c, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + t + 3 * o + 5 * c)
    dy = torch.randn(t, o, generator=g, device="cuda").to(dt)
    x = torch.randn(t, c, generator=g, device="cuda") * (0.2 + torch.rand(c, generator=g, device="cuda"))
    return dy, *trop.activation_pack(x.to(dt))


def check(trop, dy, codes, scales, to=None, bias=True):
    dw, db = trop.activation_weight_grad(dy, codes, scales, out_dtype=to, want_bias=bias)
    dt = to or dy.dtype
    assert dw.dtype == dt and (db is None) == (not bias)
    x = trop.activation_values(codes, scales, dy.dtype).double().reshape(-1, codes.shape[-1])
    d = dy.double().reshape(-1, dy.shape[-1])
    half = 0.0 if dt == F else torch.finfo(dt).eps / 2
    tiny = 0.0 if dt != H else 2.0 ** -25  # half a step of f16's subnormal numbers
    for name, got, want, size in (("dw", dw, d.T @ x, d.abs().T @ x.abs()), ("db", db, d.sum(0), d.abs().sum(0))):
        if got is None:
            continue
        assert got.shape == want.shape and bool(got.isfinite().all()), name
        lost = (d.shape[0] / 16 + 2) * 2.0 ** -24 * size
        most = lost + half * (want.abs() + lost) + tiny
        over = (got.double() - want).abs() - most
        assert got.numel() == 0 or float(over.max()) <= 0, (name, float(over.max()))
    return dw, db


SIZES = [(1, 1, 1), (1, 8, 32), (7, 64, 96), (63, 40, 33), (64, 256, 256), (65, 257, 255), (128, 300, 1000), (129, 1000, 31),
         (1021, 203, 700), (500, 1, 2000), (4100, 96, 64), (20000, 24, 40), (513, 2049, 513)]


@pytest.mark.parametrize("to", [None, F])
@pytest.mark.parametrize("dt", [B, H])
@pytest.mark.parametrize("t, o, c", SIZES)
def test_sizes(trop, t, o, c, dt, to):
    check(trop, *make(trop, t, o, c, dt), to=to)


@pytest.mark.parametrize("t, o, c", [(1024, 4096, 2048), (300, 8192, 1024), (8192, 512, 768)])
def test_many_tiles(trop, t, o, c):
    """More tiles than pairs of CTAs, and more tokens than a split's."""
    check(trop, *make(trop, t, o, c, B), bias=False)
    check(trop, *make(trop, t, o, c, H), to=F)


@pytest.mark.parametrize("dt", [B, H])
def test_strides(trop, dt):
    dy, codes, scales = make(trop, 150, 72, 96, dt)
    want = check(trop, dy, codes, scales)
    wide = torch.zeros(150, 80, dtype=dt, device="cuda")
    wide[:, 3:75] = dy
    for d in (dy.t().contiguous().t(), wide[:, 3:75], dy.flip(0).flip(0)):
        for a, b in zip(trop.activation_weight_grad(d, codes, scales, want_bias=True), want):
            assert torch.equal(a, b)
    for pitch in (96, 97, 112):  # rows of codes on 16 bytes, off them
        c = torch.zeros(150, pitch, dtype=torch.int8, device="cuda")[:, :96]
        c.copy_(codes)
        s = torch.zeros(150, 5, dtype=torch.uint8, device="cuda")[:, 1:4]
        s.copy_(scales)
        for a, b in zip(trop.activation_weight_grad(dy, c, s, want_bias=True), want):
            assert torch.equal(a, b)
    one = trop.activation_weight_grad(dy[:1].expand(150, 72), codes, scales)[0]
    x = trop.activation_values(codes, scales, dt).double()
    assert float((one.double() - dy[:1].double().expand(150, 72).T @ x).norm() / one.double().norm()) < torch.finfo(dt).eps


def test_leading_axes(trop):
    dy, codes, scales = make(trop, 60, 40, 64, B)
    want = trop.activation_weight_grad(dy, codes, scales, want_bias=True)
    v = lambda t: t.view(3, 4, 5, -1)  # noqa: E731
    got = trop.activation_weight_grad(v(dy), v(codes), v(scales), want_bias=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("t, o, c", [(0, 5, 7), (4, 0, 7), (4, 5, 0), (0, 0, 0)])
@pytest.mark.parametrize("to", [None, F])
def test_empty(trop, t, o, c, to):
    dy = torch.ones(t, o, dtype=B, device="cuda")
    codes, scales = trop.activation_pack(torch.ones(t, c, dtype=B, device="cuda"))
    dw, db = trop.activation_weight_grad(dy, codes, scales, out_dtype=to, want_bias=True)
    assert dw.shape == (o, c) and bool((dw == 0).all()) and torch.equal(db, torch.full_like(db, t))


def test_values_out_of_range_and_bad_groups(trop):
    """A group that held a NaN spoils its columns' gradients and no others; f16 makes infinities of what it cannot hold."""
    dy, codes, scales = make(trop, 100, 64, 160, B)
    want = trop.activation_weight_grad(dy, codes, scales)[0]
    scales[50, 2] = 255
    got = trop.activation_weight_grad(dy, codes, scales)[0]
    cols = torch.zeros(160, dtype=torch.bool, device="cuda")
    cols[64:96] = True
    assert bool(got[:, cols].isnan().all()) and torch.equal(got[:, ~cols], want[:, ~cols])
    big = torch.full((70, 64), 1e6, device="cuda")
    codes, scales = trop.activation_pack(big)
    assert bool(trop.activation_weight_grad(torch.ones(70, 8, dtype=H, device="cuda"), codes, scales)[0].isinf().all())


def test_repeats_bit_for_bit_on_streams_in_graphs(trop):
    """Split sums too: results do not depend on what runs beside."""
    args = make(trop, 6000, 200, 300, B)
    want = trop.activation_weight_grad(*args, want_bias=True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(trop.activation_weight_grad(*args, want_bias=True), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = trop.activation_weight_grad(*args, want_bias=True, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = trop.activation_weight_grad(*args, want_bias=True)
        graphs.append((g, out))
    args[0].mul_(0.5)
    want = trop.activation_weight_grad(*args, want_bias=True)
    sides = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(3):
        for (g, _), side in zip(graphs, sides):
            with torch.cuda.stream(side):
                g.replay()
        eager = trop.activation_weight_grad(*args, want_bias=True)
        torch.cuda.synchronize()
        for out in (*[o for _, o in graphs], eager):
            assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("bias", [True, False])
def test_linear8(trop, bias):
    g = torch.Generator(device="cuda").manual_seed(4)
    x, w, b = (torch.randn(*s, generator=g, device="cuda").to(B).requires_grad_() for s in ((3, 50, 96), (40, 96), (40,)))
    dy = torch.randn(3, 50, 40, generator=g, device="cuda").to(B)
    y = trop.Linear8.apply(x, w, b) if bias else trop.Linear8.apply(x, w)
    y.backward(dy)
    assert torch.equal(y, torch.nn.functional.linear(x, w, b if bias else None))
    codes, scales = trop.activation_pack(x.detach())
    dw, db = trop.activation_weight_grad(dy, codes, scales, want_bias=True)
    assert torch.equal(w.grad, dw) and torch.equal(x.grad, dy @ w.detach()) and (not bias or torch.equal(b.grad, db))
    # an element of x is off by 1/64 of its group's largest at most: so is the gradient, of the sum of magnitudes
    top = x.detach().double().view(150, 3, 32).abs().amax(2).repeat_interleave(32, 1)
    exact, size = dy.double().view(150, 40).T @ x.detach().double().view(150, 96), dy.double().view(150, 40).abs().T @ top
    assert bool(((dw.double() - exact).abs() <= size / 64 + exact.abs() / 128).all())
    frozen = trop.Linear8.apply(x, w.detach())
    assert [t for t in frozen.grad_fn.saved_tensors if t is not None and t.dtype == torch.int8] == []


def test_refusals(trop):
    dy, codes, scales = make(trop, 20, 8, 64, B)

    def name(f, *a, **k):
        with pytest.raises(trop.TropicalError) as e:
            f(*a, **k)
        return e.value.name

    f = trop.activation_weight_grad
    assert name(f, dy.float(), codes, scales) == "DTYPE"
    assert name(f, dy, codes, scales, out_dtype=H) == "DTYPE"
    assert name(f, dy, codes, scales, out_dtype=torch.float64) == "DTYPE"
    assert name(f, dy[:19], codes, scales) == "SHAPE"
    assert name(f, dy, codes, scales[:, :1]) == "SHAPE"
    assert name(f, dy, codes.to(torch.uint8), scales) == "DTYPE"
    assert name(f, dy.cpu(), codes, scales) == "DEVICE_MISMATCH"
    assert name(f, dy, codes.t().contiguous().t(), scales) == "UNSUPPORTED"
    assert name(trop.Linear8.apply, dy.float(), torch.ones(4, 8, device="cuda")) == "DTYPE"
