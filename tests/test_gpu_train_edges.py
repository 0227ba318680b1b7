"""The training operators at the edges of their interface: streams, layouts, autograd's corners, captures, extreme values."""

import pytest
import torch

pytestmark = pytest.mark.gpu

F, B, H = torch.float32, torch.bfloat16, torch.float16
IGNORE = -100


@pytest.fixture(scope="module")
def trop():
    import einsum_device_side_gb300 as t
    t.load()
    return t


def _normal(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda")


# ------------------------------------------------------------------ streams


def test_rows_that_are_copied_follow_the_stream_given(trop):
    """The leading axes do not merge, so the call copies them: on the stream given, not behind the caller's own work."""
    x, dy, w = _normal(1, 6, 9, 64)[:, :5], _normal(2, 6, 9, 64)[:, :5], _normal(3, 64)
    want = trop.layer_norm(x.contiguous(), w)
    stats = [s.T.contiguous().T for s in want[1:]]  # of another order, so copied too
    grads = trop.layer_norm_backward(dy.contiguous(), x.contiguous(), *want[1:], w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # the caller's stream is busy for some 50 ms
    got = trop.layer_norm(x, w, stream=side)
    back = trop.layer_norm_backward(dy, x, *stats, w, stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        same = [torch.equal(a, b) for a, b in zip((*got, *back), (*want, *grads))]
    assert all(same), same


@pytest.mark.parametrize("bits", [32, 8])
def test_a_plan_is_ready_for_any_stream_when_it_is_made(trop, bits):
    """A plan of many tensors (its table lies in device memory), stepped at once on a stream that waits for nothing."""
    sizes = [300 + i for i in range(400)]
    hyper = dict(lr=1e-2, weight_decay=0.0)
    p, g = [_normal(i, n) for i, n in enumerate(sizes)], [_normal(1000 + i, n) for i, n in enumerate(sizes)]
    q = [t.clone() for t in p]
    dtypes = (F, F) if bits == 32 else (torch.int8, torch.uint8)
    make = lambda: [[torch.zeros(n, dtype=d, device="cuda") for n in sizes] for d in dtypes] + (  # noqa: E731
        [] if bits == 32 else [[torch.zeros(-(-n // 256), device="cuda") for n in sizes] for _ in range(2)])
    a, b, values = make(), make(), [[torch.empty(n, device="cuda") for n in sizes] for _ in range(2)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    plan = trop.AdamWPlan(p, g, *a, values=tuple(values) if bits == 8 else None)
    plan.step(1, stream=side, **hyper)
    if bits == 8:
        plan.state_values(stream=side)
    side.synchronize()
    trop.adamw_step(q, g, *b, step=1, **hyper)
    assert all(torch.equal(x, y) for x, y in zip(p, q))
    assert all(torch.equal(x, y) for s, t in zip(a, b) for x, y in zip(s, t))
    if bits == 8:
        want = trop.adamw_state_values(*b)
        assert all(torch.equal(x, y) for s, t in zip(values, want) for x, y in zip(s, t))
    plan.close()


# ------------------------------------------------------------------ autograd


def test_a_gradient_penalty_raises(trop):
    x, w = _normal(1, 5, 32).requires_grad_(), _normal(2, 32).requires_grad_()
    y = trop.LayerNorm.apply(x, w)
    dx, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.square().sum().backward()
    h, v = _normal(3, 5, 32).to(B).requires_grad_(), _normal(4, 9, 32).to(B).requires_grad_()
    loss = trop.LinearCrossEntropy.apply(h, v, torch.arange(5, device="cuda"))
    dh, = torch.autograd.grad(loss.square(), h, create_graph=True)
    with pytest.raises(RuntimeError):
        dh.float().square().sum().backward()


# ------------------------------------------------------------------ layouts


@pytest.mark.parametrize("dt", [F, B])
@pytest.mark.parametrize("cols", [64, 33])
def test_layer_norm_of_leading_axes_in_any_order(trop, dt, cols):
    """[T, B, C] read as [B, T, C] and the other way, x and dy exchanged separately: bit for bit what contiguous rows give."""
    w, b = _normal(3, cols).to(dt), _normal(4, cols).to(dt)
    plain = _normal(1, 7, 5, cols).to(dt), _normal(2, 7, 5, cols).to(dt)
    want = trop.layer_norm(plain[0], w, b)
    grads = trop.layer_norm_backward(plain[1], plain[0], *want[1:], w)
    for swap_x in (False, True):
        for swap_dy in (False, True):
            x, dy = (t.transpose(0, 1).contiguous().transpose(0, 1) if s else t for t, s in zip(plain, (swap_x, swap_dy)))
            got = trop.layer_norm(x, w, b)
            assert all(torch.equal(p, q) for p, q in zip(got, want))
            assert all(torch.equal(p, q) for p, q in zip(trop.layer_norm_backward(dy, x, *want[1:], w), grads))
            leaf = x.detach().requires_grad_()
            trop.LayerNorm.apply(leaf, w, b).backward(dy)
            assert torch.equal(leaf.grad, grads[0])
    with pytest.raises(trop.TropicalError) as e:
        trop.layer_norm(plain[0], w, b, out=torch.empty(5, 7, cols, device="cuda", dtype=dt).transpose(0, 1))
    assert e.value.name == "UNSUPPORTED"
    y16 = trop.layer_norm(plain[0].float().transpose(0, 1), out_dtype=H)[0]
    assert y16.dtype == H and y16.shape == (5, 7, cols)


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_the_loss_may_be_changed_in_place(trop, reduction):
    h, v, t = _normal(3, 50, 32).to(B).requires_grad_(), _normal(4, 90, 32).to(B), torch.arange(50, device="cuda")
    plain = trop.LinearCrossEntropy.apply(h, v, t, reduction)
    value = plain.detach().clone()
    want, = torch.autograd.grad((plain / 4).sum(), h)
    loss = trop.LinearCrossEntropy.apply(h, v, t, reduction)
    loss /= 4
    assert torch.equal(loss.detach(), value / 4)
    loss.detach().mul_(2)  # what a program that logs the loss may do
    got, = torch.autograd.grad(loss.sum(), h)
    assert torch.equal(got, want)
