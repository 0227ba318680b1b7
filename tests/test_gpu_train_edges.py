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
