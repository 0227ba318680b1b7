"""The training operators' host side at its edges, with stand-ins for the device.  No GPU."""

import contextlib

import pytest
import torch


@pytest.fixture()
def train(monkeypatch):
    """train.py with the C calls replaced by a record of them: (name, arguments, current stream)."""
    from einsum_device_side_gb300 import train as module

    class Library:
        def __getattr__(self, name):
            def call(*args):
                module.calls.append((name, args, module.current[-1]))
                return module.answers.pop(0) if module.answers else 0
            return call

    class Stream:
        def __init__(self, handle):
            self.cuda_stream, self.device = handle, None

    @contextlib.contextmanager
    def use(stream):
        module.current.append(stream)
        yield
        module.current.pop()

    home = Stream(1)
    for name, value in (("calls", []), ("answers", []), ("current", [home]), ("Side", Stream), ("recorded", [])):
        monkeypatch.setattr(module, name, value, raising=False)
    monkeypatch.setattr(module._pkg, "_lib", Library())
    monkeypatch.setattr(module._pkg, "_fc", None)
    monkeypatch.setattr(module, "_fast", lambda: None)
    monkeypatch.setattr(module._pkg, "_stream", lambda stream=None, like=None: (stream or module.current[-1]).cuda_stream)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: module.current[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: module.recorded.append((t.data_ptr(), s.cuda_stream)),
                        raising=False)
    return module


def test_copies_and_results_belong_to_the_stream_given(train, monkeypatch):
    """Rows whose leading axes do not merge are copied: the copy, like the results, has to be made on the stream that the
    kernel uses."""
    side, made = train.Side(7), []
    reshape, empty, empty_like = torch.Tensor.reshape, torch.empty, torch.empty_like
    monkeypatch.setattr(torch.Tensor, "reshape", lambda t, *s: made.append(train.current[-1]) or reshape(t, *s))
    monkeypatch.setattr(train, "_empty", lambda *a, **k: made.append(train.current[-1]) or empty(*a, **k))
    monkeypatch.setattr(train, "_empty_like", lambda *a, **k: made.append(train.current[-1]) or empty_like(*a, **k))
    x = torch.zeros(3, 9, 8)[:, :5]
    y, mean, rstd = train.layer_norm(x, stream=side)
    assert made and all(s is side for s in made)
    made.clear()
    dx, _, _ = train.layer_norm_backward(x, x, mean, rstd, want_weight=False, want_bias=False, stream=side)
    assert made and all(s is side for s in made)
    assert [c[0] for c in train.calls] == ["tropical_layer_norm", "tropical_layer_norm_backward"]
    assert all(c[1][-1] == side.cuda_stream for c in train.calls)
    # the allocator knows: inputs are used on the side stream, results on the caller's
    assert (x.data_ptr(), 7) in train.recorded
    assert all((t.data_ptr(), 1) in train.recorded for t in (y, mean, rstd, dx))


def test_a_plan_s_tensors_outlive_its_steps_on_another_stream(train, monkeypatch):
    import ctypes
    t = [torch.zeros(4) for _ in range(4)]

    def create(*args):
        ctypes.cast(args[-1], ctypes.POINTER(ctypes.c_void_p))[0] = 5
        return 0

    monkeypatch.setattr(type(train._pkg._lib), "tropical_adamw_plan_create", staticmethod(create), raising=False)
    plan = train.AdamWPlan(*([x] for x in t))
    plan.step(1, stream=train.Side(7))
    assert not train.recorded
    plan.close()
    assert sorted(train.recorded) == sorted((x.data_ptr(), 7) for x in t)


@pytest.mark.parametrize("given", [1, 2, 3])
def test_layer_norm_differentiates_with_any_of_its_arguments(train, given):
    args = [torch.zeros(3, 8, requires_grad=True), torch.ones(8, requires_grad=True), torch.zeros(8, requires_grad=True)]
    train.LayerNorm.apply(*args[:given]).sum().backward()
    assert [a.grad is not None for a in args] == [i < given for i in range(3)]


def test_second_derivatives_are_refused(train):
    """What the C calls return has no graph: a second derivative would silently lack these operators' part."""
    x = torch.zeros(3, 8, requires_grad=True)
    w = torch.ones(8, requires_grad=True)
    y = train.LayerNorm.apply(x, w)
    dx, = torch.autograd.grad((y * y).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        dx.sum().backward()
    h = torch.zeros(3, 8, dtype=torch.bfloat16, requires_grad=True)
    v = torch.zeros(5, 8, dtype=torch.bfloat16, requires_grad=True)
    loss = train.LinearCrossEntropy.apply(h, v, torch.zeros(3, dtype=torch.int64))
    dh, = torch.autograd.grad(loss * loss, h, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        dh.sum().backward()


def test_leading_axes_in_any_order(train):
    """A dense input with its leading axes exchanged: empty_like would keep the exchanged strides, which make no rows."""
    x = torch.zeros(5, 4, 8).transpose(0, 1)
    y, mean, rstd = train.layer_norm(x)
    assert y.shape == (4, 5, 8) and y.is_contiguous()
    dx, dw, db = train.layer_norm_backward(x, x, mean, rstd)
    assert dx.shape == (4, 5, 8) and dx.is_contiguous()
    with pytest.raises(train._pkg.TropicalError) as e:
        train.layer_norm(x, out=torch.zeros(5, 4, 8).transpose(0, 1))
    assert e.value.name == "UNSUPPORTED"


def test_the_loss_is_no_view_and_may_be_changed_in_place(train):
    h = torch.zeros(3, 8, dtype=torch.bfloat16, requires_grad=True)
    v = torch.zeros(5, 8, dtype=torch.bfloat16)
    target = torch.zeros(3, dtype=torch.int64)
    for reduction in ("mean", "sum", "none"):
        loss, _, kept = train.linear_cross_entropy(h.detach(), v, target, reduction)
        assert loss._base is None and kept._base is None and loss.shape == ((3,) if reduction == "none" else ())
        loss = train.LinearCrossEntropy.apply(h, v, target, reduction)
        loss /= 4
        loss.detach().mul_(2)
        loss.sum().backward()


def test_a_refused_step_does_not_count(train, monkeypatch):
    import ctypes

    def create(*args):
        ctypes.cast(args[-1], ctypes.POINTER(ctypes.c_void_p))[0] = 5
        return 0

    monkeypatch.setattr(type(train._pkg._lib), "tropical_adamw_plan_create", staticmethod(create), raising=False)
    monkeypatch.setattr(train, "_capturing", lambda stream: False)
    monkeypatch.setattr(type(train._pkg._lib), "tropical_last_error", staticmethod(lambda: b"refused"), raising=False)
    opt = train.AdamW([torch.zeros(4)], [torch.zeros(4)])
    opt.step()
    train.answers.append(-1)
    with pytest.raises(train._pkg.TropicalError):
        opt.step()
    after = opt.steps
    opt._plan._h = None  # (no plan of the library's)
    assert after == 1


@pytest.mark.parametrize("fast", [False, True])
def test_no_room_for_the_workspace(train, monkeypatch, fast):
    """The library's workspace is not torch's: before a call gives up, torch's idle memory is given back."""
    emptied = []
    monkeypatch.setattr(torch.cuda, "empty_cache", lambda: emptied.append(1))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(type(train._pkg._lib), "tropical_last_error", staticmethod(lambda: b"no room"), raising=False)
    if fast:
        class Fast:
            def __getattr__(self, name):
                return lambda *args: train.answers.pop(0) if train.answers else 0 if name.endswith("_t") else 1
        monkeypatch.setattr(train, "_fast", lambda binding=Fast(): binding)
    h, v = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16)
    t, s, x, w = torch.zeros(3, dtype=torch.int64), torch.zeros(3), torch.zeros(3, 8), torch.zeros(8)
    calls = (lambda: train.linear_cross_entropy(h, v, t), lambda: train.linear_cross_entropy_backward(s, h, v, t, s),
             lambda: train.layer_norm_backward(x, x, s, s, w), lambda: train.layer_norm_backward(x, x, s, s))
    for i, call in enumerate(calls):
        train.answers[:] = [-9, 0 if not fast or i in (1, 3) else 1]
        call()
        assert len(emptied) == i + 1
    train.answers[:] = [-9, -9]
    with pytest.raises(train._pkg.TropicalError) as e:
        calls[1]()
    assert e.value.name == "OOM"
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    train.answers[:] = [-9]
    emptied.clear()
    with pytest.raises(train._pkg.TropicalError):
        calls[1]()
    assert not emptied


def test_a_parameter_s_new_gradient_buffer_is_noticed(train, monkeypatch):
    """zero_grad drops the buffers by default and backward makes new ones, which the plan does not know."""
    import ctypes

    def create(*args):
        ctypes.cast(args[-1], ctypes.POINTER(ctypes.c_void_p))[0] = 5
        return 0

    monkeypatch.setattr(type(train._pkg._lib), "tropical_adamw_plan_create", staticmethod(create), raising=False)
    monkeypatch.setattr(train, "_capturing", lambda stream: False)
    p = torch.zeros(4, requires_grad=True)
    p.sum().backward()
    opt = train.AdamW([p])
    opt.step()
    p.grad.zero_()
    p.sum().backward()
    opt.step()
    refused = []
    for grad in (None, torch.ones(4)):
        p.grad = grad
        try:
            opt.step()
        except train._pkg.TropicalError as e:
            refused.append(e.name)
    steps = opt.steps
    opt._plan._h = None  # (no plan of the library's)
    assert refused == ["INVALID_ARG"] * 2 and steps == 2
