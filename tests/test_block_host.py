"""Host-side checks of the residual block's entry points: argument errors that are found before any device work, and the
wrappers' own checks.  No GPU."""

import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def trop():
    from einsum_device_side_gb300 import build
    build.build()
    import einsum_device_side_gb300 as t
    t.load()
    return t


F32, I32, I64, F64, BF16, F16, I8, U8 = range(8)


def _tensor(trop, dtype, shape, stride=None):
    t = trop.TropTensor()
    t.data, t.dtype, t.rank = 4096, dtype, len(shape)
    if stride is None:
        stride, acc = [], 1
        for n in reversed(shape):
            stride.insert(0, acc)
            acc *= n
    for i, (n, s) in enumerate(zip(shape, stride)):
        t.shape[i], t.stride[i] = n, s
    return t


def _kept(block, u=None, gate=None, r=None):
    table = (block._Kept * 3)()
    for to, pair in zip(table, (u, gate, r)):
        if pair is not None:
            to.codes, to.scales = map(ctypes.pointer, pair)
    return table


@pytest.fixture
def block(trop):
    from einsum_device_side_gb300 import block as b
    return b


def test_activation_argument_errors(trop):
    t = lambda *a, **k: _tensor(trop, *a, **k)  # noqa: E731

    def call(x, codes, scales, pack=True):
        at = lambda d: None if d is None else ctypes.byref(d)  # noqa: E731
        f = trop._lib.tropical_activation_pack if pack else trop._lib.tropical_activation_values
        args = (x, codes, scales) if pack else (codes, scales, x)
        return trop.ERRORS.get(f(*map(at, args), None))

    for pack in (True, False):
        good = t(BF16, (4, 40)), t(I8, (4, 40)), t(U8, (4, 2))
        assert call(t(F64, (4, 40)), *good[1:], pack) == "DTYPE"
        assert call(good[0], t(U8, (4, 40)), good[2], pack) == "DTYPE"
        assert call(good[0], good[1], t(I8, (4, 2)), pack) == "DTYPE"
        assert call(good[0], t(I8, (4, 41)), good[2], pack) == "SHAPE"
        assert call(good[0], t(I8, (3, 40)), good[2], pack) == "SHAPE"
        assert call(good[0], good[1], t(U8, (4, 1)), pack) == "SHAPE"
        assert call(t(BF16, (40,)), *good[1:], pack) == "INVALID_ARG"
        assert call(None, *good[1:], pack) == "INVALID_ARG"
        assert call(good[0], good[1], None, pack) == "INVALID_ARG"
        assert call(t(BF16, (4, 40), (1, 4)), *good[1:], pack) == "UNSUPPORTED"
        assert call(good[0], t(I8, (4, 40), (1, 4)), good[2], pack) == "UNSUPPORTED"
        assert call(t(BF16, (4, 40), (-40, 1)), *good[1:], pack) == "INVALID_ARG"
        assert call(t(BF16, (1 << 31, 32)), t(I8, (1 << 31, 32)), t(U8, (1 << 31, 1)), pack) == "UNSUPPORTED"
    # written rows that overlap
    assert call(t(BF16, (4, 40)), t(I8, (4, 40), (8, 1)), t(U8, (4, 2))) == "INVALID_ARG"
    assert call(t(BF16, (4, 40), (8, 1)), t(I8, (4, 40)), t(U8, (4, 2)), False) == "INVALID_ARG"


def test_weight_grad_argument_errors(trop):
    t = lambda *a, **k: _tensor(trop, *a, **k)  # noqa: E731

    def call(dy, codes, scales, dw):
        return trop.ERRORS.get(trop._lib.tropical_activation_weight_grad(*(ctypes.byref(d) for d in (dy, codes, scales, dw)), None, None))

    dy, k, s, dw = t(BF16, (6, 8)), t(I8, (6, 40)), t(U8, (6, 2)), t(BF16, (8, 40))
    assert call(t(F32, (6, 8)), k, s, dw) == "DTYPE"
    assert call(dy, t(U8, (6, 40)), s, dw) == "DTYPE"
    assert call(dy, k, s, t(F16, (8, 40))) == "DTYPE"
    assert call(t(BF16, (5, 8)), k, s, dw) == "SHAPE"
    assert call(dy, k, t(U8, (6, 1)), dw) == "SHAPE"
    assert call(dy, k, s, t(BF16, (40, 8))) == "SHAPE"
    assert call(dy, k, s, t(BF16, (8, 40), (1, 8))) == "UNSUPPORTED"
    assert call(dy, k, s, t(BF16, (8, 40), (20, 1))) == "INVALID_ARG"


def test_residual_norm_argument_errors(trop, block):
    t = lambda *a, **k: _tensor(trop, *a, **k)  # noqa: E731

    def call(x=(BF16, (4, 40)), u=(BF16, (4, 40)), y=(BF16, (4, 40)), r=None, gate=None, kept=None, **o):
        v = dict(norm=0, post_norm=1, gate_act=0, wdtype=BF16, alpha=1.0, scale=1.0, eps=1e-5) | o
        opt = block._Options(**v)
        at = lambda d: None if d is None else ctypes.byref(t(*d))  # noqa: E731
        return trop.ERRORS.get(trop._lib.tropical_residual_norm(ctypes.byref(opt), at(x), at(u), at(gate), at(y), at(r or x), None, kept, None))

    assert call(x=None, r=(BF16, (4, 40))) == "INVALID_ARG"
    assert call(x=(BF16, (40,))) == "INVALID_ARG"
    assert call(x=(F64, (4, 40))) == "DTYPE"
    assert call(u=(F16, (4, 40))) == "DTYPE"
    assert call(u=(F32, (4, 40))) == "DTYPE"
    assert call(y=(F32, (4, 40))) == "DTYPE"
    assert call(x=(F32, (4, 40)), y=(F16, (4, 40))) == "DTYPE"
    assert call(r=(F32, (4, 40))) == "DTYPE"
    assert call(u=(BF16, (4, 39))) == "SHAPE"
    assert call(y=(BF16, (5, 40))) == "SHAPE"
    assert call(r=(BF16, (5, 40))) == "SHAPE"
    assert call(*[(BF16, (4, 0))] * 3) == "SHAPE"
    assert call(*[(BF16, (1 << 31, 8))] * 3) == "UNSUPPORTED"
    assert call(x=(BF16, (4, 40), (1, 4)), r=(BF16, (4, 40))) == "UNSUPPORTED"
    assert call(r=(BF16, (4, 40), (20, 1))) == "INVALID_ARG"
    for bad in (dict(norm=2), dict(gate_act=3), dict(gate_act=-1), dict(eps=-1.0), dict(eps=math.nan), dict(alpha=math.inf),
                dict(scale=math.nan), dict(post_norm=0, post_weight=4096)):
        assert call(**bad) == "INVALID_ARG", bad
    assert call(weight=4096, wdtype=F16) == "DTYPE"
    assert call(gate=(BF16, (4, 2))) == "SHAPE"
    assert call(gate=(BF16, (3, 40))) == "SHAPE"
    assert call(gate=(F32, (4, 40))) == "DTYPE"
    pair = t(I8, (4, 40)), t(U8, (4, 2))
    assert call(kept=_kept(block, u=pair)) == "INVALID_ARG"
    assert call(kept=_kept(block, u=pair, gate=pair, r=pair)) == "INVALID_ARG"
    assert call(kept=_kept(block, u=pair, r=(t(I8, (4, 40)), t(U8, (4, 1))))) == "SHAPE"
    assert call(gate=(BF16, (4, 40)), kept=_kept(block, u=pair, r=pair)) == "INVALID_ARG"


def test_residual_norm_backward_argument_errors(trop, block):
    t = lambda *a, **k: _tensor(trop, *a, **k)  # noqa: E731
    like = (BF16, (4, 40))

    def call(dy=like, dr=None, r=like, u=like, gate=None, kept=None, grads=None, types=(BF16, BF16), **o):
        v = dict(norm=0, post_norm=1, gate_act=0, wdtype=BF16, alpha=1.0, scale=1.0, eps=0.0) | o
        at = lambda d: None if d is None else ctypes.byref(t(*d))  # noqa: E731
        g = block._Grads()
        for name, value in (grads or {}).items():
            setattr(g, name, ctypes.pointer(t(*value)) if isinstance(value, tuple) else value)
        opt = block._Options(**v)
        return trop.ERRORS.get(trop._lib.tropical_residual_norm_backward(ctypes.byref(opt), at(dy), at(dr), at(r), at(u), at(gate), 4096,
                                                                         kept, *types, ctypes.byref(g), None))

    pair = t(I8, (4, 40)), t(U8, (4, 2))
    copies = dict(r=None, u=None, kept=_kept(block, u=pair, r=pair))
    assert call(dy=(F32, (4, 40))) == "DTYPE"
    assert call(dr=(F32, (4, 40))) == "DTYPE"
    assert call(dr=(BF16, (4, 39))) == "SHAPE"
    assert call(r=None) == "INVALID_ARG"
    assert call(u=(BF16, (3, 40))) == "SHAPE"
    assert call(kept=_kept(block, u=pair, r=pair)) == "INVALID_ARG"
    assert call(**copies, types=(I32, BF16)) == "DTYPE"
    assert call(**copies, gate=(BF16, (4, 40))) == "INVALID_ARG"
    assert call(grads=dict(dx=(F32, (4, 40)))) == "DTYPE"
    assert call(grads=dict(du=(BF16, (4, 41)))) == "SHAPE"
    assert call(grads=dict(du=(BF16, (4, 40), (0, 1)))) == "INVALID_ARG"
    assert call(grads=dict(dgate=like)) == "INVALID_ARG"
    assert call(gate=(BF16, (4, 1)), grads=dict(dgate=like)) == "SHAPE"
    assert call(grads=dict(dscale=4096)) == "INVALID_ARG"
    assert call(post_norm=0, grads=dict(dpost_bias=4096)) == "INVALID_ARG"
    assert call(wdtype=F16, grads=dict(dweight=4096)) == "DTYPE"


def test_wrappers_refuse_host_tensors_and_wrong_words(trop):
    """Whatever the arguments, an error of the package's own kind."""
    x = torch.zeros(3, 8)

    def refused(f, *a, **k):
        with pytest.raises(trop.TropicalError) as e:
            f(*a, **k)
        return e.value.name

    assert refused(trop.residual_norm, x, x, norm="batch") == "INVALID_ARG"
    assert refused(trop.residual_norm, x, x, gate_act="relu") == "INVALID_ARG"
    assert refused(trop.residual_norm, torch.zeros(()), torch.zeros(())) == "INVALID_ARG"
    assert refused(trop.residual_norm, x, x[:2]) == "SHAPE"
    assert refused(trop.residual_norm, x, x, gate=torch.zeros(())) == "SHAPE"
    assert refused(trop.residual_norm, x, x, scale=torch.zeros(7)) == "SHAPE"
    st = torch.zeros(4, 3)
    assert refused(trop.residual_norm_backward, x, None, (x, x), x, st) == "INVALID_ARG"
    assert refused(trop.residual_norm_backward, x, None, x, x, st, gate=(x, x)) == "INVALID_ARG"
    assert refused(trop.residual_norm_backward, x, None, x, x, st, gate=torch.zeros(())) == "SHAPE"
    assert refused(trop.residual_norm_backward, x, None, x, x[:2], st) == "SHAPE"
    assert refused(trop.residual_norm_backward, torch.zeros(()), None, x, x, st) == "INVALID_ARG"
    assert refused(trop.activation_values, torch.zeros(3, 8, dtype=torch.int8), torch.zeros(())) == "INVALID_ARG"
    assert refused(trop.activation_weight_grad, x.bfloat16(), torch.zeros(3, 8, dtype=torch.int8), torch.zeros(())) == "INVALID_ARG"
    if not torch.cuda.is_available():  # (which stream the call would go to is asked first)
        return
    for f, a in ((trop.residual_norm, (x, x)), (trop.activation_pack, (x,)), (trop.residual_norm_backward, (x, None, x, x, st)),
                 (trop.activation_values, (torch.zeros(3, 8, dtype=torch.int8), torch.zeros(3, 1, dtype=torch.uint8)))):
        assert refused(f, *a) in ("HOST_POINTER", "CUDA", "DEVICE_MISMATCH")


@pytest.mark.parametrize("want", [("x", "weigth"), "post weight", ["dx"]])
def test_unknown_names_of_gradients_are_refused(trop, want):
    """A misspelt name would leave a gradient out in silence."""
    x = torch.zeros(3, 8)
    with pytest.raises(trop.TropicalError) as e:
        trop.residual_norm_backward(x, None, x, x, torch.zeros(4, 3), want=want)
    assert e.value.name == "INVALID_ARG" and "want" in str(e.value)


@pytest.mark.parametrize("lead, wrong", [((3,), (3, 4)), ((4,), (16,)), ((2, 6), (12, 4)), ((2, 6), (4, 6, 2)), ((3,), (4, 3, 1)), ((), (1, 4))])
def test_statistics_of_another_shape_are_refused(trop, lead, wrong):
    """As many elements in another order would be read as other rows' statistics."""
    x = torch.zeros(*lead, 8)
    with pytest.raises(trop.TropicalError) as e:
        trop.residual_norm_backward(x, None, x, x, torch.zeros(wrong))
    assert e.value.name == "SHAPE" and "stats" in str(e.value)


def test_statistics_and_gradients_start_on_an_element(trop, block):
    """As the vectors do: an address inside an element would be a misaligned access."""
    at = lambda *d: ctypes.byref(_tensor(trop, *d))  # noqa: E731
    like = (BF16, (4, 40))

    def forward(stats):
        o = block._Options(norm=0, post_norm=1, gate_act=0, wdtype=BF16, alpha=1.0, scale=1.0, eps=1e-5)
        return trop.ERRORS.get(trop._lib.tropical_residual_norm(ctypes.byref(o), at(*like), at(*like), None, at(*like), at(*like), stats, None, None))

    def backward(stats, wdtype, **grads):
        o = block._Options(norm=0, post_norm=1, gate_act=0, wdtype=wdtype, alpha=1.0, scale=1.0, eps=0.0, scale_vector=4096)
        g = block._Grads(**grads)
        return trop.ERRORS.get(trop._lib.tropical_residual_norm_backward(ctypes.byref(o), at(*like), None, at(*like), at(*like), None, stats, None,
                                                                         BF16, BF16, ctypes.byref(g), None))

    assert forward(4098) == "INVALID_ARG"
    assert backward(4098, BF16, dweight=4096) == "INVALID_ARG"
    for name in ("dscale", "dweight", "dbias", "dpost_weight", "dpost_bias"):
        assert backward(4096, BF16, **{name: 4097}) == "INVALID_ARG"
        assert backward(4096, F32, **{name: 4098}) == "INVALID_ARG"
