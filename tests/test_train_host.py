"""Host-side checks of the training operators' entry points: argument errors that are found before any
device work, the package's names, and the 8-bit codes' bounds from their definition.  No GPU."""

import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def trop():
    from einsum_device_side_gb300 import build
    build.build()
    import einsum_device_side_gb300 as t
    t.load()
    return t


F32, I32, I64, F64, BF16, F16 = range(6)


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
    return ctypes.byref(t)


def _norm(trop, x, y, wdtype=F32, w=None, b=None, eps=1e-5):
    return trop.ERRORS.get(trop._lib.tropical_layer_norm(x, w, b, wdtype, eps, y, None, None, None))


def test_layer_norm_argument_errors(trop):
    t = lambda *a, **k: _tensor(trop, *a, **k)  # noqa: E731
    assert _norm(trop, t(F64, (2, 8)), t(F64, (2, 8))) == "DTYPE"
    assert _norm(trop, t(BF16, (2, 8)), t(F32, (2, 8))) == "DTYPE"
    assert _norm(trop, t(BF16, (2, 8)), t(F16, (2, 8))) == "DTYPE"
    assert _norm(trop, t(BF16, (2, 8)), t(BF16, (2, 8)), wdtype=F16, w=4096) == "DTYPE"
    assert _norm(trop, t(F32, (2, 8)), t(F32, (2, 9))) == "SHAPE"
    assert _norm(trop, t(F32, (2, 0)), t(F32, (2, 0))) == "SHAPE"
    assert _norm(trop, t(F32, (8,)), t(F32, (8,))) == "INVALID_ARG"
    assert _norm(trop, t(F32, (2, 8)), t(F32, (2, 8)), eps=-1.0) == "INVALID_ARG"
    assert _norm(trop, t(F32, (2, 8)), t(F32, (2, 8)), eps=math.nan) == "INVALID_ARG"
    assert _norm(trop, t(F32, (2, 8), (1, 2)), t(F32, (2, 8))) == "UNSUPPORTED"
    assert _norm(trop, t(F32, (2, 8)), t(F32, (2, 8), (4, 1))) == "INVALID_ARG"  # rows of y overlap
    assert _norm(trop, t(F32, (1 << 31, 8)), t(F32, (1 << 31, 8))) == "UNSUPPORTED"
    assert _norm(trop, None, t(F32, (2, 8))) == "INVALID_ARG"


def test_linear_cross_entropy_argument_errors(trop):
    t = lambda *a, **k: _tensor(trop, *a, **k)  # noqa: E731

    def call(x, w, target):
        rc = trop._lib.tropical_linear_cross_entropy(x, w, target, -100, 1, None, 4096, None, None, None)
        return trop.ERRORS.get(rc)

    good = t(BF16, (4, 16)), t(BF16, (32, 16)), t(I64, (4,))
    assert call(t(F32, (4, 16)), t(F32, (32, 16)), good[2]) == "DTYPE"
    assert call(good[0], t(F16, (32, 16)), good[2]) == "DTYPE"
    assert call(good[0], good[1], t(F32, (4,))) == "DTYPE"
    assert call(good[0], t(BF16, (32, 8)), good[2]) == "SHAPE"
    assert call(good[0], good[1], t(I64, (5,))) == "SHAPE"
    assert call(good[0], t(BF16, (0, 16)), good[2]) == "SHAPE"
    assert call(t(BF16, (4, 0)), t(BF16, (32, 0)), good[2]) == "SHAPE"
    assert call(good[0], good[1], t(I64, (4, 1))) == "INVALID_ARG"
    assert call(t(BF16, (1 << 31, 16)), good[1], t(I64, (1 << 31,))) == "UNSUPPORTED"
    rc = trop._lib.tropical_linear_cross_entropy(*good, -100, 1, None, None, None, None, None)
    assert trop.ERRORS.get(rc) == "INVALID_ARG"  # nowhere to put the log-sum-exp


def test_linear_cross_entropy_backward_argument_errors(trop):
    t = lambda *a, **k: _tensor(trop, *a, **k)  # noqa: E731
    x, w, target = t(BF16, (4, 16)), t(BF16, (32, 16)), t(I64, (4,))

    def call(dx, dw):
        rc = trop._lib.tropical_linear_cross_entropy_backward(4096, 1, x, w, target, -100, 4096, None, dx, dw, None)
        return trop.ERRORS.get(rc, rc)

    assert call(None, None) == 0  # nothing wanted
    assert call(t(F32, (4, 16)), None) == "DTYPE"
    assert call(t(BF16, (4, 8)), None) == "SHAPE"
    assert call(None, t(BF16, (32, 16), (1, 32))) == "UNSUPPORTED"
    assert call(None, t(BF16, (32, 16), (8, 1))) == "INVALID_ARG"


def test_adamw_argument_errors(trop):
    from einsum_device_side_gb300.train import _Options, _Tensor
    table = (_Tensor * 1)()

    def call(p=F32, g=F32, bits=32, n=0, tensors=table, **options):
        o = _Options(**{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0, step=1), **options})
        return trop.ERRORS.get(trop._lib.tropical_adamw_step(n, tensors, p, g, bits, 0, ctypes.byref(o), None))

    assert call(p=I32) == "DTYPE" and call(g=F64) == "DTYPE" and call(p=BF16, g=F16) == "DTYPE"
    assert call(bits=16) == "INVALID_ARG" and call(n=-1) == "INVALID_ARG" and call(n=1, tensors=None) == "INVALID_ARG"
    for bad in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(lr=math.inf), dict(grad_scale=math.nan)):
        assert call(**bad) == "INVALID_ARG", bad
    plan = ctypes.c_void_p()
    assert trop.ERRORS.get(trop._lib.tropical_adamw_plan_create(0, None, F32, F32, 16, 0, None, ctypes.byref(plan))) == "INVALID_ARG"
    assert plan.value is None
    assert trop.ERRORS.get(trop._lib.tropical_adamw_plan_step(None, None, None)) == "INVALID_ARG"
    assert trop._lib.tropical_adamw_plan_destroy(None) == 0


def test_tropical_operations_refuse_the_16_bit_types(trop):
    x, y = _tensor(trop, BF16, (2, 3)), _tensor(trop, BF16, (3, 2))
    assert trop.ERRORS.get(trop._lib.tropical_permute_trace(x, b"ij->ji", 0, y, None, None)) == "DTYPE"


@pytest.mark.parametrize("levels", [127, 255])
def test_square_law_codes_bound_their_error(levels):
    """c = round(levels sqrt(u)) stands for (c / levels)^2: off by at most sqrt(u) / levels + 1 / (4 levels^2)."""
    for i in range(100001):
        u = i / 100000
        c = round(levels * math.sqrt(u))
        assert abs((c / levels) ** 2 - u) <= math.sqrt(u) / levels + 0.25 / levels ** 2 + 1e-12
