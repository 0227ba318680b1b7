"""The residual block's operators at the borders of what they accept: matrices and vectors that start anywhere in a buffer,
few columns in many rows.

Limits as in test_gpu_residual_norm.py: a stored value is off by at most eps / 2 of its type relative to itself, sums in
32 bits lose less than 1e-5 of the terms that a result is the sum of."""

import pytest
import torch

from test_gpu_residual_norm import check, make

pytestmark = pytest.mark.gpu

F, B, H = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def trop():
    import einsum_device_side_gb300 as t
    t.load()
    return t


@pytest.mark.parametrize("S, U, Y", [(F, F, F), (B, B, B), (F, B, B), (F, F, H)])
@pytest.mark.parametrize("shift", [1, 2, 3, 5, 7])
def test_few_rows_from_any_element_on(trop, S, U, Y, shift):
    """Matrices that start anywhere between 16 bytes, of so few rows that most vectors reach over the matrix's own ends, which no
    copy may start from; rows with and without gaps between them."""
    for rows, cols, gap in ((1, 40, 0), (2, 33, 0), (3, 100, 4), (4, 1001, 0), (2, 8193, 7)):
        t, o = make(rows, cols, S, U, Y, gate_act="silu", seed=shift)
        for k in ("x", "u", "gate", "dy", "dr"):
            flat = torch.empty(shift + rows * (cols + gap), dtype=t[k].dtype, device="cuda")
            t[k] = flat.as_strided((rows, cols), (cols + gap, 1), shift).copy_(t[k])
        for keep in (False, True):
            check(trop, t, o, S, U, Y, keep)


def off16(v):
    """The same vector one element behind the start of a buffer."""
    to = torch.empty(v.numel() + 1, dtype=v.dtype, device=v.device)[1:]
    return to.copy_(v)


@pytest.mark.parametrize("name", ["weight", "bias", "post_weight", "post_bias", "scale"])
@pytest.mark.parametrize("S, U, Y, W", [(B, B, B, B), (H, H, H, H), (F, B, B, B), (F, B, B, F), (F, F, F, F), (F, F, B, B)])
def test_one_vector_off_16_bytes(trop, S, U, Y, W, name):
    """As a view of a flat buffer of parameters has it, the other vectors on 16 bytes: short rows, rows of one block and of a
    cluster, plain and from copies."""
    for rows, cols in ((90, 64), (40, 1024), (6, 4096), (3, 8192)):
        t, o = make(rows, cols, S, U, Y, W, gate_act="silu")
        t[name] = off16(t[name])
        assert t[name].data_ptr() % 16
        for keep in (False, True):
            check(trop, t, o, S, U, Y, keep)


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("dt", [F, B, H])
@pytest.mark.parametrize("cols", [1, 2, 3, 4, 5])
def test_few_columns_in_many_rows(trop, cols, dt, keep):
    """More rows than a grid's second dimension counts.  The column sums of up to 65535 blocks are joined by 32 warps, each a chain of
    1024 additions over sums of two (and one of 32): up to 1060 2^-24 = 6.3e-5 of the terms."""
    t, o = make(70001, cols, dt, dt, dt, norm="rms", gate_act="sigmoid")
    check(trop, t, o, dt, dt, dt, keep, lost=7e-5)
