"""The residual block's operators at the borders of what they accept.

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
