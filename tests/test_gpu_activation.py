"""Activations in 8 bits: codes, scales and values bit for bit against the format's definition, computed on the host
with exact powers of two."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F, B, H = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def trop():
    import einsum_device_side_gb300 as t
    t.load()
    return t


def pack(x):
    """Codes and scales of a matrix by the definition, in 64 bits."""
    x = x.detach().cpu().double().numpy()
    rows, cols = x.shape
    groups = -(-cols // 32)
    blocks = np.zeros((rows, groups * 32))
    blocks[:, :cols] = x
    blocks = blocks.reshape(rows, groups, 32)
    bad = ~np.isfinite(blocks).all(2)
    top = np.where(bad[..., None], 0.0, np.abs(blocks)).max(2)
    _, power = np.frexp(top)  # top in [2^(power - 1), 2^power)
    scale = np.where(top > 0, power - 1 + 127, 0)
    scale = np.where(bad, 255, np.maximum(scale, 6)).astype(np.int64)
    with np.errstate(invalid="ignore"):
        codes = np.clip(np.rint(np.ldexp(blocks, (133 - scale)[..., None].astype(int))), -127, 127)
    codes = np.where(bad[..., None], 0, codes).reshape(rows, -1)[:, :cols]
    return torch.from_numpy(codes.astype(np.int8)), torch.from_numpy(scale.astype(np.uint8))


def values(codes, scales, dtype):
    codes, scales = codes.cpu().numpy().astype(np.float64), scales.cpu().numpy().astype(np.int64)
    each = np.repeat(scales, 32, axis=1)[:, :codes.shape[1]]
    v = np.where(each == 255, np.nan, np.ldexp(codes, (each - 133).astype(int)))
    return torch.from_numpy(v).to(dtype)


def same(a, b):
    a, b = a.cpu(), b.cpu()
    assert a.dtype == b.dtype and a.shape == b.shape
    assert torch.equal(torch.nan_to_num(a.double(), nan=1e300), torch.nan_to_num(b.double(), nan=1e300))


def check(trop, x, dtypes=(F, B, H)):
    codes, scales = trop.activation_pack(x)
    want, ws = pack(x.reshape(-1, x.shape[-1]))
    same(codes.reshape(want.shape), want)
    same(scales.reshape(ws.shape), ws)
    for dt in dtypes:
        got = trop.activation_values(codes, scales, dt)
        assert got.shape == x.shape
        same(got.reshape(want.shape), values(want, ws, dt))
    return codes, scales


def make(rows, cols, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(2 * torch.randn(cols, generator=g, device="cuda"))
    return x.to(dt)


@pytest.mark.parametrize("dt", [F, B, H])
@pytest.mark.parametrize("rows, cols", [(1, 1), (1, 31), (1, 32), (3, 33), (5, 64), (7, 100), (2, 1001), (513, 96), (40, 4096),
                                        (1300, 63), (3, 20001), (700, 1024)])
def test_codes_and_values(trop, rows, cols, dt):
    check(trop, make(rows, cols, dt))


@pytest.mark.parametrize("dt", [F, B, H])
@pytest.mark.parametrize("pad, shift", [(8, 0), (3, 0), (4, 1), (9, 5)])
def test_strided_rows(trop, dt, pad, shift):
    x = make(37, 200 + pad + shift, dt)[:, shift:shift + 200]
    codes, scales = check(trop, x)
    # codes and scales in rows of any pitch, and copies without gaps
    for cp, sp in ((201, 9), (232, 7), (200, 7)):
        c, s = torch.empty(37, cp, dtype=torch.int8, device="cuda"), torch.empty(37, sp, dtype=torch.uint8, device="cuda")
        c, s = c[:, :200], s[:, :7]
        c.copy_(codes)
        s.copy_(scales)
        same(trop.activation_values(c, s, dt), trop.activation_values(codes, scales, dt))


def test_leading_axes(trop):
    x = make(24, 96, B).view(2, 3, 4, 96)
    codes, scales = check(trop, x)
    assert codes.shape == x.shape and scales.shape == (2, 3, 4, 3)
    t = x.transpose(0, 2)  # axes that do not merge
    c2, s2 = trop.activation_pack(t)
    same(c2, codes.transpose(0, 2).contiguous())
    same(s2, scales.transpose(0, 2).contiguous())
    same(trop.activation_values(codes.transpose(0, 2), scales.transpose(0, 2), B), trop.activation_values(c2, s2, B))
    one = trop.activation_pack(x[0, 0, 0])
    assert one[0].shape == (96,) and one[1].shape == (3,)
    same(one[0], codes[0, 0, 0])


@pytest.mark.parametrize("shape", [(0, 40), (4, 0), (0, 0)])
def test_empty(trop, shape):
    x = torch.empty(shape, device="cuda")
    codes, scales = trop.activation_pack(x)
    assert codes.shape == x.shape and scales.shape == (shape[0], -(-shape[1] // 32))
    assert trop.activation_values(codes, scales, F).shape == x.shape


@pytest.mark.parametrize("dt", [F, B, H])
def test_extreme_groups(trop, dt):
    """Zeros, the smallest and largest numbers, ties, values that round up past 127 units, infinities and NaN."""
    info = torch.finfo(dt)
    rows = []
    for v in (0.0, info.tiny, info.smallest_normal / 8, info.max, 1.0, 127 / 128, 1.9921875, 2 - 2.0 ** -6):
        row = torch.linspace(-1, 1, 64, dtype=torch.float64) * v
        row[5] = v
        rows.append(row)
    rows.append(torch.arange(64).double() * 0.5 + 0.25)  # ties in the first group's unit of a half and beyond
    rows.append(torch.arange(64).double() - 0.5)
    for bad in (float("inf"), float("-inf"), float("nan")):
        row = torch.ones(64, dtype=torch.float64)
        row[40] = bad
        rows.append(row)
    x = torch.stack(rows).to(dt).cuda()
    check(trop, x)
    check(trop, x[:, :61])  # off the 16 bytes
    if dt == F:
        tiny = torch.full((2, 32), 2.0 ** -149, device="cuda")
        tiny[1] = 2.0 ** -121 * 1.5
        check(trop, tiny)


def test_error_bound(trop):
    """An element is off by at most 1/128 of its group's largest magnitude (under 127.5 units; there less than a unit, 1/64)."""
    x = make(500, 640, F)
    v = trop.activation_values(*trop.activation_pack(x), F)
    top = x.view(500, 20, 32).abs().amax(2, keepdim=True)
    off = (v.view(500, 20, 32) - x.view(500, 20, 32)).abs()
    near = x.view(500, 20, 32).abs() <= 127.5 * torch.exp2(torch.floor(torch.log2(top)) - 6)
    assert bool((off[near.expand_as(off)] <= (top / 128).expand_as(off)[near]).all()) and bool((off < top / 64).all())
    same(trop.activation_values(*trop.activation_pack(v), F), v)  # a top of 64 units keeps 64: the copy's copy is itself


def test_many_elements(trop):
    """Addresses past 2^31 bytes."""
    rows, cols = 70001, 32768
    x = torch.zeros(rows, cols, dtype=H, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    last = torch.randn(2, cols, generator=g, device="cuda").to(H)
    x[-2:] = last
    codes, scales = trop.activation_pack(x)
    want, ws = pack(last)
    same(codes[-2:], want)
    same(scales[-2:], ws)
    assert int(codes[:-2].abs().max()) == 0 and bool((scales[:-2] == 6).all())
    same(trop.activation_values(codes, scales, H)[-2:], values(want, ws, H))


def test_streams_and_graphs(trop):
    x = make(200, 333, B)
    codes, scales = trop.activation_pack(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c2, s2 = trop.activation_pack(x, stream=s)
    v2 = trop.activation_values(c2, s2, B, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    same(c2, codes)
    same(s2, scales)
    same(v2, trop.activation_values(codes, scales, B))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c3, s3 = trop.activation_pack(x)
        v3 = trop.activation_values(c3, s3, B)
    x.copy_(make(200, 333, B, seed=9))
    g.replay()
    want, ws = pack(x)
    same(c3, want)
    same(s3, ws)
    same(v3, values(want, ws, B))


def test_refusals(trop):
    x = make(4, 64, B)
    codes, scales = trop.activation_pack(x)

    def name(f, *a):
        with pytest.raises(trop.TropicalError) as e:
            f(*a)
        return e.value.name

    assert name(trop.activation_pack, x.double()) == "DTYPE"
    assert name(trop.activation_pack, x.t()) == "UNSUPPORTED"
    assert name(trop.activation_pack, x.cpu()) in ("HOST_POINTER", "INVALID_ARG")
    assert name(trop.activation_values, codes, scales[:, :1], B) == "SHAPE"
    assert name(trop.activation_values, codes, scales[:3], B) == "SHAPE"
    assert name(trop.activation_values, codes.to(torch.uint8), scales, B) == "DTYPE"
    assert name(trop.activation_values, codes, scales.to(torch.int8), B) == "DTYPE"
    assert name(trop.activation_values, codes, scales, torch.float64) == "DTYPE"
    assert name(trop.activation_values, codes, scales.cpu(), B) == "DEVICE_MISMATCH"


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cols", [16, 17, 31, 33, 100, 1001, 4097])
def test_values_of_ragged_rows_anywhere_in_memory(trop, cols, dt):
    """Results that start on any element, without gaps between their rows; nothing beside them is written."""
    from einsum_device_side_gb300 import train
    g = torch.Generator(device="cuda").manual_seed(cols)
    for rows, shift in ((2, 0), (3, 1), (257, 3), (64, 6), (1000, 7)):
        x = torch.randn(rows, cols, generator=g, device="cuda") * torch.rand(rows, 1, generator=g, device="cuda") * 50
        codes, scales = trop.activation_pack(x)
        if shift == 3:  # copies without gaps
            codes = codes.contiguous()
        scales[0, 0] = 255  # a group that is not finite
        units = torch.exp2(scales.double() - 133).repeat_interleave(32, 1)[:, :cols]
        units[0, :32] = float("nan")
        want = (codes.double() * units).to(dt)
        buf = torch.full((rows * cols + 24,), -3.0, dtype=dt, device="cuda")
        out = buf[8 + shift:8 + shift + rows * cols].view(rows, cols)
        assert trop._lib.tropical_activation_values(train._desc(codes), train._desc(scales), train._desc(out), None) == 0
        torch.cuda.synchronize()
        assert torch.equal(out.nan_to_num(nan=1e4), want.nan_to_num(nan=1e4))
        assert bool((buf[:8 + shift] == -3).all()) and bool((buf[8 + shift + rows * cols:] == -3).all())
