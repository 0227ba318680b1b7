"""The training operators against plain implementations in 64 bits: layer norm, the linear head's cross
entropy and AdamW, forward and backward, at the sizes, strides and masks where they can go wrong.

Tolerances (fixed from the formats, u = 2^-24 for f32):
 * f32 results of n-term f32 sums: each of the few roundings per term costs u relative to the terms' magnitudes, and
   blocked sums of random terms grow slower than sqrt(n) u; 32 u of the terms' root mean square (times sqrt(n) for a
   sum) covers the sizes here with a margin of several.
 * a value rounded once to bf16 (f16) is off by at most 2^-8 (2^-11) relative, beside its f32 error.
 * logits on the tensor cores: f32 accumulation that may drop the bits below the accumulator's last place, one
   place per 16 products: D / 16 * 2^-23 of sqrt(sum of the squared terms' magnitudes) at most.
 * dx and dw: P is rounded to the operands' type for the products (2^-9 or 2^-12 relative per entry, in the mean), and
   so is the result: 2^-7 (2^-10) in the 2-norm has a margin of two over both together.
 * AdamW is compared bit for bit with the same chain of f32 operations, and in the 2-norm with 64 bits.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F, B, H = torch.float32, torch.bfloat16, torch.float16
U = 2.0 ** -24
ROUND = {F: 0.0, B: 2.0 ** -8, H: 2.0 ** -11}


@pytest.fixture(scope="module")
def trop():
    import einsum_device_side_gb300 as t
    t.load()
    return t


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(seed, *shape):
    return torch.randn(*shape, generator=_gen(seed), device="cuda")


def _close(got, want, dtype, slack):
    """Every entry within its rounding to dtype, and `slack` (an absolute f32 error, a tensor or number)."""
    assert got.dtype == dtype and got.shape == want.shape
    err = (got.double() - want).abs()
    limit = want.abs() * ROUND[dtype] + slack + (2.0 ** -25 if dtype == H else 0.0)
    assert bool((err <= limit).all()), f"worst {float((err - limit).max())} over its limit"


def _norm(got, want):
    return float((got.double() - want).norm() / want.norm().clamp(min=1e-300))


# ------------------------------------------------------------------ layer norm


def _norm_case(rows, cols, dt, seed, offset=1.0):
    x = (2 * _normal(seed, rows, cols) + offset).to(dt)
    return x, _normal(seed + 1, cols), _normal(seed + 2, cols), _normal(seed + 3, rows, cols)


def _norm_plain(x, w, b, eps):
    x = x.double()
    mu = x.mean(1, keepdim=True)
    sd = (x - mu).square().mean(1, keepdim=True).add(eps).sqrt()
    z = (x - mu) / sd
    y = z * w.double() if w is not None else z
    return (y + b.double() if b is not None else y), mu[:, 0], 1 / sd[:, 0], z


def _norm_plain_back(dy, z, rstd, w):
    dy = dy.double()
    u = dy * w.double() if w is not None else dy
    dx = rstd[:, None] * (u - u.mean(1, keepdim=True) - z * (u * z).mean(1, keepdim=True))
    return dx, (dy * z).sum(0), dy.sum(0)


NORM_SIZES = [(1, 1), (1, 2), (2, 7), (5, 32), (9, 33), (130, 128), (3, 255), (70, 256), (33, 1000), (41, 1001),
              (17, 2048), (5, 4095), (6, 8192), (3, 12288), (3, 16384), (2, 16385), (2, 40000), (4000, 64), (1500, 96)]


@pytest.mark.parametrize("dt", [F, B, H])
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
def test_layer_norm_both_directions(trop, rows, cols, dt):
    x, w, b, dy = _norm_case(rows, cols, dt, rows + cols)
    w, b, dy = w.to(dt), b.to(dt), dy.to(dt)
    y, mean, rstd = trop.layer_norm(x, w, b, eps=1e-5)
    wy, wm, wr, z = _norm_plain(x, w, b, 1e-5)
    # the mean's error moves every centred value; its effect on y is over the row's deviation
    shift = 32 * U * (x.double().abs().amax(1, keepdim=True))
    assert bool(((mean.double() - wm).abs() <= shift[:, 0]).all())
    slack = (shift * wr[:, None] + 32 * U * (z.abs() + 1)) * (w.double().abs() + 1) + 32 * U * b.double().abs()
    _close(y, wy, dt, slack)
    assert _norm(rstd, wr) <= 32 * U or cols == 1
    dx, dw, db = trop.layer_norm_backward(dy, x, mean, rstd, w)
    # (the backward's inputs are the statistics given)
    z = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    wx, ww, wb = _norm_plain_back(dy, z, rstd.double(), w)
    u = (dy.double() * w.double()).abs()
    slack = 32 * U * rstd.double()[:, None] * (u + u.mean(1, keepdim=True) + z.abs() * (u * z.abs()).mean(1, keepdim=True))
    _close(dx, wx, dt, slack)
    _close(dw, ww, dt, 32 * U * (dy.double() * z).abs().sum(0))
    _close(db, wb, dt, 32 * U * dy.double().abs().sum(0))


# many rows of which most start off the 16-byte granules: every offset, a row of one vector, and the widths
# around each change of the kernels' shapes
OFF_SIZES = [(2500, 3), (2477, 33), (2600, 129), (2433, 257), (2700, 510), (2600, 1001), (2440, 4093), (2433, 8189),
             (1300, 2047), (1250, 4097), (1217, 16375), (19500, 1001)]


@pytest.mark.parametrize("dt", [F, B, H])
@pytest.mark.parametrize("rows,cols", OFF_SIZES)
def test_layer_norm_of_many_rows_off_the_granules(trop, rows, cols, dt):
    test_layer_norm_both_directions(trop, rows, cols, dt)


@pytest.mark.parametrize("dt", [F, B])
@pytest.mark.parametrize("cols,pad", [(64, 1), (100, 3), (200, 7), (96, 4)])
def test_layer_norm_of_many_strided_rows_off_the_granules(trop, cols, pad, dt):
    rows = 2500
    wide, w, b, dy = _norm_case(rows, cols + pad, dt, cols + pad)
    w, b = w[:cols], b[:cols]
    x, dy = wide[:, pad:], dy.to(dt)[:, pad:]
    y, mean, rstd = trop.layer_norm(x, w, b)
    wy, _, _, _ = _norm_plain(x, w, b, 1e-5)
    _close(y, wy, dt, 64 * U * (x.double().abs().amax(1, keepdim=True) + 4) * (w.double().abs() + 1) + 64 * U * b.double().abs())
    dx, dw, db = trop.layer_norm_backward(dy, x, mean, rstd, w)
    z = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    wx, ww, wb = _norm_plain_back(dy, z, rstd.double(), w)
    assert _norm(dx, wx) <= max(ROUND[dt], 64 * U) and _norm(dw, ww) <= 64 * U and _norm(db, wb) <= 64 * U


@pytest.mark.parametrize("ydt", [B, H])
def test_layer_norm_of_f32_gives_16_bits(trop, ydt):
    x, w, b, dy = _norm_case(37, 520, F, 5)
    y, mean, rstd = trop.layer_norm(x, w, b, out_dtype=ydt)
    wy, _, wr, z = _norm_plain(x, w, b, 1e-5)
    _close(y, wy, ydt, 64 * U * (z.abs() + 4) * (w.double().abs() + 1))
    dx, dw, db = trop.layer_norm_backward(dy.to(ydt), x, mean, rstd, w)
    wx, ww, wb = _norm_plain_back(dy.to(ydt), z, wr, w)
    assert dx.dtype == dw.dtype == db.dtype == F
    assert max(_norm(dx, wx), _norm(dw, ww), _norm(db, wb)) <= 64 * U


@pytest.mark.parametrize("dt", [B, H])
@pytest.mark.parametrize("cols", [96, 97])
def test_layer_norm_f32_weights_of_16_bit_rows(trop, dt, cols):
    x, w, b, dy = _norm_case(50, cols, dt, 9)
    y, mean, rstd = trop.layer_norm(x, w, b)
    wy, _, wr, z = _norm_plain(x, w, b, 1e-5)
    _close(y, wy, dt, 64 * U * (z.abs() + 4) * (w.double().abs() + 1))
    dx, dw, db = trop.layer_norm_backward(dy.to(dt), x, mean, rstd, w)
    wx, ww, wb = _norm_plain_back(dy.to(dt), z, wr, w)
    assert dw.dtype == db.dtype == F and _norm(dw, ww) <= 64 * U and _norm(db, wb) <= 64 * U
    assert _norm(dx, wx) <= ROUND[dt]


@pytest.mark.parametrize("has_w,has_b", [(False, False), (True, False), (False, True)])
def test_layer_norm_without_weight_or_bias(trop, has_w, has_b):
    x, w, b, dy = _norm_case(20, 132, F, 3)
    w, b = w if has_w else None, b if has_b else None
    y, mean, rstd = trop.layer_norm(x, w, b)
    wy, _, wr, z = _norm_plain(x, w, b, 1e-5)
    assert _norm(y, wy) <= 64 * U
    dx, dw, db = trop.layer_norm_backward(dy, x, mean, rstd, w)
    for g, e in zip((dx, dw, db), _norm_plain_back(dy, z, wr, w)):
        assert _norm(g, e) <= 64 * U


@pytest.mark.parametrize("cols", [64, 65])
def test_layer_norm_strided_rows_leading_axes_and_views(trop, cols):
    big = _normal(1, 6, 7, cols + 5)
    x = big[:, :, 3:3 + cols]  # rows of another pitch, off the vectors' alignment
    y, mean, rstd = trop.layer_norm(x)
    assert y.shape == x.shape and mean.shape == (6, 7)
    want = _norm_plain(x.reshape(-1, cols), None, None, 1e-5)[0]
    assert _norm(y.reshape(-1, cols), want) <= 64 * U
    same = x[0, :1].expand(5, cols)  # one row read five times
    y5, m5, r5 = trop.layer_norm(same)
    assert bool((y5 == y5[0]).all()) and bool((y5[0] == y[0, 0]).all())
    out = torch.full((6, 7, cols), 7.0, device="cuda")
    assert trop.layer_norm(x, out=out)[0] is out and bool((out == y).all())
    dx, dw, db = trop.layer_norm_backward(y, x, mean, rstd)
    assert dx.shape == x.shape


def test_layer_norm_constant_rows_large_means_and_non_finite_rows(trop):
    x = torch.full((4, 300), 5.0, device="cuda")
    x[1] = 1e4 + torch.arange(300, device="cuda") * 2.0 ** -6  # a mean far above the deviation
    x[2, 7] = float("inf")
    x[3, 9] = float("nan")
    y, mean, rstd = trop.layer_norm(x)
    assert bool((y[0] == 0).all())
    want = _norm_plain(x[1:2], None, None, 1e-5)[0]
    # the row's f32 values carry a mean known to u * 1e4, against a deviation of about 1.35
    assert float((y[1].double() - want[0]).abs().max()) <= 32 * U * 1e4 / 1.35
    assert bool(y[2].isnan().any()) and bool(y[3].isnan().all()) and bool(y[0].isfinite().all())


def test_layer_norm_gradient_against_differences(trop):
    x, w, b, dy = _norm_case(3, 40, F, 11)
    _, mean, rstd = trop.layer_norm(x, w, b)
    dx, dw, db = trop.layer_norm_backward(dy, x, mean, rstd, w)
    f = lambda x, w, b: float((_norm_plain(x, w, b, 1e-5)[0] * dy.double()).sum())  # noqa: E731
    for t, g in ((x, dx), (w, dw), (b, db)):
        d = torch.randn(t.shape, generator=_gen(2), device="cuda", dtype=torch.float64)
        args = [a.double() for a in (x, w, b)]
        at = [i for i, a in enumerate((x, w, b)) if a is t][0]
        hi, lo = list(args), list(args)
        hi[at], lo[at] = args[at] + 1e-5 * d, args[at] - 1e-5 * d
        slope = (f(*hi) - f(*lo)) / 2e-5
        want = float((g.double() * d).sum())
        assert abs(slope - want) <= 1e-5 * float((g.double() * d).abs().sum()) + 1e-7


def test_layer_norm_one_gradient_at_a_time_and_no_rows(trop):
    x, w, b, dy = _norm_case(40, 72, F, 4)
    _, mean, rstd = trop.layer_norm(x, w, b)
    every = trop.layer_norm_backward(dy, x, mean, rstd, w)
    for i, k in enumerate(("want_x", "want_weight", "want_bias")):
        want = {n: n == k for n in ("want_x", "want_weight", "want_bias")}
        one = trop.layer_norm_backward(dy, x, mean, rstd, w, **want)
        assert [t is not None for t in one] == [j == i for j in range(3)]
        assert torch.equal(one[i], every[i])
    e = x[:0]
    y, mean, rstd = trop.layer_norm(e, w, b)
    assert y.shape == (0, 72)
    dx, dw, db = trop.layer_norm_backward(e, e, mean, rstd, w)
    assert dx.shape == (0, 72) and not bool(dw.any()) and not bool(db.any())


def test_layer_norm_refusals(trop):
    x, w, b, dy = _norm_case(4, 16, F, 1)

    def refused(name, f):
        with pytest.raises(trop.TropicalError) as e:
            f()
        assert e.value.name == name

    refused("DTYPE", lambda: trop.layer_norm(x.double()))
    refused("DTYPE", lambda: trop.layer_norm(x.to(B), out_dtype=F))
    refused("DTYPE", lambda: trop.layer_norm(x, w.to(B)))
    refused("DTYPE", lambda: trop.layer_norm(x, w, b.to(B)))
    refused("SHAPE", lambda: trop.layer_norm(x, w[:8]))
    refused("SHAPE", lambda: trop.layer_norm(x[:, :0]))
    refused("SHAPE", lambda: trop.layer_norm(x, out=torch.empty(4, 15, device="cuda")))
    refused("UNSUPPORTED", lambda: trop.layer_norm(x.T.contiguous().T))
    refused("INVALID_ARG", lambda: trop.layer_norm(x, eps=-1.0))
    refused("DEVICE_MISMATCH", lambda: trop.layer_norm(x, w.cpu()))
    refused("HOST_POINTER", lambda: trop.layer_norm(x.cpu(), out=x.cpu()))
    _, mean, rstd = trop.layer_norm(x)
    refused("DTYPE", lambda: trop.layer_norm_backward(dy.to(torch.int32), x, mean, rstd))
    refused("SHAPE", lambda: trop.layer_norm_backward(dy[:2], x, mean, rstd))
    refused("SHAPE", lambda: trop.layer_norm_backward(dy, x, mean[:2], rstd))


# ------------------------------------------------------------------ cross entropy of a linear head

IGNORE = -100


def _head(n, d, v, dt, seed, spread=2.0, drop=0.1):
    x = _normal(seed, n, d).to(dt)
    w = (_normal(seed + 1, v, d) * (spread / math.sqrt(d))).to(dt)
    t = torch.randint(0, v, (n,), generator=_gen(seed + 2), device="cuda")
    t[torch.rand(n, generator=_gen(seed + 3), device="cuda") < drop] = IGNORE
    return x, w, t


def _head_plain(x, w, t):
    l = x.double() @ w.double().T
    lse = torch.logsumexp(l, 1)
    k = t != IGNORE
    at = l.gather(1, torch.where(k, t, 0).long()[:, None])[:, 0]
    return torch.where(k, lse - at, 0.0), lse, k, l


def _head_plain_back(g, x, w, t, l, lse, k):
    p = torch.exp(l - lse[:, None])
    p.scatter_add_(1, torch.where(k, t, 0).long()[:, None], torch.full((len(t), 1), -1.0, device="cuda", dtype=torch.float64))
    p = torch.where(k, g.double(), 0.0)[:, None] * p
    return p @ w.double(), p.T @ x.double()


def _logit_error(x, w):
    """The largest error of a logit: one last place per 16 products, of the terms' summed magnitude at most."""
    d = x.shape[1]
    size = float(x.double().norm(dim=1).max() * w.double().norm(dim=1).max())
    return (d / 16 + 4) * 2.0 ** -23 * size / math.sqrt(max(1.0, d / 64))


HEAD_SIZES = [(1, 8, 1), (1, 8, 2), (1, 64, 300), (2, 7, 5), (4, 64, 256), (127, 64, 255), (128, 72, 256), (129, 100, 257),
              (255, 8, 513), (256, 256, 256), (257, 65, 1000), (300, 513, 77), (33, 1000, 2049), (600, 40, 5003), (16, 2048, 4096),
              (37, 1031, 515), (140, 2049, 300),  # (long rows at every offset)
              (2100, 72, 300), (1999, 65, 130)]  # (dw's tokens split)


@pytest.mark.parametrize("dt", [B, H])
@pytest.mark.parametrize("n,d,v", HEAD_SIZES)
def test_head_both_directions(trop, n, d, v, dt):
    x, w, t = _head(n, d, v, dt, n + d + v)
    loss, lse, kept = trop.linear_cross_entropy(x, w, t, "none")
    want, wlse, k, l = _head_plain(x, w, t)
    e = _logit_error(x, w) + 16 * U * float(wlse.abs().max())
    assert float((lse.double() - wlse).abs().max()) <= e
    assert float((loss.double() - want).abs().max()) <= 2 * e
    assert int(kept) == int(k.sum()) and not bool(loss[~k].any())
    g = torch.rand(n, generator=_gen(8), device="cuda") + 0.5
    dx, dw = trop.linear_cross_entropy_backward(g, x, w, t, lse)
    assert dx.dtype == dw.dtype == dt
    wx, ww = _head_plain_back(g, x, w, t, l, lse.double(), k)
    for got, exact in ((dx, wx), (dw, ww)):
        # the floor: entries that cancel (a vocabulary of one) leave errors of the logits only
        floor = e * float(g.max()) * float(max(x.double().abs().max(), w.double().abs().max())) * math.sqrt(got.numel())
        assert float((got.double() - exact).norm()) <= 2 * ROUND[dt] * float(exact.norm()) + floor
    assert not bool(dx[~k].any())


@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_head_reductions_and_scalar_gradient(trop, reduction):
    x, w, t = _head(700, 96, 1500, B, 21)
    each, lse0, kept0 = trop.linear_cross_entropy(x, w, t, "none")
    loss, lse, kept = trop.linear_cross_entropy(x, w, t, reduction)
    assert torch.equal(lse, lse0) and float(kept) == float(kept0) == int((t != IGNORE).sum())
    want = each.double().sum() / (float(kept) if reduction == "mean" else 1)
    assert abs(float(loss) - float(want)) <= 32 * U * float(want)
    mean = reduction == "mean"
    one = torch.tensor(3.0, device="cuda")
    dx, dw = trop.linear_cross_entropy_backward(one, x, w, t, lse, kept if mean else None)
    flat = torch.full((700,), 3.0 / float(kept) if mean else 3.0, device="cuda")
    ex, ew = trop.linear_cross_entropy_backward(flat, x, w, t, lse)
    assert _norm(dx, ex.double()) <= 2.0 ** -8 and _norm(dw, ew.double()) <= 2.0 ** -8


def test_head_int32_targets_strides_and_broadcasts(trop):
    x, w, t = _head(50, 48, 300, B, 2)
    loss, lse, _ = trop.linear_cross_entropy(x, w, t, "none")
    dx, dw = trop.linear_cross_entropy_backward(loss + 1, x, w, t, lse)

    def again(x2, w2, t2):
        l2, s2, _ = trop.linear_cross_entropy(x2, w2, t2, "none")
        assert torch.equal(l2, loss) and torch.equal(s2, lse)
        dx2, dw2 = trop.linear_cross_entropy_backward(loss + 1, x2, w2, t2, s2)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)

    again(x, w, t.int())
    again(x, w, torch.stack([t, t], 1)[:, 0])  # strided targets
    again(x.T.contiguous().T, w, t)            # column-major tokens
    again(x, w.T.contiguous().T, t)            # the head stored [D, V]
    wide = torch.zeros(50, 64, device="cuda", dtype=B)
    wide[:, 3:51] = x
    again(wide[:, 3:51], w, t)                 # rows off the 16-byte boundaries
    rows = torch.zeros(100, 48, device="cuda", dtype=B)
    rows[::2] = x
    again(rows[::2], w, t)
    one = x[:1].expand(50, 48)                 # one token read fifty times
    l1 = trop.linear_cross_entropy(one, w, t, "none")[1]
    assert bool((l1 == l1[0]).all()) and bool(l1[0] == lse[0])


def test_head_all_ignored_bad_targets_and_no_tokens(trop):
    x, w, t = _head(40, 64, 100, B, 6, drop=0.0)
    none = torch.full_like(t, IGNORE)
    loss, lse, kept = trop.linear_cross_entropy(x, w, none)
    assert bool(loss.isnan()) and float(kept) == 0
    dx, dw = trop.linear_cross_entropy_backward(torch.ones((), device="cuda"), x, w, none, lse, kept)
    assert not bool(dx.any()) and not bool(dw.any())
    assert float(trop.linear_cross_entropy(x, w, none, "sum")[0]) == 0
    bad = t.clone()
    bad[3], bad[5] = 100, -1
    loss, lse, kept = trop.linear_cross_entropy(x, w, bad, "none")
    assert loss.isnan().nonzero()[:, 0].tolist() == [3, 5] and float(kept) == 40
    dx, _ = trop.linear_cross_entropy_backward(torch.ones(40, device="cuda"), x, w, bad, lse)
    assert dx.isnan().any(1).nonzero()[:, 0].tolist() == [3, 5]
    t7 = t.clone()
    t7[2] = 7
    loss7 = trop.linear_cross_entropy(x, w, t7, "none", ignore_index=7)[0]
    assert float(loss7[2]) == 0
    e = x[:0]
    loss, lse, kept = trop.linear_cross_entropy(e, w, t[:0], "sum")
    assert float(loss) == 0 and float(kept) == 0 and lse.shape == (0,)
    assert bool(trop.linear_cross_entropy(e, w, t[:0])[0].isnan())
    dx, dw = trop.linear_cross_entropy_backward(torch.ones((), device="cuda"), e, w, t[:0], lse)
    assert dx.shape == (0, 64) and not bool(dw.any())


def test_head_large_logits_and_non_finite_rows(trop):
    x, w, t = _head(64, 64, 600, B, 12, spread=60.0, drop=0.0)  # logits in the hundreds
    loss, lse, _ = trop.linear_cross_entropy(x, w, t, "none")
    want, wlse, _, _ = _head_plain(x, w, t)
    e = _logit_error(x, w) + 16 * U * float(wlse.abs().max())
    assert float((lse.double() - wlse).abs().max()) <= e and float((loss.double() - want).abs().max()) <= 2 * e
    x[4, 5] = float("nan")
    _, lse2, _ = trop.linear_cross_entropy(x, w, t, "none")
    assert bool(lse2[4].isnan())
    keep = torch.arange(64, device="cuda") != 4
    assert torch.equal(lse2[keep], lse[keep])
    x[4] = 0  # a token of zeros: equal logits
    _, lse3, _ = trop.linear_cross_entropy(x, w, t, "none")
    assert abs(float(lse3[4]) - math.log(600)) <= 8 * U * math.log(600)


def test_head_several_pieces_of_the_vocabulary(trop):
    """More columns than one piece of the backward's workspace holds (2^28 entries of P)."""
    n, d, v = 30000, 16, 20001
    x, w, t = _head(n, d, v, B, 31)
    loss, lse, kept = trop.linear_cross_entropy(x, w, t, "mean")
    dx, dw = trop.linear_cross_entropy_backward(torch.ones((), device="cuda"), x, w, t, lse, kept)
    k = t != IGNORE
    wx = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    ww = torch.zeros(v, d, dtype=torch.float64, device="cuda")
    g = torch.ones(n, device="cuda") / float(kept)
    for a in range(0, n, 3000):
        r = slice(a, a + 3000)
        l = x[r].double() @ w.double().T
        assert float((torch.logsumexp(l, 1) - lse[r].double()).abs().max()) <= 1e-4
        px, pw = _head_plain_back(g[r], x[r], w, t[r], l, lse[r].double(), k[r])
        wx[r] = px
        ww += pw
    assert _norm(dx, wx) <= 2 * ROUND[B] and _norm(dw, ww) <= 2 * ROUND[B]


def test_head_one_gradient_at_a_time_and_repeats(trop):
    x, w, t = _head(300, 200, 3000, H, 17)
    _, lse, kept = trop.linear_cross_entropy(x, w, t)
    one = torch.ones((), device="cuda") * 64
    dx, dw = trop.linear_cross_entropy_backward(one, x, w, t, lse, kept)
    assert torch.equal(trop.linear_cross_entropy_backward(one, x, w, t, lse, kept, want_w=False)[0], dx)
    assert torch.equal(trop.linear_cross_entropy_backward(one, x, w, t, lse, kept, want_x=False)[1], dw)
    for _ in range(3):
        again = trop.linear_cross_entropy_backward(one, x, w, t, lse, kept)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
        assert torch.equal(trop.linear_cross_entropy(x, w, t)[1], lse)


def test_head_small_probabilities_survive_half_precision(trop):
    """A mean over many tokens makes P's entries far smaller than f16 resolves; the stored P is scaled."""
    x, w, t = _head(2000, 64, 4000, H, 19, spread=1.0, drop=0.0)
    _, lse, kept = trop.linear_cross_entropy(x, w, t)
    scale = torch.tensor(2.0 ** 14, device="cuda")  # the loss scale that keeps dw itself in f16's range
    dx, dw = trop.linear_cross_entropy_backward(scale, x, w, t, lse, kept)
    _, _, k, l = _head_plain(x, w, t)
    g = torch.full((2000,), 2.0 ** 14 / 2000, device="cuda")
    wx, ww = _head_plain_back(g, x, w, t, l, lse.double(), k)
    assert _norm(dx, wx) <= 2 * ROUND[H] and _norm(dw, ww) <= 2 * ROUND[H]


def test_head_gradient_against_differences(trop):
    x, w, t = _head(12, 24, 50, B, 23)
    loss, lse, kept = trop.linear_cross_entropy(x, w, t)
    dx, dw = trop.linear_cross_entropy_backward(torch.ones((), device="cuda"), x, w, t, lse, kept)
    f = lambda x, w: float(_head_plain(x, w, t)[0].sum() / float(kept))  # noqa: E731
    for at, g in ((0, dx), (1, dw)):
        args = [x.double(), w.double()]
        d = g.double() / g.double().norm()  # along the gradient itself
        hi, lo = list(args), list(args)
        hi[at], lo[at] = args[at] + 1e-4 * d, args[at] - 1e-4 * d
        slope = (f(*hi) - f(*lo)) / 2e-4
        assert abs(slope - float(g.double().norm())) <= 2.0 ** -7 * float(g.double().norm())


def test_head_refusals(trop):
    x, w, t = _head(8, 32, 64, B, 1)

    def refused(name, f):
        with pytest.raises(trop.TropicalError) as e:
            f()
        assert e.value.name == name

    refused("DTYPE", lambda: trop.linear_cross_entropy(x.float(), w.float(), t))
    refused("DTYPE", lambda: trop.linear_cross_entropy(x, w.to(H), t))
    refused("DTYPE", lambda: trop.linear_cross_entropy(x, w, t.float()))
    refused("SHAPE", lambda: trop.linear_cross_entropy(x, w[:, :16], t))
    refused("SHAPE", lambda: trop.linear_cross_entropy(x, w, t[:4]))
    refused("SHAPE", lambda: trop.linear_cross_entropy(x, w[:0], t))
    refused("SHAPE", lambda: trop.linear_cross_entropy(x[:, :0], w[:, :0], t))
    refused("INVALID_ARG", lambda: trop.linear_cross_entropy(x[0], w, t))
    refused("INVALID_ARG", lambda: trop.linear_cross_entropy(x, w, t, "max"))
    refused("DEVICE_MISMATCH", lambda: trop.linear_cross_entropy(x, w.cpu(), t))
    _, lse, kept = trop.linear_cross_entropy(x, w, t)
    one = torch.ones(8, device="cuda")
    refused("DTYPE", lambda: trop.linear_cross_entropy_backward(one.double(), x, w, t, lse))
    refused("SHAPE", lambda: trop.linear_cross_entropy_backward(one[:4], x, w, t, lse))
    refused("SHAPE", lambda: trop.linear_cross_entropy_backward(one, x, w, t, lse[:4]))


# ------------------------------------------------------------------ AdamW


def _sizes_of(kind):
    return {"one": [1], "odd": [1, 2, 255, 256, 257, 511, 4095, 4096, 4097, 9001], "many": [300 + i for i in range(470)],
            "empty": [0, 5, 0, 300]}[kind]


def _encode(v, codes):
    """Codes and scales of one tensor's blocks: v signed for 127 levels, nonnegative for 255."""
    n = v.numel()
    rows = torch.cat([v, v.new_zeros(-n % 256)]).reshape(-1, 256)
    top = rows.abs().amax(1, keepdim=True)
    c = torch.round(torch.sqrt((rows.abs() * torch.where(top > 0, 1 / top, 0.0)).clamp(max=1)) * codes)
    if codes == 255:
        c = torch.where(rows > 0, c.clamp(min=1), c)
    return torch.copysign(c, rows).reshape(-1)[:n], (top * float(1 / (codes * codes)))[:, 0]


def _decode(c, scale):
    c = c.float()
    return (c * c.abs()) * scale.repeat_interleave(256)[:c.numel()]


def _adamw_plain(p, g, m, v, k, h):
    """The step in f32 in the documented order of operations; exact to the last bit."""
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + (g * g) * (1 - h["beta2"])
    r = torch.sqrt(v)
    q = m / (r * (1 / math.sqrt(1 - h["beta2"] ** k)) + h["eps"])
    return p * (1 - h["lr"] * h["weight_decay"]) - q * (h["lr"] / (1 - h["beta1"] ** k)), m, v, r


HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.98, eps=1e-8, weight_decay=0.05)


@pytest.mark.parametrize("kind", ["one", "odd", "many", "empty"])
@pytest.mark.parametrize("pdt,gdt", [(F, F), (F, B), (F, H), (B, B), (B, F), (H, H), (H, F)])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_bitwise(trop, kind, pdt, gdt, bits):
    sizes = _sizes_of(kind)
    p = [_normal(i, n).to(pdt) for i, n in enumerate(sizes)]
    grads = [(0.1 * _normal(1000 + i, n) * 10.0 ** -(i % 4)).to(gdt) for i, n in enumerate(sizes)]
    opt = trop.AdamW(p, grads, state_bits=bits, **HYPER)
    want = [x.clone() for x in p]
    m = [torch.zeros(n, device="cuda") for n in sizes]
    v = [torch.zeros(n, device="cuda") for n in sizes]
    for k in (1, 2, 3):
        opt.step()
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            q, m[i], v[i], r = _adamw_plain(want[i].float(), grads[i].float(), m[i], v[i], k, HYPER)
            want[i] = q.to(pdt)
            if bits == 8:
                cm, ms = _encode(m[i], 127)
                cr, rs = _encode(r, 255)
                assert torch.equal(opt.exp_avg[i], cm.to(torch.int8)) and torch.equal(opt.exp_avg_scale[i], ms)
                assert torch.equal(opt.exp_avg_sq[i], cr.to(torch.uint8)) and torch.equal(opt.exp_avg_sq_scale[i], rs)
                m[i], v[i] = _decode(cm, ms), _decode(cr, rs) ** 2
            else:
                assert torch.equal(opt.exp_avg[i], m[i]) and torch.equal(opt.exp_avg_sq[i], v[i])
            assert torch.equal(p[i], want[i])
    if bits == 8:
        mv, vv = trop.adamw_state_values(opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale)
        assert all(torch.equal(a, b) for a, b in zip(mv + list(vv), m + v))


def test_adamw_against_64_bits(trop):
    p = [_normal(3, 5000)]
    g = [_normal(4, 5000) * 0.01]
    want, m, v = p[0].double(), 0.0, 0.0
    opt = trop.AdamW(p, g, **HYPER)
    for k in range(1, 6):
        opt.step()
        m = HYPER["beta1"] * m + (1 - HYPER["beta1"]) * g[0].double()
        v = HYPER["beta2"] * v + (1 - HYPER["beta2"]) * g[0].double() ** 2
        hat = (m / (1 - HYPER["beta1"] ** k)) / ((v / (1 - HYPER["beta2"] ** k)).sqrt() + HYPER["eps"])
        want = want - HYPER["lr"] * (hat + HYPER["weight_decay"] * want)
    # five steps of three roundings of p each
    assert _norm(p[0], want) <= 16 * U


def test_adamw_unaligned_tensors_copies_and_gradient_scale(trop):
    base = [_normal(i, 1500) for i in range(4)]
    for shift in (0, 1, 3):
        p, g, m, v = (t[shift:shift + 1203].clone() for t in base)
        v = v.abs()
        store = [torch.zeros(1300, device="cuda") for _ in range(4)]
        views = [s[shift:shift + 1203] for s in store]
        for a, t in zip(views, (p, g, m, v)):
            a.copy_(t)
        copy = torch.zeros(1300, device="cuda", dtype=B)[shift:shift + 1203]
        trop.adamw_step([views[0]], [views[1]], [views[2]], [views[3]], step=7, grad_scale=0.25, copies=[copy], **HYPER)
        q, m, v, _ = _adamw_plain(p, g * 0.25, m, v, 7, HYPER)
        assert torch.equal(views[0], q) and torch.equal(views[2], m) and torch.equal(views[3], v)
        assert torch.equal(copy, q.to(B))
        for s in store[:1] + store[2:]:  # nothing beside the views
            assert not bool(s[:shift].any()) and not bool(s[shift + 1203:].any())


def test_adamw_zero_and_non_finite_gradients(trop):
    p, g = [_normal(1, 600)], [torch.zeros(600, device="cuda")]
    before = p[0].clone()
    opt = trop.AdamW(p, g, state_bits=8, weight_decay=0.0)
    opt.step()
    assert torch.equal(p[0], before) and not bool(opt.exp_avg[0].any()) and not bool(opt.exp_avg_sq[0].any())
    g[0][300] = float("nan")
    opt.step()
    assert p[0].isnan().nonzero()[:, 0].tolist() == [300]
    mv, vv = trop.adamw_state_values(opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale)
    nan = torch.zeros(600, dtype=torch.bool, device="cuda")
    nan[256:512] = True  # its block, and no other
    assert torch.equal(mv[0].isnan(), nan) and torch.equal(vv[0].isnan(), nan)


def test_adamw_plan_equals_the_call(trop):
    make = lambda: [_normal(i, 777 + i) for i in range(40)]  # noqa: E731
    sets = []
    for _ in range(2):
        p, g = make(), make()
        sets.append((p, g, [torch.zeros_like(t) for t in p], [torch.zeros_like(t) for t in p]))
    plan = trop.AdamWPlan(*sets[0])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for k in (1, 2):
        plan.step(k, stream=stream, **HYPER)
        trop.adamw_step(*sets[1], step=k, **HYPER)
    torch.cuda.current_stream().wait_stream(stream)
    for a, b in zip(sets[0], sets[1]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    plan.close()
    with pytest.raises(RuntimeError):
        plan.step(3)


def test_adamw_refusals(trop):
    p, g = [_normal(1, 10)], [_normal(2, 10)]
    m, v = [torch.zeros(10, device="cuda")], [torch.zeros(10, device="cuda")]

    def refused(name, f):
        with pytest.raises(trop.TropicalError) as e:
            f()
        assert e.value.name == name

    refused("INVALID_ARG", lambda: trop.adamw_step(p, g, m, v, step=0))
    refused("INVALID_ARG", lambda: trop.adamw_step(p, g, m, v, step=1, beta1=1.0))
    refused("INVALID_ARG", lambda: trop.adamw_step(p, g, m, v, step=1, lr=float("nan")))
    refused("SHAPE", lambda: trop.adamw_step(p, [], m, v, step=1))
    refused("SHAPE", lambda: trop.adamw_step(p, [g[0][:5]], m, v, step=1))
    refused("DTYPE", lambda: trop.adamw_step(p, g, [m[0].to(B)], v, step=1))
    refused("DTYPE", lambda: trop.adamw_step([p[0].double()], g, m, v, step=1))
    refused("DTYPE", lambda: trop.adamw_step([p[0].to(B)], [g[0].to(H)], m, v, step=1))
    refused("DTYPE", lambda: trop.adamw_step([p[0].to(B)], [g[0].to(B)], m, v, step=1, copies=[p[0].to(H)]))
    refused("INVALID_ARG", lambda: trop.adamw_step([torch.zeros(20, device="cuda")[::2]], g, m, v, step=1))
    refused("INVALID_ARG", lambda: trop.adamw_step(p, g, m, v, m, step=1))
    refused("DEVICE_MISMATCH", lambda: trop.adamw_step(p, [g[0].cpu()], m, v, step=1))
    trop.adamw_step([], [], [], [], step=1)


# ------------------------------------------------------------------ streams, autograd, and the operators together


def test_operators_on_another_stream(trop):
    x, w, t = _head(200, 64, 900, B, 40)
    want = trop.linear_cross_entropy(x, w, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = trop.linear_cross_entropy(x, w, t)
        y = trop.layer_norm(x)
    given = trop.linear_cross_entropy(x, w, t, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a in (got, given):
        assert all(torch.equal(p, q) for p, q in zip(a, want))
    assert all(torch.equal(p, q) for p, q in zip(y, trop.layer_norm(x)))
    assert trop.stats()["stream_syncs"] == 0 and trop.device_wait_timeouts() == 0


def test_autograd_and_the_example_learn(trop):
    x = _normal(1, 30, 48).requires_grad_()
    w = _normal(2, 48).requires_grad_()
    b = _normal(3, 48).requires_grad_()
    head = (0.2 * _normal(4, 70, 48)).to(B).requires_grad_()
    t = torch.randint(0, 70, (30,), generator=_gen(5), device="cuda")
    loss = trop.LinearCrossEntropy.apply(trop.LayerNorm.apply(x, w, b, 1e-5, B), head, t, "mean", IGNORE)
    loss.backward()
    ref = [a.detach().double().requires_grad_() for a in (x, w, b, head)]
    y = torch.nn.functional.layer_norm(ref[0], (48,), ref[1], ref[2])
    torch.nn.functional.cross_entropy(y @ ref[3].T, t).backward()
    for a, r in zip((x, w, b, head), ref):
        assert _norm(a.grad, r.grad) <= 2.0 ** -6  # y, P and the gradients between are rounded to bf16

    from einsum_device_side_gb300 import tropical_net
    losses = tropical_net.train(steps=60, seed=3)
    assert losses[-1] < 0.7 * losses[0] and all(math.isfinite(v) for v in losses)
