"""The residual block's operators at the borders of what they accept: matrices and vectors that start anywhere in a buffer,
few columns in many rows, values near the ends of their types, the routes that calls take.

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


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("S, U, Y", [(F, F, F), (B, B, B), (F, B, B)])
@pytest.mark.parametrize("cols", [64, 1001, 4096, 8192, 20001])
def test_squares_past_the_range_of_f32(trop, cols, S, U, Y, norm):
    """A finite row whose squares pass f32's range has an infinite deviation: its norm is zero, as layer_norm's is, what comes back
    through it too, and the rows beside it are what they are without it."""
    t, o = make(9, cols, S, U, Y, norm=norm, gate="row")
    tensors = {k: t[k] for k in ("gate", "scale", "post_weight", "post_bias")}

    def call():
        y, r, stats, _ = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], **tensors, **o)
        return y, r, stats, trop.residual_norm_backward(t["dy"], t["dr"], r, t["u"], stats, t["weight"], t["bias"], **tensors, **o)

    y0, r0, stats0, g0 = call()
    t["x"][2] *= 1e25
    t["u"][5] *= 1e25
    y, r, stats, g = call()
    assert torch.equal(y[2], t["bias"].to(Y)) and float(stats[3, 2]) == 0 and float(stats[1, 5]) == 0
    assert all(bool(v.isfinite().all()) for v in (y, r, stats, *g))
    assert not bool(g[1][5].any())
    # with a norm of zero all of d comes from dr: alpha dr, one rounding in f32 and one to the type
    want = 0.7 * t["dr"][2].double()
    assert bool(((g[0][2].double() - want).abs() <= (torch.finfo(S).eps / 2 + 2 ** -23) * want.abs()).all())
    others = [0, 1, 3, 4, 6, 7, 8]
    for a, b in zip((y, r, *g[:3]), (y0, r0, *g0[:3])):
        assert torch.equal(a[others], b[others])
    if Y == F and norm == "layer":
        x = t["x"]
        mine = trop.residual_norm(x, torch.zeros_like(x), None, t["bias"], post_norm=False)[0]
        assert torch.equal(mine[2], trop.layer_norm(x, torch.ones_like(t["bias"]), t["bias"])[0][2])


@pytest.mark.parametrize("S, U, Y, W", [(F, F, F, F), (B, B, B, B), (B, B, B, F), (F, B, B, B), (F, B, B, F), (F, F, B, B), (F, F, B, F)])
def test_rows_on_16_bytes_take_no_long_rows_kernels(trop, S, U, Y, W):
    """Backward, whatever is given beside the rows: one kernel over the rows and one that joins the column sums, where the long rows'
    take a third for the sums.  Few rows and as many as fill the device, up to the widest that a cluster shares."""
    for rows, widths in ((1300, (16, 32, 64, 128, 256, 272, 320, 400, 512, 528, 1024)), (2, (48, 528, 2048, 4096, 4112, 8192, 12288, 20000, 32768))):
        for cols in widths:
            t, o = make(rows, cols, S, U, Y, W)
            for keep in (False, True):
                y, r, stats, kept = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], scale=t["scale"], gate=t["gate"], post_weight=t["post_weight"],
                                                       post_bias=t["post_bias"], out_dtype=Y if Y != U else None, keep=keep, **o)
                u, g, r = kept if keep else (t["u"], t["gate"], r)
                for gate in (g, None):
                    for dr in (t["dr"], None):
                        before = trop.stats()["kernel_launches"]
                        trop.residual_norm_backward(t["dy"], dr, r, u, stats, t["weight"], t["bias"], scale=t["scale"], gate=gate, x_dtype=S, u_dtype=U,
                                                    post_weight=t["post_weight"], post_bias=t["post_bias"], **o)
                        assert trop.stats()["kernel_launches"] - before == 2, (rows, cols, keep, gate is None, dr is None)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("S, U", [(F, B), (F, H)])
@pytest.mark.parametrize("rows, cols", [(7, 272), (1300, 264), (1300, 512), (9000, 400)])
def test_32_bit_vectors_where_blocks_are_small(trop, rows, cols, S, U, act):
    """Blocks of 64 threads whose two stages, beside 32-bit vectors, an eighth of the shared memory does not hold."""
    t, o = make(rows, cols, S, U, U, F, gate_act=act, seed=rows)
    # column sums of 9000 rows: 152 x 7 blocks' at a time, chains of fewer additions than test_few_columns_in_many_rows
    check(trop, t, o, S, U, U)


@pytest.mark.parametrize("kind", ["full", "row"])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("cols", [5, 100, 1024, 20001])
def test_32_bit_gates_far_from_zero(trop, cols, act, kind):
    """Element by element, relative to each: the stream's value is the gate's, whose gradient is its slope.  The exponential is good to 2
    units in the last place (2^-22), the reciprocal to one (2^-23), the denominator and the product with the gate round by 2^-24 each, as
    do the three products with ones: the sigmoid is off by 4.2e-7, the value by less than 2^-20.  The slopes are s (1 - s), and s + g s
    (1 - s), whose terms cancel to no less than a quarter of them up to g = -2: below five times the sigmoid's and some
    roundings, 2^-18."""
    rows = 65
    g = torch.linspace(-87, -2, rows * (cols if kind == "full" else 1), device="cuda").view(rows, -1)
    one = torch.ones(rows, cols, device="cuda")
    y, r, stats, _ = trop.residual_norm(torch.zeros_like(one), one, gate=g, gate_act=act, post_norm=False)
    wide = g.double().requires_grad_()
    want = (torch.sigmoid if act == "sigmoid" else torch.nn.functional.silu)(wide)
    assert bool(((r.double() - want) / want).abs().max() <= 2 ** -20)
    slope, = torch.autograd.grad(want.sum(), wide)
    # dy zero and dr one: all that reaches the gate is its slope; of a gate of a row, summed over equal elements
    dg = trop.residual_norm_backward(torch.zeros_like(one), one, r, one, stats, gate=g, gate_act=act, post_norm=False, want="gate")[2]
    want = slope if kind == "full" else slope * cols
    assert bool(((dg.double() - want) / want).abs().max() <= 2 ** -18)


@pytest.mark.parametrize("kind", ["full", "row"])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("S, U, Y", [(F, F, F), (B, B, B), (F, B, B)])
@pytest.mark.parametrize("rows, cols", [(2500, 33), (1300, 512), (700, 1001), (90, 4097), (330, 8192), (9, 20001)])
def test_rows_beside_others_that_hold_anything(trop, rows, cols, S, U, Y, keep, kind):
    """A row's results are the same bits whatever the rows beside it hold, forward and backward: other values, infinities, NaN."""
    t, o = make(rows, cols, S, U, Y, gate_act="silu", gate=kind)

    def call():
        tensors = {k: t[k] for k in ("gate", "scale", "post_weight", "post_bias")}
        y, r, stats, kept = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], **tensors, **o, keep=keep)
        ku, kg, kr = kept if keep else (t["u"], t["gate"], r)
        tensors["gate"] = kg
        g = trop.residual_norm_backward(t["dy"], t["dr"], kr, ku, stats, t["weight"], t["bias"], **tensors, **o, x_dtype=S, u_dtype=U)
        copies = [v for pair in (kept or ()) if isinstance(pair, tuple) for v in pair]
        return [y, r, stats.t(), *g[:3], *copies]

    before = call()
    gen = torch.Generator(device="cuda").manual_seed(7)
    others = torch.rand(rows, generator=gen, device="cuda") < 0.5
    others[1::4] = False  # (some of each)
    others[0] = True
    for k in ("x", "u", "gate", "dy", "dr"):
        new = torch.randn(t[k].shape, generator=gen, device="cuda") * 100
        at = torch.rand(t[k].shape, generator=gen, device="cuda")
        new[at < 0.02] = float("inf")
        new[at > 0.98] = float("nan")
        t[k] = torch.where(others[:, None], new.to(t[k].dtype), t[k])
    for a, b in zip(call(), before):
        assert torch.equal(a[~others], b[~others])


def test_scales_of_other_leading_axes_are_refused(trop):
    """As many rows in another order would be read as other rows' scales, of each of the three copies."""
    t, o = make(6, 64, B, B, B)
    v = lambda a: a.view(2, 3, -1)  # noqa: E731
    y, r, stats, kept = trop.residual_norm(v(t["x"]), v(t["u"]), gate=v(t["gate"]), **o, keep=True)
    args = lambda k: (v(t["dy"]), v(t["dr"]), k[2], k[0], stats)  # noqa: E731
    want = trop.residual_norm_backward(*args(kept), gate=kept[1], **o)
    for i in range(3):
        for wrong in (kept[i][1].view(3, 2, -1), kept[i][1].view(6, -1), kept[i][1].view(2, 6, -1)):
            bad = [*kept]
            bad[i] = (kept[i][0], wrong)
            with pytest.raises(trop.TropicalError) as e:
                trop.residual_norm_backward(*args(bad), gate=bad[1], **o)
            assert e.value.name == "SHAPE"
    # and by the matrices of the same rows
    flat = [tuple(c.reshape(6, -1) for c in k) for k in kept]
    got = trop.residual_norm_backward(t["dy"], t["dr"], flat[2], flat[0], stats.view(4, 6), gate=flat[1], **o)
    assert all(torch.equal(a.reshape(6, -1), b) for a, b in zip(want[:3], got[:3]))


@pytest.mark.parametrize("dt", [B, H])
@pytest.mark.parametrize("tokens, out, cols", [(4096, 4864, 2048), (7000, 4864, 2047), (2049, 130, 70), (16500, 64, 96), (40000, 300, 1000), (65536, 2050, 258)])
def test_long_sums_of_32_bit_weight_gradients(trop, tokens, out, cols, dt):
    """No chain of accumulations of a 32-bit result is longer than 2048 tokens: one over 8192 is off by six times what the plain 32-bit
    product is.  Products are exact, and a chain is taken to lose up to a last place every 16 of them; the chains' sums and the
    splits' are joined by as many roundings."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    dy, x = torch.randn(tokens, out, generator=g, device="cuda").to(dt), torch.randn(tokens, cols, generator=g, device="cuda").to(dt)
    codes, scales = trop.activation_pack(x)
    dw, _ = trop.activation_weight_grad(dy, codes, scales, out_dtype=F)
    want, size = torch.zeros(out, cols, dtype=torch.float64, device="cuda"), torch.zeros(out, cols, dtype=torch.float64, device="cuda")
    for i in range(0, tokens, 4096):
        d, v = dy[i:i + 4096].double(), trop.activation_values(codes[i:i + 4096], scales[i:i + 4096], F).double()
        want += d.T @ v
        size += d.abs().T @ v.abs()
    assert bool(((dw.double() - want).abs() <= (2048 / 16 + tokens / 2048 + 64) * 2.0 ** -24 * size).all())
    assert torch.equal(dw, trop.activation_weight_grad(dy, codes, scales, out_dtype=F)[0])
    if out == 4864:  # of 152 tiles, no split: the chains one after another
        parts = [trop.activation_weight_grad(dy[i:i + 2048], codes[i:i + 2048], scales[i:i + 2048], out_dtype=F)[0] for i in range(0, tokens, 2048)]
        total = parts[0]
        for p in parts[1:]:
            total = total + p
        assert torch.equal(dw, total)


def test_threads_at_once(trop):
    """Host threads, each on a stream of its own and with other sizes, as bit for bit what one thread gives."""
    import threading

    sizes = [(300, 1001), (700, 2048), (90, 8192), (64, 64)]
    jobs = []
    for rows, cols in sizes:
        t, o = make(rows, cols, B, B, B, gate_act="silu")
        tensors = {k: t[k] for k in ("gate", "scale", "post_weight", "post_bias")}

        def step(t=t, o=o, tensors=tensors):
            y, r, stats, kept = trop.residual_norm(t["x"], t["u"], t["weight"], t["bias"], **tensors, **o, keep=True)
            g = trop.residual_norm_backward(t["dy"], t["dr"], kept[2], kept[0], stats, t["weight"], t["bias"], **{**tensors, "gate": kept[1]}, **o)
            return (y, r, stats, *g, trop.activation_values(*kept[2], B), *trop.activation_weight_grad(t["dy"], *kept[0], out_dtype=F, want_bias=True))

        jobs.append((step, step()))
    torch.cuda.synchronize()
    wrong = []

    def work(step, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(25):
                    got = step()
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        wrong.append("differs")
        except Exception as e:
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=j) for j in jobs + jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong, wrong[:3]
