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


# ------------------------------------------------------------------ layer norm: shared memory


@pytest.mark.parametrize("rows,cols,dt,wdt", [(700, 6101, F, F), (700, 6111, B, F), (700, 12231, H, H), (4900, 4001, B, F)])
def test_layer_norm_where_static_and_dynamic_shared_memory_meet_48_kb(trop, rows, cols, dt, wdt):
    """Widths whose dynamic shared memory is just below 48 KB, with the kernel's static arrays above it."""
    x, dy, w, b = _normal(1, rows, cols).to(dt), _normal(2, rows, cols).to(dt), _normal(3, cols).to(wdt), _normal(4, cols).to(wdt)
    y, mean, rstd = trop.layer_norm(x, w, b)
    dx, dw, db = trop.layer_norm_backward(dy, x, mean, rstd, w)
    ref = [t.double().requires_grad_() for t in (x, w, b)]
    torch.nn.functional.layer_norm(ref[0], (cols,), ref[1], ref[2]).backward(dy.double())
    # f32 sums of up to 12231 terms, and one rounding to the result's type (2^-8, 2^-11) in the 2-norm
    for got, want in ((dx, ref[0].grad), (dw, ref[1].grad), (db, ref[2].grad)):
        limit = {F: 0.0, B: 2.0 ** -8, H: 2.0 ** -11}[got.dtype] + 64 * 2.0 ** -24
        assert float((got.double() - want).norm() / want.norm()) <= limit
    z = (x.double() - mean.double()[:, None]) * rstd.double()[:, None] * w.double() + b.double()
    assert float((y.double() - z).norm() / z.norm()) <= {F: 0.0, B: 2.0 ** -8, H: 2.0 ** -11}[dt] + 64 * 2.0 ** -24


def test_layer_norm_from_two_threads_with_other_widths(trop):
    """Two host threads, each with its stream, on one kernel with different amounts of shared memory: no call may lose its
    limit to the other's."""
    import threading

    cases, errors = [], []
    for seed, (rows, cols) in enumerate(((640, 4096), (2560, 1024))):
        x, dy, w = _normal(seed, rows, cols), _normal(seed + 2, rows, cols), _normal(seed + 4, cols)
        _, mean, rstd = trop.layer_norm(x, w)
        cases.append((dy, x, mean, rstd, w))
    want = [trop.layer_norm_backward(*c) for c in cases]
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(1500):
                    got = trop.layer_norm_backward(*cases[i])
                assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors


# ------------------------------------------------------------------ captured by the caller


def _captured(f):
    """f's results in a graph: (graph, results)."""
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    return graph, out


def _replayed_beside_eager_calls(f, inputs, others):
    """A captured f replays with new inputs on another stream, while the stream of the capture and the current one make
    eager calls of the same sizes."""
    f()  # the device's first call, outside the capture
    torch.cuda.synchronize()
    graph, out = _captured(f)
    side = torch.cuda.Stream()
    for k in range(4):
        values = [t.clone() if k % 2 else u.clone() for t, u in zip(inputs, others)]
        for t, u in zip(inputs, values):
            t.copy_(u)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        eager = [f() for _ in range(3)]  # (in the way of the replay's workspace, if it were shared)
        torch.cuda.synchronize()
        for e in eager:
            assert all(torch.equal(a, b) for a, b in zip(out, e))


@pytest.mark.parametrize("rows,cols,dt", [(3, 40, F), (2500, 1001, B), (700, 2048, F)])
def test_layer_norm_captured(trop, rows, cols, dt):
    x, dy, w = _normal(1, rows, cols).to(dt), _normal(2, rows, cols).to(dt), _normal(3, cols).to(dt)

    def f():
        y, mean, rstd = trop.layer_norm(x, w)
        return (y, mean, rstd, *trop.layer_norm_backward(dy, x, mean, rstd, w))

    _replayed_beside_eager_calls(f, (x, dy, w), (2 * x.flip(0), dy.flip(1), w.flip(0)))


@pytest.mark.parametrize("n,d,v", [(7, 64, 300), (300, 96, 1000), (1100, 65, 9001)])
def test_head_captured(trop, n, d, v):
    x, w = _normal(1, n, d).to(B), (_normal(2, v, d) / 4).to(B)
    t = torch.randint(0, v, (n,), device="cuda")
    t[::5] = IGNORE
    g = torch.rand(n, device="cuda") + 0.5

    def f():
        loss, lse, kept = trop.linear_cross_entropy(x, w, t)
        return (loss, lse, kept, *trop.linear_cross_entropy_backward(g, x, w, t, lse))

    _replayed_beside_eager_calls(f, (x, w, t, g), (x.flip(0), w.flip(0), t.flip(0), g.flip(0)))


# ------------------------------------------------------------------ what is kept between calls


def test_threads_that_end_leave_their_workspace_to_the_next(trop):
    import threading

    x, dy, w = _normal(1, 2400, 2048), _normal(2, 2400, 2048), _normal(3, 2048)
    _, mean, rstd = trop.layer_norm(x, w)
    want = trop.layer_norm_backward(dy, x, mean, rstd, w)
    out = []

    def work():
        out.append(trop.layer_norm_backward(dy, x, mean, rstd, w))

    def run(n):
        for _ in range(n):
            t = threading.Thread(target=work)
            t.start()
            t.join()
            got = out.pop()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        torch.cuda.synchronize()

    run(4)
    before = torch.cuda.mem_get_info()[0]
    run(40)  # (a block of this call is some MB)
    assert before - torch.cuda.mem_get_info()[0] < 8 << 20


def test_kept_workspace_grows_once(trop):
    """A small call, then larger ones: the block is replaced once for each doubling, and kept from then on."""
    cases = []
    for cols in (64, 256, 1024, 4096):
        x, w = _normal(1, 2400, cols), _normal(3, cols)
        cases.append((_normal(2, 2400, cols), x, *trop.layer_norm(x, w)[1:], w))
    with torch.cuda.stream(torch.cuda.Stream()):
        for c in cases:
            want = trop.layer_norm_backward(*c)
        for _ in range(3):  # (the results' own memory)
            got = trop.layer_norm_backward(*cases[-1])
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        for _ in range(20):
            got = trop.layer_norm_backward(*cases[-1])
        torch.cuda.synchronize()
        assert before - torch.cuda.mem_get_info()[0] < 8 << 20
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_destroyed_stream_s_workspace_is_not_the_next_one_s(trop):
    """A stream destroyed with its work still on its way: its handle may come back at once for a new stream, whose calls run
    beside that work."""
    import ctypes

    runtime = torch.cuda.cudart()
    x, dy, w = _normal(1, 2400, 1024), _normal(2, 2400, 1024), _normal(3, 1024)
    _, mean, rstd = trop.layer_norm(x, w)
    sets = [(dy * k, x, mean, rstd, w) for k in (1.0, 3.0)]
    want = [trop.layer_norm_backward(*s) for s in sets]
    torch.cuda.synchronize()
    results = []
    for i in range(20):
        handle = ctypes.c_void_p()
        assert int(runtime.cudaStreamCreate(ctypes.addressof(handle))) == 0
        stream = torch.cuda.ExternalStream(handle.value)
        with torch.cuda.stream(stream):
            torch.cuda._sleep(200_000)
            results.append(trop.layer_norm_backward(*sets[i % 2]))
        assert int(runtime.cudaStreamDestroy(handle.value)) == 0
    torch.cuda.synchronize()
    for i, got in enumerate(results):
        assert all(torch.equal(a, b) for a, b in zip(got, want[i % 2]))


def test_a_destroyed_stream_s_ticket_is_not_the_next_one_s(trop):
    """The same for the counter by which the head's last block to finish joins the pairs."""
    import ctypes

    runtime = torch.cuda.cudart()
    t = torch.randint(0, 3000, (700,), device="cuda")
    sets = [((_normal(1, n, 64) * k).to(B), (_normal(2, 3000, 64) / 4).to(B), t[:n]) for n in (20, 700) for k in (1.0, 3.0)]
    want = [trop.linear_cross_entropy(*s) for s in sets]
    torch.cuda.synchronize()
    results = []
    for i in range(40):
        handle = ctypes.c_void_p()
        assert int(runtime.cudaStreamCreate(ctypes.addressof(handle))) == 0
        stream = torch.cuda.ExternalStream(handle.value)
        with torch.cuda.stream(stream):
            torch.cuda._sleep(200_000)
            results.append(trop.linear_cross_entropy(*sets[i % 4]))
        assert int(runtime.cudaStreamDestroy(handle.value)) == 0
    torch.cuda.synchronize()
    for i, got in enumerate(results):
        assert all(torch.equal(a, b) for a, b in zip(got, want[i % 4]))


def test_more_streams_than_blocks_are_kept(trop):
    """Calls on streams beyond those: workspace from the pool, a ticket of their own."""
    import ctypes

    runtime = torch.cuda.cudart()
    trop.release_pool()
    x, w, t = _normal(1, 300, 64).to(B), (_normal(2, 3000, 64) / 4).to(B), torch.randint(0, 3000, (300,), device="cuda")
    rows, dy, weight = _normal(3, 400, 256), _normal(4, 400, 256), _normal(5, 256)
    stats = trop.layer_norm(rows, weight)[1:]

    def f():
        return (*trop.linear_cross_entropy(x, w, t), *trop.layer_norm_backward(dy, rows, *stats, weight))

    want = f()
    torch.cuda.synchronize()
    handles, results = [], []
    for _ in range(70):
        handle = ctypes.c_void_p()
        assert int(runtime.cudaStreamCreate(ctypes.addressof(handle))) == 0
        handles.append(handle.value)
        with torch.cuda.stream(torch.cuda.ExternalStream(handle.value)):
            results += [f(), f()]
    torch.cuda.synchronize()
    for got in results:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for h in handles:
        assert int(runtime.cudaStreamDestroy(h)) == 0
    trop.release_pool()


# ------------------------------------------------------------------ the head's gradients


@pytest.mark.parametrize("dt", [B, H])
@pytest.mark.parametrize("n", [60, 300])
def test_a_padded_token_s_gradient_counts_nowhere(trop, n, dt):
    """Whatever it is, the others' gradients stay as they are, bit for bit."""
    x, w = _normal(1, n, 64).to(dt), (_normal(2, 900, 64) / 4).to(dt)
    t = torch.randint(0, 900, (n,), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    t[5], t[n - 1] = IGNORE, IGNORE
    _, lse, _ = trop.linear_cross_entropy(x, w, t, "none")
    g = torch.full((n,), 1 / 8192, device="cuda")
    dx, dw = trop.linear_cross_entropy_backward(g, x, w, t, lse)
    for pad in (1e9, float("inf"), float("nan")):
        g[5], g[n - 1] = pad, -pad
        px, pw = trop.linear_cross_entropy_backward(g, x, w, t, lse)
        assert torch.equal(px, dx) and torch.equal(pw, dw)
    # a kept token's infinite gradient is its own row's
    g[5] = g[n - 1] = 1 / 8192
    g[7] = float("inf")
    px, _ = trop.linear_cross_entropy_backward(g, x, w, t, lse)
    rest = torch.arange(n, device="cuda") != 7
    assert torch.equal(px[rest], dx[rest]) and not bool(px[7].isfinite().any())


@pytest.mark.parametrize("each", [False, True])
@pytest.mark.parametrize("n", [60, 300])
def test_gradients_of_a_subnormal_loss_gradient(trop, n, each):
    """A gradient of 2^-130: in bf16 the gradients of 1 times 2^-130, to a place of the subnormals; in f16 zero."""
    for dt in (B, H):
        x, w = _normal(1, n, 64).to(dt), (_normal(2, 900, 64) / 4).to(dt)
        t = torch.randint(0, 900, (n,), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
        _, lse, _ = trop.linear_cross_entropy(x, w, t, "none")
        one = torch.ones(n if each else (), device="cuda")
        want = trop.linear_cross_entropy_backward(one, x, w, t, lse)
        got = trop.linear_cross_entropy_backward(one * 2.0 ** -130, x, w, t, lse)
        for a, b in zip(got, want):
            if dt == H:
                assert not bool(a.any())
            else:
                assert float((a.double() - b.double() * 2.0 ** -130).abs().max()) <= 2.0 ** -133


# ------------------------------------------------------------------ AdamW


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), 1e30, float("nan")])
def test_an_8_bit_block_with_a_state_that_is_not_finite_reads_back_as_nan(trop, bad):
    """All of the block, the entry itself among it (of 1e30 the square overflows: v, not m)."""
    p, g = [_normal(1, 600)], [_normal(2, 600)]
    g[0][300] = bad
    opt = trop.AdamW(p, g, state_bits=8)
    opt.step()
    m, v = trop.adamw_state_values(opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale)
    block = torch.zeros(600, dtype=torch.bool, device="cuda")
    block[256:512] = True
    assert torch.equal(v[0].isnan(), block) and bool(v[0][~block].isfinite().all())
    assert torch.equal(m[0].isnan(), block) if bad != 1e30 else bool(m[0].isfinite().all())


def test_a_captured_step_is_refused_where_its_number_would_repeat(trop):
    """AdamW counts steps on the host; the plan, which is given the number, may be captured."""
    p, g = [_normal(1, 600)], [_normal(2, 600)]
    opt = trop.AdamW(p, g)
    opt.step()
    m, v = [torch.zeros(600, device="cuda")], [torch.zeros(600, device="cuda")]
    plan = trop.AdamWPlan(p, g, m, v)
    q, n, u = [p[0].clone()], [m[0].clone()], [v[0].clone()]
    graph = torch.cuda.CUDAGraph()
    refused = None
    with torch.cuda.graph(graph):
        try:
            opt.step()
        except trop.TropicalError as e:
            refused = e.name
        plan.step(1000)
    assert refused == "UNSUPPORTED" and opt.steps == 1
    for _ in range(2):
        graph.replay()
        trop.adamw_step(q, g, n, u, step=1000)
    assert torch.equal(p[0], q[0]) and torch.equal(m[0], n[0]) and torch.equal(v[0], u[0])


# ------------------------------------------------------------------ layer norm: values


@pytest.mark.parametrize("rows,cols", [(3, 61), (2500, 61), (2500, 244), (700, 3904), (5, 3904), (2, 31232)])
def test_constant_rows_give_the_bias(trop, rows, cols):
    """Whole numbers whose sums are exact in f32: the mean is the row's value, so nothing of it is left."""
    most = (1 << 24) // cols - 1
    value = torch.randint(most // 2, most, (rows, 1), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).float()
    b = _normal(2, cols)
    y, mean, _ = trop.layer_norm(value.expand(rows, cols).contiguous(), torch.ones(cols, device="cuda"), b)
    assert torch.equal(mean, value[:, 0]) and torch.equal(y, b.expand(rows, cols))


@pytest.mark.parametrize("cols", [1, 3, 7, 41, 61, 244, 1000, 4093, 20011])
def test_means_are_the_nearest_quotients(trop, cols):
    """Whole numbers whose sums are exact in f32, over the number of columns: the division's own rounding."""
    gen = torch.Generator("cuda").manual_seed(cols)
    most = (1 << 24) // cols
    x = torch.randint(-most, most + 1, (500, cols), device="cuda", generator=gen).float() * 2.0 ** -20
    x[0] = 0
    _, mean, _ = trop.layer_norm(x)
    assert torch.equal(mean.cpu(), (x.double().sum(1).cpu().float() / torch.tensor(float(cols))))


def test_a_training_step_captured_through_autograd(trop):
    """Forward and backward (the latter from autograd's thread) in one graph, replayed on new inputs."""
    x, w, b = _normal(1, 70, 5, 64), _normal(2, 64).requires_grad_(), _normal(3, 64).requires_grad_()
    head, t = (_normal(4, 200, 64) / 4).to(B).requires_grad_(), torch.randint(0, 200, (350,), device="cuda")
    leaves = (w, b, head)

    def step():
        y = trop.LayerNorm.apply(x, w, b, 1e-5, B)
        loss = trop.LinearCrossEntropy.apply(y.view(350, 64), head, t)
        return (loss.detach(), *torch.autograd.grad(loss, leaves))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph, out = _captured(step)
    for k in range(3):
        x.mul_(-0.5)
        graph.replay()
        assert all(torch.equal(a, e) for a, e in zip(out, step()))
