"""GPU: layer norm and its gradients against the 64-bit oracle.

The bounds are a priori ones of oracle/layernorm_oracle.py: no sum of a row meets more than
cols / 64 + 16 additions in a lane and across lanes, and no sum over rows more than rows + 16,
whatever the kernel's division of the work."""
import numpy as np
import pytest

import oracle.layernorm_oracle as L
import tensor_gradient_compression_amd as tg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 1e-5
TYPES = [("f32", "f32"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")]
SHAPES = [(1, 1), (3, 2), (5, 7), (64, 64), (33, 65), (257, 128), (4, 255), (130, 256), (9, 257), (1, 513),
          (70, 1000), (300, 1024), (6, 1026), (2, 2048), (3, 4099), (5, 8192), (2, 16384), (3, 16385), (1, 70001)]


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def inputs(rows, cols, dtype, wdtype, seed, shift=0.5, offset=0, gap=0):
    """x with rows of their own level, dy, weight, bias; x and dy start `offset` elements into
    their allocation and have `gap` unused elements between rows."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    def rows_in(t):
        buf = torch.full((rows * (cols + gap) + offset,), float("nan"), device="cuda").to(tg.torch_dtype(dtype))
        v = buf[offset:].view(rows, cols + gap)[:, :cols]
        v.copy_(t)
        return v

    x = rows_in(normal(rows, cols) * torch.exp(normal(rows, 1)) + shift * normal(rows, 1))
    dy = rows_in(normal(rows, cols))
    w = (1 + 0.2 * normal(cols)).to(tg.torch_dtype(wdtype))
    b = (0.2 * normal(cols)).to(tg.torch_dtype(wdtype))
    return x, dy, w, b


def close(got, true, bound, what):
    off = np.abs(host(got) - true)
    assert np.all(off <= bound), f"{what}: {np.nanmax(off / bound):.3g} of the bound"


def check(x, dy, w, b, dtype, wdtype, params=True, eps=EPS):
    rows, cols = x.shape
    seq = cols / 64 + 16
    X, W, B = host(x), host(w), host(b)
    y, mean, rstd = tg.layer_norm_forward(x, w, b, eps=eps)
    assert y.dtype == x.dtype and y.shape == x.shape and mean.shape == rstd.shape == (rows,)
    for got, true, bound, what in zip((y, mean, rstd), L.forward(X, W, B, eps),
                                      L.forward_bounds(X, W, B, eps, dtype, seq), ("y", "mean", "rstd")):
        close(got, true, bound, what)
    dx, dw, db = tg.layer_norm_backward(dy, x, w, mean, rstd, params=params)
    assert dx.dtype == x.dtype and dx.shape == x.shape
    true = L.backward(host(dy), X, W, host(mean), host(rstd))
    bounds = L.backward_bounds(host(dy), X, W, host(mean), host(rstd), dtype, wdtype, seq, rows + 16)
    close(dx, true[0], bounds[0], "dx")
    if not params:
        assert dw is None and db is None
        return
    assert dw.dtype == db.dtype == (w if w is not None else x).dtype
    close(dw, true[1], bounds[1], "dweight")
    close(db, true[2], bounds[2], "dbias")


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,wdtype", TYPES)
def test_against_the_oracle(rows, cols, dtype, wdtype):
    print(f"CASE layer norm {rows} x {cols} {dtype} {wdtype}", flush=True)
    check(*inputs(rows, cols, dtype, wdtype, seed=rows + cols), dtype, wdtype)


@pytest.mark.parametrize("rows,cols", [(5, 64), (7, 333), (40, 1024), (3, 8192), (2, 20000)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("offset,gap", [(1, 0), (0, 1), (3, 5), (0, 8), (8, 64)])
def test_rows_apart_and_unaligned(rows, cols, dtype, offset, gap):
    check(*inputs(rows, cols, dtype, dtype, seed=1, offset=offset, gap=gap), dtype, dtype)


@pytest.mark.parametrize("rows,cols", [(9, 1025), (7, 1536), (600, 2001), (9, 4096), (5, 8191), (4, 9001), (3, 16383)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("offset,gap", [(0, 0), (1, 0), (0, 1), (1, 2), (2, 3)])
def test_rows_that_start_at_odd_values(rows, cols, dtype, offset, gap):
    """Rows of several waves; the values before and after each row are NaN."""
    check(*inputs(rows, cols, dtype, "f32", seed=12, offset=offset, gap=gap), dtype, "f32")


@pytest.mark.parametrize("cols", [64, 1000, 8192])
def test_without_weight_bias_or_parameter_gradients(cols):
    x, dy, w, b = inputs(37, cols, "bf16", "f32", seed=2)
    check(x, dy, None, None, "bf16", "bf16")
    check(x, dy, w, None, "bf16", "f32")
    check(x, dy, w, b, "bf16", "f32", params=False)
    y0, mean, rstd = tg.layer_norm_forward(x, None, b)
    close(y0, L.forward(host(x), None, host(b), EPS)[0], L.forward_bounds(host(x), None, host(b), EPS, "bf16", cols / 64 + 16)[0], "y")


@pytest.mark.parametrize("rows,cols", [(70000, 8), (66000, 64), (4097, 256), (2500, 1024)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(rows, cols, dtype):
    check(*inputs(rows, cols, dtype, "f32", seed=3), dtype, "f32")


@pytest.mark.parametrize("cols", [5, 256, 1024, 5000])
def test_rows_far_from_zero(cols):
    """A mean 1000 times the deviation: the bounds hold the variance to what the rounding of x's
    own distances allows, which the mean of squares less the squared mean would not meet."""
    check(*inputs(20, cols, "f32", "f32", seed=4, shift=1000.0), "f32", "f32")


@pytest.mark.parametrize("cols", [1, 3, 256, 3000])
def test_constant_rows(cols):
    """A variance of zero: n is 0, y the bias, rstd 1 / sqrt(eps)."""
    x = torch.full((6, cols), 0.5, device="cuda")
    _, dy, w, b = inputs(6, cols, "f32", "f32", seed=5)
    y, mean, rstd = tg.layer_norm_forward(x, w, b, eps=EPS)
    assert torch.equal(y, b.expand(6, cols)) and torch.equal(mean, torch.full((6,), 0.5, device="cuda"))
    assert abs(float(rstd[0]) * np.sqrt(EPS) - 1) < 4 * L.EPS32
    check(x, dy, w, b, "f32", "f32")


@pytest.mark.parametrize("rows,cols", [(r * t + more, c) for r, t, c in ((256, 8, 5), (64, 8, 27), (8, 8, 256), (4, 8, 333),
                                                                        (4, 4, 1000), (1, 4, 2050), (1, 4, 9000))
                                       for t in (1, t) for more in (0, 1)])
@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("bf16", "bf16")])
def test_a_workgroup_alone_and_two(rows, cols, dtype, wdtype):
    """The most rows that one workgroup takes, and one more; the gradient of x is the same
    without those of the parameters."""
    x, dy, w, b = inputs(rows, cols, dtype, wdtype, seed=8)
    check(x, dy, w, b, dtype, wdtype)
    _, mean, rstd = tg.layer_norm_forward(x, w, b)
    assert torch.equal(tg.layer_norm_backward(dy, x, w, mean, rstd, params=False)[0],
                       tg.layer_norm_backward(dy, x, w, mean, rstd)[0])


@pytest.mark.parametrize("rows", [2, 3, 32, 33, 128, 129])
@pytest.mark.parametrize("cols", [2050, 8192, 9001, 16384])
@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_few_long_rows(rows, cols, dtype, wdtype):
    check(*inputs(rows, cols, dtype, wdtype, seed=15), dtype, wdtype)


@pytest.mark.parametrize("rows,cols", [(5, 333), (100, 333), (2, 20000), (0, 64)])
@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_one_of_the_parameters_gradients(rows, cols, dtype, wdtype):
    """dweight or dbias may be NULL at the C entry; the other is the same as with both."""
    x, dy, w, _ = inputs(rows, cols, dtype, wdtype, seed=13)
    _, mean, rstd = tg.layer_norm_forward(x, w)
    both = tg.layer_norm_backward(dy, x, w, mean, rstd)
    lib, code = tg.load_library(), tg.DTYPE_CODES
    ws = torch.empty(max(16, lib.tgrad_layer_norm_workspace(rows, cols)), dtype=torch.uint8, device="cuda")
    for which in (0, 1):
        dx, out = torch.empty_like(x), torch.full_like(w, float("nan"))
        p = [None, None]
        p[which] = out.data_ptr()
        rc = lib.tgrad_layer_norm_backward(dy.data_ptr(), cols, x.data_ptr(), cols, w.data_ptr(), mean.data_ptr(),
                                           rstd.data_ptr(), dx.data_ptr(), p[0], p[1], rows, cols, code[dtype],
                                           code[wdtype], ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        assert torch.equal(dx, both[0]) and torch.equal(out, both[1 + which])


@pytest.mark.parametrize("rows,cols,dtype", [(40000, 2001, "bf16"), (20000, 4096, "f16"), (300000, 255, "bf16"), (20000, 2050, "f32")])
def test_calls_larger_than_the_caches(rows, cols, dtype):
    """Such calls read past the caches: rows come out as in calls on a few of them, and the sums
    over rows within their bounds."""
    gen = torch.Generator(device="cuda").manual_seed(14)
    t = tg.torch_dtype(dtype)
    x, dy = (torch.randn(rows, cols, generator=gen, device="cuda").to(t) for _ in range(2))
    w = 1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")
    y, mean, rstd = tg.layer_norm_forward(x, w, w)
    dx, dw, db = tg.layer_norm_backward(dy, x, w, mean, rstd)
    for at in (0, rows // 3, rows - 64):
        r = slice(at, at + 64)
        part = tg.layer_norm_forward(x[r], w, w)
        assert torch.equal(y[r], part[0]) and torch.equal(mean[r], part[1]) and torch.equal(rstd[r], part[2])
        assert torch.equal(dx[r], tg.layer_norm_backward(dy[r], x[r], w, mean[r], rstd[r], params=False)[0])
    n = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for got, terms, what in ((dw, dy.double() * n, "dweight"), (db, dy.double(), "dbias")):
        close(got, host(terms.sum(0)), L.gamma(rows + 16) * host(terms.abs().sum(0)), what)


@pytest.mark.parametrize("rows", [1, 300, 1705])
@pytest.mark.parametrize("dtype,wdtype", TYPES)
def test_one_column_has_no_gradient_of_x(rows, dtype, wdtype):
    """n is 0 and h its own mean, so dx and dweight are 0 and not the rounding of a product."""
    x, dy, w, _ = inputs(rows, 1, dtype, wdtype, seed=7)
    dx, dw, _ = tg.layer_norm_backward(dy, x, w, x[:, 0].float(), torch.full((rows,), EPS ** -0.5, device="cuda"))
    assert not dx.any() and not dw.any()


@pytest.mark.parametrize("cols", [2, 8, 64, 512, 1024, 2048, 8192, 16384])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_the_same_gradient_in_every_column_has_none_of_x(cols, dtype):
    """Neighbours k and -k, and dy of 0.75 everywhere: every sum is exact in any order, and
    h - mean(h) and mean(h n) are 0."""
    k = torch.arange(cols // 2, device="cuda") % 8 + 1
    x = torch.stack([k, -k], 1).reshape(1, cols).expand(5, cols).to(tg.torch_dtype(dtype)).contiguous()
    dx, _, db = tg.layer_norm_backward(torch.full_like(x, 0.75), x, None, torch.zeros(5, device="cuda"),
                                       torch.full((5,), 0.7, device="cuda"))
    assert not dx.any() and bool((db == 3.75).all())


@pytest.mark.parametrize("cols", [1, 3, 7, 13, 28, 41, 47, 111, 127, 410, 511, 1000, 1023, 2047, 4095])
def test_constant_rows_of_any_level(cols):
    """Values of 12 bits, so every sum is exact and the mean is the value itself: y is the bias
    and not eps's multiple of a mean that is off by a unit. The same for mean(dy w)."""
    level = torch.arange(2048.0, 4096.0, device="cuda") * 0.125
    x = level[:, None].expand(2048, cols).contiguous()
    b = torch.linspace(-1, 1, cols, device="cuda")
    y, mean, rstd = tg.layer_norm_forward(x, None, b, eps=EPS)
    assert torch.equal(mean, level) and torch.equal(y, b.expand(2048, cols))
    dx, _, _ = tg.layer_norm_backward(x, x, None, mean, rstd)
    assert not dx.any()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("cols", [64, 1000, 8192])
def test_rows_that_are_not_finite_stay_apart(bad, cols):
    x, dy, w, b = inputs(9, cols, "f32", "f32", seed=6)
    x[4, 3] = bad
    y, mean, rstd = tg.layer_norm_forward(x, w, b)
    dx, _, db = tg.layer_norm_backward(dy, x, w, mean, rstd)
    ok = [i for i in range(9) if i != 4]
    assert bool(y[4].isnan().all()) and bool(y[ok].isfinite().all())
    assert bool(dx[4].isnan().all()) and bool(dx[ok].isfinite().all()) and bool(db.isfinite().all())


def test_no_rows():
    for cols in (3, 1024):
        x = torch.empty(0, cols, device="cuda")
        w = torch.ones(cols, device="cuda")
        y, mean, rstd = tg.layer_norm_forward(x, w, w)
        dx, dw, db = tg.layer_norm_backward(x, x, w, mean, rstd)
        assert y.shape == dx.shape == (0, cols) and mean.shape == (0,)
        assert torch.equal(dw, torch.zeros_like(w)) and torch.equal(db, torch.zeros_like(w))


def test_shapes_of_several_axes():
    x, dy, w, b = inputs(6 * 5, 96, "bf16", "f32", seed=7)
    y, mean, rstd = tg.layer_norm_forward(x, w, b)
    x3 = x.reshape(6, 5, 96)
    y3, mean3, rstd3 = tg.layer_norm_forward(x3, w, b)
    assert torch.equal(y3.view(30, 96), y) and mean3.shape == (6, 5)
    # every second row block of a larger tensor, and one row
    z = torch.stack([x3, x3], 2)[:, :, 0]
    assert torch.equal(tg.layer_norm_forward(z, w, b)[0], y3)
    y1, m1, _ = tg.layer_norm_forward(x[0], w, b)
    assert torch.equal(y1, y[0]) and m1.shape == ()
    dx = tg.layer_norm_backward(dy.reshape(6, 5, 96), z, w, mean3, rstd3)[0]
    assert torch.equal(dx.view(30, 96), tg.layer_norm_backward(dy, x, w, mean, rstd)[0])


def test_sums_over_rows_repeat():
    x, dy, w, b = inputs(5000, 300, "bf16", "f32", seed=8)
    _, mean, rstd = tg.layer_norm_forward(x, w, b)
    first = tg.layer_norm_backward(dy, x, w, mean, rstd)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, tg.layer_norm_backward(dy, x, w, mean, rstd)))


def test_differentiable():
    x, dy, w, b = inputs(50, 200, "f32", "f32", seed=9)
    a = [t.clone().requires_grad_() for t in (x, w, b)]
    tg.layer_norm(*a, eps=EPS).backward(dy)
    _, mean, rstd = tg.layer_norm_forward(x, w, b, eps=EPS)
    for t, g in zip(a, tg.layer_norm_backward(dy, x, w, mean, rstd)):
        assert torch.equal(t.grad, g)
    # an expanded gradient, and inputs that need none
    x2 = x.clone().requires_grad_()
    tg.layer_norm(x2).sum().backward()
    assert float(x2.grad.abs().max()) < 1e-4
    w2 = w.clone().requires_grad_()
    tg.layer_norm(x, w2, b).sum().backward()
    assert w2.grad is not None


def test_another_stream_and_graph_replay():
    x, dy, w, b = inputs(500, 256, "bf16", "f32", seed=10)
    eager = tg.layer_norm_forward(x, w, b)
    back = tg.layer_norm_backward(dy, x, w, *eager[1:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tg.layer_norm_forward(x, w, b)
        got += tg.layer_norm_backward(dy, x, w, *got[1:])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(eager + back, got))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tg.layer_norm_forward(x, w, b)
        out += tg.layer_norm_backward(dy, x, w, *out[1:])
    for k in range(4):
        x.mul_(1.5)
        graph.replay()
        eager = tg.layer_norm_forward(x, w, b)
        eager += tg.layer_norm_backward(dy, x, w, *eager[1:])
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(eager, out)), f"replay {k}"


def test_refusals():
    x, dy, w, b = inputs(4, 32, "bf16", "f32", seed=11)
    _, mean, rstd = tg.layer_norm_forward(x, w, b)
    half = w.half()
    for args, what in (((x.cpu(), w, b), "GPU"), ((x.double(), w, b), "dtype"), ((x, w[:31], b), "weight"),
                       ((x, half, half), "weight"), ((x, w, b.bfloat16()), "bias"), ((x.t(), w, b), "last axis"),
                       ((x[:, :0], None, None), "empty"), ((x, w.cpu(), b), "weight"),
                       ((torch.zeros(32, 4, 4, device="cuda").transpose(0, 1).expand(4, 32, 4), None, None), "strides"),
                       ((x[:1].expand(4, 32), w, b), "overlap")):
        with pytest.raises(ValueError, match=what):
            tg.layer_norm_forward(*args)
    with pytest.raises(tg.TGradError, match="invalid argument"):
        tg.layer_norm_forward(x, w, b, eps=-1.0)
    for args, what in (((dy[:3], x, w, mean, rstd), "dy"), ((dy.float(), x, w, mean, rstd), "dy"),
                       ((dy, x, w, mean[:3], rstd), "mean"), ((dy, x, w, mean, rstd.double()), "rstd")):
        with pytest.raises(ValueError, match=what):
            tg.layer_norm_backward(*args)


def test_a_bias_alone_gets_a_gradient_of_its_own_precision():
    x, dy, _, b = inputs(400, 96, "bf16", "f32", seed=10)
    b.requires_grad_()
    tg.layer_norm(x, None, b).backward(dy)
    close(b.grad, host(dy).sum(0), L.gamma(416) * np.abs(host(dy)).sum(0), "dbias")


@pytest.mark.parametrize("shape,to", [((4, 1, 16), (4, 8, 16)), ((1, 8, 16), (4, 8, 16)), ((1, 1, 16), (4, 8, 16)),
                                      ((3, 1, 2, 16), (3, 8, 2, 16)), ((3, 2, 1, 16), (3, 2, 8, 16)),
                                      ((3, 1, 1, 16), (3, 8, 1, 16)), ((4, 1, 1), (4, 8, 1))])
def test_expanded_leading_axes_are_refused(shape, to):
    """Such rows lie in memory once and not evenly spaced: refused before a launch, as x and as
    dy, and taken once they are contiguous."""
    gen = torch.Generator(device="cuda").manual_seed(16)
    x = torch.randn(*shape, generator=gen, device="cuda").expand(*to)
    full = x.contiguous()
    for f in (tg.layer_norm_forward, tg.layer_norm):
        with pytest.raises(ValueError, match="x: .*contiguous"):
            f(x)
    y, mean, rstd = tg.layer_norm_forward(full)
    for args, what in (((full, x), "x"), ((x, full), "dy")):
        with pytest.raises(ValueError, match=f"{what}: .*contiguous"):
            tg.layer_norm_backward(*args, None, mean, rstd)
    flat = full.view(-1, to[-1])
    close(y.view_as(flat), L.forward(host(flat), None, None, EPS)[0],
          L.forward_bounds(host(flat), None, None, EPS, "f32", 17)[0], "y")


def test_more_columns_than_one_launch_has_threads_for():
    """2^27 + 33 columns, of which 32 threads each add up the sums over rows. With x of 1 and -1,
    a mean of 0 and a deviation of 1 every product is exact, and one row's sums are its own values."""
    cols = (1 << 27) + 33
    print("CASE layer norm 1 x 2^27 + 33", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(17)
    dy = torch.randn(1, cols, generator=gen, device="cuda").bfloat16()
    x = torch.ones_like(dy)
    x[:, ::3] = -1
    mean, rstd = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    dx, dw, db = tg.layer_norm_backward(dy, x, None, mean, rstd)
    assert torch.equal(db, dy[0]) and torch.equal(dw, (dy * x)[0])
    s, u, h = (float(t.sum(dtype=torch.float64)) / cols for t in (dy, dy * x, dy.abs()))
    bound = 2 * L.gamma(cols / 1024 + 26) * h
    for r in (slice(0, 4096), slice(cols - 4096, cols)):
        true = host(dy[0, r]) - s - host(x[0, r]) * u
        close(dx[0, r], true, bound + L.rounding(np.abs(true) + bound, "bf16"), "dx")


@pytest.mark.parametrize("rows", [(1 << 16) + 3, (1 << 22) + 1])
def test_many_rows_beyond_the_registers(rows):
    """Rows of 16385 columns, a workgroup each at a time: more than one launch of them, and more
    than one launch's threads. Rows of zeros but for some; each comes out as in a call on it alone."""
    import gc
    cols, dt = 16385, torch.bfloat16
    gc.collect()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 4 * rows * cols + (8 << 30):
        pytest.skip("needs x and one more tensor of its size")
    print(f"CASE layer norm {rows} x {cols}", flush=True)
    x = torch.zeros(rows, cols, dtype=dt, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(18)
    some = torch.tensor([0, 1, (1 << 16) - 1, 1 << 16, rows - 2, rows - 1], device="cuda")
    x[some] = torch.randn(6, cols, generator=gen, device="cuda").to(dt)
    w = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda"))
    few = tg.layer_norm_forward(x[some], w, w)
    zero = tg.layer_norm_forward(x[2:3], w, w)
    y, mean, rstd = tg.layer_norm_forward(x, w, w)
    mine = torch.zeros(rows, dtype=torch.bool, device="cuda")
    mine[some] = True
    for got, one, none in zip((y, mean, rstd), few, zero):
        assert torch.equal(got[some], one)
        assert torch.equal(got[:64][~mine[:64]], none.expand_as(got[:64])[~mine[:64]])
    assert bool((mean[~mine] == zero[1]).all()) and bool((rstd[~mine] == zero[2]).all())
    middle = slice(rows // 2, rows // 2 + 64)
    assert torch.equal(y[middle], zero[0].expand(64, cols))
    del y, got, one, none
    torch.cuda.empty_cache()
    dx = tg.layer_norm_backward(x, x, w, mean, rstd, params=False)[0]
    assert torch.equal(dx[some], tg.layer_norm_backward(x[some], x[some], w, mean[some], rstd[some], params=False)[0])
    assert not dx[middle].any() and not dx[2:64].any()
    del x, dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,cols", [(70000, 8), (300000, 5), (66000, 64), (300000, 255), (4097, 256), (1000, 333),
                                       (2500, 1024), (40000, 2001), (20000, 4096), (8192, 8192), (3000, 9001),
                                       (131, 16384), (2000, 16384), (513, 20000), (1, 70001)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gap", [0, 1])
def test_every_row_counts_once_in_the_sums(rows, cols, dtype, gap):
    """x at a distance of 1 / rstd from its mean, whole gradients from 1 to 7: products and sums
    below 2^24 are exact in any order, and a row that is lost or taken twice shows."""
    print(f"CASE layer norm sums {rows} x {cols} {dtype} gap {gap}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(19)
    t = tg.torch_dtype(dtype)

    def whole(lo, hi, *s):
        return torch.randint(lo, hi, s, generator=gen, device="cuda", dtype=torch.int32)

    sign, dy, mean, e = (whole(0, 2, rows, cols) * 2 - 1).char(), whole(1, 8, rows, cols).char(), whole(-8, 9, rows), whole(0, 3, rows)
    x = torch.zeros(rows, cols + gap, dtype=t, device="cuda")[:, :cols]
    g = torch.zeros(rows, cols + gap, dtype=t, device="cuda")[:, :cols]
    x.copy_(mean[:, None] + (sign << e[:, None]))
    g.copy_(dy)
    w = torch.ones(cols, device="cuda")
    dw, db = tg.layer_norm_backward(g, x, w, mean.float(), torch.exp2(-e.float()))[1:]
    assert torch.equal(dw, (sign * dy).sum(0, dtype=torch.int64).float())
    assert torch.equal(db, dy.sum(0, dtype=torch.int64).float())


@pytest.mark.parametrize("rows,cols", [(70000, 8), (66000, 64), (300000, 255), (40000, 2001), (20000, 4096)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sums_over_many_rows_as_near_as_their_depth_allows(rows, cols, dtype):
    """A thread adds at most rows / 256 of its own (a walk takes 256 rows at a time or more where
    they are this many), then come up to 64 + 4 of its workgroup's and 768 / 32 + 32 of the
    workgroups'."""
    x, dy, w, _ = inputs(rows, cols, dtype, "f32", seed=20)
    _, mean, rstd = tg.layer_norm_forward(x, w)
    dw, db = tg.layer_norm_backward(dy, x, w, mean, rstd)[1:]
    bound = L.gamma(rows / 256 + 68 + 56)
    n = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for got, terms, what in ((dw, dy.double() * n, "dweight"), (db, dy.double(), "dbias")):
        true = host(terms.sum(0))
        close(got, true, bound * host(terms.abs().sum(0)) + L.rounding(np.abs(true), "f32"), what)


@pytest.mark.parametrize("rows", [255, 256, 257])
@pytest.mark.parametrize("cols", [2050, 9001, 16384])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_some_hundred_long_rows(rows, cols, dtype):
    check(*inputs(rows, cols, dtype, "f32", seed=21), dtype, "f32")
