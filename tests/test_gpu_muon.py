"""GPU: Newton-Schulz orthogonalisation and the Muon step against the 64-bit oracle, within
what the kernels' formats allow (oracle/muon_oracle.py)."""
import ctypes
import math

import numpy as np
import pytest

import oracle.muon_oracle as M
import tensor_gradient_compression_amd as tg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = ["f32", "f16", "bf16"]
SHAPES = [(1, 1), (1, 9), (9, 1), (2, 3), (8, 8), (5, 200), (200, 5), (63, 65), (64, 64), (65, 63), (130, 72), (72, 130),
          (257, 100), (100, 257), (128, 128)]


def host(t):
    return t.detach().double().cpu().numpy()


def matrix(gen, rows, cols):
    """Directions of falling size and noise, as a gradient's."""
    k = min(rows, cols) // 4 + 1
    x = torch.randn(rows, k, generator=gen, device="cuda") / torch.arange(1, k + 1, device="cuda")
    return x @ torch.randn(k, cols, generator=gen, device="cuda") + 0.1 * torch.randn(rows, cols, generator=gen, device="cuda")


def near(got, u, dtype, what, size=1.0, **ns):
    """`got` against size times the orthogonalised u, rounded to dtype."""
    true = M.orthogonalize(u, **ns)
    e2, em = M.bounds(u, true, dtype, **ns)
    off, r = host(got) - size * true, M.HALF_ULP[dtype]
    a, b = np.linalg.norm(off), size * e2 + r * np.linalg.norm(size * true)
    assert a <= b, f"{what}: 2-norm {a / b:.3g} of the bound"
    a, b = np.abs(off), size * em + M.rounding(size * true, dtype) + r * size * em
    assert np.all(a <= b), f"{what}: {np.max(a / b):.3g} of the bound"


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_orthogonalize(rows, cols, dtype):
    print(f"CASE orthogonalize {rows} x {cols} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(rows * 7 + cols)
    x = (0.01 * matrix(gen, rows, cols)).to(tg.torch_dtype(dtype))
    y = tg.orthogonalize(x)
    assert y.shape == x.shape and y.dtype == x.dtype and y.is_contiguous()
    near(y, host(x), dtype, "orthogonalize")


@pytest.mark.parametrize("rows,cols,dtype", [(700, 530, "bf16"), (530, 700, "f16"), (1100, 260, "f32"), (300, 2050, "bf16")])
def test_orthogonalize_over_several_tiles(rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = matrix(gen, rows, cols).to(tg.torch_dtype(dtype))
    near(tg.orthogonalize(x), host(x), dtype, "orthogonalize")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("count,rows,cols", [(3, 20, 33), (300, 8, 8), (40, 64, 64), (7, 130, 70)])
def test_stacks(dtype, count, rows, cols):
    """Every matrix of a stack is as it is alone, bit for bit where its tiles are the same."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.stack([matrix(gen, rows, cols) for _ in range(count)]).to(tg.torch_dtype(dtype))
    y = tg.orthogonalize(x)
    for i in range(0, count, max(1, count // 4)):
        near(y[i], host(x[i]), dtype, f"matrix {i}")
    y4 = tg.orthogonalize(x.view(1, count, 1, rows, cols))
    assert torch.equal(y4.view_as(y), y)


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(dtype):
    """Rows and matrices apart, unaligned starts; what lies between is NaN."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.stack([matrix(gen, 21, 37) for _ in range(3)]).to(tg.torch_dtype(dtype))
    y = tg.orthogonalize(x)
    buf = torch.full((1 + 3 * 25 * 41,), float("nan"), device="cuda").to(x.dtype)
    v = buf[1:].view(3, 25, 41)[:, :21, :37]
    v.copy_(x)
    assert torch.equal(tg.orthogonalize(v), y)
    near(tg.orthogonalize(v[1]), host(x[1]), dtype, "one of them")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("steps,coefficients,eps", [(1, (1.5, -0.5, 0.0), 0.0), (8, (2.0, -1.5, 0.5), 1e-3), (3, M.COEFFICIENTS, 1.0)])
def test_other_iterations(dtype, steps, coefficients, eps):
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = matrix(gen, 40, 72).to(tg.torch_dtype(dtype))
    ns = dict(steps=steps, coefficients=coefficients, eps=eps)
    near(tg.orthogonalize(x, **ns), host(x), dtype, "orthogonalize", **ns)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e6, 1e30])
def test_any_size(size):
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = matrix(gen, 30, 20) * size
    near(tg.orthogonalize(x, eps=0.0), host(x), "f32", "orthogonalize", eps=0.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_zeros_and_nan(dtype):
    ty = tg.torch_dtype(dtype)
    x = torch.zeros(3, 20, 30, device="cuda", dtype=ty)
    assert not tg.orthogonalize(x).any()
    gen = torch.Generator(device="cuda").manual_seed(6)
    x[0], x[2] = matrix(gen, 20, 30).to(ty), matrix(gen, 20, 30).to(ty)
    clean = tg.orthogonalize(x)
    x[1, 3, 4] = float("nan")
    y = tg.orthogonalize(x)
    assert y[1].isnan().all() and torch.equal(y[0], clean[0]) and torch.equal(y[2], clean[2])
    assert tg.orthogonalize(x[:0]).shape == (0, 20, 30)


def tensors(shapes, dtype, grad, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w, g = [], []
    for s in shapes:
        n = math.prod(s[:-2])
        w.append((0.02 * torch.randn(*s, generator=gen, device="cuda")).to(tg.torch_dtype(dtype)))
        g.append((0.01 * torch.stack([matrix(gen, *s[-2:]) for _ in range(n)] or [torch.zeros(s[-2:], device="cuda")])
                  [:n].reshape(s)).to(tg.torch_dtype(grad)))
    return w, g


def check_step(opt, w, g, m, before, clip=1.0):
    """The weights w after a step from `before` with momentum m (flat, before)."""
    for i, s in enumerate(opt.shapes):
        n = math.prod(s)
        flat = m[opt.offsets[i]:opt.offsets[i] + n]
        new = host(opt.state["momentum"])[opt.offsets[i]:opt.offsets[i] + n]
        gi = host(g[i]).reshape(-1) * clip
        mom, u = M.momentum(gi, flat, opt.momentum, opt.nesterov)
        # two products and a sum of fp32, of a gradient whose product with the coefficient is one more
        assert np.all(np.abs(new - mom) <= 5 * 2.0 ** -24 * (np.abs(gi) + np.abs(flat)) + 1e-44)
        u, W, B = u.reshape(-1, *s[-2:]), host(w[i]).reshape(-1, *s[-2:]), host(before[i]).reshape(-1, *s[-2:])
        for k in range(len(u)):
            step = opt.lr * opt.scale[i]
            ns = dict(steps=opt.steps, coefficients=opt.coefficients, eps=opt.eps)
            true = M.orthogonalize(u[k], **ns)
            e2, em = M.bounds(u[k], true, opt.dtypes[i], **ns)
            want = B[k] * (1 - opt.lr * opt.weight_decay[i]) - step * true
            mine = 8 * 2.0 ** -24 * (np.abs(B[k]) + step * np.abs(true))
            off = W[k] - want
            r = M.HALF_ULP[opt.dtypes[i]]
            a, b = np.linalg.norm(off), step * e2 + np.linalg.norm(mine) + r * np.linalg.norm(want) + 2.0 ** -25 * len(want)
            assert a <= b, f"tensor {i} matrix {k}: 2-norm {a / b:.3g} of the bound"
            b = step * em + mine + M.rounding(np.abs(want) + step * em, opt.dtypes[i])
            assert np.all(np.abs(off) <= b), f"tensor {i} matrix {k}: {np.max(np.abs(off) / b):.3g} of the bound"


@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("nesterov,scale", [(True, "spectral"), (False, "rms")])
def test_muon_steps(dtype, grad, nesterov, scale):
    """Three steps over matrices of every shape, stacks and an empty stack among them."""
    print(f"CASE muon {dtype} {grad} {nesterov} {scale}", flush=True)
    shapes = [(1, 1), (30, 20), (3, 17, 33), (64, 64), (0, 5, 6), (5, 130), (2, 2, 9, 8), (130, 70)]
    w, _ = tensors(shapes, dtype, grad, 1)
    opt = tg.Muon(shapes, dtype, grad, lr=0.02, momentum=0.9, nesterov=nesterov, weight_decay=0.1, scale=scale)
    for t in range(3):
        _, g = tensors(shapes, dtype, grad, 10 + t)
        before, m = [x.clone() for x in w], host(opt.state["momentum"])
        opt.step(w, g)
        check_step(opt, w, g, m, before)


def test_muon_types_scales_and_decays_of_their_own():
    shapes = [(20, 30), (40, 10), (33, 33)]
    w, g = [], []
    for s, d, k in zip(shapes, ("f32", "bf16", "f16"), ("f32", "f32", "f16")):
        a, b = tensors([s], d, k, 2)
        w += a
        g += b
    opt = tg.Muon(shapes, ["f32", "bf16", "f16"], ["f32", "f32", "f16"], lr=0.1, weight_decay=[0.0, 0.5, 0.1],
                  scale=[0.3, "rms", "spectral"], steps=4)
    before = [x.clone() for x in w]
    opt.step(w, g)
    check_step(opt, w, g, np.zeros(opt.state["momentum"].numel()), before)


def test_more_tensors_than_a_launch_names():
    shapes = [(3 + i % 5, 4 + i % 3) for i in range(500)]
    w, g = tensors(shapes, "f32", "f32", 3)
    opt = tg.Muon(shapes, "f32", lr=0.02)
    before = [x.clone() for x in w]
    opt.step(w, g)
    check_step(opt, w, g, np.zeros(opt.state["momentum"].numel()), before)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_clipping_and_a_step_that_is_left_out(dtype):
    shapes = [(40, 24), (24, 40), (5, 16, 16)]
    w, g = tensors(shapes, dtype, dtype, 4)
    opt = tg.Muon(shapes, dtype, lr=0.02)
    norm = tg.AdamW([x.numel() for x in w], dtype)
    clip = norm.grad_norm(g, max_norm=0.05)
    before = [x.clone() for x in w]
    opt.step(w, g, clip=clip)
    check_step(opt, w, g, np.zeros(opt.state["momentum"].numel()), before, clip=float(clip[1]))
    after, m = [x.clone() for x in w], opt.state["momentum"].clone()
    g[1][3, 3] = float("inf")
    opt.step(w, g, clip=norm.grad_norm(g, max_norm=0.05))
    assert all(torch.equal(a, b) for a, b in zip(w, after)) and torch.equal(m, opt.state["momentum"])


def test_muon_is_orthogonalize():
    """A step from no momentum without decay moves a weight by lr * scale times what orthogonalize
    gives for its gradient (the factor in front of u cancels but for eps)."""
    w, g = tensors([(50, 80)], "f32", "f32", 5)
    opt = tg.Muon([(50, 80)], "f32", lr=0.5, weight_decay=0.0, scale=1.0, eps=0.0)
    before = w[0].clone()
    opt.step(w, g)
    o = tg.orthogonalize(g[0], eps=0.0)
    assert torch.linalg.norm((before - w[0]) / 0.5 - o) <= 1e-5 * torch.linalg.norm(o)


def test_muon_unaligned_tensors():
    """Weights and gradients that start at any element."""
    shapes = [(17, 13), (9, 21)]
    w, g = tensors(shapes, "bf16", "f32", 6)

    def moved(t, by):
        buf = torch.zeros(t.numel() + by, device="cuda", dtype=t.dtype)
        buf[by:].copy_(t.reshape(-1))
        return buf[by:].view(t.shape)

    a, b = (tg.Muon(shapes, "bf16", "f32", lr=0.02) for _ in range(2))
    w2, g2 = [moved(x, 1) for x in w], [moved(x, 3) for x in g]
    a.step(w, g)
    b.step(w2, g2)
    assert all(torch.equal(x, y) for x, y in zip(w, w2))


def test_muon_runs_repeat_replay_and_resume():
    shapes = [(70, 40), (3, 20, 50)]
    grads = [tensors(shapes, "bf16", "bf16", 20 + t)[1] for t in range(4)]

    def fresh():
        return tensors(shapes, "bf16", "bf16", 7)[0], tg.Muon(shapes, "bf16", lr=0.02)

    w, opt = fresh()
    want = []
    for g in grads:
        opt.step(w, g)
        want.append([x.clone() for x in w])
    # replayed, with eager work between
    w, opt = fresh()
    static = [x.clone() for x in grads[0]]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        opt.step(w, static)
    for g, v in zip(grads, want):
        for s, x in zip(static, g):
            s.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(w, v))
    # stopped and resumed, on a stream of its own
    w, opt = fresh()
    for g in grads[:2]:
        opt.step(w, g)
    saved = opt.state_dict()
    opt.close()
    other = tg.Muon(shapes, "bf16", lr=0.02)
    other.load_state_dict(saved)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for g in grads[2:]:
        other.step(w, g, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(w, want[-1]))
    with pytest.raises(ValueError, match="shapes"):
        tg.Muon([(70, 40)], "bf16").load_state_dict(saved)
    with pytest.raises(ValueError, match="momentum"):
        tg.Muon(shapes, "bf16", momentum=0.5).load_state_dict(saved)


def test_muon_set_lr():
    w, g = tensors([(20, 20)], "f32", "f32", 8)
    opt = tg.Muon([(20, 20)], "f32", lr=0.5)
    opt.set_lr(0.01)
    before = [x.clone() for x in w]
    opt.step(w, g)
    check_step(opt, w, g, np.zeros(opt.state["momentum"].numel()), before)
    with pytest.raises(tg.TGradError):
        opt.set_lr(-1.0)


def test_orthogonalize_replays():
    gen = torch.Generator(device="cuda").manual_seed(9)
    a, b = (torch.stack([matrix(gen, 70, 50) for _ in range(3)]) for _ in range(2))
    x = a.clone()
    tg.orthogonalize(x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = tg.orthogonalize(x)
    for v in (a, b, a):
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, tg.orthogonalize(v))


def test_refusals():
    x = torch.zeros(4, 6, 8, device="cuda")
    for bad, match in ((x[..., ::2], "contiguous"), (x.transpose(1, 2), "contiguous"), (x[0, 0], "two axes"),
                       (x[0, :1].expand(6, 8), "overlap"), (x[:1].expand(4, 6, 8), "overlap"), (x[:, :0], "empty"),
                       (x[..., :0], "empty"), (x.to(torch.float64), "dtype"), (x.cpu(), "GPU"),
                       (x.view(2, 2, 6, 8).transpose(0, 1), "strides")):
        with pytest.raises(ValueError, match=match):
            tg.orthogonalize(bad)
    for kw in (dict(steps=0), dict(steps=101), dict(coefficients=(1.0, 2.0))):
        with pytest.raises(ValueError):
            tg.orthogonalize(x, **kw)
    for kw in (dict(eps=-1.0), dict(coefficients=(1.0, float("nan"), 0.0))):
        with pytest.raises(tg.TGradError):
            tg.orthogonalize(x, **kw)
    opt = tg.Muon([(6, 8)], "f32")
    w, g = x[0].clone(), x[1].clone()
    for ws, gs, match in (([w, w], [g], "weights"), ([w], [g, g], "grads"), ([w.half()], [g], "weights"),
                          ([w], [g.half()], "grads"), ([w.T], [g], "weights"), ([w], [g[:5]], "grads"),
                          ([w.cpu()], [g], "weights"), ([w], [None], "grads")):
        with pytest.raises(ValueError, match=match):
            opt.step(ws, gs)
    with pytest.raises(ValueError, match="clip"):
        opt.step([w], [g], clip=torch.zeros(3, device="cuda"))


SPLIT = [(1, 300, 3000, "f32"), (1, 3000, 200, "f16"), (1, 260, 5000, "bf16"), (1, 900, 900, "f16"), (3, 300, 1500, "bf16"),
         (2, 1500, 260, "f32")]


@pytest.mark.parametrize("count,rows,cols,dtype", SPLIT)
def test_sums_that_workgroups_share(count, rows, cols, dtype):
    """Long sums of few tiles: against the oracle, again, and replayed with other work between."""
    print(f"CASE split {count} {rows} {cols} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    a, b = (torch.stack([matrix(gen, rows, cols) for _ in range(count)]).to(tg.torch_dtype(dtype)) for _ in range(2))
    y = tg.orthogonalize(a)
    near(y[-1], host(a[-1]), dtype, "orthogonalize")
    z = tg.orthogonalize(b)
    x = a.clone()
    tg.orthogonalize(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tg.orthogonalize(x)
    for v, w in ((b, z), (a, y), (a, y), (b, z)):
        x.copy_(v)
        graph.replay()
        assert torch.equal(tg.orthogonalize(v), w)
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def test_split_sums_on_two_streams():
    gen = torch.Generator(device="cuda").manual_seed(21)
    xs = [matrix(gen, 300, 2000).half(), matrix(gen, 2000, 280)]
    want = [tg.orthogonalize(x) for x in xs]
    sides, got = [torch.cuda.Stream() for _ in xs], [[], []]
    torch.cuda.synchronize()
    for _ in range(4):
        for i, s in enumerate(sides):
            with torch.cuda.stream(s):
                got[i].append(tg.orthogonalize(xs[i]))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert all(torch.equal(r, w) for r in runs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_muon_steps_of_split_sums(dtype):
    """Matrices that a workgroup holds beside larger ones whose sums are split, twice."""
    shapes = [(300, 2500), (20, 30), (2, 400, 260), (1030, 130)]
    w, _ = tensors(shapes, dtype, dtype, 22)
    opt = tg.Muon(shapes, dtype, lr=0.05, weight_decay=0.1)
    for t in range(2):
        _, g = tensors(shapes, dtype, dtype, 23 + t)
        before, m = [x.clone() for x in w], host(opt.state["momentum"])
        opt.step(w, g)
        check_step(opt, w, g, m, before)


@pytest.mark.parametrize("rows,cols", [(261, 520), (520, 261), (700, 300), (257, 257)])
@pytest.mark.parametrize("dtype", TYPES)
def test_nothing_around_a_matrix_is_read(rows, cols, dtype):
    """A matrix between NaNs, after its workspace's memory held NaNs."""
    gen = torch.Generator(device="cuda").manual_seed(24)
    x = matrix(gen, rows, cols).to(tg.torch_dtype(dtype))
    want = tg.orthogonalize(x)
    buf = torch.full((rows + 8, cols + 40), float("nan"), device="cuda").to(x.dtype)
    v = buf[3:3 + rows, 17:17 + cols]
    v.copy_(x)
    fill = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(8)]
    del fill
    assert torch.equal(tg.orthogonalize(v), want)


def test_weights_that_overlap():
    """Two matrices' workgroups would write the same values."""
    opt = tg.Muon([(6, 8), (4, 8), (0, 3, 3)], "f32")
    buf, g = torch.zeros(12, 8, device="cuda"), torch.zeros(6, 8, device="cuda")
    none = torch.zeros(0, 3, 3, device="cuda")
    for second in (buf[:4], buf[5:9]):
        with pytest.raises(tg.TGradError):
            opt.step([buf[:6], second, none], [g, g[:4], none])
    opt.step([buf[6:], buf[:4], none], [g, g[:4], none])


def test_in_place():
    """The C call's result may be its input."""
    gen = torch.Generator(device="cuda").manual_seed(25)
    for shape in ((40, 30), (300, 700)):
        x = matrix(gen, *shape)
        want = tg.orthogonalize(x)
        lib = tg.load_library()
        n = lib.tgrad_orthogonalize_workspace(1, *shape, 0)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        co = (ctypes.c_double * 3)(*M.COEFFICIENTS)
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert lib.tgrad_orthogonalize(x.data_ptr(), x.numel(), shape[1], x.data_ptr(), 1, *shape, 0, 5, co, 1e-7,
                                       ws.data_ptr(), stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(x, want)


@pytest.mark.parametrize("rows,cols", [(2, 2), (1, 7), (5, 3), (32, 32), (8, 128)])
def test_few_values_in_bf16_are_exact_but_for_their_rounding(rows, cols):
    """Within what fp32 results are off, and half a step."""
    gen = torch.Generator(device="cuda").manual_seed(31)
    x = torch.stack([matrix(gen, rows, cols) for _ in range(6)]).bfloat16()
    for got, u in zip(tg.orthogonalize(x), host(x)):
        true = M.orthogonalize(u)
        e2, em = M.bounds(u, true, "f32")
        assert np.all(np.abs(host(got) - true) <= em + M.rounding(np.abs(true) + em, "bf16"))


@pytest.mark.parametrize("size", [1e-36, 1e-41])
@pytest.mark.parametrize("rows,cols", [(30, 20), (70, 130), (300, 200)])
def test_norms_whose_reciprocal_fp32_does_not_hold(size, rows, cols):
    """eps = 0 and values down to fp32's subnormal ones, for orthogonalize and a Muon step from no
    momentum and weights of zeros (whose update, 0.05 + 0.95 x 0.05 of the gradient, has its direction
    up to four roundings, which among subnormal numbers are 2^-150 each)."""
    gen = torch.Generator(device="cuda").manual_seed(32)
    x = matrix(gen, rows, cols) * size
    near(tg.orthogonalize(x, eps=0.0), host(x), "f32", "orthogonalize", eps=0.0)
    if size < 1e-38:
        return
    w = torch.zeros(rows, cols, device="cuda")
    opt = tg.Muon([(rows, cols)], "f32", lr=1.0, weight_decay=0.0, scale=1.0, eps=0.0)
    opt.step([w], [x])
    near(-w, host(x), "f32", "step", eps=0.0)


def test_shapes_that_are_others():
    """A weight or gradient whose last axes do not form rows of cols values is refused, and not taken as
    another matrix of as many elements; flat values, axes that do form them and several matrices' rows in one
    axis are taken."""
    opt = tg.Muon([(72, 24), (2, 16, 27), (5, 1)], "f32", lr=0.02)

    def given(*shapes):
        gen = torch.Generator(device="cuda").manual_seed(33)
        return [torch.randn(math.prod(s), generator=gen, device="cuda").view(s) for s in shapes]

    right = ((72, 24), (2, 16, 27), (5, 1))
    for i, other in ((0, (24, 72)), (0, (36, 48)), (1, (2, 27, 16)), (1, (27, 32)), (1, (864, 1))):
        bad = [s if k != i else other for k, s in enumerate(right)]
        with pytest.raises(ValueError, match="weights"):
            opt.step(given(*bad), given(*right))
        with pytest.raises(ValueError, match="grads"):
            opt.step(given(*right), given(*bad))
    assert not opt.state["momentum"].any()
    want = None
    for form in (right, ((1728,), (32, 3, 3, 3), (5,)), ((8, 9, 24), (2, 16, 3, 9), (1, 5)), ((72, 2, 12), (32, 27), (5, 1, 1))):
        opt.state["momentum"].zero_()
        w = given(*form)
        opt.step(w, given(*form))
        flat = torch.cat([x.reshape(-1) for x in w])
        want = flat if want is None else want
        assert torch.equal(flat, want)


def test_as_many_matrices_as_a_launch_takes():
    """2^21 of them, each of a workgroup of 1024 threads: a row's only singular value goes through the
    iteration's polynomial from 1 on."""
    n = 1 << 21
    x = torch.ones(n, 1, 288, device="cuda", dtype=torch.bfloat16)
    x[:, 0, 0] = 1 - 2 * (torch.arange(n, device="cuda") % 2)
    y = tg.orthogonalize(x)
    a, b, c = M.COEFFICIENTS
    s = 1.0
    for _ in range(5):
        s = s * (a + b * s ** 2 + c * s ** 4)
    value = s / math.sqrt(288)
    assert torch.all((y * x).float().sub_(value).abs_() <= 2.0 ** -8 * value)


# By 128 x 128 and 256 x 256, in one workgroup a unit and in two, wide and tall, of one product of parts and of
# three, sums whole and shared: A, B and B X each meet all of them among these. (Up to 48 of 500 x 500 A is of 128 x 128
# tiles, from 24 of 1000 x 1000 on 256 x 256; B X of 64 of 500 x 500 is of 256 x 256.)
TILES = [(48, 499, 501, "bf16"), (48, 501, 499, "f16"), (24, 1001, 499, "bf16"), (24, 1001, 499, "f32"), (12, 257, 771, "bf16"),
         (12, 771, 257, "bf16"), (64, 1001, 499, "f16"), (12, 771, 257, "f32"), (12, 257, 771, "f16"), (24, 499, 501, "bf16"),
         (64, 499, 501, "bf16"), (64, 507, 499, "bf16"), (48, 507, 499, "bf16"), (24, 499, 501, "f32"), (64, 499, 501, "f32"),
         (24, 1001, 1003, "bf16"), (24, 999, 1001, "f32"), (24, 1007, 1001, "bf16"), (24, 1555, 777, "f16"),
         (6, 777, 3885, "f16"), (6, 3885, 777, "f32"), (8, 499, 1497, "f32"), (8, 1497, 499, "f16"), (3, 777, 3885, "bf16"),
         (3, 3885, 777, "bf16"), (1, 1501, 1509, "f16"), (1, 1509, 1501, "f32")]


@pytest.mark.parametrize("count,rows,cols,dtype", TILES)
def test_larger_tiles(count, rows, cols, dtype):
    """The first and the last matrix, against the oracle; all of them again, bit for bit."""
    print(f"CASE tiles {count} {rows} {cols} {dtype}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.stack([matrix(gen, rows, cols) for _ in range(count)]).to(tg.torch_dtype(dtype))
    y = tg.orthogonalize(x)
    for i in {0, count - 1}:
        near(y[i], host(x[i]), dtype, f"matrix {i}")
    assert torch.equal(tg.orthogonalize(x), y)


@pytest.mark.parametrize("count,rows,cols,dtype", [(24, 1001, 1003, "bf16"), (24, 1007, 1001, "f16"), (48, 499, 501, "f32")])
def test_muon_steps_by_larger_tiles(count, rows, cols, dtype):
    w, g = tensors([(count, rows, cols)], dtype, dtype, 34)
    opt = tg.Muon([(count, rows, cols)], dtype, lr=0.05, weight_decay=0.1)
    before = [x.clone() for x in w]
    opt.step(w, g)
    # the last matrix alone, as a tensor of its own
    last = tg.Muon([(rows, cols)], dtype, lr=0.05, weight_decay=0.1)
    last.state["momentum"][:rows * cols] = opt.state["momentum"][(count - 1) * rows * cols:count * rows * cols]
    check_step(last, [w[0][-1]], [g[0][-1]], np.zeros(rows * cols), [before[0][-1]])
