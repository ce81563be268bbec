"""CPU-only: the oracles of orthogonalisation, the Muon step and the gated linear layer against
closed forms, differences and torch, and the argument checks of their C functions."""
import ctypes
import os

import numpy as np
import pytest

import oracle.gated_oracle as G
import oracle.muon_oracle as M
import tensor_gradient_compression_amd as tg


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tg.LIB_PATH):
        from tensor_gradient_compression_amd import build
        build.build(verbose=False)
    return tg.load_library()


# ---------------------------------------------------------------- oracles

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (6, 1), (5, 5), (4, 9), (9, 4)])
def test_orthogonalisation_is_a_polynomial_of_singular_values(rows, cols):
    rng = np.random.default_rng(rows * 10 + cols)
    g = rng.standard_normal((rows, cols))
    u, s, v = np.linalg.svd(g, full_matrices=False)
    s = s / (np.linalg.norm(s) + 1e-7)
    a, b, c = M.COEFFICIENTS
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    np.testing.assert_allclose(M.orthogonalize(g), u * s @ v, atol=1e-12)


def test_orthogonalisation_of_zeros_and_of_any_size():
    assert not M.orthogonalize(np.zeros((3, 4))).any()
    g = np.random.default_rng(0).standard_normal((6, 4))
    np.testing.assert_allclose(M.orthogonalize(1e20 * g, eps=0.0), M.orthogonalize(g, eps=0.0), atol=1e-12)
    np.testing.assert_allclose(M.orthogonalize(g.T), M.orthogonalize(g).T, atol=1e-12)


def few_strong(m, n, rng, strong=16, noise=0.01):
    return rng.standard_normal((m, strong)) @ rng.standard_normal((strong, n)) + noise * rng.standard_normal((m, n))


def test_the_parts_keep_weak_directions():
    """16 strong directions and 1% of noise, whose directions the five steps raise by up to 485.
    An X held in fp16 alone is rounded in all of its 128 left directions; with X in two parts the
    rounding enters by B alone, whose weight lies in the 16 strong ones: nearer by the root of
    128 / 16 at least."""
    g = few_strong(128, 160, np.random.default_rng(1))
    true = M.orthogonalize(g)
    a, b, c = M.COEFFICIENTS
    x = M.start(g, 1e-7)
    for _ in range(5):
        x = M.parts(x, 4096.0)[0].astype(np.float64)
        p = x @ x.T
        x = a * x + (b * p + c * p @ p) @ x
    near = np.linalg.norm(M.in_parts(g, "bf16") - true)
    assert np.sqrt(128 / 16) * near < np.linalg.norm(x - true)
    assert np.linalg.norm(M.in_parts(g, "f32") - true) < 1e-4 * np.linalg.norm(true)


def test_muon_step_is_torchs_recipe():
    """The momentum by torch's lerp, with and without Nesterov's, and the decoupled decay."""
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(2)
    w, g, m = (rng.standard_normal((5, 7)) for _ in range(3))
    for nesterov in (True, False):
        buf = torch.from_numpy(m.copy())
        buf.lerp_(torch.from_numpy(g), 1 - 0.9)
        u = torch.from_numpy(g).lerp(buf, 0.9) if nesterov else buf
        new, mom = M.step(w, g, m, 0.1, 0.9, 0.02, 0.7, nesterov)
        np.testing.assert_allclose(mom, buf.numpy(), atol=1e-14)
        np.testing.assert_allclose(new, w * (1 - 0.002) - 0.07 * M.orthogonalize(u.numpy()), atol=1e-12)


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid", "relu"])
def test_gated_gradients_are_difference_quotients(act):
    rng = np.random.default_rng(3)
    args = [rng.standard_normal(s) for s in ((4, 3), (5, 3), (5, 3), (5,), (5,))]
    dy = rng.standard_normal((4, 5))
    grads = G.backward(dy, *args, act)
    h = 1e-6
    for k, (arr, g) in enumerate(zip(args, grads)):
        for i in np.ndindex(arr.shape):
            moved = [x.copy() for x in args]
            moved[k][i] += h
            up = (G.forward(*moved, act) * dy).sum()
            moved[k][i] -= 2 * h
            assert abs((up - (G.forward(*moved, act) * dy).sum()) / (2 * h) - g[i]) < 1e-7


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid", "relu"])
def test_activations_are_torchs(act):
    torch = pytest.importorskip("torch")
    g = torch.linspace(-30, 30, 601, dtype=torch.float64, requires_grad=True)
    f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "sigmoid": torch.sigmoid,
         "relu": torch.relu}[act]
    y = f(g)
    y.sum().backward()
    a, s = G.activate(g.detach().numpy(), act)
    np.testing.assert_allclose(a, y.detach().numpy(), atol=1e-14)
    np.testing.assert_allclose(s, g.grad.numpy(), atol=1e-13)


# ---------------------------------------------------------------- refusals of the C functions

I64, INT, DBL, P = ctypes.c_int64, ctypes.c_int, ctypes.c_double, ctypes.c_void_p
CO = (DBL * 3)(*M.COEFFICIENTS)


def arr(t, v):
    return (t * max(len(v), 1))(*v)


def test_orthogonalize_refuses(lib):
    def call(x=4096, mstr=12, rstr=4, out=8192, n=2, rows=3, cols=4, dt=0, steps=5, co=CO, eps=1e-7, ws=4096):
        return lib.tgrad_orthogonalize(P(x), mstr, rstr, P(out), n, rows, cols, dt, steps, co, eps, P(ws), None)

    inf = (DBL * 3)(1.0, float("inf"), 0.0)
    for kw in (dict(x=None), dict(out=None), dict(ws=4104), dict(x=4098), dict(out=4097), dict(n=-1),
               dict(rows=0), dict(cols=0), dict(rows=(1 << 19) + 1), dict(cols=1 << 20), dict(dt=3), dict(dt=-1),
               dict(steps=0), dict(steps=101), dict(co=None), dict(co=inf), dict(eps=-1.0), dict(eps=float("nan")),
               dict(rstr=3), dict(mstr=11), dict(n=1 << 22, mstr=12)):
        assert call(**kw) == tg.EINVAL, kw
    assert call(ws=None, rows=300, cols=400, rstr=400, mstr=120000) == tg.EINVAL
    assert call(n=0, x=None, out=None, ws=None) == tg.OK
    assert lib.tgrad_orthogonalize_workspace(2, 300, 400, 0) > 0
    for bad in ((-1, 3, 4, 0), (1, 0, 4, 0), (1, 3, 0, 0), (1, 3, 4, 3), (1 << 40, 3, 4, 0), (1 << 20, 1 << 19, 1 << 19, 0)):
        assert lib.tgrad_orthogonalize_workspace(*bad) == -1


def test_muon_sizes(lib):
    def values(count, rows, cols):
        return lib.tgrad_muon_state_values(len(rows), arr(I64, count), arr(I64, rows), arr(I64, cols))

    assert values([1, 2, 0], [3, 8, 5], [4, 16, 5]) == 128 + 256
    for bad in (([-1], [3], [4]), ([1], [0], [4]), ([1], [3], [0]), ([1], [(1 << 19) + 1], [4]), ([1 << 39], [64], [64]),
                ([], [], [])):
        assert values(*bad) == -1
    assert lib.tgrad_muon_state_values(1, None, arr(I64, [1]), arr(I64, [1])) == -1


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(count=[-1]), dict(rows=[0]), dict(cols=[0]), dict(dtype=[3]), dict(dtype=[9]), dict(grad=[1]),
    dict(dtype=[1], grad=[2]), dict(wd=[-1.0]), dict(wd=[float("nan")]), dict(scale=[-1.0]), dict(scale=[float("inf")]),
    dict(lr=-1.0), dict(lr=float("inf")), dict(mu=1.0), dict(mu=-0.1), dict(steps=0), dict(steps=101),
    dict(co=(1.0, float("nan"), 1.0)), dict(eps=-1.0), dict(state=0), dict(state=8), dict(count=[1 << 22]),
    dict(count=[1 << 12], rows=[1 << 19], cols=[1 << 10]),
])
def test_muon_init_refuses(lib, kw):
    a = dict(n=1, count=[1], rows=[3], cols=[4], dtype=[0], grad=None, wd=[0.0], scale=[1.0], lr=1e-3, mu=0.9, steps=5,
             co=M.COEFFICIENTS, eps=1e-7, state=4096)
    a.update(kw)
    h = P(1)
    rc = lib.tgrad_muon_init(ctypes.byref(h), a["n"], arr(I64, a["count"]), arr(I64, a["rows"]), arr(I64, a["cols"]),
                             arr(INT, a["dtype"]), arr(INT, a["grad"] or a["dtype"]), arr(DBL, a["wd"]),
                             arr(DBL, a["scale"]), a["lr"], a["mu"], 1, a["steps"], (DBL * 3)(*a["co"]), a["eps"],
                             P(a["state"]))
    assert rc == tg.EINVAL and not h.value


def test_muon_null_handles(lib):
    assert lib.tgrad_muon_destroy(None) == tg.OK
    assert lib.tgrad_muon_step(None, None, None, None, None) == tg.EINVAL
    assert lib.tgrad_muon_set_lr(None, 1.0) == tg.EINVAL
    assert lib.tgrad_muon_last_error(None) == b""


def test_gated_linear_refuses(lib):
    def fwd(x=4096, xstr=8, wg=4096, wu=4096, bg=None, bu=None, y=4096, rows=2, i=8, h=5, dt=0, act=0, ws=4096):
        return lib.tgrad_gated_linear_forward(P(x), xstr, P(wg), P(wu), P(bg), P(bu), P(y), rows, i, h, dt, act, P(ws), None)

    for kw in (dict(x=None), dict(y=None), dict(wg=None), dict(wu=None), dict(ws=None), dict(ws=4104), dict(rows=-1),
               dict(i=0), dict(h=0), dict(dt=3), dict(act=4), dict(act=-1), dict(xstr=7), dict(x=4098), dict(wg=4097),
               dict(wu=4098), dict(bg=4098), dict(bu=4097), dict(y=4098), dict(rows=1 << 31), dict(i=(1 << 19) + 1),
               dict(h=1 << 20)):
        assert fwd(**kw) == tg.EINVAL, kw
    assert fwd(rows=0, x=None, y=None, ws=None) == tg.OK

    def bwd(dy=4096, dstr=5, x=4096, xstr=8, wg=4096, wu=4096, bg=None, bu=None, dx=4096, dwg=4096, dwu=4096, dbg=4096,
            dbu=4096, rows=2, i=8, h=5, dt=0, act=0, ws=4096):
        return lib.tgrad_gated_linear_backward(P(dy), dstr, P(x), xstr, P(wg), P(wu), P(bg), P(bu), P(dx), P(dwg), P(dwu),
                                               P(dbg), P(dbu), rows, i, h, dt, act, P(ws), None)

    for kw in (dict(dy=None), dict(x=None), dict(wg=None), dict(wu=None), dict(ws=None), dict(ws=4100), dict(dstr=4),
               dict(xstr=7), dict(dwg=None), dict(dwu=None), dict(dbg=None), dict(dbu=None), dict(dx=4098), dict(dwg=4097),
               dict(dbu=4098), dict(dt=3), dict(act=9), dict(rows=-1), dict(h=0)):
        assert bwd(**kw) == tg.EINVAL, kw


def test_gated_linear_workspace(lib):
    def size(x=4096, xstr=16, wg=4096, wu=4096, rows=10, i=16, h=24, dt=2, back=0):
        return lib.tgrad_gated_linear_workspace(P(x), xstr, P(wg), P(wu), rows, i, h, dt, back)

    assert size() == 0                        # everything lies as the products take it
    assert size(back=1) >= 10 * 2 * 24 * 2
    for kw in (dict(x=4098), dict(xstr=17), dict(wg=4104), dict(wu=4098), dict(i=15, xstr=15), dict(dt=0)):
        assert size(**kw) > 0, kw
    for kw in (dict(rows=-1), dict(i=0), dict(h=0), dict(dt=3), dict(xstr=15), dict(i=1 << 20, xstr=1 << 20)):
        assert size(**kw) == -1, kw


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refuses_what_is_not_on_a_gpu(lib):
    torch = pytest.importorskip("torch")
    x, w, b = torch.zeros(2, 8), torch.zeros(4, 8), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        tg.orthogonalize(x)
    with pytest.raises(ValueError, match="GPU"):
        tg.gated_linear_forward(x, w, w, b, b)
    with pytest.raises(ValueError, match="dtype"):
        tg.orthogonalize(x.double())
    with pytest.raises(ValueError, match="Tensor"):
        tg.orthogonalize([1.0])
    with pytest.raises(ValueError, match="activation"):
        tg.gated_linear_forward(x, w, w, activation="tanh")
    with pytest.raises(ValueError):
        tg.orthogonalize(x, coefficients=(1.0, 2.0))


@pytest.mark.parametrize("kw", [
    dict(shapes=[]), dict(shapes=[(3,)]), dict(shapes=[(0, 4)]), dict(shapes=[(4, 0)]), dict(dtypes="c64"),
    dict(dtypes=["f32", "f32"]), dict(scale="large"), dict(scale=[1.0, 2.0]), dict(weight_decay=[0.1, 0.1]),
    dict(coefficients=(1.0, 2.0)), dict(shapes=[(1 << 20, 4)]),
])
def test_muon_refuses(kw):
    pytest.importorskip("torch")
    a = dict(shapes=[(3, 4)], dtypes="f32")
    a.update(kw)
    with pytest.raises(ValueError):
        tg.Muon(a.pop("shapes"), a.pop("dtypes"), **a)
