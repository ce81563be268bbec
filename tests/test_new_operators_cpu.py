"""CPU-only: the oracles of AdamW and layer norm against differences, torch and closed forms,
and the argument checks of their C functions that need no device."""
import ctypes
import os

import numpy as np
import pytest

import oracle.adamw_oracle as A
import oracle.layernorm_oracle as L
import tensor_gradient_compression_amd as tg


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tg.LIB_PATH):
        from tensor_gradient_compression_amd import build
        build.build(verbose=False)
    return tg.load_library()


def test_adamw_oracle_is_torchs():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    w = torch.from_numpy(rng.standard_normal(50)).requires_grad_()
    opt = torch.optim.AdamW([w], lr=1e-2, betas=(0.8, 0.97), eps=1e-6, weight_decay=0.1)
    x, m, v = w.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        w.grad = torch.from_numpy(g.copy())
        opt.step()
        x, m, v = A.step64(x, g, m, v, t, 1e-2, 0.8, 0.97, 1e-6, 0.1)
        np.testing.assert_allclose(x, w.detach().numpy(), rtol=1e-13)


@pytest.mark.parametrize("bits", [A.M_BITS, A.Q_BITS])
def test_codes_are_a_grid(bits):
    """All codes of a group: ascending, exact in bf16, and a value on the grid stays there for
    any random bits."""
    n = 121 if bits == A.M_BITS else 241      # a group's largest is below 2^(f - 126): code 120 or 240
    f = np.full(2, 120, np.uint8)
    code = np.zeros(256, np.int64)
    code[:n] = np.arange(n)
    val = A.decode(code, f, bits)[:n]
    assert np.all(np.diff(val) > 0) and val[0] == 0
    top = 2.0 ** (120 - 126)
    assert val[-1] == top
    mant = np.frexp(val)[0] * 2 ** (bits + 1)
    assert np.array_equal(mant, np.round(mant))
    grid = np.zeros(256)
    grid[:n - 1] = val[:-1]
    for low in (0, (1 << 19) - 1):
        again = A.encode_exact(grid, f, bits, np.full(256, low), 19)
        assert np.array_equal(again, grid)


def test_rounding_goes_up_with_its_share():
    """Half way between two codes, half of the random numbers go up."""
    f = np.array([120], np.uint8)
    unit, pos = A.unit_and_position(np.full(128, 2.0 ** -7 * 1.0625), f, 3)
    assert np.all(pos == 8.5)
    low = np.arange(128) * (1 << 13)
    got = A.encode_exact(np.full(128, 2.0 ** -7 * 1.0625), f, 3, low, 20) / unit
    assert (got == 8).sum() == 64 and (got == 9).sum() == 64


def test_random_bits_are_even():
    """Each of the 32 bits is set in half of 2^16 places within 6 standard deviations, in two
    steps, and the steps' bits differ in half."""
    n = 1 << 16
    a, b = A.random_bits(3, 1, np.arange(n)), A.random_bits(3, 2, np.arange(n))
    for h in (a, b, a ^ b):
        for k in range(32):
            assert abs(int(((h >> np.uint32(k)) & np.uint32(1)).sum()) - n / 2) < 6 * np.sqrt(n) / 2


def test_layer_norm_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 5)), rng.standard_normal((3, 5))
    w, b = rng.standard_normal(5), rng.standard_normal(5)

    def f(x, w, b):
        return (L.forward(x, w, b, 1e-3)[0] * dy).sum()

    mean, rstd = L.statistics(x, 1e-3)
    grads = L.backward(dy, x, w, mean, rstd)
    h = 1e-6
    for k, (arr, g) in enumerate(zip((x, w, b), grads)):
        for i in np.ndindex(arr.shape):
            args = [x.copy(), w.copy(), b.copy()]
            args[k][i] += h
            up = f(*args)
            args[k][i] -= 2 * h
            assert abs((up - f(*args)) / (2 * h) - g[i]) < 1e-8


I64, INT, DBL, P = ctypes.c_int64, ctypes.c_int, ctypes.c_double, ctypes.c_void_p


def arr(t, v):
    return (t * max(len(v), 1))(*v)


def test_state_sizes(lib):
    n, d = arr(I64, [1, 128, 129, 0]), arr(INT, [0, 1, 2, 3])
    assert lib.tgrad_adamw_state_values(4, n, d) == 128 + 128 + 256
    assert lib.tgrad_adamw_state_bytes(4, n, d, 32) == 512 * 8
    assert lib.tgrad_adamw_state_bytes(4, n, d, 8) == 512 * 2 + 8
    assert lib.tgrad_adamw_state_values(1, arr(I64, [65]), arr(INT, [3])) == 256
    for bad in (lib.tgrad_adamw_state_bytes(4, n, d, 16), lib.tgrad_adamw_state_values(0, n, d),
                lib.tgrad_adamw_state_values(1, arr(I64, [-1]), d), lib.tgrad_adamw_state_values(1, n, arr(INT, [4])),
                lib.tgrad_adamw_state_values(1, None, d), lib.tgrad_adamw_state_values(1, n, None)):
        assert bad == -1


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(numel=[-1]), dict(dtype=[9]), dict(grad=[1]), dict(dtype=[1], grad=[2]), dict(wd=[-1.0]),
    dict(wd=[float("nan")]), dict(bits=16), dict(lr=-1.0), dict(lr=float("inf")), dict(b1=1.0), dict(b2=-0.1),
    dict(eps=-1.0), dict(eps=float("nan")), dict(state=0), dict(state=8),
])
def test_adamw_init_refuses(lib, kw):
    a = dict(n=1, numel=[4], dtype=[0], grad=None, wd=[0.0], bits=32, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, state=4096)
    a.update(kw)
    h = P(1)
    rc = lib.tgrad_adamw_init(ctypes.byref(h), a["n"], arr(I64, a["numel"]), arr(INT, a["dtype"]),
                              arr(INT, a["grad"] or a["dtype"]), arr(DBL, a["wd"]), a["bits"], a["lr"], a["b1"],
                              a["b2"], a["eps"], 0, P(a["state"]))
    assert rc == tg.EINVAL and not h.value


def test_null_handles(lib):
    n = I64()
    assert lib.tgrad_adamw_destroy(None) == tg.OK
    assert lib.tgrad_adamw_step(None, None, None, None, None, None, None) == tg.EINVAL
    assert lib.tgrad_adamw_grad_norm(None, None, 1.0, 1.0, None, None) == tg.EINVAL
    assert lib.tgrad_adamw_set_lr(None, 1.0) == tg.EINVAL
    assert lib.tgrad_adamw_get_steps(None, ctypes.byref(n)) == tg.EINVAL
    assert lib.tgrad_adamw_set_steps(None, 0) == tg.EINVAL
    assert lib.tgrad_adamw_last_error(None) == b""


def test_layer_norm_refuses(lib):
    def fwd(x=4096, stride=8, w=None, b=None, y=4096, mean=4096, rstd=4096, rows=2, cols=8, dt=0, wdt=0, eps=1e-5):
        return lib.tgrad_layer_norm_forward(P(x), stride, P(w), P(b), P(y), P(mean), P(rstd), rows, cols, dt, wdt,
                                            eps, None)

    for kw in (dict(x=None), dict(y=None), dict(mean=None), dict(rstd=None), dict(rows=-1), dict(cols=0), dict(dt=3),
               dict(wdt=1), dict(dt=1, wdt=2), dict(stride=7), dict(x=4098), dict(w=4098), dict(b=2),
               dict(eps=-1.0), dict(eps=float("nan")), dict(rows=1 << 31), dict(cols=1 << 31)):
        assert fwd(**kw) == tg.EINVAL, kw
    assert fwd(rows=0, x=None, y=None, mean=None, rstd=None) == tg.OK

    def bwd(dy=4096, dstr=8, x=4096, xstr=8, w=None, mean=4096, rstd=4096, dx=4096, dw=4096, db=4096, rows=2, cols=8,
            dt=0, wdt=0, ws=4096):
        return lib.tgrad_layer_norm_backward(P(dy), dstr, P(x), xstr, P(w), P(mean), P(rstd), P(dx), P(dw), P(db),
                                             rows, cols, dt, wdt, P(ws), None)

    for kw in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(ws=None),
               dict(ws=4100), dict(dstr=7), dict(xstr=7), dict(dw=4098), dict(db=4097), dict(dt=3), dict(cols=0)):
        assert bwd(**kw) == tg.EINVAL, kw
    assert lib.tgrad_layer_norm_workspace(-1, 8) == -1 and lib.tgrad_layer_norm_workspace(1, 0) == -1
    assert lib.tgrad_layer_norm_workspace(5, 8) > 0


@pytest.mark.parametrize("lacks", ["torch", "a C++ compiler"])
def test_the_library_builds_without_what_the_binding_needs(lacks, tmp_path, monkeypatch, capsys):
    """libtgrad.so is a C library: hipcc is enough for it."""
    import importlib.util
    from tensor_gradient_compression_amd import build
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.hip").write_text('extern "C" int one() { return 1; }\n')
    for name, at in (("CSRC", src), ("BUILD", tmp_path / "_build"), ("LIB", tmp_path / "libtgrad.so"),
                     ("BINDING", tmp_path / "_tgrad_torch.so")):
        monkeypatch.setattr(build, name, str(at))
    if lacks == "torch":
        monkeypatch.setattr(importlib.util, "find_spec", lambda *a: None)
        build.build()
        assert "torch" in capsys.readouterr().out
    else:
        def fails():
            raise RuntimeError("g++ not found")
        monkeypatch.setattr(build, "_compile_binding", fails)
        with pytest.raises(RuntimeError, match="g\\+\\+"):
            build.build()
    assert ctypes.CDLL(build.LIB).one() == 1
    assert not os.path.exists(build.BINDING)


@pytest.mark.parametrize("numel,dtype", [([1 << 40], 0), ([1 << 40], 3), ([1 << 38, 1], 2), ([1 << 39] * 4, 1)])
def test_adamw_init_refuses_more_than_a_card_could_hold(lib, numel, dtype):
    """Before tables of 80 bytes for every 2048 values take the host's memory."""
    h, n = P(1), len(numel)
    rc = lib.tgrad_adamw_init(ctypes.byref(h), n, arr(I64, numel), arr(INT, [dtype] * n), arr(INT, [dtype] * n),
                              arr(DBL, [0.0] * n), 8, 1e-3, 0.9, 0.99, 1e-8, 0, P(4096))
    assert rc == tg.EINVAL and not h.value
