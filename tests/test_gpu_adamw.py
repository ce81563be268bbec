"""GPU: AdamW over many tensors through the Python binding, each step against the oracle.

Every step is checked on its own: the oracle starts from the state and weights that the
library had before it. The stored state must follow the fp32 order of operations bit for bit;
weights must be within what those roundings can add up to of the step in 64 bits:
  m: the gradient's scaling, two products and a sum, 4 eps of |b1 m| + |(1 - b1) g|
  q = sqrt(v): six roundings under the root and its own, 4 eps; the denominator 8 eps
  u = step m / denominator: 16 eps of itself beside m's error; w: 4 eps and its own rounding
with eps = 2^-24."""
import math

import numpy as np
import pytest

import oracle.adamw_oracle as A
import tensor_gradient_compression_amd as tg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HALF = {"f32": E, "c64": E, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -150, "c64": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
HYPER = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8)


def values(t):
    """A tensor's real values as float64 (exact)."""
    if t.is_complex():
        t = torch.view_as_real(t)
    return t.detach().reshape(-1).double().cpu().numpy()


def random_tensor(n, dtype, gen, scale, offset=0):
    """n elements that start `offset` elements into their allocation."""
    real = torch.float32 if dtype == "c64" else tg.torch_dtype(dtype)
    per = 2 if dtype == "c64" else 1
    x = torch.randn((n + offset) * per, generator=gen, device="cuda")
    x = x * torch.exp(torch.randn(x.shape, generator=gen, device="cuda")) * scale
    x = x.to(real)
    if dtype == "c64":
        x = torch.view_as_complex(x.view(-1, 2))
    return x[offset:]


class Case:
    """An optimizer with weights of its own and a step that checks itself."""

    def __init__(self, numels, dtypes, grads=None, bits=32, decay=0.01, offset=0, seed=7, hyper=HYPER):
        n = len(numels)
        self.dtypes = [dtypes] * n if isinstance(dtypes, str) else list(dtypes)
        self.gtypes = self.dtypes if grads is None else ([grads] * n if isinstance(grads, str) else list(grads))
        self.decay = [decay] * n if not isinstance(decay, (list, tuple)) else list(decay)
        self.numels, self.bits, self.seed, self.offset, self.hyper = numels, bits, seed, offset, hyper
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w = [random_tensor(m, d, self.gen, 0.02, offset) for m, d in zip(numels, self.dtypes)]
        self.opt = tg.AdamW(numels, self.dtypes, self.gtypes, weight_decay=self.decay, state_bits=bits,
                            seed=seed, **hyper)
        self.t = 0

    def gradients(self, scale=0.01):
        return [random_tensor(m, d, self.gen, scale, self.offset) for m, d in zip(self.numels, self.gtypes)]

    def snapshot(self):
        return [values(w) for w in self.w], {k: v.cpu().numpy().copy() for k, v in self.opt.state.items()}

    def checked_step(self, g, clip=None, moments=None):
        w0, s0 = self.snapshot()
        self.opt.step(self.w, g, clip=clip, moments=moments)
        self.t += 1
        w1, s1 = self.snapshot()
        coef = 1.0 if clip is None else float(clip[1])
        b1, b2 = self.hyper["betas"]
        lr, eps = self.hyper["lr"], self.hyper["eps"]
        for i, n in enumerate(self.numels):
            per = 2 if self.dtypes[i] == "c64" else 1
            gi, vals, at = values(g[i]), n * per, self.opt.offsets[i]
            end = at + -(-vals // A.GROUP) * A.GROUP
            gi_all = np.zeros(end - at)
            gi_all[:vals] = gi
            grp = slice(at // A.GROUP, end // A.GROUP)
            if self.bits == 32:
                m0, v0 = s0["m"][at:end], s0["v"][at:end]
            else:
                m0 = A.decode_m(s0["m"][at:end], s0["m_scale"][grp])
                q0 = A.decode_q(s0["root_v"][at:end], s0["root_v_scale"][grp]).astype(np.float32)
                v0 = q0 * q0
            m32, v32 = A.step32(gi_all.astype(np.float32), m0, v0, b1, b2, np.float32(coef))
            if self.bits == 32:
                assert np.array_equal(s1["m"][at:end], m32), f"tensor {i}: m"
                assert np.array_equal(s1["v"][at:end], v32), f"tensor {i}: v"
            else:
                self.check_codes(i, s1, at, end, grp, m32, np.sqrt(v32), moments)
            w64, m64, v64 = A.step64(w0[i], gi, m0[:vals], v0[:vals], self.t, lr, b1, b2, eps, self.decay[i], coef)
            terms = b1 * np.abs(m0[:vals]) + (1 - b1) * np.abs(gi * coef)
            den = np.sqrt(v64 / (1 - b2 ** self.t)) + eps
            tol = lr / (1 - b1 ** self.t) / den * (4 * E * terms + 16 * E * np.abs(m64)) + 4 * E * np.abs(w0[i])
            tol = tol + (np.abs(w64) + tol) * HALF[self.dtypes[i]] + TINY[self.dtypes[i]]
            off = np.abs(w1[i] - w64)
            assert np.all(off <= tol), f"tensor {i}: w off by {(off / tol).max():.3g} of the bound"

    def check_codes(self, i, s, at, end, grp, m, q, moments):
        places = np.arange(at, end)
        h = A.random_bits(self.seed, self.t, places)
        fm, fq = A.fields(m), A.fields(q)
        assert np.array_equal(s["m_scale"][grp], fm) and np.array_equal(s["root_v_scale"][grp], fq)
        em = A.encode_exact(m, fm, A.M_BITS, h >> 12, 20) * np.sign(m)
        eq = A.encode_exact(q, fq, A.Q_BITS, h & 0x7FFFF, 19)
        eq = np.where(q > 0, np.maximum(eq, A.least(fq, A.Q_BITS)), 0.0)
        gm, gq = A.decode_m(s["m"][at:end], fm), A.decode_q(s["root_v"][at:end], fq)
        assert np.array_equal(gm, em), f"tensor {i}: codes of m"
        assert np.array_equal(gq, eq), f"tensor {i}: codes of sqrt(v)"
        if moments is not None:
            assert np.array_equal(values(moments[0])[at:end], gm)
            assert np.array_equal(values(moments[1])[at:end], gq)

    def moment_buffers(self):
        total = self.opt.state["m"].numel()
        return [torch.full((total,), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]


SIZES = [1, 7, 8, 0, 127, 128, 129, 2047, 2048, 2049, 5000]
TYPES = [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("c64", "c64")]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,grad", TYPES)
@pytest.mark.parametrize("offset", [0, 1])
def test_steps_against_the_oracle(bits, dtype, grad, offset):
    """Sizes around the vector, group and workgroup lengths, aligned and not, from a zero
    state; the second step on meets a real one."""
    print(f"CASE adamw {bits} {dtype} {grad} offset {offset}", flush=True)
    c = Case(SIZES, dtype, grad, bits, decay=[0.01 * (i % 3) for i in range(len(SIZES))], offset=offset)
    mo = c.moment_buffers() if bits == 8 else None
    for k in range(4):
        c.checked_step(c.gradients(10.0 ** -k), moments=mo if k % 2 else None)
    assert c.opt.t == 4


@pytest.mark.parametrize("bits", [32, 8])
def test_mixed_types_and_many_tensors(bits):
    """More tensors than one launch carries, of every type."""
    rng = np.random.default_rng(3)
    n = 2 * 240 + 13
    kinds = [TYPES[i % len(TYPES)] for i in range(n)]
    c = Case([int(x) for x in rng.integers(0, 700, n)], [k[0] for k in kinds], [k[1] for k in kinds], bits)
    for _ in range(2):
        c.checked_step(c.gradients(), clip=c.opt.grad_norm(c.gradients(), max_norm=0.5))


@pytest.mark.parametrize("bits,dtype", [(32, "bf16"), (8, "f16"), (8, "f32")])
def test_chunks_of_several_passes(bits, dtype):
    """Enough values that a workgroup takes several passes over its chunk."""
    c = Case([9_000_011, 300_001], dtype, bits=bits)
    for _ in range(2):
        c.checked_step(c.gradients())


@pytest.mark.parametrize("betas,eps,lr", [((0.0, 0.0), 1e-8, 1e-3), ((0.95, 0.9999), 1e-6, 0.0), ((0.9, 0.99), 0.5, 1.0)])
@pytest.mark.parametrize("bits", [32, 8])
def test_hyperparameters(bits, betas, eps, lr):
    c = Case([1000, 33], "f32", bits=bits, hyper=dict(lr=lr, betas=betas, eps=eps))
    for _ in range(3):
        c.checked_step(c.gradients())


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_and_wide_ranges(bits):
    """Gradients of zero leave zero moments and a decayed weight; within one group, values 2^40
    apart keep a positive sqrt(v), so that no update explodes."""
    c = Case([256, 300], "f32", bits=bits)
    c.checked_step([torch.zeros(256, device="cuda"), torch.zeros(300, device="cuda")])
    w0 = values(c.w[0])
    g = torch.full((256,), 1e-9, device="cuda")
    g[::64] = 1e3
    for _ in range(3):
        c.checked_step([g, g.new_zeros(300)])
    assert np.all(np.abs(values(c.w[0]) - w0) < 3 * 1.1e-3 * 4)
    if bits == 8:
        assert np.all(c.opt.state["root_v"][:256].cpu().numpy() >= 1)
        assert np.all(c.opt.state["root_v"][256:].cpu().numpy() == 0)


@pytest.mark.parametrize("dtype,scale", [("f32", 1.0), ("f32", 1e25), ("f32", 1e-30), ("f16", 100.0), ("bf16", 1e18), ("c64", 1e-3)])
def test_norm_and_coefficient(dtype, scale):
    """fp64 sums: squares far outside fp32's range count; rounded to fp32 once (2^-24; squares
    and sums in fp64 are below that by 2^-20 and more)."""
    n = [5000, 1, 0, 129, 40001]
    c = Case(n, dtype)
    g = c.gradients(scale)
    if dtype == "f16":
        g = [torch.nan_to_num(x) for x in g]
    for max_norm, gs in ((math.inf, 1.0), (0.5 * scale, 1.0), (1e30, 0.125)):
        out = c.opt.grad_norm(g, max_norm=max_norm, grad_scale=gs)
        again = c.opt.grad_norm(g, max_norm=max_norm, grad_scale=gs)
        assert torch.equal(out, again)
        norm, coef = A.norm_and_coefficient([values(x) for x in g], max_norm, gs)
        assert abs(float(out[0]) - norm) <= 1.01 * E * norm + 2.0 ** -150
        assert abs(float(out[1]) - coef) <= 1.01 * E * coef + 2.0 ** -150
    zero = c.opt.grad_norm([torch.zeros_like(x) for x in g], max_norm=1.0)
    assert zero.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("numels", [[0], [0] * 300, [0] * 250 + [70], [70] + [0] * 250, [2048] * 16, [2048] * 17,
                                    [100] * 24, [100] * 25, [100] * 600])
def test_norm_of_few_and_many_tensors(numels):
    """The ways the sums are joined: one workgroup alone, a launch, several launches, none."""
    c = Case(numels, "f32")
    g = c.gradients()
    out = c.opt.grad_norm(g, max_norm=1e-3)
    norm, coef = A.norm_and_coefficient([values(x) for x in g], 1e-3, 1.0)
    assert abs(float(out[0]) - norm) <= 1.01 * E * norm
    assert abs(float(out[1]) - coef) <= 1.01 * E * coef
    for _ in range(2):
        assert torch.equal(out, c.opt.grad_norm(g, max_norm=1e-3))
        c.checked_step(g, clip=out)


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_steps(bits):
    c = Case([4000, 77], "f16", bits=bits)
    for max_norm in (0.1, 1e9):
        g = c.gradients()
        c.checked_step(g, clip=c.opt.grad_norm(g, max_norm=max_norm, grad_scale=0.5))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite_cancels_the_step(bits, bad):
    c = Case([4000, 77], "bf16", bits=bits)
    c.checked_step(c.gradients())
    w0, s0 = c.snapshot()
    g = c.gradients()
    g[1][5] = bad
    clip = c.opt.grad_norm(g, max_norm=1.0)
    assert not math.isfinite(float(clip[0]))
    mo = c.moment_buffers() if bits == 8 else None
    c.opt.step(c.w, g, clip=clip, moments=mo)
    w1, s1 = c.snapshot()
    assert all(np.array_equal(a, b) for a, b in zip(w0, w1))
    assert all(np.array_equal(s0[k], s1[k]) for k in s0)
    assert mo is None or bool(mo[0].isnan().all())
    assert c.opt.t == 1
    c.checked_step(c.gradients())       # and the next one counts as the second
    assert c.opt.t == 2


def test_values_that_are_not_finite_stay_visible():
    """Without the norm: in 32 bits the element alone is lost, in 8 bits its group of 128, and
    stays so."""
    for bits, lost in ((32, 1), (8, 128)):
        c = Case([1024], "f32", bits=bits)
        g = c.gradients()
        g[0][200] = math.inf
        c.opt.step(c.w, g)
        assert int(torch.isfinite(c.w[0]).logical_not().sum()) == 1
        mo = c.moment_buffers() if bits == 8 else None
        c.opt.step(c.w, c.gradients(), moments=mo)
        assert int(torch.isfinite(c.w[0]).logical_not().sum()) == lost
        if mo:
            assert bool(mo[0][128:256].isnan().all()) and int(mo[0].isnan().sum()) == 128
            assert bool(mo[1][128:256].isnan().all()) and int(mo[1].isnan().sum()) == 128


def test_rounding_is_unbiased():
    """One value beside its group's largest, over 2^20 elements: the mean of what is stored is
    the value. A rounding of one unit has a standard deviation of at most half a unit, so the
    mean of n is within 6 * 0.5 / sqrt(n) units (one failure in 5e8 for a fair rounding)."""
    n = 1 << 20
    c = Case([n], "f32", bits=8)
    for x in (0.3777, 0.0301):
        g = torch.full((n,), x, device="cuda")
        g[::128] = 1.0
        c.opt.state["m"].zero_()
        c.opt.state["root_v"].zero_()
        mo = c.moment_buffers()
        c.opt.step(c.w, [g], moments=mo)
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep[::128] = False
        b1, b2 = c.hyper["betas"]
        m, v = A.step32(np.float32(x), np.float32(0), np.float32(0), b1, b2)
        for got, true, bits in ((mo[0], float(m), 3), (mo[1], math.sqrt(float(v)), 4)):
            unit = 2.0 ** (math.floor(math.log2(true)) - bits)
            mean = float(got[keep].double().mean())
            assert abs(mean - true) <= 3 * unit / math.sqrt(n * 127 / 128) + 1e-6 * true


@pytest.mark.parametrize("bits", [32, 8])
def test_graph_replay_counts_and_matches_eager(bits):
    """A captured step (norm, clip and step) keeps its own count: replays with eager steps and
    synchronisations between them match an optimizer that is stepped eagerly throughout."""
    a, b = (Case([3000, 5, 257], "bf16", bits=bits) for _ in range(2))
    g = a.gradients()
    out = torch.empty(2, device="cuda")

    def step(c):
        c.opt.step(c.w, g, clip=c.opt.grad_norm(g, max_norm=0.3, out=out))

    step(a), step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for k in range(4):
        graph.replay()
        step(b)
        if k == 1:
            step(a), step(b)
        torch.cuda.synchronize()
        for x, y in zip(a.w, b.w):
            assert torch.equal(x, y), f"replay {k}"
        for n in a.opt.state:
            assert torch.equal(a.opt.state[n], b.opt.state[n])
    assert a.opt.t == b.opt.t == 6


def test_another_stream_than_the_current_one():
    a, b = (Case([100_000, 77], "f16", bits=8) for _ in range(2))
    g = a.gradients()
    side, out = torch.cuda.Stream(), torch.empty(2, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.opt.grad_norm(g, max_norm=0.3, out=out, stream=side)
        a.opt.step(a.w, g, clip=out, stream=side.cuda_stream)
        b.opt.step(b.w, g, clip=b.opt.grad_norm(g, max_norm=0.3))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(a.w, b.w))
    with pytest.raises(ValueError, match="out"):
        a.opt.grad_norm(g, stream=side)


@pytest.mark.parametrize("bits", [32, 8])
def test_saved_state_continues_the_run(bits):
    a = Case([5000, 129], "bf16", bits=bits)
    for _ in range(3):
        a.checked_step(a.gradients())
    saved, w = a.opt.state_dict(), [x.clone() for x in a.w]
    g = a.gradients()
    a.checked_step(g)
    b = Case([5000, 129], "bf16", bits=bits)
    b.opt.load_state_dict(saved)
    b.w, b.t = w, saved["t"]
    b.checked_step(g)
    assert b.opt.t == 4 and all(torch.equal(x, y) for x, y in zip(a.w, b.w))
    other = Case([5000, 128], "bf16", bits=bits)
    with pytest.raises(ValueError, match="numels"):
        other.opt.load_state_dict(saved)


def test_learning_rate_changes():
    c = Case([1000], "f32")
    c.checked_step(c.gradients())
    c.opt.set_lr(0.05)
    c.hyper = dict(HYPER, lr=0.05)
    c.checked_step(c.gradients())


def test_places_beyond_32_bits():
    """A tensor of 2^32 + 1000 values: its end is stepped like a tensor of its own, with the
    same random bits at the places 2^32 on as at 0 on."""
    n, tail = (1 << 32) + 1000, 1000
    print("CASE adamw 2^32 values", flush=True)
    big = tg.AdamW([n], "bf16", state_bits=8, seed=5, **HYPER)
    small = tg.AdamW([tail], "bf16", state_bits=8, seed=5, **HYPER)
    w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    wt = random_tensor(tail, "bf16", gen, 0.02)
    gt = random_tensor(tail, "bf16", gen, 0.01)
    w[-tail:], g[-tail:] = wt, gt
    for _ in range(2):
        big.step([w], [g])
        small.step([wt], [gt])
    assert torch.equal(w[-tail:], wt)
    for k in ("m", "root_v"):
        assert torch.equal(big.state[k][1 << 32:], small.state[k])
    assert int((w[:-tail] != 0).sum()) == 0
    norm = big.grad_norm([g])
    assert torch.equal(norm, small.grad_norm([gt]))


def test_refusals():
    c = Case([100, 50], ["bf16", "f32"], bits=8)
    g = c.gradients()
    before = c.snapshot()

    def refused(what, *a, **k):
        with pytest.raises(ValueError, match=what):
            c.opt.step(*a, **k)

    refused("weights", c.w[:1], g)
    refused("grads", c.w, g + g)
    refused(r"grads\[0\].*dtype", c.w, [g[0].float(), g[1]])
    refused(r"weights\[1\].*elements", [c.w[0], c.w[1][:49]], g)
    refused(r"weights\[1\].*GPU", [c.w[0], c.w[1].cpu()], g)
    refused(r"grads\[1\].*contiguous", c.w, [g[0], torch.zeros(100, device="cuda")[::2]])
    refused(r"grads\[0\].*Tensor", c.w, [None, g[1]])
    refused("clip", c.w, g, clip=torch.ones(3, device="cuda"))
    refused("clip", c.w, g, clip=torch.ones(2, device="cuda", dtype=torch.float64))
    mo = c.moment_buffers()
    refused("moments", c.w, g, moments=[mo[0]])
    refused("moments", c.w, g, moments=[mo[0], mo[0]])
    refused("moments", c.w, g, moments=[mo[0], mo[1].float()])
    with pytest.raises(tg.TGradError, match="invalid argument"):
        c.opt.grad_norm(g, max_norm=0.0)
    with pytest.raises(tg.TGradError, match="invalid argument"):
        c.opt.grad_norm(g, grad_scale=math.inf)
    with pytest.raises(tg.TGradError, match="invalid argument"):
        c.opt.set_lr(-1.0)
    d = Case([100], "f32")
    with pytest.raises(ValueError, match="moments"):
        d.opt.step(d.w, d.gradients(), moments=[torch.empty(128, dtype=torch.bfloat16, device="cuda")] * 2)
    after = c.snapshot()
    assert all(np.array_equal(x, y) for x, y in zip(before[0], after[0])) and c.opt.t == 0
    for kw in (dict(lr=-1.0), dict(betas=(1.0, 0.9)), dict(eps=math.nan), dict(weight_decay=-0.1)):
        with pytest.raises(tg.TGradError, match="invalid argument"):
            tg.AdamW([4], "f32", **kw)
    for kw in (dict(state_bits=16), dict(grad_dtypes=["f32"] * 3), dict(weight_decay=[0.1, 0.2])):
        with pytest.raises(ValueError):
            tg.AdamW([4], "f32", **kw)
    with pytest.raises(tg.TGradError, match="invalid argument"):
        tg.AdamW([4], "f32", "bf16")
    with pytest.raises(ValueError):
        tg.AdamW([], "f32")
    with pytest.raises(ValueError):
        tg.AdamW([-1], "f32")


def test_autograd_sees_the_change():
    """A step is an in-place change: a graph that saved a weight before it refuses to run."""
    c = Case([64], "f32")
    w = c.w[0].requires_grad_()
    y = (w * w).sum()
    c.opt.step([w], c.gradients())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_autograd_sees_the_results_that_are_written_in_place():
    """The values of the moments and the norm, which go into the caller's tensors, change as the
    weights do."""
    c = Case([64], "f32", bits=8)
    mo, out = c.moment_buffers(), torch.ones(2, device="cuda")
    for t in mo + [out]:
        x = torch.ones_like(t).requires_grad_()
        y = (x * t).sum()                      # saves t
        c.opt.step(c.w, c.gradients(), clip=c.opt.grad_norm(c.gradients(), out=out), moments=mo)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    with torch.inference_mode():               # tensors that have no version
        out, mo = torch.ones(2, device="cuda"), c.moment_buffers()
        c.opt.step(c.w, c.gradients(), clip=c.opt.grad_norm(c.gradients(), out=out), moments=mo)


def test_more_values_than_one_launch_has_threads_for():
    """A tensor of 2^35 + 1000 values, 2^24 workgroups' and one more: its end and a piece in its
    middle are stepped like tensors of their own, with the same random bits at multiples of 2^32."""
    import gc
    tail, at = 1000, (5 << 32, 1 << 35)
    n = at[1] + tail
    gc.collect()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 6.2 * n + (8 << 30):
        pytest.skip("needs weights, gradients and state of 2^35 values")
    print("CASE adamw 2^35 values", flush=True)
    big = tg.AdamW([n], "bf16", state_bits=8, seed=5, **HYPER)
    small = tg.AdamW([tail], "bf16", state_bits=8, seed=5, **HYPER)
    w, g = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(1)
    wt, gt = random_tensor(tail, "bf16", gen, 0.02), random_tensor(tail, "bf16", gen, 0.01)
    for a in at:
        w[a:a + tail], g[a:a + tail] = wt, gt
    for _ in range(2):
        big.step([w], [g])
        small.step([wt], [gt])
    whole = tail // A.GROUP * A.GROUP
    for a in at:
        assert torch.equal(w[a:a + tail], wt)
        for k in ("m", "root_v"):
            assert torch.equal(big.state[k][a:a + whole], small.state[k][:whole])
    norm = math.sqrt(2 * float((gt.double() ** 2).sum()))
    assert abs(float(big.grad_norm([g])[0]) - norm) <= 1.01 * E * norm
    assert big.t == 2
    del w, g
    big.close()
    del big
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "c64"])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("numels", [[9_000_011, 300_001], [130_000_003, 5]])
def test_norm_of_spans_of_several_passes(dtype, offset, numels):
    """Spans of 8192 to 98304 values, several passes of a workgroup, with ragged ends. fp64 sums
    in another order differ far less than fp32's rounding."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    opt = tg.AdamW(numels, dtype, state_bits=8)
    g = [random_tensor(n, dtype, gen, 1.0, offset) for n in numels]
    squares = 0.0
    for x in g:
        v = torch.view_as_real(x).reshape(-1) if x.is_complex() else x
        for part in v.split(1 << 26):
            squares += float((part.double() ** 2).sum())
    out = opt.grad_norm(g, max_norm=2.0, grad_scale=0.5)
    norm = 0.5 * math.sqrt(squares)
    coef = 0.5 * min(1.0, 2.0 / norm)
    assert abs(float(out[0]) - norm) <= 1.01 * E * norm
    assert abs(float(out[1]) - coef) <= 1.01 * E * coef
    g[0].reshape(-1)[-1] = math.inf              # the very last value of a span
    assert float(opt.grad_norm(g)[0]) == math.inf


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-37, 1e-39, 1e-45, 1e-60])
def test_eps_below_fp32s_normal_numbers(bits, eps):
    """Any eps above zero keeps a value that has had no gradient at its decayed weight, where 0 / 0
    would lose it, and is nothing beside the root of the others' v."""
    c = Case([300, 5], "f32", bits=bits, hyper=dict(lr=1e-2, betas=(0.9, 0.999), eps=eps))
    for _ in range(2):
        g = c.gradients()
        g[0][::3] = 0
        c.checked_step(g)
    assert all(bool(w.isfinite().all()) for w in c.w)
