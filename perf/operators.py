"""Cases of the operators beside the TensorGRaD step, with their plain forms.

A TensorGRaD handle optimises the large weight tensors of a model. What is left of a training
step on the same model is measured here:

* adamw: one AdamW step over all the other tensors at once, with fp32 moments or with
  moments held in 8 bits, optionally after the global gradient norm (clipping, and no step
  where that norm is not finite);
* ln_fwd, ln_bwd: layer norm over the last axis, and its gradients, the reduction of the
  weight's and the bias's gradient over all rows included. These are among the tensors that
  the AdamW step takes.

The tensors of an AdamW case are views of one flat buffer, each starting at a multiple of
128 values (where an allocator would start it), so that the updated weights come back whole.
"""
import itertools
import math
import random

import torch

own = False

F32 = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "c64": torch.complex64}
GROUP = 128          # values that share one scale; every tensor's state starts at a multiple of it
LR, B1, B2, EPS, DECAY, SEED = 1e-3, 0.9, 0.999, 1e-8, 0.01, 1234
STEPS_BEFORE = 100   # the state is that of a run that has made this many steps
MAX_NORM = 1.0
LN_EPS = 1e-5


def listed():
    return [
        # biases, norm weights and skip products of one narrow layer: a step is launch latency
        {"name": "adamw32_layer_f32", "op": "adamw", "bits": 32, "dtype": "f32", "grad": "f32", "clip": True,
         "tensors": 12, "lo": 64, "hi": 4096, "mix": 1},
        # every tensor of a middle-sized model in bf16 with gradient clipping
        {"name": "adamw32_model_bf16", "op": "adamw", "bits": 32, "dtype": "bf16", "grad": "bf16", "clip": True,
         "tensors": 150, "lo": 64, "hi": 1 << 20, "mix": 2},
        # the tensor of the bf16 (64,64,48,48,25) workload, stepped without compression
        {"name": "adamw32_tensor_bf16", "op": "adamw", "bits": 32, "dtype": "bf16", "grad": "bf16", "clip": False,
         "tensors": 1, "lo": 235929600, "hi": 235929600, "mix": 3},
        # a small fp16 model under loss scaling, odd sizes
        {"name": "adamw8_small_f16", "op": "adamw", "bits": 8, "dtype": "f16", "grad": "f16", "clip": True,
         "tensors": 40, "lo": 33, "hi": 20011, "mix": 4},
        # fp32 weights of odd sizes from one value up
        {"name": "adamw8_odd_f32", "op": "adamw", "bits": 8, "dtype": "f32", "grad": "f32", "clip": False,
         "tensors": 61, "lo": 1, "hi": 1 << 20, "mix": 5},
        # the four layers of the fp16 (64,64,64,64) workload
        {"name": "adamw8_layers_f16", "op": "adamw", "bits": 8, "dtype": "f16", "grad": "f16", "clip": True,
         "tensors": 4, "lo": 16777216, "hi": 16777216, "mix": 6},
        # a few points of a narrow layer
        {"name": "ln_fwd_small_f32", "op": "ln_fwd", "rows": 64, "cols": 64, "dtype": "f32", "weight": "f32"},
        # 16 fields of 64 x 64 points with 256 channels
        {"name": "ln_fwd_fields_bf16", "op": "ln_fwd", "rows": 65536, "cols": 256, "dtype": "bf16", "weight": "f32"},
        # rows that no vector width divides
        {"name": "ln_fwd_odd_f16", "op": "ln_fwd", "rows": 8191, "cols": 4099, "dtype": "f16", "weight": "f16"},
        {"name": "ln_bwd_odd_f32", "op": "ln_bwd", "rows": 1000, "cols": 333, "dtype": "f32", "weight": "f32"},
        {"name": "ln_bwd_fields_bf16", "op": "ln_bwd", "rows": 65536, "cols": 256, "dtype": "bf16", "weight": "f32"},
        # wide rows of a mixed-precision transformer
        {"name": "ln_bwd_wide_bf16", "op": "ln_bwd", "rows": 8192, "cols": 8192, "dtype": "bf16", "weight": "bf16"},
    ]


def log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        bits = rng.choice((32, 8))
        dtype = rng.choice(("f32", "f16", "bf16", "bf16", "c64"))
        grad = rng.choice((dtype, dtype, "f32")) if dtype in ("f16", "bf16") else dtype
        total, n = log_uniform(rng, 1e3, 2e7), log_uniform(rng, 1, 300)
        lo = log_uniform(rng, 1, 1e4)
        hi = max(lo, 3 * total // n)
        # an fp32 weight's second step shows where two sums of squares, rounded apart, put a
        # moment on either side of an 8-bit rounding: those cases run without the norm
        clip = rng.random() < 0.5 and not (bits == 8 and dtype in ("f32", "c64"))
        return {"op": "adamw", "bits": bits, "dtype": dtype, "grad": grad, "clip": clip,
                "tensors": n, "lo": lo, "hi": hi, "mix": rng.randrange(1 << 20)}
    cols = log_uniform(rng, 1, 16384)
    rows = log_uniform(rng, 1, max(1, min(200000, 60000000 // cols)))
    if rng.random() < 0.4:
        cols = max(8, cols // 8 * 8)
    dtype = rng.choice(("f32", "f16", "bf16"))
    return {"op": rng.choice(("ln_fwd", "ln_bwd")), "rows": rows, "cols": cols, "dtype": dtype,
            "weight": rng.choice(("f32", dtype))}


# ------------------------------------------------------------------------------- adamw

def sizes_of(case):
    """Elements of each tensor (a complex element is one)."""
    rng = random.Random(case["mix"])
    return [log_uniform(rng, case["lo"], case["hi"]) for _ in range(case["tensors"])]


def layout(case):
    """(elements, first value, values) of each tensor in the flat buffers, and their length."""
    per, sizes = 2 if case["dtype"] == "c64" else 1, sizes_of(case)
    ends = list(itertools.accumulate(-(-n * per // GROUP) * GROUP for n in sizes))
    return [(n, at, n * per) for n, at in zip(sizes, [0] + ends)], ends[-1]


def random_bits(t, n, device):
    """32 random bits for each value of the state at step t, as int64: SplitMix64's output for
    the state seed + t * 0x9E3779B97F4A7C15 keys a mix of the value's place."""
    mask = (1 << 64) - 1
    z = (SEED + t * 0x9E3779B97F4A7C15) & mask
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
    key = (z ^ (z >> 31)) & 0xFFFFFFFF
    h = (torch.arange(n, dtype=torch.int64, device=device) & 0xFFFFFFFF) ^ key
    h = (h * 0xBF58476D) & 0xFFFFFFFF
    h = h ^ (h >> 16)
    h = (h * 0x94D049BB) & 0xFFFFFFFF
    return h ^ (h >> 13)


def power(e):
    """2 ** e as fp32, for exponents of the normal range."""
    return ((e + 127) << 23).view(torch.float32)


def pack(x, shift, r):
    """fp32 values x of whole groups, none negative, as 8-bit floats without a sign: a code of
    the group's exponent field f (of its largest value) stands for the fp32 value with the
    bits code << shift, times 2 ** (f - 14). r: the random low bits that are added before the
    rest is cut off."""
    x = x.view(-1, GROUP)
    f = x.amax(1).view(torch.int32) >> 23
    y = (x * power(14 - f).unsqueeze(1)).view(torch.int32) + r.view(-1, GROUP).to(torch.int32)
    return (y >> shift).reshape(-1), f.to(torch.uint8)


def unpack(code, f, shift):
    y = (code.to(torch.int32) << shift).view(torch.float32).view(-1, GROUP)
    return (y * power(f.to(torch.int32) - 14).unsqueeze(1)).reshape(-1)


def pack_state(m, q, rm, rq):
    """8-bit moments: m as a sign and an E4M3 code, q = sqrt(v) as an E4M4 code, where a q
    above zero keeps at least the least code, so that no update divides by zero."""
    cm, fm = pack(m.abs(), 20, rm)
    cq, fq = pack(q, 19, rq)
    cm = cm | (m < 0).to(torch.int32) * 128
    cq = torch.maximum(cq, (q > 0).to(torch.int32))
    return cm.to(torch.uint8), cq.to(torch.uint8), fm, fq


def values_of(cm, cq, fm, fq):
    m = unpack(cm & 127, fm, 20)
    return torch.where(cm >= 128, -m, m), unpack(cq, fq, 19)


def prepare_adamw(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    tensors, total = layout(case)
    ends = torch.tensor([at + n for _, at, n in tensors], device=dev)
    room = torch.tensor([-(-n // GROUP) * GROUP for _, _, n in tensors], device=dev)
    live = torch.arange(total, device=dev) < ends.repeat_interleave(room)

    def normal():
        return torch.randn(total, generator=gen, device=dev)

    # gradients and moments spread over several orders of magnitude, as a model's are
    size = (normal() * 0.7).exp_()
    g = normal() * size * (0.01 * live)
    m = normal() * size * (0.003 * live)
    q = (0.2 * normal()).exp_() * size * (0.01 * live)
    w = normal() * (0.02 * live)

    def store(x, kind):
        return torch.view_as_complex(x.view(-1, 2)) if kind == "c64" else x.to(F32[kind])

    s = {"case": case, "t": STEPS_BEFORE, "w": store(w, case["dtype"]), "g": store(g, case["grad"])}
    if case["bits"] == 8:
        half = torch.full((total,), 1 << 19, dtype=torch.int64, device=dev)
        s["m"], s["v"], s["fm"], s["fv"] = pack_state(m, q, half, half >> 1)
    else:
        s["m"], s["v"] = m, q * q
    if own:
        import tensor_gradient_compression_amd as tg
        per = 2 if case["dtype"] == "c64" else 1
        s["ws"] = [s["w"][at // per:at // per + n] for n, at, _ in tensors]
        s["gs"] = [s["g"][at // per:at // per + n] for n, at, _ in tensors]
        opt = tg.AdamW([n for n, _, _ in tensors], case["dtype"], grad_dtypes=case["grad"], lr=LR, betas=(B1, B2),
                       eps=EPS, weight_decay=DECAY, state_bits=case["bits"], seed=SEED)
        for k, v in zip(opt.state, (s["m"], s["v"]) + ((s["fm"], s["fv"]) if case["bits"] == 8 else ())):
            opt.state[k].copy_(v)
        opt.t = STEPS_BEFORE
        s["opt"] = opt
        if case["bits"] == 8:
            s["values"] = [torch.empty(total, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    return s


def real(x):
    return torch.view_as_real(x).reshape(-1) if x.is_complex() else x


def run_adamw(s):
    case = s["case"]
    if own:
        opt = s["opt"]
        clip = opt.grad_norm(s["gs"], max_norm=MAX_NORM) if case["clip"] else None
        if case["bits"] == 8:
            opt.step(s["ws"], s["gs"], clip=clip, moments=s["values"])
            out = [s["w"], *s["values"]]
        else:
            opt.step(s["ws"], s["gs"], clip=clip)
            out = [s["w"], opt.state["m"], opt.state["v"]]
        return out + ([clip] if case["clip"] else [])
    s["t"] += 1
    t, g = s["t"], real(s["g"]).float()
    out = []
    if case["clip"]:
        norm = (g * g).sum().sqrt()
        coef = (MAX_NORM / norm).clamp(max=1.0)
        out = [torch.stack((norm, coef))]
        g = g * coef
    if case["bits"] == 8:
        m, q = values_of(s["m"], s["v"], s["fm"], s["fv"])
        v = q * q
    else:
        m, v = s["m"], s["v"]
    m = B1 * m + (1 - B1) * g
    v = B2 * v + (1 - B2) * (g * g)
    w = real(s["w"]).float() * (1 - LR * DECAY) - LR * ((m / (1 - B1 ** t)) / ((v / (1 - B2 ** t)).sqrt() + EPS))
    real(s["w"]).copy_(w)
    if case["bits"] == 8:
        h = random_bits(t, m.numel(), m.device)
        s["m"], s["v"], s["fm"], s["fv"] = pack_state(m, v.sqrt(), h >> 12, h & 0x7FFFF)
        m, v = (x.to(torch.bfloat16) for x in values_of(s["m"], s["v"], s["fm"], s["fv"]))
    else:
        s["m"], s["v"] = m, v
    return [s["w"], m, v] + out


def exact_adamw(case, seed):
    s, t = prepare_adamw(case, seed), STEPS_BEFORE + 1
    g = real(s["g"]).double()
    out = []
    if case["clip"]:
        norm = (g * g).sum().sqrt()
        coef = (MAX_NORM / norm).clamp(max=1.0)
        out = [torch.stack((norm, coef))]
        g = g * coef

    def value(code, f, bits):
        """A code with `bits` of mantissa: below 2 ** bits it counts the least steps."""
        code, f = code.long(), f.long().repeat_interleave(GROUP)
        e, frac = code >> bits, (code & ((1 << bits) - 1)).double() / (1 << bits)
        y = torch.where(e > 0, 1 + frac, frac)
        return torch.ldexp(y, (e.clamp(min=1) - 127 + f - 14).double())

    if case["bits"] == 8:
        m = value(s["m"] & 127, s["fm"], 3) * torch.where(s["m"] >= 128, -1.0, 1.0)
        v = value(s["v"], s["fv"], 4) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = B1 * m + (1 - B1) * g
    v = B2 * v + (1 - B2) * g * g
    w = real(s["w"]).double()
    w = w - LR * DECAY * w - LR * (m / (1 - B1 ** t)) / ((v / (1 - B2 ** t)).sqrt() + EPS)
    if s["w"].is_complex():
        w = torch.view_as_complex(w.view(-1, 2))
    if case["bits"] == 8:
        h = random_bits(t, m.numel(), m.device)

        def rounded(x, bits, u):
            """x, not negative, on the codes: down or up by u, uniform in [0, 1)."""
            top = x.view(-1, GROUP).amax(1)
            f = torch.where(top > 0, torch.frexp(top)[1].long() + 126, 0).clamp(min=0)
            f = f.repeat_interleave(GROUP)
            e = torch.frexp(x)[1].long() - 1 - f + 14 + 127       # the code's exponent field
            unit = torch.ldexp(torch.ones_like(x), (e.clamp(min=1) - 127 + f - 14 - bits).double())
            return torch.floor(x / unit + u) * unit, torch.ldexp(torch.ones_like(x), (f - 14 - 126 - bits).double())

        a, _ = rounded(m.abs(), 3, (h >> 12).double() / (1 << 20))
        b, least = rounded(v.sqrt(), 4, (h & 0x7FFFF).double() / (1 << 19))
        m, v = a * torch.sign(m), torch.where(v > 0, torch.maximum(b, least), 0.0)
    return [w, m, v] + out


def work_adamw(case):
    n = sum(v for _, _, v in layout(case)[0])
    size = {"f32": 4, "c64": 4, "f16": 2, "bf16": 2}
    w, g = size[case["dtype"]], size[case["grad"]]
    # 8 bits: the codes and a scale byte for 128 of them, in and out, and the values that come back
    state = 16 if case["bits"] == 32 else 4 + 4 / GROUP + 4
    return {"bytes": n * (2 * w + g + state), "flops": n * (16 + (3 if case["clip"] else 0))}


# -------------------------------------------------------------------------- layer norm

def prepare_ln(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rows, cols = case["rows"], case["cols"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    # activations: rows of their own level, a few channels that are much larger
    loud = 1 + 9 * (torch.rand(cols, generator=gen, device=dev) < 0.02)
    x = ((normal(rows, cols) + 0.5 * normal(rows, 1)) * loud + 0.3 * normal(cols)).to(F32[case["dtype"]])
    s = {"case": case, "x": x, "w": (1 + 0.1 * normal(cols)).to(F32[case["weight"]]),
         "b": (0.1 * normal(cols)).to(F32[case["weight"]])}
    if case["op"] == "ln_bwd":
        xf = x.float()
        s["mean"] = xf.mean(1)
        s["rstd"] = ((xf - s["mean"][:, None]) ** 2).mean(1).add(LN_EPS).rsqrt()
        s["dy"] = (0.1 * normal(rows, cols) + 0.02 * normal(cols)).to(F32[case["dtype"]])
    return s


def run_ln(s):
    back = s["case"]["op"] == "ln_bwd"
    if own:
        import tensor_gradient_compression_amd as tg
        if back:
            return list(tg.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"]))
        return list(tg.layer_norm_forward(s["x"], s["w"], s["b"], eps=LN_EPS))
    x, w = s["x"].float(), s["w"].float()
    if not back:
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = 1.0 / ((c * c).mean(1) + LN_EPS).sqrt()
        y = c * rstd[:, None] * w + s["b"].float()
        return [y.to(s["x"].dtype), mean, rstd]
    dy = s["dy"].float()
    n = (x - s["mean"][:, None]) * s["rstd"][:, None]
    h = dy * w
    dx = s["rstd"][:, None] * (h - h.mean(1, keepdim=True) - n * (h * n).mean(1, keepdim=True))
    return [dx.to(s["x"].dtype), (dy * n).sum(0).to(s["w"].dtype), dy.sum(0).to(s["w"].dtype)]


def exact_ln(case, seed):
    s = prepare_ln(case, seed)
    x, w = s["x"].double(), s["w"].double()
    mean = x.sum(1, keepdim=True) / case["cols"]
    var = ((x - mean) ** 2).sum(1, keepdim=True) / case["cols"]
    rstd = (var + LN_EPS) ** -0.5
    n = (x - mean) * rstd
    if case["op"] == "ln_fwd":
        return [n * w + s["b"].double(), mean[:, 0], rstd[:, 0]]
    dy = s["dy"].double()
    h = dy * w
    dx = (h - h.sum(1, keepdim=True) / case["cols"] - n * ((h * n).sum(1, keepdim=True) / case["cols"])) * rstd
    return [dx, (dy * n).sum(0), dy.sum(0)]


def work_ln(case):
    e = {"f32": 4, "f16": 2, "bf16": 2}
    n, r, c = case["rows"] * case["cols"], case["rows"], case["cols"]
    if case["op"] == "ln_fwd":
        return {"bytes": n * 2 * e[case["dtype"]] + 8 * r + 2 * c * e[case["weight"]], "flops": 8 * n}
    return {"bytes": n * 3 * e[case["dtype"]] + 8 * r + 3 * c * e[case["weight"]], "flops": 14 * n}


def prepare(case, seed):
    return prepare_adamw(case, seed) if case["op"] == "adamw" else prepare_ln(case, seed)


def run(state):
    return run_adamw(state) if state["case"]["op"] == "adamw" else run_ln(state)


def exact(case, seed):
    return exact_adamw(case, seed) if case["op"] == "adamw" else exact_ln(case, seed)


def work(case):
    return work_adamw(case) if case["op"] == "adamw" else work_ln(case)
