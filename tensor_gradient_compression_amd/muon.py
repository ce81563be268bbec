"""Muon over many matrices at once, and the orthogonalisation it steps by (tgrad_muon_*,
tgrad_orthogonalize in include/tgrad.h)."""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Union

import tensor_gradient_compression_amd as _tg

GROUP = 128     # every tensor's momentum starts at a multiple
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonalize(x, steps: int = 5, coefficients: Sequence[float] = COEFFICIENTS, eps: float = 1e-7):
    """Every matrix of x (..., rows, cols) with its singular values brought near 1 by `steps`
    Newton-Schulz products, on the current stream, as a new tensor. x: float32, float16 or
    bfloat16, its rows contiguous and its matrices evenly spaced. Autograd records nothing."""
    a, b, c = coefficients
    return _tg.binding().orthogonalize(x, steps, a, b, c, eps)


def _stream(stream) -> Optional[int]:
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _scale(scale, rows: int, cols: int) -> float:
    if scale == "spectral":
        return math.sqrt(max(1.0, rows / cols))
    if scale == "rms":
        return 0.2 * math.sqrt(max(rows, cols))
    if isinstance(scale, str):
        raise ValueError(f"unknown scale {scale!r}: 'spectral', 'rms' or a number")
    return float(scale)


class Muon:
    """One Muon optimizer for a list of tensors of `shapes`: (rows, cols), or (..., rows, cols)
    for as many matrices one after the other.

    dtypes, grad_dtypes: "f32", "f16" or "bf16", one for all tensors or one each; a 16-bit weight
    may have fp32 gradients. weight_decay: one for all or one each. scale: what multiplies an
    update beside the learning rate, "spectral" (sqrt(max(1, rows / cols))), "rms"
    (0.2 sqrt(max(rows, cols)), an update of the size of AdamW's) or a number; one or one each.

    The momentum is `state`["momentum"], one flat float32 GPU tensor in which tensor i's values
    start at offsets[i]. The learning rate takes effect at the next step (set_lr)."""

    def __init__(self, shapes: Sequence[Sequence[int]], dtypes: Union[str, Sequence[str]],
                 grad_dtypes: Union[None, str, Sequence[str]] = None, lr: float = 1e-3,
                 momentum: float = 0.95, nesterov: bool = True,
                 weight_decay: Union[float, Sequence[float]] = 0.1, scale="spectral", steps: int = 5,
                 coefficients: Sequence[float] = COEFFICIENTS, eps: float = 1e-7):
        import torch
        self._h = None
        self._lib = _tg.load_library()
        bind = _tg.binding()
        n = len(shapes)
        if n < 1:
            raise ValueError("shapes: at least one tensor")
        self.shapes = tuple(tuple(int(x) for x in s) for s in shapes)
        for s in self.shapes:
            if len(s) < 2 or min(s) < 0 or s[-1] < 1 or s[-2] < 1:
                raise ValueError(f"shapes: {s} is no matrix or matrices")
        each = lambda v: (v,) * n if isinstance(v, str) or not isinstance(v, Sequence) else tuple(v)  # noqa: E731
        self.dtypes = each(dtypes)
        self.grad_dtypes = self.dtypes if grad_dtypes is None else each(grad_dtypes)
        self.weight_decay = tuple(float(x) for x in each(weight_decay))
        scales = each(scale)
        for what, v in (("dtypes", self.dtypes), ("grad_dtypes", self.grad_dtypes),
                        ("weight_decay", self.weight_decay), ("scale", scales)):
            if len(v) != n:
                raise ValueError(f"{what}: {len(v)} given for {n} tensors")
        for d in self.dtypes + self.grad_dtypes:
            if d not in ("f32", "f16", "bf16"):
                raise ValueError(f"dtype {d!r}: 'f32', 'f16' or 'bf16'")
        self.scale = tuple(_scale(x, s[-2], s[-1]) for x, s in zip(scales, self.shapes))
        if len(tuple(coefficients)) != 3:
            raise ValueError("coefficients: three numbers")
        self.lr, self.momentum, self.nesterov = float(lr), float(momentum), bool(nesterov)
        self.steps, self.eps = int(steps), float(eps)
        self.coefficients = tuple(float(c) for c in coefficients)
        counts = [math.prod(s[:-2]) for s in self.shapes]
        i64, i32, f64 = ctypes.c_int64 * n, ctypes.c_int * n, ctypes.c_double * n
        cc, cr, ck = i64(*counts), i64(*[s[-2] for s in self.shapes]), i64(*[s[-1] for s in self.shapes])
        total = self._lib.tgrad_muon_state_values(n, cc, cr, ck)
        if total < 0:
            raise ValueError("shapes: more than the library takes")
        dts = [_tg.DTYPE_CODES[d] for d in self.dtypes]
        gts = [_tg.DTYPE_CODES[d] for d in self.grad_dtypes]
        numels = [math.prod(s) for s in self.shapes]
        at, self.offsets = 0, []
        for x in numels:
            self.offsets.append(at)
            at += -(-x // GROUP) * GROUP
        self.device_index = torch.cuda.current_device()
        self.state = {"momentum": torch.zeros(total, device=f"cuda:{self.device_index}")}
        h = ctypes.c_void_p()
        rc = self._lib.tgrad_muon_init(ctypes.byref(h), n, cc, cr, ck, i32(*dts), i32(*gts), f64(*self.weight_decay),
                                       f64(*self.scale), self.lr, self.momentum, int(self.nesterov), self.steps,
                                       (ctypes.c_double * 3)(*self.coefficients), self.eps,
                                       ctypes.c_void_p(self.state["momentum"].data_ptr()))
        if rc != _tg.OK:
            raise _tg.TGradError(f"tgrad_muon_init: {self._lib.tgrad_status_string(rc).decode()}")
        self._h = h
        self._plan = bind.muon_plan(h.value, self.device_index, numels, dts, gts, list(ck))
        self._step = bind.muon_step

    # ---------------------------------------------------------------- lifecycle
    def close(self):
        if getattr(self, "_h", None):
            self._plan = None
            self._lib.tgrad_muon_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---------------------------------------------------------------- hot path
    def step(self, weights, grads, clip=None, stream=None):
        """One step of every tensor: weights[i] is updated in place from grads[i] (contiguous
        GPU tensors of as many elements as shapes[i], flat or by axes of which the last join to a row; no
        weight overlaps another or a gradient). clip: what AdamW.grad_norm returned, the norm over this
        optimizer's gradients or over more; where it is not finite, nothing changes."""
        self._step(self._plan, weights, grads, clip, _stream(stream))

    def set_lr(self, lr: float):
        rc = self._lib.tgrad_muon_set_lr(self._h, float(lr))
        if rc != _tg.OK:
            raise _tg.TGradError(f"tgrad_muon_set_lr: {self._lib.tgrad_status_string(rc).decode()}")
        self.lr = float(lr)

    # ---------------------------------------------------------------- state
    def state_dict(self) -> dict:
        """A copy of the momentum and what it depends on."""
        return {"shapes": self.shapes, "momentum_factor": self.momentum,
                "state": {k: v.clone() for k, v in self.state.items()}}

    def load_state_dict(self, saved: dict):
        """Continue from a state_dict of an optimizer of the same shapes and momentum factor."""
        if saved["shapes"] != self.shapes:
            raise ValueError(f"shapes: the state has {saved['shapes']}, the optimizer {self.shapes}")
        if saved["momentum_factor"] != self.momentum:
            raise ValueError(f"momentum: the state has {saved['momentum_factor']}, the optimizer {self.momentum}")
        for k, v in self.state.items():
            x = saved["state"][k]
            if x.shape != v.shape or x.dtype != v.dtype:
                raise ValueError(f"state {k}: {tuple(x.shape)} of {x.dtype}, expected {tuple(v.shape)} of {v.dtype}")
        for k, v in self.state.items():
            v.copy_(saved["state"][k])
