"""AdamW over many tensors at once (tgrad_adamw_* in include/tgrad.h)."""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Union

import tensor_gradient_compression_amd as _tg

GROUP = 128     # values that share a scale of the 8-bit state


def _stream(stream) -> Optional[int]:
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


class AdamW:
    """One AdamW optimizer for a list of tensors of `numels` elements.

    dtypes, grad_dtypes: "f32", "f16", "bf16" or "c64", one for all tensors or one each; a
    16-bit weight may have fp32 gradients. weight_decay: one for all or one each. state_bits:
    32 for fp32 moments, 8 for moments of one byte each.

    The state lives in `state`, a dict of flat GPU tensors: "m" and "v" (32 bits), or "m",
    "root_v", "m_scale" and "root_v_scale" (8 bits, the format of include/tgrad.h). Tensor i's
    values start at offsets[i]; complex elements count as two."""

    def __init__(self, numels: Sequence[int], dtypes: Union[str, Sequence[str]],
                 grad_dtypes: Union[None, str, Sequence[str]] = None, lr: float = 1e-3,
                 betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: Union[float, Sequence[float]] = 0.01, state_bits: int = 32,
                 seed: int = 0):
        import torch
        self._h = None
        self._lib = _tg.load_library()
        bind = _tg.binding()
        n = len(numels)
        if n < 1:
            raise ValueError("numels: at least one tensor")
        self.numels = tuple(int(x) for x in numels)
        self.dtypes = (dtypes,) * n if isinstance(dtypes, str) else tuple(dtypes)
        self.grad_dtypes = self.dtypes if grad_dtypes is None else (
            (grad_dtypes,) * n if isinstance(grad_dtypes, str) else tuple(grad_dtypes))
        decay = (tuple(float(x) for x in weight_decay) if isinstance(weight_decay, Sequence)
                 else (float(weight_decay),) * n)
        for what, v in (("dtypes", self.dtypes), ("grad_dtypes", self.grad_dtypes),
                        ("weight_decay", decay)):
            if len(v) != n:
                raise ValueError(f"{what}: {len(v)} given for {n} tensors")
        for d in self.dtypes + self.grad_dtypes:
            if d not in _tg.DTYPE_CODES:
                raise ValueError(f"unknown dtype {d!r}")
        self.lr, self.betas, self.eps = float(lr), (float(betas[0]), float(betas[1])), float(eps)
        self.weight_decay, self.state_bits = decay, int(state_bits)
        self.seed = int(seed) & 0xFFFFFFFFFFFFFFFF
        num = (ctypes.c_int64 * n)(*self.numels)
        dts = [_tg.DTYPE_CODES[d] for d in self.dtypes]
        gts = [_tg.DTYPE_CODES[d] for d in self.grad_dtypes]
        cd, cg = (ctypes.c_int * n)(*dts), (ctypes.c_int * n)(*gts)
        nbytes = self._lib.tgrad_adamw_state_bytes(n, num, cd, self.state_bits)
        if nbytes < 0:
            raise ValueError("numels must be >= 0 and state_bits 32 or 8")
        total = self._lib.tgrad_adamw_state_values(n, num, cd)
        at, self.offsets = 0, []
        for x, d in zip(self.numels, self.dtypes):
            self.offsets.append(at)
            at += -(-x * (2 if d == "c64" else 1) // GROUP) * GROUP
        self.device_index = torch.cuda.current_device()
        self._buf = torch.zeros(nbytes, dtype=torch.uint8, device=f"cuda:{self.device_index}")
        h = ctypes.c_void_p()
        rc = self._lib.tgrad_adamw_init(ctypes.byref(h), n, num, cd, cg, (ctypes.c_double * n)(*decay),
                                        self.state_bits, self.lr, *self.betas, self.eps, self.seed,
                                        ctypes.c_void_p(self._buf.data_ptr()))
        if rc != _tg.OK:
            raise _tg.TGradError(f"tgrad_adamw_init: {self._lib.tgrad_status_string(rc).decode()}")
        self._h = h
        self._plan = bind.adamw_plan(h.value, self.device_index, self.state_bits, total,
                                     list(self.numels), dts, gts)
        self._step, self._norm = bind.adamw_step, bind.adamw_grad_norm
        b, g = self._buf, total // GROUP
        if self.state_bits == 32:
            self.state = {"m": b[:4 * total].view(torch.float32), "v": b[4 * total:].view(torch.float32)}
        else:
            self.state = {"m": b[:total], "root_v": b[total:2 * total],
                          "m_scale": b[2 * total:2 * total + g], "root_v_scale": b[2 * total + g:]}

    # ---------------------------------------------------------------- lifecycle
    def close(self):
        if getattr(self, "_h", None):
            self._plan = None
            self._lib.tgrad_adamw_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, rc: int, what: str):
        if rc != _tg.OK:
            msg = self._lib.tgrad_status_string(rc).decode()
            detail = self._lib.tgrad_adamw_last_error(self._h).decode() if self._h else ""
            raise _tg.TGradError(f"{what}: {msg} {detail}".strip())

    # ---------------------------------------------------------------- hot path
    def step(self, weights, grads, clip=None, moments=None, stream=None):
        """One step of every tensor: weights[i] is updated in place from grads[i] (contiguous
        GPU tensors of numels[i] elements). clip: what grad_norm returned; where its norm is
        not finite, nothing changes. moments (8-bit states): two bf16 tensors of the flat
        state's length, which receive the new m and sqrt(v) as values."""
        self._step(self._plan, weights, grads, clip, moments, _stream(stream))

    def grad_norm(self, grads, max_norm: float = math.inf, grad_scale: float = 1.0, out=None,
                  stream=None):
        """Two floats on the GPU: the norm of all gradients together, times grad_scale (1 over
        the loss scale), and the coefficient that scales and clips them to max_norm. With a
        stream of your own, give `out` (memory that is ordered with it) as well."""
        return self._norm(self._plan, grads, max_norm, grad_scale, out, _stream(stream))

    def set_lr(self, lr: float):
        self._check(self._lib.tgrad_adamw_set_lr(self._h, float(lr)), "tgrad_adamw_set_lr")
        self.lr = float(lr)

    # ---------------------------------------------------------------- state
    @property
    def t(self) -> int:
        """Steps made (synchronises; a step left out for its norm does not count)."""
        n = ctypes.c_int64()
        self._check(self._lib.tgrad_adamw_get_steps(self._h, ctypes.byref(n)), "tgrad_adamw_get_steps")
        return n.value

    @t.setter
    def t(self, steps: int):
        self._check(self._lib.tgrad_adamw_set_steps(self._h, int(steps)), "tgrad_adamw_set_steps")

    def state_dict(self) -> dict:
        """Copies of the state, the step count and what the state depends on."""
        return {"numels": self.numels, "dtypes": self.dtypes, "state_bits": self.state_bits,
                "betas": self.betas, "eps": self.eps, "seed": self.seed, "t": self.t,
                "state": {k: v.clone() for k, v in self.state.items()}}

    def load_state_dict(self, saved: dict):
        """Continue from a state_dict of an optimizer of the same tensors, betas, eps and state
        format (the learning rate and the weight decay may differ, as a schedule changes them)."""
        for k in ("numels", "dtypes", "state_bits", "betas", "eps", "seed"):
            if saved[k] != getattr(self, k):
                raise ValueError(f"{k}: the state has {saved[k]}, the optimizer {getattr(self, k)}")
        for k, v in self.state.items():
            x = saved["state"][k]
            if x.shape != v.shape or x.dtype != v.dtype:
                raise ValueError(f"state {k}: {tuple(x.shape)} of {x.dtype}, expected {tuple(v.shape)} of {v.dtype}")
        for k, v in self.state.items():
            v.copy_(saved["state"][k])
        self.t = int(saved["t"])
