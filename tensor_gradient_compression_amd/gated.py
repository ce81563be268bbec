"""Gated linear layer (tgrad_gated_linear_* in include/tgrad.h), on the current stream."""
from __future__ import annotations

import tensor_gradient_compression_amd as _tg

ACTIVATIONS = {"silu": 0, "gelu": 1, "sigmoid": 2, "relu": 3}


def _code(activation: str) -> int:
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}: one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[activation]


def gated_linear_forward(x, w_gate, w_up, b_gate=None, b_up=None, activation: str = "silu"):
    """y = act(x w_gate^T + b_gate) * (x w_up^T + b_up) over x's last axis (float32, float16 or
    bfloat16; the last axis contiguous, the leading ones evenly spaced). w_gate, w_up: contiguous
    (hidden, in); b_gate, b_up: None or hidden values; all of x's type. activation: "silu",
    "gelu" (the exact one), "sigmoid" or "relu". Autograd records nothing of this call:
    gated_linear is the differentiable one."""
    return _tg.binding().gated_linear_forward(x, w_gate, w_up, b_gate, b_up, _code(activation))


def gated_linear_backward(dy, x, w_gate, w_up, b_gate=None, b_up=None, activation: str = "silu",
                          need_dx: bool = True, need_weights: bool = True):
    """(dx, dw_gate, dw_up, db_gate, db_up) from forward's inputs alone; db is None for a bias
    that is None, and all but dx are where need_weights is false. Autograd records nothing of
    this call."""
    bias = need_weights and (b_gate is not None or b_up is not None)
    dx, dwg, dwu, dbg, dbu = _tg.binding().gated_linear_backward(
        dy, x, w_gate, w_up, b_gate, b_up, _code(activation), need_dx, need_weights, bias)
    return dx, dwg, dwu, dbg if b_gate is not None else None, dbu if b_up is not None else None


_function = None


def _gated_linear_function():
    global _function
    if _function is None:
        import torch

        class GatedLinear(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, w_gate, w_up, b_gate, b_up, activation):
                ctx.save_for_backward(x, w_gate, w_up, b_gate, b_up)
                ctx.activation = activation
                return gated_linear_forward(x, w_gate, w_up, b_gate, b_up, activation)

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dy):
                need = ctx.needs_input_grad
                # a gradient that autograd expanded (of a sum, say) has stride 0
                grads = gated_linear_backward(dy.contiguous(), *ctx.saved_tensors, activation=ctx.activation,
                                              need_dx=need[0], need_weights=any(need[1:5]))
                return tuple(g if n else None for g, n in zip(grads, need)) + (None,)

        _function = GatedLinear
    return _function


def gated_linear(x, w_gate, w_up, b_gate=None, b_up=None, activation: str = "silu"):
    """gated_linear_forward with gradients (of the first order, in reverse mode). The backward
    pass forms the two products again from x: nothing but the inputs is kept for it."""
    return _gated_linear_function().apply(x, w_gate, w_up, b_gate, b_up, activation)
