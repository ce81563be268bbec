"""Layer norm over the last axis (tgrad_layer_norm_* in include/tgrad.h), on the current
stream."""
from __future__ import annotations

import tensor_gradient_compression_amd as _tg


def layer_norm_forward(x, weight=None, bias=None, eps: float = 1e-5):
    """(y, mean, rstd) of x (float32, float16 or bfloat16; the last axis contiguous, the
    leading ones evenly spaced). weight, bias: None, or one value per column in float32 or
    x's type. mean and rstd are float32, of x's shape without the last axis. Autograd records
    nothing of this call, whatever its inputs require: layer_norm is the differentiable one."""
    return _tg.binding().layer_norm_forward(x, weight, bias, eps)


def layer_norm_backward(dy, x, weight, mean, rstd, params: bool = True):
    """(dx, dweight, dbias) from forward's inputs and statistics; dweight and dbias in the
    weight's type (x's without a weight), None where params is false. Autograd records nothing
    of this call."""
    return _tg.binding().layer_norm_backward(dy, x, weight, mean, rstd, params)


_function = None


def _layer_norm_function():
    global _function
    if _function is None:
        import torch

        class LayerNorm(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, weight, bias, eps):
                y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
                if weight is None and bias is not None and bias.dtype != x.dtype:
                    weight = torch.ones_like(bias)   # backward gives dbias the weight's type
                ctx.save_for_backward(x, weight, mean, rstd)
                return y

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dy):
                x, weight, mean, rstd = ctx.saved_tensors
                need = ctx.needs_input_grad
                # a gradient that autograd expanded (of a sum, say) has stride 0
                dx, dw, db = layer_norm_backward(dy.contiguous(), x, weight, mean, rstd,
                                                 params=bool(need[1] or need[2]))
                return (dx if need[0] else None, dw if need[1] else None, db if need[2] else None, None)

        _function = LayerNorm
    return _function


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """y = (x - mean) / sqrt(var + eps) * weight + bias over the last axis, with gradients (of
    the first order, in reverse mode). Inputs as those of layer_norm_forward."""
    return _layer_norm_function().apply(x, weight, bias, eps)
