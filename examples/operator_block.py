"""A training loop in which every tensor of a small model has its optimizer.

The model is one block of a Fourier neural operator in miniature: layer norm over the channels,
a product with a weight of its own for each of the modes (the large tensor, stepped by TGrad in
a compressed space), and a pointwise product with a bias beside it. The layer norm's weight and
bias and the pointwise part are stepped together by AdamW, here with moments of 8 bits, after
their gradients are clipped to a common norm; a step whose gradients are not finite is left out.

    python examples/operator_block.py [steps]
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tensor_gradient_compression_amd as tg  # noqa: E402

CHANNELS, MODES, BATCH = 8, (6, 6), 64


def block(u, norm_w, norm_b, modes_w, point_w, point_b):
    """u: (batch, modes, modes, channels)"""
    h = tg.layer_norm(u, norm_w, norm_b)
    mixed = (h.unsqueeze(-1) * modes_w.permute(2, 3, 0, 1)).sum(-2)
    return mixed + h @ point_w + point_b


def train(steps=200, state_bits=8, seed=0):
    """The losses of a run against a block with other weights."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale):
        return scale * torch.randn(*shape, generator=gen, device="cuda")

    def parameters():
        return [1 + normal(CHANNELS, scale=0.1), normal(CHANNELS, scale=0.1),
                normal(CHANNELS, CHANNELS, *MODES, scale=0.3), normal(CHANNELS, CHANNELS, scale=0.3),
                normal(CHANNELS, scale=0.1)]

    teacher = parameters()
    params = [p.requires_grad_() for p in parameters()]
    large, small = params[2], params[:2] + params[3:]
    tgrad = tg.TGrad(tuple(large.shape), (4, 4, 3, 3), "f32", sparse_ratio=0.05, T=20, lr=1e-2)
    # no decay for biases and norm weights
    adamw = tg.AdamW([p.numel() for p in small], "f32", lr=1e-2, weight_decay=[0.0, 0.0, 1e-4, 0.0],
                     state_bits=state_bits, seed=seed)
    losses = []
    for _ in range(steps):
        u = normal(BATCH, *MODES, CHANNELS, scale=1.0)
        loss = (block(u, *params) - block(u, *teacher)).square().mean()
        grads = torch.autograd.grad(loss, params)
        small_grads = [g.contiguous() for g in grads[:2] + grads[3:]]
        tgrad.step(large.detach(), grads[2].contiguous())
        adamw.step(small, small_grads, clip=adamw.grad_norm(small_grads, max_norm=1.0))
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    losses = train(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:5d}  loss {losses[i]:.4f}")
    print(f"last        loss {losses[-1]:.4f}")
