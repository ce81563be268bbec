"""A training loop for a block whose matrices are trained by Muon.

The block mixes the channels of every point of a field: layer norm, a gated linear layer that
expands them, and a product that contracts them again, with the input added. Its three matrices
are stepped by Muon, the norm's weight and bias and the gate's biases by AdamW; the gradients of
both are clipped by the norm over all of them, and a step whose gradients are not finite is left
out by both.

    python examples/channel_mixer.py [steps]
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tensor_gradient_compression_amd as tg  # noqa: E402

CHANNELS, HIDDEN, POINTS = 24, 72, 400


def block(x, norm_w, norm_b, gate_b, up_b, gate_w, up_w, down_w):
    """x: (points, channels)"""
    h = tg.gated_linear(tg.layer_norm(x, norm_w, norm_b), gate_w, up_w, gate_b, up_b, activation="gelu")
    return x + h @ down_w


class Loop:
    """A block, its optimizers, and another block whose outputs it learns."""

    def __init__(self, dtype=torch.float32, seed=0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype = dtype
        self.teacher = self.parameters()
        self.params = [p.requires_grad_() for p in self.parameters()]
        name = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[dtype]
        self.muon = tg.Muon([tuple(p.shape) for p in self.params[4:]], name, lr=0.02, weight_decay=0.01)
        # the norm is that of all gradients, in an optimizer's handle that steps nothing
        self.norm = tg.AdamW([p.numel() for p in self.params], name)
        self.adamw = tg.AdamW([p.numel() for p in self.params[:4]], name, lr=1e-2, weight_decay=0.0)

    def normal(self, *shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=self.gen, device="cuda")).to(self.dtype)

    def parameters(self):
        return [1 + self.normal(CHANNELS, scale=0.1), self.normal(CHANNELS, scale=0.1),
                self.normal(HIDDEN, scale=0.1), self.normal(HIDDEN, scale=0.1),
                self.normal(HIDDEN, CHANNELS, scale=CHANNELS ** -0.5), self.normal(HIDDEN, CHANNELS, scale=CHANNELS ** -0.5),
                self.normal(HIDDEN, CHANNELS, scale=HIDDEN ** -0.5)]

    def gradients(self, x):
        """(loss, gradients) at the inputs x"""
        loss = (block(x, *self.params) - block(x, *self.teacher)).float().square().mean()
        return loss.detach(), [g.contiguous() for g in torch.autograd.grad(loss, self.params)]

    def step(self, grads, max_norm=1.0):
        weights = [p.detach() for p in self.params]
        clip = self.norm.grad_norm(grads, max_norm=max_norm)
        self.adamw.step(weights[:4], grads[:4], clip=clip)
        self.muon.step(weights[4:], grads[4:], clip=clip)


def train(steps=200, dtype=torch.float32, seed=0):
    """The losses of a run."""
    loop = Loop(dtype, seed)
    losses = []
    for _ in range(steps):
        loss, grads = loop.gradients(loop.normal(POINTS, CHANNELS))
        loop.step(grads)
        losses.append(loss)
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    losses = train(int(sys.argv[1]) if len(sys.argv) > 1 else 200)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:5d}  loss {losses[i]:.4f}")
    print(f"last        loss {losses[-1]:.4f}")
