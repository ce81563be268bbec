"""GPU: layer norm, the gated linear layer, the shared norm, AdamW and Muon together, as the example
runs them: its gradients, its steps, and a captured step."""
import os
import sys

import numpy as np
import pytest

import oracle.muon_oracle as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def host(t):
    return t.detach().double().cpu()


def plain_block(x, nw, nb, gb, ub, gw, uw, dw):
    h = torch.nn.functional.layer_norm(x, x.shape[-1:], nw, nb)
    return x + (torch.nn.functional.gelu(h @ gw.T + gb) * (h @ uw.T + ub)) @ dw


def plain_gradients(loop, x):
    params = [host(p).requires_grad_() for p in loop.params]
    loss = (plain_block(host(x), *params) - plain_block(host(x), *[host(p) for p in loop.teacher])).square().mean()
    return float(loss.detach()), torch.autograd.grad(loss, params)


@pytest.mark.parametrize("dtype,eps", [(torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)])
def test_its_gradients(dtype, eps):
    """Against the same block in 64 bits. A value of the block goes through six roundings (norm, gate
    and up, their product, the contraction, the sum) each way and every gradient sums 400 points or
    more, whose roundings are independent: 16 roundings' worth of the gradient's 2-norm, and the loss's
    residual, a difference of two blocks about as large as either, twice that again."""
    import channel_mixer as ex
    loop = ex.Loop(dtype, seed=1)
    x = loop.normal(ex.POINTS, ex.CHANNELS)
    loss, grads = loop.gradients(x)
    want, true = plain_gradients(loop, x)
    assert abs(float(loss) - want) <= 32 * eps * want
    for g, t in zip(grads, true):
        assert (host(g) - t).norm() <= 32 * eps * t.norm()


def test_a_step_is_the_recipe():
    """From its own gradients: the norm over all of them, AdamW's first step and Muon's, in 64 bits."""
    import channel_mixer as ex
    loop = ex.Loop(seed=2)
    loss, grads = loop.gradients(loop.normal(ex.POINTS, ex.CHANNELS))
    before = [host(p) for p in loop.params]
    max_norm = 0.5 * float(sum(host(g).square().sum() for g in grads).sqrt())
    loop.step(grads, max_norm=max_norm)
    for i, (p, b, g) in enumerate(zip(loop.params, before, grads)):
        g = host(g) * 0.5
        if i < 4:       # the first moments' ratio is the gradient's sign
            want = b - 1e-2 * g / (g.abs() + 1e-8)
            # the step's own roundings, and the coefficient's in a ratio that a small eps lets move
            assert torch.all((host(p) - want).abs() <= 2.0 ** -24 * (b.abs() + 1e-2 * 16) + 1e-2 * 2.0 ** -20)
            continue
        opt = loop.muon
        m, u = M.momentum(g.numpy(), 0.0, opt.momentum, opt.nesterov)
        true = M.orthogonalize(u)
        e2, em = M.bounds(u, true, "f32")
        step = opt.lr * opt.scale[i - 4]
        want = b.numpy() * (1 - opt.lr * 0.01) - step * true
        off = np.abs(host(p).numpy() - want)
        # the norm of u is rounded nowhere that a change of the gradient's coefficient by 2^-23 would show
        assert np.all(off <= step * (em + 2.0 ** -20) + 8 * 2.0 ** -24 * (np.abs(want) + step))


def test_gradients_that_are_not_finite_leave_both_out():
    import channel_mixer as ex
    loop = ex.Loop(seed=3)
    loss, grads = loop.gradients(loop.normal(ex.POINTS, ex.CHANNELS))
    grads[0][3] = float("inf")
    before = [p.detach().clone() for p in loop.params]
    loop.step(grads)
    assert all(torch.equal(p, b) for p, b in zip(loop.params, before))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_captured_loop_is_the_eager_one(dtype):
    """Forward, backward and both steps in one graph, replayed on other inputs, bit for bit."""
    import channel_mixer as ex

    def run(loop, inputs, captured):
        x = inputs[0].clone()

        def once():
            out, grads = loop.gradients(x)
            loop.step(grads)
            return out

        losses = []
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                first = once()
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            losses.append(first.clone())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                loss = once()
            for v in inputs[1:]:
                x.copy_(v)
                graph.replay()
                torch.cuda.synchronize()
                losses.append(loss.clone())
        else:
            for v in inputs:
                x.copy_(v)
                losses.append(once().clone())
        return losses, [p.detach().clone() for p in loop.params]

    gen = torch.Generator(device="cuda").manual_seed(7)
    inputs = [torch.randn(ex.POINTS, ex.CHANNELS, generator=gen, device="cuda").to(dtype) for _ in range(5)]
    eager = run(ex.Loop(dtype, seed=4), inputs, False)
    replayed = run(ex.Loop(dtype, seed=4), inputs, True)
    assert all(torch.equal(a, b) for a, b in zip(eager[1], replayed[1]))
    assert all(torch.equal(a, b) for a, b in zip(eager[0], replayed[0]))


def test_it_runs_and_repeats():
    import channel_mixer as ex
    losses = ex.train(5)
    assert len(losses) == 5 and all(np.isfinite(losses)) and ex.train(5) == losses
