"""The operators together, as a decoder's training step runs them: the example
runs, and its gradients are those of the same model in 64-bit autograd.

The bound on a gradient is statistical: each of the chain's L = 12 stored bfloat16 tensors per layer carries a relative rounding of at
most 2^-8 (rms 2^-8 / sqrt(3)); over two layers forward and backward that is sqrt(2 * 2 * 12) * 2^-8 / sqrt(3) = 0.016 of a
gradient's norm if they add as independent errors, and three times that is allowed.
"""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_gpt  # noqa: E402

pytestmark = pytest.mark.gpu


def model64(w, model, ids, labels, lengths, positions):
    h, kv, d = model.heads, model.kv_heads, model.dim
    norm = lambda x, g, b: torch.nn.functional.layer_norm(x, x.shape[-1:], g, b, 1e-5)  # noqa: E731
    f = 10000.0 ** (-2 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    a = (positions.double()[:, None] * f)[:, None]

    def turn(x):
        u, v = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()], -1)

    x = w["E"][ids]
    for i in range(model.layers):
        q, k, v = (norm(x, w[f"{i}.g1"], w[f"{i}.b1"]) @ w[f"{i}.Wqkv"] + w[f"{i}.bqkv"]).view(-1, h + 2 * kv, d).split([h, kv, kv], 1)
        q, k = turn(q), turn(k)
        outs, at = [], 0
        for n in lengths:
            s = slice(at, at + n)
            at += n
            kk, vv = (y[s].repeat_interleave(h // kv, 1).transpose(0, 1) for y in (k, v))
            z = q[s].transpose(0, 1) @ kk.transpose(1, 2) * d ** -0.5
            z = z.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)
            outs.append((z.softmax(-1) @ vv).transpose(0, 1))
        x = x + torch.cat(outs).flatten(1) @ w[f"{i}.Wo"]
        x = x + torch.nn.functional.gelu(norm(x, w[f"{i}.g2"], w[f"{i}.b2"]) @ w[f"{i}.W1"] + w[f"{i}.c1"]) @ w[f"{i}.W2"]
    return torch.nn.functional.cross_entropy(norm(x, w["gf"], w["bf"]) @ w["E"].t(), labels)


def test_gradients_of_the_chain():
    lengths = (200, 1, 77, 300, 129)
    model = train_gpt.Model()
    ids, labels, offsets, positions = train_gpt.text(301, lengths, torch.Generator("cuda").manual_seed(3))
    loss, grads = model.loss_and_grads(ids, labels, offsets, positions, p=0.0)
    w = {n: x.double().requires_grad_() for n, x in model.w.items()}
    want = model64(w, model, ids, labels, lengths, positions)
    want.backward()
    assert abs(float(loss) - float(want)) < 0.01 * float(want)
    for n, x in w.items():
        assert grads[n].shape == x.shape
        off = float((grads[n].double() - x.grad).norm() / x.grad.norm())
        assert off < 3 * 0.016, (n, off)


@pytest.mark.parametrize("bits", [8, 32])
def test_example_runs(bits):
    losses = train_gpt.train(steps=5, bits=bits)
    assert len(losses) == 5 and all(math.isfinite(x) for x in losses)


def test_captured_step():
    """Forward, backward and optimizer step as one graph, replayed: the same numbers as without it."""
    lengths = (100, 29)
    models = [train_gpt.Model(bits=8) for _ in range(2)]
    ids, labels, offsets, positions = train_gpt.text(301, lengths, torch.Generator("cuda").manual_seed(3))
    for m in models:  # warm up the products' workspaces
        m.update(m.loss_and_grads(ids, labels, offsets, positions)[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grads = models[0].loss_and_grads(ids, labels, offsets, positions)
        models[0].update(grads)
    graph.replay()
    other, grads = models[1].loss_and_grads(ids, labels, offsets, positions)
    models[1].update(grads)
    assert abs(float(loss) - float(other)) < 1e-3 * float(other)
    off = [float((a - b).abs().max()) for a, b in zip(models[0].master.values(), models[1].master.values())]
    # torch's products and index_add may add in another order; a step moves an element by at most about lr * 10.
    assert max(off) <= 2 * 10 * 3e-3
