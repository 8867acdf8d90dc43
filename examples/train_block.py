"""Trains a small pre-norm feed-forward block with a weight-tied head, forward
and backward by hand, on the library's operators:

    e = E[ids] + P                      broadcast add
    f = gelu(norm(e) W1 + b1) W2        layer norm, broadcast add, GeLU
    h = e + dropout(f)                  dropout with its residual
    loss = xent(norm(h) E^T, next id)   layer norm, cross entropy of the head

The matrix products are torch's.  The text is one synthetic batch, in which
every character is followed by a fixed other one three times out of four; the
block learns it by heart, so the loss falls from log(vocab) towards 0.

    python examples/train_block.py [steps] [bf16|f32]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import broadcast_elementwise_shape_gb300 as zr  # noqa: E402


def text(vocab, batch, length, gen):
    """ids [batch, length] of the synthetic source."""
    follow = torch.randperm(vocab, generator=gen, device="cuda")
    ids = torch.randint(0, vocab, (batch, length), generator=gen, device="cuda")
    for t in range(1, length):
        jump = torch.rand(batch, generator=gen, device="cuda") < 0.25
        ids[:, t] = torch.where(jump, ids[:, t], follow[ids[:, t - 1]])
    return ids


def train(steps=60, dtype=torch.bfloat16, vocab=301, width=192, batch=32, length=64, p=0.1, lr=0.01, seed=1):
    """The loss of every step (one read at the end)."""
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    w = {"E": normal(vocab, width, std=0.05), "P": normal(length, width, std=0.02),
         "g1": torch.ones(width, dtype=dtype, device="cuda"), "b1": torch.zeros(width, dtype=dtype, device="cuda"),
         "W1": normal(width, 4 * width, std=width ** -0.5),
         "c1": torch.zeros(4 * width, dtype=dtype, device="cuda"),
         "W2": normal(4 * width, width, std=0.5 * width ** -0.5),
         "g2": torch.ones(width, dtype=dtype, device="cuda"), "b2": torch.zeros(width, dtype=dtype, device="cuda")}
    master = {k: v.float() for k, v in w.items()}
    m1 = {k: torch.zeros_like(v) for k, v in master.items()}
    m2 = {k: torch.zeros_like(v) for k, v in master.items()}
    ids = text(vocab, batch, length + 1, gen)
    inputs, labels = ids[:, :-1], ids[:, 1:].clone()
    labels[:, ::16] = -100  # positions that are not trained on
    one = torch.ones((), device="cuda")
    offset, losses = 0, []
    for step in range(steps):
        # Forward.
        e = zr.zr_binary_fwd("add", w["E"][inputs], w["P"])
        n, mu1, rs1 = zr.zr_layer_norm_fwd(e, w["g1"], w["b1"])
        a = zr.zr_binary_fwd("add", n @ w["W1"], w["c1"])
        u = zr.zr_unary_fwd("gelu", a)
        f = u @ w["W2"]
        h = zr.zr_dropout_fwd(f, p, seed, offset, residual=e)
        y, mu2, rs2 = zr.zr_layer_norm_fwd(h, w["g2"], w["b2"])
        loss, lse = zr.zr_linear_xent_fwd(y, w["E"], labels)
        losses.append(loss)
        # Backward.
        g = {}
        gy, g["E"] = zr.zr_linear_xent_bwd(one, y, w["E"], labels, lse)
        gh, g["g2"], g["b2"] = zr.zr_layer_norm_bwd(gy, h, w["g2"], mu2, rs2)
        gf = zr.zr_dropout_bwd(gh, p, seed, offset)
        g["W2"] = u.flatten(0, 1).t() @ gf.flatten(0, 1)
        ga = zr.zr_unary_bwd("gelu", gf @ w["W2"].t(), a)
        ga, g["c1"] = zr.zr_binary_bwd("add", ga, a, w["c1"])
        g["W1"] = n.flatten(0, 1).t() @ ga.flatten(0, 1)
        ge, g["g1"], g["b1"] = zr.zr_layer_norm_bwd(ga @ w["W1"].t(), e, w["g1"], mu1, rs1)
        ge = zr.zr_binary_fwd("add", ge, gh)
        _, g["P"] = zr.zr_binary_bwd("add", ge, e, w["P"])
        g["E"] = g["E"].float().index_add_(0, inputs.flatten(), ge.flatten(0, 1).float())
        offset += (f.numel() + 3) // 4  # the next step's own mask
        # Adam on binary32 masters.
        for k, x in master.items():
            d = g[k].float()
            m1[k].lerp_(d, 0.1)
            m2[k].lerp_(d * d, 0.01)
            x -= lr * (m1[k] / (1 - 0.9 ** (step + 1))) / ((m2[k] / (1 - 0.99 ** (step + 1))).sqrt() + 1e-8)
            w[k] = x.to(dtype)
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 60
    dtype = torch.float32 if sys.argv[2:] == ["f32"] else torch.bfloat16
    losses = train(steps, dtype)
    for i in range(0, steps, max(1, steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {steps - 1:4d}  loss {losses[-1]:.4f}  (log vocab {math.log(301):.4f})")
