"""Trains a small pre-norm decoder with a weight-tied head, forward and backward
by hand, on the library's operators:

    x = E[ids]
    per layer:  q, k, v = norm(x) Wqkv + bqkv, q and k turned by their position
                x = x + dropout(attention(q, k, v) Wo)
                x = x + dropout(gelu(norm(x) W1 + b1) W2)
    loss = xent(norm(x) E^T, next id)

Documents of different lengths are packed one behind the other: attention and
positions stay within a document.  AdamW keeps binary32 parameters, their
bfloat16 copies are what the model computes with, and the optimizer's states are
held in 8 bits (or 32).  The matrix products are torch's.

    python examples/train_gpt.py [steps] [8|32]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import broadcast_elementwise_shape_gb300 as zr  # noqa: E402


class Model:
    """Parameters, their copies, and the optimizer's states."""

    def __init__(self, vocab=301, width=192, heads=6, kv_heads=2, layers=2, bits=8, seed=1):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.layers, self.bits = heads, kv_heads, width // heads, layers, bits
        self.plan = zr.zr_rotary_plan(self.dim)
        rows = (heads + 2 * kv_heads) * self.dim
        shapes = {"E": (vocab, width), "gf": (width,), "bf": (width,)}
        for i in range(layers):
            shapes |= {f"{i}.g1": (width,), f"{i}.b1": (width,), f"{i}.Wqkv": (width, rows), f"{i}.bqkv": (rows,), f"{i}.Wo": (width, width),
                       f"{i}.g2": (width,), f"{i}.b2": (width,), f"{i}.W1": (width, 4 * width), f"{i}.c1": (4 * width,), f"{i}.W2": (4 * width, width)}
        self.master = {}
        for n, s in shapes.items():
            if len(s) == 2:
                std = 0.05 if n == "E" else s[0] ** -0.5 * (0.5 if n.endswith(("Wo", "W2")) else 1)
                self.master[n] = torch.randn(s, generator=gen, device="cuda") * std
            else:
                self.master[n] = torch.ones(s, device="cuda") if n.split(".")[-1][0] == "g" else torch.zeros(s, device="cuda")
        self.w = {n: x.bfloat16() for n, x in self.master.items()}
        state = torch.uint8 if bits == 8 else torch.float32
        self.m, self.v = ([torch.zeros(x.shape, dtype=state, device="cuda") for x in self.master.values()] for _ in range(2))
        self.scales = [[torch.zeros(-(-x.numel() // 256), device="cuda") for x in self.master.values()] for _ in range(2)] if bits == 8 else (None, None)
        self.decay = [0.1 if x.dim() == 2 else 0.0 for x in self.master.values()]
        self.step = 0

    def loss_and_grads(self, ids, labels, offsets, positions, p=0.1, seed=1):
        """The mean loss of packed tokens and every parameter's gradient."""
        w, h, kv, d = self.w, self.heads, self.kv_heads, self.dim
        counter = self.step << 40  # each step and dropout its own mask

        def drop(i):
            return seed, counter + (i << 32)

        x = w["E"][ids]
        kept = []
        for i in range(self.layers):
            n1, mu1, rs1 = zr.zr_layer_norm_fwd(x, w[f"{i}.g1"], w[f"{i}.b1"])
            qkv = zr.zr_binary_fwd("add", n1 @ w[f"{i}.Wqkv"], w[f"{i}.bqkv"]).view(-1, h + 2 * kv, d)
            zr.zr_rotary_fwd(qkv[:, :h + kv], self.plan, positions, out=qkv[:, :h + kv])
            q, k, v = qkv.split([h, kv, kv], 1)
            a, lse, low = zr.zr_attention_fwd(q, k, v, None, offsets, keep_low=True)
            x1 = zr.zr_dropout_fwd(a.flatten(1) @ w[f"{i}.Wo"], p, *drop(2 * i), residual=x)
            n2, mu2, rs2 = zr.zr_layer_norm_fwd(x1, w[f"{i}.g2"], w[f"{i}.b2"])
            f = zr.zr_binary_fwd("add", n2 @ w[f"{i}.W1"], w[f"{i}.c1"])
            u = zr.zr_unary_fwd("gelu", f)
            kept.append((x, n1, mu1, rs1, q, k, v, a, lse, low, x1, n2, mu2, rs2, f, u))
            x = zr.zr_dropout_fwd(u @ w[f"{i}.W2"], p, *drop(2 * i + 1), residual=x1)
        y, mu, rs = zr.zr_layer_norm_fwd(x, w["gf"], w["bf"])
        loss, lse = zr.zr_linear_xent_fwd(y, w["E"], labels)
        g = {}
        gy, g["E"] = zr.zr_linear_xent_bwd(torch.ones((), device="cuda"), y, w["E"], labels, lse)
        gx, g["gf"], g["bf"] = zr.zr_layer_norm_bwd(gy, x, w["gf"], mu, rs)
        for i in reversed(range(self.layers)):
            x, n1, mu1, rs1, q, k, v, a, lse, low, x1, n2, mu2, rs2, f, u = kept[i]
            gf = zr.zr_dropout_bwd(gx, p, *drop(2 * i + 1))
            g[f"{i}.W2"] = u.t() @ gf
            gu = zr.zr_unary_bwd("gelu", gf @ w[f"{i}.W2"].t(), f)
            gu, g[f"{i}.c1"] = zr.zr_binary_bwd("add", gu, f, w[f"{i}.c1"])
            g[f"{i}.W1"] = n2.t() @ gu
            gn, g[f"{i}.g2"], g[f"{i}.b2"] = zr.zr_layer_norm_bwd(gu @ w[f"{i}.W1"].t(), x1, w[f"{i}.g2"], mu2, rs2)
            gx = zr.zr_binary_fwd("add", gx, gn)
            ga = zr.zr_dropout_bwd(gx, p, *drop(2 * i))
            g[f"{i}.Wo"] = a.flatten(1).t() @ ga
            grad = torch.empty(len(ids), h + 2 * kv, d, dtype=torch.bfloat16, device="cuda")
            zr.zr_attention_bwd((ga @ w[f"{i}.Wo"].t()).view_as(a), q, k, v, a, lse, low, None, offsets, grads=grad.split([h, kv, kv], 1))
            zr.zr_rotary_bwd(grad[:, :h + kv], self.plan, positions, grad_x=grad[:, :h + kv])
            grad = grad.flatten(1)
            grad, g[f"{i}.bqkv"] = zr.zr_binary_bwd("add", grad, grad, w[f"{i}.bqkv"])
            g[f"{i}.Wqkv"] = n1.t() @ grad
            gn, g[f"{i}.g1"], g[f"{i}.b1"] = zr.zr_layer_norm_bwd(grad @ w[f"{i}.Wqkv"].t(), x, w[f"{i}.g1"], mu1, rs1)
            gx = zr.zr_binary_fwd("add", gx, gn)
        g["E"] = g["E"].float().index_add_(0, ids, gx.float()).bfloat16()
        return loss, g

    def update(self, grads, lr=3e-3):
        self.step += 1
        zr.zr_adamw_step(list(self.master.values()), [grads[n].contiguous() for n in self.master], self.m, self.v, self.step, lr, (0.9, 0.99), 1e-8,
                         self.decay, copies=list(self.w.values()), m_scales=self.scales[0], v_scales=self.scales[1], seed=7)


def text(vocab, lengths, gen):
    """Packed ids and next ids of documents in which every character is followed by a fixed other one three times out of four."""
    follow = torch.randperm(vocab, generator=gen, device="cuda")
    ids, labels, positions = [], [], []
    for n in lengths:
        d = torch.randint(0, vocab, (n + 1,), generator=gen, device="cuda")
        keep = torch.rand(n + 1, generator=gen, device="cuda") < 0.75
        for t in range(1, n + 1):
            d[t] = torch.where(keep[t], follow[d[t - 1]], d[t])
        ids.append(d[:-1])
        labels.append(d[1:])
        positions.append(torch.arange(n, device="cuda"))
    offsets = torch.tensor([0, *lengths], device="cuda").cumsum(0).int()
    return torch.cat(ids), torch.cat(labels), offsets, torch.cat(positions)


def train(steps=60, bits=8, lengths=(200, 1, 77, 300, 129), seed=1):
    """The loss of every step (one read at the end)."""
    model = Model(bits=bits, seed=seed)
    ids, labels, offsets, positions = text(301, lengths, torch.Generator("cuda").manual_seed(seed))
    losses = []
    for _ in range(steps):
        loss, grads = model.loss_and_grads(ids, labels, offsets, positions)
        losses.append(loss)
        model.update(grads)
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 60
    losses = train(steps, int(sys.argv[2]) if len(sys.argv) > 2 else 8)
    for i in range(0, steps, max(1, steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {steps - 1:4d}  loss {losses[-1]:.4f}  (log vocab {math.log(301):.4f})")
