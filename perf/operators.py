"""Layer norm, dropout with its residual, and the cross entropy of a linear
head: the cases they are measured on.

A case names an operator (``op``), a direction (``way``), an element type
(``dtype``) and its sizes.  ``run`` with ``own`` false computes the plain
form in elementary torch operations (32-bit arithmetic, rounded once at the
end); with ``own`` true it calls this package.  ``exact`` is the definition
in 64 bits.

* ``layer_norm``: x [rows, dim], ``pitch`` extra elements between rows.
  way ``fwd`` gives (y, mean, rstd), ``bwd`` (grad_x, grad_gamma, grad_beta).
* ``dropout``: x [rows, dim]; element i (row-major) is kept when word i mod 4
  of Philox4x32-10 (J. K. Salmon, M. A. Moraes, R. O. Dror and D. E. Shaw,
  "Parallel random numbers: as easy as 1, 2, 3", SC 2011) at counter
  offset + i div 4, keyed by the seed, is at least round(p * 2^32).
  way ``fwd`` gives residual + keep * x / (1 - p), ``bwd`` keep * g / (1 - p).
* ``xent``: hidden rows x [rows, dim], head weight w [vocab, dim], labels
  [rows], some of them ignored.  way ``fwd`` gives (mean loss, per-row log of
  the sum of exponentials), ``step`` also the gradients of x and w.
"""
import math

import numpy as np
import torch

own = False

IGNORE = -100
EPS = 1e-5
_M = 0xFFFFFFFF


def listed():
    return [
        # One token's residual stream between two blocks while generating: latency counts.
        dict(name="ln_fwd_token", op="layer_norm", way="fwd", dtype="bf16", rows=1, dim=768, pitch=0),
        # The batch of the affine workload, [16, 1024, 768], in 32 bits.
        dict(name="ln_fwd_batch", op="layer_norm", way="fwd", dtype="f32", rows=16384, dim=768, pitch=0),
        dict(name="ln_bwd_batch", op="layer_norm", way="bwd", dtype="f32", rows=16384, dim=768, pitch=0),
        # Odd width and an odd number of rows, cut out of a wider buffer.
        dict(name="ln_bwd_ragged", op="layer_norm", way="bwd", dtype="bf16", rows=4093, dim=1001, pitch=23),
        # A long-context batch in bf16.
        dict(name="ln_bwd_large", op="layer_norm", way="bwd", dtype="bf16", rows=65536, dim=1024, pitch=0),
        # The residual after one 256-token sequence of a small model of width 384.
        dict(name="drop_fwd_small", op="dropout", way="fwd", dtype="f32", rows=256, dim=384),
        # The batch of the affine workload in bf16, with its residual.
        dict(name="drop_fwd_batch", op="dropout", way="fwd", dtype="bf16", rows=16384, dim=768),
        # The gradient of a large batch.
        dict(name="drop_bwd_large", op="dropout", way="bwd", dtype="f32", rows=65536, dim=1536),
        # Scoring one token against a large vocabulary.
        dict(name="xent_fwd_token", op="xent", way="fwd", dtype="bf16", rows=1, vocab=50001, dim=768),
        # A small character-level model in 32 bits: 16 sequences of 256 less one token, an odd vocabulary.
        dict(name="xent_step_chars", op="xent", way="step", dtype="f32", rows=4080, vocab=5003, dim=384),
        # An ordinary training batch.
        dict(name="xent_step_batch", op="xent", way="step", dtype="bf16", rows=4096, vocab=32000, dim=1024),
        # A large batch and an odd, large vocabulary.
        dict(name="xent_step_large", op="xent", way="step", dtype="bf16", rows=16384, vocab=50001, dim=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "dropout", "xent"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "xent":
        # A 32-bit product costs several 16-bit ones: fewer of them, so that no draw costs more than the largest case.
        most = 16384 * 50001 * 768 // (12 if dtype == "f32" else 1)
        dim = _log(rng, 64, 2048)
        if rng.random() < 0.5:
            dim = -(-dim // 64) * 64
        vocab = _log(rng, 500, 130000)
        rows = _log(rng, 1, max(1, min(16384, most // (dim * vocab))))
        return dict(op=op, way=rng.choice(["fwd", "step"]), dtype=dtype, rows=rows, vocab=vocab, dim=dim)
    dim = _log(rng, 48, 8192)
    if rng.random() < 0.6:
        dim = -(-dim // 64) * 64
    rows = _log(rng, 1, 65536 * 1536 // dim)
    case = dict(op=op, way=rng.choice(["fwd", "bwd"]), dtype=dtype, rows=rows, dim=dim)
    if op == "layer_norm":
        case["pitch"] = rng.choice([0, 0, rng.randrange(1, 64)])
    return case


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, rows, dim = _dtype(case), case["rows"], case["dim"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    state = {"case": case}
    if case["op"] == "layer_norm":
        # A residual stream: channels of different size and mean, a few of them large.
        wide = dim + case["pitch"]
        size = torch.exp(0.5 * normal(wide)) * (1 + 6 * (uniform(0, 1, wide) < 0.01))
        x = normal(rows, wide).mul_(size).add_(0.5 * normal(wide)).to(dt)[:, :dim]
        state.update(x=x, gamma=uniform(0.5, 1.5, dim).to(dt), beta=(0.1 * normal(dim)).to(dt))
        if case["way"] == "bwd":
            xf = x.float()
            mean = xf.sum(1) / dim
            var = (xf - mean[:, None]).square_().sum(1) / dim
            state.update(grad=normal(rows, wide).to(dt)[:, :dim], mean=mean, rstd=1 / torch.sqrt(var + EPS))
    elif case["op"] == "dropout":
        state.update(x=normal(rows, dim).to(dt), p=0.2, seed=0x9E3779B97F4A7C15 ^ seed, offset=(seed * 7919 + 12345 << 20) & (1 << 62) - 1)
        if case["way"] == "fwd":
            state.update(residual=(2 * normal(rows, dim)).to(dt))
    else:
        # Rows of unit variance that lean towards their label's weight by an amount of their own, so that some labels
        # are near certain and some are lost in the vocabulary; about one row in sixteen is padding.
        vocab = case["vocab"]
        w = (normal(vocab, dim) / math.sqrt(dim)).to(dt)
        labels = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        x = (normal(rows, dim) + uniform(0, 12, rows, 1) * w[labels].float()).to(dt)
        labels = torch.where(uniform(0, 1, rows) < 1 / 16, torch.full_like(labels, IGNORE), labels) if rows > 1 else labels
        state.update(x=x, w=w, labels=labels)
        if case["way"] == "step":
            state["grad_loss"] = uniform(0.5, 1.0, 1)  # 1 / (accumulated batches), as a loss scale gives it
    return state


def _plain_layer_norm_fwd(s):
    dim = s["x"].shape[1]
    x = s["x"].float()
    mean = x.sum(1) / dim
    c = x - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).sum(1) / dim + EPS)
    y = c * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    return y.to(s["x"].dtype), mean, rstd


def _plain_layer_norm_bwd(s):
    dim, dt = s["x"].shape[1], s["x"].dtype
    g = s["grad"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    q = g * s["gamma"].float()
    gx = s["rstd"][:, None] * (q - q.sum(1, keepdim=True) / dim - xhat * ((q * xhat).sum(1, keepdim=True) / dim))
    return gx.to(dt), (g * xhat).sum(0).to(dt), g.sum(0).to(dt)


def _keep(n, p, seed, offset, device):
    """Which of n elements are kept: Philox4x32-10 in 64-bit integers, whose products wrap as unsigned ones do."""
    k = torch.arange((n + 3) // 4, device=device, dtype=torch.int64)
    low = (offset & _M) + k
    c0, c1 = low & _M, ((offset >> 32) + (low >> 32)) & _M
    c2 = c3 = torch.zeros_like(c0)
    k0, k1 = seed & _M, (seed >> 32) & _M
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & _M) ^ c1 ^ k0, b & _M, ((a >> 32) & _M) ^ c3 ^ k1, a & _M
        k0, k1 = (k0 + 0x9E3779B9) & _M, (k1 + 0xBB67AE85) & _M
    return torch.stack((c0, c1, c2, c3), 1).reshape(-1)[:n] >= round(p * 2 ** 32)


def _plain_dropout(s, residual):
    x, p = s["x"], s["p"]
    keep = _keep(x.numel(), p, s["seed"], s["offset"], x.device).view(x.shape)
    y = torch.where(keep, x.float() * (1 / (1 - p)), torch.zeros((), device=x.device))
    if residual is not None:
        y = residual.float() + y
    return y.to(x.dtype)


def _plain_xent(s, step):
    x, w, labels = s["x"].float(), s["w"].float(), s["labels"]
    valid = labels != IGNORE
    safe = torch.where(valid, labels, torch.zeros_like(labels))
    count = valid.sum().clamp(min=1)
    logits = x @ w.t()
    top = logits.max(1).values
    e = torch.exp(logits - top[:, None])
    z = e.sum(1)
    lse = top + torch.log(z)
    at = logits.gather(1, safe[:, None])[:, 0]
    loss = torch.where(valid, lse - at, torch.zeros_like(lse)).sum() / count
    if not step:
        return loss, lse
    del logits
    scale = torch.where(valid, s["grad_loss"] / count, torch.zeros_like(lse))
    e *= (scale / z)[:, None]
    e[torch.arange(len(labels), device=e.device), safe] -= scale
    return loss, lse, (e @ w).to(s["x"].dtype), (e.t() @ x).to(s["w"].dtype)


def _own(s):
    import broadcast_elementwise_shape_gb300 as zr

    op, way = s["case"]["op"], s["case"]["way"]
    if op == "layer_norm" and way == "fwd":
        return zr.zr_layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS)
    if op == "layer_norm":
        return zr.zr_layer_norm_bwd(s["grad"], s["x"], s["gamma"], s["mean"], s["rstd"])
    if op == "dropout" and way == "fwd":
        return zr.zr_dropout_fwd(s["x"], s["p"], s["seed"], s["offset"], residual=s["residual"])
    if op == "dropout":
        return zr.zr_dropout_bwd(s["x"], s["p"], s["seed"], s["offset"])
    loss, lse = zr.zr_linear_xent_fwd(s["x"], s["w"], s["labels"], ignore_index=IGNORE)
    if way == "fwd":
        return loss, lse
    gx, gw = zr.zr_linear_xent_bwd(s["grad_loss"], s["x"], s["w"], s["labels"], lse, ignore_index=IGNORE)
    return loss, lse, gx, gw


def run(state):
    if own:
        return _own(state)
    op, way = state["case"]["op"], state["case"]["way"]
    if op == "layer_norm":
        return _plain_layer_norm_fwd(state) if way == "fwd" else _plain_layer_norm_bwd(state)
    if op == "dropout":
        return _plain_dropout(state, state.get("residual"))
    return _plain_xent(state, way == "step")


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    rows, dim, fwd = case["rows"], case["dim"], case["way"] == "fwd"
    n = rows * dim
    if case["op"] == "layer_norm":
        if fwd:
            return {"bytes": es * (2 * n + 2 * dim) + 8 * rows, "flops": 8 * n}
        return {"bytes": es * (3 * n + 3 * dim) + 8 * rows, "flops": 15 * n}
    if case["op"] == "dropout":
        return {"bytes": es * n * (3 if fwd else 2), "flops": 2 * n}
    # The step's three products are those of the logits and of the two gradients.
    vocab = case["vocab"]
    inputs = es * (n + vocab * dim) + 8 * rows
    if fwd:
        return {"bytes": inputs + 4 * rows, "flops": 2 * n * vocab}
    return {"bytes": inputs + 4 * rows + es * (n + vocab * dim), "flops": 6 * n * vocab}


def _exact_layer_norm(s, way):
    x = s["x"].double()
    dim = x.shape[1]
    if way == "fwd":
        mean = x.mean(1, keepdim=True)
        rstd = (x.var(1, unbiased=False, keepdim=True) + EPS).rsqrt()
        y = torch.addcmul(s["beta"].double(), (x - mean) * rstd, s["gamma"].double())
        return y, mean[:, 0], rstd[:, 0]
    mean, rstd, g = s["mean"].double(), s["rstd"].double(), s["grad"].double()
    xhat = x.sub(mean[:, None]).mul_(rstd[:, None])
    # The projection onto what the norm leaves: q less its parts along 1 and along xhat.
    q = g * s["gamma"].double()
    along = torch.einsum("rd,rd->r", q, xhat) / dim
    gx = (q - q.mean(1, keepdim=True) - along[:, None] * xhat) * rstd[:, None]
    return gx, torch.einsum("rd,rd->d", g, xhat), g.sum(0)


def _philox(counters, seed):
    """Philox4x32-10 of 64-bit counters, [n, 4] words, in numpy's unsigned integers."""
    c = [counters & np.uint64(_M), counters >> np.uint64(32), np.zeros_like(counters), np.zeros_like(counters)]
    key = [seed & _M, seed >> 32 & _M]
    for r in range(10):
        if r:
            key = [(key[0] + 0x9E3779B9) & _M, (key[1] + 0xBB67AE85) & _M]
        p = np.uint64(0xD2511F53) * c[0]
        q = np.uint64(0xCD9E8D57) * c[2]
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(key[0]), q & np.uint64(_M),
             (p >> np.uint64(32)) ^ c[3] ^ np.uint64(key[1]), p & np.uint64(_M)]
    return np.stack(c, 1)


def _exact_dropout(s):
    n, p = s["x"].numel(), s["p"]
    at = np.uint64(s["offset"]) + np.arange((n + 3) // 4, dtype=np.uint64)
    words = _philox(at, s["seed"]).reshape(-1)[:n]
    drop = torch.from_numpy(words < round(p * 2 ** 32)).cuda().view(s["x"].shape)
    y = (s["x"].double() / (1 - p)).masked_fill_(drop, 0)
    return y if "residual" not in s else y + s["residual"].double()


def _exact_xent(s, way):
    labels = s["labels"]
    w = s["w"].double()
    rows = int((labels != IGNORE).sum())
    lse, loss, gx = [], 0.0, []
    gw = torch.zeros_like(w) if way == "step" else None
    for at in range(0, len(labels), 2048):  # some rows at a time, so that 64 bits fit
        x, y = s["x"][at:at + 2048].double(), labels[at:at + 2048]
        l = x @ w.t()
        z = torch.logsumexp(l, 1)
        used = torch.nonzero(y != IGNORE)[:, 0]
        lse.append(z)
        loss += float((z[used] - l[used, y[used]]).sum())
        if way == "step":
            p = torch.exp(l - z[:, None])
            p[used, y[used]] -= 1
            p[y == IGNORE] = 0
            p *= float(s["grad_loss"]) / max(rows, 1)
            gx.append(p @ w)
            gw += p.t() @ x
    loss = torch.tensor(loss / max(rows, 1), dtype=torch.float64)
    if way == "fwd":
        return loss, torch.cat(lse)
    return loss, torch.cat(lse), torch.cat(gx), gw


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer_norm":
        return _exact_layer_norm(s, case["way"])
    if case["op"] == "dropout":
        return _exact_dropout(s)
    return _exact_xent(s, case["way"])
