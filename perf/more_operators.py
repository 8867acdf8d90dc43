"""Causal attention, rotary positions and the AdamW step: the cases they are
measured on.

A case names an operator (``op``), an element type (``dtype``) and its sizes.
``run`` with ``own`` false computes the plain form in elementary torch
operations (32-bit arithmetic, rounded once at the end; angles in 64 bits);
with ``own`` true it calls this package.  ``exact`` is the definition in 64
bits.

* ``attention``: one projection's rows [tokens, heads + 2 * kv_heads, dim],
  whose heads are the queries, then the keys, then the values; query head h
  reads key and value head h * kv_heads // heads.  ``lengths`` are packed one
  behind the other, and a token sees those before it in its own sequence and
  itself.  With ``batch`` the rows are [batch, length, ...] instead.
  way ``fwd`` gives (out, per-row log of the sum of exponentials), ``step``
  also the gradient of the projection's rows.
* ``rotary``: x [tokens, heads, dim], the first ``part`` elements of a head in
  pairs (j, j + part / 2), or (2j, 2j + 1) where ``interleaved``, turned by the
  token's position times base^(-2j / part).  With ``factor`` over 1 the
  frequencies are divided by it, all of them, or with ``original`` those that
  turn less than once over so many positions, none that turn over 32 times,
  and between the two a blend (B. Peng, J. Quesnelle, H. Fan and E. Shippole,
  "YaRN: efficient context window extension of large language models", 2023).
  way ``fwd`` gives y, ``bwd`` the gradient of x.
* ``adamw``: the tensors of a small decoder (``layers``, ``width``, ``vocab``),
  or ``count`` tensors of ragged sizes.  Parameters are 32-bit with a bf16
  copy, gradients of ``dtype``, states of ``bits``.  States of 8 bits are
  blocks of 256 elements with a power of two each: m a sign, 4 bits of exponent
  and 3 of mantissa, v 5 bits of exponent and 3 of mantissa, the block's
  largest in the last binade but one; they are rounded up with the probability
  of what is cut off, drawn by Philox4x32-10 (Salmon, Moraes, Dror and Shaw, SC
  2011) at counter (i div 4, tensor, step), word i mod 4: its low half for m,
  its high half for v.  Gives (parameters, copies, m, v), of all tensors one
  behind the other.
"""
import math

import torch

own = False

_M = 0xFFFFFFFF
BLOCK = 256
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.999, 1e-8, 0.1


def listed():
    return [
        # A handful of short prompts packed together, one of them a single token: latency counts.
        dict(name="attn_fwd_small", op="attention", way="fwd", dtype="bf16", lengths="5,1,17,64", heads=6, kv_heads=6, dim=64, batch=0),
        # A small character-level model in 32 bits: 16 sequences of 256 less one token.
        dict(name="attn_step_chars", op="attention", way="step", dtype="f32", lengths="255", heads=6, kv_heads=6, dim=64, batch=16),
        # The attention-score workload, [8, 12, 1024, 1024], as a training step.
        dict(name="attn_step_batch", op="attention", way="step", dtype="bf16", lengths="1024", heads=12, kv_heads=12, dim=64, batch=8),
        # Documents of very different lengths packed into one long row, four query heads to a key head.
        dict(name="attn_step_packed", op="attention", way="step", dtype="bf16", lengths="8192,3,2047,130,4001,777,1,1233", heads=32, kv_heads=8, dim=128, batch=0),
        # One new token of a small model.
        dict(name="rot_fwd_token", op="rotary", way="fwd", dtype="bf16", tokens=1, heads=24, dim=64, part=64, interleaved=False, factor=1.0, original=0, first=1000),
        # The queries and keys of a training batch, [8, 1024] tokens, in 32 bits, neighbours paired.
        dict(name="rot_fwd_batch", op="rotary", way="fwd", dtype="f32", tokens=8192, heads=24, dim=64, part=64, interleaved=True, factor=1.0, original=0, first=0),
        # A part of an odd head, an odd number of tokens, the gradient, positions stretched to four times the context.
        dict(name="rot_bwd_part", op="rotary", way="bwd", dtype="bf16", tokens=4093, heads=20, dim=81, part=32, interleaved=True, factor=4.0, original=0, first=3000),
        # A long context, far positions, frequencies blended.
        dict(name="rot_fwd_long", op="rotary", way="fwd", dtype="bf16", tokens=65536, heads=40, dim=128, part=128, interleaved=False, factor=16.0, original=8192, first=900000),
        # The block of the training example, width 192: a handful of small tensors.
        dict(name="adamw_small", op="adamw", dtype="f32", bits=32, layers=1, width=192, vocab=301, count=0),
        # Many ragged tensors, gradients in 16 bits, states in 8.
        dict(name="adamw_ragged8", op="adamw", dtype="bf16", bits=8, layers=0, width=0, vocab=0, count=301),
        # A decoder of 12 layers of width 768 and a vocabulary of 50001.
        dict(name="adamw_model", op="adamw", dtype="f32", bits=32, layers=12, width=768, vocab=50001, count=0),
        dict(name="adamw_model8", op="adamw", dtype="bf16", bits=8, layers=12, width=768, vocab=50001, count=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "rotary", "adamw"])
    if op == "attention":
        dtype = rng.choice(["f32", "bf16", "bf16"])
        dim = rng.choice([64, 128, 8 * rng.randrange(2, 17), rng.randrange(16, 129)])
        kv = rng.choice([1, 2, 3, 4, 6, 8])
        heads = kv * rng.choice([1, 1, 2, 3, 4])
        # The largest listed case's products, or an eighth of them in 32 bits.
        left = 8192 * 8192 * 32 * 128 // (8 if dtype == "f32" else 1) // (heads * dim)
        if rng.random() < 0.3:
            length = _log(rng, 1, min(4096, math.isqrt(left)))
            batch = _log(rng, 1, max(1, min(64, left // (length * length), (1 << 19) // (length * heads))))
            return dict(op=op, way=rng.choice(["fwd", "step"]), dtype=dtype, lengths=str(length), heads=heads, kv_heads=kv, dim=dim, batch=batch)
        lengths = []
        for _ in range(rng.randrange(1, 13)):
            n = _log(rng, 1, 8192)
            if n * n <= left:
                left -= n * n
                lengths.append(n)
        return dict(op=op, way=rng.choice(["fwd", "step"]), dtype=dtype, lengths=",".join(map(str, lengths or [1])), heads=heads, kv_heads=kv, dim=dim, batch=0)
    if op == "rotary":
        dim = rng.choice([64, 128, 8 * rng.randrange(2, 33), rng.randrange(16, 257)])
        part = dim // 2 * 2 if rng.random() < 0.6 else 2 * rng.randrange(1, dim // 2 + 1)
        heads = rng.randrange(1, 65)
        factor = rng.choice([1.0, 1.0, 4.0, 10.5])
        return dict(op=op, way=rng.choice(["fwd", "bwd"]), dtype=rng.choice(["f32", "bf16"]), tokens=_log(rng, 1, 65536 * 40 * 64 // (heads * dim)), heads=heads, dim=dim,
                    part=part, interleaved=rng.random() < 0.5, factor=factor, original=rng.choice([0, 4096]) if factor > 1 else 0, first=rng.choice([0, _log(rng, 1, 1 << 20)]))
    case = dict(op=op, dtype=rng.choice(["f32", "bf16"]), bits=rng.choice([8, 32]), layers=0, width=0, vocab=0, count=0)
    if rng.random() < 0.4:
        return {**case, "count": _log(rng, 1, 700)}
    return {**case, "layers": rng.randrange(1, 13), "width": _log(rng, 64, 768), "vocab": _log(rng, 100, 50000)}


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _sizes(case):
    """The element counts of the tensors of an adamw case."""
    if case["count"]:
        # Biases of a few elements to matrices of some hundred thousands, hardly one of them round.
        return [1 + (7919 * i * i + 104729 * i) % (37 if i % 3 == 0 else 1013 if i % 3 == 1 else 400009) for i in range(case["count"])]
    c, v = case["width"], case["vocab"]
    layer = [c, c, 3 * c * c, 3 * c, c * c, c, c, c, 4 * c * c, 4 * c, 4 * c * c, c]
    return [v * c, 1024 * c] + layer * case["layers"] + [c, c]


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    state = {"case": case}
    if case["op"] == "attention":
        h, kv, d, b = case["heads"], case["kv_heads"], case["dim"], case["batch"]
        lead = (b, _lengths(case)[0]) if b else (sum(_lengths(case)),)
        # Heads of different temperatures, keys with a mean of their own, values and gradients of unit size.
        x = normal(*lead, h + 2 * kv, d)
        x[..., :h, :] *= uniform(0.5, 3, h, 1)
        x[..., h:h + kv, :] += 0.5 * normal(kv, d)
        state.update(qkv=x.to(dt), scale=d ** -0.5)
        if not b:
            ends = torch.tensor(_lengths(case)).cumsum(0)
            state["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(torch.int32).cuda()
        if case["way"] == "step":
            state["grad"] = normal(*lead, h, d).to(dt)
    elif case["op"] == "rotary":
        n = case["tokens"]
        # Positions that run on, as a packed batch or a continued prompt has them.
        state.update(x=normal(n, case["heads"], case["dim"]).to(dt),
                     positions=case["first"] + torch.arange(n, device="cuda") % 70000 + torch.randint(0, 100, (1,), generator=g, device="cuda"))
        state["freqs"] = _freqs(case).cuda()
        state["magnitude"] = 0.1 * math.log(case["factor"]) + 1 if case["original"] else 1.0
        state["plan"] = dict(base=10000.0, interleaved=case["interleaved"], factor=case["factor"], original=case["original"] or None, magnitude=state["magnitude"])
    else:
        sizes = _sizes(case)
        n = sum(sizes)

        def split(flat, by=1):
            return list(flat.split([-(-s // by) for s in sizes]))

        p = 0.02 * normal(n)
        grad = normal(n) * torch.exp(2 * normal(n) - 6)
        v = (grad * grad).mul_(uniform(0.2, 2, n))
        m = 0.3 * torch.sqrt(v) * normal(n)
        state.update(p=p, copy=torch.empty(n, dtype=torch.bfloat16, device="cuda"), grad=grad.to(dt), step=100 + seed % 1000, seed=0x9E3779B97F4A7C15 ^ seed)
        if case["bits"] == 8:
            half = torch.full((), 1 << 19, dtype=torch.int32, device="cuda")
            made = [[_encode(x, half, signed) for x in split(t)] for t, signed in ((m, True), (v, False))]
            state.update(m=torch.cat([c for c, _ in made[0]]), v=torch.cat([c for c, _ in made[1]]),
                         m_scale=torch.cat([s for _, s in made[0]]), v_scale=torch.cat([s for _, s in made[1]]))
            state["scales"] = (split(state["m_scale"], BLOCK), split(state["v_scale"], BLOCK))
        else:
            state.update(m=m, v=v)
        state["tensors"] = {k: split(state[k]) for k in ("p", "grad", "m", "v", "copy")}
    return state


def _freqs(case):
    """The turning rates of the pairs, in 64 bits."""
    j = torch.arange(case["part"] // 2, dtype=torch.float64)
    f = 10000.0 ** (-2 * j / case["part"])
    if not case["original"]:
        return f / case["factor"]
    w = ((case["original"] * f / (2 * math.pi) - 1) / (32 - 1)).clamp(0, 1)
    return f * (w + (1 - w) / case["factor"])


def _plain_sequence(q, k, v, scale, go):
    """Attention of sequences of one length: q, go [..., T, H, D], k and v [..., T, K, D], in 32 bits."""
    t, h, d = q.shape[-3:]
    kv = k.shape[-2]
    q = q.transpose(-3, -2).unflatten(-3, (kv, h // kv))  # [..., K, H / K, T, D]
    k, v = k.transpose(-3, -2).unsqueeze(-3), v.transpose(-3, -2).unsqueeze(-3)
    at = torch.arange(t, device=q.device)
    s = (q @ k.transpose(-2, -1)).mul_(scale)
    s.masked_fill_(at[None, :] > at[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp_(s.sub_(top))
    z = p.sum(-1, keepdim=True)
    p /= z
    out = p @ v
    lse = (top + torch.log(z)).squeeze(-1).flatten(-3, -2).transpose(-2, -1)
    back = lambda x: x.flatten(-4, -3).transpose(-3, -2)  # noqa: E731
    if go is None:
        return back(out), lse
    go = go.transpose(-3, -2).unflatten(-3, (kv, h // kv))
    gv = (p.transpose(-2, -1) @ go).sum(-3)
    dp = go @ v.transpose(-2, -1)
    dp -= (dp * p).sum(-1, keepdim=True)
    ds = p.mul_(dp).mul_(scale)
    gq = ds @ k
    gk = (ds.transpose(-2, -1) @ q).sum(-3)
    return back(out), lse, back(gq), gk.transpose(-3, -2), gv.transpose(-3, -2)


def _plain_attention(s):
    case = s["case"]
    h, kv = case["heads"], case["kv_heads"]
    parts = [s["qkv"]] if case["batch"] else list(s["qkv"].split(_lengths(case)))
    gos = [None] * len(parts) if case["way"] == "fwd" else [s["grad"]] if case["batch"] else list(s["grad"].split(_lengths(case)))
    got = [_plain_sequence(*x.float().split([h, kv, kv], -2), s["scale"], None if go is None else go.float()) for x, go in zip(parts, gos)]
    out, lse, *grads = (torch.cat(x) for x in zip(*got))
    if not grads:
        return out.to(s["qkv"].dtype), lse
    return out.to(s["qkv"].dtype), lse, torch.cat(grads, -2).to(s["qkv"].dtype)


def _plain_rotary(s):
    case, x = s["case"], s["x"]
    part = case["part"]
    a = s["positions"].double()[:, None] * s["freqs"]
    c, n = ((s["magnitude"] * f(a)).float()[:, None] for f in (torch.cos, torch.sin))
    if case["way"] == "bwd":
        n = -n
    xf = x.float()
    y = xf.clone()
    i, j = (slice(0, part, 2), slice(1, part, 2)) if case["interleaved"] else (slice(0, part // 2), slice(part // 2, part))
    y[..., i] = xf[..., i] * c - xf[..., j] * n
    y[..., j] = xf[..., j] * c + xf[..., i] * n
    return y.to(x.dtype)


def _words(n, tensor, step, seed, device):
    """The words of Philox4x32-10 of n elements, in 64-bit integers, whose products wrap as unsigned ones do."""
    c0 = torch.arange((n + 3) // 4, device=device, dtype=torch.int64)
    c1, c2, c3 = (torch.full_like(c0, x) for x in (tensor, step & _M, step >> 32))
    k0, k1 = seed & _M, (seed >> 32) & _M
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & _M) ^ c1 ^ k0, b & _M, ((a >> 32) & _M) ^ c3 ^ k1, a & _M
        k0, k1 = (k0 + 0x9E3779B9) & _M, (k1 + 0xBB67AE85) & _M
    return torch.stack((c0, c1, c2, c3), 1).reshape(-1)[:n]


def _blocks(x):
    return torch.nn.functional.pad(x, (0, -len(x) % BLOCK)).view(-1, BLOCK)


def _encode(x, cut, signed):
    """x's codes and its blocks' powers of two; ``cut`` in [0, 2^20) is added below the last place that is kept."""
    b = _blocks(x)
    e = ((b.abs().amax(1).view(torch.int32) >> 23) - 127).clamp(min=-90)
    scale, inverse = (((127 + k * e) << 23).view(torch.float32) for k in (1, -1))
    y = (b.abs() * inverse[:, None] * (2.0 ** -113 if signed else 2.0 ** -97)).view(-1)[:len(x)]
    code = (y.view(torch.int32) + cut) >> 20
    if signed:
        code = code | (torch.signbit(x).int() << 7)
    return code.to(torch.uint8), scale


def _decode(code, scale, signed):
    c = code.int()
    y = (((c & 127) if signed else c) << 20).view(torch.float32) * (2.0 ** 113 if signed else 2.0 ** 97)
    if signed:
        y = torch.where(c > 127, -y, y)
    return (_blocks(y) * scale[:, None]).view(-1)[:len(code)]


def _plain_adamw(s):
    bits, t, seed = s["case"]["bits"], s["step"], s["seed"]
    parts = s["tensors"]
    if bits == 8:
        m, v = (torch.cat([_decode(c, x, k == "m") for c, x in zip(parts[k], scales)]) for k, scales in zip("mv", s["scales"]))
    else:
        m, v = s["m"], s["v"]
    g = s["grad"].float()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    root = torch.sqrt(v) * (1 - BETA2 ** t) ** -0.5 + EPS
    s["p"] -= (LR * DECAY) * s["p"] + LR / (1 - BETA1 ** t) * (m / root)
    s["copy"].copy_(s["p"])
    if bits == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return s["p"], s["copy"], s["m"], s["v"]
    sizes = [len(c) for c in parts["m"]]
    words = [_words(n, i, t, seed, g.device).int() for i, n in enumerate(sizes)]
    out = []
    for k, x, cuts, scales in (("m", m, [(w & 0xFFFF) << 4 | 8 for w in words], s["scales"][0]),
                               ("v", v, [(w >> 16 & 0xFFFF) << 4 | 8 for w in words], s["scales"][1])):
        made = [_encode(y, cut, k == "m") for y, cut in zip(x.split(sizes), cuts)]
        s[k].copy_(torch.cat([c for c, _ in made]))
        s[k + "_scale"].copy_(torch.cat([x for _, x in made]))
        out.append(torch.cat([_decode(c, x, k == "m") for c, x in zip(parts[k], scales)]).bfloat16())  # four bits and a power of two: exact
    return s["p"], s["copy"], *out


def _own(s):
    import broadcast_elementwise_shape_gb300 as zr

    case = s["case"]
    if case["op"] == "attention":
        h, kv = case["heads"], case["kv_heads"]
        q, k, v = s["qkv"].split([h, kv, kv], -2)
        offsets = s.get("offsets")
        if case["way"] == "fwd":
            out, lse, _ = zr.zr_attention_fwd(q, k, v, s["scale"], offsets)
            return out, lse
        out, lse, low = zr.zr_attention_fwd(q, k, v, s["scale"], offsets, keep_low=True)
        grads = torch.empty_like(s["qkv"])
        zr.zr_attention_bwd(s["grad"], q, k, v, out, lse, low, s["scale"], offsets, grads=grads.split([h, kv, kv], -2))
        return out, lse, grads
    if case["op"] == "rotary":
        if type(s["plan"]) is dict:  # made once, by the first call
            s["plan"] = zr.zr_rotary_plan(case["part"], **s["plan"])
        turn = zr.zr_rotary_fwd if case["way"] == "fwd" else zr.zr_rotary_bwd
        return turn(s["x"], s["plan"], s["positions"])
    t = s["tensors"]
    scales = s.get("scales", (None, None))
    zr.zr_adamw_step(t["p"], t["grad"], t["m"], t["v"], s["step"], LR, (BETA1, BETA2), EPS, DECAY, copies=t["copy"], m_scales=scales[0], v_scales=scales[1], seed=s["seed"])
    if case["bits"] == 32:
        return s["p"], s["copy"], s["m"], s["v"]
    if "values" not in s:  # room for the states' values, made by the first call
        s["values"] = [torch.empty_like(s["copy"]) for _ in range(2)]
        s["views"] = [list(x.split([len(y) for y in t["p"]])) for x in s["values"]]
    zr.zr_adamw_state(t["m"], t["v"], *scales, out=s["views"])
    return s["p"], s["copy"], *s["values"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_attention(state) if op == "attention" else _plain_rotary(state) if op == "rotary" else _plain_adamw(state)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attention":
        h, kv, d = case["heads"], case["kv_heads"], case["dim"]
        n = sum(_lengths(case)) * max(1, case["batch"])
        pairs = sum(t * (t + 1) // 2 for t in _lengths(case)) * max(1, case["batch"])  # of a query and a key that it sees
        moved = es * n * (2 * h + 2 * kv) * d + 4 * n * h
        if case["way"] == "fwd":
            return {"bytes": moved, "flops": 4 * pairs * h * d}
        # Two products forward; five backward, one of them the logits once more.
        return {"bytes": moved + es * n * (2 * h + 2 * kv) * d, "flops": 14 * pairs * h * d}
    if case["op"] == "rotary":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * es * n * case["dim"] + 8 * case["tokens"], "flops": 3 * n * case["part"]}
    n = sum(_sizes(case))
    # Parameters read and written, their copies, gradients, states read and written; those of 8 bits also come as values.
    return {"bytes": n * (10 + es + (16 if case["bits"] == 32 else 4 + 4)), "flops": 15 * n}


def _exact_heads(q, k, v, scale, go):
    """One sequence and one key head: q, go [H, T, D], k and v [T, D], in 64 bits."""
    t = k.shape[0]
    s = torch.einsum("htd,sd->hts", q, k) * scale
    s += torch.full((t, t), -math.inf, dtype=s.dtype, device=s.device).triu(1)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    out = torch.einsum("hts,sd->htd", p, v)
    if go is None:
        return out, lse
    gv = torch.einsum("hts,htd->sd", p, go)
    # The softmax's gradient: each logit's weight times how far its own product is from the row's.
    ds = p * (torch.einsum("htd,sd->hts", go, v) - (go * out).sum(-1, keepdim=True)) * scale
    return out, lse, torch.einsum("hts,sd->htd", ds, k), torch.einsum("hts,htd->sd", ds, q), gv


def _exact_attention(s):
    case = s["case"]
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    lengths = _lengths(case) * max(1, case["batch"])
    x = s["qkv"].view(-1, h + 2 * kv, d)
    n = x.shape[0]
    out = torch.empty(n, h, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(n, h, dtype=torch.float64, device="cuda")
    grad = torch.empty(n, h + 2 * kv, d, dtype=torch.float64, device="cuda")
    at = 0
    for t in lengths:
        rows = slice(at, at + t)
        at += t
        for k in range(kv):
            mine = slice(k * h // kv, (k + 1) * h // kv)
            go = s["grad"].view(n, h, d)[rows, mine].double().transpose(0, 1) if "grad" in s else None
            got = _exact_heads(x[rows, mine].double().transpose(0, 1), x[rows, h + k].double(), x[rows, h + kv + k].double(), s["scale"], go)
            out[rows, mine], lse[rows, mine] = got[0].transpose(0, 1), got[1].t()
            if go is not None:
                grad[rows, mine], grad[rows, h + k], grad[rows, h + kv + k] = got[2].transpose(0, 1), got[3], got[4]
    lead = s["qkv"].shape[:-2]
    out, lse, grad = out.view(*lead, h, d), lse.view(*lead, h), grad.view(*lead, h + 2 * kv, d)
    return (out, lse, grad) if "grad" in s else (out, lse)


def _exact_rotary(s):
    case = s["case"]
    part = case["part"]
    x = s["x"].double()
    turn = torch.polar(torch.full((), s["magnitude"], dtype=torch.float64, device="cuda"), s["positions"].double()[:, None] * s["freqs"])[:, None]
    if case["way"] == "bwd":
        turn = turn.conj()
    if case["interleaved"]:
        z = torch.view_as_complex(x[..., :part].unflatten(-1, (-1, 2)).contiguous()) * turn
        return torch.cat([torch.view_as_real(z).flatten(-2), x[..., part:]], -1)
    z = torch.complex(x[..., :part // 2], x[..., part // 2:part]) * turn
    return torch.cat([z.real, z.imag, x[..., part:]], -1)


def _exact_round(x, cut, places):
    """x of one tensor, in blocks whose largest is in the last binade but one of 2^(places - 3) of them, rounded by ``cut``."""
    b = _blocks(x.abs())
    top = torch.frexp(b.amax(1)).exponent - 1  # floor of the base-2 logarithm
    top = torch.where(b.amax(1) > 0, top, -90).clamp(min=-90)
    least = top - ((1 << (places - 3)) - 3)  # the first binade with its leading bit in place
    e = torch.maximum(torch.frexp(b).exponent - 1, least[:, None])
    step = torch.ldexp(torch.ones((), dtype=torch.float64, device=x.device), (e - 3).double()).view(-1)[:len(x)]
    return torch.copysign(torch.floor(x.abs() / step + cut.double() / 2 ** 20) * step, x)


def _exact_adamw(s):
    case, t = s["case"], s["step"]
    parts, p, g = s["tensors"], s["p"].double(), s["grad"].double()
    m, v = s["m"], s["v"]
    if case["bits"] == 8:
        m, v = (torch.cat([_decode(c, x, k == "m") for c, x in zip(parts[k], scales)]) for k, scales in zip("mv", s["scales"]))
    m, v = torch.lerp(g, m.double(), BETA1), torch.lerp(g * g, v.double(), BETA2)
    update = m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    p = p - LR * (update + DECAY * p)
    if case["bits"] == 8:
        sizes = [len(c) for c in parts["m"]]
        words = [_words(n, i, t, s["seed"], g.device) for i, n in enumerate(sizes)]
        m = torch.cat([_exact_round(x, w % 65536 * 16 + 8, 7) for x, w in zip(m.split(sizes), words)])
        v = torch.cat([_exact_round(x, w // 65536 * 16 + 8, 8) for x, w in zip(v.split(sizes), words)])
    return p, p, m, v


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attention(s) if case["op"] == "attention" else _exact_rotary(s) if case["op"] == "rotary" else _exact_adamw(s)
