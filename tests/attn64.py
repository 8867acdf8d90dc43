"""Causal attention and its gradients in 64 bits, and how far a result may be
off, element by element (shared by the attention's GPU tests).

With u the half step of what is rounded to as an operand (bf16 2^-8; binary32
tensors: 0), e = 2^-24 and A_ij = |scale| sum |q k|:
* a score is off by at most ds = (D + 4) e A, and a weight exp(s - lse), whose
  lse moves as far at most and is kept to e |lse| (and times log2(e) once more), by the factor 1 + w, w = 2 max_j ds + 4 e (|lse| + A) + 8 e;
* out: (u + w + (T + 4) e) sum p |v|, and the rounding of the result;
* grad_v: the same of sum p |grad_out|;
* ds = p (dp - delta): p's factor w, dp's (D + 4) e sum |grad_out v|, delta's: out's own error and (D + 4) e,
  of sum |grad_out| |out|, and where low is not given out's rounding; ds is rounded to u as an operand.
* Weights below 2^-126 may be taken as 0 (the exponential flushes them): a weight is off by F = 2^-126 besides, which adds
  F sum |grad_out| to grad_v, and to ds F |scale| (|dp| + |delta|) + F (ds itself may flush).
The tensor core truncates where it adds, at most 2 e per 16 terms, which (D + 4) e and (T + 4) e cover.
"""
import torch

E, F = 2.0 ** -24, 2.0 ** -126
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def sequences(t, offsets):
    if offsets is None:
        return [(0, t)]
    o = offsets.tolist()
    return [(max(0, min(a, t)), max(0, min(b, t))) for a, b in zip(o[:-1], o[1:]) if b > a]


def heads(q, k, v, scale, go, u, rows_low):
    """One sequence, one batch entry, [T, H, D]: values and bounds, as dicts."""
    t, h, d = q.shape
    g = h // k.shape[1]
    q, k, v = (x.double().transpose(0, 1) for x in (q, k, v))
    k, v = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
    mask = torch.ones(t, t, dtype=torch.bool, device=q.device).triu(1)
    s = (q @ k.transpose(1, 2) * scale).masked_fill(mask, -torch.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    out = p @ v
    a = (q.abs() @ k.abs().transpose(1, 2) * abs(scale)).masked_fill(mask, 0)
    w = (2 * (d + 4) * E * a).amax(-1) + 4 * E * (lse.abs() + a.amax(-1)) + 8 * E
    w = w.expm1() if bool((w > 0.1).any()) else 1.1 * w
    val = {"out": out, "lse": lse}
    raw = (u + w + (t + 4) * E)[..., None] * (p @ v.abs())  # before out is rounded
    off = {"out": raw, "lse": w}
    if go is not None:
        go = go.double().transpose(0, 1)
        dp, size = go @ v.transpose(1, 2), go.abs() @ v.abs().transpose(1, 2)
        delta = (go * out).sum(-1, keepdim=True)
        ds = p * (dp - delta) * scale
        o_size = (go.abs() * out.abs()).sum(-1, keepdim=True)
        e_delta = (go.abs() * raw).sum(-1, keepdim=True) + (d + 4) * E * o_size + rows_low * o_size
        e_ds = abs(scale) * p * (w[..., None] * (dp.abs() + delta.abs()) + (1 + w[..., None]) * ((d + 4) * E * size + e_delta) + 4 * E * (dp.abs() + delta.abs()))
        e_ds = e_ds + F * (abs(scale) * (dp.abs() + delta.abs()) + 1).masked_fill(mask, 0)
        e_ds = e_ds + (u + 2 * E) * (ds.abs() + e_ds)
        fold = lambda x: x.unflatten(0, (-1, g)).sum(1)  # noqa: E731
        val |= {"gq": ds @ k, "gk": fold(ds.transpose(1, 2) @ q), "gv": fold(p.transpose(1, 2) @ go)}
        n = (t * g + 4) * E
        off |= {"gq": e_ds @ k.abs() + n * (ds.abs() @ k.abs()), "gk": fold(e_ds.transpose(1, 2) @ q.abs() + n * (ds.abs().transpose(1, 2) @ q.abs())),
                "gv": fold(((u + n + w[..., None]) * p + F * ~mask).transpose(1, 2) @ go.abs())}
    turn = lambda x: x.transpose(0, 1)  # noqa: E731
    return {n: turn(x) for n, x in val.items()}, {n: turn(x) for n, x in off.items()}


def reference(q, k, v, scale, offsets=None, go=None, exact=False, low=True):
    """{name: (value, bound)} of [B, T, H, D] or [T, H, D]; rows in no sequence are NaN with bound NaN.
    exact: the operands stay binary32."""
    batched = q.dim() == 4
    if not batched:
        q, k, v = q[None], k[None], v[None]
        go = None if go is None else go[None]
    u = 0.0 if exact else HALF[q.dtype]
    rows_low = E if q.dtype == torch.float32 else (2.0 ** -16 if low else 2.0 ** -8)
    shapes = {"out": q.shape, "lse": q.shape[:-1]}
    if go is not None:
        shapes |= {"gq": q.shape, "gk": k.shape, "gv": v.shape}
    got = {n: [torch.full(s, torch.nan, dtype=torch.float64, device=q.device) for _ in range(2)] for n, s in shapes.items()}
    for b in range(q.shape[0]):
        for lo, hi in sequences(q.shape[1], offsets):
            val, off = heads(q[b, lo:hi], k[b, lo:hi], v[b, lo:hi], scale, None if go is None else go[b, lo:hi], u, rows_low)
            for n in got:
                got[n][0][b, lo:hi], got[n][1][b, lo:hi] = val[n], off[n]
    half = HALF[q.dtype]
    for n, (val, off) in got.items():
        off += (E if n == "lse" else half) * (val.abs() + off) + 1e-38
    return {n: tuple(x if batched else x[0] for x in pair) for n, pair in got.items()}


def check(got, want):
    val, off = want
    inside = ~torch.isnan(val)
    err = (got.double() - val).abs()
    bad = inside & ~(err <= off)
    assert not bool(bad.any()), f"{int(bad.sum())} of {int(inside.sum())} off, worst {float((err / off)[bad].max()) if bool(bad.any()) else 0}"


def run(zr, q, k, v, scale=None, offsets=None, go=None, low=True, exact=False, **kw):
    """Runs the forward, and the backward where go is given, and checks them."""
    want = reference(q, k, v, q.shape[-1] ** -0.5 if scale is None else scale, offsets, go, exact, low)
    out, lse, lo = zr.zr_attention_fwd(q, k, v, scale, offsets, keep_low=low and go is not None, **kw)
    check(out, want["out"])
    check(lse, want["lse"])
    if go is None:
        return out, lse
    grads = zr.zr_attention_bwd(go, q, k, v, out, lse, lo, scale, offsets)
    for n, g in zip(("gq", "gk", "gv"), grads):
        check(g, want[n])
    return out, lse, *grads
