"""Plain 64-bit references of latent attention, draft verification and rotary
positions with several axes (torch, on the tensors' device), and the bounds
that results in fp16 are held to."""
from __future__ import annotations

import math

import numpy as np
import torch

F64 = torch.float64
H = 2.0 ** -11   # half a step of fp16, relative


def quantized(x, bits, G):
    """Vectors x [m, r] (fp16) as the cache restores them: zero + code * scale
    of groups of G channels (fp32 arithmetic, fp16 scale and zero), in 64 bits."""
    m, r = x.shape
    y = x.float().view(m, r // G, G)
    lo, hi = y.amin(2, keepdim=True), y.amax(2, keepdim=True)
    s = ((hi - lo) / torch.full_like(hi, 2 ** bits - 1)).half()   # (by a number torch multiplies with its reciprocal)
    sf, z = s.float(), lo.half().float()
    q = torch.where(sf > 0, torch.round((y - z) / torch.where(sf > 0, sf, torch.ones_like(sf))), torch.zeros_like(y))
    return (q.clamp(0, 2 ** bits - 1).to(F64) * sf.to(F64) + z.to(F64)).view(m, r)


def cached(c, T, R, bits, G):
    """The first T of a sequence's vectors c as attention sees them."""
    k = max(0, T - R)
    return torch.cat((quantized(c[:k], bits, G), c[k:T].to(F64))) if k else c[:T].to(F64)


def half(x):
    """64-bit x in fp16, rounded once (torch rounds to fp32 on the way)."""
    return torch.from_numpy(x.cpu().numpy().astype(np.float16)).to(x.device)


def attend(q, keys, values, first, scale):
    """Rows q [n, d] at positions first.. over keys [S, d] and values [S, dv] at
    0..: the output, sum_s w |v|, and each row's largest scale sum |q k|."""
    q, keys, values = q.to(F64), keys.to(F64), values.to(F64)
    n, S = q.shape[0], keys.shape[0]
    see = torch.arange(S, device=q.device) <= torch.arange(first, first + n, device=q.device).view(n, 1)
    w = torch.softmax((scale * (q @ keys.t())).masked_fill(~see, -math.inf), 1)
    mag = (scale * (q.abs() @ keys.abs().t())).masked_fill(~see, 0).amax(1)
    return w @ values, w @ values.abs(), mag


def attn_bound(wabs, mag, S, d, scores=1.0, values=1.0):
    """What an attention output may be off by before it is rounded.  scores:
    roundings to fp16 among a score's factors (half a step of every product: H
    mag each), d products summed in fp32 (d 2^-23 mag; a tensor core may cut off
    where it could round).  A weight is off by a factor exp(that), and so is their
    sum; rounded itself (H, below 2^-14 of its reference by 2^-25 of it: S of them
    against a sum of at least 2^-8 of 2^7-lifted ones: 2^-17 / 2^7 S); values:
    roundings of the values (H each); fp32 sums of S (2^-23 S)."""
    e = scores * H + d * 2.0 ** -23
    rel = torch.expm1(2 * e * mag).unsqueeze(1) + (1 + values) * H + S * (2.0 ** -23 + 2.0 ** -24)
    return wabs * rel


def check(got, ref, bound, what=""):
    """Every element within the bound and one rounding to fp16; and, the
    roundings being independent, the whole within 1.5e-3: six of H / sqrt(3) =
    2.8e-4 each, those of the scores' factors times the spread of their products
    (up to 2.2): sqrt(2 (2.2)^2 + 4) 2.8e-4 = 1.05e-3."""
    got = got.to(F64)
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    over = (got - ref).abs() - (bound + ref.abs() * H + 2.0 ** -24)
    assert float(over.max()) <= 0, f"{what}: {float(over.max()):.3e} over the bound"
    den = float(torch.linalg.norm(ref))
    if den > 0:
        rel = float(torch.linalg.norm(got - ref)) / den
        assert rel <= 1.5e-3, f"{what}: relative L2 error {rel:.3e}"


def latent(qn, qr, c, kr, wk, wv, first, scale, absorbed, restored=False):
    """One head's rows over tokens c (64 bits), kr: the output [n, 128] and what it
    may be off by before its last rounding.  Absorbed: q Wk, the restored c (as
    key and as value), the weights and the sums ol round to fp16; expanded: Wk c
    and Wv c (products of r terms in fp32: r 2^-23 of their size each), the
    weights, and with restored c too (H of every product's size)."""
    qn, qr, kr, wk, wv, c = (x.to(F64) for x in (qn, qr, kr, wk, wv, c))
    S, r = c.shape
    if absorbed:
        ql = qn @ wk
        spread = (qn.abs() @ wk.abs())             # |ql| plus what its own fp32 sum may lose
        q, keys = torch.cat((ql, qr), 1), torch.cat((c, kr), 1)
        o, wabs, mag = attend(q, keys, c, first, scale)
        mag = mag + 128 * 2.0 ** -12 * scale * (spread @ c.abs().t()).amax(1)
        e = attn_bound(wabs, mag, S, r + 64, scores=2.0)
        e = e + o.abs() * H + 2.0 ** -24           # ol is rounded
        out = o @ wv.t()
        return out, e @ wv.abs().t() + r * 2.0 ** -23 * (o.abs() @ wv.abs().t())
    k, v = c @ wk.t(), c @ wv.t()
    ka, va = c.abs() @ wk.abs().t(), c.abs() @ wv.abs().t()
    o, wabs, mag = attend(torch.cat((qn, qr), 1), torch.cat((k, kr), 1), v, first, scale)
    own = r * 2.0 ** -12 + (1 if restored else 0)
    mag = mag + own * scale * (qn.abs() @ ka.t()).amax(1)
    return o, attn_bound(wabs + own * va.amax(0), mag, S, 192)


def verify(p, q, draft, u, n):
    """One sequence's tokens (numpy; p [ns + 1, V], q [ns, V] or None, n drafted):
    whole numbers throughout, Python's own for the mark."""
    def units(row):
        x = row.astype(np.float64)
        return np.floor(np.where(x > 0, np.minimum(x, 1.0), 0.0) * 2.0 ** 40).astype(np.int64)

    ns, V = p.shape[0] - 1, p.shape[1]
    out, r = np.full(ns + 1, -1, np.int32), 0
    while r < n:
        x = int(draft[r])
        if not 0 <= x < V:
            break
        if not float(u[r]) * (1.0 if q is None else float(q[r, x])) < float(p[r, x]):
            break
        out[r] = x
        r += 1
    plain = units(p[r])
    w = plain
    if r < n:
        if q is None:
            w = plain.copy()
            if 0 <= int(draft[r]) < V:
                w[int(draft[r])] = 0
        else:
            w = np.maximum(plain - units(q[r]), 0)
        if not w.any():
            w = plain
    total = int(w.sum())
    if total:
        x = float(u[ns])
        U = int(min(x, 1.0 - 2.0 ** -24) * 2.0 ** 30) if x > 0 else 0
        out[r] = np.searchsorted(np.cumsum(w), U * total >> 30, side="right")
    return out, r
