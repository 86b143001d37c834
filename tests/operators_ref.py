"""Plain 64-bit references of the serving operators (rotary positions,
sliding-window and chunk attention over the quantized cache), and the bound
their fp16 results are held to."""
from __future__ import annotations

import numpy as np


def counters(t, R):
    """Quantized keys and values after a prefill of t tokens."""
    return t - t % R, max(t - R, 0)


def counters_after(T, Tqk, Tqv, n, R):
    """... and after n one-token appends (a full key window flushes, and a
    value queue of R + 1 pops, at the start of the next append)."""
    for _ in range(n):
        if T - Tqk == R:
            Tqk += R
        if T - Tqv == R + 1:
            Tqv += 1
        T += 1
    return T, Tqk, Tqv


def _quant(x, bits, axis):
    """zero + code * scale of groups along `axis` (fp32 arithmetic, fp16
    scale and zero), in 64 bits."""
    x = x.astype(np.float32)
    lo, hi = x.min(axis, keepdims=True), x.max(axis, keepdims=True)
    s = ((hi - lo) / np.float32(2 ** bits - 1)).astype(np.float16)
    z = lo.astype(np.float16).astype(np.float32)
    sf = s.astype(np.float32)
    q = np.where(sf > 0, np.rint((x - z) / np.where(sf > 0, sf, np.float32(1))), 0)
    q = np.clip(q, 0, 2 ** bits - 1)
    return q.astype(np.float64) * sf.astype(np.float64) + z.astype(np.float64)


def restore(K, V, Tqk, Tqv, kb, vb, G):
    """One slice's keys and values [t, d] (fp16) as attention sees them."""
    k, v = K.astype(np.float64), V.astype(np.float64)
    d = K.shape[1]
    if Tqk:
        k[:Tqk] = _quant(K[:Tqk].reshape(Tqk // G, G, d), kb, 1).reshape(Tqk, d)
    if Tqv:
        v[:Tqv] = _quant(V[:Tqv].reshape(Tqv, d // G, G), vb, 2).reshape(Tqv, d)
    return k, v


def visible(pos, S, window, sinks):
    """[n, S] truth values: what queries at positions pos see of tokens 0..S-1."""
    p, s = np.asarray(pos)[:, None], np.arange(S)[None, :]
    see = s <= p
    if window:
        see &= (p - s < window) | (s < sinks)
    return see


def attend(q, k, v, see):
    """Rows q [n, d] over k, v [S, d]: the output [n, d], and what bounds its
    error: sum_s w |v| [n, d] and the largest visible sum_c |q_c k_c| / sqrt(d)
    [n]."""
    q = q.astype(np.float64)
    d = q.shape[1]
    x = np.where(see, q @ k.T / np.sqrt(d), -np.inf)
    w = np.exp(x - x.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    mag = np.where(see, np.abs(q) @ np.abs(k).T / np.sqrt(d), 0).max(1)
    return w @ v, w @ np.abs(v), mag


def check_rounded(got, ref, wabs, mag, S, what=""):
    """The chunk attention's result against the reference.

    Pointwise: each restored key is rounded to fp16 (half a step: 2^-11), so
    a score is off by at most 2^-11 mag and a weight, after normalizing, by a
    factor exp(2 * 2^-11 mag); a weight and a value are rounded once each
    (2^-11), a weight below 2^-14 of its row's reference by at most 2^-25 of
    it (S of them against a sum of at least 2^-8: 2^-17 S, weights being up
    to 2^8 above the reference never lowers this), 32-bit sums add S 2^-23,
    and the output is rounded (2^-11).
    In norm: the roundings are independent and about 2^-11 / sqrt(3) = 2.8e-4
    relative each (four of them, the score's times the keys' spread, < 2.2):
    1e-3 covers them; 1.5e-3 is the bar."""
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    h = 2.0 ** -11
    rel = np.expm1(2 * h * mag)[:, None] + 2 * h + S * 2.0 ** -23
    bound = wabs * rel + np.abs(ref) * h + np.abs(wabs) * S * 2.0 ** -25 + 2.0 ** -24
    err = np.abs(got - ref)
    assert np.all(err <= bound), f"{what}: error {(err - bound).max():.3e} over the bound at {np.argmax(err - bound)}"
    den = np.linalg.norm(ref)
    if den > 0:
        r = np.linalg.norm(got - ref) / den
        assert r <= 1.5e-3, f"{what}: relative L2 error {r:.3e}"


def rotate(x, pos, inv_freq, factor, rot, interleaved, inverse=False):
    """Rows x [n, d] at positions pos [n]."""
    x = np.asarray(x, np.float64)
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq)[None, :]
    c, s = factor * np.cos(a), factor * np.sin(a) * (-1 if inverse else 1)
    y = x.copy()
    i0 = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    i1 = i0 + 1 if interleaved else i0 + rot // 2
    y[:, i0] = x[:, i0] * c - x[:, i1] * s
    y[:, i1] = x[:, i1] * c + x[:, i0] * s
    return y
