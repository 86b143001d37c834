"""What the chunk attention's 16-bit roundings can do to its result: a bound
for every element, and the expected size of the whole error."""
from __future__ import annotations

import numpy as np

H = 2.0 ** -11   # half a step of fp16, relative
F = 2.0 ** -25   # ... in its subnormals


def attend(q, k, v, see, restored=True):
    """Rows q [n, d] over k, v [S, d] in 64 bits: the output [n, d], the error's
    bound of each element and its expected square.

    Bound.  A restored key is off by at most H |k| + F, so a score by at most
    e = (H sum |q k| + F sum |q|) / sqrt(d) and a normalized weight by a factor
    exp(2 e).  A weight is rounded by H of itself, or in the subnormals by F
    where the reference's own weight is 2^7: 2^-32 of a weight that is at most
    the row's largest, for each visible token, times its value.  A value is
    rounded by H of itself, the output by H of itself and F; the 32-bit
    exponent, exponential and sums add 2^-19 and S 2^-23 of sum w |v|.

    Expected square.  The roundings of different keys, weights and values are
    independent, each uniform within half a step at most, so of variance at
    most H^2 / 3 relative: a score's variance is sum (q k)^2 / d times that,
    and it moves the output by w (v - out).

    restored: False where keys and values are fp16 as they come: they are not
    rounded then."""
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    d, S = q.shape[1], k.shape[0]
    x = np.where(see, q @ k.T / np.sqrt(d), -np.inf)
    w = np.exp(x - x.max(1, keepdims=True))
    L = w.sum(1, keepdims=True)
    w /= L
    out, wabs = w @ v, w @ np.abs(v)
    e = np.where(see, (H * np.abs(q) @ np.abs(k).T + F * np.abs(q).sum(1, keepdims=True)) / np.sqrt(d), 0).max(1, keepdims=True)
    if not restored:
        e = e * 0
    bound = (wabs * (np.expm1(2 * e) + (1 + restored) * H + 2.0 ** -19 + S * 2.0 ** -23) + H * np.abs(out) +
             2.0 ** -32 * (see @ np.abs(v)) / L + 2 * F)
    u = H * H / 3
    w2, s2 = w * w, np.where(see, (q * q) @ (k * k).T / d, 0) * u
    ws = w2 * s2   # sum_s w^2 var (v - out)^2, expanded
    moved = ws @ (v * v) - 2 * out * (ws @ v) + out * out * ws.sum(1, keepdims=True)
    return out, bound, moved * restored + (1 + restored) * u * (w2 @ (v * v)) + u * out * out


def check(got, want, what=""):
    """got and want = [(output, bound, expected square), ...] of the same rows:
    every element within its bound, and the whole within 1.5 times its expected
    size."""
    got = [np.asarray(g, np.float64) for g in got]
    for g, (o, b, _) in zip(got, want):
        assert np.all(np.isfinite(g)), f"{what}: non-finite output"
        over = np.abs(g - o) - b
        assert np.all(over <= 0), f"{what}: {over.max():.3e} over the bound at {np.unravel_index(np.argmax(over), over.shape)}"
    err = np.sqrt(sum(((g - o) ** 2).sum() for g, (o, _, _) in zip(got, want)))
    size = np.sqrt(sum(s.sum() for _, _, s in want))
    assert err <= 1.5 * size, f"{what}: error {err:.3e}, expected {size:.3e}"
