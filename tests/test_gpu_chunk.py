"""Chunk attention over the cache, the chunk append and the extend path
against 64-bit references and the one-token calls."""
import numpy as np
import pytest

from tests import kivi_testutil as U
from tests import operators_ref as R


def _cuda(*xs):
    import torch
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in xs]


def _setup(b, hq, h, d, kb, vb, G, Rw, T, steps, n, seed, extra=0):
    """A cache filled with T[i] tokens and `steps` appends, and a chunk."""
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    rng = np.random.default_rng(seed)
    t, ns = max(max(T), 1), max(max(n), 1) + 2
    Kh, Vh = (rng.standard_normal((b, h, t, d)).astype(np.float16) for _ in range(2))
    ks, vs = (rng.standard_normal((steps, b, h, d)).astype(np.float16) for _ in range(2))
    c = K.KiviCache(b, h, d, kb, vb, G, Rw, t + steps + max(max(n), 1) + extra)
    c.prefill(*_cuda(Kh, Vh), T)
    for s in range(steps):
        c.append(*_cuda(ks[s], vs[s]))
    Q = rng.standard_normal((b, hq, ns, d)).astype(np.float16)
    Kn, Vn = (rng.standard_normal((b, h, ns, d)).astype(np.float16) for _ in range(2))
    Kn[:, :, -2:], Vn[:, :, -2:] = np.nan, np.inf   # rows past every chunk: never read
    keys = [np.concatenate([Kh[i, :, :T[i]], ks[:, i].swapaxes(0, 1)], 1) for i in range(b)]
    vals = [np.concatenate([Vh[i, :, :T[i]], vs[:, i].swapaxes(0, 1)], 1) for i in range(b)]
    return c, Q, Kn, Vn, keys, vals


CASES = [
    # b, hq, h, d, kb, vb, G, R, T, appends, n, window, sinks
    (1, 1, 1, 64, 2, 2, 32, 32, [0], 0, [1], 0, 0),             # one token, nothing cached
    (1, 4, 1, 128, 2, 2, 32, 128, [200], 0, [1], 0, 0),
    (1, 3, 3, 64, 4, 4, 16, 16, [100], 0, [70], 0, 0),          # key blocks half window (R = 16)
    (2, 8, 1, 128, 4, 2, 64, 64, [321, 64], 33, [5, 40], 0, 0),
    (3, 6, 2, 64, 2, 4, 16, 48, [0, 500, 77], 3, [130, 0, 65], 0, 0),   # a sequence left out
    (2, 10, 2, 128, 2, 2, 128, 128, [1000, 128], 130, [64, 3], 0, 0),   # groups over two blocks
    (1, 4, 2, 128, 2, 2, 32, 128, [2000], 0, [4], 0, 0),        # few rows: split and joined
    (1, 8, 2, 64, 4, 4, 32, 96, [3001], 7, [9], 0, 0),
    (1, 4, 1, 128, 2, 2, 32, 128, [900], 0, [200], 0, 0),       # rows over several CTAs of two slots
    (1, 7, 1, 64, 2, 4, 64, 64, [10], 0, [300], 0, 0),          # seven heads a kv head
    (2, 4, 2, 128, 4, 4, 32, 32, [700, 90], 5, [150, 33], 100, 4),
    (1, 4, 1, 128, 2, 2, 32, 128, [3000], 0, [7], 500, 3),      # windows with few rows
    (1, 2, 1, 64, 2, 2, 16, 32, [600], 0, [260], 1, 0),         # a token sees only itself
    (1, 2, 1, 64, 2, 2, 16, 32, [600], 0, [200], 64, 130),
    (1, 2, 1, 64, 2, 2, 16, 32, [40], 0, [200], 100000, 100000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("b,hq,h,d,kb,vb,G,Rw,T,steps,n,window,sinks", CASES)
def test_chunk_attention(b, hq, h, d, kb, vb, G, Rw, T, steps, n, window, sinks):
    import torch
    c, Q, Kn, Vn, keys, vals = _setup(b, hq, h, d, kb, vb, G, Rw, T, steps, n, 17 + sum(T))
    Qt, Kt, Vt = _cuda(Q, Kn, Vn)
    before = c.export()
    out = torch.full_like(Qt, 7.0)
    assert c.chunk_attn(Qt, Kt, Vt, n, window, sinks, out=out) is out
    again = c.chunk_attn(Qt, Kt, Vt, n, window, sinks)
    got = out.float().cpu().numpy()
    assert c.check() == 0
    g = hq // h
    for i in range(b):
        assert np.all(got[i, :, n[i]:] == 7.0)
        assert torch.equal(again[i, :, :n[i]], out[i, :, :n[i]]) and not again[i, :, n[i]:].any()
        if n[i] == 0:
            continue
        t = T[i] + steps
        _, qk, qv = R.counters_after(T[i], *R.counters(T[i], Rw), steps, Rw)
        for j in range(h):
            k, v = R.restore(keys[i][j], vals[i][j], qk, qv, kb, vb, G)
            k = np.concatenate([k, Kn[i, j, :n[i]].astype(np.float64)])
            v = np.concatenate([v, Vn[i, j, :n[i]].astype(np.float64)])
            see = R.visible(t + np.arange(n[i]), t + n[i], window, sinks)
            for e in range(j * g, (j + 1) * g):
                ref, wabs, mag = R.attend(Q[i, e, :n[i]], k, v, see)
                R.check_rounded(got[i, e, :n[i]], ref, wabs, mag, t + n[i], f"sequence {i} head {e}")
    after = c.export()
    assert all(np.array_equal(before[x], after[x]) for x in before)   # read-only
    c.close()


def _attention_case(b, hq, h, d, kb, vb, G, Rw, T, steps, n, window, sinks):
    c, Q, Kn, Vn, keys, vals = _setup(b, hq, h, d, kb, vb, G, Rw, T, steps, n, 5 + d + G + sum(n))
    out = c.chunk_attn(*_cuda(Q, Kn, Vn), n, window, sinks).float().cpu().numpy()
    for i in range(b):
        t = T[i] + steps
        _, qk, qv = R.counters_after(T[i], *R.counters(T[i], Rw), steps, Rw)
        for j in range(h):
            k, v = R.restore(keys[i][j], vals[i][j], qk, qv, kb, vb, G)
            k = np.concatenate([k, Kn[i, j, :n[i]].astype(np.float64)])
            v = np.concatenate([v, Vn[i, j, :n[i]].astype(np.float64)])
            see = R.visible(t + np.arange(n[i]), t + n[i], window, sinks)
            for e in range(j * (hq // h), (j + 1) * (hq // h)):
                ref, wabs, mag = R.attend(Q[i, e, :n[i]], k, v, see)
                R.check_rounded(out[i, e, :n[i]], ref, wabs, mag, t + n[i], f"sequence {i} head {e}")
    assert c.check() == 0
    c.close()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb", [2, 4])
@pytest.mark.parametrize("vb", [2, 4])
@pytest.mark.parametrize("G", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [3, 45])
def test_chunk_attention_formats(d, kb, vb, G, n):
    """Every record format, with few rows and with many."""
    if G > d:
        pytest.skip("needs d % G == 0")
    _attention_case(1, 4, 1, d, kb, vb, G, max(G, 32), [413], G // 8, [n], 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("n,hq", [(1, 8), (2, 8), (5, 5), (8, 2), (16, 4), (13, 8), (17, 8), (64, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 70), (3, 0)])
def test_chunk_attention_row_counts(n, hq, window, sinks):
    """Row counts around the row tiles' sizes, even and odd numbers of blocks."""
    _attention_case(2, hq, 1, 128, 2, 4, 32, 32, [700, 10], 1, [n, max(n - 1, 1)], window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 40])
def test_growing_scores(n):
    """Keys grow along the sequence, so the running maximum rises by far more
    than 2^8 in weight again and again."""
    from bit_quantized_kv_quantize_gb300 import kivi as K
    rng = np.random.default_rng(4)
    t, d = 1500, 64
    Kh, Vh = (rng.standard_normal((1, 1, t, d)).astype(np.float16) for _ in range(2))
    Kh[:] = np.abs(Kh) * (np.arange(t) / 150.0).astype(np.float16)[None, None, :, None]
    Q = np.abs(rng.standard_normal((1, 2, n, d))).astype(np.float16)
    Kn, Vn = (rng.standard_normal((1, 1, n, d)).astype(np.float16) for _ in range(2))
    c = K.KiviCache(1, 1, d, 4, 4, 32, 64, t + n)
    c.prefill(*_cuda(Kh, Vh), t)
    out = c.chunk_attn(*_cuda(Q, Kn, Vn), n).float().cpu().numpy()
    k, v = R.restore(Kh[0, 0], Vh[0, 0], *R.counters(t, 64), 4, 4, 32)
    k, v = np.concatenate([k, Kn[0, 0].astype(np.float64)]), np.concatenate([v, Vn[0, 0].astype(np.float64)])
    for e in range(2):
        ref, wabs, mag = R.attend(Q[0, e], k, v, R.visible(t + np.arange(n), t + n, 0, 0))
        got, h = out[0, e].astype(np.float64), 2.0 ** -11
        # (the pointwise part of check_rounded: few tokens carry these rows, so
        # their roundings do not average)
        bound = wabs * (np.expm1(2 * h * mag)[:, None] + 2 * h + (t + n) * 2.0 ** -23) + np.abs(ref) * h
        assert np.all(np.abs(got - ref) <= bound + wabs * (t + n) * 2.0 ** -25 + 2.0 ** -24)
    c.close()


@pytest.mark.gpu
@pytest.mark.parametrize("b,h,d,kb,vb,G,Rw,T,steps,n", [
    (1, 1, 64, 2, 2, 32, 32, [0], 0, 1),
    (1, 1, 64, 2, 2, 32, 32, [0], 0, 200),
    (2, 2, 128, 2, 4, 32, 128, [300, 128], 0, 1),
    (2, 2, 128, 4, 2, 64, 64, [321, 5], 33, 95),
    (1, 3, 64, 4, 4, 16, 48, [47], 1, 48),      # the first append flushes
    (1, 3, 64, 4, 4, 16, 48, [47], 2, 49),
    (1, 1, 256, 2, 2, 128, 128, [130], 129, 300),
    (1, 2, 256, 4, 4, 16, 16, [17], 0, 130),
    (1, 2, 128, 2, 2, 128, 256, [100], 0, 700),
    (1, 2, 128, 2, 2, 32, 4096, [1000], 0, 5000),
])
def test_append_chunk_is_n_appends(b, h, d, kb, vb, G, Rw, T, steps, n):
    """Whole export equal, live and stale slots alike, and the counters; then
    both caches take one more token."""
    from bit_quantized_kv_quantize_gb300 import kivi as K
    c, _, Kn, Vn, _, _ = _setup(b, h, h, d, kb, vb, G, Rw, T, steps, [n] * b, 3, extra=1)
    e, _, _, _, _, _ = _setup(b, h, h, d, kb, vb, G, Rw, T, steps, [n] * b, 3, extra=1)
    Kt, Vt = _cuda(Kn, Vn)
    c.append_chunk(Kt, Vt, n)
    for r in range(n):
        e.append(Kt[:, :, r].contiguous(), Vt[:, :, r].contiguous())
    for x, y in zip(c.lengths(), e.lengths()):
        assert np.array_equal(x, y)
    for _ in range(2):
        a, f = c.export(), e.export()
        for name in a:
            assert np.array_equal(a[name], f[name]), name
        if c.lengths()[0].max() < c.max_tokens:
            for z in (c, e):
                z.append(Kt[:, :, 0].contiguous(), Vt[:, :, 0].contiguous())
    q = _cuda(np.random.default_rng(1).standard_normal((b, h, d)).astype(np.float16))[0]
    assert (c.decode(q) == e.decode(q)).all()
    assert c.check() == 0
    with pytest.raises(K.CapacityError):
        c.append_chunk(Kt, Vt, n)
    c.close()
    e.close()


@pytest.mark.gpu
def test_append_chunk_ragged():
    """Each sequence as if alone."""
    from bit_quantized_kv_quantize_gb300 import kivi as K
    b, h, d, T, n = 4, 2, 64, [100, 0, 33, 64], [0, 77, 1, 40]
    c, _, Kn, Vn, keys, vals = _setup(b, h, h, d, 2, 4, 16, 32, T, 0, n, 8)
    Kt, Vt = _cuda(Kn, Vn)
    c.append_chunk(Kt, Vt, n)
    gex = c.export()
    cap = c.max_tokens
    gg = U.geometry(b, h, d, 2, 4, 16, 32, cap)
    for i in range(b):
        e = K.KiviCache(1, h, d, 2, 4, 16, 32, cap)
        if T[i]:
            e.prefill(*_cuda(keys[i][None], vals[i][None]), T[i])
        for r in range(n[i]):
            e.append(Kt[i:i + 1, :, r].contiguous(), Vt[i:i + 1, :, r].contiguous())
        Te, qk, qv = (int(x[0]) for x in e.lengths())
        assert [int(x[i]) for x in c.lengths()] == [Te, qk, qv]
        eex, ge = e.export(), U.geometry(1, h, d, 2, 4, 16, 32, cap)
        for j in range(h):
            U.compare_slice(gex, gg, i, j, eex, ge, 0, j, Te, qk, qv, f"sequence {i}")
        e.close()
    c.close()


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 4)])
def test_extend_in_pieces(window, sinks):
    """A prompt taken in ragged pieces with rotary positions, then a decode
    step: each piece against the 64-bit reference, and the cache bitwise the
    one that the rotated tokens leave one at a time."""
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    rng = np.random.default_rng(21)
    b, hq, h, d, kb, vb, G, Rw = 2, 4, 2, 64, 4, 4, 16, 32
    pieces = [[40, 1], [17, 100], [0, 64], [33, 5]]
    rope = K.Rope(d, base=5e5)
    c = K.KiviCache(b, h, d, kb, vb, G, Rw, 200)
    e = [K.KiviCache(1, h, d, kb, vb, G, Rw, 200) for _ in range(b)]
    keys = [np.zeros((h, 0, d), np.float16) for _ in range(b)]
    vals = [np.zeros((h, 0, d), np.float16) for _ in range(b)]
    cnt = [(0, 0, 0)] * b
    for n in pieces:
        ns = max(n)
        Q = rng.standard_normal((b, hq, ns, d)).astype(np.float16)
        Kn, Vn = (rng.standard_normal((b, h, ns, d)).astype(np.float16) for _ in range(2))
        Qt, Kt, Vt = _cuda(Q, Kn, Vn)
        Qr, Kr = (x.cpu().numpy() for x in rope.apply(Qt, Kt, [x[0] for x in cnt], n=n))
        out = c.extend(Qt, Kt, Vt, n, window, sinks, rope=rope).float().cpu().numpy()
        assert torch.equal(Kt.cpu(), torch.from_numpy(Kn))   # the caller's keys stay
        for i in range(b):
            T, qk, qv = cnt[i]
            assert not out[i, :, n[i]:].any()
            for j in range(h):
                k, v = R.restore(keys[i][j], vals[i][j], qk, qv, kb, vb, G)
                k = np.concatenate([k, Kr[i, j, :n[i]].astype(np.float64)])
                v = np.concatenate([v, Vn[i, j, :n[i]].astype(np.float64)])
                for q in range(j * 2, j * 2 + 2):
                    if n[i]:
                        ref, wabs, mag = R.attend(Qr[i, q, :n[i]], k, v,
                                                  R.visible(T + np.arange(n[i]), T + n[i], window, sinks))
                        R.check_rounded(out[i, q, :n[i]], ref, wabs, mag, T + n[i])
            keys[i] = np.concatenate([keys[i], Kr[i, :, :n[i]]], 1)
            vals[i] = np.concatenate([vals[i], Vn[i, :, :n[i]]], 1)
            cnt[i] = R.counters_after(T, qk, qv, n[i], Rw)
            for r in range(n[i]):
                e[i].append(*_cuda(Kr[i:i + 1, :, r], Vn[i:i + 1, :, r]))
        assert [list(x) for x in np.stack(c.lengths()).T] == [list(x) for x in cnt]
    gex, gg = c.export(), U.geometry(b, h, d, kb, vb, G, Rw, 200)
    q = rng.standard_normal((b, hq, d)).astype(np.float16)
    got = c.decode(*_cuda(q), window=window, sinks=sinks).float().cpu().numpy()
    ref = np.zeros_like(got, np.float64)
    for i in range(b):
        eex, ge = e[i].export(), U.geometry(1, h, d, kb, vb, G, Rw, 200)
        for j in range(h):
            U.compare_slice(gex, gg, i, j, eex, ge, 0, j, *cnt[i], f"sequence {i}")
            k, v = R.restore(keys[i][j], vals[i][j], cnt[i][1], cnt[i][2], kb, vb, G)
            ref[i, 2 * j:2 * j + 2] = R.attend(q[i, 2 * j:2 * j + 2], k, v,
                                               R.visible([cnt[i][0] - 1] * 2, cnt[i][0], window, sinks))[0]
        e[i].close()
    U.compare_output(got, ref, "decode after the pieces")
    assert c.check() == 0
    c.close()


@pytest.mark.gpu
def test_draft_left_out_leaves_no_trace():
    """Verify a draft, keep part of it: the cache is the one without it."""
    c, Q, Kn, Vn, _, _ = _setup(2, 4, 2, 128, 2, 2, 32, 128, [500, 129], 3, [6, 6], 4)
    e, _, _, _, _, _ = _setup(2, 4, 2, 128, 2, 2, 32, 128, [500, 129], 3, [6, 6], 4)
    Qt, Kt, Vt = _cuda(Q, Kn, Vn)
    c.chunk_attn(Qt, Kt, Vt, 6)
    for z in (c, e):
        z.append_chunk(Kt, Vt, [2, 5])
    a, f = c.export(), e.export()
    assert all(np.array_equal(a[x], f[x]) for x in a)
    c.close()
    e.close()


@pytest.mark.gpu
def test_other_stream_and_graph():
    import torch
    c, Q, Kn, Vn, _, _ = _setup(1, 4, 1, 128, 2, 2, 32, 128, [2100], 0, [5], 2)
    Qt, Kt, Vt = _cuda(Q, Kn, Vn)
    ref = c.chunk_attn(Qt, Kt, Vt, 5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.chunk_attn(Qt, Kt, Vt, 5, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, ref)
    out = torch.zeros_like(Qt)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.chunk_attn(Qt, Kt, Vt, 5, out=out)
    Q2 = torch.randn_like(Qt)
    Qt.copy_(Q2)
    g.replay()
    assert torch.equal(out, c.chunk_attn(Q2, Kt, Vt, 5))
    c.close()


@pytest.mark.gpu
def test_refusals():
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    c, Q, Kn, Vn, _, _ = _setup(2, 4, 2, 64, 2, 2, 32, 32, [50, 60], 0, [4, 4], 2)
    Qt, Kt, Vt = _cuda(Q, Kn, Vn)

    def status(f):
        with pytest.raises(K.KiviError) as e:
            f()
        return e.value.status

    assert status(lambda: c.chunk_attn(Qt, Kt, Vt, 7)) == 1            # n above n_stride
    assert status(lambda: c.chunk_attn(Qt, Kt, Vt, [-1, 2])) == 1
    assert status(lambda: c.chunk_attn(Qt, Kt, Vt, 2, window=-1)) == 1
    assert status(lambda: c.chunk_attn(Qt[:, :3].contiguous(), Kt, Vt, 2)) == 1   # h_q not a multiple of h_kv
    assert status(lambda: c.append_chunk(Kt, Vt, [6, 6])) == 3          # capacity: 60 + 6 > 64
    with pytest.raises(K.CapacityError):
        c.extend(Qt, Kt, Vt, [1, 5])
    for bad in (lambda: c.chunk_attn(Qt, Kt, Vt, [1, 2, 3]), lambda: c.chunk_attn(Qt, Kt, Vt, 1.5),
                lambda: c.chunk_attn(Qt, Kt[:, :1], Vt, 1), lambda: c.append_chunk(Kt.float(), Vt, 1)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    assert c.lengths()[0].tolist() == [50, 60]
    c.chunk_attn(Qt, Kt, Vt, 0)
    c.append_chunk(Kt, Vt, 0)
    assert c.lengths()[0].tolist() == [50, 60]
    c.append_chunk(Kt, Vt, [6, 4])
    assert c.lengths()[0].tolist() == [56, 64]
    c.close()
    w = K.KiviCache(1, 1, 256, 2, 2, 32, 32, 64)
    x = torch.zeros(1, 1, 4, 256, device="cuda").half()
    assert status(lambda: w.chunk_attn(x, x, x, 1)) == 2                # d = 256
    w.append_chunk(x, x, 4)
    w.close()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 90])
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 64, 2**31, 2**40])
def test_window_beyond_every_position(n, window):
    """A window that no position reaches is no window, in every call; both
    row-tile forms."""
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    rng = np.random.default_rng(window % 97 + n)
    b, h, hq, d, t = 2, 2, 4, 64, 200
    c = K.KiviCache(b, h, d, 2, 4, 32, 32, t + n)
    Q, Kp, Vp = _cuda(*(rng.standard_normal((b, x, t, d)).astype(np.float16) for x in (hq, h, h)))
    plain = c.prefill_attn(Q, Kp, Vp, t)
    # (another kernel than the plain prompt's: each rounds the weights to fp16
    # and its output, by 2^-11 of at most max |V|)
    diff = (c.prefill_attn(Q, Kp, Vp, t, window=window).float() - plain.float()).abs().max()
    assert diff <= 4 * 2.0 ** -11 * Vp.abs().max().float()
    q = Q[:, :, :n].contiguous()
    k, v = Kp[:, :, :n].contiguous(), Vp[:, :, :n].contiguous()
    assert torch.equal(c.chunk_attn(q, k, v, n, window=window, sinks=2**31), c.chunk_attn(q, k, v, n))
    assert torch.equal(c.decode(q[:, :, 0].contiguous(), window=window, sinks=2**40), c.decode(q[:, :, 0].contiguous()))
    assert torch.equal(c.chunk_attn(q, k, v, n, window=7, sinks=2**32 + 1), c.chunk_attn(q, k, v, n, window=7, sinks=2**31 - 1))
    for bad in (-1, -2**31, -2**32, -2**40):
        with pytest.raises(K.KiviError):
            c.chunk_attn(q, k, v, n, window=bad)
        with pytest.raises(K.KiviError):
            c.decode(q[:, :, 0].contiguous(), window=4, sinks=bad)
        with pytest.raises(K.KiviError):
            c.prefill_attn(Q, Kp, Vp, t, window=bad)
    for bad in (4.0, "4", None):
        with pytest.raises(TypeError):
            c.chunk_attn(q, k, v, n, window=bad)
    assert c.check() == 0
    c.close()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,vb", [(2, 2), (2, 4), (4, 2), (4, 4)])
@pytest.mark.parametrize("G", [16, 32, 64, 128])
def test_few_rows_over_long_sequences(d, kb, vb, G):
    """Few query rows over 32 blocks and more have row tiles of their own:
    every record format, a short and an empty sequence beside the long one."""
    if G > d:
        pytest.skip("needs d % G == 0")
    _attention_case(3, 4, 1, d, kb, vb, G, max(G, 32), [2413, 90, 0], G // 8, [3, 4, 2], 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("n,hq", [(1, 8), (2, 8), (5, 3), (8, 2), (16, 1), (4, 4)])
@pytest.mark.parametrize("T", [2040, 2300])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2035, 0), (2100, 70)])
def test_few_rows_counts_and_windows(n, hq, T, window, sinks):
    """Row counts up to a whole tile, at the length from which they have their
    own row tiles, windows that end inside a block."""
    _attention_case(2, hq, 1, 128, 2, 4, 32, 32, [T, 10], 1, [n, max(n - 1, 1)], window, sinks)


@pytest.mark.gpu
def test_growing_scores_few_rows():
    """As test_growing_scores, long enough for few rows' own tiles."""
    from bit_quantized_kv_quantize_gb300 import kivi as K
    rng = np.random.default_rng(4)
    t, d, n = 2600, 64, 2
    Kh, Vh = (rng.standard_normal((1, 1, t, d)).astype(np.float16) for _ in range(2))
    Kh[:] = np.abs(Kh) * (np.arange(t) / 260.0).astype(np.float16)[None, None, :, None]
    Q = np.abs(rng.standard_normal((1, 2, n, d))).astype(np.float16)
    Kn, Vn = (rng.standard_normal((1, 1, n, d)).astype(np.float16) for _ in range(2))
    c = K.KiviCache(1, 1, d, 4, 4, 32, 64, t + n)
    c.prefill(*_cuda(Kh, Vh), t)
    out = c.chunk_attn(*_cuda(Q, Kn, Vn), n).float().cpu().numpy()
    k, v = R.restore(Kh[0, 0], Vh[0, 0], *R.counters(t, 64), 4, 4, 32)
    k, v = np.concatenate([k, Kn[0, 0].astype(np.float64)]), np.concatenate([v, Vn[0, 0].astype(np.float64)])
    for e in range(2):
        ref, wabs, mag = R.attend(Q[0, e], k, v, R.visible(t + np.arange(n), t + n, 0, 0))
        got, h = out[0, e].astype(np.float64), 2.0 ** -11
        # (the pointwise part of check_rounded: few tokens carry these rows, so
        # their roundings do not average)
        bound = wabs * (np.expm1(2 * h * mag)[:, None] + 2 * h + (t + n) * 2.0 ** -23) + np.abs(ref) * h
        assert np.all(np.abs(got - ref) <= bound + wabs * (t + n) * 2.0 ** -25 + 2.0 ** -24)
    c.close()
