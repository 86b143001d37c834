"""Sliding window with sinks: decode over the cache and the prompt's
attention against 64-bit references.  Hidden tokens carry large values, so
that one seen by mistake shows."""
import numpy as np
import pytest

from tests import kivi_testutil as U
from tests import operators_ref as R


def _inputs(rng, b, h, t, d, loud):
    K = rng.standard_normal((b, h, t, d)).astype(np.float16)
    V = rng.standard_normal((b, h, t, d)).astype(np.float16)
    if loud is not None:   # tokens [lo, hi) of every sequence
        lo, hi = loud
        V[:, :, lo:hi] += 64
    return K, V


@pytest.mark.gpu
@pytest.mark.parametrize("b,hq,h,d,kb,vb,G,Rw,T,steps,window,sinks", [
    (1, 4, 1, 64, 2, 2, 32, 32, [300], 0, 40, 0),
    (1, 4, 1, 64, 2, 2, 32, 32, [300], 5, 1, 0),          # only itself
    (2, 4, 2, 128, 4, 4, 32, 128, [1000, 1], 3, 200, 4),
    (2, 8, 1, 128, 2, 4, 64, 64, [129, 640], 70, 64, 64),
    (3, 3, 3, 64, 4, 2, 16, 48, [0, 700, 65], 2, 17, 70),  # sinks past a block, an empty sequence
    (1, 5, 1, 256, 2, 2, 128, 128, [900], 1, 333, 1),
    (1, 4, 2, 128, 2, 2, 32, 128, [500], 0, 10000, 9),    # a window longer than the sequence
    (1, 4, 2, 128, 2, 2, 32, 128, [500], 0, 77, 10000),   # sinks longer than the sequence
    (2, 16, 4, 128, 2, 2, 32, 128, [5000, 9001], 0, 1024, 4),
])
def test_decode_window(b, hq, h, d, kb, vb, G, Rw, T, steps, window, sinks):
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    rng = np.random.default_rng(sum(T) + window)
    t = max(max(T), 1)
    Kh, Vh = _inputs(rng, b, h, t + steps, d, None)
    for i in range(b):   # loud where hidden
        p = T[i] + steps - 1
        if p - window >= sinks:
            Vh[i, :, sinks:p - window + 1] += 64
    c = K.KiviCache(b, h, d, kb, vb, G, Rw, t + steps)
    seq = [np.concatenate([Kh[i, :, :T[i]], Kh[i, :, t:]], 1) for i in range(b)]
    vseq = [np.concatenate([Vh[i, :, :T[i]], Vh[i, :, t:]], 1) for i in range(b)]
    for i in range(b):   # the appended tokens' share of the loudness follows their position
        p = T[i] + steps - 1
        vseq[i][:, T[i]:] = rng.standard_normal(vseq[i][:, T[i]:].shape).astype(np.float16)
        if p - window >= sinks:
            vseq[i][:, max(sinks, T[i]):p - window + 1] += 64
    c.prefill(torch.from_numpy(Kh[:, :, :t]).cuda().contiguous(), torch.from_numpy(Vh[:, :, :t]).cuda().contiguous(), T)
    for s in range(steps):
        c.append(torch.from_numpy(np.stack([x[:, T[i] + s] for i, x in enumerate(seq)])).cuda(),
                 torch.from_numpy(np.stack([x[:, T[i] + s] for i, x in enumerate(vseq)])).cuda())
    q = rng.standard_normal((b, hq, d)).astype(np.float16)
    qt = torch.from_numpy(q).cuda()
    out = c.decode(qt, window=window, sinks=sinks)
    assert torch.equal(out, c.decode(qt, window=window, sinks=sinks))   # repeatable
    got = out.float().cpu().numpy()
    ref = np.zeros_like(got, np.float64)
    for i in range(b):
        n = T[i] + steps
        if n == 0:
            continue
        _, qk, qv = R.counters_after(T[i], *R.counters(T[i], Rw), steps, Rw)
        for j in range(h):
            k, v = R.restore(seq[i][j], vseq[i][j], qk, qv, kb, vb, G)
            g = hq // h
            ref[i, j * g:(j + 1) * g] = R.attend(q[i, j * g:(j + 1) * g], k, v,
                                                 R.visible([n - 1] * g, n, window, sinks))[0]
    U.compare_output(got, ref, "windowed decode")
    assert c.check() == 0
    c.close()


@pytest.mark.gpu
@pytest.mark.parametrize("b,hq,h,d,T,window,sinks", [
    (1, 2, 2, 64, [300], 50, 0),
    (1, 2, 2, 64, [300], 1, 0),
    (2, 4, 2, 128, [500, 1], 64, 4),       # two heads a CTA
    (2, 3, 3, 128, [700, 0], 65, 70),      # two query tiles a CTA, an empty sequence
    (1, 3, 1, 128, [1100], 129, 1),
    (1, 4, 1, 128, [1100], 300, 0),
    (1, 2, 1, 128, [400], 5000, 2),        # a window longer than the prompt
    (1, 2, 1, 128, [400], 33, 5000),       # sinks longer than the prompt
    (1, 1, 1, 64, [1500], 128, 200),
])
def test_prompt_window(b, hq, h, d, T, window, sinks):
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    rng = np.random.default_rng(sum(T) + window)
    t = max(T)
    Kh, Vh = _inputs(rng, b, h, t, d, None)
    Vh[:, :, ::7] += 16   # uneven, so that a token seen by mistake shows
    Q = rng.standard_normal((b, hq, t, d)).astype(np.float16)
    c = K.KiviCache(b, h, d, 2, 4, 32, 64, t + 8)
    w = K.KiviCache(b, h, d, 2, 4, 32, 64, t + 8)
    Qt, Kt, Vt = (torch.from_numpy(x).cuda() for x in (Q, Kh, Vh))
    out = torch.full_like(Qt, 7.0)
    assert c.prefill_attn(Qt, Kt, Vt, T, out=out, window=window, sinks=sinks) is out
    w.prefill(Kt, Vt, T)
    a, e = c.export(), w.export()
    for name in a:   # the cache takes every token, as the plain prefill does
        assert np.array_equal(a[name], e[name]), name
    got = out.float().cpu().numpy()
    for i in range(b):
        assert np.all(got[i, :, T[i]:] == 7.0)
        for e_ in range(hq):
            if T[i] == 0:
                continue
            j = e_ // (hq // h)
            ref, wabs, mag = R.attend(Q[i, e_, :T[i]], Kh[i, j, :T[i]].astype(np.float64),
                                      Vh[i, j, :T[i]].astype(np.float64),
                                      R.visible(np.arange(T[i]), T[i], window, sinks))
            R.check_rounded(got[i, e_, :T[i]], ref, wabs, mag, T[i], f"sequence {i} head {e_}")
    assert c.check() == 0
    c.close()
    w.close()


@pytest.mark.gpu
def test_window_zero_is_everything_and_refusals():
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    c = K.KiviCache(1, 1, 64, 2, 2, 32, 32, 200)
    x = torch.randn(1, 1, 150, 64, device="cuda").half()
    c.prefill(x, x, 150)
    q = torch.randn(1, 2, 64, device="cuda").half()
    assert torch.equal(c.decode(q), c.decode(q, window=0, sinks=3))
    qq = torch.randn(1, 2, 150, 64, device="cuda").half()
    a = c.prefill_attn(qq, x, x, 150)
    assert torch.equal(a, c.prefill_attn(qq, x, x, 150, window=0, sinks=3))
    for kw in (dict(window=-1), dict(window=5, sinks=-1)):
        with pytest.raises(K.KiviError) as e:
            c.decode(q, **kw)
        assert e.value.status == 1
        with pytest.raises(K.KiviError):
            c.prefill_attn(qq, x, x, 150, **kw)
    assert c.lengths()[0].tolist() == [150]
    c.close()


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 70])
def test_other_stream_and_graph(window):
    """A prompt and a step on a stream of their own, their outputs made there
    too (the current stream is busy meanwhile), and captured and replayed."""
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    rng = np.random.default_rng(5)
    b, h, hq, d, ts, t = 2, 2, 4, 64, 150, [150, 90]
    c = K.KiviCache(b, h, d, 2, 2, 32, 64, 256)
    Q, Kp, Vp = (torch.from_numpy(rng.standard_normal((b, x, ts, d)).astype(np.float16)).cuda() for x in (hq, h, h))
    q = Q[:, :, 7].contiguous()
    want, step = c.prefill_attn(Q, Kp, Vp, t, window=window, sinks=3), c.decode(q, window=window, sinks=3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    got = c.prefill_attn(Q, Kp, Vp, t, stream=s, window=window, sinks=3)
    dec = c.decode(q, stream=s, window=window, sinks=3)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(dec, step)
    g = torch.cuda.CUDAGraph()
    got.zero_()
    with torch.cuda.graph(g):
        c.prefill_attn(Q, Kp, Vp, t, out=got, window=window, sinks=3)
        c.decode(q, out=dec, window=window, sinks=3)
    for _ in range(2):
        dec.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(dec, step)
    assert c.check() == 0
    c.close()
