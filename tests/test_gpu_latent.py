"""The latent cache and latent attention (kivi_latent_*, kivi_head_product;
kivi.LatentCache, latent_prompt_attn, head_product) against 64-bit references,
and their refusals."""
import ctypes

import numpy as np
import pytest

SCALE = 192 ** -0.5


def _K():
    from bit_quantized_kv_quantize_gb300 import kivi as K
    return K


def _L():
    from tests import latent_ref as L
    return L


# ---- refusals (no GPU) ---------------------------------------------------------

@pytest.mark.parametrize("args,code", [
    ((0, 512, 4, 32, 128, 100), 1), ((1, 0, 4, 32, 128, 100), 1), ((1, 512, 4, 0, 128, 100), 1),
    ((1, 512, 4, 32, 0, 100), 1), ((1, 512, 4, 32, 128, 0), 1),
    ((1025, 512, 4, 32, 128, 100), 2), ((1, 384, 4, 32, 128, 100), 2), ((1, 512, 8, 32, 128, 100), 2),
    ((1, 512, 4, 16, 128, 100), 2), ((1, 512, 4, 256, 128, 100), 2), ((1, 512, 4, 32, 100, 100), 2),
    ((1, 512, 4, 32, 128, 2 ** 30 + 1), 2),
])
def test_create_refuses(args, code):
    K = _K()
    h = ctypes.c_void_p()
    assert K.lib.kivi_latent_create(*args, ctypes.byref(h)) == code and not h.value
    assert K.lib.kivi_last_error()


def test_handles_and_calls_without_one_refuse():
    K = _K()
    p, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4104)   # never dereferenced: every call below is refused
    n = np.array([1], np.int32)
    vp = ctypes.c_void_p
    bogus = ctypes.cast(ctypes.create_string_buffer(64), vp)
    for h in (None, bogus):
        assert K.lib.kivi_latent_destroy(h) == 1
        assert K.lib.kivi_latent_prefill(h, p, p, n.ctypes.data, 1, None) == 1
        assert K.lib.kivi_latent_append(h, p, p, n.ctypes.data, 1, None) == 1
        assert K.lib.kivi_latent_attn(h, p, p, p, p, n.ctypes.data, 1, 1, 1.0, p, None) == 1
        assert K.lib.kivi_latent_lengths(h, None, None) == 1
        assert K.lib.kivi_latent_restore(h, None, None, 0, None) == 1
        assert K.lib.kivi_latent_rows(h, p, p, n.ctypes.data, 1, p, p, 1, None) == 1

    def product(x=p, w=p, b=1, hx=1, h=4, ns=1, n=n, k=128, nn=128, out=p):
        return K.lib.kivi_head_product(x, w, b, hx, h, ns, None if n is None else n.ctypes.data, k, nn, 0, out, None)

    assert product(b=0) == 1 and product(h=0) == 1 and product(hx=2) == 1 and product(ns=-1) == 1 and product(n=None) == 1
    assert product(n=np.array([2], np.int32)) == 1 and product(n=np.array([-1], np.int32)) == 1
    assert product(x=None) == 1 and product(w=odd) == 1 and product(out=odd) == 1
    assert product(b=1025) == 2 and product(k=96) == 2 and product(nn=192) == 2 and product(h=1025) == 2 and product(k=16448) == 2

    def prompt(q=p, v=p, b=1, h=1, t=n, ts=1, scale=1.0, out=p):
        return K.lib.kivi_latent_prompt_attn(q, p, p, p, v, b, h, None if t is None else t.ctypes.data, ts, scale, out, None)

    assert prompt(b=0) == 1 and prompt(h=0) == 1 and prompt(t=None) == 1 and prompt(ts=-1) == 1 and prompt(q=None) == 1
    assert prompt(scale=0.0) == 1 and prompt(scale=float("nan")) == 1 and prompt(scale=float("inf")) == 1
    assert prompt(v=odd) == 1 and prompt(t=np.array([2], np.int32)) == 1
    T = np.array([0], np.int32)

    def expanded(T=T, n=n, ns=1, ss=1):
        a = lambda x: None if x is None else x.ctypes.data   # noqa: E731
        return K.lib.kivi_latent_expanded_attn(p, p, p, p, odd, 1, 1, a(T), a(n), ns, ss, 1.0, p, None)

    assert expanded(T=None) == 1 and expanded(n=None) == 1 and expanded(ss=0) == 1 and expanded(T=np.array([-1], np.int32)) == 1
    assert expanded(T=np.array([1], np.int32)) == 1 and expanded(ss=2 ** 26 + 1) == 2 and expanded() == 1
    assert prompt(b=1025) == 2 and prompt(ts=2 ** 26 + 1) == 2 and prompt(h=1025) == 2 and prompt(h=1024, ts=2 ** 21) == 2


# ---- inputs ----------------------------------------------------------------------

class _Made:
    """Random tokens, queries and weights."""

    def __init__(self, seed, b, h, r):
        import torch
        self.torch, self.b, self.h, self.r = torch, b, h, r
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.wk, self.wv = (self.rand(h, 128, r, by=r ** -0.5) for _ in range(2))

    def rand(self, *shape, by=1.0):
        return (self.torch.randn(*shape, generator=self.g, device="cuda") * by).half()

    def tokens(self, n):
        c = self.rand(self.b, n, self.r)
        c[:, :, 5] *= 6.0                         # a large channel
        if n > 2:
            c[:, 1] = 0.25                        # a group of equal values: scale 0
        return c, self.rand(self.b, n, 64)

    def queries(self, n):
        return self.rand(self.b, self.h, n, 128), self.rand(self.b, self.h, n, 64)


# ---- the cache ---------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("r", [256, 512])
@pytest.mark.parametrize("bits,G,R", [(4, 32, 64), (4, 64, 128), (4, 128, 192), (2, 32, 128), (2, 64, 64), (2, 128, 1024)])
def test_cache_holds_its_tokens(r, bits, G, R):
    """Restored rows, whatever calls brought the tokens: prefill, chunks longer and
    shorter than the window, single tokens, a sequence left out."""
    torch = pytest.importorskip("torch")
    K, L = _K(), _L()
    m = _Made(r + bits + R, 3, 1, r)
    cache = K.LatentCache(3, r, bits, G, R, max_tokens=1200)
    T, rows, keys = [0, 0, 0], [[], [], []], [[], [], []]
    assert [int(x.max()) for x in cache.lengths()] == [0, 0]
    first = True
    for n in ([300, 0, 65], [1, 1, 0], [200, 5, 64], [1, 1, 1], [0, 500, 130], [3, 64, 1], [64, 63, 63]):
        c, kr = m.tokens(max(n))
        (cache.prefill if first else cache.append)(c, kr, n)
        first = False
        for i in range(3):
            rows[i].append(c[i, :n[i]])
            keys[i].append(kr[i, :n[i]])
            T[i] += n[i]
        gt, gq = cache.lengths()
        assert list(gt) == T and list(gq) == [max(0, t - R) for t in T]
        gc, gk = cache.restore()
        for i in range(3):
            c_all = torch.cat(rows[i])
            ref = L.cached(c_all, T[i], R, bits, G)
            # scale code + zero in one rounding
            assert torch.equal(gc[i, :T[i]], L.half(ref))
            assert torch.equal(gk[i, :T[i]], torch.cat(keys[i]))
            assert not gc[i, T[i]:].any()
    with pytest.raises(K.CapacityError):
        cache.append(*m.tokens(900), [900, 0, 0])
    assert list(cache.lengths()[0]) == T and cache.check() == 0
    c, kr = m.tokens(70)
    cache.prefill(c, kr, 70)                      # anew
    assert torch.equal(cache.restore()[0][2], L.half(L.cached(c[2], 70, R, bits, G)))
    cache.close()


# ---- products ------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("b,h,n,K_,N,transposed,shared", [
    (1, 1, 1, 128, 512, True, False), (64, 3, 1, 128, 256, True, False), (3, 2, 130, 512, 128, False, False),
    (2, 5, 301, 512, 128, False, True), (1, 2, 128, 64, 128, False, False), (2, 1, 77, 192, 384, True, True),
    (5, 128, 2, 256, 128, False, False),
    # rows of all heads alike over several heads a CTA: an odd number of heads, two column tiles, ragged ends
    (3, 61, 260, 512, 128, False, True), (1, 7, 5000, 192, 256, False, True), (1, 200, 127, 64, 128, False, True),
    # ... in tiles of two column tiles, of which the last has one
    (1, 24, 5000, 512, 128, False, True), (2, 23, 4999, 320, 128, False, True), (1, 8, 5000, 64, 384, False, True),
])
def test_head_product(b, h, n, K_, N, transposed, shared):
    torch = pytest.importorskip("torch")
    K = _K()
    g = torch.Generator(device="cuda").manual_seed(n + K_)
    x = torch.randn((b, n, K_) if shared else (b, h, n, K_), generator=g, device="cuda").half()
    w = torch.randn((h, K_, N) if transposed else (h, N, K_), generator=g, device="cuda").half()
    cnt = [n] + [(7 * i) % (n + 1) for i in range(1, b)]
    out = torch.full((b, h, n, N), 7.0, dtype=torch.float16, device="cuda")
    K.head_product(x, w, cnt, transposed, out)
    xd = (x.unsqueeze(1) if shared else x).double()
    wd = w.double() if transposed else w.double().transpose(1, 2)
    ref, size = xd @ wd, xd.abs() @ wd.abs()
    for i in range(b):
        # one rounding, and K terms in fp32
        bound = ref[i, :, :cnt[i]].abs() * 2.0 ** -11 + 2.0 ** -25 + size[i, :, :cnt[i]] * K_ * 2.0 ** -23
        assert bool(((out[i, :, :cnt[i]].double() - ref[i, :, :cnt[i]]).abs() <= bound).all()), i
        assert bool((out[i, :, cnt[i]:] == 7.0).all())
    assert K.device_check() == 0


# ---- attention over the cache ---------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("b,h,r,bits,G,R,t,n", [
    (1, 1, 512, 4, 32, 64, [0], [1]),                 # nothing cached, one token
    (1, 16, 512, 4, 32, 64, [1], [1]),
    (2, 16, 256, 4, 64, 64, [63, 64], [1, 1]),
    (3, 16, 512, 4, 32, 128, [300, 0, 129], [1, 1, 0]),
    (2, 128, 512, 4, 128, 128, [257, 1000], [1, 1]),  # two row tiles a sequence
    (2, 5, 512, 2, 32, 64, [200, 500], [13, 4]),      # rows that do not fill a tile, an odd number of heads
    (2, 12, 256, 2, 64, 192, [700, 190], [40, 33]),
    (1, 3, 256, 4, 32, 1024, [900], [150]),           # fp16 tiles, whole tiles of new tokens
    (2, 8, 512, 4, 64, 64, [0, 100], [200, 3]),
    (3, 2, 256, 4, 32, 128, [61, 700, 0], [300, 0, 129]),   # several row tiles behind cached tokens that end inside a tile
    (1, 2, 512, 2, 64, 64, [127], [257]),
    (1, 64, 256, 2, 128, 64, [5000], [2]),            # cut into shares
    (4, 16, 512, 4, 32, 128, [4000, 3, 2500, 64], [1, 1, 1, 1]),
    (1, 1, 512, 2, 128, 64, [3000], [5]),
    (40, 7, 256, 4, 32, 64, None, None),
])
def test_attention_over_the_cache(b, h, r, bits, G, R, t, n):
    torch = pytest.importorskip("torch")
    K, L = _K(), _L()
    m = _Made(r + h + R, b, h, r)
    if t is None:
        t, n = [(37 * i) % 600 for i in range(b)], [i % 4 for i in range(b)]
    ts, ns = max(max(t), 1), max(n)
    cache = K.LatentCache(b, r, bits, G, R, max_tokens=ts)
    c, kr = m.tokens(ts)
    cache.prefill(c, kr, t)
    c1, kr1 = m.tokens(ns)
    qn, qr = m.queries(ns)
    ql = m.rand(b, h, ns, r, by=0.7)
    for i in range(b):                                # rows behind a sequence hold anything
        c1[i, n[i]:], kr1[i, n[i]:], qn[i, :, n[i]:], ql[i, :, n[i]:] = float("nan"), float("inf"), float("nan"), float("nan")
    lat = torch.full((b, h, ns, r), 7.0, dtype=torch.float16, device="cuda")
    cache.attn_latent(ql, qr, c1, kr1, n, out=lat)
    again = cache.attn_latent(ql, qr, c1, kr1, n, out=torch.full_like(lat, 7.0))
    out = torch.full((b, h, ns, 128), 7.0, dtype=torch.float16, device="cuda")
    cache.attn(qn, qr, c1, kr1, n, m.wk, m.wv, out=out, form="absorbed")
    exp = cache.attn(qn, qr, c1, kr1, n, m.wk, m.wv, out=torch.full_like(out, 7.0), form="expanded")
    pick = cache.attn(qn, qr, c1, kr1, n, m.wk, m.wv, out=torch.full_like(out, 7.0))
    assert cache.check() == 0 and K.device_check() == 0
    assert torch.equal(lat, again) and (torch.equal(pick, out) or torch.equal(pick, exp))
    for i in range(b):
        assert all(bool((x[i, :, n[i]:] == 7.0).all()) for x in (lat, out, exp))
        if n[i] == 0:
            continue
        cs = torch.cat((L.cached(c[i], t[i], R, bits, G), c1[i, :n[i]].double()))
        ks = torch.cat((kr[i, :t[i]], kr1[i, :n[i]])).double()
        got, ref, err = [], [], []
        for e in range(h):
            o, wabs, mag = L.attend(torch.cat((ql[i, e, :n[i]], qr[i, e, :n[i]]), 1), torch.cat((cs, ks), 1), cs, t[i], SCALE)
            got.append(lat[i, e, :n[i]])
            ref.append(o)
            err.append(L.attn_bound(wabs, mag, cs.shape[0], r + 64))
        L.check(torch.stack(got), torch.stack(ref), torch.stack(err), f"latent {i}")
        full = [L.latent(qn[i, e, :n[i]], qr[i, e, :n[i]], cs, ks, m.wk[e], m.wv[e], t[i], SCALE, True) for e in range(h)]
        L.check(out[i, :, :n[i]], torch.stack([x for x, _ in full]), torch.stack([x for _, x in full]), f"out {i}")
        full = [L.latent(qn[i, e, :n[i]], qr[i, e, :n[i]], cs, ks, m.wk[e], m.wv[e], t[i], SCALE, False, True) for e in range(h)]
        L.check(exp[i, :, :n[i]], torch.stack([x for x, _ in full]), torch.stack([x for _, x in full]), f"expanded {i}")
    cache.close()


@pytest.mark.gpu
@pytest.mark.parametrize("r", [256, 512])
def test_growing_scores_and_a_sink(r):
    """Scores that rise by far more than 2^8 from tile to tile, so that the
    references are raised again and again, some rows only; and one token that
    takes all of the weight."""
    torch = pytest.importorskip("torch")
    K, L = _K(), _L()
    b, h, t, n = 1, 40, 600, 2
    m = _Made(11, b, h, r)
    cache = K.LatentCache(b, r, 4, 32, 64, max_tokens=t)
    c, kr = m.tokens(t)
    kr[0, :, 0] = torch.linspace(-60, 60, t, device="cuda").half()
    kr[0, 17, 1] = 100.0
    cache.prefill(c, kr, t)
    c1, kr1 = m.tokens(n)
    ql, qr = m.rand(b, h, n, r, by=0.2), m.rand(b, h, n, 64, by=0.2)
    qr[0, :, :, 0] = torch.linspace(-8, 8, h, device="cuda").half().view(h, 1)
    qr[0, 3, :, 1], qr[0, 5, :, 1] = 20.0, -20.0
    out = cache.attn_latent(ql, qr, c1, kr1, n)
    cs = torch.cat((L.cached(c[0], t, 64, 4, 32), c1[0].double()))
    ks = torch.cat((kr[0], kr1[0])).double()
    for e in range(h):
        o, wabs, mag = L.attend(torch.cat((ql[0, e], qr[0, e]), 1), torch.cat((cs, ks), 1), cs, t, SCALE)
        # (the rotary part of a key is exact: the bound's roundings are of the rest, and fp32 sums of all)
        part = SCALE * (ql[0, e].double().abs() @ cs.abs().t()).amax(1)
        err = L.attn_bound(wabs, part + mag * (r + 64) * 2.0 ** -12, cs.shape[0], r + 64)
        L.check(out[0, e], o, err, f"head {e}")
    assert cache.check() == 0


# ---- prompts -----------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("b,h,r,t", [
    (1, 1, 512, [1]), (1, 2, 256, [63]), (1, 3, 512, [64]), (2, 2, 256, [65, 0]), (1, 2, 512, [128]), (3, 2, 256, [129, 1, 255]),
    (2, 1, 512, [256, 257]), (1, 4, 512, [700]), (3, 5, 256, [513, 300, 1000]),
])
def test_prompt(b, h, r, t):
    torch = pytest.importorskip("torch")
    K, L = _K(), _L()
    m = _Made(r + sum(t), b, h, r)
    ts = max(t)
    c, kr = m.tokens(ts)
    qn, qr = m.queries(ts)
    for i in range(b):                                # rows behind a sequence hold anything
        c[i, t[i]:], kr[i, t[i]:], qn[i, :, t[i]:] = float("nan"), float("inf"), float("nan")
    out = torch.full((b, h, ts, 128), 7.0, dtype=torch.float16, device="cuda")
    K.latent_prompt_attn(qn, qr, c, kr, t, m.wk, m.wv, out=out)
    assert K.device_check() == 0
    cache = K.LatentCache(b, r, 4, 32, 64, max_tokens=ts)
    again = cache.prefill_attn(qn, qr, c, kr, t, m.wk, m.wv, out=torch.full_like(out, 7.0))
    assert torch.equal(out, again) and list(cache.lengths()[0]) == t
    for i in range(b):
        assert bool((out[i, :, t[i]:] == 7.0).all())
        if t[i] == 0:
            continue
        full = [L.latent(qn[i, e, :t[i]], qr[i, e, :t[i]], c[i, :t[i]], kr[i, :t[i]], m.wk[e], m.wv[e], 0, SCALE, False)
                for e in range(h)]
        L.check(out[i, :, :t[i]], torch.stack([x for x, _ in full]), torch.stack([x for _, x in full]), f"prompt {i}")


@pytest.mark.gpu
def test_prompt_growing_scores_and_dead_values():
    """Rising scores (raises and rescalings in every tile), and inputs behind the
    sequences and in its last tile that must not reach the output."""
    torch = pytest.importorskip("torch")
    K, L = _K(), _L()
    b, h, t = 2, 2, [390, 201]
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(b, h, 400, 128, generator=g, device="cuda").half() for _ in range(3))
    qr, kr = torch.randn(b, h, 400, 64, generator=g, device="cuda").half(), torch.randn(b, 400, 64, generator=g, device="cuda").half()
    kr[:, :, 0] = torch.linspace(-100, 100, 400, device="cuda").half()
    qr[:, :, :, 0] = 9.0
    qr[:, :, ::3, 0] = -9.0
    for i in range(b):
        for x in (q, k, v, qr):
            x[i, :, t[i]:] = float("nan")
        kr[i, t[i]:] = float("nan")
    out = torch.zeros_like(q)
    n = np.array(t, np.int32)
    st = torch.cuda.current_stream().cuda_stream
    assert K.lib.kivi_latent_prompt_attn(q.data_ptr(), qr.data_ptr(), k.data_ptr(), kr.data_ptr(), v.data_ptr(), b, h,
                                         n.ctypes.data, 400, SCALE, out.data_ptr(), st) == 0
    assert K.device_check() == 0
    for i in range(b):
        for e in range(h):
            o, wabs, mag = L.attend(torch.cat((q, qr), 3)[i, e, :t[i]], torch.cat((k[i, e], kr[i]), 1)[:t[i]], v[i, e, :t[i]], 0, SCALE)
            err = L.attn_bound(wabs, mag, t[i], 192, scores=0.0, values=0.0)   # (every input is fp16 as it is)
            L.check(out[i, e, :t[i]], o, err, f"{i} {e}")
        assert not out[i, :, t[i]:].any()


# ---- together ------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("b,h,r,t,n", [
    (1, 1, 256, [4100], [300]),             # two row tiles, eight shares each
    (2, 3, 512, [5000, 0], [130, 700]),     # shares without tiles; rows that see nothing of a share
    (3, 7, 256, [1500, 900, 1100], [1, 0, 257]),
    (1, 20, 512, [2600], [17]),
])
def test_row_tiles_that_ctas_share(b, h, r, t, n):
    """The expanded form of few row tiles over many tokens, in shares that are
    joined; scores that rise along the tokens for some rows and fall for others.
    (The joined factors' roundings, 2^-22 relative a share, are within the bound's
    S 2^-24.)"""
    torch = pytest.importorskip("torch")
    K, L = _K(), _L()
    m = _Made(47, b, h, r)
    bits, G, R, ns = 4, 32, 64, max(n)
    cache = K.LatentCache(b, r, bits, G, R, max_tokens=max(t))
    c, kr = m.tokens(max(t))
    kr[:, :, 0] = torch.linspace(-8, 8, max(t), device="cuda").half()
    cache.prefill(c, kr, t)
    c1, kr1 = m.tokens(ns)
    qn, qr = m.queries(ns)
    qr[:, :, :, 0] = torch.linspace(-12, 12, ns, device="cuda").half()
    out = cache.attn(qn, qr, c1, kr1, n, m.wk, m.wv, out=torch.full_like(qn, 7.0), form="expanded")
    again = cache.attn(qn, qr, c1, kr1, n, m.wk, m.wv, out=torch.full_like(qn, 7.0), form="expanded")
    assert cache.check() == 0 and K.device_check() == 0 and torch.equal(out, again)
    for i in range(b):
        assert bool((out[i, :, n[i]:] == 7.0).all())
        if n[i] == 0:
            continue
        cs = torch.cat((L.cached(c[i], t[i], R, bits, G), c1[i, :n[i]].double()))
        ks = torch.cat((kr[i, :t[i]], kr1[i, :n[i]])).double()
        full = [L.latent(qn[i, e, :n[i]], qr[i, e, :n[i]], cs, ks, m.wk[e], m.wv[e], t[i], SCALE, False, True) for e in range(h)]
        L.check(out[i, :, :n[i]], torch.stack([x for x, _ in full]), torch.stack([x for _, x in full]), f"{i}")
    cache.close()
    # a prompt alone
    t = [x + y for x, y in zip(t, n)]
    c, kr = m.tokens(max(t))
    qn, qr = m.queries(max(t))
    out = K.latent_prompt_attn(qn, qr, c, kr, t, m.wk, m.wv, out=torch.full_like(qn, 7.0))
    assert K.device_check() == 0
    i = t.index(max(t))
    first = t[i] - 300
    for e in (0, h - 1):
        o, w = L.latent(qn[i, e, first:t[i]], qr[i, e, first:t[i]], c[i, :t[i]], kr[i, :t[i]], m.wk[e], m.wv[e], first, SCALE, False)
        L.check(out[i, e, first:t[i]], o, w, f"prompt {e}")


def _outputs(torch, m, cache, qn, qr, c, kr, c1, kr1, t, n, R, bits, G, rows):
    """Both forms against the reference: the given (sequence, head) pairs."""
    K, L = _K(), _L()
    for form in ("absorbed", "expanded"):
        out = cache.attn(qn, qr, c1, kr1, n, m.wk, m.wv, out=torch.full_like(qn, 7.0), form=form)
        assert cache.check() == 0 and K.device_check() == 0
        assert all(bool((out[i, :, k:] == 7.0).all()) for i, k in enumerate(n) if k < out.shape[2])
        for i, e in rows:
            cs = torch.cat((L.cached(c[i, :t[i]], t[i], R, bits, G), c1[i, :n[i]].double()))
            ks = torch.cat((kr[i, :t[i]], kr1[i, :n[i]])).double()
            o, w = L.latent(qn[i, e, :n[i]], qr[i, e, :n[i]], cs, ks, m.wk[e], m.wv[e], t[i], SCALE, form == "absorbed",
                            form == "expanded")
            L.check(out[i, e, :n[i]], o, w, f"{form} {i} {e}")


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A cache of 5 GB of records, most of it empty, and its last sequences; keys
    and values of more than 4 GB."""
    torch = pytest.importorskip("torch")
    K = _K()
    b, h, r, R = 1024, 2, 512, 64
    m = _Made(3, b, h, r)
    cache = K.LatentCache(b, r, 4, 32, R, max_tokens=16384)
    t, n = [0] * b, [0] * b
    t[1000], t[1023], n[1000], n[1022], n[1023] = 129, 300, 1, 2, 3
    c, kr = m.tokens(300)
    cache.prefill(c, kr, t)
    c1, kr1 = m.tokens(3)
    _outputs(torch, m, cache, *m.queries(3), c, kr, c1, kr1, t, n, R, 4, 32, [(1000, 1), (1022, 0), (1023, 0), (1023, 1)])
    cache.close()
    del cache, c, kr
    b, h, t, n = 1, 128, [140000], [2]
    m = _Made(4, b, h, r)
    cache = K.LatentCache(b, r, 4, 32, R, max_tokens=t[0])
    c, kr = m.tokens(t[0])
    cache.prefill(c, kr, t)
    c1, kr1 = m.tokens(2)
    _outputs(torch, m, cache, *m.queries(2), c, kr, c1, kr1, t, n, R, 4, 32, [(0, 0), (0, 127)])
    cache.close()


@pytest.mark.gpu
@pytest.mark.parametrize("r,bits,G,R,axes", [(512, 4, 32, 64, False), (256, 2, 64, 128, True)])
def test_a_prompt_pieces_drafts_and_steps(r, bits, G, R, axes):
    """As a program serves: a rotated prompt, a piece, a draft that is verified and
    kept in part, single tokens; the cache against the tokens that it was given."""
    torch = pytest.importorskip("torch")
    K, L = _K(), _L()
    b, h = 2, 6
    m = _Made(5, b, h, r)
    cache = K.LatentCache(b, r, bits, G, R, max_tokens=500)
    rope = K.Rope(64, axes=K.rope_axes([10, 11, 11]) if axes else None)
    seen, keys, T = [torch.zeros(0, r).half().cuda()] * b, [torch.zeros(0, 64).half().cuda()] * b, [0, 0]
    for n, what in (([210, 77], "prompt"), ([50, 64], "piece"), ([4, 3], "draft"), ([1, 1], "step"), ([1, 1], "step")):
        ns = max(n)
        c, kr = m.tokens(ns)
        qn, qr = m.queries(ns)
        pos = torch.stack([torch.tensor(T).view(b, 1) + torch.arange(ns)] * 3).int().cuda()
        pos[1:] //= 7
        at = pos if axes else T
        qrot, krot = rope.apply(qr, kr.unsqueeze(1), at)
        krot = krot.squeeze(1)
        keep = n
        if what == "prompt":
            out = cache.prefill_attn(qn, qrot, c, krot, n, m.wk, m.wv)
        elif what == "draft":
            out = cache.attn(qn, qrot, c, krot, n, m.wk, m.wv)
            p = torch.softmax(torch.randn(b, ns + 1, 100, generator=m.g, device="cuda"), 2)
            q = torch.softmax(torch.randn(b, ns, 100, generator=m.g, device="cuda"), 2)
            draft = q.argmax(2).int()
            u = torch.rand(b, ns + 1, generator=m.g, device="cuda")
            tokens, acc = K.verify(p, q, draft, u, n)
            for i in range(b):
                ref, a = L.verify(p[i].cpu().numpy(), q[i].cpu().numpy(), draft[i].cpu().numpy(), u[i].cpu().numpy(), n[i])
                assert a == int(acc[i]) and np.array_equal(ref, tokens[i].cpu().numpy())
            keep = acc.tolist()
            cache.append(c, krot, keep)
        else:
            out = cache.extend(qn, qr, c, kr, n, m.wk, m.wv, rope=rope, pos=pos if axes else None)
        for i in range(b):
            cs = torch.cat((L.cached(seen[i], T[i], R, bits, G), c[i, :n[i]].double()))
            ks = torch.cat((keys[i], krot[i, :n[i]]))
            absorbed = what in ("draft", "step")          # (the piece expands: 16 queries and more over a short cache)
            full = [L.latent(qn[i, e, :n[i]], qrot[i, e, :n[i]], cs, ks, m.wk[e], m.wv[e], T[i], SCALE, absorbed, what == "piece")
                    for e in range(h)]
            L.check(out[i, :, :n[i]], torch.stack([x for x, _ in full]), torch.stack([x for _, x in full]), f"{what} {i}")
            seen[i], keys[i] = torch.cat((seen[i], c[i, :keep[i]])), torch.cat((keys[i], krot[i, :keep[i]]))
            T[i] += keep[i]
        assert list(cache.lengths()[0]) == T
    gc, gk = cache.restore()
    for i in range(b):
        assert torch.equal(gc[i, :T[i]], L.half(L.cached(seen[i], T[i], R, bits, G))) and torch.equal(gk[i, :T[i]], keys[i])
    assert cache.check() == 0 and K.device_check() == 0


@pytest.mark.gpu
def test_streams_and_graphs():
    """The whole of attn on another stream and captured (its first split call's
    buffer included), replayed with other contents."""
    torch = pytest.importorskip("torch")
    K = _K()
    b, h, r, t, n = 2, 16, 512, 2000, 2
    m = _Made(9, b, h, r)
    cache = K.LatentCache(b, r, max_tokens=t + 10)
    cache.prefill(*m.tokens(t), t)
    args = (*m.queries(n), *m.tokens(n))
    torch.cuda.synchronize()
    out = torch.zeros(b, h, n, 128, dtype=torch.float16, device="cuda")
    K.head_product(args[0], m.wk, transposed=True)   # (loads the kernels)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attn(*args, n, m.wk, m.wv, out=out)
        prompt = K.latent_prompt_attn(*args, n, m.wk, m.wv)
    for x, y in zip(args, (*m.queries(n), *m.tokens(n))):
        x.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    ref = cache.attn(*args, n, m.wk, m.wv, stream=st)
    refp = K.latent_prompt_attn(*args, n, m.wk, m.wv, stream=st)
    st.synchronize()
    assert torch.equal(out, ref) and torch.equal(prompt, refp) and cache.check() == 0


@pytest.mark.gpu
def test_shared_row_tiles_on_streams_and_in_graphs():
    """A chunk whose row tiles CTAs share, on another stream and captured twice,
    the graphs replayed in turn; and a step behind it in the same graph."""
    torch = pytest.importorskip("torch")
    K = _K()
    b, h, r, t, n = 1, 3, 256, 2100, 40
    m = _Made(9, b, h, r)
    cache = K.LatentCache(b, r, 4, 32, 64, max_tokens=t)
    c, kr = m.tokens(t)
    cache.prefill(c, kr, t)
    c1, kr1 = m.tokens(n)
    qn, qr = m.queries(n)
    want = [cache.attn(qn, qr, c1, kr1, k, m.wk, m.wv, out=torch.full_like(qn, 7.0)) for k in (n, 1)]
    st, outs, graphs = torch.cuda.Stream(), [], []
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        o = [torch.full_like(qn, 7.0) for _ in want]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for k, x in zip((n, 1), o):
                cache.attn(qn, qr, c1, kr1, k, m.wk, m.wv, out=x)
        outs.append(o)
        graphs.append(g)
    for g in graphs + graphs:
        g.replay()
    side = torch.full_like(qn, 7.0)
    st.wait_stream(torch.cuda.current_stream())
    cache.attn(qn, qr, c1, kr1, n, m.wk, m.wv, out=side, stream=st)
    torch.cuda.synchronize()
    assert cache.check() == 0 and K.device_check() == 0
    assert all(torch.equal(x, y) for o in outs for x, y in zip(o, want)) and torch.equal(side, want[0])
    cache.close()


@pytest.mark.gpu
def test_binding_refuses():
    torch = pytest.importorskip("torch")
    K = _K()
    m = _Made(1, 2, 4, 256)
    cache = K.LatentCache(2, 256, max_tokens=64)
    (qn, qr), (c, kr) = m.queries(3), m.tokens(3)
    for bad in ((qn.float(), qr, c, kr), (qn, qr.cpu(), c, kr)):
        with pytest.raises(TypeError):
            cache.attn(*bad, 3, m.wk, m.wv)
    for bad in ((qn, qr[:, :2], c, kr), (qn, qr, c[:, :2], kr), (qn.transpose(1, 2), qr, c, kr), (qn, qr, c, kr[:1])):
        with pytest.raises(ValueError):
            cache.attn(*bad, 3, m.wk, m.wv)
    with pytest.raises(ValueError):
        cache.attn(qn, qr, c, kr, 3, m.wk[:2], m.wv)
    with pytest.raises(ValueError):
        cache.extend(qn, qr, c, kr, 3, m.wk, m.wv, rope=K.Rope(128))
    with pytest.raises(K.KiviError):
        cache.attn(qn, qr, c, kr, 4, m.wk, m.wv)
    for form in ("absorbed", "expanded"):
        with pytest.raises(K.KiviError):
            cache.attn(qn, qr, c, kr, 4, m.wk, m.wv, form=form)
        with pytest.raises(K.KiviError):
            cache.attn(qn, qr, c, kr, -1, m.wk, m.wv, form=form)
    with pytest.raises(ValueError):
        cache.attn(qn, qr, c, kr, 3, m.wk, m.wv, form="other")
    with pytest.raises(K.KiviError):
        cache.attn(qn, qr, c, kr, 3, m.wk, m.wv, scale=-1.0)
    cache.prefill(c, kr, 3)
    with pytest.raises(K.KiviError):                  # refused before the cache changes
        cache.prefill_attn(qn, qr, c, kr, 2, m.wk, m.wv, scale=0.0)
    with pytest.raises(K.CapacityError):
        cache.prefill_attn(*m.queries(65), *m.tokens(65), 65, m.wk, m.wv)
    assert list(cache.lengths()[0]) == [3, 3]
    big = m.tokens(62)
    with pytest.raises(K.CapacityError):
        cache.extend(*m.queries(62), *big, 62, m.wk, m.wv)
    with pytest.raises(K.KiviError):
        K.head_product(qn, m.rand(4, 96, 128))
    assert list(cache.lengths()[0]) == [3, 3]
    cache.close()
    with pytest.raises(K.KiviError):
        cache.append(c, kr, 1)
