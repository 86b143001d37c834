"""Latent attention with more heads than its absorbed form takes: prompts, pieces,
drafts and steps, all expanded."""
import pytest


@pytest.mark.gpu
@pytest.mark.parametrize("h,r", [(129, 512), (200, 256), (1024, 256)])
def test_many_heads(h, r):
    torch = pytest.importorskip("torch")
    from bit_quantized_kv_quantize_gb300 import kivi as K
    from tests import latent_ref as L
    b, R, scale = 2, 64, 192 ** -0.5
    g = torch.Generator(device="cuda").manual_seed(h)
    rand = lambda *s, by=1.0: (torch.randn(*s, generator=g, device="cuda") * by).half()   # noqa: E731
    wk, wv = rand(h, 128, r, by=r ** -0.5), rand(h, 128, r, by=r ** -0.5)
    cache = K.LatentCache(b, r, 4, 32, R, 400)
    seen, keys, T = [rand(0, r)] * b, [rand(0, 64)] * b, [0] * b
    for n in ([200, 77], [1, 1], [3, 0], [20, 2], [1, 1]):
        ns = max(n)
        c, kr, qn, qr = rand(b, ns, r), rand(b, ns, 64), rand(b, h, ns, 128), rand(b, h, ns, 64)
        if T == [0, 0]:
            out = cache.prefill_attn(qn, qr, c, kr, n, wk, wv)
        else:
            out = cache.extend(qn, qr, c, kr, n, wk, wv)
        for i in range(b):
            if n[i] == 0:
                continue
            cs = torch.cat((L.cached(seen[i], T[i], R, 4, 32), c[i, :n[i]].double()))
            ks = torch.cat((keys[i], kr[i, :n[i]]))
            heads = (0, 1, 64, 127, 128, h - 1)
            full = [L.latent(qn[i, e, :n[i]], qr[i, e, :n[i]], cs, ks, wk[e], wv[e], T[i], scale, False, T[i] > 0) for e in heads]
            L.check(out[i, heads, :n[i]], torch.stack([x for x, _ in full]), torch.stack([x for _, x in full]), f"{n} {i}")
            seen[i], keys[i], T[i] = torch.cat((seen[i], c[i, :n[i]])), ks, T[i] + n[i]
    assert list(cache.lengths()[0]) == T and cache.check() == 0 and K.device_check() == 0
    with pytest.raises(K.KiviError):                  # asked for: refused
        cache.attn(qn, qr, c, kr, 1, wk, wv, form="absorbed")
    cache.close()
