"""Appends to the latent cache that are longer than its ring of fp16 tokens: what
leaves the window is quantized from its own values."""
import pytest


@pytest.mark.gpu
@pytest.mark.parametrize("r,bits,G,R,T,n", [
    (512, 4, 32, 64, 100, 300), (256, 2, 64, 64, 100, 300), (512, 4, 32, 128, 2000, 300), (256, 4, 128, 128, 7, 500),
    (512, 2, 32, 192, 257, 900), (256, 4, 32, 256, 1000, 1300), (512, 4, 64, 128, 1, 257),
])
def test_chunks_longer_than_the_ring(r, bits, G, R, T, n):
    """Every sequence at lengths of its own around T and n, several times over."""
    torch = pytest.importorskip("torch")
    from bit_quantized_kv_quantize_gb300 import kivi as K
    from tests import latent_ref as L
    b = 24
    g = torch.Generator(device="cuda").manual_seed(T + n)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").half()   # noqa: E731
    t, m = [T + 5 * i for i in range(b)], [n + 11 * (i % 9) - 3 * (i % 4) for i in range(b)]
    t[0], m[0] = T, n
    c, kr, c1, kr1 = rand(b, max(t), r), rand(b, max(t), 64), rand(b, max(m), r), rand(b, max(m), 64)
    want = [L.half(L.cached(torch.cat((c[i, :t[i]], c1[i, :m[i]])), t[i] + m[i], R, bits, G)) for i in range(b)]
    cache = K.LatentCache(b, r, bits, G, R, max_tokens=max(t) + max(m))
    for _ in range(4):
        cache.prefill(c, kr, t)
        cache.append(c1, kr1, m)
        gc, gk = cache.restore()
        for i in range(b):
            assert torch.equal(gc[i, :t[i] + m[i]], want[i]), i
            assert torch.equal(gk[i, :t[i] + m[i]], torch.cat((kr[i, :t[i]], kr1[i, :m[i]]))), i
    assert cache.check() == 0
    cache.close()
