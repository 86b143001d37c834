"""A latent cache that is filled anew after tokens that were not finite: nothing of
them is left in the blocks that the new tokens do not fill."""
import pytest


@pytest.mark.gpu
@pytest.mark.parametrize("r,bits,R", [(512, 4, 64), (256, 2, 128), (256, 4, 192), (512, 4, 1024)])
def test_filled_anew(r, bits, R):
    """As a cache that held nothing before, bit for bit: after the fill, and while
    tokens are appended one by one and by chunks into block after block."""
    torch = pytest.importorskip("torch")
    from bit_quantized_kv_quantize_gb300 import kivi as K
    b, h, most = 3, 5, 900
    g = torch.Generator(device="cuda").manual_seed(r + R)
    rand = lambda *s, by=1.0: (torch.randn(*s, generator=g, device="cuda") * by).half()   # noqa: E731
    wk, wv = rand(h, 128, r, by=r ** -0.5), rand(h, 128, r, by=r ** -0.5)
    used, new = (K.LatentCache(b, r, bits, 32, R, most) for _ in range(2))
    bad = torch.full((b, most, r), float("nan"), device="cuda").half()
    bad[:, ::2] = float("inf")
    used.prefill(bad, torch.full((b, most, 64), float("nan"), device="cuda").half(), most)
    t = [100, 129, 0]
    c, kr = rand(b, max(t), r), rand(b, max(t), 64)
    for x in (used, new):
        x.prefill(c, kr, t)
    for n in ([1, 1, 1], [3, 0, 5], [27, 126, 1], [1, 1, 1], [130, 1, 122], [1, 1, 1], [1, 1, 1], [5, 2, 126], [300, 1, 1], [1, 1, 0]):
        c, kr, qn, qr = rand(b, max(n), r), rand(b, max(n), 64), rand(b, h, max(n), 128), rand(b, h, max(n), 64)
        for form in ("absorbed", "expanded"):
            out, want = (x.attn(qn, qr, c, kr, n, wk, wv, form=form) for x in (used, new))
            assert bool(torch.isfinite(out).all()) and torch.equal(out, want), (n, form)
        for x in (used, new):
            x.append(c, kr, n)
    assert all(torch.equal(x, y) for x, y in zip(used.restore(), new.restore()))
    assert used.check() == 0 and new.check() == 0
    used.close()
    new.close()
