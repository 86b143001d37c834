"""Device memory of the latent cache: no records for tokens that are never
quantized."""
import pytest


@pytest.mark.gpu
@pytest.mark.parametrize("R,most", [(16384, 16384), (32768, 16000), (8192, 16384), (8192, 16001)])
def test_records_are_for_quantized_tokens(R, most):
    """16 sequences of up to 16k tokens: fp16 rows of the window and of one block more,
    rotary keys, and records of what can leave the window (320 bytes a token), each
    allocation up to 2 MB larger."""
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K

    def free():
        torch.cuda.synchronize()
        return torch.cuda.mem_get_info()[0]

    b, r = 16, 512
    K.LatentCache(1, r, 4, 32, 64, 200).close()
    up = lambda x: -(-x // 128) * 128   # noqa: E731
    before = free()
    c = K.LatentCache(b, r, 4, 32, R, most)
    need = b * ((min(up(R), up(most)) + 128) * r * 2 + up(most) * 128 + up(max(0, most - R)) * 320)
    assert 0 <= before - free() - need + (1 << 20) <= 9 << 20
    g = torch.Generator(device="cuda").manual_seed(R)
    x, kr = torch.randn(b, most, r, generator=g, device="cuda").half(), torch.randn(b, most, 64, generator=g, device="cuda").half()
    c.prefill(x[:, :most - 1].contiguous(), kr[:, :most - 1].contiguous(), most - 1)
    c.append(x[:, most - 1:].contiguous(), kr[:, most - 1:].contiguous(), 1)
    gc, gk = c.restore()
    T, Tq = c.lengths()
    assert list(T) == [most] * b and list(Tq) == [max(0, most - R)] * b
    k = int(Tq[0])
    assert torch.equal(gc[:, k:], x[:, k:]) and torch.equal(gk, kr)
    if k:   # codes: within half a step and the roundings of scale, zero and value
        y = x[:, :k].float().view(b, k, -1, 32)
        step = (y.amax(3) - y.amin(3)) / 15
        bound = step * (0.5 + 16 * 2.0 ** -11) + y.abs().amax(3) * 2.0 ** -10
        assert bool(((gc[:, :k].float().view(b, k, -1, 32) - y).abs().amax(3) <= bound).all())
    assert c.check() == 0
    held = free()                                     # (with torch's tensors)
    c.close()
    assert abs(free() - held - need) <= 9 << 20
