"""Device memory of the chunk attention: none before a call needs it, and the
first call may be a captured one."""
import pytest


def _free():
    import torch
    torch.cuda.synchronize()
    return torch.cuda.mem_get_info()[0]


@pytest.mark.gpu
def test_a_cache_without_chunks_keeps_no_partials():
    """What 8 caches of 256 tokens need is far below 8 MB each (the decode's
    partials: 8 heads of 304 slots of 132 floats, 1.3 MB)."""
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    x = torch.zeros(1, 1, 64, 128, device="cuda").half()

    def use(c):
        c.prefill(x, x, 64)
        c.decode(x[:, :, 0].contiguous())
        c.chunk_attn(x, x, x, 64)   # nothing to split
        return c

    new = lambda: K.KiviCache(1, 1, 128, 2, 2, 32, 128, 256)   # noqa: E731
    use(new()).close()   # (the kernels' code is loaded)
    start = _free()
    caches = [use(new()) for _ in range(8)]
    assert start - _free() < 8 * (8 << 20)
    for c in caches:
        c.close()
    assert abs(_free() - start) < 8 << 20


@pytest.mark.gpu
@pytest.mark.parametrize("n,window", [(3, 0), (40, 0), (300, 200)])
def test_first_call_is_captured(n, window):
    """Few rows, many, a window: captured without a call before it."""
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    g = torch.Generator(device="cuda").manual_seed(n)
    rows = lambda h, t: torch.randn(1, h, t, 128, device="cuda", generator=g).half()   # noqa: E731
    c, e = (K.KiviCache(1, 1, 128, 2, 2, 32, 128, 6000) for _ in range(2))
    Kp, Vp = rows(1, 5000), rows(1, 5000)
    for z in (c, e):
        z.prefill(Kp, Vp, 5000)
    Q, Kn, Vn = rows(2, n), rows(1, n), rows(1, n)
    out = torch.zeros_like(Q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.chunk_attn(Q, Kn, Vn, n, window=window, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, e.chunk_attn(Q, Kn, Vn, n, window=window))
    assert c.check() == 0 and e.check() == 0
    del graph
    c.close()
    e.close()


@pytest.mark.gpu
def test_first_windowed_prompt_is_captured():
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    g = torch.Generator(device="cuda").manual_seed(2)
    Q, Kp, Vp = (torch.randn(1, h, 3100, 64, device="cuda", generator=g).half() for h in (2, 1, 1))
    c, e = (K.KiviCache(1, 1, 64, 2, 2, 32, 128, 3200) for _ in range(2))
    out = torch.zeros_like(Q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.prefill_attn(Q, Kp, Vp, 3100, out=out, window=700, sinks=4)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, e.prefill_attn(Q, Kp, Vp, 3100, window=700, sinks=4))
    assert c.check() == 0
    del graph
    c.close()
    e.close()
