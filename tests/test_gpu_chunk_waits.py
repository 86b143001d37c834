"""A chunk attention in which some warps give up, as if a wait had run out: the
others stop too, with copies under way; it reports that, ends at once, and
leaves nothing behind."""
import time

import pytest


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,hq", [
    (2000, 40, 8),    # 256-row tiles over records
    (0, 500, 2),      # ... whose first tiles are copies already on their way
    (130, 300, 3),    # ... three heads a kv head: queries without copies
    (100, 400, 1),    # ... one slot
    (4000, 3, 2),     # few rows
    (2050, 2, 8),
])
@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_runs_out(monkeypatch, T, n, hq, d):
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    g = torch.Generator(device="cuda").manual_seed(T + n)
    rows = lambda h, t: torch.randn(2, h, t, d, device="cuda", generator=g).half()   # noqa: E731
    c = K.KiviCache(2, 2, d, 2, 4, 32, 64, 5000)
    if T:
        c.prefill(rows(2, T), rows(2, T), T)
    Q, Kn, Vn = rows(2 * hq, n), rows(2, n), rows(2, n)
    want = c.chunk_attn(Q, Kn, Vn, n)
    assert c.check() == 0
    for quit in ("0", "2", "0"):   # warps that restore tiles, or the one that copies records after so many
        monkeypatch.setenv("KIVI_CHUNK_QUIT", quit)
        t0 = time.perf_counter()
        c.chunk_attn(Q, Kn, Vn, n)
        flags = c.check()
        assert flags & 2 and time.perf_counter() - t0 < 1.0
    monkeypatch.delenv("KIVI_CHUNK_QUIT")
    assert torch.equal(c.chunk_attn(Q, Kn, Vn, n), want)
    assert c.check() == 0
    c.close()
