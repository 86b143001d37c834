"""The chunk attention's 16-bit roundings where they matter most: many tokens
far below one, keys with a few large channels; few query rows and many."""
import numpy as np
import pytest

from tests import operators_ref as R
from tests import rounding_ref as E


def _cuda(*xs):
    import torch
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in xs]


def _run(Kh, Vh, Q, Kn, Vn, kb, vb, G, Rw):
    """out [hq, n, d] of one sequence of one kv head (and what it should be)."""
    from bit_quantized_kv_quantize_gb300 import kivi as K
    t, n, d, hq = Kh.shape[0], Kn.shape[0], Kh.shape[1], Q.shape[0]
    c = K.KiviCache(1, 1, d, kb, vb, G, Rw, t + n)
    c.prefill(*_cuda(Kh[None, None], Vh[None, None]), t)
    got = c.chunk_attn(*_cuda(Q[None], Kn[None, None], Vn[None, None]), n).float().cpu().numpy()[0]
    assert c.check() == 0
    c.close()
    k, v = R.restore(Kh, Vh, *R.counters(t, Rw), kb, vb, G)
    k, v = np.concatenate([k, Kn.astype(np.float64)]), np.concatenate([v, Vn.astype(np.float64)])
    see = R.visible(t + np.arange(n), t + n, 0, 0)
    return got, [E.attend(Q[e], k, v, see) for e in range(hq)]


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("nats", [14.0, 17.5, 19.0])
def test_flat_background_under_a_sink(n, nats):
    """The first token scores `nats` above 32k equal ones whose values add up:
    each of their weights is next to nothing, their sum is not.  As many kv
    heads as SMs, all alike, so that no sequence is cut into shares (a share
    without the first token would take its weights against its own largest)."""
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    t, d = 32768, 64
    h = torch.cuda.get_device_properties(0).multi_processor_count
    Kh, Vh = np.zeros((t, d), np.float16), np.ones((t, d), np.float16)
    Kh[0], Vh[0] = nats / np.sqrt(d), 0.0   # (with q = 1: score sum(k) / 8)
    c = K.KiviCache(1, h, d, 2, 2, 32, 128, t + n)
    c.prefill(*(x[None, None].expand(1, h, t, d).contiguous() for x in _cuda(Kh, Vh)), t)
    one = torch.ones(1, h, n, d, device="cuda").half()
    got = c.chunk_attn(one, torch.zeros_like(one), one, n).float().cpu().numpy()[0]
    assert c.check() == 0
    c.close()
    k, v = R.restore(Kh, Vh, *R.counters(t, 128), 2, 2, 32)
    k, v = np.concatenate([k, np.zeros((n, d))]), np.concatenate([v, np.ones((n, d))])
    o, b, _ = E.attend(np.ones((n, d)), k, v, R.visible(t + np.arange(n), t + n, 0, 0))
    assert np.all(b < 0.1 * np.abs(o) + 1.5e-5)   # the bound says something
    assert np.all(np.abs(got - o) <= b), f"{np.abs(got - o).max():.3e} against {b.max():.3e} of {o.max():.3e}"


@pytest.mark.gpu
@pytest.mark.parametrize("d,kb,vb,G", [(128, 2, 2, 32), (64, 4, 4, 64), (128, 4, 2, 16)])
@pytest.mark.parametrize("n,big", [(3, 1.0), (3, 8.0), (150, 1.0), (150, 8.0)])
def test_keys_with_large_channels(d, kb, vb, G, n, big):
    """Two channels of every key are `big` times the others."""
    rng = np.random.default_rng(d + n + int(big))
    t, hq = 2500, 4
    Kh, Vh = (rng.standard_normal((t, d)).astype(np.float16) for _ in range(2))
    Kn, Vn = (rng.standard_normal((n, d)).astype(np.float16) for _ in range(2))
    ch = rng.choice(d, 2, replace=False)
    Kh[:, ch] *= np.float16(big)
    Kn[:, ch] *= np.float16(big)
    Q = rng.standard_normal((hq, n, d)).astype(np.float16)
    got, want = _run(Kh, Vh, Q, Kn, Vn, kb, vb, G, 128)
    E.check(got, want, f"channels times {big}")
