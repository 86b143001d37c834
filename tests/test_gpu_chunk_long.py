"""Row tiles cut into many shares, and several row tiles over a long cache."""
import numpy as np
import pytest

from tests import operators_ref as R
from tests import rounding_ref as E


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,hq,h,window,sinks", [
    (33000, 40, 1, 1, 0, 0),      # one row tile in about 64 shares: the join's lanes go round twice
    (33000, 130, 2, 1, 0, 0),     # ... two row tiles
    (70001, 3, 2, 1, 0, 0),       # few rows, about 68 shares
    (70001, 3, 2, 1, 40000, 100),  # ... with a window
    (2600, 70, 8, 1, 0, 0),       # three row tiles of 256 rows over 40 tiles and more
    (3333, 170, 4, 2, 1500, 7),
    (1999, 129, 5, 1, 0, 0),      # ... five heads a kv head
])
@pytest.mark.parametrize("d", [64, 128])
def test_long(T, n, hq, h, window, sinks, d):
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    rng = np.random.default_rng(T + n + d)
    Kh, Vh = (rng.standard_normal((1, h, T, d)).astype(np.float16) for _ in range(2))
    Q, Kn, Vn = (rng.standard_normal((1, x, n, d)).astype(np.float16) for x in (hq, h, h))
    Kh[..., 0] += np.linspace(-2, 2, T).astype(np.float16)   # the shares' maxima differ
    Q[..., 0] += 4
    c = K.KiviCache(1, h, d, 2, 4, 32, 64, T + n)
    c.prefill(*(torch.from_numpy(x).cuda() for x in (Kh, Vh)), T)
    got = c.chunk_attn(*(torch.from_numpy(x).cuda() for x in (Q, Kn, Vn)), n, window, sinks).float().cpu().numpy()
    assert c.check() == 0
    c.close()
    see = R.visible(T + np.arange(n), T + n, window, sinks)
    rows = []
    for j in range(h):
        k, v = R.restore(Kh[0, j], Vh[0, j], *R.counters(T, 64), 2, 4, 32)
        k, v = np.concatenate([k, Kn[0, j].astype(np.float64)]), np.concatenate([v, Vn[0, j].astype(np.float64)])
        for e in range(j * hq // h, (j + 1) * hq // h):
            rows.append((got[0, e], E.attend(Q[0, e], k, v, see)))
    E.check([x for x, _ in rows], [y for _, y in rows])
