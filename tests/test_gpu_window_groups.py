"""The windowed prompt with every group size, within what the rounding of its
weights allows."""
import numpy as np
import pytest

from tests import operators_ref as R
from tests import rounding_ref as E


@pytest.mark.gpu
@pytest.mark.parametrize("d,G", [(128, 128), (128, 32), (64, 64), (64, 16)])
@pytest.mark.parametrize("hq,h,T,window,sinks", [(2, 2, [300, 129], 40, 0), (4, 1, [700, 0], 128, 5), (3, 1, [128, 1], 1, 200),
                                                 (2, 1, [2500, 1300], 900, 4)])
def test_prompt_window_groups(hq, h, T, window, sinks, d, G):
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    rng = np.random.default_rng(T[0] + window)
    b, t = 2, max(T)
    Q, Kp, Vp = (rng.standard_normal((b, x, t, d)).astype(np.float16) for x in (hq, h, h))
    Qt, Kt, Vt = (torch.from_numpy(x).cuda() for x in (Q, Kp, Vp))
    c, w = (K.KiviCache(b, h, d, 2, 4, G, 128, t + 8) for _ in range(2))
    got = c.prefill_attn(Qt, Kt, Vt, T, window=window, sinks=sinks).float().cpu().numpy()
    w.prefill(Kt, Vt, T)
    a, e = c.export(), w.export()
    assert all(np.array_equal(a[x], e[x]) for x in a)   # the cache of the plain prefill
    assert all(np.array_equal(x, y) for x, y in zip(c.lengths(), w.lengths()))
    for i in range(b):
        assert not got[i, :, T[i]:].any()
        if T[i]:
            see = R.visible(np.arange(T[i]), T[i], window, sinks)
            rows = [(got[i, q, :T[i]], E.attend(Q[i, q, :T[i]], Kp[i, q * h // hq, :T[i]], Vp[i, q * h // hq, :T[i]], see, False))
                    for q in range(hq)]
            E.check([x for x, _ in rows], [y for _, y in rows], f"sequence {i}")
    if G > 64:   # without a window the attention's CTAs pack, up to G = 64
        with pytest.raises(K.KiviError) as r:
            c.prefill_attn(Qt, Kt, Vt, T)
        assert r.value.status == 2
    assert c.check() == 0
    c.close()
    w.close()
