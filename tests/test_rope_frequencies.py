"""The yarn scaling of rope_frequencies against the method's ramp, and against
what its documentation says of each pair's turns."""
import numpy as np
import pytest


def _ramp(rot, base, factor, length, fast, slow):
    """The published ramp: it runs between the (real) pair indices that turn
    `fast` and `slow` times over the original length, rounded outwards and kept
    inside [0, rot - 1]: past the last pair where that still turns often."""
    at = [rot * np.log(length / (r * 2 * np.pi)) / (2 * np.log(base)) for r in (fast, slow)]
    lo, hi = max(np.floor(at[0]), 0), min(np.ceil(at[1]), rot - 1)
    m = np.arange(rot // 2)
    f = float(base) ** (-2.0 * m / rot)
    keep = 1 - np.clip((m - lo) / max(hi - lo, 1e-3), 0, 1)
    return f / factor * (1 - keep) + f * keep


@pytest.mark.parametrize("rot", [64, 128])
@pytest.mark.parametrize("base", [1e4, 5e5])
@pytest.mark.parametrize("length", [2048, 8192, 32768, 65536, 131072, 1 << 20])
def test_yarn_ramp(rot, base, length):
    from bit_quantized_kv_quantize_gb300 import kivi as K
    f, m = K.rope_frequencies(rot, base, "yarn", 4.0, length)
    assert np.allclose(f, _ramp(rot, base, 4.0, length, 32.0, 1.0), rtol=1e-12)
    assert np.isclose(m, 0.1 * np.log(4.0) + 1)
    plain = K.rope_frequencies(rot, base)[0]
    turns = length * plain / (2 * np.pi)
    # a pair that turns more than once is not yet divided by the whole factor
    # (1.0001: away from the border), one that turns 32 times more is kept
    assert np.all(f[turns > 1.0001] > plain[turns > 1.0001] / 4 * (1 + 1e-9))
    last = np.floor(rot * np.log(length / (64 * np.pi)) / (2 * np.log(base)))
    assert np.allclose(f[np.arange(rot // 2) <= last], plain[np.arange(rot // 2) <= last])
