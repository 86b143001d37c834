"""The largest sizes of the chunk and window calls: what passes the kernels'
32-bit counts is refused before anything is launched."""
import numpy as np
import pytest


def _call(K, c, fn, x, n, stride, hq, window):
    """One call of the library with counts that the tensor x does not have: it
    must be refused before the GPU sees them."""
    cnt = np.array([n], np.int32)
    p = x.data_ptr()
    return fn(c.handle, p, p, p, cnt.ctypes.data, stride, hq, window, 0, p, None)


@pytest.mark.gpu
def test_work_beyond_32_bits_is_refused():
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    c = K.KiviCache(1, 1, 64, 2, 2, 32, 32, 64)
    x = torch.zeros(1, 8, 4, 64, device="cuda").half()
    big = 1 << 26   # 2^21 row tiles of 2^19 key tiles on average: 2^40 of them
    assert _call(K, c, K.lib.kivi_chunk_attn, x, big, big, 8, 0) == 2
    assert b"2^31" in K.lib.kivi_last_error()
    assert _call(K, c, K.lib.kivi_chunk_attn, x, 4, big + 1, 8, 0) == 2
    assert c.lengths()[0].tolist() == [0] and c.check() == 0
    assert torch.equal(c.chunk_attn(x, x[:, :1].contiguous(), x[:, :1].contiguous(), 4), x)   # still usable
    c.close()


@pytest.mark.gpu
def test_windowed_prompt_beyond_its_stride_is_refused():
    """Row indices of up to 8 heads a kv head must stay below 2^29."""
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    c = K.KiviCache(1, 1, 64, 2, 2, 32, 32, 64)
    x = torch.zeros(1, 8, 4, 64, device="cuda").half()
    assert _call(K, c, K.lib.kivi_prefill_attn_window, x, 4, (1 << 26) + 1, 8, 7) == 2
    assert c.lengths()[0].tolist() == [0] and c.check() == 0
    c.close()
