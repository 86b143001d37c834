"""extend() before it reaches the GPU: the library's calls are faked."""
import pytest


class _Lib:
    """Records the calls made of it; all succeed."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


class _Tensor:
    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 4096


@pytest.fixture
def cache(monkeypatch):
    """A cache of device 0 with a faked library, and the device that is current."""
    import torch
    from bit_quantized_kv_quantize_gb300 import kivi as K
    lib, current = _Lib(), [0]
    monkeypatch.setattr(K, "lib", lib)
    monkeypatch.setattr(K, "_rows16", lambda x, shape, dev, name: 4096)
    monkeypatch.setattr(K, "_stream", lambda s: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    for make in ("empty_like", "zeros_like"):
        monkeypatch.setattr(torch, make, lambda x: x)
    c = object.__new__(K.KiviCache)
    c.b, c.h_kv, c.d, c.max_tokens, c._dev, c._h = 1, 1, 64, 100, 0, None
    return c, lib, current


@pytest.mark.parametrize("rope", [False, True])
def test_extend_on_another_device_launches_nothing(cache, rope):
    from bit_quantized_kv_quantize_gb300 import kivi as K
    c, lib, current = cache
    r = K.Rope(64) if rope else None
    x = _Tensor(1, 1, 4, 64)
    c.extend(x, x, x, 3, rope=r)
    launches = [n for n in lib.calls if n != "kivi_cache_lengths"]
    assert launches == ["kivi_rope"] * rope + ["kivi_chunk_attn", "kivi_append_chunk"]
    lib.calls.clear()
    current[0] = 1
    with pytest.raises(K.KiviError) as e:
        c.extend(x, x, x, 3, rope=r)
    assert e.value.status == 1
    assert not [n for n in lib.calls if n != "kivi_cache_lengths"]
