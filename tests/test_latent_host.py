"""The latent cache's calls before they reach the GPU: the library's are faked."""
import pytest


class _Lib:
    """Records the calls made of it; all succeed, and the cache holds T tokens."""

    def __init__(self):
        self.calls, self.T = [], 0

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, a))
            if name == "kivi_latent_lengths":
                import ctypes
                ctypes.cast(a[1], ctypes.POINTER(ctypes.c_int))[0] = self.T
            return 0
        return call

    def names(self):
        return [n for n, _ in self.calls if n != "kivi_latent_lengths"]


@pytest.fixture
def cache(monkeypatch):
    """An empty latent cache of one sequence on device 0, its library, and a call of
    its attention with h heads, n of ns tokens."""
    torch = pytest.importorskip("torch")
    from bit_quantized_kv_quantize_gb300 import kivi as K
    lib = _Lib()
    monkeypatch.setattr(K, "lib", lib)
    monkeypatch.setattr(K, "_rows16", lambda x, shape, dev, name: 4096)
    monkeypatch.setattr(K, "_stream", lambda s: 0)
    monkeypatch.setattr(K, "_space", lambda stream, dev, *halves: (None, [4096] * len(halves)))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    c = object.__new__(K.LatentCache)
    c.b, c.r, c.max_tokens, c._dev, c._device, c._sms, c._h = 1, 512, 1 << 20, 0, None, 152, None

    def attn(h, n, ns=None, form=None):
        lib.calls.clear()
        rows = lambda *s: torch.empty(s, device="meta", dtype=torch.float16)   # noqa: E731
        ns = n if ns is None else ns
        q = rows(1, h, ns, 128)
        c.attn(q, rows(1, h, ns, 64), rows(1, ns, 512), rows(1, ns, 64), n, rows(h, 128, 512), rows(h, 128, 512), out=q, form=form)
        return lib.names()
    return c, lib, attn


def _absorbed(names):
    return "kivi_latent_attn" in names


def _expanded(names):
    return "kivi_latent_rows" in names and not _absorbed(names)


def test_the_form_that_takes_the_call(cache):
    """More heads, or rows, than the absorbed attention takes: expanded, whatever the
    number of tokens and the size of keys and values."""
    _, lib, attn = cache
    assert _absorbed(attn(128, 1)) and _absorbed(attn(16, 15)) and _expanded(attn(16, 1, form="expanded"))
    lib.T = 100
    for h in (129, 1024):
        for n in (1, 15, 16, 300):
            assert _expanded(attn(h, n)), (h, n)
    lib.T = 80000                               # (keys and values of more than 4 GB)
    assert _absorbed(attn(128, 1024)) and _expanded(attn(129, 1024))
    lib.T = 1 << 19
    assert _absorbed(attn(128, 40, ns=(1 << 17) - 1)) and _expanded(attn(128, 40, ns=1 << 17))
    assert _expanded(attn(128, 1, ns=1 << 17))
    assert _absorbed(attn(129, 1, form="absorbed"))   # (asked for: the library refuses it)


def test_every_call_of_a_cache_reports_to_it(cache):
    """Products and expanded attention too: kivi_latent_check tells of a wait that ran
    out in any of them."""
    c, lib, attn = cache
    import torch
    c._h = object()
    rows = lambda *s: torch.empty(s, device="meta", dtype=torch.float16)   # noqa: E731
    w = rows(8, 128, 512)

    def all_of_it(names):
        assert all(a[0] is c._h for _, a in lib.calls), [n for n, a in lib.calls if a[0] is not c._h]
        return names

    for form in ("absorbed", "expanded"):
        names = all_of_it(attn(8, 20, form=form))
        assert len(names) == (3 if form == "absorbed" else 4)
    lib.calls.clear()
    q = rows(1, 8, 30, 128)
    c.prefill_attn(q, rows(1, 8, 30, 64), rows(1, 30, 512), rows(1, 30, 64), 30, w, w, out=q)
    assert len(all_of_it(lib.names())) == 4
    lib.calls.clear()
    c.extend(q, rows(1, 8, 30, 64), rows(1, 30, 512), rows(1, 30, 64), 30, w, w, out=q)
    assert all_of_it(lib.names())[-1] == "kivi_latent_append"


def test_a_caches_products_and_expanded_attention_refuse():
    import ctypes

    import numpy as np
    from bit_quantized_kv_quantize_gb300 import kivi as K
    p, n = ctypes.c_void_p(4096), np.array([1], np.int32)   # never dereferenced: every call below is refused
    bogus = ctypes.cast(ctypes.create_string_buffer(64), ctypes.c_void_p)
    for h in (None, bogus):
        assert K.lib.kivi_latent_product(h, p, p, 1, 4, 1, n.ctypes.data, 128, 128, 0, p, None) == 1
        for T in (None, n.ctypes.data):
            assert K.lib.kivi_latent_expanded(h, p, p, p, p, p, 4, T, n.ctypes.data, 1, 2, 1.0, p, None) == 1
        assert b"latent cache handle" in K.lib.kivi_last_error()
