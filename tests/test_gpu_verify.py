"""Draft verification (kivi_verify, kivi.verify) against whole-number
arithmetic of its definition, exactly, and its refusals."""
import ctypes

import numpy as np
import pytest

from tests import latent_ref as L


def _K():
    from bit_quantized_kv_quantize_gb300 import kivi as K
    return K


def test_refusals_before_cuda():
    K = _K()
    p = ctypes.c_void_p(4096)   # never dereferenced: every call below is refused
    odd = ctypes.c_void_p(4097)

    def call(p=p, q=p, size=4, draft=p, u=p, b=1, ns=2, V=10, n=(1,), tokens=p, accepted=p):
        a = None if n is None else np.array(n, np.int32)
        return K.lib.kivi_verify(p, q, size, draft, u, b, ns, V, None if a is None else a.ctypes.data, tokens, accepted, None)

    assert call(b=0) == 1 and call(ns=-1) == 1 and call(V=0) == 1
    assert call(b=1025) == 2 and call(V=2 ** 20 + 1) == 2 and call(ns=2 ** 20 + 1) == 2 and call(size=8) == 2
    assert call(p=None) == 1 and call(draft=None) == 1 and call(u=None) == 1 and call(n=None) == 1
    assert call(tokens=None) == 1 and call(accepted=None) == 1
    assert call(n=(3,)) == 1 and call(n=(-1,)) == 1
    assert call(p=odd) == 1 and call(q=odd) == 1 and call(u=odd) == 1 and call(tokens=odd) == 1


def test_reference_draws_from_the_target():
    """Tokens of 1 + draft, over many numbers, are distributed as p (Leviathan
    et al.'s identity): a check of the reference itself."""
    rng = np.random.default_rng(0)
    V, m = 5, 20000
    p, q = rng.dirichlet(np.ones(V)).astype(np.float32), rng.dirichlet(np.ones(V)).astype(np.float32)
    seen = np.zeros(V)
    for _ in range(m):
        x = rng.choice(V, p=q.astype(np.float64) / q.astype(np.float64).sum())
        out, _ = L.verify(np.stack([p, p]), q[None], [x], rng.random(2).astype(np.float32), 1)
        seen[out[0]] += 1
    # four standard deviations of a count
    assert np.all(np.abs(seen / m - p) <= 4 * np.sqrt(p * (1 - p) / m) + 1e-6)


def _run(torch, p, q, draft, u, n, **kw):
    K = _K()
    dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()   # noqa: E731
    t, a = K.verify(dev(p), dev(q), dev(draft.astype(np.int32)), dev(u), list(n), **kw)
    t, a = t.cpu().numpy(), a.cpu().numpy()
    for i in range(p.shape[0]):
        ref, r = L.verify(p[i], None if q is None else q[i], draft[i], u[i], n[i])
        assert a[i] == r, (i, a[i], r)
        assert np.array_equal(t[i], ref), (i, t[i], ref)
    return t, a


def _case(rng, b, ns, V, dt, certain, near=0.5):
    z = 2 * rng.standard_normal((b, ns + 1, V))
    y = z[:, :ns] + near * rng.standard_normal((b, ns, V))
    p = np.exp(z - z.max(2, keepdims=True))
    q = np.exp(y - y.max(2, keepdims=True)) if ns else np.zeros((b, 0, V))
    p, q = (p / p.sum(2, keepdims=True)).astype(dt), (q / np.maximum(q.sum(2, keepdims=True), 1e-30)).astype(dt)
    draft = np.zeros((b, ns), np.int32)
    for i in range(b):
        for r in range(ns):
            w = q[i, r].astype(np.float64)
            draft[i, r] = y[i, r].argmax() if certain else rng.choice(V, p=w / w.sum())
    return p, None if certain else q, draft, rng.random((b, ns + 1)).astype(np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [np.float32, np.float16])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("b,ns,V", [(1, 1, 1), (3, 0, 7), (2, 1, 33), (5, 4, 1000), (3, 40, 515), (4, 3, 4097), (2, 5, 32001),
                                    (2, 2, 150001)])
def test_matches(b, ns, V, certain, dt):
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(b * 1000 + ns * 10 + V)
    p, q, draft, u = _case(rng, b, ns, V, dt, certain)
    for n in ([ns] * b, rng.integers(0, ns + 1, b)):
        _run(torch, p, q, draft, u, [int(x) for x in n])


@pytest.mark.gpu
@pytest.mark.parametrize("V", [5, 2048, 40000])
def test_edges(V):
    """u of 0 and just below 1, equal rows (nothing is left of the difference),
    rows without any probability, negative, infinite and NaN ones, drafted tokens
    outside the vocabulary, all of the weight on the first or last token."""
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(V)
    b, ns = 12, 2
    p, q, draft, u = _case(rng, b, ns, V, np.float32, False)
    u[0] = 0.0
    u[1] = 1.0 - 2.0 ** -24
    u[2], q[2] = 1.0 - 2.0 ** -24, p[2, :ns]
    p[2] *= np.float32(0.75)                     # p < q everywhere: drawn from p
    p[3, 0] = 0.0                                # not kept, and nothing to draw from
    p[4, 0, 1:], p[4, 0, 0] = 0.0, 1.0
    draft[4, 0], u[4, 0] = V - 1, 0.5
    p[5, 0, :-1], p[5, 0, -1], draft[5, 0] = 0.0, 1.0, 0
    draft[6] = [V, 0]
    draft[7] = [-1, 0]
    p[8, 0, ::2], draft[8, 0] = np.nan, 0
    q[9, 0, 1::2], draft[9, 0] = np.nan, 1
    p[10, 0, 0], p[10, 0, 1], draft[10, 0] = -1.0, np.inf, 0
    p[11, ns], u[11, :ns], q[11] = 2.0 ** -60, 0.0, 0.5     # kept; then less than a unit anywhere
    t, a = _run(torch, p, q, draft, u, [ns] * b)
    assert a[3] == 0 and np.all(t[3] == -1)
    assert a[4] == 0 and t[4, 0] == 0 and a[5] == 0 and t[5, 0] == V - 1
    assert a[6] == 0 and a[7] == 0 and a[11] == ns and t[11, ns] == -1
    _run(torch, p, None, draft, u, [ns] * b)


@pytest.mark.gpu
def test_streams_graphs_and_outputs():
    """On another stream, captured and replayed with new contents, into given
    outputs; rows of other calls untouched."""
    torch = pytest.importorskip("torch")
    K = _K()
    rng = np.random.default_rng(5)
    p, q, draft, u = _case(rng, 4, 3, 5000, np.float32, False)
    dev = [torch.from_numpy(x).cuda() for x in (p, q, draft, u)]
    tokens, accepted = torch.zeros((4, 4), dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    K.verify(*dev, tokens=tokens, accepted=accepted, stream=st)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.verify(*dev, tokens=tokens, accepted=accepted)
    for seed in (6, 7):
        p, q, draft, u = _case(np.random.default_rng(seed), 4, 3, 5000, np.float32, False)
        for x, y in zip(dev, (p, q, draft, u)):
            x.copy_(torch.from_numpy(y))
        g.replay()
        torch.cuda.synchronize()
        for i in range(4):
            ref, r = L.verify(p[i], q[i], draft[i], u[i], 3)
            assert accepted[i] == r and np.array_equal(tokens[i].cpu().numpy(), ref)


@pytest.mark.gpu
def test_binding_refuses():
    torch = pytest.importorskip("torch")
    K = _K()
    p, q = torch.rand(2, 3, 9, device="cuda"), torch.rand(2, 2, 9, device="cuda")
    d, u = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.rand(2, 3, device="cuda")
    for bad in ((p.double(), q, d, u), (p, q.half(), d, u), (p, q, d.long(), u), (p.cpu(), q, d, u)):
        with pytest.raises(TypeError):
            K.verify(*bad)
    for bad in ((p[0], q, d, u), (p, q[:, :1], d, u), (p.transpose(0, 1), q, d, u), (p, q, d, u[:, :2])):
        with pytest.raises(ValueError):
            K.verify(*bad)
    with pytest.raises(K.KiviError):
        K.verify(p, q, d, u, 3)
    with pytest.raises(ValueError):
        K.verify(p, q, d, u, [1])
