"""Rotary positions with several axes (kivi_rope_axes, Rope(axes=...)) against
a 64-bit reference, the inverse as the gradient, and refusals."""
import ctypes

import numpy as np
import pytest

from tests import operators_ref as R


def _K():
    from bit_quantized_kv_quantize_gb300 import kivi as K
    return K


def test_axes_of_pairs():
    K = _K()
    assert K.rope_axes([2, 1, 3]) == [0, 0, 1, 2, 2, 2]
    assert K.rope_axes([2, 1, 3], in_turn=True) == [0, 1, 2, 0, 2, 2]
    assert K.rope_axes([0, 2]) == [1, 1]
    for bad in ([], [0, 0], [-1, 3]):
        with pytest.raises(ValueError):
            K.rope_axes(bad)
    r = K.Rope(64, axes=K.rope_axes([16, 8, 8]))
    assert r.axes == 3 and len(r._axis) == 32
    for bad in ([0] * 31, [0] * 31 + [-1], [0] * 31 + [255]):
        with pytest.raises(ValueError):
            K.Rope(64, axes=bad)


def test_refusals_before_cuda():
    K = _K()
    p = ctypes.c_void_p(4096)   # never dereferenced: every call below is refused
    n, turns, axis = np.array([1], np.int32), np.zeros(64, np.uint64), np.zeros(64, np.uint8)
    axis[63] = 2

    def call(q=p, k=p, b=1, hq=2, hk=1, ns=1, d=128, n=n, pos=p, axes=3, axis=axis, turns=turns, rot=128, f=1.0, qo=p, ko=p):
        a = lambda x: None if x is None else x.ctypes.data   # noqa: E731
        return K.lib.kivi_rope_axes(q, k, b, hq, hk, ns, d, a(n), pos, axes, a(axis), a(turns), rot, 0, f, 0, qo, ko, None)

    assert call(axes=0) == 1 and call(axes=256) == 1 and call(axes=2) == 1 and call(axis=None) == 1 and call(pos=None) == 1
    assert call(pos=ctypes.c_void_p(4098)) == 1 and call(n=np.array([2], np.int32)) == 1 and call(f=float("nan")) == 1
    assert call(d=96) == 2 and call(rot=24) == 2 and call(b=1025) == 2 and call(q=None) == 1
    assert call(qo=ctypes.c_void_p(4104)) == 1


def _check(got, x, pos, rope, inverse=False):
    """Rows x [n, d] at positions pos [axes, n]: the bound of the one-axis
    rotation (one rounding to fp16 of a 32-bit result whose sine and cosine are
    within 2^-22: 2^-21 (|x| + |y|) covers them), pair by pair."""
    rot = rope.rot_dim
    ref = x.astype(np.float64).copy()
    mag = np.zeros_like(ref)
    for m in range(rot // 2):
        i, j = (2 * m, 2 * m + 1) if rope.interleaved else (m, m + rot // 2)
        a = pos[rope._axis[m]].astype(np.float64) * rope.inv_freq[m] * (-1 if inverse else 1)
        c, s = rope.factor * np.cos(a), rope.factor * np.sin(a)
        e, o = x[:, i].astype(np.float64), x[:, j].astype(np.float64)
        ref[:, i], ref[:, j] = e * c - o * s, o * c + e * s
        mag[:, i] = mag[:, j] = np.abs(e) + np.abs(o)
    bound = np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + abs(rope.factor) * mag * 2.0 ** -21
    assert np.all(np.abs(got.astype(np.float64) - ref) <= bound)
    assert np.array_equal(got[:, rot:], x[:, rot:])


@pytest.mark.gpu
@pytest.mark.parametrize("b,hq,hk,n,d,rot,sections,in_turn,inter,far", [
    (1, 1, 1, 1, 64, 64, [16, 8, 8], False, False, 0),
    (3, 4, 2, 1, 128, 128, [16, 24, 24], False, False, 1000),
    (2, 5, 1, 37, 128, 96, [16, 16, 16], True, True, 2 ** 30),
    (1, 8, 8, 300, 64, 32, [16], False, True, 70000),
    (2, 3, 3, 129, 256, 256, [40, 44, 44], True, False, -5),
    (1, 2, 1, 20, 64, 16, [1, 0, 2, 5], False, False, 2 ** 31 - 100),
])
def test_matches(b, hq, hk, n, d, rot, sections, in_turn, inter, far):
    torch = pytest.importorskip("torch")
    K = _K()
    rng = np.random.default_rng(n + d)
    f, m = K.rope_frequencies(rot, 10000.0, "yarn", 4.0, 4096) if rot > 16 else K.rope_frequencies(rot)
    rope = K.Rope(d, rot_dim=rot, interleaved=inter, inv_freq=f, factor=m, axes=K.rope_axes(sections, in_turn))
    A = len(sections)
    q, k = (rng.standard_normal((b, h, n, d)).astype(np.float16) for h in (hq, hk))
    pos = (far + rng.integers(-50, 51, (A, b, n)).clip(-2 ** 31 - far, 2 ** 31 - 1 - far)).astype(np.int32)
    cnt = [n] + [int(x) for x in rng.integers(0, n + 1, b - 1)]
    pt = torch.from_numpy(pos).cuda()
    for inverse in (False, True):
        qo, ko = rope.apply(torch.from_numpy(q).cuda(), torch.from_numpy(k).cuda(), pt, n=cnt, inverse=inverse)
        for got, x in ((qo.cpu().numpy(), q), (ko.cpu().numpy(), k)):
            for i in range(b):
                assert not got[i, :, cnt[i]:].any()
                for h in range(x.shape[1]):
                    _check(got[i, h, :cnt[i]], x[i, h, :cnt[i]], pos[:, i, :cnt[i]], rope, inverse)


@pytest.mark.gpu
def test_equal_positions_are_one_axis_and_the_inverse_is_the_gradient():
    """The same position on every axis gives the one-axis result bit for bit; and
    <R(x), g> differs by <dx, R^-1(g)> between x and x + dx (the map is linear:
    the difference quotient is exact but for roundings)."""
    torch = pytest.importorskip("torch")
    K = _K()
    g = torch.Generator(device="cuda").manual_seed(3)
    axes = K.rope_axes([22, 21, 21], in_turn=True)
    rope, one = K.Rope(128, axes=axes), K.Rope(128)
    x, dx, go = (torch.randn(2, 3, 65, 128, generator=g, device="cuda").half() for _ in range(3))
    same = (torch.arange(65, device="cuda") + 7).expand(3, 2, 65).int().contiguous()
    assert torch.equal(rope.apply(x, None, same), one.apply(x, None, 7))
    assert torch.equal(rope.apply(x, None, 7), one.apply(x, None, 7))
    pos = torch.randint(0, 5000, (3, 2, 65), generator=g, device="cuda").int()
    y0, y1 = rope.apply(x, None, pos).double(), rope.apply((x + dx).half(), None, pos).double()
    d = (x + dx).half().double() - x.double()
    lhs, grad = ((y1 - y0) * go.double()), rope.apply(go, None, pos, inverse=True).double()
    # each of the three rotations rounds by 2^-11 of its values (2^-21 of the pair's size before that)
    size = ((y0.abs() + y1.abs()) * go.double().abs()).sum() + (d.abs() * grad.abs()).sum()
    assert abs(float(lhs.sum() - (d * grad).sum())) <= 2.0 ** -10 * float(size)


@pytest.mark.gpu
def test_graph_stream_in_place_and_refusals():
    torch = pytest.importorskip("torch")
    K = _K()
    g = torch.Generator(device="cuda").manual_seed(4)
    rope = K.Rope(64, axes=K.rope_axes([10, 11, 11]))
    q, k = torch.randn(2, 4, 64, generator=g, device="cuda").half(), torch.randn(2, 1, 64, generator=g, device="cuda").half()
    pos = torch.randint(0, 999, (3, 2, 1), generator=g, device="cuda").int()
    ref = rope.apply(q, k, pos)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    a, b = q.clone(), k.clone()
    st.wait_stream(torch.cuda.current_stream())
    rope.apply(a, b, pos, q_out=a, k_out=b, stream=st)
    st.synchronize()
    assert torch.equal(a, ref[0]) and torch.equal(b, ref[1])
    gr = torch.cuda.CUDAGraph()
    out = torch.zeros_like(q)
    with torch.cuda.graph(gr):
        rope.apply(q, None, pos, q_out=out)
    pos.add_(5)
    gr.replay()
    assert torch.equal(out, rope.apply(q, None, pos))
    for bad in (pos.long(), pos[:2].contiguous(), pos.transpose(0, 1), torch.zeros(2, 1, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            rope.apply(q, k, bad)


@pytest.mark.gpu
def test_extend_at_given_positions():
    """KiviCache.extend with positions of its own: as rotating by hand."""
    torch = pytest.importorskip("torch")
    K = _K()
    g = torch.Generator(device="cuda").manual_seed(8)
    rope = K.Rope(64, axes=K.rope_axes([10, 11, 11]))
    Q, Kn, V = (torch.randn(2, h, 9, 64, generator=g, device="cuda").half() for h in (4, 2, 2))
    pos = torch.randint(0, 999, (3, 2, 9), generator=g, device="cuda").int()
    a, b = K.KiviCache(2, 2, 64, max_tokens=100), K.KiviCache(2, 2, 64, max_tokens=100)
    q1, k1 = rope.apply(Q, Kn, pos)
    assert torch.equal(a.extend(Q, Kn, V, [9, 4], rope=rope, pos=pos), b.extend(q1, k1, V, [9, 4]))
    with pytest.raises(ValueError):
        a.extend(Q, Kn, V, 9, rope=rope, pos=pos[:2].contiguous())
    assert a.check() == 0 and [int(x) for x in a.lengths()[0]] == [9, 4]


@pytest.mark.gpu
def test_positions_without_a_rope_are_refused():
    torch = pytest.importorskip("torch")
    K = _K()
    half = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.float16)   # noqa: E731
    pos = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    cache = K.KiviCache(1, 2, 64, max_tokens=100)
    with pytest.raises(ValueError):
        cache.extend(half(1, 4, 3, 64), half(1, 2, 3, 64), half(1, 2, 3, 64), 3, pos=pos)
    latent = K.LatentCache(1, 256, max_tokens=100)
    with pytest.raises(ValueError):
        latent.extend(half(1, 2, 3, 128), half(1, 2, 3, 64), half(1, 3, 256), half(1, 3, 64), 3, half(2, 128, 256), half(2, 128, 256),
                      pos=pos)
    assert int(cache.lengths()[0][0]) == 0 and int(latent.lengths()[0][0]) == 0
