"""Rotary positions (kivi_rope, kivi.Rope) against a 64-bit reference, and
their refusals."""
import ctypes

import numpy as np
import pytest

from tests import operators_ref as R


def _K():
    from bit_quantized_kv_quantize_gb300 import kivi as K
    return K


def _check(got, x, pos, rope, inverse=False):
    """One rounding to fp16 (2^-11 relative, 2^-25 in the subnormals) of a
    32-bit result whose sine and cosine are within 2^-22 (sincospi: 2^-23;
    the angle as a 32-bit float: pi 2^-25), three 32-bit roundings more:
    2^-21 (|x| + |y|) factor covers them."""
    rot = rope.rot_dim
    ref = R.rotate(x, pos, rope.inv_freq, rope.factor, rot, rope.interleaved, inverse)
    xa = np.abs(x.astype(np.float64))
    i0 = np.arange(0, rot, 2) if rope.interleaved else np.arange(rot // 2)
    i1 = i0 + 1 if rope.interleaved else i0 + rot // 2
    mag = np.zeros_like(xa)
    mag[:, i0] = mag[:, i1] = xa[:, i0] + xa[:, i1]
    bound = np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + abs(rope.factor) * mag * 2.0 ** -21
    assert np.all(np.abs(got.astype(np.float64) - ref) <= bound)
    assert np.array_equal(got[:, rot:], x[:, rot:])


# ---- host side ----------------------------------------------------------------

def test_frequencies():
    K = _K()
    f, m = K.rope_frequencies(128, 10000.0)
    assert m == 1.0 and f[0] == 1.0 and np.isclose(f[-1], 10000.0 ** (-126 / 128), rtol=1e-14)
    assert np.allclose(K.rope_frequencies(128, 1e4, "linear", 8.0)[0], f / 8)
    g, _ = K.rope_frequencies(128, 1e4, "ntk", 8.0)
    assert g[0] == 1.0 and np.isclose(g[-1], f[-1] / 8, rtol=1e-12)
    y, m = K.rope_frequencies(128, 1e4, "yarn", 4.0, 4096)
    assert np.isclose(m, 0.1 * np.log(4.0) + 1) and y[0] == f[0] and np.isclose(y[-1], f[-1] / 4)
    assert np.all(y <= f * (1 + 1e-15)) and np.all(y >= f / 4 * (1 - 1e-15))
    z, m = K.rope_frequencies(128, 5e5, "bands", 8.0, 8192)
    base = K.rope_frequencies(128, 5e5)[0]
    turns = 8192 * base / (2 * np.pi)
    assert m == 1.0 and np.allclose(z[turns > 4], base[turns > 4]) and np.allclose(z[turns < 1], base[turns < 1] / 8)
    for bad in (dict(rot_dim=7), dict(rot_dim=64, base=1.0), dict(rot_dim=64, scaling="other"),
                dict(rot_dim=64, factor=0.5), dict(rot_dim=2, scaling="ntk")):
        with pytest.raises(ValueError):
            K.rope_frequencies(**bad)


def test_turns_are_fixed_point_fractions():
    K = _K()
    r = K.Rope(64, inv_freq=[2 * np.pi * 0.25] + [0.0] * 30 + [-2 * np.pi * 0.25])
    assert int(r._turns[0]) == 2 ** 62 and int(r._turns[1]) == 0 and int(r._turns[31]) == 2 ** 64 - 2 ** 62
    with pytest.raises(ValueError):
        K.Rope(64, inv_freq=[1.0] * 31)
    with pytest.raises(ValueError):
        K.Rope(64, inv_freq=[np.nan] * 32)


def test_refusals_before_cuda():
    """The C entry refuses bad sizes and pointers before any CUDA call."""
    K = _K()
    p = ctypes.c_void_p(4096)   # never dereferenced: every call below is refused
    n, pos0 = np.array([1], np.int32), np.array([0], np.int32)
    turns = np.zeros(64, np.uint64)

    def call(q=p, k=p, b=1, hq=2, hk=1, ns=1, d=128, n=n, pos0=pos0, pos=None, turns=turns, rot=128, f=1.0, qo=p, ko=p):
        a = lambda x: None if x is None else x.ctypes.data   # noqa: E731
        return K.lib.kivi_rope(q, k, b, hq, hk, ns, d, a(n), a(pos0), pos, a(turns), rot, 0, f, 0, qo, ko, None)

    assert call(b=0) == 1 and call(ns=-1) == 1 and call(hq=0, hk=0) == 1 and call(hq=-1) == 1
    assert call(b=1025) == 2 and call(d=96) == 2 and call(rot=24) == 2 and call(rot=0) == 2 and call(rot=144) == 2
    assert call(n=None) == 1 and call(turns=None) == 1 and call(pos0=None) == 1 and call(pos=p) == 1
    assert call(n=np.array([2], np.int32)) == 1 and call(n=np.array([-1], np.int32)) == 1
    assert call(f=float("inf")) == 1 and call(f=float("nan")) == 1
    assert call(q=None) == 1 and call(ko=None) == 1 and call(qo=ctypes.c_void_p(4104)) == 1
    assert call(pos0=None, pos=ctypes.c_void_p(4097)) == 1
    assert call(n=np.array([0], np.int32)) == 0   # nothing to do


# ---- on the GPU -----------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("b,n,hq,hk,d,rot,interleaved", [
    (1, 1, 1, 1, 64, 64, False),
    (5, 1, 32, 8, 128, 128, False),
    (3, 7, 9, 3, 128, 96, True),
    (2, 33, 4, 1, 64, 16, False),
    (2, 100, 6, 2, 256, 256, True),
    (1, 517, 40, 8, 128, 64, True),
    (1, 1000, 3, 3, 256, 128, False),
])
def test_matches_reference(b, n, hq, hk, d, rot, interleaved):
    import torch
    K = _K()
    rng = np.random.default_rng(n)
    rope = K.Rope(d, rot_dim=rot, interleaved=interleaved, factor=1.25)
    q = rng.standard_normal((b, hq, n, d)).astype(np.float16)
    k = rng.standard_normal((b, hk, n, d)).astype(np.float16)
    first = rng.integers(0, 2_000_000, b)
    args = [torch.from_numpy(x).cuda() for x in (q, k)]
    if n == 1:
        args = [x.squeeze(2) for x in args]
    out = rope.apply(*args, first.tolist())
    inv = rope.apply(*args, first.tolist(), inverse=True)
    for x, y, z in zip((q, k), out, inv):
        y, z = (t.cpu().numpy().reshape(x.shape) for t in (y, z))
        for i in range(b):
            for h in range(x.shape[1]):
                pos = first[i] + np.arange(n)
                _check(y[i, h], x[i, h], pos, rope)
                _check(z[i, h], x[i, h], pos, rope, inverse=True)


@pytest.mark.gpu
def test_ragged_rows_positions_and_in_place():
    import torch
    K = _K()
    rng = np.random.default_rng(5)
    b, n, hq, hk, d = 4, 19, 5, 2, 64
    rope = K.Rope(d, rot_dim=32, interleaved=True, inv_freq=K.rope_frequencies(32, 5e5, "bands", 8.0)[0])
    q = rng.standard_normal((b, hq, n, d)).astype(np.float16)
    k = rng.standard_normal((b, hk, n, d)).astype(np.float16)
    lens = [0, 19, 1, 7]
    pos = rng.integers(-2 ** 31, 2 ** 31, (b, n)).astype(np.int32)   # any 32-bit position, in any order
    pos[1, :4] = [2 ** 31 - 1, -2 ** 31, 0, -1]
    qt, kt, pt = (torch.from_numpy(x).cuda() for x in (q, k, pos))
    qo, ko = torch.full_like(qt, 7.0), torch.full_like(kt, 7.0)
    got = rope.apply(qt, kt, pt, n=lens, q_out=qo, k_out=ko)
    assert got[0] is qo and got[1] is ko
    for x, y in ((q, qo.cpu().numpy()), (k, ko.cpu().numpy())):
        for i, m in enumerate(lens):
            assert np.all(y[i, :, m:] == 7.0)
            for h in range(x.shape[1]):
                _check(y[i, h, :m], x[i, h, :m], pos[i, :m], rope)
    new = rope.apply(qt, None, pt, n=lens)   # a new output is zero past the tokens
    assert torch.equal(new, torch.where(qo == 7.0, torch.zeros_like(qo), qo))
    rope.apply(qt, kt, pt, n=lens, q_out=qt, k_out=kt)
    for x, y, z in ((q, qt, qo), (k, kt, ko)):
        y, z = y.cpu().numpy(), z.cpu().numpy()
        for i, m in enumerate(lens):
            assert np.array_equal(y[i, :, :m], z[i, :, :m]) and np.array_equal(y[i, :, m:], x[i, :, m:])


@pytest.mark.gpu
def test_inverse_is_the_gradient():
    """<g, R x> = <R^T g, x>, and against differences of the linear map."""
    import torch
    K = _K()
    rng = np.random.default_rng(9)
    rope = K.Rope(128, rot_dim=64, factor=1.5)
    x = rng.standard_normal((1, 2, 11, 128)).astype(np.float16)
    g = rng.standard_normal((1, 2, 11, 128)).astype(np.float16)
    xt, gt = torch.from_numpy(x).cuda(), torch.from_numpy(g).cuda()
    y = rope.apply(xt, None, 123456).double().cpu().numpy()
    dx = rope.apply(gt, None, 123456, inverse=True).double().cpu().numpy()
    lhs, rhs = float((g.astype(np.float64) * y).sum()), float((dx * x.astype(np.float64)).sum())
    # each of 2816 products is off by at most 2^-11 |g y|; independent signs
    assert abs(lhs - rhs) <= 2.0 ** -11 * 4 * np.sqrt(2 * (g.astype(np.float64) ** 2 * y ** 2).sum())
    for c in (0, 5, 32, 63, 64, 127):   # d<g, R x>/dx_c by a unit step (the map is linear)
        e = np.zeros_like(x)
        e[0, 1, 4, c] = 1.0
        r = rope.apply(torch.from_numpy(e).cuda(), None, 123456).double().cpu().numpy()
        diff = float((g.astype(np.float64) * r).sum())
        assert abs(diff - dx[0, 1, 4, c]) <= 2.0 ** -11 * 4 * np.abs(g[0, 1, 4]).max() * 1.5


@pytest.mark.gpu
def test_streams_and_graph():
    import torch
    K = _K()
    rope = K.Rope(128)
    q, k = (torch.randn(2, h, 65, 128, device="cuda").half() for h in (8, 2))
    pos = torch.arange(130, dtype=torch.int32, device="cuda").view(2, 65).contiguous()
    ref = rope.apply(q, k, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = rope.apply(q, k, pos, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(side[0], ref[0]) and torch.equal(side[1], ref[1])
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope.apply(q, k, pos, q_out=qo, k_out=ko)
    pos += 1000   # a replay reads the positions of the moment
    g.replay()
    ref = rope.apply(q, k, [1000, 1065])
    assert torch.equal(qo, ref[0]) and torch.equal(ko, ref[1])


@pytest.mark.gpu
def test_binding_refusals():
    import torch
    K = _K()
    rope = K.Rope(128)
    q = torch.zeros(2, 4, 8, 128, device="cuda").half()
    for bad in (lambda: rope.apply(q.float(), None, 0), lambda: rope.apply(q.transpose(1, 2), None, 0),
                lambda: rope.apply(q[0, 0], None, 0), lambda: rope.apply(q, None, [0, 1, 2]),
                lambda: rope.apply(q, None, 0.5), lambda: rope.apply(q, None, 2 ** 31),
                lambda: rope.apply(q, None, torch.zeros(2, 8, device="cuda", dtype=torch.int64)),
                lambda: rope.apply(q, None, 0, n=9), lambda: rope.apply(q, q[:1], 0),
                lambda: K.Rope(128, rot_dim=24).apply(q, None, 0)):
        with pytest.raises((TypeError, ValueError, K.KiviError)):
            bad()
