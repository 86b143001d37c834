"""Which warp of a latent cache's append reads and writes which place of the ring
(csrc/kivi_latent_places.h, the kernel's own lines, compiled for the host): a place
is one warp's, and every token that leaves the window is quantized once, from its
own place; the places of a new block that hold no tokens yet are zeroed."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_kv_quantize_gb300", "csrc")
SHIM = """
#include "kivi_latent_places.h"
extern "C" int moves(int T, int n, int R, int W, int *out) {   // [warps][3]
    const int warps = lat_end(T, n) - T;
    for (int x = 0; x < warps; ++x) {
        const LatMoves m = lat_moves(T, n, R, W, x);
        out[3 * x] = m.own;
        out[3 * x + 1] = m.under;
        out[3 * x + 2] = m.codes;
    }
    return warps;
}
extern "C" int restored(int T, int n, int R, int o) { return lat_restored(T, n, R, o); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("places")
    src, so = d / "places.cpp", d / "places.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def _ring(R):
    return ((R + 127) // 128 + 1) * 128


def _walk(lib, T, n, R):
    """The append of n tokens to T: who touches each place, what is quantized from
    where, and the ring as it is afterwards (place -> token)."""
    W = _ring(R)
    out = (ctypes.c_int * (3 * (n + 128)))()
    warps = lib.moves(T, n, R, W, out)
    Tq, Tq1, B = max(0, T - R), max(0, T + n - R), max(0, T + n - R) // 128 * 128
    reads, writes, coded = {}, {}, []
    ring = {o % W: o for o in range(Tq // 128 * 128, T)}
    stored = {}

    def leave(x, o):
        assert Tq <= o < min(T, Tq1), (x, o)          # a cached token that leaves the window
        reads.setdefault(o % W, set()).add(x)
        coded.append(o)
        if lib.restored(T, n, R, o):
            write(x, o)

    def write(x, o):
        writes.setdefault(o % W, set()).add(x)
        assert stored.setdefault(o % W, o) == o       # (no two tokens into one place)

    for x in range(warps):
        own, under, codes = out[3 * x:3 * x + 3]
        if own >= 0:
            leave(x, own)
        if under >= 0:
            leave(x, under)
        tau = T + x
        assert codes == (tau < Tq1)
        if codes:
            coded.append(tau)
        if not codes or lib.restored(T, n, R, tau):
            write(x, tau)
    shared = [p for p, w in writes.items() if len(w | reads.get(p, set())) > 1]
    assert not shared, f"T {T}, n {n}, R {R}: {len(shared)} places of several warps, such as {shared[0]}"
    assert sorted(coded) == list(range(Tq, Tq1)), f"T {T}, n {n}, R {R}: quantized {len(coded)} of {Tq1 - Tq}"
    ring.update(stored)
    assert all(ring[o % W] == o for o in range(B, T + n)), f"T {T}, n {n}, R {R}: a block is not whole"
    last = (T + n - 1) // 128 * 128                   # (a block begun before: by the append that did)
    assert all(stored.get(f % W) == f for f in range(T + n, last + 128)) == (last >= T or (T + n) % 128 == 0)


@pytest.mark.parametrize("R", [64, 128, 192, 256, 1024])
def test_a_place_is_one_warps(lib, R):
    W = _ring(R)
    rng = random.Random(R)
    ends = [0, 1, 63, 64, 65, 127, 128, 129, R - 1, R, R + 1, W - 1, W, W + 1, W + 127, 2 * W, 2 * W + 77, 100, 2000]
    sizes = [1, 2, 63, 64, 127, 128, 129, R, R + 1, W - 128, W - 1, W, W + 1, W + 60, 2 * W, 3 * W + 5, 300, 500]
    for T in ends:
        for n in sizes:
            _walk(lib, T, n, R)
    for _ in range(400):
        _walk(lib, rng.randrange(4 * W), rng.randrange(1, 3 * W), R)
