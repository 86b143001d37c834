"""Thin Python binding of libkivi's C ABI (include/kivi.h).

Argument marshalling only: every step of the cache and of decode attention
runs in the library's CUDA kernels.  torch supplies device memory and the
current CUDA stream.  There is no fallback: if libkivi.so is missing or
fails to load, importing this module raises.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import math
import operator
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkivi.so")

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "capacity exceeded",
          4: "poisoned", 5: "CUDA error", 6: "out of memory"}

EXPORTS = ["kivi_cache_create", "kivi_cache_destroy", "kivi_prefill", "kivi_append",
           "kivi_decode_attn", "kivi_cache_lengths", "kivi_cache_export_sizes",
           "kivi_cache_export", "kivi_cache_check", "kivi_profile_enable", "kivi_profile_read",
           "kivi_decode_plan", "kivi_status_str", "kivi_last_error", "kivi_abi_version",
           "kivi_decode_attn_noalloc", "kivi_cache_export_records", "kivi_append_decode",
           "kivi_decode_attn_probs", "kivi_plan_preview", "kivi_prefill_attn", "kivi_prefill_attn_window",
           "kivi_decode_attn_window", "kivi_chunk_attn", "kivi_append_chunk", "kivi_rope"]


class KiviError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class CapacityError(KiviError):
    pass


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_int
    L.kivi_cache_create.argtypes = [i32] * 8 + [ctypes.POINTER(vp)]
    L.kivi_cache_destroy.argtypes = [vp]
    L.kivi_prefill.argtypes = [vp, vp, vp, vp, i32, vp]
    L.kivi_prefill_attn.argtypes = [vp, vp, vp, vp, vp, i32, i32, vp, vp]
    L.kivi_append.argtypes = [vp, vp, vp, vp]
    L.kivi_decode_attn.argtypes = [vp, vp, i32, vp, vp]
    L.kivi_decode_attn_probs.argtypes = [vp, vp, i32, vp, vp, vp, ctypes.c_int64, vp]
    L.kivi_prefill_attn_window.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp]
    L.kivi_decode_attn_window.argtypes = [vp, vp, i32, i32, i32, vp, vp]
    L.kivi_chunk_attn.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp]
    L.kivi_append_chunk.argtypes = [vp, vp, vp, vp, i32, vp]
    L.kivi_rope.argtypes = [vp, vp] + [i32] * 5 + [vp] * 4 + [i32, i32, ctypes.c_float, i32, vp, vp, vp]
    L.kivi_plan_preview.argtypes = [i32] * 9 + [vp, vp, vp, i32, vp]
    L.kivi_cache_lengths.argtypes = [vp, vp, vp, vp]
    L.kivi_cache_export_sizes.argtypes = [vp, ctypes.POINTER(ctypes.c_size_t)]
    L.kivi_cache_export.argtypes = [vp] * 8
    L.kivi_cache_check.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
    L.kivi_profile_enable.argtypes = [vp, i32]
    L.kivi_profile_read.argtypes = [vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i32)]
    L.kivi_decode_plan.argtypes = [vp, ctypes.POINTER(i32), ctypes.POINTER(i32)]
    L.kivi_status_str.restype = ctypes.c_char_p
    L.kivi_status_str.argtypes = [st]
    L.kivi_last_error.restype = ctypes.c_char_p
    for name in EXPORTS:
        f = getattr(L, name)
        if name not in ("kivi_status_str", "kivi_last_error"):
            f.restype = ctypes.c_int
    return L


lib = _load()


def _check(rc: int):
    if rc != 0:
        msg = lib.kivi_last_error().decode()
        raise (CapacityError if rc == 3 else KiviError)(rc, msg)


def _stream(stream):
    import torch
    if stream is None:   # the current stream's handle, without an object for it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _dev_f32_rows(x, lead, name):
    """Pointer of a contiguous CUDA fp32 tensor [*lead, ld]."""
    import torch
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype == torch.float32):
        raise TypeError(f"{name} must be a CUDA float32 tensor")
    if x.dim() != len(lead) + 1 or tuple(x.shape[:-1]) != tuple(lead) or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{', '.join(map(str, lead))}, ld] tensor")
    return x.data_ptr()


def _dev_fp16(x, shape, name):
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != torch.float16:
        raise TypeError(f"{name} must be a CUDA float16 tensor")
    if tuple(x.shape) != tuple(shape) or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got {tuple(x.shape)}")
    return ctypes.c_void_p(x.data_ptr())


def _on(stream):
    """Context in which torch allocates (and launches) on `stream`."""
    import torch
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _counts(n, b, name="n"):
    """Per-sequence counts (an integer or b of them) as an array of C ints."""
    if not isinstance(n, (int, list, tuple)) or isinstance(n, bool):
        a = np.asarray(n)
        if a.dtype.kind not in "iu" or a.ndim > 1:
            raise ValueError(f"{name} must be an integer or {b} integers")
        n = a.tolist()
    if isinstance(n, int):
        n = (n,) * b
    if len(n) != b:
        raise ValueError(f"{name} must be an integer or {b} integers")
    try:
        return array.array("i", n)
    except TypeError:
        raise ValueError(f"{name} must be an integer or {b} integers") from None
    except OverflowError:
        raise ValueError(f"{name} outside 32 bits") from None


def _visible(window, sinks):
    """A window and a number of sinks as C ints; those past 32 bits mean the
    same as the largest (or, negative, are refused alike)."""
    return tuple(max(-1, min(operator.index(x), 2**31 - 1)) for x in (window, sinks))


def _addr(a):
    """Address of an array.array's items."""
    return a.buffer_info()[0]


def _rows16(x, shape, dev, name):
    """Address of a contiguous CUDA fp16 tensor of this shape on device dev."""
    import torch
    if type(x) is not torch.Tensor and not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if x.dtype is not torch.float16 or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA float16 tensor")
    if x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}, got {tuple(x.shape)}")
    if x.get_device() != dev:
        raise ValueError(f"{name} must be on device cuda:{dev}")
    return x.data_ptr()


def rope_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, original_length=8192, beta_fast=32.0,
                     beta_slow=1.0, low=1.0, high=4.0):
    """Rotary frequencies (radians a position, float64 [rot_dim / 2]) and the
    factor on the rotated channels, for Rope.

    scaling: None, base ** (-2 m / rot_dim); "linear", divided by factor;
    "ntk", the base raised so that the lowest frequency is divided by factor;
    "yarn", divided by factor below beta_slow turns over original_length,
    kept above beta_fast, a linear ramp (in m) between, and the rotated part
    times 0.1 ln(factor) + 1; "bands", divided below `low` turns over
    original_length, kept above `high`, linear (in turns) between."""
    if rot_dim < 2 or rot_dim % 2 or not (base > 1 and factor >= 1):
        raise ValueError("need an even rot_dim >= 2, base > 1 and factor >= 1")
    m = np.arange(rot_dim // 2, dtype=np.float64)
    f = float(base) ** (-2.0 * m / rot_dim)
    if scaling is None:
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs rot_dim >= 4")
        return (base * factor ** (rot_dim / (rot_dim - 2))) ** (-2.0 * m / rot_dim), 1.0
    if scaling == "yarn":
        at = [rot_dim * math.log(original_length / (r * 2 * math.pi)) / (2 * math.log(base))
              for r in (beta_fast, beta_slow)]
        # (the ramp ends past the last pair where that turns more than beta_slow times)
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot_dim - 1)
        ramp = np.clip((m - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if scaling == "bands":
        if not high > low:
            raise ValueError("bands scaling needs high > low")
        keep = np.clip((original_length * f / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
        return f / factor * (1 - keep) + f * keep, 1.0
    raise ValueError(f"unknown scaling {scaling!r}")


class Rope:
    """Rotary positions for heads of dimension d: the first rot_dim channels
    (default all) turn, pairs (m, m + rot_dim / 2) or, interleaved, (2 m,
    2 m + 1), at the frequencies inv_freq (default base ** (-2 m / rot_dim);
    rope_frequencies has the long-context scalings) times factor."""

    def __init__(self, d, rot_dim=None, base=10000.0, interleaved=False, inv_freq=None, factor=1.0):
        self.d, self.rot_dim = d, d if rot_dim is None else rot_dim
        self.interleaved, self.factor = int(bool(interleaved)), float(factor)
        f = rope_frequencies(self.rot_dim, base)[0] if inv_freq is None else np.asarray(inv_freq, np.float64)
        if f.shape != (self.rot_dim // 2,) or not np.all(np.isfinite(f)):
            raise ValueError(f"inv_freq must be {self.rot_dim // 2} finite numbers")
        self.inv_freq = f.copy()
        # fractions of a turn, 2^64 = one turn
        self._turns = array.array("Q", [int(round(x / (2 * math.pi) * 2.0**64)) % 2**64 for x in f.tolist()])

    def apply(self, q, k, pos, n=None, q_out=None, k_out=None, inverse=False, stream=None):
        """Rotate q (CUDA fp16 [b, h_q, t, d] or [b, h_q, d]) and k (same with
        h_kv heads, or None).  pos: first position of each sequence (an
        integer or b integers), or every position (CUDA int32 [b, t]).  n:
        tokens of each sequence (default t; rows past them stay as they are in
        the outputs, zero in new ones).  inverse: the transposed map.  Returns
        (q_out, k_out), or q_out alone when k is None."""
        import torch
        if not isinstance(q, torch.Tensor) or q.dim() not in (3, 4):
            raise ValueError("q must be a [b, heads, t, d] or [b, heads, d] tensor")
        if not q.is_cuda:
            raise TypeError("q must be a CUDA float16 tensor")
        dev = q.get_device()
        if dev != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self.apply(q, k, pos, n, q_out, k_out, inverse, stream)
        shape, step = q.shape, q.dim() == 3
        b, hq, t = shape[0], shape[1], 1 if step else shape[2]
        hk = 0 if k is None else k.shape[1]
        qs = (b, hq, self.d) if step else (b, hq, t, self.d)
        ks = (b, hk, self.d) if step else (b, hk, t, self.d)
        qp, kp = _rows16(q, qs, dev, "q"), None if k is None else _rows16(k, ks, dev, "k")
        cnt = _counts(t if n is None else n, b)
        posp, pos0 = None, None
        if isinstance(pos, torch.Tensor) and pos.is_cuda:
            if pos.dtype is not torch.int32 or tuple(pos.shape) != (b, t) or not pos.is_contiguous() or pos.get_device() != dev:
                raise ValueError(f"pos must be a contiguous int32 tensor [{b}, {t}] on device cuda:{dev}")
            posp = pos.data_ptr()
        else:
            pos0 = _counts(pos, b, "pos")
        if q_out is None or (k_out is None and k is not None):
            new = torch.empty_like if n is None or min(cnt) == t else torch.zeros_like
            with _on(stream):
                q_out = new(q) if q_out is None else q_out
                k_out = new(k) if k_out is None and k is not None else k_out
        self._call(qp, kp, b, hq, hk, t, cnt, pos0, posp, inverse, _rows16(q_out, qs, dev, "q_out"),
                   None if k is None else _rows16(k_out, ks, dev, "k_out"), _stream(stream))
        return q_out if k is None else (q_out, k_out)

    def _call(self, qp, kp, b, hq, hk, t, cnt, pos0, posp, inverse, qo, ko, stream):
        _check(lib.kivi_rope(qp, kp, b, hq, hk, t, self.d, _addr(cnt), None if pos0 is None else _addr(pos0), posp,
                             _addr(self._turns), self.rot_dim, self.interleaved, self.factor, 1 if inverse else 0,
                             qo, ko, stream))


class KiviCache:
    """A KIVI quantized KV cache of b sequences x h_kv heads on the current GPU.

    Calls on one cache must not overlap on the GPU, on two streams or in two
    captured graphs replayed at once: those that only read it (decode,
    chunk_attn) share its buffers too."""

    def __init__(self, b, h_kv, d, k_bits=2, v_bits=2, G=32, R=128, max_tokens=4096):
        self.b, self.h_kv, self.d = b, h_kv, d
        self.k_bits, self.v_bits, self.G, self.R = k_bits, v_bits, G, R
        self.max_tokens = max_tokens
        self._h = ctypes.c_void_p()
        _check(lib.kivi_cache_create(b, h_kv, d, k_bits, v_bits, G, R, max_tokens,
                                     ctypes.byref(self._h)))
        import torch
        self._dev = torch.cuda.current_device()   # the handle's memory is there

    # -- lifecycle ---------------------------------------------------------
    def close(self):
        if self._h:
            h, self._h = self._h, ctypes.c_void_p()
            _check(lib.kivi_cache_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    # -- hot path ----------------------------------------------------------
    def prefill(self, K, V, t, stream=None):
        """K, V: CUDA fp16 [b, h_kv, t_stride, d]; t: per-sequence token counts."""
        t = np.ascontiguousarray(np.broadcast_to(np.asarray(t, np.int32), (self.b,)))
        ts = K.shape[2]
        kp = _dev_fp16(K, (self.b, self.h_kv, ts, self.d), "K")
        vp = _dev_fp16(V, (self.b, self.h_kv, ts, self.d), "V")
        _check(lib.kivi_prefill(self._h, kp, vp, t.ctypes.data, ts, _stream(stream)))

    def _here(self, *tensors):
        """The tensors are on the cache's device."""
        if any(x is not None and x.device.index != self._dev for x in tensors):
            raise ValueError(f"tensors must be on the cache's device cuda:{self._dev}")

    def prefill_attn(self, Q, K, V, t, out=None, stream=None, window=0, sinks=0):
        """prefill(K, V, t) and the prompt's causal attention: Q CUDA fp16
        [b, h_q, t_stride, d] -> out (same shape; rows past each sequence's
        length untouched).  One launch.  With window > 0 a query sees only the
        last `window` tokens up to its own and the sequence's first `sinks`
        (several launches)."""
        import torch
        t = np.ascontiguousarray(np.broadcast_to(np.asarray(t, np.int32), (self.b,)))
        ts, hq = K.shape[2], Q.shape[1]
        qp = _dev_fp16(Q, (self.b, hq, ts, self.d), "Q")
        kp = _dev_fp16(K, (self.b, self.h_kv, ts, self.d), "K")
        vp = _dev_fp16(V, (self.b, self.h_kv, ts, self.d), "V")
        if out is None:
            with _on(stream):
                out = torch.zeros_like(Q)
        op = _dev_fp16(out, (self.b, hq, ts, self.d), "out")
        if window or sinks:
            self._here(Q, K, V, out)
            _check(lib.kivi_prefill_attn_window(self._h, qp, kp, vp, t.ctypes.data, ts, hq, *_visible(window, sinks), op,
                                                _stream(stream)))
        else:
            _check(lib.kivi_prefill_attn(self._h, qp, kp, vp, t.ctypes.data, ts, hq, op, _stream(stream)))
        return out

    def _chunk(self, K, V, n):
        """Addresses of a chunk's keys and values, its counts and stride."""
        if K.dim() != 4:
            raise ValueError("K must be [b, h_kv, n_stride, d]")
        shape = (self.b, self.h_kv, K.shape[2], self.d)
        return (_rows16(K, shape, self._dev, "K"), _rows16(V, shape, self._dev, "V"), _counts(n, self.b),
                K.shape[2])

    def _chunk_out(self, Q, ns, out, stream):
        """Address of a chunk's queries, its output (a new one is zero) and that's address."""
        import torch
        if Q.dim() != 4:
            raise ValueError("Q must be [b, h_q, n_stride, d]")
        shape = (self.b, Q.shape[1], ns, self.d)
        qp = _rows16(Q, shape, self._dev, "Q")
        if out is None:
            with _on(stream):
                out = torch.zeros_like(Q)
        return qp, out, _rows16(out, shape, self._dev, "out")

    def chunk_attn(self, Q, K, V, n, window=0, sinks=0, out=None, stream=None):
        """Attention of n new tokens of each sequence (an integer or b of
        them) over the cache and the chunk itself: Q CUDA fp16 [b, h_q, ns, d],
        K and V [b, h_kv, ns, d] -> out (rows past n untouched, zero in a new
        tensor).  Does not append (append_chunk, extend)."""
        kp, vp, cnt, ns = self._chunk(K, V, n)
        qp, out, op = self._chunk_out(Q, ns, out, stream)
        _check(lib.kivi_chunk_attn(self._h, qp, kp, vp, _addr(cnt), ns, Q.shape[1], *_visible(window, sinks), op,
                                   _stream(stream)))
        return out

    def append_chunk(self, K, V, n, stream=None):
        """Append n tokens of each sequence (an integer or b of them; K, V CUDA
        fp16 [b, h_kv, ns, d]): n one-token appends in one call."""
        kp, vp, cnt, ns = self._chunk(K, V, n)
        _check(lib.kivi_append_chunk(self._h, kp, vp, _addr(cnt), ns, _stream(stream)))

    def extend(self, Q, K, V, n, window=0, sinks=0, rope=None, out=None, stream=None):
        """Take the next chunk of every sequence: rotate its queries and keys
        at the positions behind the cached tokens (rope: a Rope, or None),
        attend (chunk_attn; returns its out) and append it (append_chunk)."""
        import torch
        if torch.cuda.current_device() != self._dev:   # (before the rotation, which runs on the current one)
            raise KiviError(1, f"the cache belongs to device {self._dev}, which is not current")
        kp, vp, cnt, ns = self._chunk(K, V, n)
        win, snk = _visible(window, sinks)
        T = array.array("i", bytes(4 * self.b))
        _check(lib.kivi_cache_lengths(self._h, _addr(T), None, None))
        for i in range(self.b):
            if cnt[i] > self.max_tokens - T[i]:
                raise CapacityError(3, f"sequence {i} would exceed max_tokens")
        qp, out, op = self._chunk_out(Q, ns, out, stream)
        hq, st, cp = Q.shape[1], _stream(stream), _addr(cnt)
        if rope is not None:
            if rope.d != self.d:
                raise ValueError(f"rope is for heads of dimension {rope.d}")
            with _on(stream):   # rows past n are not read
                rq, rk = torch.empty_like(Q), torch.empty_like(K)
            rope._call(qp, kp, self.b, hq, self.h_kv, ns, cnt, T, None, False, rq.data_ptr(), rk.data_ptr(), st)
            qp, kp = rq.data_ptr(), rk.data_ptr()
        _check(lib.kivi_chunk_attn(self._h, qp, kp, vp, cp, ns, hq, win, snk, op, st))
        _check(lib.kivi_append_chunk(self._h, kp, vp, cp, ns, st))
        return out

    def append(self, k, v, stream=None):
        """k, v: CUDA fp16 [b, h_kv, d]."""
        kp = _dev_fp16(k, (self.b, self.h_kv, self.d), "k")
        vp = _dev_fp16(v, (self.b, self.h_kv, self.d), "v")
        _check(lib.kivi_append(self._h, kp, vp, _stream(stream)))

    def decode(self, q, out=None, stream=None, window=0, sinks=0):
        """q: CUDA fp16 [b, h_q, d] -> out CUDA fp16 [b, h_q, d].  With
        window > 0 the query sees only the last `window` tokens and the
        sequence's first `sinks`."""
        import torch
        hq = q.shape[1]
        qp = _dev_fp16(q, (self.b, hq, self.d), "q")
        if out is None:
            with _on(stream):
                out = torch.empty_like(q)
        op = _dev_fp16(out, (self.b, hq, self.d), "out")
        if window or sinks:
            self._here(q, out)
            _check(lib.kivi_decode_attn_window(self._h, qp, hq, *_visible(window, sinks), op, _stream(stream)))
        else:
            _check(lib.kivi_decode_attn(self._h, qp, hq, op, _stream(stream)))
        return out

    def decode_probs(self, q, probs, mass=None, out=None, stream=None):
        """decode(q), and each token's softmax weight into probs (CUDA fp32
        [b, h_q, ld], ld >= every sequence's length; entries past a
        sequence's length untouched); mass (same shape, optional) += probs.
        Returns out."""
        import torch
        hq = q.shape[1]
        qp = _dev_fp16(q, (self.b, hq, self.d), "q")
        if out is None:
            out = torch.empty_like(q)
        op = _dev_fp16(out, (self.b, hq, self.d), "out")
        pp = _dev_f32_rows(probs, (self.b, hq), "probs")
        mp = 0
        if mass is not None:
            if tuple(mass.shape) != tuple(probs.shape):
                raise ValueError("mass must have the shape of probs")
            mp = _dev_f32_rows(mass, (self.b, hq), "mass")
        _check(lib.kivi_decode_attn_probs(self._h, qp, hq, op, pp, mp or None, probs.shape[2],
                                          _stream(stream)))
        return out

    def append_decode(self, k, v, q, out=None, stream=None):
        """append(k, v) then decode(q) in one call; returns out.

        One launch where the decode kernel appends the token itself (see
        kivi_append_decode in kivi.h for when), else the append kernel and
        the decode kernel as its programmatic dependent."""
        import torch
        hq = q.shape[1]
        kp = _dev_fp16(k, (self.b, self.h_kv, self.d), "k")
        vp = _dev_fp16(v, (self.b, self.h_kv, self.d), "v")
        qp = _dev_fp16(q, (self.b, hq, self.d), "q")
        if out is None:
            out = torch.empty_like(q)
        op = _dev_fp16(out, (self.b, hq, self.d), "out")
        _check(lib.kivi_append_decode(self._h, kp, vp, qp, hq, op, _stream(stream)))
        return out

    # -- inspection ----------------------------------------------------------
    def lengths(self):
        T = np.zeros(self.b, np.int32)
        Tqk = np.zeros(self.b, np.int32)
        Tqv = np.zeros(self.b, np.int32)
        _check(lib.kivi_cache_lengths(self._h, T.ctypes.data, Tqk.ctypes.data, Tqv.ctypes.data))
        return T, Tqk, Tqv

    def export(self, stream=None):
        """The whole device state in the packed format (host numpy arrays)."""
        sz = (ctypes.c_size_t * 6)()
        _check(lib.kivi_cache_export_sizes(self._h, sz))
        dt = [np.uint32, np.uint16, np.uint32, np.uint16, np.uint16, np.uint16]
        arrs = [np.zeros(int(n) // np.dtype(t).itemsize, t) for n, t in zip(sz, dt)]
        _check(lib.kivi_cache_export(self._h, *[a.ctypes.data for a in arrs], _stream(stream)))
        return dict(zip(["Kc", "Ksz", "Vc", "Vsz", "Kf", "Vf"], arrs))

    def export_records(self, stream=None) -> np.ndarray:
        """The packed arrays as the device stores them (block records, uint8)."""
        n = ctypes.c_size_t(0)
        _check(lib.kivi_cache_export_records(self._h, None, ctypes.byref(n), _stream(stream)))
        buf = np.zeros(int(n.value), np.uint8)
        _check(lib.kivi_cache_export_records(self._h, buf.ctypes.data, ctypes.byref(n), _stream(stream)))
        return buf

    def check(self, stream=None) -> int:
        f = ctypes.c_uint32(0)
        _check(lib.kivi_cache_check(self._h, ctypes.byref(f), _stream(stream)))
        return int(f.value)

    def profile(self, on: bool):
        _check(lib.kivi_profile_enable(self._h, 1 if on else 0))

    def profile_read(self):
        ms = ctypes.c_double(0)
        n = ctypes.c_int(0)
        _check(lib.kivi_profile_read(self._h, ctypes.byref(ms), ctypes.byref(n)))
        return float(ms.value), int(n.value)

    def plan(self):
        s = ctypes.c_int(0)
        n = ctypes.c_int(0)
        _check(lib.kivi_decode_plan(self._h, ctypes.byref(s), ctypes.byref(n)))
        return int(s.value), int(n.value)
