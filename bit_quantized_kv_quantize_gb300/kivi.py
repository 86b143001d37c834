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
           "kivi_decode_attn_window", "kivi_chunk_attn", "kivi_append_chunk", "kivi_rope",
           "kivi_rope_axes", "kivi_verify", "kivi_latent_create", "kivi_latent_destroy", "kivi_latent_prefill",
           "kivi_latent_append", "kivi_latent_attn", "kivi_latent_lengths", "kivi_latent_restore",
           "kivi_latent_check", "kivi_latent_rows", "kivi_latent_expanded_attn", "kivi_head_product",
           "kivi_latent_prompt_attn", "kivi_latent_product", "kivi_latent_expanded", "kivi_device_check"]


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
    L.kivi_rope_axes.argtypes = [vp, vp] + [i32] * 5 + [vp, vp, i32, vp, vp, i32, i32, ctypes.c_float, i32, vp, vp, vp]
    L.kivi_verify.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp]
    L.kivi_latent_create.argtypes = [i32] * 6 + [ctypes.POINTER(vp)]
    L.kivi_latent_destroy.argtypes = [vp]
    L.kivi_latent_prefill.argtypes = L.kivi_latent_append.argtypes = [vp, vp, vp, vp, i32, vp]
    L.kivi_latent_attn.argtypes = [vp] * 6 + [i32, i32, ctypes.c_float, vp, vp]
    L.kivi_latent_lengths.argtypes = [vp, vp, vp]
    L.kivi_latent_restore.argtypes = [vp, vp, vp, i32, vp]
    L.kivi_latent_check.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
    L.kivi_head_product.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, i32, i32, vp, vp]
    L.kivi_latent_prompt_attn.argtypes = [vp] * 5 + [i32, i32, vp, i32, ctypes.c_float, vp, vp]
    L.kivi_latent_rows.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, vp]
    L.kivi_latent_expanded_attn.argtypes = [vp] * 5 + [i32, i32, vp, vp, i32, i32, ctypes.c_float, vp, vp]
    L.kivi_latent_product.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, i32, i32, vp, vp]
    L.kivi_latent_expanded.argtypes = [vp] * 6 + [i32, vp, vp, i32, i32, ctypes.c_float, vp, vp]
    L.kivi_device_check.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
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
    if isinstance(n, array.array):
        n = n.tolist()
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


def _rows(x, shape, dtype, dev, name):
    """Address of a contiguous CUDA tensor of this shape and type on device dev."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype is not dtype:
        raise TypeError(f"{name} must be a CUDA {str(dtype)[6:]} tensor")
    if tuple(x.shape) != tuple(shape) or not x.is_contiguous():
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


def rope_axes(sections, in_turn=False):
    """The axis of each channel pair for Rope: sections[a] pairs turn by axis a,
    one section after another, or, in_turn, dealt to the axes in turn while they
    last (0, 1, 2, 0, 1, 2, ...)."""
    left = [operator.index(x) for x in sections]
    if not left or min(left) < 0 or sum(left) < 1:
        raise ValueError("sections must be numbers of pairs")
    if not in_turn:
        return [a for a, k in enumerate(left) for _ in range(k)]
    return [a for k in range(max(left)) for a, m in enumerate(left) if k < m]


class Rope:
    """Rotary positions for heads of dimension d: the first rot_dim channels
    (default all) turn, pairs (m, m + rot_dim / 2) or, interleaved, (2 m,
    2 m + 1), at the frequencies inv_freq (default base ** (-2 m / rot_dim);
    rope_frequencies has the long-context scalings) times factor.  axes: the
    axis of each pair's position (rot_dim / 2 numbers from 0 on; rope_axes makes
    the usual ones), for tokens that stand on several."""

    def __init__(self, d, rot_dim=None, base=10000.0, interleaved=False, inv_freq=None, factor=1.0, axes=None):
        self.d, self.rot_dim = d, d if rot_dim is None else rot_dim
        self.interleaved, self.factor = int(bool(interleaved)), float(factor)
        f = rope_frequencies(self.rot_dim, base)[0] if inv_freq is None else np.asarray(inv_freq, np.float64)
        if f.shape != (self.rot_dim // 2,) or not np.all(np.isfinite(f)):
            raise ValueError(f"inv_freq must be {self.rot_dim // 2} finite numbers")
        self.inv_freq = f.copy()
        self.axes = None
        if axes is not None:
            a = [operator.index(x) for x in axes]
            if len(a) != self.rot_dim // 2 or min(a) < 0 or max(a) > 254:
                raise ValueError(f"axes must be {self.rot_dim // 2} numbers from 0 to 254")
            self.axes, self._axis = max(a) + 1, array.array("B", a)
        # fractions of a turn, 2^64 = one turn
        self._turns = array.array("Q", [int(round(x / (2 * math.pi) * 2.0**64)) % 2**64 for x in f.tolist()])

    def apply(self, q, k, pos, n=None, q_out=None, k_out=None, inverse=False, stream=None):
        """Rotate q (CUDA fp16 [b, h_q, t, d] or [b, h_q, d]) and k (same with
        h_kv heads, or None).  pos: first position of each sequence (an
        integer or b integers), or every position (CUDA int32 [b, t], with
        axes [axes, b, t]; a first position stands on every axis).  n: tokens of each sequence (default t; rows past them stay as they are in
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
            posp = self._pos(pos, b, t, dev)
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

    def _pos(self, pos, b, t, dev):
        """Address of every token's position."""
        import torch
        shape = (b, t) if self.axes is None else (self.axes, b, t)
        if pos.dtype is not torch.int32 or tuple(pos.shape) != shape or not pos.is_contiguous() or pos.get_device() != dev:
            raise ValueError(f"pos must be a contiguous int32 tensor {list(shape)} on device cuda:{dev}")
        return pos.data_ptr()

    def _call(self, qp, kp, b, hq, hk, t, cnt, pos0, posp, inverse, qo, ko, stream):
        if posp is not None and self.axes is not None:
            _check(lib.kivi_rope_axes(qp, kp, b, hq, hk, t, self.d, _addr(cnt), posp, self.axes, _addr(self._axis),
                                      _addr(self._turns), self.rot_dim, self.interleaved, self.factor,
                                      1 if inverse else 0, qo, ko, stream))
            return
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

    def extend(self, Q, K, V, n, window=0, sinks=0, rope=None, out=None, stream=None, pos=None):
        """Take the next chunk of every sequence: rotate its queries and keys
        at the positions behind the cached tokens (rope: a Rope, or None; or at
        pos, as Rope.apply takes every position), attend (chunk_attn; returns
        its out) and append it (append_chunk)."""
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
        if rope is None and pos is not None:
            raise ValueError("positions without a rope")
        if rope is not None:
            if rope.d != self.d:
                raise ValueError(f"rope is for heads of dimension {rope.d}")
            posp = None if pos is None else rope._pos(pos, self.b, ns, self._dev)
            with _on(stream):   # rows past n are not read
                rq, rk = torch.empty_like(Q), torch.empty_like(K)
            rope._call(qp, kp, self.b, hq, self.h_kv, ns, cnt, T if posp is None else None, posp, False, rq.data_ptr(),
                       rk.data_ptr(), st)
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


def verify(p, q, draft, u, n=None, tokens=None, accepted=None, stream=None):
    """Verification of drafted tokens (kivi_verify): p CUDA fp32 or fp16 [b, ns +
    1, vocab], the target's probabilities; q [b, ns, vocab] of the same type, the
    draft's, or None where each drafted token was certain; draft CUDA int32 [b,
    ns]; u CUDA fp32 [b, ns + 1], uniform in [0, 1); n: drafted tokens of each
    sequence (an integer or b of them, default ns).  Returns tokens (int32 [b, ns
    + 1]: those kept, the one drawn behind them, then -1) and accepted (int32 [b]:
    how many were kept)."""
    import torch
    if not isinstance(p, torch.Tensor) or p.dim() != 3 or p.shape[1] < 1:
        raise ValueError("p must be a [b, ns + 1, vocab] tensor")
    if not p.is_cuda or p.dtype not in (torch.float32, torch.float16):
        raise TypeError("p must be a CUDA float32 or float16 tensor")
    dev = p.get_device()
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return verify(p, q, draft, u, n, tokens, accepted, stream)
    b, ns, V = p.shape[0], p.shape[1] - 1, p.shape[2]
    cnt = _counts(ns if n is None else n, b)
    args = [_rows(p, p.shape, p.dtype, dev, "p"), None if q is None else _rows(q, (b, ns, V), p.dtype, dev, "q"),
            p.element_size(), _rows(draft, (b, ns), torch.int32, dev, "draft"),
            _rows(u, (b, ns + 1), torch.float32, dev, "u")]
    if tokens is None or accepted is None:
        with _on(stream):
            tokens = torch.empty((b, ns + 1), dtype=torch.int32, device=p.device) if tokens is None else tokens
            accepted = torch.empty((b,), dtype=torch.int32, device=p.device) if accepted is None else accepted
    _check(lib.kivi_verify(*args, b, ns, V, _addr(cnt), _rows(tokens, (b, ns + 1), torch.int32, dev, "tokens"),
                           _rows(accepted, (b,), torch.int32, dev, "accepted"), _stream(stream)))
    return tokens, accepted


def device_check(stream=None) -> int:
    """The current device's status word of the calls without a handle
    (kivi_device_check): head_product, latent_prompt_attn."""
    f = ctypes.c_uint32(0)
    _check(lib.kivi_device_check(ctypes.byref(f), _stream(stream)))
    return int(f.value)


LATENT_HEAD, LATENT_ROPE = 128, 64   # channels of a head without positions (and of its values), of the rotary key


def head_product(x, w, n=None, transposed=False, out=None, stream=None):
    """A matrix of each head times its rows (kivi_head_product): x CUDA fp16 [b,
    h, t, K] or [b, t, K] (rows of all heads alike), w [h, N, K] or, transposed,
    [h, K, N] -> out [b, h, t, N] (rows past n untouched, zero in a new tensor)."""
    import torch
    if not isinstance(x, torch.Tensor) or not isinstance(w, torch.Tensor) or x.dim() not in (3, 4) or w.dim() != 3:
        raise ValueError("x must be [b, h, t, K] or [b, t, K], w [h, N, K]")
    if not x.is_cuda:
        raise TypeError("x must be a CUDA float16 tensor")
    dev = x.get_device()
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return head_product(x, w, n, transposed, out, stream)
    b, t, K, h = x.shape[0], x.shape[-2], x.shape[-1], w.shape[0]
    N = w.shape[2] if transposed else w.shape[1]
    hx = 1 if x.dim() == 3 else h
    xp = _rows16(x, (b, t, K) if x.dim() == 3 else (b, h, t, K), dev, "x")
    wp = _rows16(w, (h, K, N) if transposed else (h, N, K), dev, "w")
    cnt = _counts(t if n is None else n, b)
    if out is None:
        with _on(stream):
            out = (torch.empty if n is None or min(cnt) == t else torch.zeros)((b, h, t, N), dtype=x.dtype, device=x.device)
    _check(lib.kivi_head_product(xp, wp, b, hx, h, t, _addr(cnt), K, N, 1 if transposed else 0,
                                 _rows16(out, (b, h, t, N), dev, "out"), _stream(stream)))
    return out


def _latent_args(qn, qr, c, kr, wk, wv, out, stream, dev):
    """Checks of a latent call's tensors: (b, h, t, r) and their addresses."""
    import torch
    if any(not isinstance(x, torch.Tensor) for x in (qn, qr, c, kr, wk, wv)):
        raise TypeError("queries, latent vectors and weights must be tensors")
    if qn.dim() != 4 or c.dim() != 3:
        raise ValueError("qn must be [b, h, t, 128] and c [b, t, r]")
    (b, h, t, _), r = qn.shape, c.shape[2]
    qnp, qrp = _rows16(qn, (b, h, t, LATENT_HEAD), dev, "qn"), _rows16(qr, (b, h, t, LATENT_ROPE), dev, "qr")
    cp, krp = _rows16(c, (b, t, r), dev, "c"), _rows16(kr, (b, t, LATENT_ROPE), dev, "kr")
    wkp, wvp = _rows16(wk, (h, LATENT_HEAD, r), dev, "wk"), _rows16(wv, (h, LATENT_HEAD, r), dev, "wv")
    if out is None:
        with _on(stream):
            out = torch.zeros_like(qn)
    return (b, h, t, r), (qnp, qrp, cp, krp, wkp, wvp, _rows16(out, (b, h, t, LATENT_HEAD), dev, "out")), out


def _space(stream, dev, *halves):
    """A workspace of several fp16 arrays: the tensor that holds it (kept until the
    calls that use it are issued) and their addresses.  (One allocation: each takes
    longer than a call's checks.)"""
    import torch
    at = [0]
    for n in halves:
        at.append(at[-1] + (n + 127) // 128 * 128)
    with _on(stream):
        t = torch.empty(at[-1], dtype=torch.float16, device=dev)
    p = t.data_ptr()
    return t, [p + 2 * a for a in at[:-1]]


def _latent_scale(scale):
    return 1.0 / math.sqrt(LATENT_HEAD + LATENT_ROPE) if scale is None else float(scale)


def latent_prompt_attn(qn, qr, c, kr, t, wk, wv, scale=None, out=None, stream=None):
    """Latent attention of prompts, expanded: every head's keys and values are
    formed (head_product) and attended to causally (kivi_latent_prompt_attn).  qn
    CUDA fp16 [b, h, ts, 128], qr [b, h, ts, 64] (rotated), c [b, ts, r], kr [b,
    ts, 64] (rotated), wk and wv [h, 128, r], t tokens of each sequence -> out [b,
    h, ts, 128] (rows past t untouched, zero in a new tensor).  scale: default 1 /
    sqrt(192).  Keys and values are fp16: wk c and wv c must stay below 65504."""
    import torch
    if not isinstance(qn, torch.Tensor) or not qn.is_cuda:
        raise TypeError("qn must be a CUDA float16 tensor")
    dev = qn.get_device()
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return latent_prompt_attn(qn, qr, c, kr, t, wk, wv, scale, out, stream)
    dims, ptrs, out = _latent_args(qn, qr, c, kr, wk, wv, out, stream, dev)
    (b, h, ts, r), (qnp, qrp, cp, krp, wkp, wvp, op) = dims, ptrs
    cnt, scale, st = _counts(t, b, "t"), _latent_scale(scale), _stream(stream)
    keep, (K, V) = _space(stream, qn.device, *[b * h * ts * LATENT_HEAD] * 2)   # (rows past t are not read)
    for w, x in ((wkp, K), (wvp, V)):
        _check(lib.kivi_head_product(cp, w, b, 1, h, ts, _addr(cnt), r, LATENT_HEAD, 0, x, st))
    _check(lib.kivi_latent_prompt_attn(qnp, qrp, K, krp, V, b, h, _addr(cnt), ts, scale, op, st))
    return out


class LatentCache:
    """A quantized cache of latent vectors for b sequences on the current GPU:
    one vector c [r] a token (r 256 or 512), from which every head's keys and
    values are products, and one rotary key kr [64].  The newest R tokens (a
    multiple of 64) are fp16, older ones quantized to `bits` in groups of G
    channels of a token.

    Calls on one cache must not overlap on the GPU, as for KiviCache."""

    def __init__(self, b, r, bits=4, G=32, R=128, max_tokens=4096):
        self.b, self.r, self.bits, self.G, self.R, self.max_tokens = b, r, bits, G, R, max_tokens
        self._h = ctypes.c_void_p()
        _check(lib.kivi_latent_create(b, r, bits, G, R, max_tokens, ctypes.byref(self._h)))
        import torch
        self._dev = torch.cuda.current_device()   # the handle's memory is there
        self._device = torch.device("cuda", self._dev)
        self._sms = torch.cuda.get_device_properties(self._dev).multi_processor_count

    def close(self):
        if self._h:
            h, self._h = self._h, ctypes.c_void_p()
            _check(lib.kivi_latent_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def _tokens(self, c, kr, n, name="n"):
        """Addresses of new tokens' rows, their counts and stride."""
        import torch
        if not isinstance(c, torch.Tensor) or c.dim() != 3:
            raise ValueError(f"c must be a [b, {name}, r] tensor")
        ns = c.shape[1]
        return (_rows16(c, (self.b, ns, self.r), self._dev, "c"),
                _rows16(kr, (self.b, ns, LATENT_ROPE), self._dev, "kr"), _counts(n, self.b, name), ns)

    def _here(self):
        import torch
        if torch.cuda.current_device() != self._dev:   # (before anything is launched)
            raise KiviError(1, f"the latent cache belongs to device {self._dev}, which is not current")

    def prefill(self, c, kr, t, stream=None):
        """Every sequence anew, with its first t tokens (an integer or b of them):
        c CUDA fp16 [b, ts, r], kr [b, ts, 64]."""
        cp, krp, cnt, ts = self._tokens(c, kr, t, "t")
        _check(lib.kivi_latent_prefill(self._h, cp, krp, _addr(cnt), ts, _stream(stream)))

    def append(self, c, kr, n, stream=None):
        """n more tokens of each sequence (an integer or b of them)."""
        cp, krp, cnt, ns = self._tokens(c, kr, n)
        _check(lib.kivi_latent_append(self._h, cp, krp, _addr(cnt), ns, _stream(stream)))

    def attn_latent(self, ql, qr, c, kr, n, scale=None, out=None, stream=None):
        """The absorbed attention itself (kivi_latent_attn): ql CUDA fp16 [b, h,
        ns, r], qr [b, h, ns, 64] -> out [b, h, ns, r] (rows past n untouched,
        zero in a new tensor)."""
        import torch
        if not isinstance(ql, torch.Tensor) or ql.dim() != 4:
            raise ValueError("ql must be a [b, h, ns, r] tensor")
        cp, krp, cnt, ns = self._tokens(c, kr, n)
        h = ql.shape[1]
        shape = (self.b, h, ns, self.r)
        qlp, qrp = _rows16(ql, shape, self._dev, "ql"), _rows16(qr, (self.b, h, ns, LATENT_ROPE), self._dev, "qr")
        if out is None:
            with _on(stream):
                out = torch.zeros_like(ql)
        _check(lib.kivi_latent_attn(self._h, qlp, qrp, cp, krp, _addr(cnt), ns, h, _latent_scale(scale),
                                    _rows16(out, shape, self._dev, "out"), _stream(stream)))
        return out

    def _form(self, form, cnt, T, h, ns):
        """Whether attn forms every head's keys and values (expanded) rather than
        absorbing them, and the longest sequence with its new tokens.

        None, the faster by these times on a GB300 (us; r = 512, at 256 0.55 and 0.67
        of the second terms): absorbed 35 and one for 250,000 (query, head, token);
        expanded 10, one for 2,800 (token, head), and 0.8 for 64 tokens while every SM
        has a row tile of 256 queries of a head, or a share of one, with 3 to join
        them.  16 heads over 8000 tokens: 64 queries 64 and 76, 128 108 and 77, 512 305
        and 96; 128 heads over 4000: 64 queries 184 and 223, 256 636 and 240.
        Expanded from 16 queries on, where keys and values take up to 4 GB; and
        whatever they take where the absorbed attention refuses the call."""
        S = [t + n if n > 0 else 0 for t, n in zip(T, cnt)]
        if form not in (None, "absorbed", "expanded"):
            raise ValueError('form must be None, "absorbed" or "expanded"')
        if form is not None:
            return form == "expanded", max(S)
        if not self._absorbs(h, ns):
            return True, max(S)
        if max(cnt) < 16 or 4 * self.b * max(S) * h * LATENT_HEAD > 1 << 32:
            return False, max(S)
        absorbed = 35 + h * sum(n * s for n, s in zip(cnt, S)) * (self.r + 64) / 144e6
        rt = h * sum((n + 255) // 256 for n in cnt)
        c = max(1, min(6, self._sms * 9 // 10 // rt))
        expanded = 10 + h * sum(S) * (self.r + 256) / 2.15e6 + -(-rt // self._sms) * max(S) / (80 * c) + 3 * (c > 1)
        return expanded < absorbed, max(S)

    @staticmethod
    def _absorbs(h, ns):
        """Whether kivi_latent_attn takes h heads of a stride of ns tokens."""
        return h <= 128 and h * ns < 1 << 24

    def _expand(self, dims, ptrs, qrp, c, kr, K, V, T, cnt, tok, S, scale, st):
        """Every head's keys K and values V of tok tokens c, and the attention to them."""
        (_, h, ns, r), (qnp, _, _, _, wkp, wvp, op) = dims, ptrs
        for w, x in ((wkp, K), (wvp, V)):
            _check(lib.kivi_latent_product(self._h, c, w, 1, h, S, _addr(tok), r, LATENT_HEAD, 0, x, st))
        _check(lib.kivi_latent_expanded(self._h, qnp, qrp, K, kr, V, h, None if T is None else _addr(T), _addr(cnt), ns, S,
                                        scale, op, st))

    def _expanded(self, dims, ptrs, qrp, krp, cnt, T, S, scale, stream, st):
        (b, h, ns, r), cp = dims, ptrs[2]
        keep, (c_all, kr_all, K, V) = _space(stream, self._device, b * S * r, b * S * LATENT_ROPE,
                                             *[b * h * S * LATENT_HEAD] * 2)   # (rows past a sequence's tokens are not read)
        _check(lib.kivi_latent_rows(self._h, cp, krp, _addr(cnt), ns, c_all, kr_all, S, st))
        tok = array.array("i", [t + n if n else 0 for t, n in zip(T, cnt)])
        self._expand(dims, ptrs, qrp, c_all, kr_all, K, V, T, cnt, tok, S, scale, st)

    def _lengths(self):
        T = array.array("i", bytes(4 * self.b))
        _check(lib.kivi_latent_lengths(self._h, _addr(T), None))
        return T

    def _attn(self, dims, ptrs, qrp, krp, cnt, scale, form, stream, st):
        (b, h, ns, r), (qnp, _, cp, _, wkp, wvp, op) = dims, ptrs
        if form is not None or max(cnt) >= 16 or not self._absorbs(h, ns):
            T = self._lengths()
            expanded, S = self._form(form, cnt, T, h, ns)
            if expanded:
                return self._expanded(dims, ptrs, qrp, krp, cnt, T, S, scale, stream, st)
        keep, (ql, ol) = _space(stream, self._device, b * h * ns * r, b * h * ns * r)   # (rows past n are not read)
        _check(lib.kivi_latent_product(self._h, qnp, wkp, h, h, ns, _addr(cnt), LATENT_HEAD, r, 1, ql, st))
        _check(lib.kivi_latent_attn(self._h, ql, qrp, cp, krp, _addr(cnt), ns, h, scale, ol, st))
        _check(lib.kivi_latent_product(self._h, ol, wvp, h, h, ns, _addr(cnt), r, LATENT_HEAD, 0, op, st))

    def _args(self, qn, qr, c, kr, wk, wv, out, stream):
        dims, ptrs, out = _latent_args(qn, qr, c, kr, wk, wv, out, stream, self._dev)
        if dims[0] != self.b or dims[3] != self.r:
            raise ValueError(f"the latent cache holds {self.b} sequences of vectors of {self.r}")
        return dims, ptrs, out

    def attn(self, qn, qr, c, kr, n, wk, wv, scale=None, out=None, stream=None, form=None):
        """Latent attention of n new tokens of each sequence (an integer or b of
        them) over the cache and over themselves, absorbed or expanded (form;
        default the faster, which for long chunks is the latter, and expanded where
        the other is refused: more than 128 heads, h ns of 2^24 and more): qn CUDA fp16
        [b, h, ns, 128], qr [b, h, ns, 64], c [b, ns, r], kr [b, ns, 64], wk and wv [h,
        128, r] -> out [b, h, ns, 128] (rows past n untouched, zero in a new tensor).
        Queries and keys rotated.  Does not append (append, extend).

        What lies between the products is fp16: wk^T qn (absorbed) or wk c and wv c of
        every token (expanded) must stay below 65504, or out is not finite."""
        self._here()
        dims, ptrs, out = self._args(qn, qr, c, kr, wk, wv, out, stream)
        self._attn(dims, ptrs, ptrs[1], ptrs[3], _counts(n, self.b), _latent_scale(scale), form, stream, _stream(stream))
        return out

    def prefill_attn(self, qn, qr, c, kr, t, wk, wv, scale=None, out=None, stream=None):
        """prefill(c, kr, t) and the prompt's attention (latent_prompt_attn)."""
        self._here()
        dims, ptrs, out = self._args(qn, qr, c, kr, wk, wv, out, stream)
        cnt, st = _counts(t, self.b, "t"), _stream(stream)
        if max(cnt) > self.max_tokens:
            raise CapacityError(3, "a prompt exceeds max_tokens")
        b, h, ts, _ = dims
        keep, (K, V) = _space(stream, self._device, *[b * h * ts * LATENT_HEAD] * 2)   # (rows past t are not read)
        # (refuses before the cache changes)
        self._expand(dims, ptrs, ptrs[1], ptrs[2], ptrs[3], K, V, None, cnt, cnt, ts, _latent_scale(scale), st)
        _check(lib.kivi_latent_prefill(self._h, ptrs[2], ptrs[3], _addr(cnt), dims[2], st))
        return out

    def extend(self, qn, qr, c, kr, n, wk, wv, rope=None, pos=None, scale=None, out=None, stream=None, form=None):
        """Take the next n tokens of every sequence (a chunk, or one): rotate qr
        and kr at the positions behind the cached tokens (rope: a Rope of 64
        channels, or None; or at pos, as Rope.apply takes every position), attend
        (attn; returns its out) and append them."""
        import torch
        self._here()
        dims, ptrs, out = self._args(qn, qr, c, kr, wk, wv, out, stream)
        (b, h, ns, _), cnt, st = dims, _counts(n, self.b), _stream(stream)
        qrp, krp = ptrs[1], ptrs[3]
        if rope is None and pos is not None:
            raise ValueError("positions without a rope")
        T = self._lengths()
        for i in range(b):
            if cnt[i] > self.max_tokens - T[i]:
                raise CapacityError(3, f"sequence {i} would exceed max_tokens")
        if rope is not None:
            if rope.d != LATENT_ROPE:
                raise ValueError(f"rope is for heads of dimension {rope.d}")
            posp = None if pos is None else rope._pos(pos, b, ns, self._dev)
            keep, (rq, rk) = _space(stream, self._device, b * h * ns * LATENT_ROPE, b * ns * LATENT_ROPE)   # (rows past n are not read)
            rope._call(qrp, krp, b, h, 1, ns, cnt, T if posp is None else None, posp, False, rq, rk, st)
            qrp, krp = rq, rk
        self._attn(dims, ptrs, qrp, krp, cnt, _latent_scale(scale), form, stream, st)
        _check(lib.kivi_latent_append(self._h, ptrs[2], krp, _addr(cnt), ns, st))
        return out

    # -- inspection ----------------------------------------------------------
    def lengths(self):
        """Tokens of each sequence, and how many of them are quantized."""
        T, Tq = np.zeros(self.b, np.int32), np.zeros(self.b, np.int32)
        _check(lib.kivi_latent_lengths(self._h, T.ctypes.data, Tq.ctypes.data))
        return T, Tq

    def restore(self, stream=None):
        """The cached latent vectors and rotary keys as attention sees them: CUDA
        fp16 [b, t, r] and [b, t, 64] (t: the longest sequence; zero past each)."""
        import torch
        t = max(1, int(self.lengths()[0].max()))
        with _on(stream):
            c = torch.zeros((self.b, t, self.r), dtype=torch.float16, device=f"cuda:{self._dev}")
            kr = torch.zeros((self.b, t, LATENT_ROPE), dtype=torch.float16, device=f"cuda:{self._dev}")
        _check(lib.kivi_latent_restore(self._h, c.data_ptr(), kr.data_ptr(), t, _stream(stream)))
        return c, kr

    def check(self, stream=None) -> int:
        """The status word of every call of this cache's methods (kivi_latent_check)."""
        f = ctypes.c_uint32(0)
        _check(lib.kivi_latent_check(self._h, ctypes.byref(f), _stream(stream)))
        return int(f.value)
