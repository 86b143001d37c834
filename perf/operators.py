"""Cases for measuring the cache's serving operators, with their plain forms.

  rope           rotary positions of a step's or prompt's queries and keys
  window_decode  one decode step over the quantized cache, each query seeing
                 a sliding window of tokens and the first few (sinks)
  window_prompt  the prompt's causal attention with the same visibility
  chunk          attention of a chunk of new tokens over the quantized cache
                 and the chunk itself (a long prompt taken in pieces, or the
                 tokens of a speculative step to verify)
  extend         the pieces as a program runs them: fill the cache, rotate
                 the next chunk, attend and append it, decode one token

A query at position p sees token s when s <= p and (window == 0 or
p - s < window or s < sinks).
"""
import math

import torch

own = False

F32, F64 = torch.float32, torch.float64


# ---- the cases ---------------------------------------------------------------

def _rope(name, b, n, hq, hkv, d, rot, interleaved, far, ragged=False, scaling="none"):
    return {"name": name, "op": "rope", "b": b, "n": n, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "far": far, "ragged": ragged, "scaling": scaling}


def _cached(name, op, b, hq, hkv, d, kbits, vbits, G, R, t, ragged, n, window, sinks):
    return {"name": name, "op": op, "b": b, "hq": hq, "hkv": hkv, "d": d, "kbits": kbits, "vbits": vbits,
            "G": G, "R": R, "t": t, "ragged": ragged, "n": n, "window": window, "sinks": sinks}


def listed():
    return [
        # the serving batch's decode step: one token of 64 sequences, latency counts
        _rope("rope_step", 64, 1, 32, 8, 128, 128, False, 4096),
        # four prompts of 8k tokens
        _rope("rope_prompt", 4, 8192, 32, 8, 128, 128, False, 0),
        # ragged chunks far into long contexts, half of each head rotated, pairs side by side
        _rope("rope_far_partial", 3, 1777, 12, 4, 64, 32, True, 900000, True, "yarn"),
        # 8 long conversations whose queries see 4k tokens back
        _cached("window_decode_32k", "window_decode", 8, 32, 8, 128, 2, 2, 32, 128, 32767, False, 1, 4096, 4),
        # the ragged serving batch, 4-bit, with a window shorter than most of its sequences
        _cached("window_decode_serving", "window_decode", 64, 32, 8, 128, 4, 4, 32, 128, 4096, True, 1, 1000, 5),
        # a 4k prompt, every head with its own keys
        _cached("window_prompt_4k", "window_prompt", 1, 32, 32, 128, 2, 2, 32, 128, 4096, False, 0, 1024, 4),
        # an 8k prompt, grouped heads
        _cached("window_prompt_8k", "window_prompt", 1, 32, 8, 128, 2, 2, 32, 128, 8191, False, 0, 2048, 64),
        # a speculative step: 4 tokens of each of 8 sequences to verify over 32k tokens
        _cached("chunk_verify_32k", "chunk", 8, 32, 8, 128, 2, 2, 32, 128, 32767, False, 4, 0, 0),
        # the next 2048 tokens of a long prompt
        _cached("chunk_prompt_16k", "chunk", 1, 32, 8, 128, 2, 2, 32, 128, 16500, False, 2048, 0, 0),
        # ragged pieces over ragged 4-bit sequences, sliding window
        _cached("chunk_window_ragged", "chunk", 6, 16, 4, 64, 4, 4, 16, 48, 5000, True, 333, 777, 3),
        # a prompt in two pieces, then a step
        _cached("extend_prompt", "extend", 1, 32, 8, 128, 2, 2, 32, 128, 4000, False, 2000, 0, 0),
        # the same for a small ragged batch with every head its own keys
        _cached("extend_ragged", "extend", 4, 8, 8, 128, 4, 2, 64, 64, 900, True, 150, 256, 4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "window_decode", "window_prompt", "chunk", "chunk", "extend"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 8])
    if op == "rope":
        b, n = _log(rng, 1, 64), _log(rng, 1, 8192)
        n = max(1, min(n, 4 * 8192 * 40 * 128 // (b * (hq + hkv) * d)))
        c = _rope("", b, n, hq, hkv, d, rng.choice([d, d // 2, 16, d // 4 * 3]), rng.random() < 0.5,
                  _log(rng, 1, 2000000), rng.random() < 0.5, rng.choice(["none", "linear", "ntk", "yarn"]))
    else:
        G = rng.choice([16, 32, 64])
        R = G * rng.randint(1, 4)
        kb, vb = rng.choice([2, 4]), rng.choice([2, 4])
        ragged = rng.random() < 0.5
        window, sinks = _log(rng, 16, 5000), rng.choice([0, 1, 4, 70])
        b, n = 1, 1
        if op == "window_decode":
            b, t = _log(rng, 1, 32), _log(rng, 100, 32767)
            t = max(1, min(t, 8 * 8 * 32767 // (b * hkv)))
        elif op == "window_prompt":
            t, n = _log(rng, 100, 8192), 0
            hq, hkv = (hq, hkv) if hq <= 32 else (32, 8)
        elif op == "chunk":
            b, t = _log(rng, 1, 8), _log(rng, 50, 32767)
            hq, hkv = (hq, hkv) if hq <= 32 else (32, 8)
            n = _log(rng, 1, 2048)
            n = max(1, min(n, 32 * 2048 * 16500 // (b * hq * t)))
            if rng.random() < 0.5:
                window = sinks = 0
        else:
            b, t, n = _log(rng, 1, 4), _log(rng, 50, 3000), _log(rng, 1, 1500)
            hq, hkv = (hq, hkv) if hq <= 32 else (32, 8)
            n = max(1, min(n, 32 * 2000 * 4000 // (b * hq * t)))
            if rng.random() < 0.5:
                window = sinks = 0
        c = _cached("", op, b, hq, hkv, d, kb, vb, G, R, t, ragged, n, window, sinks)
    del c["name"]
    return c


# ---- inputs ------------------------------------------------------------------

def _lens(gen_seed, n, b, ragged, low):
    if not ragged:
        return [n] * b
    g = torch.Generator().manual_seed(gen_seed)
    r = torch.randint(min(low, n), n + 1, (b,), generator=g).tolist()
    r[0] = n
    return r


def _inv_freq(c):
    """Angular frequencies (radians a position, 64 bits) and the factor on the rotated part."""
    rot, base, factor, old = c["rot"], 500000.0, 4.0, 8192
    i = torch.arange(0, rot, 2, dtype=F64)
    f = base ** (-i / rot)
    if c["scaling"] == "linear":
        return f / factor, 1.0
    if c["scaling"] == "ntk":
        return (base * factor ** (rot / (rot - 2))) ** (-i / rot), 1.0
    if c["scaling"] == "yarn":
        at = [rot * math.log(old / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot // 2 - 1)
        ramp = ((torch.arange(rot // 2, dtype=F64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32)


def _keys(g, b, h, n, d, channels):
    """Keys with a few large channels per head."""
    k = _randn(g, b, h, n, d)
    return k.scatter(3, channels.expand(b, h, n, channels.shape[3]),
                     8.0 * torch.gather(k, 3, channels.expand(b, h, n, channels.shape[3]))).half()


def _data(c, seed):
    """The inputs, a pure function of the case and the seed."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    b, hq, h, d = c["b"], c["hq"], c["hkv"], c["d"]
    if c["op"] == "rope":
        n = c["n"]
        lens = _lens(seed, n, b, c["ragged"], 0)
        first = [max(0, c["far"] - 17 * i) for i in range(b)]
        return {"q": _randn(g, b, hq, n, d).half(), "k": _randn(g, b, h, n, d).half(), "n": lens, "first": first}
    t, n = c["t"], c["n"]
    ch = torch.rand((b, h, 1, d), generator=g, device="cuda").topk(max(1, round(0.02 * d)), dim=3).indices
    s = {"K": _keys(g, b, h, t, d, ch), "V": _randn(g, b, h, t, d).half(), "t": _lens(seed, t, b, c["ragged"], t // 4)}
    if c["op"] == "window_prompt":
        s["q"] = _randn(g, b, hq, t, d).half()
    elif c["op"] == "window_decode":
        s["q"] = _randn(g, b, hq, d).half()
    else:
        s |= {"q": _randn(g, b, hq, n, d).half(), "k": _keys(g, b, h, n, d, ch), "v": _randn(g, b, h, n, d).half(),
              "n": _lens(seed + 1, n, b, c["ragged"], 0)}
        if c["op"] == "extend":
            s |= {"q1": _randn(g, b, hq, d).half(), "rope": dict(rot=d, scaling="none")}
    return s


def _counters(t, R):
    """Quantized keys and values of a sequence filled with t tokens at once."""
    return t - t % R, max(t - R, 0)


def _counters_after(t, n, R):
    """... and after n more, one at a time."""
    qk, qv = _counters(t, R)
    return (qk, qv) if n == 0 else (max(qk, (t + n - 1) // R * R), max(qv, t + n - R - 1))


def prepare(case, seed):
    c = case
    s = _data(c, seed)
    s["case"] = c
    b, d, R = c["b"], c["d"], c.get("R")
    dev = dict(device="cuda")
    if c["op"] == "rope":
        f, factor = _inv_freq(c)
        s["freq"], s["factor"] = f.cuda(), factor
        s["pos0"], s["len"] = torch.tensor(s["first"], **dev), torch.tensor(s["n"], **dev)
        s["q_out"], s["k_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
        if own:
            from bit_quantized_kv_quantize_gb300 import kivi as K
            s["handle"] = K.Rope(d, rot_dim=c["rot"], interleaved=c["interleaved"], inv_freq=f.tolist(),
                                 factor=factor)
        return s
    s["T"] = torch.tensor(s["t"], **dev)
    s["out"] = torch.zeros_like(s["q"])
    if c["op"] in ("chunk", "extend"):
        s["len"] = torch.tensor(s["n"], **dev)
    if c["op"] in ("window_decode", "chunk"):
        s["cache"] = _pack(s["K"], s["V"], [_counters(t, R)[0] for t in s["t"]],
                           [_counters(t, R)[1] for t in s["t"]], c)
    if c["op"] == "extend":
        s["freq"] = _inv_freq(dict(rot=d, scaling="none"))[0].cuda()
        s["out1"] = torch.zeros_like(s["q1"])
    if own:
        from bit_quantized_kv_quantize_gb300 import kivi as K
        s["handle"] = K.KiviCache(b, c["hkv"], d, c["kbits"], c["vbits"], c["G"], R, c["t"] + c["n"] + 1)
        if c["op"] in ("window_decode", "chunk"):
            s["handle"].prefill(s["K"], s["V"], s["t"])
            del s["cache"]
        if c["op"] == "extend":
            s["rope_handle"] = K.Rope(d, inv_freq=s["freq"].tolist())
    return s


# ---- plain forms -------------------------------------------------------------

def _quant(x, bits):
    """Codes, scale and zero of groups along the last axis of x [..., G] (16-bit scale and zero, 32-bit arithmetic)."""
    x = x.to(F32)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s, z = ((hi - lo) / (2 ** bits - 1)).half(), lo.half()
    sf = s.to(F32)
    q = torch.where(sf > 0, ((x - z.to(F32)) / torch.where(sf > 0, sf, 1.0)).round(), 0.0)
    return q.clamp(0, 2 ** bits - 1).to(torch.uint8), s, z


def _pack(K, V, qk, qv, c):
    """The cache in plain tensors: codes with 16-bit scales and zeros (keys per channel along G tokens, values per
    token along G channels), the 16-bit rows, and how many of each are quantized."""
    b, h, t, d = K.shape
    G = c["G"]
    tg = -(-t // G) * G
    Kp = torch.nn.functional.pad(K, (0, 0, 0, tg - t))
    kc, ks, kz = _quant(Kp.view(b, h, tg // G, G, d).transpose(3, 4), c["kbits"])
    vc, vs, vz = _quant(V.view(b, h, t, d // G, G), c["vbits"])
    return {"kc": kc, "ks": ks, "kz": kz, "vc": vc, "vs": vs, "vz": vz, "K": K, "V": V,
            "qk": torch.tensor(qk, device="cuda"), "qv": torch.tensor(qv, device="cuda")}


def _unpack(p, dt=F32):
    """Keys and values as attention sees them [b, h, t, d]: quantized tokens restored, the others as they are."""
    b, h, t, d = p["K"].shape
    at = torch.arange(t, device="cuda").view(1, 1, t, 1)
    k = (p["kc"].to(dt) * p["ks"].to(dt) + p["kz"].to(dt)).transpose(3, 4).reshape(b, h, -1, d)[:, :, :t]
    v = (p["vc"].to(dt) * p["vs"].to(dt) + p["vz"].to(dt)).reshape(b, h, t, d)
    return (torch.where(at < p["qk"].view(b, 1, 1, 1), k, p["K"].to(dt)),
            torch.where(at < p["qv"].view(b, 1, 1, 1), v, p["V"].to(dt)))


def _attend(q, k, v, pos, kpos, kok, window, sinks):
    """softmax(q k^T / sqrt(d)) v with q [b, hq, n, d], k, v [b, h, S, d], query positions pos [b, n], token positions
    kpos [b, S] and tokens that exist kok [b, S]."""
    b, hq, n, d = q.shape
    h, S = k.shape[1], k.shape[2]
    see = kok.view(b, 1, S) & (kpos.view(b, 1, S) <= pos.view(b, n, 1))
    if window:
        see &= (pos.view(b, n, 1) - kpos.view(b, 1, S) < window) | (kpos.view(b, 1, S) < sinks)
    s = torch.matmul(q.to(F32).reshape(b, h, hq // h * n, d), k.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    s = s.view(b, h, hq // h, n, S).masked_fill_(~see.view(b, 1, 1, n, S), -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    o = torch.matmul(s.view(b, h, hq // h * n, S), v).view(b, h, hq // h, n, d)
    o = o / s.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.view(b, hq, n, d)


def _rotate(x, pos, freq, factor, rot, interleaved):
    """x [b, h, n, d], pos [b, n]."""
    a = pos.to(F64)[:, None, :, None] * freq
    cos, sin = (torch.cos(a) * factor).to(F32), (torch.sin(a) * factor).to(F32)
    y = x.to(F32)
    r = y[..., :rot]
    if interleaved:
        e, o = r[..., 0::2], r[..., 1::2]
        r = torch.stack((e * cos - o * sin, o * cos + e * sin), -1).flatten(-2)
    else:
        e, o = r[..., : rot // 2], r[..., rot // 2:]
        r = torch.cat((e * cos - o * sin, o * cos + e * sin), -1)
    return torch.cat((r, y[..., rot:]), -1)


def _inside(lens, n):
    return torch.arange(n, device="cuda").view(1, n) < lens.view(-1, 1)


def _run_plain(s):
    c = s["case"]
    op, b = c["op"], c["b"]
    if op == "rope":
        n = c["n"]
        pos = s["pos0"].view(b, 1) + torch.arange(n, device="cuda")
        keep = _inside(s["len"], n).view(b, 1, n, 1)
        return tuple(torch.where(keep, _rotate(s[x], pos, s["freq"], s["factor"], c["rot"], c["interleaved"]), 0.0)
                     .half() for x in ("q", "k"))
    t, window, sinks = c["t"], c["window"], c["sinks"]
    at = torch.arange(t, device="cuda").expand(b, t)
    if op == "window_decode":
        k, v = _unpack(s["cache"])
        return _attend(s["q"].unsqueeze(2), k, v, s["T"].view(b, 1) - 1, at, _inside(s["T"], t), window,
                       sinks).squeeze(2).half()
    if op == "window_prompt":
        inside = _inside(s["T"], t)
        o = _attend(s["q"], s["K"].to(F32), s["V"].to(F32), at, at, inside, window, sinks)
        return torch.where(inside.view(b, 1, t, 1), o, 0.0).half()
    n = c["n"]
    pos = s["T"].view(b, 1) + torch.arange(n, device="cuda")
    kpos = torch.cat((at, pos), 1)
    kok = torch.cat((_inside(s["T"], t), _inside(s["len"], n)), 1)
    keep = _inside(s["len"], n).view(b, 1, n, 1)
    if op == "chunk":
        k, v = _unpack(s["cache"])
        o = _attend(s["q"], torch.cat((k, s["k"].to(F32)), 2), torch.cat((v, s["v"].to(F32)), 2), pos, kpos, kok,
                    window, sinks)
        return torch.where(keep, o, 0.0).half()
    R, d = c["R"], c["d"]
    q = _rotate(s["q"], pos, s["freq"], 1.0, d, False).half()
    kn = _rotate(s["k"], pos, s["freq"], 1.0, d, False).half()
    k, v = _unpack(_pack(s["K"], s["V"], [_counters(x, R)[0] for x in s["t"]],
                         [_counters(x, R)[1] for x in s["t"]], c))
    o = _attend(q, torch.cat((k, kn.to(F32)), 2), torch.cat((v, s["v"].to(F32)), 2), pos, kpos, kok, window, sinks)
    # the sequences with the chunk behind their own last token
    src = torch.arange(t + n, device="cuda").expand(b, t + n)
    src = torch.where(src < s["T"].view(b, 1), src, src - s["T"].view(b, 1) + t).clamp_max(t + n - 1)
    src = src.view(b, 1, t + n, 1).expand(b, c["hkv"], t + n, d)
    after = [_counters_after(x, y, R) for x, y in zip(s["t"], s["n"])]
    k, v = _unpack(_pack(torch.cat((s["K"], kn), 2).gather(2, src), torch.cat((s["V"], s["v"]), 2).gather(2, src),
                         [x for x, _ in after], [y for _, y in after], c))
    total = s["T"] + s["len"]
    o1 = _attend(s["q1"].unsqueeze(2), k, v, total.view(b, 1) - 1, torch.arange(t + n, device="cuda").expand(b, t + n),
                 _inside(total, t + n), window, sinks)
    return torch.where(keep, o, 0.0).half(), o1.squeeze(2).half()


def run(state):
    s = state
    if not own:
        return _run_plain(s)
    c, h = s["case"], s["handle"]
    if c["op"] == "rope":
        return h.apply(s["q"], s["k"], s["first"], n=s["n"], q_out=s["q_out"], k_out=s["k_out"])
    if c["op"] == "window_decode":
        return h.decode(s["q"], window=c["window"], sinks=c["sinks"], out=s["out"])
    if c["op"] == "window_prompt":
        return h.prefill_attn(s["q"], s["K"], s["V"], s["t"], window=c["window"], sinks=c["sinks"], out=s["out"])
    if c["op"] == "chunk":
        return h.chunk_attn(s["q"], s["k"], s["v"], s["n"], window=c["window"], sinks=c["sinks"], out=s["out"])
    h.prefill(s["K"], s["V"], s["t"])
    o = h.extend(s["q"], s["k"], s["v"], s["n"], window=c["window"], sinks=c["sinks"], rope=s["rope_handle"],
                 out=s["out"])
    return o, h.decode(s["q1"], window=c["window"], sinks=c["sinks"], out=s["out1"])


# ---- what a pass cannot do without -------------------------------------------

def _seen(t, n, window, sinks):
    """Visible (query, token) pairs of n queries at positions t .. t + n - 1, and the tokens that any of them sees."""
    pairs, w = 0, window or t + n
    for p in range(t, t + n):
        first = max(0, p + 1 - w)
        pairs += p + 1 - first + min(sinks if window else 0, first)
    first = max(0, t + 1 - w)
    return pairs, t + n - first + min(sinks if window else 0, first)


def work(case):
    c = case
    b, hq, h, d = c["b"], c["hq"], c["hkv"], c["d"]
    if c["op"] == "rope":
        tokens = sum(_lens(1, c["n"], b, c["ragged"], 0))
        return {"bytes": 4.0 * tokens * (hq + h) * d, "flops": 3.0 * tokens * (hq + h) * c["rot"]}
    R, G, w, k = c["R"], c["G"], c["window"], c["sinks"]
    t = _lens(1, c["t"], b, c["ragged"], c["t"] // 4)
    if c["op"] == "window_prompt":
        pairs = sum(_seen(0, x, w, k)[0] for x in t)
        return {"bytes": sum(t) * d * (4.0 * hq + 4 * h + h * _token(c) / d), "flops": 4.0 * d * hq * pairs}
    if c["op"] == "window_decode":
        seen = [_seen(x - 1, 1, w, k)[1] for x in t]
        return {"bytes": b * hq * d * 4.0 + sum(_cache_bytes(c, x, y) for x, y in zip(t, seen)),
                "flops": 4.0 * d * hq * sum(seen)}
    n = _lens(2, c["n"], b, c["ragged"], 0)
    got = [_seen(x, y, w, k) if y else (0, 0) for x, y in zip(t, n)]
    chunk = {"bytes": sum(_cache_bytes(c, x, max(0, s - y)) for x, y, (_, s) in zip(t, n, got))
             + sum(n) * d * 4.0 * (hq + h), "flops": 4.0 * d * hq * sum(p for p, _ in got)}
    if c["op"] == "chunk":
        return chunk
    # extend: the fill, the rotation, the chunk with its packing, the step
    seen = [_seen(x + y - 1, 1, w, k)[1] for x, y in zip(t, n)]
    more = sum(t) * h * (4.0 * d + _token(c)) + sum(n) * (4.0 * d * (hq + h) + h * _token(c)) + 4.0 * b * hq * d
    more += sum(_cache_bytes(c, x + y, z) for x, y, z in zip(t, n, seen))
    return {"bytes": chunk["bytes"] + more, "flops": chunk["flops"] + 4.0 * d * hq * sum(seen)}


def _token(c):
    """Bytes of one quantized token of one kv head."""
    return c["d"] * (c["kbits"] + c["vbits"]) / 8 + 8 * c["d"] / c["G"]


def _cache_bytes(c, t, seen):
    """Bytes of `seen` of a sequence's t tokens, the newest R of them in 16 bits."""
    full = min(seen, c["R"])
    return c["hkv"] * (full * 4.0 * c["d"] + (seen - full) * _token(c))


# ---- the definition in 64 bits ------------------------------------------------

def _exact_rows(q, k, v, first, window, sinks):
    """Attention of rows q [n, d] at positions first.. over k, v [S, d] at positions 0..S-1."""
    n, S = q.shape[0], k.shape[0]
    p = torch.arange(first, first + n, device="cuda").view(n, 1)
    s = torch.arange(S, device="cuda").view(1, S)
    x = (q.to(F64) @ k.t()) / math.sqrt(q.shape[1])
    hidden = s > p
    if window:
        hidden = hidden | ((s <= p - window) & (s >= sinks))
    x[hidden] = -math.inf
    return torch.softmax(x, -1) @ v


def _exact_quant(x, bits, axis):
    """Groups along `axis` of x replaced by zero + code * scale, in 64 bits from 16-bit scales and zeros."""
    x = x.to(F64)
    z = x.amin(axis, keepdim=True)
    s = ((x.amax(axis, keepdim=True) - z) / (2 ** bits - 1)).to(F32).half().to(F64)
    code = torch.round((x - z) / s).clamp(0, 2 ** bits - 1)
    return torch.where(s > 0, z + s * torch.nan_to_num(code), z)


def _exact_cache(K, V, qk, qv, c):
    """One sequence's keys and values [t, d] of one kv head as the cache restores them."""
    G, d = c["G"], c["d"]
    k, v = K.to(F64).clone(), V.to(F64).clone()
    if qk:
        k[:qk] = _exact_quant(K[:qk].view(qk // G, G, d), c["kbits"], 1).view(qk, d)
    if qv:
        v[:qv] = _exact_quant(V[:qv].view(qv, d // G, G), c["vbits"], 2).view(qv, d)
    return k, v


def _exact_rotate(x, first, f, factor, rot, interleaved):
    """Rows x [n, d] at positions first.., as complex numbers times exp(i p f)."""
    n, x = x.shape[0], x.to(F64)
    p = torch.arange(first, first + n, device="cuda", dtype=F64).view(n, 1)
    turn = torch.polar(torch.full((n, rot // 2), factor, dtype=F64, device="cuda"), p * f)
    if interleaved:
        y = torch.view_as_complex(x[:, :rot].reshape(n, rot // 2, 2).contiguous()) * turn
        y = torch.view_as_real(y).reshape(n, rot)
    else:
        y = torch.complex(x[:, : rot // 2].contiguous(), x[:, rot // 2:rot].contiguous()) * turn
        y = torch.cat((y.real, y.imag), 1)
    return torch.cat((y, x[:, rot:]), 1)


def exact(case, seed):
    c = case
    s = _data(c, seed)
    b, hq, h, d = c["b"], c["hq"], c["hkv"], c["d"]
    if c["op"] == "rope":
        f, factor = _inv_freq(c)
        out = [torch.zeros(s[x].shape, dtype=F64, device="cuda") for x in ("q", "k")]
        for o, x in zip(out, (s["q"], s["k"])):
            for i in range(b):
                for j in range(x.shape[1]):
                    n = s["n"][i]
                    o[i, j, :n] = _exact_rotate(x[i, j, :n], s["first"][i], f.cuda(), factor, c["rot"],
                                                c["interleaved"])
        return tuple(out)
    w, sk, R = c["window"], c["sinks"], c.get("R")
    out = torch.zeros(s["q"].shape, dtype=F64, device="cuda")
    out1 = torch.zeros((b, hq, d), dtype=F64, device="cuda")
    if c["op"] == "extend":
        f = _inv_freq(dict(rot=d, scaling="none"))[0].cuda()
    for i in range(b):
        t = s["t"][i]
        qk, qv = _counters(t, R)
        for j in range(h):
            heads = range(j * (hq // h), (j + 1) * (hq // h))
            K, V = s["K"][i, j, :t], s["V"][i, j, :t]
            if c["op"] == "window_prompt":
                for e in heads:
                    out[i, e, :t] = _exact_rows(s["q"][i, e, :t], K.to(F64), V.to(F64), 0, w, sk)
                continue
            k, v = _exact_cache(K, V, qk, qv, c)
            if c["op"] == "window_decode":
                for e in heads:
                    out[i, e] = _exact_rows(s["q"][i, e:e + 1], k, v, t - 1, w, sk)[0]
                continue
            n = s["n"][i]
            q, kn = s["q"][i, :, :n], s["k"][i, j, :n]
            if c["op"] == "extend":
                kn = _exact_rotate(kn, t, f, 1.0, d, False).half()
            k, v = torch.cat((k, kn.to(F64))), torch.cat((v, s["v"][i, j, :n].to(F64)))
            for e in heads:
                x = _exact_rotate(q[e], t, f, 1.0, d, False).half() if c["op"] == "extend" else q[e]
                if n:
                    out[i, e, :n] = _exact_rows(x, k, v, t, w, sk)
            if c["op"] == "extend":
                k, v = _exact_cache(torch.cat((K, kn)), torch.cat((V, s["v"][i, j, :n])),
                                    *_counters_after(t, n, R), c)
                for e in heads:
                    out1[i, e] = _exact_rows(s["q1"][i, e:e + 1], k, v, t + n - 1, w, sk)[0]
    return (out, out1) if c["op"] == "extend" else out
