"""Cases for measuring latent attention with its quantized cache, rotary
positions with several axes and the verification of drafts, with their plain
forms.

  axes           rotary positions whose channel pairs turn by different axes
                 (time, height, width) of a token's position
  verify         drafted tokens against the target's probabilities, from given
                 random numbers: how many are kept, and the token after them
  latent_attn    attention of new tokens over a cache that holds one latent
                 vector a token (keys and values of every head are products of
                 it), and over the new tokens themselves
  latent_prompt  the causal attention of a prompt given as latent vectors
  latent_run     the pieces as a program runs them: a prompt with its cache
                 filled, a chunk, a single token, rotary positions throughout

Latent attention.  Token s has a latent vector c_s [r] and a rotary key kr_s
[64], shared by all heads; head h has Wk_h and Wv_h [128][r].  A query is
qn [128] and qr [64]:
  score = (qn . Wk_h c_s + qr . kr_s) / sqrt(192),   out = Wv_h sum_s w_s c_s.
The cache holds the newest R tokens' c_s as they are, older ones in 2- or 4-bit
codes with a 16-bit scale and zero for each G channels of a token, and kr_s as
it is.
"""
import math

import torch

own = False

F32, F64 = torch.float32, torch.float64
DN, DR, DV = 128, 64, 128   # a head's channels without and with positions, and of its values


# ---- the cases ---------------------------------------------------------------

def _axes(name, b, n, hq, hkv, d, rot, sections, turns, interleaved, far, ragged):
    return {"name": name, "op": "axes", "b": b, "n": n, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "sections": sections,
            "turns": turns, "interleaved": interleaved, "far": far, "ragged": ragged}


def _verify(name, b, n, vocab, half, ragged, certain):
    return {"name": name, "op": "verify", "b": b, "n": n, "vocab": vocab, "half": half, "ragged": ragged,
            "certain": certain}


def _latent(name, op, b, h, r, bits, G, R, t, ragged, n):
    return {"name": name, "op": op, "b": b, "h": h, "r": r, "bits": bits, "G": G, "R": R, "t": t, "ragged": ragged,
            "n": n}


def listed():
    return [
        # the serving batch's decode step with three axes, one token of 64 sequences: latency counts
        _axes("axes_step", 64, 1, 32, 8, 128, 128, "16,24,24", False, False, 4096, False),
        # two prompts of text and image patches, axes dealt to the pairs in turn
        _axes("axes_patches", 2, 4999, 32, 8, 128, 128, "22,21,21", True, False, 300, True),
        # a speculative step of the serving batch: 4 drafted tokens of 64 sequences
        _verify("verify_step", 64, 4, 32000, False, False, False),
        # long drafts over a large vocabulary of an odd size, 16-bit probabilities
        _verify("verify_wide", 16, 9, 150001, True, True, False),
        # the ragged serving batch's step: one token of 64 sequences of up to 4k, 16 heads (a share of a larger model's)
        _latent("latent_step", "latent_attn", 64, 16, 512, 4, 32, 128, 4096, True, 1),
        # 8 long conversations, every head on this GPU
        _latent("latent_step_32k", "latent_attn", 8, 128, 512, 4, 32, 128, 32767, False, 1),
        # a speculative step over 2-bit caches
        _latent("latent_verify", "latent_attn", 8, 32, 256, 2, 64, 192, 16001, True, 5),
        # the next 1024 tokens of a long prompt whose cache has not been quantized yet
        _latent("latent_chunk", "latent_attn", 1, 16, 512, 4, 128, 16384, 8000, False, 1024),
        # a 4k prompt
        _latent("latent_prompt_4k", "latent_prompt", 1, 32, 512, 4, 32, 128, 4096, False, 0),
        # ragged prompts, an odd number of heads
        _latent("latent_prompt_ragged", "latent_prompt", 3, 11, 256, 4, 32, 128, 1531, True, 0),
        # a prompt, its next piece and a step
        _latent("latent_run", "latent_run", 2, 16, 512, 4, 32, 128, 2000, False, 300),
        # the same for a small ragged batch
        _latent("latent_run_small", "latent_run", 4, 8, 256, 2, 64, 64, 190, True, 17),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["axes", "verify", "latent_attn", "latent_attn", "latent_attn", "latent_prompt", "latent_run"])
    if op == "axes":
        d = rng.choice([64, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 6])
        b, n = _log(rng, 1, 64), _log(rng, 1, 8192)
        n = max(1, min(n, 2 * 8192 * 40 * 128 // (b * (hq + hkv) * d)))
        rot = rng.choice([d, d // 2, d // 4 * 3])
        cuts = sorted(rng.randint(0, rot // 2) for _ in range(rng.choice([1, 2, 2, 3])))
        sections = ",".join(str(y - x) for x, y in zip([0] + cuts, cuts + [rot // 2]))
        c = _axes("", b, n, hq, hkv, d, rot, sections, rng.random() < 0.5, rng.random() < 0.5, _log(rng, 1, 2000000),
                  rng.random() < 0.5)
    elif op == "verify":
        vocab = _log(rng, 50, 200000)
        b, n = _log(rng, 1, 64), rng.randint(1, 12)
        b = max(1, min(b, 16 * 19 * 150001 // ((2 * n + 1) * vocab)))
        c = _verify("", b, n, vocab, rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.25)
    else:
        r = rng.choice([256, 512])
        h = rng.choice([1, 2, 5, 8, 12, 16, 32, 64, 128])
        bits, G, R = rng.choice([2, 4]), rng.choice([32, 64, 128]), rng.choice([64, 128, 192, 1024, 16384])
        ragged = rng.random() < 0.5
        if op == "latent_attn":
            b, t, n = _log(rng, 1, 64), _log(rng, 1, 32767), rng.choice([1, 1, _log(rng, 1, 1024)])
            t = max(1, min(t, 8 * 32767 // b))
            n = max(1, min(n, 120000000 // (b * h * t)))
            n = max(1, min(n, int(math.sqrt(120000000 / (b * h)))))
        elif op == "latent_prompt":
            b, t, n = _log(rng, 1, 8), _log(rng, 1, 4096), 0
            t = max(1, min(t, int(math.sqrt(32 * 4096 * 4096 / (b * h)))))
        else:
            b, t, n = _log(rng, 1, 4), _log(rng, 1, 2000), _log(rng, 1, 300)
            t = max(1, min(t, int(math.sqrt(32 * 2000 * 2000 / (b * h)))))
            n = max(1, min(n, 16 * 2 * 300 * 2300 // (b * h * (t + n))))
        c = _latent("", op, b, h, r, bits, G, R, t, ragged, n)
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


def _axis_of_pairs(c):
    """The axis of each pair: sections one after another, or dealt in turn while they last."""
    left = [int(x) for x in c["sections"].split(",")]
    if not c["turns"]:
        return [a for a, k in enumerate(left) for _ in range(k)]
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _freq(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=F64) / rot)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32)


def _data(c, seed):
    """The inputs, a pure function of the case and the seed."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    b = c["b"]
    if c["op"] == "axes":
        n, hq, h, d, A = c["n"], c["hq"], c["hkv"], c["d"], len(c["sections"].split(","))
        # some text, then a grid of patches behind it: a width of 37
        at = torch.arange(n, device="cuda")
        text = min(n, 11)
        patch = (at - text).clamp_min(0)
        rows = [torch.where(at < text, at, text + x) for x in (patch // (37 * 31), patch // 37 % 31, patch % 37, patch)]
        pos = torch.stack([rows[a % 4].expand(b, n) + c["far"] + 17 * torch.arange(b, device="cuda").view(b, 1)
                           for a in range(A)]).int().contiguous()
        return {"q": _randn(g, b, hq, n, d).half(), "k": _randn(g, b, h, n, d).half(), "pos": pos,
                "n": _lens(seed, n, b, c["ragged"], 0)}
    if c["op"] == "verify":
        n, V = c["n"], c["vocab"]
        dt = torch.float16 if c["half"] else F32
        logit = 2.5 * _randn(g, b, n + 1, V)
        # a draft whose distribution is near the target's
        near = logit[:, :n] + 0.7 * _randn(g, b, n, V)
        p = torch.softmax(logit, -1).to(dt)
        q = torch.softmax(near, -1).to(dt)
        # drawn from q (the smallest exponential over its rate); a certain draft is the largest
        w = _exponential(g, b, n, V)
        draft = (near.argmax(-1) if c["certain"] else (q.to(F32) / w).argmax(-1)).int()
        u = torch.rand((b, n + 1), generator=g, device="cuda", dtype=F32)
        return {"p": p, "q": None if c["certain"] else q, "draft": draft, "u": u, "n": _lens(seed, n, b, c["ragged"], 0)}
    r, h, t, n = c["r"], c["h"], c["t"], c["n"]
    spread = 0.5 + torch.rand((1, 1, r), generator=g, device="cuda", dtype=F32)

    def tokens(m):
        return (spread * _randn(g, b, m, r)).half(), _randn(g, b, m, DR).half()

    def queries(m):
        return _randn(g, b, h, m, DN).half(), _randn(g, b, h, m, DR).half()

    s = {"wk": (_randn(g, h, DN, r) / math.sqrt(r)).half(), "wv": (_randn(g, h, DV, r) / math.sqrt(r)).half(),
         "t": _lens(seed, t, b, c["ragged"], t // 4)}
    s["c"], s["kr"] = tokens(t)
    if c["op"] != "latent_attn":
        s["qn"], s["qr"] = queries(t)
    if c["op"] != "latent_prompt":
        s["c1"], s["kr1"] = tokens(n)
        s["qn1"], s["qr1"] = queries(n)
        s["n"] = _lens(seed + 1, n, b, c["ragged"], 0)
    if c["op"] == "latent_run":
        s["c2"], s["kr2"] = tokens(1)
        s["qn2"], s["qr2"] = queries(1)
    return s


def _exponential(g, *shape):
    return -torch.log(torch.rand(shape, generator=g, device="cuda", dtype=F32).clamp_min(1e-20))


def prepare(case, seed):
    c = case
    s = _data(c, seed)
    s["case"] = c
    dev = dict(device="cuda")
    b = c["b"]
    if own:
        from bit_quantized_kv_quantize_gb300 import kivi as K
    if c["op"] == "axes":
        s["freq"], s["len"] = _freq(c["rot"]).cuda(), torch.tensor(s["n"], **dev)
        s["axis"] = torch.tensor(_axis_of_pairs(c), **dev)
        s["q_out"], s["k_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
        if own:
            s["handle"] = K.Rope(c["d"], rot_dim=c["rot"], interleaved=c["interleaved"], inv_freq=_freq(c["rot"]).tolist(),
                                 axes=_axis_of_pairs(c))
        return s
    if c["op"] == "verify":
        s["len"] = torch.tensor(s["n"], **dev)
        s["tokens"] = torch.zeros((b, c["n"] + 1), dtype=torch.int32, **dev)
        s["accepted"] = torch.zeros((b,), dtype=torch.int32, **dev)
        return s
    s["T"] = torch.tensor(s["t"], **dev)
    if "n" in s:
        s["len"] = torch.tensor(s["n"], **dev)
    for x in ("", "1", "2"):
        if "qn" + x in s:
            s["out" + x] = torch.zeros(s["qn" + x].shape[:3] + (DV,), dtype=torch.float16, **dev)
    if c["op"] == "latent_run":
        s["freq"] = _freq(DR).cuda()
    if c["op"] == "latent_attn" and not own:
        s["cache"] = _pack(s["c"], s["T"] - c["R"], c)
    if own and c["op"] != "latent_prompt":
        s["handle"] = K.LatentCache(b, c["r"], bits=c["bits"], G=c["G"], R=c["R"], max_tokens=c["t"] + c["n"] + 1)
        if c["op"] == "latent_attn":
            s["handle"].prefill(s["c"], s["kr"], s["t"])
            del s["c"]
        else:
            s["rope"] = K.Rope(DR, inv_freq=_freq(DR).tolist())
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


def _pack(x, quantized, c):
    """Latent vectors [b, t, r] in plain tensors: codes, 16-bit scales and zeros, the vectors, how many are quantized."""
    b, t, r = x.shape
    code, s, z = _quant(x.view(b, t, r // c["G"], c["G"]), c["bits"])
    return {"code": code, "s": s, "z": z, "c": x, "quantized": quantized.view(b, 1, 1)}


def _unpack(p):
    """Latent vectors as attention sees them."""
    x = (p["code"].to(F32) * p["s"].to(F32) + p["z"].to(F32)).view(p["c"].shape)
    return torch.where(torch.arange(x.shape[1], device="cuda").view(1, -1, 1) < p["quantized"], x, p["c"].to(F32))


def _softmax(s, see):
    """Weights of scores s [b, h, n, S] where see [b, 1, n, S], in place."""
    s.mul_(1.0 / math.sqrt(DN + DR)).masked_fill_(~see, -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    return s.div_(s.sum(-1, keepdim=True).clamp_min(1e-30))


def _absorbed(qn, qr, c, kr, wk, wv, see):
    """Latent attention with the heads' products on the query's and the output's side."""
    b, h, n, _ = qn.shape
    r, S = c.shape[2], c.shape[1]
    ql = torch.matmul(qn.to(F32), wk.to(F32))
    s = torch.matmul(ql.view(b, h * n, r), c.transpose(1, 2))
    s += torch.matmul(qr.to(F32).reshape(b, h * n, DR), kr.to(F32).transpose(1, 2))
    w = _softmax(s.view(b, h, n, S), see)
    o = torch.matmul(w.view(b, h * n, S), c).view(b, h, n, r)
    return torch.matmul(o, wv.to(F32).transpose(1, 2))


def _expanded(qn, qr, c, kr, wk, wv, see):
    """Latent attention with every head's keys and values formed."""
    c = c.to(F32).unsqueeze(1)
    k, v = torch.matmul(c, wk.to(F32).transpose(1, 2)), torch.matmul(c, wv.to(F32).transpose(1, 2))
    s = torch.matmul(qn.to(F32), k.transpose(2, 3))
    s += torch.matmul(qr.to(F32), kr.to(F32).unsqueeze(1).transpose(2, 3))
    return torch.matmul(_softmax(s, see), v)


def _turn(x, angle, interleaved=False):
    """x [b, h, n, d] by angles [b, n, pairs]."""
    rot = 2 * angle.shape[2]
    cos, sin = torch.cos(angle).to(F32).unsqueeze(1), torch.sin(angle).to(F32).unsqueeze(1)
    y = x.to(F32)
    r = y[..., :rot]
    e, o = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rot // 2], r[..., rot // 2:])
    e, o = e * cos - o * sin, o * cos + e * sin
    r = torch.stack((e, o), -1).flatten(-2) if interleaved else torch.cat((e, o), -1)
    return torch.cat((r, y[..., rot:]), -1)


def _inside(lens, n):
    return torch.arange(n, device="cuda").view(1, n) < lens.view(-1, 1)


def _fixed(p):
    """Probabilities in units of 2^-40, rounded down (not a number and below 0: 0; above 1: 1)."""
    return (torch.where(p > 0, p.to(F64).clamp_max(1.0), 0.0) * 2.0 ** 40).long()


def _plain_verify(s):
    c = s["case"]
    b, n, V = c["b"], c["n"], c["vocab"]
    p, draft = s["p"], s["draft"].long()
    at = torch.arange(n, device="cuda").view(1, n)
    px = torch.gather(p[:, :n], 2, draft.unsqueeze(2)).squeeze(2).to(F64)
    qx = torch.ones_like(px) if s["q"] is None else torch.gather(s["q"], 2, draft.unsqueeze(2)).squeeze(2).to(F64)
    kept = (s["u"][:, :n].to(F64) * qx < px) & (at < s["len"].view(b, 1))
    first = kept.int().cumprod(1).sum(1)                       # the first that is not kept, or the row's length
    pf = _fixed(torch.gather(p, 1, first.view(b, 1, 1).expand(b, 1, V)).squeeze(1))
    row = first.clamp_max(n - 1).view(b, 1)
    if s["q"] is None:
        qf = torch.zeros_like(pf).scatter_(1, torch.gather(draft, 1, row), 2 ** 40)
    else:
        qf = _fixed(torch.gather(s["q"], 1, row.unsqueeze(2).expand(b, 1, V)).squeeze(1))
    rejected = first < s["len"]
    w = torch.where(rejected.view(b, 1), (pf - qf).clamp_min(0), pf)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, pf)
    total = w.sum(1)
    u = (s["u"][:, n].to(F64).clamp(0.0, 1.0 - 2.0 ** -24) * 2.0 ** 30).long()
    mark = u * (total >> 30) + ((u * (total & (2 ** 30 - 1))) >> 30)          # floor(u total / 2^30)
    token = (w.cumsum(1) <= mark.view(b, 1)).sum(1)
    token = torch.where(total > 0, token, -1)
    at = torch.arange(n + 1, device="cuda").view(1, n + 1)
    out = torch.where(at < first.view(b, 1), torch.nn.functional.pad(draft, (0, 1)), -1)
    out = torch.where(at == first.view(b, 1), token.view(b, 1), out)
    return out.int(), first.int()


def _run_plain(s):
    c = s["case"]
    op, b = c["op"], c["b"]
    if op == "axes":
        angle = s["pos"].to(F64)[s["axis"]].permute(1, 2, 0) * s["freq"]
        keep = _inside(s["len"], c["n"]).view(b, 1, c["n"], 1)
        return tuple(torch.where(keep, _turn(s[x], angle, c["interleaved"]), 0.0).half() for x in ("q", "k"))
    if op == "verify":
        return _plain_verify(s)
    t, n, wk, wv = c["t"], c["n"], s["wk"], s["wv"]
    at = torch.arange(t, device="cuda").expand(b, t)
    inside = _inside(s["T"], t)

    def see(pos, kpos, kok):
        return (kok.view(b, 1, 1, -1) & (kpos.view(b, 1, 1, -1) <= pos.reshape(b, 1, -1, 1)))

    pos1 = s["T"].view(b, 1) + torch.arange(max(n, 1), device="cuda")
    if op == "latent_prompt":
        o = _expanded(s["qn"], s["qr"], s["c"], s["kr"], wk, wv, see(at, at, inside))
        return torch.where(inside.view(b, 1, t, 1), o, 0.0).half()
    keep = _inside(s["len"], n)
    see1 = see(pos1, torch.cat((at, pos1), 1), torch.cat((inside, keep), 1))
    if op == "latent_attn":
        o = _absorbed(s["qn1"], s["qr1"], torch.cat((_unpack(s["cache"]), s["c1"].to(F32)), 1),
                      torch.cat((s["kr"], s["kr1"]), 1), wk, wv, see1)
        return torch.where(keep.view(b, 1, n, 1), o, 0.0).half()
    total = s["T"] + s["len"]

    def turned(x, pos):
        return _turn(x, pos.to(F64).unsqueeze(2) * s["freq"]).half()

    qr, kr = turned(s["qr"], at), turned(s["kr"].unsqueeze(1), at).squeeze(1)
    qr1, kr1 = turned(s["qr1"], pos1), turned(s["kr1"].unsqueeze(1), pos1).squeeze(1)
    qr2, kr2 = turned(s["qr2"], total.view(b, 1)), turned(s["kr2"].unsqueeze(1), total.view(b, 1)).squeeze(1)
    o = _expanded(s["qn"], qr, s["c"], kr, wk, wv, see(at, at, inside))
    o1 = _absorbed(s["qn1"], qr1, torch.cat((_unpack(_pack(s["c"], s["T"] - c["R"], c)), s["c1"].to(F32)), 1),
                   torch.cat((kr, kr1), 1), wk, wv, see1)
    # the sequences with the chunk behind their own last token
    src = torch.arange(t + n, device="cuda").expand(b, t + n)
    src = torch.where(src < s["T"].view(b, 1), src, src - s["T"].view(b, 1) + t).clamp_max(t + n - 1).unsqueeze(2)
    all_c = torch.cat((s["c"], s["c1"]), 1).gather(1, src.expand(b, t + n, c["r"]))
    all_kr = torch.cat((kr, kr1), 1).gather(1, src.expand(b, t + n, DR))
    at2 = torch.arange(t + n + 1, device="cuda").expand(b, t + n + 1)
    ok2 = (at2 < total.view(b, 1)) | (at2 == t + n)
    o2 = _absorbed(s["qn2"], qr2, torch.cat((_unpack(_pack(all_c, total - c["R"], c)), s["c2"].to(F32)), 1),
                   torch.cat((all_kr, kr2), 1), wk, wv, ok2.view(b, 1, 1, -1))
    return (torch.where(inside.view(b, 1, t, 1), o, 0.0).half(), torch.where(keep.view(b, 1, n, 1), o1, 0.0).half(),
            o2.half())


def run(state):
    s = state
    if not own:
        return _run_plain(s)
    from bit_quantized_kv_quantize_gb300 import kivi as K
    c, h = s["case"], s.get("handle")
    if c["op"] == "axes":
        return h.apply(s["q"], s["k"], s["pos"], n=s["n"], q_out=s["q_out"], k_out=s["k_out"])
    if c["op"] == "verify":
        return K.verify(s["p"], s["q"], s["draft"], s["u"], s["n"], tokens=s["tokens"], accepted=s["accepted"])
    wk, wv = s["wk"], s["wv"]
    if c["op"] == "latent_prompt":
        return K.latent_prompt_attn(s["qn"], s["qr"], s["c"], s["kr"], s["t"], wk, wv, out=s["out"])
    if c["op"] == "latent_attn":
        return h.attn(s["qn1"], s["qr1"], s["c1"], s["kr1"], s["n"], wk, wv, out=s["out1"])
    qr, kr = s["rope"].apply(s["qr"], s["kr"].unsqueeze(1), 0, n=s["t"])
    o = h.prefill_attn(s["qn"], qr, s["c"], kr.squeeze(1), s["t"], wk, wv, out=s["out"])
    o1 = h.extend(s["qn1"], s["qr1"], s["c1"], s["kr1"], s["n"], wk, wv, rope=s["rope"], out=s["out1"])
    o2 = h.extend(s["qn2"], s["qr2"], s["c2"], s["kr2"], 1, wk, wv, rope=s["rope"], out=s["out2"])
    return o, o1, o2


# ---- what a pass cannot do without -------------------------------------------

def _cached_bytes(c, t):
    """A sequence's t cached tokens, the newest R of them in 16 bits."""
    full = min(t, c["R"])
    return (full * 2.0 * c["r"] + (t - full) * (c["r"] * c["bits"] / 8 + 4 * c["r"] / c["G"])) + t * 2.0 * DR


def _products(c, rows, pairs, tokens):
    """Operations of latent attention for rows (query, head), pairs (query, head, token) and tokens: the cheaper form."""
    absorbed = 2.0 * rows * c["r"] * (DN + DV) + pairs * 2.0 * (2 * c["r"] + DR)
    expanded = 2.0 * tokens * c["h"] * c["r"] * (DN + DV) + pairs * 2.0 * (DN + DR + DV)
    return min(absorbed, expanded)


def work(case):
    c = case
    b = c["b"]
    if c["op"] == "axes":
        tokens, heads = sum(_lens(1, c["n"], b, c["ragged"], 0)), c["hq"] + c["hkv"]
        return {"bytes": 4.0 * tokens * heads * c["d"] + 4.0 * tokens * len(c["sections"].split(",")),
                "flops": 3.0 * tokens * heads * c["rot"]}
    if c["op"] == "verify":
        # one row of the target's, and of the draft's where there is one
        rows = b * (1 if c["certain"] else 2)
        return {"bytes": rows * c["vocab"] * (2.0 if c["half"] else 4.0) + b * c["n"] * 20.0,
                "flops": 2.0 * rows * c["vocab"]}
    h, r = c["h"], c["r"]
    t = _lens(1, c["t"], b, c["ragged"], c["t"] // 4)
    n = _lens(2, c["n"], b, c["ragged"], 0) if c["n"] else [0] * b
    weights = 4.0 * h * DN * r
    io = 2.0 * (h * (DN + DR + DV) + r + DR)       # a token's queries, output, latent vector and rotary key
    prompt = {"bytes": weights + sum(t) * io,
              "flops": _products(c, sum(t) * h, h * sum(x * (x + 1) / 2 for x in t), sum(t))}
    if c["op"] == "latent_prompt":
        return prompt

    def piece(t, n):
        pairs = h * sum(y * x + y * (y + 1) / 2 for x, y in zip(t, n))
        return {"bytes": weights + sum(n) * io + sum(_cached_bytes(c, x) for x, y in zip(t, n) if y),
                "flops": _products(c, sum(n) * h, pairs, sum(x + y for x, y in zip(t, n) if y))}

    chunk = piece(t, n)
    if c["op"] == "latent_attn":
        return chunk
    step = piece([x + y for x, y in zip(t, n)], [1] * b)
    fill = sum(_cached_bytes(c, x + y + 1) for x, y in zip(t, n))
    return {"bytes": prompt["bytes"] + chunk["bytes"] + step["bytes"] + fill,
            "flops": prompt["flops"] + chunk["flops"] + step["flops"]}


# ---- the definition in 64 bits ------------------------------------------------

def _exact_quant(x, c):
    """Vectors x [m, r] replaced by zero + code * scale, in 64 bits from 16-bit scales and zeros."""
    m, r = x.shape
    x = x.to(F64).view(m, r // c["G"], c["G"])
    z = x.min(2, keepdim=True).values
    s = ((x.max(2, keepdim=True).values - z) / (2 ** c["bits"] - 1)).to(F32).half().to(F64)
    code = torch.nan_to_num(torch.round((x - z) / s)).clamp(0, 2 ** c["bits"] - 1)
    return torch.where(s > 0, z + s * code, z).view(m, r)


def _exact_cache(x, c):
    """One sequence's latent vectors [t, r] as the cache restores them."""
    k = max(0, x.shape[0] - c["R"])
    return torch.cat((_exact_quant(x[:k], c), x[k:].to(F64))) if k else x.to(F64)


def _exact_rows(qn, qr, lat, kr, wk, wv, first):
    """One head's rows at positions first.. over tokens at positions 0.. (64 bits).  Few rows: the products on their
    side; many: every key and value."""
    n, S = qn.shape[0], lat.shape[0]
    qn, wk, wv = qn.to(F64), wk.to(F64), wv.to(F64)
    x = (qn @ wk) @ lat.t() if n < 200 else qn @ (lat @ wk.t()).t()
    x = (x + qr.to(F64) @ kr.to(F64).t()) / math.sqrt(DN + DR)
    hidden = torch.arange(S, device="cuda").view(1, S) > torch.arange(first, first + n, device="cuda").view(n, 1)
    w = torch.softmax(x.masked_fill_(hidden, -math.inf), -1)
    return (w @ lat) @ wv.t() if n < 200 else w @ (lat @ wv.t())


def _exact_turn(x, p, axis, f, interleaved=False):
    """Rows x [n, d] at positions p [A, n], as complex numbers times exp(i p f)."""
    x, rot = x.to(F64), 2 * f.shape[0]
    n = x.shape[0]
    a = torch.stack([p[axis[m]].to(F64) * f[m] for m in range(rot // 2)], 1)
    turn = torch.polar(torch.ones_like(a), a)
    if interleaved:
        y = torch.view_as_real(torch.view_as_complex(x[:, :rot].reshape(n, rot // 2, 2).contiguous()) * turn).reshape(n, rot)
    else:
        y = torch.complex(x[:, : rot // 2].contiguous(), x[:, rot // 2:rot].contiguous()) * turn
        y = torch.cat((y.real, y.imag), 1)
    return torch.cat((y, x[:, rot:]), 1)


def _exact_verify(c, s):
    """Each sequence's tokens by whole numbers, one sequence at a time."""
    import numpy as np
    b, n, V = c["b"], c["n"], c["vocab"]

    def units(row):
        x = row.double().cpu().numpy()
        return np.floor(np.where(x > 0, np.minimum(x, 1.0), 0.0) * 2.0 ** 40).astype(np.int64)

    out, kept = np.full((b, n + 1), -1, np.int32), np.zeros(b, np.int32)
    draft, u = s["draft"].cpu().numpy(), s["u"].double().cpu().numpy()
    for i in range(b):
        r = 0
        while r < s["n"][i]:
            x = int(draft[i, r])
            if not u[i, r] * (1.0 if s["q"] is None else float(s["q"][i, r, x])) < float(s["p"][i, r, x]):
                break
            out[i, r] = x
            r += 1
        kept[i] = r
        p = units(s["p"][i, r])
        w = p
        if r < s["n"][i]:
            if s["q"] is None:
                w = p.copy()
                w[draft[i, r]] = 0
            else:
                w = np.maximum(p - units(s["q"][i, r]), 0)
            if not w.any():
                w = p
        total = int(w.sum())
        if total:
            mark = int(min(max(u[i, n], 0.0), 1.0 - 2.0 ** -24) * 2.0 ** 30) * total >> 30
            out[i, r] = np.searchsorted(np.cumsum(w), mark, side="right")
    return torch.from_numpy(out).cuda(), torch.from_numpy(kept).cuda()


def exact(case, seed):
    c = case
    s = _data(c, seed)
    b = c["b"]
    if c["op"] == "verify":
        return _exact_verify(c, s)
    if c["op"] == "axes":
        out = [torch.zeros(s[x].shape, dtype=F64, device="cuda") for x in ("q", "k")]
        axis, f = _axis_of_pairs(c), _freq(c["rot"]).cuda()
        for o, x in zip(out, (s["q"], s["k"])):
            for i in range(b):
                m = s["n"][i]
                rows = x[i, :, :m].reshape(-1, c["d"])
                o[i, :, :m] = _exact_turn(rows, s["pos"][:, i, :m].repeat(1, x.shape[1]), axis, f,
                                          c["interleaved"]).view(-1, m, c["d"])
        return tuple(out)
    f, same = _freq(DR).cuda(), [0] * (DR // 2)

    def turned(x, first):
        """x [heads, n, 64] at positions first.."""
        return torch.stack([_exact_turn(y, torch.arange(first, first + y.shape[0], device="cuda").view(1, -1), same, f).half()
                            for y in x])

    outs = {x: torch.zeros(s["qn" + x].shape[:3] + (DV,), dtype=F64, device="cuda") for x in ("", "1", "2") if "qn" + x in s}
    for i in range(b):
        t = s["t"][i]
        lat, kr = s["c"][i, :t], s["kr"][i, :t]
        if c["op"] == "latent_run":
            kr = turned(kr.unsqueeze(0), 0)[0]
        if "" in outs:
            qr = s["qr"][i, :, :t]
            qr = turned(qr, 0) if c["op"] == "latent_run" else qr
            for e in range(c["h"]):
                outs[""][i, e, :t] = _exact_rows(s["qn"][i, e, :t], qr[e], lat.to(F64), kr, s["wk"][e], s["wv"][e], 0)
        for x, n in (("1", s["n"][i] if "n" in s else 0), ("2", 1)):
            if x not in outs or n == 0:
                continue
            first = lat.shape[0]
            new, kn, qr = s["c" + x][i, :n], s["kr" + x][i, :n], s["qr" + x][i, :, :n]
            if c["op"] == "latent_run":
                kn, qr = turned(kn.unsqueeze(0), first)[0], turned(qr, first)
            seen, kr = torch.cat((_exact_cache(lat, c), new.to(F64))), torch.cat((kr, kn))
            for e in range(c["h"]):
                outs[x][i, e, :n] = _exact_rows(s["qn" + x][i, e, :n], qr[e], seen, kr, s["wk"][e], s["wv"][e], first)
            lat = torch.cat((lat, new))
    outs = tuple(outs.values())
    return outs if len(outs) > 1 else outs[0]
