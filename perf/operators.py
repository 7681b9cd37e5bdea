"""Cases for timing the decoder-layer operators around the quantized linears.

Four operators: the residual update with the norms before and after a block
(``norm``), rotary positions (``rope``), the quantized paged key/value cache,
written and read back (``write``, ``read``), and attention of decode rows or
of a tree of drafted tokens over that cache (``attn``).  ``run`` computes
them with elementary torch operations, or, with ``own``, through this
package's entry points on the same state.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


def w4():
    import bit_weight_quantized_w4a8_gb300 as m
    return m


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one decode row between two linears: latency
        {"name": "norm 1 row", "op": "norm", "rows": 1, "n": 3584, "y": "float32", "r": "float32",
         "post": False, "gate": False, "alpha": 1.0, "beta": 1.0},
        # a decode batch: norm after the block, learned gate, 16-bit residual
        {"name": "norm 64 rows, post, gate", "op": "norm", "rows": 64, "n": 3584, "y": "float32", "r": "float16",
         "post": True, "gate": True, "alpha": 1.0, "beta": 0.5},
        # a prompt: bandwidth
        {"name": "norm 12289 rows", "op": "norm", "rows": 12289, "n": 4096, "y": "float32", "r": "float32",
         "post": False, "gate": False, "alpha": 1.25, "beta": 1.0},
        # queries of one decode row, half layout, far position
        {"name": "rope 1 row", "op": "rope", "rows": 1, "heads": 28, "dim": 128, "rot": 128, "inter": False,
         "x": "float32", "out": "float16", "base": 1e6, "factor": 1.0, "far": 131072},
        # queries of a long prompt, interleaved layout on half of the head, interpolated positions
        {"name": "rope 8191 rows", "op": "rope", "rows": 8191, "heads": 32, "dim": 128, "rot": 64, "inter": True,
         "x": "float32", "out": "float16", "base": 1e4, "factor": 8.0, "far": 32768},
        # a decode batch: q, k rotated, k and v quantized into the pages, read back
        {"name": "write 7 tokens", "op": "write", "seqs": 7, "tok": 1, "ctx": 4096, "hq": 28, "hkv": 4, "dim": 128,
         "page": 64, "bits": 8, "x": "float32", "rot": 128, "inter": False, "base": 1e6},
        # a prompt written into the cache and read back
        {"name": "write 8190 tokens", "op": "write", "seqs": 5, "tok": 1638, "ctx": 300, "hq": 32, "hkv": 2,
         "dim": 128, "page": 32, "bits": 8, "x": "float32", "rot": 64, "inter": True, "base": 1e4},
        # a long 4-bit cache read back
        {"name": "read 200000 tokens, 4 bits", "op": "read", "seqs": 3, "tok": 66666, "ctx": 0, "hkv": 4, "dim": 128,
         "page": 64, "bits": 4},
        # one token over a short cache: latency
        {"name": "attn 1 token", "op": "attn", "seqs": 1, "tok": 1, "ctx": 2047, "hq": 28, "hkv": 4, "dim": 128,
         "page": 64, "bits": 8, "tree": False},
        # a decode batch of ragged contexts
        {"name": "attn 24 sequences", "op": "attn", "seqs": 24, "tok": 1, "ctx": 32768, "hq": 28, "hkv": 4, "dim": 128,
         "page": 64, "bits": 8, "tree": False},
        # small trees over a 4-bit cache
        {"name": "attn trees of 9, 4 bits", "op": "attn", "seqs": 6, "tok": 9, "ctx": 30001, "hq": 32, "hkv": 2,
         "dim": 128, "page": 32, "bits": 4, "tree": True},
        # the largest trees over a long cache
        {"name": "attn trees of 64", "op": "attn", "seqs": 4, "tok": 64, "ctx": 32001, "hq": 28, "hkv": 4, "dim": 128,
         "page": 64, "bits": 8, "tree": True},
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rope", "write", "read", "attn", "attn"])
    ft = lambda: rng.choice(["float32", "float16"])  # noqa: E731
    if op == "norm":
        n = rng.choice([896, 3584, 4096, 8 * rng.randint(64, 1024), rng.randint(500, 9000)])
        rows = _logu(rng, 1, max(1, 50_000_000 // n))
        return {"op": op, "rows": rows, "n": n, "y": ft(), "r": ft(), "post": rng.random() < 0.5,
                "gate": rng.random() < 0.5, "alpha": rng.choice([1.0, 1.25, 0.8]), "beta": rng.choice([1.0, 0.3])}
    dim = rng.choice([64, 128, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    bits = rng.choice([8, 8, 4])
    rot = rng.choice([dim, dim // 2, dim // 4])
    inter = rng.random() < 0.5
    base = rng.choice([1e4, 1e6])
    if op == "rope":
        rows = _logu(rng, 1, max(1, 33_000_000 // (hq * dim)))
        return {"op": op, "rows": rows, "heads": hq, "dim": dim, "rot": rot, "inter": inter, "x": ft(), "out": ft(),
                "base": base, "factor": rng.choice([1.0, 4.0, 8.0]), "far": _logu(rng, 512, 1_000_000)}
    if op == "write":
        tokens = _logu(rng, 1, max(1, 36_000_000 // ((hq + 2 * hkv) * dim)))
        seqs = min(tokens, _logu(rng, 1, 64))
        # a 4-bit code next to a border is a coarse step: those keys come without positions
        return {"op": op, "seqs": seqs, "tok": max(1, tokens // seqs), "ctx": rng.randint(0, 3000), "hq": hq, "hkv": hkv,
                "dim": dim, "page": page, "bits": bits, "x": ft(), "rot": rot if bits == 8 else 0, "inter": inter,
                "base": base}
    if op == "read":
        tokens = _logu(rng, 1, 100_000_000 // (hkv * dim))
        seqs = min(tokens, _logu(rng, 1, 64))
        return {"op": op, "seqs": seqs, "tok": max(1, tokens // seqs), "ctx": rng.randint(0, 3000), "hkv": hkv,
                "dim": dim, "page": page, "bits": bits}
    tree = rng.random() < 0.6
    tok = _logu(rng, 1, 64) if tree else 1
    seqs = _logu(rng, 1, 32)
    # cached elements, and products with them, no more than the largest listed cases have
    most = min(300_000_000 / (seqs * hkv * dim), 14_000_000_000 / (seqs * tok * hq * dim), 130_000)
    ctx = _logu(rng, 1, max(2, int(most)))
    return {"op": op, "seqs": seqs, "tok": tok, "ctx": ctx, "hq": hq, "hkv": hkv, "dim": dim, "page": page,
            "bits": bits, "tree": tree}


def _lens(case):
    """Tokens and cached tokens of each sequence: ragged, a function of the case alone."""
    b = np.arange(case["seqs"])
    tok = case["tok"] - (b * 7) % (case["tok"] // 4 + 1)
    ctx = case["ctx"] - (b * 977) % (case["ctx"] // 3 + 1)
    return tok, ctx


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype="float32", std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(getattr(torch, dtype))


def _freqs(case):
    i = np.arange(case["rot"] // 2, dtype=np.float64)
    f = case["base"] ** (-2.0 * i / max(1, case["rot"])) / case.get("factor", 1.0)
    return torch.from_numpy(f).to(DEV)


def _pages(case, g):
    """Sequence offsets, starts and a page table over a shuffled pool."""
    tok, ctx = _lens(case)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(tok)]).astype(np.int32)).to(DEV)
    start = torch.from_numpy(ctx.astype(np.int32)).to(DEV)
    need = -(-(tok + ctx) // case["page"])
    width, pool = int(need.max()), int(need.sum()) + 3
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)[None, :]
    first = torch.from_numpy(np.concatenate([[0], np.cumsum(need)[:-1]])).to(DEV)[:, None]
    used = col < torch.from_numpy(need).to(DEV)[:, None]
    table = torch.where(used, perm[torch.where(used, first + col, 0)], 0).to(torch.int32).contiguous()
    return cu, start, table, pool


def _cache(case, g, pool, fill):
    shape = (pool, case["hkv"], case["page"])
    k, v = ({8: torch.zeros(shape + (case["dim"],), dtype=torch.int8, device=DEV),
             4: torch.zeros(shape + (case["dim"] // 2,), dtype=torch.uint8, device=DEV)}[case["bits"]]
            for _ in range(2))
    ks, vs = (torch.zeros(shape, device=DEV) for _ in range(2))
    if fill:  # what the quantizer leaves of normal keys and values
        for c, s in ((k, ks), (v, vs)):
            if case["bits"] == 8:
                c.copy_(torch.randn(c.shape, generator=g, device=DEV).mul_(42).round_().clamp_(-127, 127))
                s.copy_(torch.exp(torch.randn(shape, generator=g, device=DEV) * 0.2) / 42)
            else:
                lo, hi = (torch.randn(c.shape, generator=g, device=DEV).mul_(2.5).round_().clamp_(-7, 7).to(torch.int32)
                          for _ in range(2))
                c.copy_((lo & 15) | ((hi & 15) << 4))
                s.copy_(torch.exp(torch.randn(shape, generator=g, device=DEV) * 0.2) / 2.5)
    return k, v, ks, vs


def _trees(case, seed):
    """For each token the set of drafted tokens it sees: itself and its ancestors."""
    rng = np.random.default_rng(seed)
    tok, _ = _lens(case)
    words = []
    for t in tok:
        seen = []
        for i in range(int(t)):
            p = int(rng.integers(-1, i)) if i else -1
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        words += seen
    return torch.from_numpy(np.array(words, dtype=np.uint64).view(np.int64).copy()).to(DEV)


def prepare(case, seed):
    g, c = _gen(seed), case
    if c["op"] == "norm":
        s = {"y": _normal(g, (c["rows"], c["n"]), c["y"]), "r": _normal(g, (c["rows"], c["n"]), c["r"], 3.0),
             "w": 1 + _normal(g, (c["n"],), std=0.1)}
        s["post"] = 1 + _normal(g, (c["n"],), std=0.1) if c["post"] else None
        s["gate"] = _normal(g, (c["n"],), std=0.5) if c["gate"] else None
    elif c["op"] == "rope":
        s = {"x": _normal(g, (c["rows"], c["heads"], c["dim"]), c["x"]), "freqs": _freqs(c),
             "pos": torch.randint(0, c["far"], (c["rows"],), generator=g, device=DEV, dtype=torch.int32)}
    else:
        cu, start, table, pool = _pages(c, g)
        k, v, ks, vs = _cache(c, g, pool, c["op"] != "write")
        s = {"cu": cu, "start": start, "table": table, "k": k, "v": v, "ks": ks, "vs": vs}
        n = int(_lens(c)[0].sum())
        if c["op"] == "write":
            s["Q"] = _normal(g, (n, c["hq"], c["dim"]), c["x"])
            s["K"] = _normal(g, (n, c["hkv"], c["dim"]), c["x"])
            s["V"] = _normal(g, (n, c["hkv"], c["dim"]), c["x"])
            tok, ctx = _lens(c)
            s["pos"] = torch.from_numpy(np.concatenate([x + np.arange(t) for t, x in zip(tok, ctx)]).astype(np.int32)).to(DEV)
            s["freqs"] = _freqs(c) if c["rot"] else None
        elif c["op"] == "attn":
            s["q"] = _normal(g, (n, c["hq"], c["dim"]), "float16")
            s["mask"] = _trees(c, seed) if c["tree"] else None
        s["tokens"], s["most"] = n, int(_lens(c)[0].max())
    s["case"] = case
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

EPS = 1e-6


def _rms(x):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


def _norm(s):
    c = s["case"]
    u = s["y"].float()
    if s["post"] is not None:
        u = _rms(u) * s["post"]
    if s["gate"] is not None:
        u = u * s["gate"]
    r = c["alpha"] * s["r"].float() + c["beta"] * u
    return [r.to(s["r"].dtype), (_rms(r) * s["w"]).half()]


def _rotate(x, pos, freqs, inter):
    """x [tokens][heads][dim] in 32 bits; angles of far positions in 64."""
    rot = 2 * freqs.numel()
    a = pos.double()[:, None] * freqs
    cos, sin = torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]
    x = x.float()
    if inter:
        p, q = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((p * cos - q * sin, q * cos + p * sin), -1).flatten(-2)
    else:
        p, q = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((p * cos - q * sin, q * cos + p * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _places(s):
    """Page and offset of each token's slot."""
    i = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(s["cu"].long(), i, right=True) - 1
    slot = s["start"].long()[b] + i - s["cu"].long()[b]
    page = s["k"].shape[2]
    return s["table"][b, slot // page].long(), slot % page


def _codes(x, bits):
    top = 127 if bits == 8 else 7
    sc = x.abs().amax(-1) / top
    q = torch.where(sc[..., None] > 0, x / sc[..., None], torch.zeros_like(x))
    q = (torch.sign(q) * torch.floor(q.abs().double() + 0.5)).clamp(-top, top).to(torch.int32)
    if bits == 4:
        return ((q[..., 0::2] & 15) | ((q[..., 1::2] & 15) << 4)).to(torch.uint8), sc
    return q.to(torch.int8), sc


def _values(codes):
    if codes.dtype == torch.int8:
        return codes.float()
    u = codes.to(torch.int32)
    n = torch.stack((u & 15, u >> 4), -1).flatten(-2)
    return (n - ((n & 8) << 1)).float()


def _read(s):
    page, at = _places(s)
    return [(_values(c[page, :, at]) * sc[page, :, at][..., None]).half() for c, sc in ((s["k"], s["ks"]), (s["v"], s["vs"]))]


def _write(s):
    c = s["case"]
    q, k, v = s["Q"].float(), s["K"].float(), s["V"].float()
    if s["freqs"] is not None:
        q, k = (_rotate(x, s["pos"], s["freqs"], c["inter"]) for x in (q, k))
    page, at = _places(s)
    s["k"][page, :, at], s["ks"][page, :, at] = _codes(k, c["bits"])
    s["v"][page, :, at], s["vs"][page, :, at] = _codes(v, c["bits"])
    return [q.half()] + _read(s)


def _attn(s):
    """All sequences at once, padded to the longest; a row that sees nothing gives 0."""
    c = s["case"]
    B, H, G, D, T = c["seqs"], c["hkv"], c["hq"] // c["hkv"], c["dim"], s["most"]
    cu, start = s["cu"].long(), s["start"].long()
    t = torch.arange(T, device=DEV)[None, :]
    live = t < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(live, cu[:-1, None] + t, 0)
    q = s["q"][at].float().view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    tab = s["table"].long()
    L = tab.shape[1] * c["page"]

    def whole(codes, sc):
        x = _values(codes[tab]) * sc[tab][..., None]  # [B][pages][H][page][D]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, L, D)

    j = torch.arange(L, device=DEV)[None, None, :] - start[:, None, None]  # place among the drafted tokens
    if s["mask"] is None:
        sees = j <= t[..., None]
    else:
        m = s["mask"][at][..., None]
        sees = (j < 0) | ((j < 64) & (((m >> j.clamp(0, 63)) & 1) == 1))
    sees = sees & (j < (cu[1:] - cu[:-1])[:, None, None]) & live[..., None]
    sees = sees[:, None, :, None, :].expand(B, 1, T, G, L).reshape(B, 1, T * G, L)
    p = (q @ whole(s["k"], s["ks"]).transpose(-1, -2)).div_(math.sqrt(D)).masked_fill_(~sees, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    o = (p @ whole(s["v"], s["vs"])) / p.sum(-1, keepdim=True).clamp_min(1e-37)
    o = o.view(B, H, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, H * G, D)
    return o[live].half()


PLAIN = {"norm": _norm, "rope": lambda s: _rotate(s["x"], s["pos"], s["freqs"], s["case"]["inter"]).to(
    getattr(torch, s["case"]["out"])), "write": _write, "read": _read, "attn": _attn}


def run(state):
    s, c = state, state["case"]
    if not own:
        return PLAIN[c["op"]](s)
    m = w4()
    if c["op"] == "norm":
        return list(m.add_norm(s["r"], s["w"], y=s["y"], post_w=s["post"], gate=s["gate"], alpha=c["alpha"],
                               beta=c["beta"], eps=EPS))
    if c["op"] == "rope":
        return m.rope_rotate(s["x"], s["pos"], s["freqs"], interleaved=c["inter"], dtype=getattr(torch, c["out"]))
    cache, batch = m.KVQCache(s["k"], s["v"], s["ks"], s["vs"]), m.KVQBatch(s["cu"], s["start"], s["table"])
    if c["op"] == "attn":
        return m.kvq_attention(s["q"], cache, batch, mask=s["mask"])
    if c["op"] == "read":
        return list(m.kvq_read(cache, batch, s["tokens"]))
    q = m.kvq_write(cache, batch, s["K"], s["V"], Q=s["Q"], pos=s["pos"], freqs=s["freqs"], interleaved=c["inter"])
    return [q] + list(m.kvq_read(cache, batch, s["tokens"]))


# --------------------------------------------------------------------------
# least work
# --------------------------------------------------------------------------

SIZE = {"float32": 4, "float16": 2}


def work(case):
    c = case
    if c["op"] == "norm":
        mn = c["rows"] * c["n"]
        return {"bytes": mn * (SIZE[c["y"]] + 2 * SIZE[c["r"]] + 2) + 4 * c["n"] * (1 + c["post"] + c["gate"]),
                "flops": 8 * mn}
    if c["op"] == "rope":
        mn = c["rows"] * c["heads"] * c["dim"]
        return {"bytes": mn * (SIZE[c["x"]] + SIZE[c["out"]]) + 4 * c["rows"], "flops": 3 * mn}
    tok, ctx = _lens(c)
    n = int(tok.sum())
    vec = c["dim"] * c["bits"] // 8 + 4  # one key or value as it is held
    kv = n * c["hkv"] * c["dim"]
    if c["op"] == "write":
        return {"bytes": (n * c["hq"] * c["dim"] + 2 * kv) * (SIZE[c["x"]] + 2) + 2 * 2 * n * c["hkv"] * vec,
                "flops": 3 * n * c["hq"] * c["dim"] + 12 * kv}
    if c["op"] == "read":
        return {"bytes": 2 * n * c["hkv"] * vec + 2 * 2 * kv, "flops": 2 * kv}
    L = int((tok + ctx).sum())
    return {"bytes": 2 * L * c["hkv"] * vec + 2 * 2 * n * c["hq"] * c["dim"],
            "flops": 4 * int((tok * (tok + ctx)).sum()) * c["hq"] * c["dim"]}


# --------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# --------------------------------------------------------------------------

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        y, r = s["y"].double(), s["r"].double()
        if c["post"]:
            y = y * (y.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * s["post"].double()
        r = c["alpha"] * r + c["beta"] * (y if s["gate"] is None else s["gate"].double() * y)
        return [r, r * (r.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * s["w"].double()]

    def turn(x, pos, f):  # as complex numbers
        x, h = x.double(), f.numel()
        z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[:, None] * f)[:, None, :]
        out = x.clone()
        lo, hi = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if c["inter"] else (slice(0, h), slice(h, 2 * h))
        w = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * z
        out[..., lo], out[..., hi] = w.real, w.imag
        return out

    if c["op"] == "rope":
        return turn(s["x"], s["pos"], s["freqs"])
    if c["op"] == "write":
        q, k, v = s["Q"].double(), s["K"].double(), s["V"].double()
        if c["rot"]:
            q, k = turn(q, s["pos"], s["freqs"]), turn(k, s["pos"], s["freqs"])
        top = float(2 ** (c["bits"] - 1) - 1)

        def held(x):
            step = x.abs().max(-1, keepdim=True).values / top
            n = x / step.clamp_min(1e-300)
            return n.sign() * (n.abs() + 0.5).floor().clamp_max(top) * step

        return [q, held(k), held(v)]
    tok, ctx = _lens(c)

    def stored(codes, sc, b, lo, hi):  # values of slots lo..hi of sequence b, [slots][heads][dim]
        slot = torch.arange(lo, hi, device=DEV)
        pg = s["table"][b].long()[slot.div(c["page"], rounding_mode="floor")]
        x = codes[pg, :, slot.remainder(c["page"])]
        if c["bits"] == 4:
            u = x.long()
            x = torch.stack((u.remainder(16), u.div(16, rounding_mode="floor")), -1).flatten(-2)
            x = torch.where(x > 7, x - 16, x)
        return x.double() * sc[pg, :, slot.remainder(c["page"])].double()[..., None]

    if c["op"] == "read":
        return [torch.cat([stored(x, y, b, int(ctx[b]), int(ctx[b] + tok[b])) for b in range(c["seqs"])])
                for x, y in ((s["k"], s["ks"]), (s["v"], s["vs"]))]
    outs, G = [], c["hq"] // c["hkv"]
    for b in range(c["seqs"]):
        t, x, first = int(tok[b]), int(ctx[b]), int(s["cu"][b])
        k, v = (stored(a, y, b, 0, t + x) for a, y in ((s["k"], s["ks"]), (s["v"], s["vs"])))
        q = s["q"][first:first + t].double()
        see = torch.ones((t, t + x), dtype=torch.bool, device=DEV)
        if c["tree"]:
            words = s["mask"][first:first + t].cpu().numpy().view(np.uint64)
            own_bits = (words[:, None] >> np.arange(t, dtype=np.uint64)) & np.uint64(1)
            see[:, x:] = torch.from_numpy(own_bits.astype(bool)).to(DEV)
        else:
            see[:, x:] = torch.tril(see[:, x:])
        o = torch.zeros_like(q)
        for h in range(c["hkv"]):
            a = torch.einsum("tgd,ld->tgl", q[:, h * G:(h + 1) * G], k[:, h]) / c["dim"] ** 0.5
            a = torch.softmax(a.masked_fill(~see[:, None, :], -math.inf), -1)
            o[:, h * G:(h + 1) * G] = torch.einsum("tgl,ld->tgd", a, v[:, h])
        outs.append(o)
    return torch.cat(outs)
