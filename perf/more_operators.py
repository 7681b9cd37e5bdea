"""Cases for timing the operators of a serving step around the decoder layer.

Four operators: the linear with 8-bit floating-point weights and activations
and a scale for each block of 128 (``f8``), the verification of drafted tokens
against the target's logits (``verify``), the step's offsets, pages, positions
and slots from request lengths (``plan``), and rotary positions with several
axes, alone (``axes``) and in the cache's write (``axes_write``).  ``run``
computes them with elementary torch operations, or, with ``own``, through this
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
        # one decode row through an MLP projection: the weights' stream
        {"name": "f8 1 row", "op": "f8", "m": 1, "k": 3584, "n": 18944, "x": "float16", "y": "float32"},
        # a ragged decode batch through the projection with the long sum
        {"name": "f8 49 rows", "op": "f8", "m": 49, "k": 18944, "n": 3584, "x": "float16", "y": "float32"},
        # a short prompt through a fused q/k/v projection
        {"name": "f8 777 rows", "op": "f8", "m": 777, "k": 4096, "n": 4608, "x": "float16", "y": "float16"},
        # a batch of long prompts
        {"name": "f8 8192 rows", "op": "f8", "m": 8192, "k": 3584, "n": 18944, "x": "float16", "y": "float16"},
        # a chain of four drafted tokens, greedy: latency
        {"name": "verify 1 chain, greedy", "op": "verify", "seqs": 1, "tok": 5, "vocab": 152064, "l": "float32",
         "tree": False, "q": False, "greedy": True},
        # small trees without draft probabilities
        {"name": "verify 24 trees", "op": "verify", "seqs": 24, "tok": 12, "vocab": 152064, "l": "float32",
         "tree": True, "q": False, "greedy": False},
        # chains drawn from a draft model, with its probabilities
        {"name": "verify 61 chains, draft probabilities", "op": "verify", "seqs": 61, "tok": 6, "vocab": 152064,
         "l": "float32", "tree": False, "q": True, "greedy": False},
        # a decode step of 48 requests with five drafted tokens each
        {"name": "plan 48 requests", "op": "plan", "seqs": 48, "tok": 6, "ctx": 4000, "page": 64, "spare": 1.0,
         "swap": False},
        # half of many requests end, prompts take their places
        {"name": "plan 4093 requests", "op": "plan", "seqs": 4093, "tok": 257, "ctx": 1500, "page": 32, "spare": 1.0,
         "swap": True},
        # queries of one decode row behind an image: latency
        {"name": "axes 1 row", "op": "axes", "rows": 1, "heads": 28, "dim": 128, "rot": 128, "inter": False,
         "x": "float32", "out": "float16", "base": 1e6, "axes": 3, "cycled": False, "far": 131072},
        # a long prompt of images and text, interleaved axes on half of the head
        {"name": "axes 8191 rows", "op": "axes", "rows": 8191, "heads": 32, "dim": 128, "rot": 64, "inter": True,
         "x": "float32", "out": "float16", "base": 1e4, "axes": 3, "cycled": True, "far": 32768},
        # such prompts written into the cache and read back
        {"name": "axes write 8190 tokens", "op": "axes_write", "seqs": 5, "tok": 1638, "ctx": 300, "hq": 28, "hkv": 4,
         "dim": 128, "page": 64, "x": "float32", "rot": 128, "inter": False, "base": 1e6, "axes": 3, "cycled": False},
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["f8", "f8", "f8", "verify", "verify", "plan", "axes", "axes_write"])
    ft = lambda: rng.choice(["float32", "float16"])  # noqa: E731
    if op == "f8":
        k = rng.choice([3584, 4096, 13696, 18944, 16 * _logu(rng, 8, 1000)])
        n = rng.choice([512, 3584, 4608, 18944, _logu(rng, 64, 20000)])
        n = min(n, 67_000_000 // k)
        m = _logu(rng, 1, min(8192, 550_000_000_000 // (n * k)))
        return {"op": op, "m": m, "k": k, "n": n, "x": rng.choice(["float16", "float16", "float32"]), "y": ft()}
    if op == "verify":
        vocab = rng.choice([152064, 32000, 65024, _logu(rng, 1000, 160000)])
        tree = rng.random() < 0.5
        tok = _logu(rng, 1, 64 if tree else 16)
        seqs = _logu(rng, 1, max(1, min(64, 45_000_000 // (vocab * tok))))
        return {"op": op, "seqs": seqs, "tok": tok, "vocab": vocab, "l": ft(), "tree": tree, "q": rng.random() < 0.5,
                "greedy": rng.random() < 0.2}
    if op == "plan":
        seqs = _logu(rng, 1, 4093)
        tok = _logu(rng, 1, max(1, min(8000, 1_000_000 // seqs)))
        return {"op": op, "seqs": seqs, "tok": tok, "ctx": _logu(rng, 1, max(1, min(100_000, 6_000_000 // seqs))),
                "page": rng.choice([16, 32, 64, 128, 256]), "spare": rng.choice([1.0, 1.0, 0.6]),
                "swap": rng.random() < 0.5}
    dim = rng.choice([64, 128, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 7, 8])
    rot = rng.choice([dim, dim // 2])
    common = {"dim": dim, "rot": rot, "inter": rng.random() < 0.5, "x": ft(), "base": rng.choice([1e4, 1e6]),
              "axes": rng.choice([2, 3, 3, 4]), "cycled": rng.random() < 0.5}
    if op == "axes":
        rows = _logu(rng, 1, max(1, 33_000_000 // (hq * dim)))
        return {"op": op, "rows": rows, "heads": hq, "out": ft(), "far": _logu(rng, 512, 1_000_000), **common}
    tokens = _logu(rng, 1, max(1, 36_000_000 // ((hq + 2 * hkv) * dim)))
    seqs = min(tokens, _logu(rng, 1, 64))
    return {"op": op, "seqs": seqs, "tok": max(1, tokens // seqs), "ctx": rng.randint(0, 3000), "hq": hq, "hkv": hkv,
            "page": rng.choice([16, 32, 64, 128]), **common}


def _lens(case):
    """Tokens and cached tokens of each sequence: ragged, a function of the case alone."""
    b = np.arange(case["seqs"])
    tok = case["tok"] - (b * 7) % (case["tok"] // 4 + 1)
    ctx = case.get("ctx", 0) - (b * 977) % (case.get("ctx", 0) // 3 + 1)
    return tok, ctx


def _sections(case):
    """Pairs of each axis: the first has the fewest, as time does."""
    a, h = case["axes"], case["rot"] // 2
    rest = (h + a - 1) // a + (1 if h > 2 * a else 0)
    return [h - rest * (a - 1)] + [rest] * (a - 1)


def _axis_of(case):
    """Axis of each pair: blocks of pairs, or the axes in turn for as long as each has pairs left."""
    sec = _sections(case)
    if not case["cycled"]:
        return [a for a, n in enumerate(sec) for _ in range(n)]
    left, out = list(sec), []
    while len(out) < sum(sec):
        for a in range(len(sec)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype="float32", std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(getattr(torch, dtype))


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a), dtype=np.int32)).to(DEV)


def _prep_f8(c, g):
    k, n = c["k"], c["n"]
    x = torch.randn((c["m"], k), generator=g, device=DEV)
    x = x * torch.where(torch.rand(x.shape, generator=g, device=DEV) < 1e-3, 20.0, 1.0)  # outliers
    w = torch.randn((n, k), generator=g, device=DEV) * 0.02
    kb, nb = -(-k // 128), -(-n // 128)
    pad = torch.nn.functional.pad(w.abs(), (0, kb * 128 - k, 0, nb * 128 - n))
    sw = pad.view(nb, 128, kb, 128).amax((1, 3)) / 448.0
    each = sw.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    wf = (w / each).to(torch.float8_e4m3fn).view(torch.uint8)
    return {"x": x.to(getattr(torch, c["x"])).contiguous(), "wf": wf.contiguous(), "sw": sw.contiguous()}


def _trees(c, seed):
    """Parents (index in the sequence, -1 for the root) and the bit words of ancestors and self."""
    rng = np.random.default_rng(seed)
    parents, words = [], []
    for t in _lens(c)[0]:
        seen = []
        for i in range(int(t)):
            p = -1 if i == 0 else int(rng.integers(max(0, i - 8), i)) if c["tree"] else i - 1
            parents.append(p)
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        words += seen
    return np.array(parents), torch.from_numpy(np.array(words, dtype=np.uint64).view(np.int64).copy()).to(DEV)


def _prep_verify(c, g, seed):
    tok, _ = _lens(c)
    n, v = int(tok.sum()), c["vocab"]
    cu = np.concatenate([[0], np.cumsum(tok)])
    logits = torch.randn((n, v), generator=g, device=DEV) * 2
    at = torch.randint(0, v, (n, 24), generator=g, device=DEV)  # a few likely tokens a row
    logits.scatter_(1, at, 6 + 8 * torch.rand((n, 24), generator=g, device=DEV))
    logits = logits.to(getattr(torch, c["l"]))
    temp = torch.rand(c["seqs"], generator=g, device=DEV) * 0.6 + 0.6
    if c["greedy"]:
        temp.zero_()
    draft = logits.float() + torch.randn((n, v), generator=g, device=DEV) * 0.4  # a draft model: close, not equal
    parents, mask = _trees(c, seed)
    first = np.repeat(cu[:-1], tok)
    parent_row = torch.from_numpy(np.where(parents < 0, np.arange(n), first + parents)).to(DEV)
    if c["q"]:
        q = torch.softmax(draft / torch.where(temp > 0, temp, 1.0).repeat_interleave(torch.from_numpy(tok).to(DEV))[:, None], 1)
        draft = None
        ids = torch.multinomial(q, int(tok.max()), replacement=True, generator=g)
        ids = ids[parent_row, torch.from_numpy(np.arange(n) - first).to(DEV)]
    else:
        q = None
        rank = np.zeros(n, dtype=np.int64)  # among its siblings
        seen = {}
        for t in range(n):
            key = (first[t], parents[t])
            rank[t] = seen.get(key, 0)
            seen[key] = rank[t] + 1
        top = torch.topk(draft, min(64, v), 1).indices
        ids = top[parent_row, torch.from_numpy(rank).to(DEV)]
    return {"logits": logits, "q": q, "ids": ids.to(torch.int32).contiguous(), "cu": _i32(cu),
            "mask": mask if c["tree"] else None, "parent": parents,
            "temp": temp, "u": torch.rand(n, generator=g, device=DEV), "most": int(tok.max())}


def _prep_plan(c, seed):
    """Requests with their pages held, all pages of the pool in a random order."""
    rng = np.random.default_rng(seed)
    tok, ctx = _lens(c)
    page, seqs = c["page"], c["seqs"]
    most = -(-(ctx + 200 + tok) // page)
    width, pages = int(most.max()) + 1, int(most.sum()) + 3
    ctx = ctx + rng.integers(0, 200, seqs)
    held = -(-ctx // page)
    ends = (np.arange(seqs) % 2 == 0) & c["swap"]
    if c["swap"]:  # not only in the rows' order; the others' next token fits their last page
        ends = ends[rng.permutation(seqs)]
        ctx = ctx | 1
        held = -(-ctx // page)
    after = -(-(np.where(ends, 0, ctx) + tok) // page)
    if c["swap"]:
        after = np.where(ends, after, -(-(ctx + 1) // page))
    more = int(np.maximum(after - np.where(ends, 0, held), 0).sum()) - int(held[ends].sum())
    free = pages - int(held.sum())
    if c["spare"] < 1.0:  # fewer than this step wants: the last requests have to wait
        free = max(0, int(more * c["spare"]))
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((seqs, width), -1, dtype=np.int32)
    at = 0
    for b in range(seqs):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    stack = np.full(pages, -1, dtype=np.int32)
    stack[:free] = perm[at:at + free]
    s = {"table": _i32(table), "held": _i32(held), "stack": _i32(stack), "top": _i32([free]), "lens": _i32(ctx),
         "out": _i32(np.where(ends, -1, 0)), "add": _i32(tok), "tokens": int(tok.sum()) + 5}
    if c["swap"]:
        s["add"] = _i32(np.where(ends, tok, 1))
    return s


def _pages(c, g):
    tok, ctx = _lens(c)
    cu, start = _i32(np.concatenate([[0], np.cumsum(tok)])), _i32(ctx)
    need = -(-(tok + ctx) // c["page"])
    pool = int(need.sum()) + 3
    perm = torch.randperm(pool, generator=g, device=DEV).to(torch.int32).cpu().numpy()
    table = np.zeros((c["seqs"], int(need.max())), dtype=np.int32)
    at = 0
    for b in range(c["seqs"]):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    return cu, start, _i32(table), pool


def _prep_axes(c, g):
    i = np.arange(c["rot"] // 2, dtype=np.float64)
    s = {"freqs": torch.from_numpy(c["base"] ** (-2.0 * i / c["rot"])).to(DEV),
         "axis": torch.tensor(_axis_of(c), device=DEV), "axis_host": bytes(_axis_of(c))}
    if c["op"] == "axes":
        n = c["rows"]
        s["x"] = _normal(g, (n, c["heads"], c["dim"]), c["x"])
    else:
        s["cu"], s["start"], s["table"], pool = _pages(c, g)
        tok, ctx = _lens(c)
        n = int(tok.sum())
        shape = (pool, c["hkv"], c["page"])
        s["k"], s["v"] = (torch.zeros(shape + (c["dim"],), dtype=torch.int8, device=DEV) for _ in range(2))
        s["ks"], s["vs"] = (torch.zeros(shape, device=DEV) for _ in range(2))
        s["Q"] = _normal(g, (n, c["hq"], c["dim"]), c["x"])
        s["K"], s["V"] = (_normal(g, (n, c["hkv"], c["dim"]), c["x"]) for _ in range(2))
        s["tokens"] = n
    # text runs share one position on all axes, an image's tokens walk over rows and columns
    t = np.arange(n)
    base = _normal(g, ()).abs().mul(c.get("far", 4000)).long() % c.get("far", 4000)
    side = 17
    rows = [t // (side * side), t // side % side, t % side, t % 5][:c["axes"]]
    image = (t // 400) % 2 == 0
    pos = np.stack([np.where(image, r, t) for r in rows])
    s["pos"] = (torch.from_numpy(pos).to(DEV) + base).to(torch.int32).contiguous()
    return s


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"f8": lambda: _prep_f8(c, g), "verify": lambda: _prep_verify(c, g, seed), "plan": lambda: _prep_plan(c, seed),
         "axes": lambda: _prep_axes(c, g), "axes_write": lambda: _prep_axes(c, g)}[c["op"]]()
    s["case"] = case
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _e4m3(q):
    """Nearest number of four significant bits down to 2^-9, ties to even; |q| <= 448 up to a rounding."""
    e = torch.frexp(q)[1].clamp_min(-5) - 4  # exponent of the last place
    step = torch.ldexp(torch.ones_like(q), e)
    return (torch.round(q / step) * step).clamp_(-448.0, 448.0)


def _f8(s):
    c = s["case"]
    m, k, n = c["m"], c["k"], c["n"]
    kb = -(-k // 128)
    x = torch.nn.functional.pad(s["x"].float(), (0, kb * 128 - k)).view(m, kb, 128)
    sa = x.abs().amax(2, keepdim=True) * torch.tensor(1 / 448.0, dtype=torch.float32, device=DEV)
    q = torch.where(sa > 0, x.double() / sa.double(), 0.0)  # codes next to a border: the quotient in 64 bits
    x = (_e4m3(q).float() * sa).view(m, kb * 128)[:, :k]
    each = s["sw"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    w = s["wf"].view(torch.float8_e4m3fn).float() * each
    return (x @ w.t()).to(getattr(torch, c["y"]))


def _verify(s):
    """All sequences at once, drafted token by drafted token; sums in 64 bits."""
    c = s["case"]
    B, V, T = c["seqs"], c["vocab"], s["most"]
    cu, ids, u, temp = s["cu"].long(), s["ids"].long(), s["u"], s["temp"]
    n = ids.numel()
    tok = cu[1:] - cu[:-1]
    b = torch.arange(B, device=DEV)
    if s["mask"] is None:
        parent = torch.arange(n, device=DEV) - cu[torch.searchsorted(cu, torch.arange(n, device=DEV), right=True) - 1] - 1
    else:  # the highest ancestor
        own_at = torch.arange(n, device=DEV) - cu[torch.searchsorted(cu, torch.arange(n, device=DEV), right=True) - 1]
        bits = (s["mask"][:, None] >> torch.arange(64, device=DEV)) & 1
        at = torch.arange(64, device=DEV)[None, :]
        parent = torch.where((bits == 1) & (at < own_at[:, None]), at, -1).amax(1)
    greedy = (temp == 0)[:, None]
    safe = torch.where(temp == 0, 1.0, temp.double())[:, None]

    def weights(row):
        x = s["logits"][row].double()
        x = torch.exp((x - x.amax(1, keepdim=True)) / safe)
        one = torch.zeros_like(x).scatter_(1, s["logits"][row].argmax(1, keepdim=True), 1.0)
        return torch.where(greedy, one, x)

    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    e = weights(cu[:-1])
    total = e.sum(1)
    keep = torch.full((n + 1,), -1, dtype=torch.int32, device=DEV)
    out = torch.full((n + 1,), -1, dtype=torch.int32, device=DEV)
    keep[cu[:-1]] = 0
    count = torch.ones(B, dtype=torch.long, device=DEV)
    scale = total.clone()  # what the draft's probabilities are multiplied with
    for i in range(1, T):
        t = torch.where(i < tok, cu[:-1] + i, 0)
        test = (i < tok) & (parent[t] == cur)
        x = ids[t]
        w = e[b, x]
        if s["q"] is None:
            yes = test & (u[t].double() * total < w)
            e = torch.where((test & ~yes)[:, None], e.scatter(1, x[:, None], 0.0), e)
            total = torch.where(test & ~yes, total - w, total)
        else:
            q = s["q"][cu[:-1] + cur].double()
            yes = test & torch.where(greedy[:, 0], w > 0, u[t].double() * q[b, x] * scale < w)
            left = torch.where(greedy, e, (e - q * scale[:, None]).clamp_min(0))
            e = torch.where((test & ~yes)[:, None], left, e)
            total = torch.where(test & ~yes, left.sum(1), total)
            scale = torch.where(test & ~yes, total, scale)
        keep[torch.where(yes, cu[:-1] + count, n)] = i
        out[torch.where(yes, cu[:-1] + count - 1, n)] = x.to(torch.int32)
        count = count + yes.long()
        cur = torch.where(yes, i, cur)
        fresh = weights(cu[:-1] + cur)
        e = torch.where(yes[:, None], fresh, e)
        total = torch.where(yes, fresh.sum(1), total)
        scale = torch.where(yes, total, scale)
    run = e.cumsum(1)
    at = torch.searchsorted(run, (u[cu[:-1]].double() * run[:, -1])[:, None], right=True)[:, 0]
    out[cu[:-1] + count - 1] = at.clamp_max(V - 1).to(torch.int32)
    return [keep[:n].clone(), out[:n].clone(), count.to(torch.int32)]


def _plan_call(s, add):
    page, tokens = s["case"]["page"], s["tokens"]
    table, held, stack = s["table"], s["held"].long(), s["stack"]
    seqs, width = table.shape
    col = torch.arange(width, device=DEV)[None, :]
    lens, top = s["lens"].long(), s["top"].long()
    end = add < 0
    # pages come back, the last one first onto the stack
    back = torch.where(end, held, 0)
    before = back.cumsum(0) - back
    place = top + back.sum() - 1 - (before[:, None] + col)
    stack_w = torch.cat((stack, stack[:1]))
    gone = end[:, None] & (col < held[:, None])
    stack_w[torch.where(gone, place, stack.numel())] = table
    stack.copy_(stack_w[:-1])
    top = top + back.sum()
    held, lens = torch.where(end, 0, held), torch.where(end, 0, lens)
    # pages go out, rows in order, as far as they and the tokens reach
    n = add.clamp_min(0).long()
    want = (lens + n + page - 1) // page
    need = torch.where(n > 0, (want - held).clamp_min(0), 0)
    wide = want > width
    need = torch.where(wide, 0, need)
    fits = ~wide & ((need == 0) | (need.cumsum(0) <= top)) & (torch.where(wide, 0, n).cumsum(0) <= tokens)
    n, need = torch.where(fits, n, 0), torch.where(fits, need, 0)
    before = need.cumsum(0) - need
    k = col - held[:, None]
    new = (k >= 0) & (k < need[:, None])
    table.copy_(torch.where(new, stack[torch.where(new, top - 1 - before[:, None] - k, 0)], table))
    s["held"].copy_(held + need)
    s["top"].copy_(top - need.sum())
    s["lens"].copy_(lens)
    cu = torch.cat((torch.zeros(1, dtype=torch.long, device=DEV), n.cumsum(0)))
    i = torch.arange(tokens, device=DEV)
    live = i < cu[-1]
    b = torch.where(live, torch.searchsorted(cu, i, right=True) - 1, 0)
    pos = torch.where(live, lens[b] + i - cu[b], 0)
    slot = torch.where(live, table[b, pos // page].long() * page + pos % page, -1)
    return [cu.to(torch.int32), pos.to(torch.int32), slot, torch.where(live, b, -1).to(torch.int32)]


def _plan(s):
    if s["case"]["swap"]:
        _plan_call(s, s["out"])
    return _plan_call(s, s["add"]) + [s[k] for k in ("lens", "held", "table", "stack", "top")]


def _turn(x, s):
    """x [tokens][heads][dim] in 32 bits; angles of far positions in 64."""
    rot = 2 * s["freqs"].numel()
    a = s["pos"][s["axis"]].t().double() * s["freqs"]
    cos, sin = torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]
    x = x.float()
    if s["case"]["inter"]:
        p, q = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((p * cos - q * sin, q * cos + p * sin), -1).flatten(-2)
    else:
        p, q = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((p * cos - q * sin, q * cos + p * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _axes(s):
    return _turn(s["x"], s).to(getattr(torch, s["case"]["out"]))


def _axes_write(s):
    q, k, v = _turn(s["Q"], s), _turn(s["K"], s), s["V"].float()
    i = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(s["cu"].long(), i, right=True) - 1
    slot = s["start"].long()[b] + i - s["cu"].long()[b]
    page = s["k"].shape[2]
    pg, at = s["table"][b, slot // page].long(), slot % page
    outs = [q.half()]
    for x, c, sc in ((k, s["k"], s["ks"]), (v, s["v"], s["vs"])):
        step = x.abs().amax(-1) / 127
        r = torch.where(step[..., None] > 0, x / step[..., None], torch.zeros_like(x))
        c[pg, :, at] = (torch.sign(r) * torch.floor(r.abs().double() + 0.5)).clamp(-127, 127).to(torch.int8)
        sc[pg, :, at] = step
        outs.append((c[pg, :, at].float() * sc[pg, :, at][..., None]).half())
    return outs


PLAIN = {"f8": _f8, "verify": _verify, "plan": _plan, "axes": _axes, "axes_write": _axes_write}


def run(state):
    s, c = state, state["case"]
    if not own:
        return PLAIN[c["op"]](s)
    m = w4()
    if c["op"] == "f8":
        return m.f8_linear(s["x"], s["wf"], s["sw"], dtype=getattr(torch, c["y"]))
    if c["op"] == "verify":
        return list(m.draft_verify(s["logits"], s["cu"], s["ids"], s["u"], mask=s["mask"], q=s["q"], temp=s["temp"]))
    if c["op"] == "plan":
        pool = m.KVQPool(s["table"], s["held"], s["stack"], s["top"])
        if c["swap"]:
            m.kvq_plan(pool, c["page"], s["lens"], s["out"], s["tokens"])
        batch, pos, slot, seq = m.kvq_plan(pool, c["page"], s["lens"], s["add"], s["tokens"])
        return [batch.cu, pos, slot, seq] + [s[k] for k in ("lens", "held", "table", "stack", "top")]
    if c["op"] == "axes":
        return m.rope_rotate(s["x"], s["pos"], s["freqs"], interleaved=c["inter"], dtype=getattr(torch, c["out"]),
                             axis=s["axis_host"])
    cache, batch = m.KVQCache(s["k"], s["v"], s["ks"], s["vs"]), m.KVQBatch(s["cu"], s["start"], s["table"])
    q = m.kvq_write(cache, batch, s["K"], s["V"], Q=s["Q"], pos=s["pos"], freqs=s["freqs"], interleaved=c["inter"],
                    axis=s["axis_host"])
    return [q] + list(m.kvq_read(cache, batch, s["tokens"]))


# --------------------------------------------------------------------------
# least work
# --------------------------------------------------------------------------

SIZE = {"float32": 4, "float16": 2}


def work(case):
    c = case
    if c["op"] == "f8":
        m, k, n = c["m"], c["k"], c["n"]
        kb, nb = -(-k // 128), -(-n // 128)
        return {"bytes": m * k * SIZE[c["x"]] + n * k + 4 * kb * nb + m * n * SIZE[c["y"]], "flops": 2 * m * n * k}
    if c["op"] == "verify":
        n = int(_lens(c)[0].sum())
        # all logits, and of the draft's probabilities the row of each sequence's last token
        return {"bytes": n * c["vocab"] * SIZE[c["l"]] + (4 * c["seqs"] * c["vocab"] if c["q"] else 0) + 20 * n,
                "flops": 4 * n * c["vocab"]}
    if c["op"] == "plan":
        tok, ctx = _lens(c)
        pages = int((-(-(tok + ctx) // c["page"]) - -(-ctx // c["page"])).sum())
        calls = 2 if c["swap"] else 1
        return {"bytes": calls * (24 * c["seqs"] + 16 * (int(tok.sum()) + 5)) + 8 * pages,
                "flops": calls * (8 * c["seqs"] + 4 * int(tok.sum()))}
    if c["op"] == "axes":
        mn = c["rows"] * c["heads"] * c["dim"]
        return {"bytes": mn * (SIZE[c["x"]] + SIZE[c["out"]]) + 4 * c["axes"] * c["rows"], "flops": 3 * mn}
    n = int(_lens(c)[0].sum())
    kv = n * c["hkv"] * c["dim"]
    return {"bytes": (n * c["hq"] * c["dim"] + 2 * kv) * (SIZE[c["x"]] + 2) + 4 * n * c["hkv"] * (c["dim"] + 4)
            + 4 * c["axes"] * n, "flops": 3 * n * c["hq"] * c["dim"] + 12 * kv}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_f8(c, s):
    m, k, n = c["m"], c["k"], c["n"]
    # the 8-bit numbers in order; between neighbours the even code takes the tie
    code = torch.arange(0, 127, dtype=torch.uint8, device=DEV)
    val = code.view(torch.float8_e4m3fn).double()
    mid = (val[1:] + val[:-1]) / 2
    x = s["x"].double()
    xq = torch.zeros_like(x)
    for lo in range(0, k, 128):
        part = x[:, lo:lo + 128]
        top = part.abs().amax(1, keepdim=True)
        step = (top.float() * np.float32(1 / 448.0).item()).double()  # the scale as it is held
        r = torch.where(step > 0, part.abs() / step, 0.0)
        i = torch.bucketize(r, mid, right=False)  # the number of midpoints below r
        tie = (i < 126) & (r == mid[i.clamp_max(125)])
        i = torch.where(tie & (i % 2 == 1), i + 1, i)
        xq[:, lo:lo + 128] = val[i] * part.sign() * step
    w = s["wf"].view(torch.float8_e4m3fn).double()
    for lo in range(0, k, 128):
        w[:, lo:lo + 128] *= s["sw"][:, lo // 128].double().repeat_interleave(128)[:n, None]
    return xq @ w.t()


def _exact_verify(c, s):
    tok, _ = _lens(c)
    keep, out, count = [], [], []
    ids, u, temp = s["ids"].tolist(), s["u"].tolist(), s["temp"].tolist()
    first = 0
    for b in range(c["seqs"]):
        n = int(tok[b])
        par = s["parent"][first:first + n]

        def p_of(i):
            x = s["logits"][first + i].double()
            if temp[b] == 0:
                p = torch.zeros_like(x)
                p[int(torch.nonzero(x == x.max())[0])] = 1
                return p
            return torch.softmax(x / temp[b], 0)

        kept, said, node, p = [0], [], 0, p_of(0)
        i = 1
        while i < n:
            if par[i] == node:
                x = ids[first + i]
                q = s["q"][first + node].double() if s["q"] is not None else None
                got = float(p[x])
                lim = u[first + i] if q is None else u[first + i] * float(q[x])
                if (got > 0) if temp[b] == 0 else lim < got:
                    kept.append(i)
                    said.append(x)
                    node, p = i, p_of(i)
                elif temp[b] != 0:  # what is left of the target, as a distribution again
                    if q is None:
                        p[x] = 0
                    else:
                        p = (p - q).clamp_min(0)
                    p = p / p.sum()
            i += 1
        c_sum = torch.cumsum(p, 0)
        above = torch.nonzero(c_sum > u[first] * float(c_sum[-1]))
        said.append(int(above[0]))
        count.append(len(kept))
        keep += kept + [-1] * (n - len(kept))
        out += said + [-1] * (n - len(said))
        first += n
    return [_i32(keep), _i32(out), _i32(count)]


def _exact_plan(c, s):
    """Request by request, page by page."""
    page, tokens = c["page"], s["tokens"]
    lens, held, table, stack, top = (s[k].cpu().numpy().copy() for k in ("lens", "held", "table", "stack", "top"))
    top = int(top[0])
    for add in ([s["out"], s["add"]] if c["swap"] else [s["add"]]):
        add = add.cpu().numpy()
        for b in reversed(range(c["seqs"])):
            if add[b] < 0:
                for j in reversed(range(held[b])):
                    stack[top] = table[b, j]
                    top += 1
                held[b] = lens[b] = 0
        asked_pages = asked_tokens = 0
        free = top
        cu, pos, slot, seq = [0], [], [], []
        for b in range(c["seqs"]):
            n = max(int(add[b]), 0)
            want = -(-(int(lens[b]) + n) // page)
            need = max(want - int(held[b]), 0) if n else 0
            ok = want <= table.shape[1]
            if ok:
                asked_pages += need
                asked_tokens += n
                ok = (need == 0 or asked_pages <= free) and asked_tokens <= tokens
            if ok:
                for _ in range(need):
                    top -= 1
                    table[b, held[b]] = stack[top]
                    held[b] += 1
                for i in range(n):
                    x = int(lens[b]) + i
                    pos.append(x)
                    slot.append(int(table[b, x // page]) * page + x % page)
                    seq.append(b)
            cu.append(len(pos))
        rest = tokens - len(pos)
        pos, slot, seq = pos + [0] * rest, slot + [-1] * rest, seq + [-1] * rest
    return [_i32(cu), _i32(pos), torch.tensor(slot, dtype=torch.int64, device=DEV), _i32(seq), _i32(lens), _i32(held),
            _i32(table), _i32(stack), _i32([top])]


def _exact_axes(c, s):
    def turn(x):  # as complex numbers
        x, h = x.double(), s["freqs"].numel()
        out = x.clone()
        for i, a in enumerate(_axis_of(c)):
            z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["pos"][a].double() * s["freqs"][i])
            lo, hi = (2 * i, 2 * i + 1) if c["inter"] else (i, i + h)
            w = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * z[:, None]
            out[..., lo], out[..., hi] = w.real, w.imag
        return out

    if c["op"] == "axes":
        return turn(s["x"])

    def held(x):
        step = x.abs().max(-1, keepdim=True).values / 127.0
        r = x / step.clamp_min(1e-300)
        return r.sign() * (r.abs() + 0.5).floor().clamp_max(127.0) * step

    return [turn(s["Q"]), held(turn(s["K"])), held(s["V"].double())]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify" and case["seqs"] * case["tok"] * case["vocab"] > 120_000_000:
        return None
    if case["op"] in ("axes", "axes_write"):
        return _exact_axes(case, s)
    return {"f8": _exact_f8, "verify": _exact_verify, "plan": _exact_plan}[case["op"]](case, s)
