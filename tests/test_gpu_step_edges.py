"""A serving step's operators where one input makes another's error large: rows
without a distribution, sums that cancel, numbers at the ends of their types, idle
rows; and calls launched dependently behind what they read."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import guards  # noqa: E402
import step_ref as sref  # noqa: E402
from test_gpu_step import (_no_error_left, dev, drafts, make_pool, np_, run_verify, same, tree_words,  # noqa: E402,F401
                           w4)

pytestmark = pytest.mark.gpu

F32, F16, I32, I64 = np.float32, np.float16, np.int32, np.int64
NEG = F32(-np.inf)
ALMOST_ONE = F32(1 - 2.0 ** -24)


def words(*parents):
    """Masks of a tree by its tokens' parents."""
    w = []
    for i, p in enumerate(parents):
        w.append((w[p] if p >= 0 else 0) | 1 << i)
    return np.array(w, np.uint64).view(I64)


# -- verification of drafts ------------------------------------------------------------

def test_no_child_of_a_row_with_a_nan_is_taken(w4):  # noqa: F811
    """With draft probabilities and several children: a row with a NaN among ordinary logits has
    no distribution for the second and third child either."""
    rng = np.random.default_rng(31)
    seqs, v = 12, 3000
    logits = (2 * rng.standard_normal((5 * seqs, v))).astype(F32)
    q = np.exp(rng.standard_normal((5 * seqs, v)))
    q = (q / q.sum(1, keepdims=True)).astype(F32)
    ids = np.zeros(5 * seqs, I32)
    u = np.full(5 * seqs, 1e-6, F32)
    for b in range(seqs):
        # the tokens that have most left after a refusal; one child's own child behind them
        ids[5 * b + 1:5 * b + 5] = np.argsort(sref.distribution(logits[5 * b], 1.0) - q[5 * b])[-4:]
        if b % 3 < 2:
            logits[5 * b, rng.integers(0, v)] = np.nan
    mask = np.tile(words(-1, 0, 0, 0, 2), seqs)
    cu = np.arange(0, 5 * seqs + 1, 5, dtype=I32)
    got = run_verify(w4, logits, cu, ids, u, mask, q)
    same(got, sref.verify(logits, cu, ids, u, mask, q))
    bad = np.arange(seqs) % 3 < 2
    assert np.all(got[2][bad] == 1) and np.all(got[1][::5][bad] == -1) and np.all(got[2][~bad] > 1)


def test_weights_of_a_draw_are_within_four_units(w4):  # noqa: F811
    """The first token has the largest weight, 2^40 units; four others are chosen to weigh as much together,
    18 units more or less, to a unit.  With each of them within 4 units of its exact weight, half the sum passes the
    first token or not as the exact sums say."""
    rng = np.random.default_rng(32)
    n, one = 6000, 2.0 ** 40
    temp = rng.uniform(0.3, 3, n).astype(F32)
    t = temp.astype(np.float64)
    top = np.where(rng.random(n) < 0.5, 0, rng.uniform(-20, 20, n)).astype(F32)
    logits = np.zeros((n, 5), F32)
    logits[:, 0] = top
    side = np.where(rng.random(n) < 0.5, 18.0, -18.0)
    left = one + side

    def weight(l):
        return np.exp((l.astype(np.float64) - top.astype(np.float64)) / t) * one

    for k in (1, 2, 3, 4):
        want = left * rng.uniform(0.2, 0.8, n) if k == 1 else left
        l = (top + t * np.log(np.maximum(want, 0.4) / one)).astype(F32)
        for _ in range(4):  # from below
            l = np.where(weight(l) > want, np.nextafter(l, NEG), l)
        logits[:, k] = l
        left = left - weight(l)
    assert np.all(np.abs(left) < 1)
    got = run_verify(w4, logits, np.arange(n + 1, dtype=I32), np.zeros(n, I32), np.full(n, 0.5, F32), None, None, temp)
    assert np.all(got[2] == 1)
    wrong = (got[1] == 0) != (side < 0)
    assert not wrong.any(), "%d of %d" % (wrong.sum(), n)


def test_what_a_refusal_takes_off_is_rounded_once(w4):  # noqa: F811
    """A refused draft whose probabilities leave k 2^-24 of a weight of 2^40 units (the row's largest), and two tokens
    that weigh as much as what is left, 24 units more or less.  Each of the two weights may be 4 units off, hence the
    row's sum 8, and what is taken off half a unit more: less than 17 in all."""
    rng = np.random.default_rng(33)
    n, one = 3000, 2.0 ** 40
    k = rng.integers(1, 1 << rng.integers(2, 20, n))
    q0 = 1 - k * 2.0 ** -24
    side = np.where(rng.random(n) < 0.5, 24.0, -24.0)
    logits, q = np.full((2 * n, 4), NEG, F32), np.zeros((2 * n, 4), F32)
    logits[::2, 0], logits[1::2] = 0, 0
    q[::2, 0], q[::2, 1] = q0, k * 2.0 ** -25
    assert np.all(q[::2, 0].astype(np.float64) == q0)
    # rest = 2^40 - q0 (2^40 + rest) + side
    rest = left = (k * 2.0 ** 16 + side) / (1 + q0)
    for c in (2, 3):
        l = np.log(np.maximum(left, 1) / one).astype(F32)
        for _ in range(4):
            l = np.where(np.exp(l.astype(np.float64)) * one > left, np.nextafter(l, NEG), l)
        logits[::2, c] = np.where(left > 1, l, NEG)
        left = left - np.exp(logits[::2, c].astype(np.float64)) * one
    assert np.all(np.abs(left) < 4) and np.all(rest > 2.0 ** 14)
    ids = np.ones(2 * n, I32)  # a token without weight: refused
    u = np.full(2 * n, 0.5, F32)
    got = run_verify(w4, logits, np.arange(0, 2 * n + 1, 2, dtype=I32), ids, u, None, q)
    assert np.all(got[2] == 1)
    wrong = (got[1][::2] == 0) != (side < 0)
    assert not wrong.any(), "%d of %d" % (wrong.sum(), n)


def test_tests_after_refusals_that_leave_next_to_nothing(w4):  # noqa: F811
    """Sixteen refused tokens hold all but 2^-25 of the weight; what is left lies in six tokens, in shares of
    1/40.  The random numbers are odd multiples of 1/128, so that u times a sum of at most 40 shares
    is 2^-13 of it at least from a whole number of shares; the weights' roundings (half a unit of 2^-40 each,
    a share is 2^13.7 units) are a twentieth of that.  Drafts without weight are never taken."""
    rng = np.random.default_rng(34)
    seqs, v, big = 48, 900, 16
    shares = np.array([13, 11, 7, 5, 3, 1])
    par = [-1] + [0] * (big + 6)
    n = len(par)
    logits = np.full((n * seqs, v), NEG, F32)
    ids, u = np.zeros(n * seqs, I32), np.full(n * seqs, ALMOST_ONE, F32)
    for b in range(seqs):
        place = rng.permutation(v)
        row = logits[n * b]
        row[place[:big]] = 0
        row[place[big:big + 6]] = np.log(shares / 40 * 2.0 ** -21)
        logits[n * b + 1:n * (b + 1)] = rng.standard_normal((n - 1, v))
        ids[n * b + 1:n * b + 1 + big] = place[:big]
        tail = list(rng.permutation(place[big:big + 6])[:4]) + [place[700], -1]  # one without weight, one outside
        ids[n * b + 1 + big:n * (b + 1)] = rng.permutation(tail)
        u[n * b + 1 + big:n * (b + 1)] = (2 * rng.integers(0, 64, 6) + 1) / 128
        u[n * b] = (2 * rng.integers(0, 64) + 1) / 128
    mask = np.tile(words(*par), seqs)
    cu = np.arange(0, n * seqs + 1, n, dtype=I32)
    got, want = run_verify(w4, logits, cu, ids, u, mask), sref.verify(logits, cu, ids, u, mask)
    same(got[2:], want[2:], "count")
    same(got, want)
    assert 4 < (want[2] == 1).sum() < seqs - 4


def test_draws_with_probabilities_that_sum_to_a_million(w4):  # noqa: F811
    """Draft probabilities need not sum to 1: the bound on the fp32 sums grows with them, past 64 bits, and leaves the
    draw to the integers.  Half of 2^22 tokens are left, in two runs of 2^20 equal weights each; the random numbers
    put the target 2^-10 to 2^-7 of a token from the next one.  A weight is off by at most 4 units of 2^-40, 2^20 of them by
    2^-18 of a token; the fp32 weights of the second run, each off by the same up to 2^-22, by up to a quarter."""
    seqs, v = 48, 2 ** 22
    rng = np.random.default_rng(35)
    low = -rng.random(seqs).astype(F32)
    w = np.exp(low.astype(np.float64))
    total = (v // 4) * (1 + w)
    u = np.full(2 * seqs, 0.99, F32)
    for b in range(seqs):
        cand = (rng.random(20000) * 0.3 + 0.2).astype(F32)  # targets in the first run
        at = cand.astype(np.float64) * total[b]
        edge = np.abs(at - np.round(at))
        u[2 * b] = cand[np.flatnonzero((edge > 2.0 ** -10) & (edge < 2.0 ** -7))[0]]
    assert np.all(u[::2].astype(np.float64) * total < v // 4 - 1)
    want = 2 * np.floor(u[::2].astype(np.float64) * total).astype(I64)  # the even tokens are left
    logits = torch.zeros((2 * seqs, v), device="cuda")
    logits[::2, v // 2:] = dev(low)[:, None]
    q = torch.zeros((2 * seqs, v), dtype=torch.float16, device="cuda")
    q[:, 1::2] = 1
    ids = torch.ones(2 * seqs, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, 2 * seqs + 1, 2, dtype=torch.int32, device="cuda")
    keep, out, count = w4.draft_verify(logits, cu, ids, dev(u), q=q)
    assert bool((count == 1).all())
    got = np_(out)[::2]
    assert np.array_equal(got, want), "%d of %d" % ((got != want).sum(), seqs)


# -- the plan of a step ----------------------------------------------------------------

def plan_with_trees(host, add, tokens, mask, grow):
    """sref.Pool.plan with the mask laid out as `add` asks; a row whose words lie past the mask waits."""
    asked = np.maximum(np.asarray(add, np.int64), 0)
    at = np.cumsum(asked) - asked
    cu, pos, slot, seq = host.plan(np.where(at + asked > tokens, np.minimum(add, 0), add), tokens, grow)
    n = cu[-1]
    s = seq[:n]
    word = mask.view(np.uint64)[at[s] + np.arange(n) - cu[s]]
    pos[:n] = host.lens[s] + np.array([bin(int(x)).count("1") for x in word], np.int64) - 1
    return cu, pos, slot, seq


@pytest.mark.parametrize("seqs,width", [(40, 4), (1000, 3), (1500, 4), (9000, 3), (6000, 40)])
def test_kvq_plan_reads_trees_where_they_were_asked(w4, seqs, width):  # noqa: F811
    """Rows that wait, for pages or for good, between rows that go in: each row's positions come from its own tree,
    whose words the caller laid out before it could know."""
    rng = np.random.default_rng(seqs + width)
    page = 16
    lens = rng.integers(0, width * page // 2, seqs)
    pages = int((-(-lens // page)).sum()) + seqs // 40
    host = make_pool(rng, seqs, width, pages, page, lens)
    pool = w4.KVQPool(*(dev(np.asarray(a).astype(I32)) for a in (host.table, host.held, host.stack, [host.top])))
    dl = dev(lens.astype(I32))
    add = rng.integers(0, 5, seqs)
    add[rng.random(seqs) < 0.2] = 0
    if width <= 4:
        add[rng.random(seqs) < 0.05] = -1
    add[rng.random(seqs) < 0.05] = 64  # too long for a narrow table
    grow = rng.integers(0, 2, seqs)
    trees = [tree_words(int(a), rng) for a in add if a > 0]
    asked = int(np.maximum(add, 0).sum())
    waits = 0
    for tokens in (asked + 3, asked - asked // 3):
        mask = np.concatenate(trees + [np.zeros(3, I64)])[:tokens]
        outs = [guards.out((seqs + 1,), torch.int32), guards.out((tokens,), torch.int32), guards.out((tokens,), torch.int64),
                guards.out((tokens,), torch.int32)]
        ws = guards.out((w4.kvq_plan_workspace_bytes(pool, page),), torch.uint8)
        w4.kvq_plan(pool, page, dl, dev(add.astype(I32)), tokens, grow=dev(grow.astype(I32)), mask=dev(mask), cu=outs[0].t,
                    pos=outs[1].t, slot=outs[2].t, seq=outs[3].t, ws=ws.t)
        guards.check_all(*outs, ws)
        want = plan_with_trees(host, add, tokens, mask, grow)
        for o, x, name in zip(outs, want, ("cu", "pos", "slot", "seq")):
            assert np.array_equal(np_(o.t), x), name
        assert np.array_equal(np_(dl), host.lens) and int(pool.top[0]) == host.top
        inside = np.diff(want[0]) > 0
        waits += int((~inside & (add > 0))[:np.flatnonzero(inside)[-1]].sum())
    assert waits >= 2


def test_tokens_behind_a_batch_with_a_waiting_row_are_no_error(w4):  # noqa: F811
    """A step planned for more tokens than went in: the cache's write and read leave the others out, and the error
    word stays 0; offsets that are not in order, or negative, set it as ever."""
    g = torch.Generator(device="cuda").manual_seed(37)
    page, heads, dim, n = 16, 2, 64, 40
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = w4.kvq_pool(3, 2, 2)
    lens = torch.zeros(3, **i32)
    batch, pos, slot, seq = w4.kvq_plan(pool, page, lens, torch.tensor([10, 20, 5], **i32), n)
    assert batch.cu.tolist() == [0, 10, 10, 10]
    cache = w4.kvq_cache(2, page, heads, dim, 8)
    cache.ks.fill_(-3)
    q, k, v = (torch.randn((n, h, dim), device="cuda", generator=g) for h in (4, heads, heads))
    f = torch.ones(dim // 2, dtype=torch.float64, device="cuda")
    qr = w4.kvq_write(cache, batch, k, v, Q=q, pos=pos, freqs=f)
    out = torch.full((n, heads, dim), 7.0, device="cuda")
    w4.kvq_read(cache, batch, n, K=out, V=torch.empty_like(out))
    w4.kvq_attention(qr, cache, batch)
    w4.kvq_keep(cache, batch, torch.zeros(n, **i32))
    assert w4.w4a8_device_error() == 0
    turned = w4.rope_rotate(k, pos, f)
    assert float((out[:10] - turned[:10]).abs().max()) <= float(turned[:10].abs().max()) / 127 * 0.51
    assert bool((out[10:] == 7).all()) and bool((cache.ks[1, :, :10] >= 0).all())
    assert bool((cache.ks[0] == -3).all()) and bool((cache.ks[1, :, 10:] == -3).all())
    for cu in ([2, 10, 10, 10], [0, 10, 5, 40], [0, -1, -1, -1], [0, 10, 10, -5]):
        w4.kvq_write(cache, w4.KVQBatch(torch.tensor(cu, **i32), lens, pool.table), k, v)
        assert w4.w4a8_device_error() == 8, cu


def graph_us(call, reps=5):
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    times = []
    for _ in range(reps):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(1000 * a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("seqs,tokens", [(1000, 8), (8000, 8), (65536, 8), (65536, 20000)])
def test_kvq_plan_does_not_walk_over_idle_rows(w4, seqs, tokens):  # noqa: F811
    """Two tokens in seats far apart: the step of two neighbours, and about its time (a walk over 65534 idle
    rows takes a hundred times as long)."""
    us = []
    for second in (1, seqs // 2, seqs - 1):
        pool = w4.kvq_pool(seqs, 1, 16)
        lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        add = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        add[0] = 1
        add[second] = 2
        batch, pos, slot, seq = w4.kvq_plan(pool, 16, lens, add, tokens)
        assert seq[:4].tolist() == [0, second, second, -1] and slot[:4].tolist() == [15 * 16, 14 * 16, 14 * 16 + 1, -1]
        assert pos[:4].tolist() == [0, 0, 1, 0] and batch.cu[second:second + 2].tolist() == [1, 3]
        us.append(graph_us(lambda: w4.kvq_plan(pool, 16, lens, add, tokens)))
    assert max(us) < 4 * us[0] + 20, us


# -- the linear with e4m3 blocks -------------------------------------------------------

def test_f8_quotients_next_to_ties_of_the_smallest_scales(w4):  # noqa: F811
    """Subnormal scales of many bits, and values whose quotient rounds to a tie between two codes without being one: what is
    left over is less than the smallest number, and still tells the side."""
    rng = np.random.default_rng(36)
    ties = np.concatenate([(2 * np.arange(8) + 1) / 1024, *[(2 * np.arange(8, 16) + 1) * 2.0 ** (e - 4) for e in range(-6, 5)]])
    rows = []
    while len(rows) < 400:
        k = int(rng.integers(1 << 21, (1 << 23) - 1))
        top = F32(448 * k * 2.0 ** -149)
        k = int(np.float64(sref.f8_scale(np.array([top]))[0]) * 2.0 ** 149)
        x = np.round(ties * k)
        near = (x != ties * k) & ((x / k).astype(F32) == ties.astype(F32))
        if near.sum() < 4:
            continue
        row = np.zeros(128, F32)
        row[0] = top
        row[1:1 + near.sum()] = (x[near] * 2.0 ** -149 * rng.choice([-1, 1], near.sum())).astype(F32)
        rows.append(row)
    x = np.array(rows)
    xf, sa = w4.f8_quantize_rows(dev(x))
    codes, scales = sref.f8_rows(x)
    assert np.array_equal(np_(sa), scales) and np.all(scales < 2.0 ** -126)
    assert np.array_equal(sref.E4M3[np_(xf)], sref.E4M3[codes])


# -- calls launched dependently behind what they read ------------------------------------

@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("with_q", [False, True])
def test_a_step_of_dependent_launches(w4, captured, with_q):  # noqa: F811
    """A step in which each call reads what the one before writes, every launch dependent: the bits of the same step
    launched one after the other, step by step, buffers spoiled in between."""
    hidden, heads, dim, v, page = 512, 4, 64, 32000, 16
    seqs, n = 6, 48
    g = torch.Generator(device="cuda").manual_seed(38)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    wk, wl = (w4.f8_quantize_weights(rand(m, hidden) * 0.1) for m in (heads * dim, v))
    gamma, freqs = torch.ones(hidden, device="cuda"), torch.rand(dim // 2, dtype=torch.float64, device="cuda", generator=g)
    axis = w4.rope_axes((8, 12, 12))
    mask = dev(np.tile(words(-1, 0, 0, 1, 1, 2, 0, 3), seqs))
    steps = [(rand(n, hidden) * 2, torch.randint(0, v, (n,), device="cuda", generator=g, dtype=torch.int32),
              torch.rand(n, device="cuda", generator=g) * 1e-3, torch.randint(0, 500, (3, n), device="cuda", generator=g,
                                                                              dtype=torch.int32)) for _ in range(8)]
    q = torch.softmax(rand(n, v), 1) if with_q else None
    add = torch.full((seqs,), 8, **i32)

    class State:
        def __init__(self):
            self.r, self.ids, self.u, self.pos = (torch.empty_like(t) for t in steps[0])
            self.pool, self.cache = w4.kvq_pool(seqs, 4, 24), w4.kvq_cache(24, page, heads, dim, 8)
            self.lens, self.count = torch.zeros(seqs, **i32), torch.zeros(seqs, **i32)
            self.cu, self.at, self.seq = torch.zeros(seqs + 1, **i32), torch.zeros(n, **i32), torch.zeros(n, **i32)
            self.slot = torch.zeros(n, dtype=torch.int64, device="cuda")
            self.x = torch.zeros((n, hidden), dtype=torch.float16, device="cuda")
            self.xf, self.sa = torch.zeros((n, hidden), dtype=torch.uint8, device="cuda"), torch.zeros((4, n), device="cuda")
            self.k, self.logits = torch.zeros((n, heads * dim), device="cuda"), torch.zeros((n, v), device="cuda")
            self.qr, self.kr = (torch.zeros((n, heads, dim), dtype=t, device="cuda") for t in (torch.float16, torch.float32))
            self.keep, self.out = torch.zeros(n, **i32), torch.zeros(n, **i32)

        def spoil(self):
            for t in (self.x, self.sa, self.k, self.logits, self.qr, self.kr):
                t.fill_(float("nan"))
            for t in (self.xf, self.cu, self.at, self.seq, self.slot, self.keep, self.out):
                t.fill_(3)

        def run(self, flags):
            f = dict(flags=flags)
            batch, *_ = w4.kvq_plan(self.pool, page, self.lens, add, n, grow=self.count, mask=mask, cu=self.cu, pos=self.at,
                                    slot=self.slot, seq=self.seq, **f)
            w4.add_norm(self.r, gamma, X=self.x, **f)
            w4.f8_quantize_rows(self.x, Xf=self.xf, sa=self.sa, **f)
            w4.f8_gemm(self.xf, self.sa, *wk, Y=self.k, **f)
            k = self.k.view(n, heads, dim)
            w4.rope_rotate(k, self.pos, freqs, Y=self.kr, axis=axis, **f)
            w4.kvq_write(self.cache, batch, self.kr, k, Q=k, pos=self.pos, freqs=freqs, axis=axis, Q_out=self.qr, **f)
            w4.f8_linear(self.x, *wl, Y=self.logits, **f)
            w4.draft_verify(self.logits, self.cu, self.ids, self.u, mask=mask, q=q, keep=self.keep, out=self.out,
                            count=self.count, **f)
            w4.kvq_keep(self.cache, batch, self.keep, **f)

        def all(self):
            return [self.lens, self.count, self.cu, self.at, self.seq, self.slot, self.x, self.k, self.logits, self.qr, self.kr,
                    self.keep, self.out, *self.pool, *self.cache]

    want, got = State(), State()
    graph = None
    if captured:
        got.run(w4.LAUNCH_PDL)
        torch.cuda.synchronize()
        got = State()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.run(w4.LAUNCH_PDL)
    taken = 0
    for step in steps:
        for s in (want, got):
            s.spoil()
            for t, x in zip((s.r, s.ids, s.u, s.pos), step):
                t.copy_(x)
        want.run(0)
        if graph is None:
            got.run(w4.LAUNCH_PDL)
        else:
            graph.replay()
        for i, (a, b) in enumerate(zip(want.all(), got.all())):
            assert np.array_equal(np_(a), np_(b), equal_nan=a.dtype.is_floating_point), i
        taken += int(want.count.sum()) - seqs
    assert taken > 0 and w4.w4a8_device_error() == 0
