"""The decoder layer's operators on the GPU against plain 64-bit references
(layer_ref.py), within bounds counted from their roundings; what is held in
integers is bit-exact.  Outputs lie between guard bytes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import guards  # noqa: E402
import layer_ref as ref  # noqa: E402
import oracle  # noqa: E402

pytestmark = pytest.mark.gpu

F32, F16 = np.float32, np.float16
T = {F32: torch.float32, F16: torch.float16}


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_weight_quantized_w4a8_gb300 as m
    m.build()
    m.w4a8_set_tuning(reset=True)
    assert m.w4a8_device_error() == 0
    return m


@pytest.fixture(autouse=True)
def _no_error_left(w4):
    yield
    assert w4.w4a8_device_error() == 0


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def close(got, want, bound, what):
    got = got.cpu().numpy().astype(np.float64)
    off = np.abs(got - want) - bound
    bad = np.unravel_index(np.argmax(np.where(np.isnan(off), np.inf, off)), off.shape)
    assert np.all(off <= 0), "%s at %s: got %r, want %r, bound %.3g" % (what, bad, got[bad], want[bad], bound[bad])


# -- add_norm -------------------------------------------------------------------

@pytest.mark.parametrize("M,N", [(1, 3584), (64, 3584), (3, 1), (2, 7), (5, 1000), (1, 1001), (2, 8), (3, 8200),
                                 (2, 16392), (1, 32768), (1, 32767), (700, 264)])
@pytest.mark.parametrize("rt,yt,post,gate", [(F32, F32, False, None), (F16, F32, True, "vector"),
                                             (F32, F16, True, "rows"), (F16, F16, False, "vector"), (F16, None, False, None)])
def test_add_norm(w4, M, N, rt, yt, post, gate):
    rng = np.random.default_rng(M * 7 + N)
    r = (3 * rng.standard_normal((M, N))).astype(rt)
    y = None if yt is None else rng.standard_normal((M, N)).astype(yt)
    w = (1 + 0.1 * rng.standard_normal(N)).astype(F32)
    p = (1 + 0.1 * rng.standard_normal(N)).astype(F32) if post else None
    g = None if gate is None else rng.standard_normal(N if gate == "vector" else (M, N)).astype(F32)
    d = lambda a: None if a is None else dev(a)  # noqa: E731
    want_r, want_x, e_r, e_x = ref.add_norm(r, w, y, p, g, 1.25, -0.5, 1e-6)
    go, gx = guards.out((M, N), T[rt]), guards.out((M, N), torch.float16)
    codes = {}
    if N % 8 == 0:
        gq, gs = guards.out((M, N), torch.int8), guards.out((M,), torch.float32)
        codes = dict(Xq=gq.t, sa=gs.t)
    got = w4.add_norm(d(r), d(w), y=d(y), post_w=d(p), gate=d(g), alpha=1.25, beta=-0.5, r_out=go.t, X=gx.t, **codes)
    guards.check_all(go, gx)
    close(got[0], want_r, e_r + ref.out_round(want_r, rt), "r'")
    close(got[1], want_x, e_x + ref.out_round(want_x, F16), "x")
    if codes:
        guards.check_all(gq, gs)
        xq, sa = oracle.load().act_quantize(got[1].cpu().numpy())
        assert np.array_equal(got[2].cpu().numpy(), xq) and np.array_equal(got[3].cpu().numpy(), sa)


def test_add_norm_in_place_unaligned_and_partial(w4):
    rng = np.random.default_rng(5)
    M, N = 9, 512
    r, y = rng.standard_normal((M, N)).astype(F32), rng.standard_normal((M, N)).astype(F32)
    w = rng.standard_normal(N).astype(F32)
    plain = w4.add_norm(dev(r), dev(w), y=dev(y))
    rd = dev(r)
    out = w4.add_norm(rd, dev(w), y=dev(y), r_out=rd)  # r' over r
    assert out[0].data_ptr() == rd.data_ptr() and all(torch.equal(a, b) for a, b in zip(plain, out))
    # tensors on an element's alignment only: the scalar path, held to the same bounds
    buf = torch.empty(M * N + 1, device="cuda")
    odd = buf[1:].view(M, N)
    odd.copy_(dev(y))
    wr, wx, er, ex = ref.add_norm(r, w, y, None, None, 1.0, 1.0, 1e-6)
    got = w4.add_norm(dev(r), dev(w), y=odd)
    close(got[0], wr, er + ref.out_round(wr, F32), "r'")
    close(got[1], wx, ex + ref.out_round(wx, F16), "x")
    # without w: the residual alone
    r2, x2 = w4.add_norm(dev(r), y=dev(y))
    assert x2 is None and torch.equal(r2, plain[0])


def test_add_norm_zero_rows_and_codes(w4):
    """A zero row: eps keeps it finite, x = 0, scale 0 and all codes 0."""
    r = torch.zeros((2, 256), device="cuda")
    r[1] = 1.0
    w = torch.ones(256, device="cuda")
    _, x, xq, sa = w4.add_norm(r, w, codes=True)
    assert not x[0].any() and not xq[0].any() and sa[0] == 0 and bool((xq[1] == 127).all())
    # its codes feed the unfused linear as act_quantize_i8's do
    q2, s2 = w4.act_quantize_i8(x)
    assert torch.equal(xq, q2) and torch.equal(sa, s2)


# -- rotary positions -------------------------------------------------------------

@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 8), (128, 128), (128, 64), (128, 24), (256, 256), (256, 72)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("xt,yt", [(F32, F16), (F16, F16), (F16, F32), (F32, F32)])
def test_rope_rotate(w4, dim, rot, inter, xt, yt):
    rng = np.random.default_rng(dim + rot)
    n, h = 13, 5
    x = rng.standard_normal((n, h, dim)).astype(xt)
    pos = rng.integers(-100, 1_000_000, n).astype(np.int32)
    pos[:4] = [0, 1, 2 ** 31 - 1, -2 ** 31]
    freqs, ms = w4.rope_frequencies(rot, 1e4, "yarn", 4.0, old_ctx=4096)
    want, err = ref.rotate(x, pos, freqs.numpy(), inter, ms)
    g = guards.out((n, h, dim), T[yt])
    y = w4.rope_rotate(dev(x), dev(pos), freqs.cuda(), interleaved=inter, mscale=ms, Y=g.t)
    guards.check_all(g)
    close(y, want, err + ref.out_round(want, yt), "rotated")
    if rot < dim:  # what is past the rotated part is copied
        assert np.array_equal(y[..., rot:].cpu().numpy(), x[..., rot:].astype(yt))


@pytest.mark.parametrize("n,h", [(1, 1), (1, 28), (64, 33), (5000, 3)])
def test_rope_rotate_rows_and_in_place(w4, n, h):
    """Rows inside a wider projection, in place and out of place: the same bits."""
    rng = np.random.default_rng(n)
    wide = dev(rng.standard_normal((n, (h + 3) * 128)).astype(F32))
    part = wide[:, 128:(h + 1) * 128].view(n, h, 128)
    pos = dev(rng.integers(0, 40000, n).astype(np.int32))
    freqs = w4.rope_frequencies(128, 1e6)[0].cuda()
    before = wide.clone()
    want, err = ref.rotate(part.cpu().numpy(), pos.cpu().numpy(), freqs.cpu().numpy(), False)
    y = w4.rope_rotate(part, pos, freqs)
    close(y, want, err + ref.out_round(want, F32), "rotated")
    w4.rope_rotate(part, pos, freqs, Y=part)
    assert torch.equal(part, y)
    assert torch.equal(wide[:, :128], before[:, :128]) and torch.equal(wide[:, (h + 1) * 128:], before[:, (h + 1) * 128:])


# -- the cache --------------------------------------------------------------------

def make_cache(w4, pg, heads, dim, bits):
    """An empty cache between guard bytes."""
    width, dt = (dim, torch.int8) if bits == 8 else (dim // 2, torch.uint8)
    gs = [guards.out((pg.pages, heads, pg.page, width), dt) for _ in range(2)] + \
        [guards.out((pg.pages, heads, pg.page), torch.float32) for _ in range(2)]
    for g in gs:
        g.t.zero_()
    return w4.KVQCache(*(g.t for g in gs)), gs


def make_batch(w4, pg):
    return w4.KVQBatch(dev(pg.cu), dev(pg.start), dev(pg.table))


SHAPES = [((1,), (0,), 16), ((1, 0, 1, 1), (100, 5, 0, 63), 64), ((17, 64, 3), (40, 0, 130), 32), ((300,), (77,), 128),
          ((5,) * 40, tuple(range(40)), 256)]


@pytest.mark.parametrize("tok,ctx,page", SHAPES)
@pytest.mark.parametrize("dim,bits,heads,xt", [(128, 8, 4, F32), (64, 4, 3, F16), (256, 8, 1, F16), (128, 4, 2, F32),
                                               (64, 8, 9, F32), (256, 4, 2, F32)])
def test_write_without_positions_is_exact_and_reads_back(w4, tok, ctx, page, dim, bits, heads, xt):
    rng = np.random.default_rng(sum(tok) + dim)
    pg = ref.Paged(rng, tok, ctx, page)
    n = pg.tokens
    k, v = ((rng.standard_normal((n, heads, dim)) * np.exp(rng.standard_normal((n, heads, 1)))).astype(xt) for _ in range(2))
    k[0, 0] = 0                       # a zero vector: scale 0, codes 0
    v[0, -1, :2] = [300.0, -300.0]    # both ends of the range
    c, gs = make_cache(w4, pg, heads, dim, bits)
    b = make_batch(w4, pg)
    assert w4.kvq_write(c, b, dev(k), dev(v)) is None
    guards.check_all(*gs)
    p, o = pg.own()
    used = np.zeros((pg.pages, page), bool)
    used[p, o] = True
    for x, codes, scales in ((k, c.k, c.ks), (v, c.v, c.vs)):
        q, s = ref.quantize(x, bits)
        raw, sc = codes.cpu().numpy(), scales.cpu().numpy()
        assert np.array_equal(raw[p, :, o], ref.pack(q, bits))
        assert np.array_equal(sc[p, :, o], s)
        assert not raw.transpose(0, 2, 1, 3)[~used].any() and not sc.transpose(0, 2, 1)[~used].any()
    for yt in (F16, F32):
        gk, gv = guards.out((n, heads, dim), T[yt]), guards.out((n, heads, dim), T[yt])
        w4.kvq_read(c, b, n, K=gk.t, V=gv.t)
        guards.check_all(gk, gv)
        for x, g in ((k, gk), (v, gv)):
            q, s = ref.quantize(x, bits)
            assert np.array_equal(g.t.cpu().numpy(), (q.astype(F32) * s[..., None]).astype(yt))


@pytest.mark.parametrize("dim,rot,inter,bits,hq,heads,xt", [(128, 128, False, 8, 28, 4, F32), (128, 64, True, 8, 32, 2, F32),
                                                            (64, 16, False, 4, 5, 5, F16), (256, 256, True, 4, 8, 1, F32)])
@pytest.mark.parametrize("tok,ctx", [((1,), (2047,)), ((3, 0, 20), (5, 9, 0)), ((2000,), (1,))])
def test_write_with_positions(w4, dim, rot, inter, bits, hq, heads, xt, tok, ctx):
    rng = np.random.default_rng(dim + rot + sum(tok))
    pg = ref.Paged(rng, tok, ctx, 64)
    n = pg.tokens
    # one fused projection: q, k and v are slices of its rows
    wide = rng.standard_normal((n, (hq + 2 * heads) * dim)).astype(xt)
    cut = lambda t, a, m: t[:, a * dim:(a + m) * dim].reshape(n, m, dim)  # noqa: E731
    wd = dev(wide)
    q, k, v = cut(wd, 0, hq), cut(wd, hq, heads), cut(wd, hq + heads, heads)
    pos = rng.integers(0, 100000, n).astype(np.int32)
    freqs, ms = w4.rope_frequencies(rot, 1e6)
    c, gs = make_cache(w4, pg, heads, dim, bits)
    g = guards.out((n, hq, dim), torch.float16)
    out = w4.kvq_write(c, make_batch(w4, pg), k, v, Q=q, pos=dev(pos), freqs=freqs.cuda(), interleaved=inter, Q_out=g.t)
    guards.check_all(g, *gs)
    want, err = ref.rotate(cut(wide, 0, hq), pos, freqs.numpy(), inter)
    close(out, want, err + ref.out_round(want, F16), "queries")
    p, o = pg.own()
    codes, scale = ref.unpack(c.k.cpu().numpy()[p, :, o], bits), c.ks.cpu().numpy()[p, :, o]
    kw, ke = ref.rotate(cut(wide, hq, heads), pos, freqs.numpy(), inter)
    top = 127 if bits == 8 else 7
    amax, ae = np.abs(kw).max(-1), ke.max(-1)
    assert np.all(np.abs(scale - amax / top) <= ae / top + 2 * ref.U32 * amax / top)
    # each code stands for its value to half a step, as far as value and quotient are exact
    sc = scale.astype(np.float64)[..., None]
    assert np.all(np.abs(codes * sc - kw) <= sc * (0.5 + top * 4 * ref.U32) + ke + ae[..., None])
    assert np.array_equal(c.v.cpu().numpy()[p, :, o], ref.pack(ref.quantize(cut(wide, hq + heads, heads), bits)[0], bits))


@pytest.mark.parametrize("dim,bits,heads", [(128, 8, 4), (64, 4, 3), (256, 8, 2)])
def test_keep_moves_the_accepted_branch(w4, dim, bits, heads):
    rng = np.random.default_rng(dim)
    tok, ctx = (64, 0, 9, 1, 5), (30, 4, 0, 61, 200)
    pg = ref.Paged(rng, tok, ctx, 32)
    n = pg.tokens
    c, gs = make_cache(w4, pg, heads, dim, bits)
    b = make_batch(w4, pg)
    w4.kvq_write(c, b, dev(rng.standard_normal((n, heads, dim)).astype(F32)), dev(rng.standard_normal((n, heads, dim)).astype(F32)))
    keep = np.full(n, -1, np.int32)
    lists = {0: sorted(rng.choice(64, 20, replace=False)), 2: [8, 0, 3], 3: [0], 4: [0, 1, 2, 3, 4]}  # any order, all, one
    before = [t.cpu().numpy() for t in c]
    want = [t.copy() for t in before]
    for s, ids in lists.items():
        keep[pg.cu[s]:pg.cu[s] + len(ids)] = ids
        pf, of = pg.where(s, ctx[s] + np.array(ids))
        pt, ot = pg.where(s, ctx[s] + np.arange(len(ids)))
        for x, y in zip(want, before):
            x[pt, :, ot] = y[pf, :, of]
    w4.kvq_keep(c, b, dev(keep))
    guards.check_all(*gs)
    for x, t in zip(want, c):
        assert np.array_equal(t.cpu().numpy(), x)


# -- attention ----------------------------------------------------------------------

def fill(w4, rng, pg, heads, dim, bits, spread=0.3):
    """A cache whose used slots hold codes and scales as the quantizer leaves them."""
    top = 127 if bits == 8 else 7
    c, gs = make_cache(w4, pg, heads, dim, bits)
    host = []
    for codes, scales in ((c.k, c.ks), (c.v, c.vs)):
        q = np.clip(np.rint(rng.standard_normal((pg.pages, heads, pg.page, dim)) * top / 3), -top, top).astype(np.int8)
        s = (np.exp(spread * rng.standard_normal((pg.pages, heads, pg.page))) * 3 / top).astype(F32)
        codes.copy_(dev(ref.pack(q, bits)))
        scales.copy_(dev(s))
        host.append((q, s))
    return c, gs, host


def check_attention(w4, rng, pg, q, c, host, hq, heads, dim, mask, scale, got, skip=(), rows_off=()):
    got = got.cpu().numpy()
    G = hq // heads
    (kq, ks), (vq, vs) = host
    for b in range(len(pg.tok)):
        if b in skip or pg.tok[b] == 0:
            continue
        t = pg.tok[b]
        seen = ref.seen_of(pg, b, mask)
        p, o = pg.where(b, np.arange(pg.ctx[b] + t))
        lo = pg.cu[b]
        heads_done = range(heads) if pg.ctx[b] < 3000 else [0, heads - 1]
        for h in heads_done:
            rows = q[lo:lo + t, h * G:(h + 1) * G].reshape(t * G, dim)
            want, err = ref.attention(rows, kq[p, h, o], ks[p, h, o], vq[p, h, o], vs[p, h, o], np.repeat(seen, G, 0), scale)
            have = got[lo:lo + t, h * G:(h + 1) * G].reshape(t * G, dim).astype(np.float64)
            off = np.abs(have - want) - err
            off = np.where(np.isnan(off), np.inf, off)
            off[np.isin(lo + np.arange(t * G) // G, rows_off)] = 0
            i = np.unravel_index(np.argmax(off), off.shape)
            assert off[i] <= 0, "sequence %d head %d row %s: got %r, want %r, bound %.3g" % (b, h, i, have[i], want[i], err[i])


# A table this wide (slots times heads) leaves a call of 49 rows or more of a cache
# head to the kernel for many rows, whatever the lengths.
WIDE = 500_000


def wide_cols(seqs, heads, page):
    return -(-WIDE // (seqs * heads * page))


def run_attention(w4, rng, tok, ctx, page, hq, heads, dim, bits, tree, qstd=1.0, empty=(), spread=0.3, wide=False):
    pg = ref.Paged(rng, tok, ctx, page, extra_cols=wide_cols(len(tok), heads, page) if wide else 1)
    c, gs, host = fill(w4, rng, pg, heads, dim, bits, spread)
    q = (qstd * rng.standard_normal((pg.tokens, hq, dim))).astype(F16)
    mask = ref.tree_masks(rng, tok, empty) if tree else None
    g = guards.out((pg.tokens, hq, dim), torch.float16)
    b = make_batch(w4, pg)
    need = w4.kvq_attention_workspace_bytes(c, b, pg.tokens, hq)
    gw = guards.workspace(need)
    call = lambda: w4.kvq_attention(dev(q), c, b, mask=None if mask is None else dev(mask.view(np.int64)), out=g.t,  # noqa: E731
                                    ws=guards.t(gw))
    out = call()
    guards.check_all(g, gw, *gs)
    check_attention(w4, rng, pg, q, c, host, hq, heads, dim, mask, dim ** -0.5, out)
    first = out.clone()
    assert torch.equal(call(), first)  # the same bits again, on a workspace left ready
    return out


@pytest.mark.parametrize("dim,bits", [(128, 8), (128, 4), (64, 8), (64, 4), (256, 8), (256, 4)])
@pytest.mark.parametrize("hq,heads,page", [(28, 4, 64), (32, 2, 32), (3, 3, 16), (8, 1, 256)])
@pytest.mark.parametrize("tok,ctx,tree", [((1,), (0,), False), ((1,), (63,), False), ((1, 1, 0, 1), (64, 0, 7, 200), False),
                                          ((9, 2), (129, 0), True), ((33, 1), (31, 500), True)])
def test_attention(w4, dim, bits, hq, heads, page, tok, ctx, tree):
    rng = np.random.default_rng(dim + bits + hq + sum(tok) + sum(ctx))
    run_attention(w4, rng, tok, ctx, page, hq, heads, dim, bits, tree)


@pytest.mark.parametrize("dim,bits,hq,heads", [(128, 8, 28, 4), (128, 4, 32, 2), (64, 8, 6, 6), (256, 8, 4, 2)])
@pytest.mark.parametrize("tok,ctx,tree", [((64,), (1,), True), ((64, 64), (300, 1023), True), ((100,), (57,), False),
                                          ((1,) * 70, tuple(17 * i % 400 for i in range(70)), False), ((7,), (5000,), True),
                                          ((1, 3), (20000, 1), True)])
def test_attention_larger(w4, dim, bits, hq, heads, tok, ctx, tree):
    rng = np.random.default_rng(dim + bits + sum(tok) + sum(ctx))
    run_attention(w4, rng, tok, ctx, 64, hq, heads, dim, bits, tree)


@pytest.mark.parametrize("hq,heads", [(1, 1), (5, 5), (2, 1), (9, 1), (12, 1), (17, 1), (64, 1), (130, 1), (30, 6), (64, 8)])
def test_attention_head_groups(w4, hq, heads):
    run_attention(w4, np.random.default_rng(hq), (3, 1), (77, 260), 16, hq, heads, 128, 8, True)


@pytest.mark.parametrize("qstd,spread", [(0.0, 0.0), (30.0, 0.3), (1e-4, 2.0), (1000.0, 0.0)])
def test_attention_flat_and_peaked(w4, qstd, spread):
    """All logits equal; logits that leave one key; scales over a wide range."""
    run_attention(w4, np.random.default_rng(3), (4, 1), (500, 90), 32, 14, 2, 128, 8, True, qstd=qstd, spread=spread)


@pytest.mark.parametrize("dim,bits", [(128, 8), (128, 4), (64, 8), (64, 4)])
@pytest.mark.parametrize("hq,heads,page", [(28, 4, 64), (32, 2, 16), (64, 1, 256), (48, 3, 32)])
@pytest.mark.parametrize("tok,ctx,tree", [((8,), (0,), True), ((64,), (1,), True), ((17, 0, 20), (31, 9, 500), True),
                                          ((33, 1, 40), (300, 128, 127), False), ((64, 50), (2000, 1023), True),
                                          ((100,), (57,), False), ((9,), (9000,), True)])
def test_attention_many_rows(w4, dim, bits, hq, heads, page, tok, ctx, tree):
    """The kernel for many rows: one and two tiles a row block, whole and shared
    by CTAs, blocks of keys that end inside."""
    rng = np.random.default_rng(dim + bits + hq + sum(tok) + sum(ctx) + 1)
    run_attention(w4, rng, tok, ctx, page, hq, heads, dim, bits, tree, wide=True)


def test_attention_many_rows_routes(w4):
    """Wide and narrow tables take the two kernels (their workspaces tell them apart)."""
    rng = np.random.default_rng(0)
    need = []
    for cols in (1, wide_cols(1, 4, 64)):
        pg = ref.Paged(rng, (64,), (10,), 64, extra_cols=cols)
        c, _ = make_cache(w4, pg, 4, 128, 8)
        need.append(w4.kvq_attention_workspace_bytes(c, make_batch(w4, pg), 64, 28))
    assert need[0] < need[1]
    pg = ref.Paged(rng, (64,), (10,), 64, extra_cols=wide_cols(1, 4, 64))
    c, _ = make_cache(w4, pg, 4, 256, 8)  # 256 dimensions: row blocks always
    assert w4.kvq_attention_workspace_bytes(c, make_batch(w4, pg), 64, 28) < need[1]


@pytest.mark.parametrize("qstd,spread", [(0.0, 0.0), (30.0, 0.3), (1e-4, 2.0), (1000.0, 0.0), (3.0, 4.0)])
@pytest.mark.parametrize("tok", [(5, 9), (30, 20)])
def test_attention_many_rows_flat_and_peaked(w4, qstd, spread, tok):
    run_attention(w4, np.random.default_rng(4), tok, (900, 90), 32, 32, 2, 128, 8, True, qstd=qstd, spread=spread, wide=True)


def test_attention_many_rows_growing_logits(w4):
    """Keys whose logits rise along the sequence: every block raises the
    references and rescales what was summed before."""
    rng = np.random.default_rng(5)
    tok, ctx, hq, heads, dim = (6, 3), (1500, 700), 32, 2, 128
    pg = ref.Paged(rng, tok, ctx, 64, extra_cols=wide_cols(2, heads, 64))
    c, _, host = fill(w4, rng, pg, heads, dim, 8)
    (kq, ks), (vq, vs) = host
    for b in range(2):
        p, o = pg.where(b, np.arange(tok[b] + ctx[b]))
        ks[p, :, o] *= np.linspace(0.01, 12.0, len(p)).astype(F32)[:, None]
        vs[p, :, o] *= np.exp2(np.linspace(-12, 6, len(p))).astype(F32)[:, None]
    c.ks.copy_(dev(ks))
    c.vs.copy_(dev(vs))
    q = rng.standard_normal((9, hq, dim)).astype(F16)
    mask = ref.tree_masks(rng, tok)
    out = w4.kvq_attention(dev(q), c, make_batch(w4, pg), mask=dev(mask.view(np.int64)))
    check_attention(w4, rng, pg, q, c, host, hq, heads, dim, mask, dim ** -0.5, out)


def test_attention_many_rows_that_see_nothing(w4):
    rng = np.random.default_rng(6)
    out = run_attention(w4, rng, (6, 8), (0, 0), 16, 32, 2, 128, 8, True, empty=(2, 5, 6, 7, 8), wide=True)
    assert not out[[2, 5, 6, 7, 8]].any() and bool(out[0].any())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_attention_many_rows_bad_scales_in_masked_keys(w4, bits, bad, which):
    rng = np.random.default_rng(7)
    tok, ctx, hq, heads, dim = (5, 6), (170, 3), 32, 2, 128
    pg = ref.Paged(rng, tok, ctx, 16, extra_cols=wide_cols(2, heads, 16))
    c, _, host = fill(w4, rng, pg, heads, dim, bits)
    mask = ref.tree_masks(rng, tok)
    mask[:5] &= ~np.uint64(4)  # nobody but token 2 sees token 2
    mask[2] |= np.uint64(4)
    p, o = pg.where(0, [ctx[0] + 2])
    q = rng.standard_normal((pg.tokens, hq, dim)).astype(F16)
    if which != "v":
        c.ks[int(p[0]), :, int(o[0])] = bad
    if which != "k":
        c.vs[int(p[0]), :, int(o[0])] = bad
    out = w4.kvq_attention(dev(q), c, make_batch(w4, pg), mask=dev(mask.view(np.int64)))
    assert bool(torch.isfinite(out[[0, 1, 3, 4, 5, 6, 7, 8, 9, 10]]).all())
    assert not bool(torch.isfinite(out[2]).all())  # who sees it has it
    check_attention(w4, rng, pg, q, c, host, hq, heads, dim, mask, dim ** -0.5, out, rows_off=(2,))


def test_attention_many_rows_zero_scales(w4):
    """Zero values weigh and add nothing; zero keys (scale 0) have logit 0."""
    rng = np.random.default_rng(8)
    tok, heads = (4, 5), 2
    pg = ref.Paged(rng, tok, (150, 0), 32, extra_cols=wide_cols(2, heads, 32))
    c, _, host = fill(w4, rng, pg, heads, 128, 8)
    q = rng.standard_normal((9, 32, 128)).astype(F16)
    host[0][1][:, :, 1::4] = 0
    host[0][0][:, :, 1::4] = 0
    c.ks[:, :, 1::4] = 0
    c.k[:, :, 1::4] = 0
    for zero in (slice(None, None, 3), slice(None)):
        host[1][1][:, :, zero] = 0
        c.vs[:, :, zero] = 0
        out = w4.kvq_attention(dev(q), c, make_batch(w4, pg))
        check_attention(w4, rng, pg, q, c, host, 32, heads, 128, None, 128 ** -0.5, out)
    assert not out.any()


def test_attention_scale_signs(w4):
    """A negative, a zero and a large factor of the logits, both kernels."""
    rng = np.random.default_rng(9)
    for wide, hq in ((False, 8), (True, 64)):
        pg = ref.Paged(rng, (3, 2), (140, 5), 32, extra_cols=wide_cols(2, 2, 32) if wide else 1)
        c, _, host = fill(w4, rng, pg, 2, 128, 8)
        q = rng.standard_normal((5, hq, 128)).astype(F16)
        for scale in (-0.1, 0.0, 3.0):
            out = w4.kvq_attention(dev(q), c, make_batch(w4, pg), scale=scale)
            check_attention(w4, rng, pg, q, c, host, hq, 2, 128, None, scale, out)


def test_attention_many_rows_bad_pages_and_graph(w4):
    """A page out of range is seen by nobody and sets the error word; a captured
    call follows lengths changed between replays."""
    rng = np.random.default_rng(10)
    tok, ctx, hq, heads, dim = (6, 7), (300, 500), 32, 2, 128
    pg = ref.Paged(rng, tok, ctx, 32, extra_cols=wide_cols(2, heads, 32))
    c, _, host = fill(w4, rng, pg, heads, dim, 8)
    q = rng.standard_normal((13, hq, dim)).astype(F16)
    qd = dev(q)
    for entry in (-1, pg.pages, 2 ** 31 - 1, -2 ** 31):
        table = pg.table.copy()
        table[1, 3] = entry
        out = w4.kvq_attention(qd, c, w4.KVQBatch(dev(pg.cu), dev(pg.start), dev(table)))
        assert w4.w4a8_device_error() == 8
        assert bool(torch.isfinite(out).all())
        check_attention(w4, rng, pg, q, c, host, hq, heads, dim, None, dim ** -0.5, out, skip=(1,))
        # sequence 1 as if the page's slots were not there
        (kq, ks), (vq, vs) = host
        slots = np.array([j for j in range(507) if not 96 <= j < 128])
        p, o = pg.where(1, slots)
        seen = np.repeat(ref.seen_of(pg, 1, None)[:, slots], hq // heads, 0)
        for h in range(heads):
            rows = q[6:, h * 16:(h + 1) * 16].reshape(-1, dim)
            want, err = ref.attention(rows, kq[p, h, o], ks[p, h, o], vq[p, h, o], vs[p, h, o], seen, dim ** -0.5)
            got = out[6:, h * 16:(h + 1) * 16].cpu().numpy().reshape(-1, dim)
            assert np.all(np.abs(got - want) <= err)
    b = make_batch(w4, pg)
    w4.kvq_attention(qd, c, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w4.kvq_attention(qd, c, b)
    for new in ((300, 500), (2, 444), (0, 0), (127, 128)):
        b.start.copy_(dev(np.array(new, np.int32)))
        graph.replay()
        assert torch.equal(out, w4.kvq_attention(qd, c, b))
        pg.ctx, pg.start = list(new), np.array(new, np.int32)
        check_attention(w4, rng, pg, q, c, host, hq, heads, dim, None, dim ** -0.5, out)


def test_attention_rows_that_see_nothing(w4):
    """No cached token and an empty mask word: zeros; the other rows as ever."""
    rng = np.random.default_rng(9)
    out = run_attention(w4, rng, (6, 3), (0, 0), 16, 8, 2, 128, 8, True, empty=(2, 5, 6, 7, 8))
    assert not out[[2, 5, 6, 7, 8]].any() and bool(out[0].any())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_bad_scales_in_masked_keys(w4, bits, bad):
    """A drafted key whose scales are not finite harms nobody that does not see it."""
    rng = np.random.default_rng(10)
    tok, ctx, hq, heads, dim = (5, 2), (70, 3), 14, 2, 128
    pg = ref.Paged(rng, tok, ctx, 16)
    c, _, host = fill(w4, rng, pg, heads, dim, bits)
    mask = ref.tree_masks(rng, tok)
    mask[:5] &= ~np.uint64(4)  # nobody but token 2 sees token 2
    mask[2] |= np.uint64(4)
    p, o = pg.where(0, [ctx[0] + 2])
    q = rng.standard_normal((pg.tokens, hq, dim)).astype(F16)
    md = dev(mask.view(np.int64))
    clean = w4.kvq_attention(dev(q), c, make_batch(w4, pg), mask=md)
    c.ks[int(p[0]), :, int(o[0])] = bad
    c.vs[int(p[0]), :, int(o[0])] = bad
    out = w4.kvq_attention(dev(q), c, make_batch(w4, pg), mask=md)
    rows = [0, 1, 3, 4, 5, 6]
    assert bool(torch.isfinite(out[rows]).all())
    check_attention(w4, rng, pg, q, c, host, hq, heads, dim, mask, dim ** -0.5, clean)
    check_attention(w4, rng, pg, q, c, host, hq, heads, dim, mask, dim ** -0.5, out, rows_off=(2,))


def test_attention_zero_value_scales(w4):
    """Zero value vectors (scale 0) weigh in the softmax and add nothing."""
    rng = np.random.default_rng(11)
    pg = ref.Paged(rng, (2, 1), (150, 0), 32)
    c, _, host = fill(w4, rng, pg, 2, 128, 8)
    for zero in (slice(None, None, 3), slice(None)):
        host[1][1][:, :, zero] = 0
        c.vs[:, :, zero] = 0
        q = rng.standard_normal((3, 6, 128)).astype(F16)
        out = w4.kvq_attention(dev(q), c, make_batch(w4, pg))
        check_attention(w4, rng, pg, q, c, host, 6, 2, 128, None, 128 ** -0.5, out)
    assert not out.any()


def test_attention_on_another_stream_and_in_a_graph(w4):
    """A side stream; a captured call that follows lengths and pages changed
    between replays, next to eager calls."""
    rng = np.random.default_rng(12)
    hq, heads, dim = 28, 4, 128
    pg = ref.Paged(rng, (1, 1), (900, 2000), 64)
    c, _, host = fill(w4, rng, pg, heads, dim, 8)
    b = make_batch(w4, pg)
    q = rng.standard_normal((2, hq, dim)).astype(F16)
    qd = dev(q)
    base = w4.kvq_attention(qd, c, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = w4.kvq_attention(qd, c, b)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, base)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w4.kvq_attention(qd, c, b)
    for ctx in ((900, 2000), (5, 1999), (0, 64), (899, 3)):
        b.start.copy_(dev(np.array(ctx, np.int32)))
        graph.replay()
        eager = w4.kvq_attention(qd, c, b)
        assert torch.equal(out, eager)
        pg.ctx, pg.start = list(ctx), np.array(ctx, np.int32)
        check_attention(w4, rng, pg, q, c, host, hq, heads, dim, None, dim ** -0.5, out)


def test_large_pool_offsets(w4):
    """Pages whose bytes lie past 2^31 and 2^32: written, read back, attended to."""
    page, heads, dim = 256, 4, 128
    pages = (1 << 32) // (page * heads * dim) + 40
    c = w4.kvq_cache(pages, page, heads, dim)
    table = torch.tensor([[pages - 1, 3, pages - 30, (1 << 31) // (page * heads * dim) + 1]], dtype=torch.int32).cuda()
    n = 1000
    b = w4.KVQBatch(torch.tensor([0, n], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda(), table)
    rng = np.random.default_rng(13)
    k, v = (rng.standard_normal((n, heads, dim)).astype(F32) for _ in range(2))
    w4.kvq_write(c, b, dev(k), dev(v))
    rk, rv = w4.kvq_read(c, b, n, dtype=torch.float32)
    for x, r in ((k, rk), (v, rv)):
        q, s = ref.quantize(x, 8)
        assert np.array_equal(r.cpu().numpy(), q.astype(F32) * s[..., None])
    one = w4.KVQBatch(torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([n - 1], dtype=torch.int32).cuda(), table)
    qh = rng.standard_normal((1, 8, dim)).astype(F16)
    out = w4.kvq_attention(dev(qh), c, one).cpu().numpy()
    for h in range(heads):
        (kc, ks), (vc, vs) = ref.quantize(k[:, h], 8), ref.quantize(v[:, h], 8)
        want, err = ref.attention(qh[0, 2 * h:2 * h + 2], kc, ks, vc, vs, np.ones((2, n), bool), dim ** -0.5)
        assert np.all(np.abs(out[0, 2 * h:2 * h + 2] - want) <= err)


def test_bad_pages_and_offsets_set_the_error_word(w4):
    """Slots and pages out of range: nothing outside the cache is touched, the
    rest of the batch is served, bit 3 of the error word is set.  (The look-ups
    themselves are tested on the host with the same tables.)"""
    rng = np.random.default_rng(14)
    heads, dim, hq = 2, 128, 8
    pg = ref.Paged(rng, (2, 2, 1), (60, 40, 20), 16)
    c, gs, host = fill(w4, rng, pg, heads, dim, 8)
    q = rng.standard_normal((5, hq, dim)).astype(F16)
    x = rng.standard_normal((5, heads, dim)).astype(F32)
    for entry in (-1, pg.pages, 2 ** 31 - 1, -2 ** 31):
        table = pg.table.copy()
        table[1, 2] = entry  # the page of sequence 1's own tokens (slots 40, 41) and of cached ones from 32
        b = w4.KVQBatch(dev(pg.cu), dev(pg.start), dev(table))
        out = w4.kvq_attention(dev(q), c, b)
        assert w4.w4a8_device_error() == 8
        check_attention(w4, rng, pg, q, c, host, hq, heads, dim, None, dim ** -0.5, out, skip=(1,))
        assert bool(torch.isfinite(out).all())  # sequence 1: its 32 slots in range
        before = [t.clone() for t in c]
        w4.kvq_write(c, b, dev(x), dev(x))
        assert w4.w4a8_device_error() == 8
        p, o = pg.own()
        assert np.array_equal(c.ks.cpu().numpy()[p, :, o][[0, 1, 4]], ref.quantize(x, 8)[1][[0, 1, 4]])
        p1, o1 = pg.where(1, [40, 41])  # the pages of the sound table: untouched
        for t, u in zip(c, before):
            assert torch.equal(t[dev(p1).long(), :, dev(o1).long()], u[dev(p1).long(), :, dev(o1).long()])
        k0 = torch.full((5, heads, dim), 7.0, device="cuda")
        kk, vv = w4.kvq_read(c, b, 5, dtype=torch.float32, K=k0, V=torch.full_like(k0, 7.0))
        assert w4.w4a8_device_error() == 8
        assert bool((kk[2:4] == 7).all()) and bool((kk[[0, 1, 4]] != 7).any())
        w4.kvq_keep(c, b, dev(np.array([1, -1, 1, -1, 0], np.int32)))
        assert w4.w4a8_device_error() == 8
        for t, u in zip(c, before):
            t.copy_(u)
    guards.check_all(*gs)
    for start in ([60, -3, 20], [60, 10 ** 9, 20]):  # before and past the table
        b = w4.KVQBatch(dev(pg.cu), dev(np.array(start, np.int32)), dev(pg.table))
        out = w4.kvq_attention(dev(q), c, b)
        assert w4.w4a8_device_error() == 8
        check_attention(w4, rng, pg, q, c, host, hq, heads, dim, None, dim ** -0.5, out, skip=(1,))
        w4.kvq_write(c, b, dev(x), dev(x))
        assert w4.w4a8_device_error() == 8
        w4.kvq_keep(c, b, dev(np.array([0, -1, 0, -1, 0], np.int32)))
        assert w4.w4a8_device_error() == 8
        for t, u in zip(c, before):
            t.copy_(u)
    # an entry past the tree, and a tree past 64 tokens under a mask
    w4.kvq_keep(c, make_batch(w4, pg), dev(np.array([2, -1, 0, -1, 0], np.int32)))
    assert w4.w4a8_device_error() == 8
    big = ref.Paged(rng, (65, 1), (3, 40), 16)
    c2, _, host2 = fill(w4, rng, big, heads, dim, 8)
    q2 = rng.standard_normal((66, hq, dim)).astype(F16)
    mask = np.full(66, 1, np.uint64)
    out = w4.kvq_attention(dev(q2), c2, make_batch(w4, big), mask=dev(mask.view(np.int64)))
    assert w4.w4a8_device_error() == 8
    assert not out[:65].any()
    check_attention(w4, rng, big, q2, c2, host2, hq, heads, dim, mask, dim ** -0.5, out, skip=(0,))
    guards.check_all(*gs)
