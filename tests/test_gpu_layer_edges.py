"""Values at the ends of what the decoder layer's cache and attention hold, on
the GPU, against the 64-bit references and bounds of layer_ref.py: scales
that are tiny, huge, negative, zero or not finite."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import guards  # noqa: E402
import layer_ref as ref  # noqa: E402
from test_gpu_layer import (check_attention, dev, fill, make_batch, make_cache, w4,  # noqa: E402,F401
                            wide_cols)

pytestmark = pytest.mark.gpu

F32, F16 = np.float32, np.float16


@pytest.fixture(autouse=True)
def _no_error_left(w4):  # noqa: F811
    yield
    assert w4.w4a8_device_error() == 0


# -- the write's codes -------------------------------------------------------------

# Largest values of vectors: binary32's subnormals, the scales' (1.2e-38 times 127 or
# 7, and a quarter of that, where 1 / scale is no longer finite), ordinary ones.
TINY = [1e-45, 3e-45, 9e-44, 1e-42, 1e-40, 1.17e-38, 2e-38, 2.1e-38, 8e-38, 9e-38, 3.7e-37, 3.8e-37, 1.4e-36, 1.5e-36, 1e-35]


@pytest.mark.parametrize("dim,bits", [(64, 8), (128, 8), (128, 4), (256, 4)])
def test_write_of_tiny_vectors_is_exact(w4, dim, bits):  # noqa: F811
    rng = np.random.default_rng(dim + bits)
    n, heads = len(TINY), 3
    x = [rng.uniform(-1, 1, (n, heads, dim)) for _ in range(2)]
    for t in x:
        t[:, 0, 0], t[:, 1, -1] = 1, -1
        t[:, :, 5:9] = 0                # zeros inside
        t *= np.array(TINY)[:, None, None]
    k, v = (t.astype(F32) for t in x)
    pg = ref.Paged(rng, (n,), (3,), 16)
    c, gs = make_cache(w4, pg, heads, dim, bits)
    w4.kvq_write(c, make_batch(w4, pg), dev(k), dev(v))
    guards.check_all(*gs)
    p, o = pg.own()
    for t, codes, scales in ((k, c.k, c.ks), (v, c.v, c.vs)):
        q, s = ref.quantize(t, bits)
        assert np.array_equal(scales.cpu().numpy()[p, :, o], s)
        assert np.array_equal(codes.cpu().numpy()[p, :, o], ref.pack(q, bits))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dim,bits,rot,inter", [(128, 8, 0, False), (64, 4, 0, False), (128, 8, 128, False), (128, 4, 64, True)])
def test_write_keeps_what_is_not_finite_in_the_scale(w4, bad, dim, bits, rot, inter):  # noqa: F811
    """A vector with a NaN or an infinity: a scale that is neither finite nor 0,
    codes 0, so that every value reads back NaN; its neighbours as ever."""
    rng = np.random.default_rng(dim + bits + rot)
    n, heads = 6, 2
    k, v = (rng.standard_normal((n, heads, dim)).astype(F32) for _ in range(2))
    clean = [t.copy() for t in (k, v)]
    k[1, 0, 3] = k[4, 1, dim - 1] = v[2, 1, 0] = v[5, 0, 40] = bad
    k[3, 0, 7], k[3, 0, 8] = float("nan"), bad   # with a NaN beside it: NaN
    pg = ref.Paged(rng, (n,), (10,), 16)
    pos = dev(rng.integers(0, 5000, n).astype(np.int32))
    freqs = w4.rope_frequencies(rot, 1e4)[0].cuda() if rot else None
    got = []
    for a, b in ((k, v), clean):
        c, gs = make_cache(w4, pg, heads, dim, bits)
        w4.kvq_write(c, make_batch(w4, pg), dev(a), dev(b), pos=pos if rot else None, freqs=freqs, interleaved=inter)
        guards.check_all(*gs)
        got.append(c)
    c, sound = got
    p, o = pg.own()
    at = lambda t: t.cpu().numpy()[p, :, o]  # noqa: E731
    kb, vb = np.zeros((n, heads), bool), np.zeros((n, heads), bool)
    kb[[1, 4, 3], [0, 1, 0]] = True
    vb[[2, 5], [1, 0]] = True
    for codes, scales, s_codes, s_scales, b in ((c.k, c.ks, sound.k, sound.ks, kb), (c.v, c.vs, sound.v, sound.vs, vb)):
        assert not np.isfinite(at(scales)[b]).any() and not at(codes)[b].any()
        assert np.array_equal(at(scales)[~b], at(s_scales)[~b]) and np.array_equal(at(codes)[~b], at(s_codes)[~b])
    assert np.isnan(at(c.ks)[3, 0])
    rk, rv = w4.kvq_read(c, make_batch(w4, pg), n, dtype=torch.float32)
    assert np.isnan(rk.cpu().numpy()[kb]).all() and np.isnan(rv.cpu().numpy()[vb]).all()
    assert torch.isfinite(rk[dev(~kb)]).all() and torch.isfinite(rv[dev(~vb)]).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("which", ["k", "v"])
def test_a_nan_that_is_written_reaches_the_rows_that_see_it(w4, wide, which):  # noqa: F811
    rng = np.random.default_rng(21)
    tok, ctx, hq, heads, dim = (5,), (150,), 32, 2, 128
    pg = ref.Paged(rng, tok, ctx, 32, extra_cols=wide_cols(1, heads, 32) if wide else 1)
    c, _, _ = fill(w4, rng, pg, heads, dim, 8)
    mask = np.array([1, 3, 4, 9, 17], np.uint64)  # token 2 is seen by itself alone
    x = {t: rng.standard_normal((5, heads, dim)).astype(F32) for t in "kv"}
    x[which][2, :, 11] = float("nan")
    q = rng.standard_normal((5, hq, dim)).astype(F16)
    b = make_batch(w4, pg)
    w4.kvq_write(c, b, dev(x["k"]), dev(x["v"]))
    out = w4.kvq_attention(dev(q), c, b, mask=dev(mask.view(np.int64)))
    assert bool(torch.isfinite(out[[0, 1, 3, 4]]).all()) and not bool(torch.isfinite(out[2]).any())


# -- attention ------------------------------------------------------------------------

@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("big", [1e6, -1e6, 1e30, -1e30])
@pytest.mark.parametrize("tok,ctx", [((5, 6), (170, 3)), ((40, 9), (900, 90))])
def test_attention_large_values_in_masked_keys(w4, wide, bits, big, tok, ctx):  # noqa: F811
    """A drafted token with a large value vector changes only the rows that see it."""
    rng = np.random.default_rng(22)
    hq, heads, dim = 32, 2, 128
    pg = ref.Paged(rng, tok, ctx, 16, extra_cols=wide_cols(2, heads, 16) if wide else 1)
    c, _, host = fill(w4, rng, pg, heads, dim, bits)
    mask = ref.tree_masks(rng, tok)
    mask[:tok[0]] &= ~np.uint64(4)  # nobody but token 2 sees token 2
    mask[2] |= np.uint64(4)
    p, o = pg.where(0, [ctx[0] + 2])
    c.vs[int(p[0]), :, int(o[0])] = big
    q = rng.standard_normal((pg.tokens, hq, dim)).astype(F16)
    out = w4.kvq_attention(dev(q), c, make_batch(w4, pg), mask=dev(mask.view(np.int64)))
    check_attention(w4, rng, pg, q, c, host, hq, heads, dim, mask, dim ** -0.5, out, rows_off=(2,))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("scale", [0.1, -0.1])
def test_attention_negative_scales(w4, wide, bits, scale):  # noqa: F811
    """Scales of either sign are factors like any other, in both kernels."""
    rng = np.random.default_rng(23)
    tok, ctx, hq, heads, dim = (5, 3), (300, 20), 32, 2, 128
    pg = ref.Paged(rng, tok, ctx, 32, extra_cols=wide_cols(2, heads, 32) if wide else 1)
    c, _, host = fill(w4, rng, pg, heads, dim, bits)
    for (_, s), t in zip(host, (c.ks, c.vs)):
        s *= np.where(rng.random(s.shape) < 0.5, -1, 1).astype(F32)
        t.copy_(dev(s))
    q = rng.standard_normal((pg.tokens, hq, dim)).astype(F16)
    mask = ref.tree_masks(rng, tok)
    out = w4.kvq_attention(dev(q), c, make_batch(w4, pg), mask=dev(mask.view(np.int64)), scale=scale)
    check_attention(w4, rng, pg, q, c, host, hq, heads, dim, mask, scale, out)


@pytest.mark.parametrize("hq,dim", [(8, 64), (64, 64), (64, 128)])
@pytest.mark.parametrize("order", ["zeros first", "zeros last"])
def test_attention_many_zero_values(w4, hq, dim, order):  # noqa: F811
    """2^19 keys whose values are zero beside 2^15 ordinary ones, all with one
    logit: the zeros weigh as much as the others.  (8 rows and 64 take the two kernels.)"""
    rng = np.random.default_rng(24)
    zeros, rest, page = 1 << 19, 1 << 15, 256
    pg = ref.Paged(rng, (1,), (zeros + rest - 1,), page)
    c, _, host = fill(w4, rng, pg, 1, dim, 8)
    p, o = pg.where(0, np.arange(zeros) + (0 if order == "zeros first" else rest))
    vq, vs = host[1]
    vs[p, :, o] = 0
    vq[...] = np.abs(vq)  # a mean that is not 0
    c.vs.copy_(dev(vs))
    c.v.copy_(dev(vq))
    q = np.zeros((1, hq, dim), F16)
    out = w4.kvq_attention(dev(q), c, make_batch(w4, pg)).cpu().numpy().astype(np.float64)
    p, o = pg.where(0, np.arange(zeros + rest))
    (kq, ks), (vq, vs) = host
    want, err = ref.attention(q[0, :1], kq[p, 0, o], ks[p, 0, o], vq[p, 0, o], vs[p, 0, o], np.ones((1, zeros + rest), bool),
                              dim ** -0.5)
    assert np.all(np.abs(out[0] - want) <= err) and np.all(want > 0.01)


# -- dependent launches ---------------------------------------------------------------

@pytest.mark.parametrize("wide", [False, True])
def test_dependent_launches_give_the_same_bits(w4, wide):  # noqa: F811
    """A chain of all entry points, each reading what the one before wrote, with and
    without W4A8_LAUNCH_PDL: the kernels start early and wait before they read."""
    rng = np.random.default_rng(25)
    tok, ctx, hq, heads, dim, page = (9, 30), (700, 45), 32, 2, 128, 32
    pg = ref.Paged(rng, tok, ctx, page, extra_cols=wide_cols(2, heads, page) if wide else 1)
    c, gs, _ = fill(w4, rng, pg, heads, dim, 8)
    n = pg.tokens
    b = make_batch(w4, pg)
    normal = lambda *shape: dev(rng.standard_normal(shape).astype(F32))  # noqa: E731
    q, k, v, r, w = normal(n, hq, dim), normal(n, heads, dim), normal(n, heads, dim), normal(n, hq * dim), normal(hq * dim)
    pos = dev(rng.integers(0, 5000, n).astype(np.int32))
    freqs = w4.rope_frequencies(dim, 1e4)[0].cuda()
    mask = dev(ref.tree_masks(rng, tok).view(np.int64))
    keep = np.full(n, -1, np.int32)
    keep[:3], keep[9:11] = [2, 5, 8], [1, 29]
    keep = dev(keep)
    before = [t.clone() for t in c]
    ws = torch.zeros(w4.kvq_attention_workspace_bytes(c, b, n, hq), dtype=torch.uint8, device="cuda")

    def chain(flags):
        for t, u in zip(c, before):
            t.copy_(u)
        out, x = [], q
        for _ in range(3):
            x = w4.rope_rotate(x, pos, freqs, flags=flags)
            qo = w4.kvq_write(c, b, k, v, Q=x, pos=pos, freqs=freqs, flags=flags)
            a = w4.kvq_attention(qo, c, b, mask=mask, ws=ws, flags=flags)
            r2, x2 = w4.add_norm(r, w, y=a.view(n, -1), flags=flags)
            w4.kvq_keep(c, b, keep, flags=flags)
            out += [qo, a, r2, x2, *w4.kvq_read(c, b, n, flags=flags)]
            x = r2.view(n, hq, dim)
        return [t.clone() for t in out + list(c)]

    plain = chain(0)
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(plain, chain(1)))
    guards.check_all(*gs)
