"""A serving step's operators on the GPU against plain 64-bit references
(step_ref.py): within bounds counted from their roundings, and equal where what
comes out is whole numbers.  Outputs lie between guard bytes."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import guards  # noqa: E402
import layer_ref as ref  # noqa: E402
import step_ref as sref  # noqa: E402

pytestmark = pytest.mark.gpu

F32, F16, I32, I64, U8 = np.float32, np.float16, np.int32, np.int64, np.uint8
T = {F32: torch.float32, F16: torch.float16, I32: torch.int32, I64: torch.int64, U8: torch.uint8}
RANGE = 8  # bit 3 of the device error word


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bit_weight_quantized_w4a8_gb300 as m
    m.build()
    assert m.w4a8_device_error() == 0
    return m


@pytest.fixture(autouse=True)
def _no_error_left(w4):
    yield
    assert w4.w4a8_device_error() == 0


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def np_(t):
    return t.cpu().numpy()


def close(got, want, bound, what):
    got = np_(got).astype(np.float64)
    off = np.abs(got - want) - bound
    bad = np.unravel_index(np.argmax(np.where(np.isnan(off), np.inf, off)), off.shape)
    assert np.all(off <= 0), "%s at %s: got %r, want %r, bound %.3g" % (what, bad, got[bad], want[bad], bound[bad])


# -- the linear with e4m3 blocks -----------------------------------------------------

@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (8, 1040), (9, 3584), (65, 256), (200, 4096), (4100, 2048)])
@pytest.mark.parametrize("xt", [F32, F16])
def test_f8_quantize_rows(w4, M, K, xt):
    """Codes and scales bit-exact, ties between codes and quotients that round onto one included."""
    rng = np.random.default_rng(M + K)
    x = rng.standard_normal((M, K)).astype(xt)
    x[:, ::7] *= xt(30)
    x[0, :min(K, 64)] = (np.arange(min(K, 64)) * xt(0.125)).astype(xt)  # many ties when 448 / max is short
    x[-1, 0:16] = xt(0)
    if K > 128:
        x[0, 128:min(K, 256)] = 0  # a block of zeros
    gx, gs = guards.out((M, K), torch.uint8), guards.out((-(-K // 128), M), torch.float32)
    w4.f8_quantize_rows(dev(x), Xf=gx.t, sa=gs.t)
    guards.check_all(gx, gs)
    codes, scales = sref.f8_rows(x)
    assert np.array_equal(np_(gs.t), scales)
    got = np_(gx.t)
    assert np.array_equal(sref.E4M3[got], sref.E4M3[codes]) and np.array_equal(got & 127, codes & 127)


def test_f8_quantize_ties_and_tiny_scales(w4):
    """Exact ties go to the even code; quotients a rounding away from one go to
    their own side; scales below the normal numbers keep their codes."""
    m = np.float32(448 * 1.2345678)
    s = np.float64(sref.f8_scale(np.array([m]))[0])
    mids = (sref.E4M3[1:127] + sref.E4M3[:126]) / 2
    x = np.zeros((4, 128), F32)
    x[0, 0] = m
    x[0, 1:127] = (mids * s).astype(F32)
    x[1] = np.nextafter(x[0], F32(0))
    x[2] = np.nextafter(x[0], F32(1e9))
    x[3] = x[0] * F32(1e-42 / 448) * 64  # a scale of a few subnormal steps
    xf, sa = w4.f8_quantize_rows(dev(x))
    codes, scales = sref.f8_rows(x)
    assert np.array_equal(np_(sa), scales) and scales[0, 3] < 2.0 ** -126
    assert np.array_equal(sref.E4M3[np_(xf)], sref.E4M3[codes])


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (130, 144), (300, 1040), (5, 4096)])
def test_f8_quantize_weights(w4, N, K):
    rng = np.random.default_rng(N)
    w = (0.02 * rng.standard_normal((N, K))).astype(F32)
    gw, gs = guards.out((N, K), torch.uint8), guards.out((-(-N // 128), -(-K // 128)), torch.float32)
    w4.f8_quantize_weights(dev(w), Wf=gw.t, sw=gs.t)
    guards.check_all(gw, gs)
    codes, scales = sref.f8_weights(w)
    assert np.array_equal(np_(gs.t), scales) and np.array_equal(sref.E4M3[np_(gw.t)], sref.E4M3[codes])


# kernels for few rows (16, 32, 64, 128 of them; K in one piece or up to 8) and for many; sizes at
# their tile, block and piece edges
SHAPES = [(1, 16, 1), (1, 128, 128), (1, 1024, 129), (2, 112, 257), (16, 3584, 512), (17, 144, 130), (32, 2048, 127),
          (33, 4096, 384), (64, 1040, 1000), (65, 256, 300), (128, 1152, 640), (129, 512, 128), (300, 640, 513),
          (130, 256, 26000), (1000, 1040, 9001), (513, 128, 20480), (257, 272, 20001),
          (512, 3584, 512), (1500, 3584, 512), (400, 1024, 3584), (256, 1024, 4608), (500, 2064, 4601), (257, 128, 3585),
          (2560, 640, 500)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("yt", [F32, F16])
def test_f8_gemm(w4, M, K, N, yt):
    rng = np.random.default_rng(M + K + N)
    xf, wf = rng.integers(0, 127, (M, K)).astype(U8), rng.integers(0, 127, (N, K)).astype(U8)
    xf |= (rng.integers(0, 2, (M, K)) << 7).astype(U8)
    wf |= (rng.integers(0, 2, (N, K)) << 7).astype(U8)
    sa = (2.0 ** rng.uniform(-12, -6, (-(-K // 128), M))).astype(F32)
    sw = (2.0 ** rng.uniform(-12, -6, (-(-N // 128), -(-K // 128)))).astype(F32)
    sw[0, 0] = -sw[0, 0]
    y = guards.out((M, N), T[yt])
    w4.f8_gemm(dev(xf), dev(sa), dev(wf), dev(sw), Y=y.t)
    guards.check_all(y)
    want, err = sref.f8_product(xf, sa, wf, sw)
    close(y.t, want, err + ref.out_round(want, yt), "Y")


@pytest.mark.parametrize("M,K,N", [(1, 16, 65535 * 128 + 129), (2, 131072, 130), (20, 131072, 300), (300, 131072, 40),
                                   (70001, 32, 64)])
def test_f8_gemm_ends_of_the_sizes(w4, M, K, N):
    """Small whole numbers and scales of 1, sums below 2^24: exact."""
    g = torch.Generator(device="cuda").manual_seed(M)
    small = dev(sref.e4m3_codes(np.arange(-2, 3).astype(np.float64)))
    pick = lambda *s: torch.randint(0, 5, s, device="cuda", generator=g)  # noqa: E731
    x, w = pick(M, K), pick(N, K)
    kb = -(-K // 128)
    y = guards.out((M, N), torch.float32)
    w4.f8_gemm(small[x], torch.ones((kb, M), device="cuda"), small[w], torch.ones((-(-N // 128), kb), device="cuda"), Y=y.t)
    guards.check_all(y)
    for n in range(0, N, 1 << 22):
        want = (x.double() - 2) @ (w[n:n + (1 << 22)].double() - 2).T
        assert torch.equal(y.t[:, n:n + (1 << 22)].double(), want)


@pytest.mark.parametrize("M,K,N", [(1, 4096, 200), (40, 2064, 300), (100, 1024, 256), (600, 1296, 6001)])
def test_f8_gemm_whole_numbers(w4, M, K, N):
    """Small whole numbers and scales that are powers of two: every sum is exact."""
    rng = np.random.default_rng(K)
    small = sref.e4m3_codes(np.arange(-4, 5).astype(np.float64))
    xf, wf = small[rng.integers(0, 9, (M, K))], small[rng.integers(0, 9, (N, K))]
    sa = (2.0 ** rng.integers(0, 2, (-(-K // 128), M))).astype(F32)
    sw = (2.0 ** rng.integers(0, 2, (-(-N // 128), -(-K // 128)))).astype(F32)
    y = w4.f8_gemm(dev(xf), dev(sa), dev(wf), dev(sw))
    assert np.array_equal(np_(y).astype(np.float64), sref.f8_product(xf, sa, wf, sw)[0])


@pytest.mark.parametrize("M,K,N", [(1, 3584, 512), (50, 1040, 300), (700, 512, 9000)])
@pytest.mark.parametrize("xt,yt", [(F32, F16), (F16, F32)])
def test_f8_linear(w4, M, K, N, xt, yt):
    """The two steps in one call: the same bits, with a caller's workspace or its own, dependent launches too."""
    rng = np.random.default_rng(M)
    x, w = rng.standard_normal((M, K)).astype(xt), (0.05 * rng.standard_normal((N, K))).astype(F32)
    wf, sw = w4.f8_quantize_weights(dev(w))
    xf, sa = w4.f8_quantize_rows(dev(x))
    want = w4.f8_gemm(xf, sa, wf, sw, dtype=T[yt])
    y, ws = guards.out((M, N), T[yt]), guards.out((w4.f8_linear_workspace_bytes(M, K, N),), torch.uint8)
    w4.f8_linear(dev(x), wf, sw, Y=y.t, ws=ws.t)
    guards.check_all(y, ws)
    assert torch.equal(y.t, want) and torch.equal(w4.f8_linear(dev(x), wf, sw, dtype=T[yt]), want)
    assert torch.equal(w4.f8_linear(dev(x), wf, sw, dtype=T[yt], flags=w4.LAUNCH_PDL), want)
    ws2 = torch.empty(ws.nbytes - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(w4.W4A8Error):
        w4.f8_linear(dev(x), wf, sw, ws=ws2)


@pytest.mark.parametrize("M", [1, 2, 3])
@pytest.mark.parametrize("K,N", [(16, 5), (128, 128), (144, 130), (640, 200), (1040, 4000), (18944, 384), (272, 40000)])
@pytest.mark.parametrize("xt", [F32, F16])
def test_f8_linear_single_tokens(w4, M, K, N, xt):
    """Few rows take one launch, or two where the weights are many: the bits of the two steps, zero, tiny and
    not finite blocks among them, and nothing of the rows behind the last."""
    rng = np.random.default_rng(K + N)
    x = rng.standard_normal((M + 1, K)).astype(xt)
    x[0, :min(K, 128)] = np.round(8 * x[0, :min(K, 128)]) / 8  # quotients near ties
    x[M - 1, 256:384] = 0
    x[M - 1, 128:256] *= xt(1e-6)
    x[M, :] = np.nan
    wf, sw = w4.f8_quantize_weights(dev((0.05 * rng.standard_normal((N, K))).astype(F32)))
    for odd in (None, np.nan, np.inf):
        if odd is not None:
            x[0, K // 2] = odd
        a = dev(x)[:M]
        y = guards.out((M, N), torch.float32)
        for flags in (0, w4.LAUNCH_PDL):
            y.t.zero_()
            w4.f8_linear(a, wf, sw, Y=y.t, flags=flags)
            guards.check_all(y)
            want = w4.f8_gemm(*w4.f8_quantize_rows(a), wf, sw)
            assert np.array_equal(np_(y.t), np_(want), equal_nan=True)
        assert np.isnan(np_(y.t)[0]).all() == (odd is not None) and np.isfinite(np_(y.t)[1:]).all()


def test_f8_linear_not_finite(w4):
    """An infinity or a NaN stays in its row of X (and its rows of W)."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((20, 512)).astype(F16)
    x[3, 200], x[7, 300] = np.nan, np.inf
    wf, sw = w4.f8_quantize_weights(dev((0.05 * rng.standard_normal((300, 512))).astype(F32)))
    y = np_(w4.f8_linear(dev(x), wf, sw))
    bad = np.isnan(y).all(1)
    assert list(np.flatnonzero(bad)) == [3, 7] and np.isfinite(y[~bad]).all()


# -- rotary positions with several axes ------------------------------------------------

@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 64), (128, 24), (256, 256)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_rope_rotate_axes(w4, dim, rot, inter, axes):
    rng = np.random.default_rng(dim + rot + axes)
    n, h = 9, 3
    x = rng.standard_normal((n, h, dim)).astype(F32)
    pos = rng.integers(-100, 1_000_000, (axes, n)).astype(I32)
    axis = [int(a) for a in rng.integers(0, axes, rot // 2)]
    f = 1e6 ** (-2.0 * np.arange(rot // 2) / rot)
    want, err = sref.rotate_axes(x, pos, axis, f, inter, 1.25)
    y = guards.out((n, h, dim), torch.float16)
    w4.rope_rotate(dev(x), dev(pos), dev(f), interleaved=inter, mscale=1.25, Y=y.t, axis=axis)
    guards.check_all(y)
    close(y.t, want, err + ref.out_round(want, F16), "Y")


def test_rope_axes_strides_and_one_axis(w4):
    """Rows at a distance, in place, and several axes with one number are the plain call's bits."""
    rng = np.random.default_rng(4)
    fused = dev(rng.standard_normal((11, 8 * 64)).astype(F32))
    f = dev(1e4 ** (-np.arange(32) / 32))
    pos = dev(rng.integers(0, 5000, 11).astype(I32))
    three = pos[None].repeat(3, 1).contiguous()
    axis = w4.rope_axes((8, 12, 12), cycled=True)
    x = fused[:, 64:64 * 6].view(11, 5, 64)
    plain = w4.rope_rotate(x, pos, f)
    assert torch.equal(w4.rope_rotate(x, three, f, axis=axis), plain)
    before = fused.clone()
    w4.rope_rotate(x, three, f, Y=x, axis=axis)
    assert torch.equal(x, plain) and torch.equal(fused[:, :64], before[:, :64]) and torch.equal(fused[:, 384:], before[:, 384:])


def test_rope_axis_is_a_sequence_of_numbers(w4):
    x, pos = torch.zeros((2, 2, 64), device="cuda"), torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    freqs = torch.ones(32, dtype=torch.float64, device="cuda")
    with pytest.raises(TypeError):  # not a count of them
        w4.rope_rotate(x, pos, freqs, axis=32)
    with pytest.raises(ValueError, match="32 pairs, got 4"):  # entries are counted, not an array's bytes
        w4.rope_rotate(x, pos, freqs, axis=np.zeros(4, np.int64))
    with pytest.raises(ValueError):
        w4.rope_rotate(x, pos, freqs, axis=[-1] * 32)
    w4.rope_rotate(x, pos, freqs, axis=np.full(32, 2, np.int64))


@pytest.mark.parametrize("bits", [8, 4])
def test_kvq_write_axes(w4, bits):
    """Keys and queries turned by several axes in the cache's write: the write of keys
    that were turned before, bit for bit, and the queries as rope_rotate gives them."""
    rng = np.random.default_rng(bits)
    n, hq, hkv, dim, page = 70, 6, 2, 128, 16
    q, k, v = (dev(rng.standard_normal((n, h, dim)).astype(F32)) for h in (hq, hkv, hkv))
    pos = dev(rng.integers(0, 3000, (3, n)).astype(I32))
    f = dev(1e6 ** (-np.arange(64) / 64))
    axis = w4.rope_axes((16, 24, 24))
    cu, start = dev(np.array([0, 30, 70], I32)), dev(np.array([5, 0], I32))
    table = dev(np.array([[3, 0, 7], [2, 5, 1]], I32))
    batch = w4.KVQBatch(cu, start, table)
    a, b = (w4.kvq_cache(8, page, hkv, dim, bits) for _ in range(2))
    qa = w4.kvq_write(a, batch, k, v, Q=q, pos=pos, freqs=f, axis=axis)
    turned = w4.rope_rotate(k, pos, f, axis=axis)
    w4.kvq_write(b, batch, turned, v)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(qa, w4.rope_rotate(q, pos, f, dtype=torch.float16, axis=axis))


# -- verification of drafts ---------------------------------------------------------------

def tree_words(n, rng):
    words = []
    for i in range(n):
        p = int(rng.integers(0, i)) if i else -1
        words.append((words[p] if p >= 0 else 0) | 1 << i)
    return np.array(words, np.uint64).view(I64)


def drafts(rng, sizes, v, lt=F32, tree=False, with_q=False, sharp=1.0):
    """A batch whose drafts are likely enough that some are taken."""
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(I32)
    n = int(cu[-1])
    logits = (sharp * rng.standard_normal((n, v)) * 2).astype(lt)
    mask = np.concatenate([tree_words(s, rng) for s in sizes]) if tree and n else None
    q = None
    ids = np.zeros(n, I32)
    if with_q:
        near = logits.astype(np.float64) + 0.4 * rng.standard_normal((n, v))
        q = np.exp(near - near.max(1, keepdims=True))
        q = (q / q.sum(1, keepdims=True)).astype(F32)
    for b, s in enumerate(sizes):
        lo = int(cu[b])
        par = sref.parents(s, None if mask is None else [int(m) for m in mask[lo:lo + s].view(np.uint64)])
        for i in range(1, s):
            p = q[lo + par[i]].astype(np.float64) if with_q else sref.distribution(logits[lo + par[i]], 1.0) ** 0.5
            ids[lo + i] = rng.choice(v, p=p / p.sum())
    return logits, cu, ids, rng.random(n).astype(F32), mask, q


def run_verify(w4, logits, cu, ids, u, mask=None, q=None, temp=None, **kw):
    n, seqs = logits.shape[0], len(cu) - 1
    outs = [guards.out((n,), torch.int32), guards.out((n,), torch.int32), guards.out((seqs,), torch.int32)]
    for g in outs:
        g.t.fill_(-7)
    d = lambda a: None if a is None else a if isinstance(a, torch.Tensor) else dev(a)  # noqa: E731
    ws = guards.out((w4.draft_verify_workspace_bytes(*logits.shape),), torch.uint8)
    w4.draft_verify(d(logits), d(cu), d(ids), d(u), mask=d(mask), q=d(q), temp=d(temp), keep=outs[0].t, out=outs[1].t,
                    count=outs[2].t, ws=ws.t, **kw)
    guards.check_all(*outs, ws)
    return [np_(g.t) for g in outs]


def same(got, want, what=""):
    for g, w, name in zip(got, want, ("keep", "out", "count")):
        assert np.array_equal(g, w), "%s %s: got %s, want %s" % (what, name, g, w)


@pytest.mark.parametrize("v", [1, 2, 5, 127, 128, 129, 511, 512, 513, 4096, 4097, 32001])
@pytest.mark.parametrize("tree,with_q", [(False, False), (False, True), (True, False), (True, True)])
def test_draft_verify(w4, v, tree, with_q):
    rng = np.random.default_rng(v + 2 * tree + with_q)
    a = drafts(rng, [1, 6, 0, 3, 12, 2, 64] if v < 4096 else [5, 0, 9], v, tree=tree, with_q=with_q)
    temp = (0.5 + rng.random(len(a[1]) - 1)).astype(F32)
    temp[::3] = 0
    same(run_verify(w4, *a, temp), sref.verify(*a, temp))
    same(run_verify(w4, *a), sref.verify(*a))


@pytest.mark.parametrize("lt,qt", [(F16, F32), (F32, F16), (F16, F16)])
def test_draft_verify_types_rows_and_alignment(w4, lt, qt):
    """16-bit logits and probabilities; rows at a distance and off the vector's alignment."""
    rng = np.random.default_rng(8)
    logits, cu, ids, u, _, q = drafts(rng, [4, 7, 2], 1001, lt, with_q=True)
    q = q.astype(qt)
    want = sref.verify(logits, cu, ids, u, None, q)
    same(run_verify(w4, logits, cu, ids, u, None, q), want)
    wide = torch.zeros((13, 1109), dtype=T[lt], device="cuda")
    wide[:, 3:1004] = dev(logits)
    wide_q = torch.zeros((13, 1010), dtype=T[qt], device="cuda")
    wide_q[:, 1:1002] = dev(q)
    same(run_verify(w4, wide[:, 3:1004], cu, ids, u, None, wide_q[:, 1:1002]), want, "strided")


def test_draft_verify_more_than_one_slice_and_many_sequences(w4):
    rng = np.random.default_rng(9)
    a = drafts(rng, [3] * 100, 700, with_q=True)
    same(run_verify(w4, *a), sref.verify(*a))
    a = drafts(rng, [2, 3], 152064, sharp=2.0)
    same(run_verify(w4, *a), sref.verify(*a))
    a = drafts(rng, [2], 152065, with_q=True)
    same(run_verify(w4, *a), sref.verify(*a))


def test_draft_verify_flat_rows_take_the_exact_sums(w4):
    """Nearly equal weights: the fp32 sums leave the token open, the integers decide."""
    rng = np.random.default_rng(10)
    for with_q in (False, True):
        logits, cu, ids, u, mask, q = drafts(rng, [3] * 12, 50000, with_q=with_q, sharp=1e-3)
        same(run_verify(w4, logits, cu, ids, u, mask, q), sref.verify(logits, cu, ids, u, mask, q))


def test_draft_verify_masked_and_useless_rows(w4):
    rng = np.random.default_rng(11)
    v = 3000
    for with_q in (False, True):
        logits, cu, ids, u, _, q = drafts(rng, [4] * 8, v, with_q=with_q)
        logits[0:4, rng.random(v) < 0.9] = -np.inf          # most tokens masked
        logits[4:8, 1:] = -np.inf                            # one token left
        logits[8] = -np.inf                                  # nothing left at the root
        logits[13, 5] = np.nan                               # no distribution after the first draft
        logits[16, 7] = np.inf
        logits[20:24] = np.finfo(F32).min                    # the lowest value everywhere: uniform
        logits[24:28, ::2] = np.finfo(F32).min               # ... beside ordinary logits
        ids[[5, 6, 7]] = 0
        ids[29] = -1                                         # drafts outside the vocabulary
        ids[30] = v
        same(run_verify(w4, logits, cu, ids, u, None, q), sref.verify(logits, cu, ids, u, None, q))
        zero = np.zeros(8, F32)
        same(run_verify(w4, logits, cu, ids, u, None, q, zero), sref.verify(logits, cu, ids, u, None, q, zero))


def test_draft_verify_siblings_twice_and_ties(w4):
    """A token drafted twice under one parent; equal largest logits (the first counts)."""
    rng = np.random.default_rng(12)
    v = 600
    logits = rng.standard_normal((6, v)).astype(F32)
    logits[0, 17], logits[0, 400] = 9, 8.9
    logits[:, 300] = logits[:, 301] = 9.5
    mask = np.array([1, 3, 5, 9, 17, 0b100011], np.uint64).view(I64)  # four children of the root, a child of the first
    ids = np.array([0, 17, 17, 400, 400, 300], I32)
    cu = np.array([0, 6], I32)
    for u1 in (0.0, 0.3, 0.6, 0.99):
        u = np.array([0.5, u1, 0.01, u1, 0.02, 0.5], F32)
        same(run_verify(w4, logits, cu, ids, u, mask), sref.verify(logits, cu, ids, u, mask), u1)
    zero = np.zeros(1, F32)
    ids[1:] = [301, 300, 300, 301, 300]
    same(run_verify(w4, logits, cu, ids, u, mask, None, zero), sref.verify(logits, cu, ids, u, mask, None, zero))


@pytest.mark.parametrize("u0", [0.0, 1.0 - 2.0 ** -24, 0.5, 2.0 ** -24, 2.0 ** -126])
def test_draft_verify_ends_of_the_random_numbers(w4, u0):
    rng = np.random.default_rng(13)
    logits, cu, ids, u, mask, q = drafts(rng, [1, 2, 3], 2000, with_q=True)
    u[:] = u0
    same(run_verify(w4, logits, cu, ids, u, mask, q), sref.verify(logits, cu, ids, u, mask, q))
    low = logits.copy()
    low[:, :7] = low[:, -7:] = -np.inf  # neither end's token may come out
    got = run_verify(w4, low, cu, ids, u)
    assert np.all((got[1][[0, 1, 3]] >= 7) & (got[1][[0, 1, 3]] < 1993))


def test_draft_verify_random_numbers_outside(w4):
    """u >= 1, negative and NaN: a token of the vocabulary all the same."""
    logits = np.zeros((4, 1000), F32)
    got = run_verify(w4, logits, np.arange(5, dtype=I32), np.zeros(4, I32), np.array([1.0, 7.0, -3.0, np.nan], F32))
    assert list(got[1][:3]) == [999, 999, 0] and 0 <= got[1][3] < 1000 and list(got[2]) == [1] * 4


def test_draft_verify_tests_with_numbers_outside(w4):
    """The same of a draft's random number and probability: a token without weight is never taken, a token
    with all of it always."""
    rng = np.random.default_rng(22)
    v = 700
    logits = rng.standard_normal((16, v)).astype(F32)
    logits[::2, :350] = -np.inf
    logits[8, 400:] = logits[8, :399] = -np.inf  # token 399 has it all
    ids = np.full(16, 5, I32)
    ids[[9, 11]] = 399, 500
    u = np.full(16, 0.5, F32)
    u[1::2] = [-1, -np.inf, np.nan, 0, 1, np.nan, 0, 0]
    cu = np.arange(0, 17, 2, dtype=I32)
    got = run_verify(w4, logits, cu, ids, u)
    inside = u.copy()
    inside[1::2] = [0, 0, 0, 0, 1 - 2.0 ** -24, 0, 0, 0]
    same(got, sref.verify(logits, cu, ids, inside))
    assert list(got[2]) == [1, 1, 1, 1, 2, 2, 1, 1]
    q = np.exp(rng.standard_normal((16, v)))
    q = (q / q.sum(1, keepdims=True)).astype(F32)
    wild = q.copy()
    wild[0, 5], wild[2, 5], wild[4, 5], wild[8, 399], wild[10, 500] = -0.5, np.nan, np.inf, 3.0, -np.inf
    wild[6, 400:440], wild[12, 500:], wild[14, 350:] = -2.0, np.nan, np.inf
    got = run_verify(w4, logits, cu, ids, u, None, wild)
    same(got, sref.verify(logits, cu, ids, inside, None, np.where(np.isnan(wild), 0, np.clip(wild, 0, 1)).astype(F32)))


@pytest.mark.parametrize("temp", [2.0 ** -20, 1e-3, 30.0, 1e30, np.inf])
def test_draft_verify_temperatures(w4, temp):
    rng = np.random.default_rng(14)
    logits, cu, ids, u, mask, q = drafts(rng, [3, 4], 1500)
    logits[2, 40:90] = -np.inf
    t = np.full(2, temp, F32)
    want = sref.verify(logits, cu, ids, u, mask, q, np.minimum(t, F32(2.0 ** 60)))
    same(run_verify(w4, logits, cu, ids, u, mask, q, t), want)
    bad = np.array([-1.0, np.nan], F32)  # greedy
    same(run_verify(w4, logits, cu, ids, u, mask, q, bad), sref.verify(logits, cu, ids, u, mask, q, np.zeros(2, F32)))


def test_draft_verify_far_logits(w4):
    """Rows far from zero: the weights depend on differences alone."""
    rng = np.random.default_rng(15)
    logits, cu, ids, u, mask, q = drafts(rng, [3, 4, 5], 900)
    far = (np.round(logits * 64) / 64 + 30000).astype(F32)
    same(run_verify(w4, far, cu, ids, u), sref.verify(far, cu, ids, u))
    same(run_verify(w4, -far, cu, ids, u), sref.verify(-far, cu, ids, u))


def test_draft_verify_rows_that_no_sequence_holds_and_too_long(w4):
    """Rows behind the last sequence, and in front of the first, are left as they were; a
    sequence of more than 64 tokens is refused on the device."""
    rng = np.random.default_rng(16)
    logits, _, ids, u, _, _ = drafts(rng, [90], 300)
    cu = np.array([2, 5, 70, 80], I32)  # 3, 65 and 10 tokens; 2 rows before, 10 behind
    got = run_verify(w4, logits, cu, ids, u)
    assert w4.w4a8_device_error() == RANGE
    want = sref.verify(logits[:80], np.array([2, 5, 5, 70, 80], I32)[[0, 1, 1, 3, 4]], ids[:80], u[:80])
    for g, w in zip(got[:2], want[:2]):
        assert np.array_equal(g[2:5], w[2:5]) and np.array_equal(g[70:80], w[70:80])
        assert np.all(g[:2] == -7) and np.all(g[80:] == -7) and np.all(g[5:70] == -1)
    assert got[2][1] == 0
    logits, _, ids, u, _, _ = drafts(rng, [64], 300)
    same(run_verify(w4, logits, np.array([0, 64], I32), ids, u), sref.verify(logits, np.array([0, 64]), ids, u))


def test_draft_verify_bad_offsets(w4):
    logits, ids, u = np.zeros((6, 50), F32), np.zeros(6, I32), np.zeros(6, F32)
    for cu in ([0, 7], [-1, 3], [4, 2], [0, 2 ** 31 - 1]):
        got = run_verify(w4, logits, np.array(cu, I32), ids, u)
        assert got[2][0] == 0 and w4.w4a8_device_error() == RANGE


def test_draft_verify_refusals_before_a_row_of_no_use(w4):
    """Two siblings refused over the whole row, then a third taken whose own row holds no distribution:
    the next token is -1."""
    rng = np.random.default_rng(18)
    seqs, v = 24, 20000
    logits = rng.standard_normal((4 * seqs, v)).astype(F32)
    q = np.exp(rng.standard_normal((4 * seqs, v)))
    q[:, 7] = 0
    q = (q / q.sum(1, keepdims=True)).astype(F32)
    ids, u = np.zeros(4 * seqs, I32), rng.random(4 * seqs).astype(F32)
    for b in range(seqs):
        ids[4 * b + 1:4 * b + 3] = np.argsort(q[4 * b] / sref.distribution(logits[4 * b], 1.0))[-2:]
        ids[4 * b + 3] = 7
    logits[3::4] = np.nan
    u[1::4] = u[2::4] = 0.999
    mask = np.tile(np.array([1, 3, 5, 9], np.uint64).view(I64), seqs)
    cu = np.arange(0, 4 * seqs + 1, 4, dtype=I32)
    got = run_verify(w4, logits, cu, ids, u, mask, q)
    same(got, sref.verify(logits, cu, ids, u, mask, q))
    assert np.all(got[2] == 2) and np.all(got[1].reshape(seqs, 4)[:, :2] == [7, -1])


def test_draft_verify_largest_vocabulary_many_refusals(w4):
    """2^22 equal weights and eight refusals of one token at the root: what is taken off adds up to 2^66 of
    the units of 2^-40.  Roundings: half a unit a weight and a refusal's, 2^-20 of a weight after 2^22."""
    rng = np.random.default_rng(23)
    v, kids = 2 ** 22, 8
    logits = np.zeros((kids + 1, v), F32)
    q = rng.random(v)
    q[77] = 0
    q *= 0.4 / q.sum()
    q[77] = 0.6
    q = np.tile(q.astype(F32), (kids + 1, 1))
    ids = np.full(kids + 1, 77, I32)
    u = np.full(kids + 1, 0.99, F32)
    mask = np.array([1] + [1 | 1 << i for i in range(1, kids + 1)], np.uint64).view(I64)
    cu = np.array([0, kids + 1], I32)
    for u0 in (0.0, 0.123, 0.5, 0.987):
        u[0] = u0
        got, want = run_verify(w4, logits, cu, ids, u, mask, q), sref.verify(logits, cu, ids, u, mask, q)
        assert got[2][0] == 1 and abs(int(got[1][0]) - int(want[1][0])) <= 1


def test_draft_verify_roundings_of_a_long_tail_do_not_add_up(w4):
    """A draw among 2^20 tokens that hold 2^-29 of the largest weight each, of which the draft's
    probabilities leave about half: some 2^10 of the units of 2^-40 that the sums are made of.  A weight is
    the difference of two numbers rounded to nearest, off by at most a unit and by 0.41 in the root mean
    square, so that a sum over 2^20 is off by about 420 units, half a token; six times that are less than 3
    tokens.  Numbers all cut off on one side would be off by up to 2^19 units, hundreds of tokens."""
    g = torch.Generator(device="cuda").manual_seed(19)
    seqs, v = 16, 2 ** 20
    logits = -20 + 0.1 * torch.randn((2 * seqs, v), device="cuda", generator=g)
    logits[:, 0] = 0
    logits[:, v - 1] = -20 + math.log(v)
    p = torch.softmax(logits.double(), 1)
    q = p * (0.3 + 0.4 * torch.rand((2 * seqs, v), device="cuda", generator=g))
    q[:, v - 1] = 0
    q[:, 0] = 0
    q[:, 0] = 1 - q.sum(1)
    q = q.float()
    u = torch.full((2 * seqs,), 0.99999, device="cuda")
    u[::2] = torch.linspace(0.01, 0.3, seqs, device="cuda")
    cu = torch.arange(0, 2 * seqs + 1, 2, dtype=torch.int32, device="cuda")
    keep, out, count = w4.draft_verify(logits, cu, torch.zeros(2 * seqs, dtype=torch.int32, device="cuda"), u, q=q)
    run = (p[::2] - q[::2].double()).clamp_min(0).cumsum(1)
    want = torch.searchsorted(run, u[::2, None].double() * run[:, -1:], right=True)[:, 0]
    assert bool((count == 1).all()) and bool((want < v - 1).all())
    off = (out[::2].long() - want).abs().max()
    assert int(off) <= 3, off


def test_draft_verify_follows_the_target(w4):
    """Over a grid of random numbers, the drafts taken with their probabilities, the first
    token said has the target's distribution: 24576 sequences in one call."""
    rng = np.random.default_rng(17)
    v, g = 6, 64
    row = rng.standard_normal(v).astype(F32)
    q = np.array([0.3, 0.05, 0.2, 0.25, 0.1, 0.1], F32)
    x, i1, i0 = (a.reshape(-1) for a in np.meshgrid(np.arange(v), np.arange(g), np.arange(g), indexing="ij"))
    s = len(x)
    ids = np.zeros(2 * s, I32)
    ids[1::2] = x
    u = np.zeros(2 * s, F32)
    u[::2], u[1::2] = (i0 + 0.5) / g, (i1 + 0.5) / g
    cu = np.arange(0, 2 * s + 1, 2, dtype=I32)
    got = run_verify(w4, np.tile(row, (2 * s, 1)), cu, ids, u, None, np.tile(q, (2 * s, 1)))
    freq = np.bincount(got[1][::2], weights=q[x].astype(np.float64) / g ** 2, minlength=v)
    assert np.all(np.abs(freq - sref.distribution(row, 1.0)) < 2.5 / g)


# -- the plan of a step ----------------------------------------------------------------------

def make_pool(rng, seqs, width, pages, page, lens):
    held = -(-lens // page)
    perm = rng.permutation(pages).astype(I32)
    table = np.full((seqs, width), -1, I32)
    at = 0
    for b in range(seqs):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    stack = np.full(pages, -1, I32)
    stack[:pages - at] = perm[at:]
    return sref.Pool(table, held.astype(I32), stack, pages - at, lens, page)


class Planner:
    """The device's pool beside the host's, call by call."""

    def __init__(self, w4, host):
        self.w4, self.host = w4, host
        self.g = [guards.Guarded(a.shape, torch.int32) for a in (host.table, host.held, host.stack)]
        self.g += [guards.Guarded((1,), torch.int32), guards.Guarded(host.lens.shape, torch.int32)]
        for g, a in zip(self.g, (host.table, host.held, host.stack, np.array([host.top]), host.lens)):
            g.t.copy_(dev(np.asarray(a).astype(I32)))
        self.pool, self.lens = w4.KVQPool(*(g.t for g in self.g[:4])), self.g[4].t

    def plan(self, add, tokens, grow=None, mask=None, **kw):
        d = lambda a, t: None if a is None else dev(np.asarray(a, t))  # noqa: E731
        outs = [guards.out((len(add) + 1,), torch.int32), guards.out((tokens,), torch.int32),
                guards.out((tokens,), torch.int64), guards.out((tokens,), torch.int32)]
        ws = guards.out((self.w4.kvq_plan_workspace_bytes(self.pool, self.host.page),), torch.uint8)
        self.w4.kvq_plan(self.pool, self.host.page, self.lens, d(add, I32), tokens, grow=d(grow, I32), mask=d(mask, I64),
                         cu=outs[0].t, pos=outs[1].t, slot=outs[2].t, seq=outs[3].t, ws=ws.t, **kw)
        guards.check_all(*outs, ws, *self.g)
        want = self.host.plan(np.asarray(add), tokens, None if grow is None else np.asarray(grow), mask)
        for g, w, name in zip(outs, want, ("cu", "pos", "slot", "seq")):
            assert np.array_equal(np_(g.t), w), name
        h = self.host
        held, table = np_(self.pool.held), np_(self.pool.table)
        assert np.array_equal(held, h.held) and np.array_equal(np_(self.lens), h.lens)
        assert int(self.pool.top[0]) == h.top and np.array_equal(np_(self.pool.stack)[:h.top], h.stack[:h.top])
        for b in range(len(held)):
            assert np.array_equal(table[b, :held[b]], h.table[b, :held[b]])
        return want


# one CTA; a cluster that writes the step; one with a second launch; several rows a thread
@pytest.mark.parametrize("seqs,tokens,width", [(1, 1, 1), (1, 5000, 400), (3, 40, 4), (48, 300, 70), (1024, 4096, 20),
                                               (1025, 4000, 20), (700, 3000, 500), (300, 16384, 60), (300, 16388, 60),
                                               (5000, 60001, 12), (8192, 9000, 4), (8193, 20000, 4), (65536, 70000, 3)])
def test_kvq_plan(w4, seqs, tokens, width):
    rng = np.random.default_rng(seqs + tokens)
    page = int(rng.choice([16, 32, 64]))
    lens = rng.integers(0, max(1, (width - 1) * page // 2), seqs)
    pages = int((-(-lens // page)).sum()) + seqs * 2 + 40
    p = Planner(w4, make_pool(rng, seqs, width, pages, page, lens))
    each = max(1, tokens // seqs)
    first = rng.integers(0, each + 1, seqs)
    p.plan(first, tokens)
    p.plan(np.where(rng.random(seqs) < 0.3, -1, rng.integers(0, 2 * each + 1, seqs)), tokens, grow=first)
    p.plan(rng.integers(0, each + 2, seqs), tokens, grow=rng.integers(0, 2, seqs), flags=w4.LAUNCH_PDL)
    p.plan(np.full(seqs, -1), tokens)
    assert p.host.top == pages  # all of it came back


def test_kvq_plan_waiting_requests(w4):
    """Too few pages, too few tokens, rows too long for the table: those wait, rows that need nothing do not."""
    rng = np.random.default_rng(1)
    lens = np.array([10, 16, 0, 3, 40, 5, 0, 15])
    p = Planner(w4, make_pool(rng, 8, 4, 20, 16, lens))
    got = p.plan([6, 1, 40, 2, 5, 3, 16, 1], 100)     # enough for all
    assert list(np.diff(got[0])) == [6, 1, 40, 2, 5, 3, 16, 1]
    q = Planner(w4, make_pool(rng, 8, 4, 10, 16, lens))
    got = q.plan([6, 1, 40, 2, 100, 3, 16, 1], 100)  # the third asks for more than is free, the fifth can never fit
    assert list(np.diff(got[0])) == [6, 1, 0, 2, 0, 3, 0, 1]
    q.plan([0, 0, 0, -1, -1, 0, 16, 0], 100)          # pages that come back serve the same call
    r = Planner(w4, make_pool(rng, 8, 4, 60, 16, lens))
    got = r.plan([4, 4, 4, 4, 4, 4, 4, 4], 18)        # room for four rows of tokens and a half
    assert list(np.diff(got[0])) == [4, 4, 4, 4, 0, 0, 0, 0]


def test_kvq_plan_depths_of_a_tree(w4):
    rng = np.random.default_rng(2)
    p = Planner(w4, make_pool(rng, 3, 5, 20, 16, np.array([7, 30, 0])))
    mask = np.concatenate([tree_words(5, rng), tree_words(9, rng), tree_words(2, rng), np.zeros(4, I64)])
    p.plan([5, 9, 2], 20, mask=mask)


def test_kvq_plan_optional_outputs(w4):
    L, p = w4.lib(), w4.kvq_pool(2, 4, 8)
    import ctypes
    from bit_weight_quantized_w4a8_gb300 import _binding as B
    lens, add, cu = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, 0], [3, 20], [0, 0, 0]))
    arg = ctypes.byref(B._Pool(*(t.data_ptr() for t in p), 2, 4, 8, 16))
    ws = torch.empty(w4.kvq_plan_workspace_bytes(p, 16), dtype=torch.uint8, device="cuda")
    st = L.kvq_plan(arg, lens.data_ptr(), None, add.data_ptr(), None, 30, cu.data_ptr(), None, None, None, ws.data_ptr(),
                    ws.numel(), 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and cu.tolist() == [0, 3, 23] and p.held.tolist() == [1, 2] and p.top.tolist() == [5]
    assert p.table[0, 0] == 7 and p.table[1, :2].tolist() == [6, 5]


def test_kvq_plan_counters_out_of_range(w4):
    """Cut to their range and reported; nothing outside the arrays is touched (guard bytes)."""
    rng = np.random.default_rng(3)
    for held, top, lens in (([99, -5], 3, [4, 4]), ([1, 1], 10 ** 9, [4, 4]), ([1, 1], -4, [4, 4]), ([0, 0], 3, [-9, 2 ** 31 - 1])):
        p = Planner(w4, make_pool(rng, 2, 3, 8, 16, np.array([4, 4])))
        p.pool.held.copy_(dev(np.array(held, I32)))
        p.pool.top.fill_(top)
        p.lens.copy_(dev(np.array(lens, I32)))
        for add in ([1, 1], [-1, 1], [-1, -1]):
            w4.kvq_plan(p.pool, 16, p.lens, dev(np.array(add, I32)), 40)
            guards.check_all(*p.g)
            assert 0 <= int(p.pool.top[0]) <= 8 and int(p.pool.held.min()) >= 0 and int(p.pool.held.max()) <= 3
        assert w4.w4a8_device_error() == RANGE


# -- several streams, graphs --------------------------------------------------------------------

def test_calls_on_two_streams_and_in_a_graph(w4):
    """The same call at once on two streams, captured twice and replayed in turn: the same results."""
    rng = np.random.default_rng(20)
    logits, cu, ids, u, mask, q = drafts(rng, [5, 9, 3], 5000, tree=True, with_q=True)
    want = sref.verify(logits, cu, ids, u, mask, q)
    a = [dev(x) for x in (logits, cu, ids, u)]
    m, qd = dev(mask), dev(q)
    x = dev(rng.standard_normal((40, 1024)).astype(F16))
    wf, sw = w4.f8_quantize_weights(dev((0.05 * rng.standard_normal((700, 1024))).astype(F32)))
    y0 = w4.f8_linear(x, wf, sw)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                got.append((w4.draft_verify(*a, mask=m, q=qd), w4.f8_linear(x, wf, sw)))
    torch.cuda.synchronize()
    for v, y in got:
        same([np_(t) for t in v], want)
        assert torch.equal(y, y0)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((w4.draft_verify(*a, mask=m, q=qd), w4.f8_linear(x, wf, sw)))
        graphs.append(g)
    for i in (0, 1, 1, 0):
        for v, y in outs:
            for t in v:
                t.fill_(-9)
            y.zero_()
        graphs[i].replay()
        w4.draft_verify(*a)  # an eager call in between
        torch.cuda.synchronize()
        same([np_(t) for t in outs[i][0]], want)
        assert torch.equal(outs[i][1], y0)


def test_wide_linear_twice_at_once(w4):
    """Two calls of the kernel for many rows, whose CTAs hold all of their SMs' tensor memory."""
    rng = np.random.default_rng(21)
    x = dev(rng.standard_normal((1500, 512)).astype(F16))
    wf, sw = w4.f8_quantize_weights(dev((0.05 * rng.standard_normal((9000, 512))).astype(F32)))
    y0 = w4.f8_linear(x, wf, sw, dtype=torch.float16)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    ys = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                ys.append(w4.f8_linear(x, wf, sw, dtype=torch.float16, flags=w4.LAUNCH_PDL))
    torch.cuda.synchronize()
    assert all(torch.equal(y, y0) for y in ys)
