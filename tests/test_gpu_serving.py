"""The serving loop of examples/decoder_layer.py: plan, layer, verification and the
kept branch as they follow one another, each against its reference on what the one before
gave; and the loop captured into a graph against the same calls made one by one."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref  # noqa: E402
import step_ref as sref  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIDDEN, HEADS, KV, DIM, INNER, VOCAB = 512, 8, 2, 64, 1024, 300
SIZES = (100, 0, 164, 72)  # a row without a request


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.w4.build()
    return m


def np_(t):
    return t.cpu().numpy()


def server(ex, bits=8):
    layer = ex.DecoderLayer(HIDDEN, HEADS, KV, DIM, INNER, prompts=True)
    return ex.Server(layer, VOCAB, len(SIZES), 6, 24, page=64, bits=bits)


def prompts(ex, srv):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    add = torch.tensor(SIZES, dtype=torch.int32, device="cuda")
    pos = torch.cat([ex.image_positions(8, 8, n - 64) for n in SIZES if n], 1).cuda()
    axis = ex.w4.rope_axes((8, 12, 12), cycled=True)
    x = torch.randn((sum(SIZES), HIDDEN), generator=g, device="cuda")
    return add, x, pos, axis


def test_prompt_stages(ex):
    """A prompt with images through the layer: linears with e4m3 blocks, positions of three axes."""
    srv = server(ex)
    add, x, pos, axis = prompts(ex, srv)
    batch, p, slot, _ = ex.w4.kvq_plan(srv.pool, srv.page, srv.lens, add, x.shape[0])
    t = {}
    srv.layer.prompt(x, None, srv.cache, batch, pos, axis, trace=t)
    f = np_(srv.layer.freqs)
    for name, w in zip("qkv", srv.layer.f8):
        xf, sa = sref.f8_rows(np_(t["x1"]))
        want, err = sref.f8_product(xf, sa, np_(w[0]), np_(w[1]))
        assert np.all(np.abs(np_(t[name]).reshape(want.shape) - want) <= err + ref.out_round(want, np.float32))
    want, err = sref.rotate_axes(np_(t["q"]), np_(pos), list(axis), f, False)
    assert np.all(np.abs(np_(t["qr"]).astype(np.float64) - want) <= err + ref.out_round(want, np.float16))
    # the cache's rows at the plan's slots hold the turned keys
    want, err = sref.rotate_axes(np_(t["k"]), np_(pos), list(axis), f, False)
    codes, scale = np_(srv.cache.k), np_(srv.cache.ks)
    s = np_(slot)[:, None]
    page, at, h = s // srv.page, s % srv.page, np.arange(KV)[None, :]
    sc = scale[page, h, at].astype(np.float64)[..., None]
    off = np.abs(codes[page, h, at] * sc - want)
    assert np.all(off <= sc * (0.5 + 127 * 4 * ref.U32) + err + err.max(-1, keepdims=True))
    for name, w, src in (("yo", srv.layer.f8[3], np_(t["a"]).reshape(x.shape[0], -1)), ("yd", srv.layer.f8[6], np_(t["h"]))):
        xf, sa = sref.f8_rows(src)
        want, err = sref.f8_product(xf, sa, np_(w[0]), np_(w[1]))
        assert np.all(np.abs(np_(t[name]) - want) <= err + ref.out_round(want, np.float32))
    assert ex.w4.w4a8_device_error() == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_steps_of_a_run(ex, bits):
    """Prompts, then drafted steps, a request that ends and one that comes: every stage's result."""
    rng = np.random.default_rng(bits)
    srv = server(ex, bits)
    host = sref.Pool(np_(srv.pool.table), np_(srv.pool.held), np_(srv.pool.stack), 24, np.zeros(4, np.int64), 64)
    add, x, pos, axis = prompts(ex, srv)
    roots = np_(srv.prompt(add, x, pos, axis).argmax(1)).astype(np.int32)
    host.plan(list(SIZES), x.shape[0])
    grow = np.array(SIZES)
    taken = 0
    for it in range(5):
        adds = np.array([9, 0, 7, 12], np.int32)
        if it == 2:
            adds[2] = -1   # one request ends ...
        if it >= 3:
            adds[1], adds[2] = 5, 0   # ... a row without a prompt begins with its first token
        n = int(np.maximum(adds, 0).sum())
        words = []
        for m in np.maximum(adds, 0):
            par = [-1] + [int(rng.integers(0, i)) for i in range(1, m)]
            words += list(np_(ex.tree_mask(par[:m])))
        mask = np.array(words, np.int64)
        ids = rng.integers(0, VOCAB, n).astype(np.int32)
        cu = np.concatenate([[0], np.cumsum(np.maximum(adds, 0))])
        ids[cu[:-1][adds > 0]] = roots[adds > 0]
        u = (rng.random(n) * 0.004).astype(np.float32)  # as small as 1 / VOCAB: some of the random drafts are taken
        u[cu[:-1][adds > 0]] = rng.random(int((adds > 0).sum()))
        temp = np.array([0.0, 0.7, 1.0, 30.0], np.float32)
        d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        t = {}
        got = [np_(a) for a in srv.step(d(adds), d(ids), d(mask), d(u), d(temp), trace=t)]
        want = host.plan(adds, n, grow, mask)
        for a, w in zip((t["batch"].cu, t["pos"], t["slot"], t["seq"]), want):
            assert np.array_equal(np_(a), w)
        assert np.array_equal(np_(srv.lens), host.lens) and int(srv.pool.top[0]) == host.top
        ver = sref.verify(np_(t["logits"]), cu, ids, u, mask, None, temp)
        for a, w in zip(got, ver):
            assert np.array_equal(a, w)
        # the kept tokens' keys and values lie together
        after = ex.w4.kvq_read(srv.cache, t["batch"], n)
        for b in range(4):
            for i in range(got[2][b]):
                for x0, x1 in zip(t["before"], after):
                    assert torch.equal(x1[cu[b] + i], x0[cu[b] + got[0][cu[b] + i]])
        grow = got[2]
        taken += int(np.maximum(grow - 1, 0).sum())
        for b in np.flatnonzero(adds > 0):
            roots[b] = got[1][cu[b] + grow[b] - 1]
    assert taken > 0 and ex.w4.w4a8_device_error() == 0


def test_a_captured_step_follows_the_lengths(ex):
    """One captured step replayed: the tokens, lengths and pages of the same steps made one by one."""
    runs = []
    for captured in (False, True):
        srv = server(ex)
        add, x, pos, axis = prompts(ex, srv)
        roots = srv.prompt(add, x, pos, axis).argmax(1).to(torch.int32)
        seqs, par = len(SIZES), [-1, 0, 0, 1, 1, 2]
        add = torch.tensor([len(par) if n else 0 for n in SIZES], dtype=torch.int32, device="cuda")
        live = [b for b, n in enumerate(SIZES) if n]
        mask = ex.tree_mask(par).cuda().repeat(len(live))
        g = torch.Generator(device="cuda")
        g.manual_seed(9)
        tokens = len(live) * len(par)
        ids = torch.zeros(tokens, dtype=torch.int32, device="cuda")
        u = torch.zeros(tokens, device="cuda")
        temp = torch.full((seqs,), 5.0, device="cuda")
        grow = srv.grow.clone()
        srv.grow = grow
        out = []

        def one():
            keep, said, count = srv.step(add, ids, mask, u, temp)
            grow.copy_(count)
            srv.grow = grow
            return said, count

        graph = None
        if captured:
            # what a step changes is put back after the run that warms it up
            keepers = [srv.lens, grow, *srv.pool, *srv.cache]
            saved = [k.clone() for k in keepers]
            one()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                said, count = one()
            for k, s in zip(keepers, saved):
                k.copy_(s)
        root = roots[live]
        for _ in range(6):
            ids.copy_(torch.randint(0, VOCAB, (tokens,), generator=g, device="cuda", dtype=torch.int32))
            ids.view(len(live), -1)[:, 0] = root
            u.copy_(torch.rand(tokens, generator=g, device="cuda") * 0.004)
            if graph is None:
                said, count = one()
            else:
                graph.replay()
            root = said.view(len(live), -1).gather(1, (count[live].long() - 1)[:, None])[:, 0]
            out += [said.clone(), count.clone(), srv.lens.clone()]
        out += [srv.pool.held.clone(), srv.pool.top.clone()]
        runs.append(out)
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    assert ex.w4.w4a8_device_error() == 0
