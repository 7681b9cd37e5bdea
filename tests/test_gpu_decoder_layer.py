"""The decoder layer of examples/decoder_layer.py: every stage against the plain
reference or the oracle on the values that the stage before gave, token by token
and over a tree; and a tree's accepted branch against the same tokens decoded one by one."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref  # noqa: E402
import oracle  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIDDEN, HEADS, KV, DIM, INNER = 512, 8, 2, 64, 1024


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


def stages(ex, layer, t, r, cache, table, starts, tok, pos, mask, bits):
    """Checks of one step's trace."""
    orc = oracle.load()
    M = r.shape[0]
    want_r, want_x, e_r, e_x = ref.add_norm(np_(r), np_(layer.norm1), None, None, None, 1.0, 1.0, 1e-6)
    assert np.all(np.abs(np_(t["r1"]) - want_r) <= e_r + ref.out_round(want_r, np.float32))
    assert np.all(np.abs(np_(t["x1"]).astype(np.float64) - want_x) <= e_x + ref.out_round(want_x, np.float16))
    for name, (w, s) in zip("qkv", layer.qkv):
        assert np.array_equal(np_(t[name]).reshape(M, -1), orc.w4a8_linear(np_(t["x1"]), np_(w), np_(s))[0])
    want, err = ref.rotate(np_(t["q"]), np_(pos), np_(layer.freqs), False)
    assert np.all(np.abs(np_(t["qr"]).astype(np.float64) - want) <= err + ref.out_round(want, np.float16))
    # attention over what the cache holds, of which the call's keys are the rotated ones' codes
    k, v, ks, vs = (np_(c) for c in cache)
    page = k.shape[2]
    kw, ke = ref.rotate(np_(t["k"]), np_(pos), np_(layer.freqs), False)
    top = 127 if bits == 8 else 7
    at = 0
    for b, n in enumerate(tok):
        if n == 0:
            continue
        slots = np.arange(starts[b] + n)
        p, o = table[b, slots // page], slots % page
        own = slice(at, at + n)
        codes, sc = ref.unpack(k[p[-n:], :, o[-n:]], bits), ks[p[-n:], :, o[-n:]].astype(np.float64)[..., None]
        assert np.all(np.abs(codes * sc - kw[own]) <= sc * (0.5 + top * 4 * ref.U32) + ke[own] + ke[own].max(-1, keepdims=True))
        seen = np.ones((n, starts[b] + n), bool)
        if mask is None:
            seen[:, starts[b]:] = np.tril(np.ones((n, n), bool))
        else:
            words = np_(mask)[own].view(np.uint64)
            seen[:, starts[b]:] = (words[:, None] >> np.arange(n, dtype=np.uint64)) & np.uint64(1)
        G = HEADS // KV
        for h in range(KV):
            q = np_(t["qr"])[own, h * G:(h + 1) * G].reshape(n * G, DIM)
            want, err = ref.attention(q, ref.unpack(k[p, h, o], bits), ks[p, h, o], ref.unpack(v[p, h, o], bits), vs[p, h, o],
                                      np.repeat(seen, G, 0), DIM ** -0.5)
            got = np_(t["a"])[own, h * G:(h + 1) * G].reshape(n * G, DIM)
            assert np.all(np.abs(got - want) <= err)
        at += n
    assert np.array_equal(np_(t["yo"]), orc.w4a8_linear(np_(t["a"]).reshape(M, -1), *(np_(x) for x in layer.o))[0])
    want_r, want_x, e_r, e_x = ref.add_norm(np_(t["r1"]), np_(layer.norm2), np_(t["yo"]), None, None, 1.0, 1.0, 1e-6)
    assert np.all(np.abs(np_(t["r2"]) - want_r) <= e_r + ref.out_round(want_r, np.float32))
    assert np.all(np.abs(np_(t["x2"]).astype(np.float64) - want_x) <= e_x + ref.out_round(want_x, np.float16))
    assert np.array_equal(np_(t["yd"]), orc.w4a8_linear(np_(t["h"]), *(np_(x) for x in layer.down))[0])


@pytest.mark.parametrize("bits", [8, 4])
def test_layer_stage_by_stage(ex, bits):
    w4 = ex.w4
    layer = ex.DecoderLayer(HIDDEN, HEADS, KV, DIM, INNER)
    rng = np.random.default_rng(bits)
    perm = rng.permutation(12).astype(np.int32)
    table = np.stack([perm[:6], perm[6:]])
    cache = w4.kvq_cache(12, 16, KV, DIM, bits)
    td = torch.from_numpy(table).cuda()
    lens = [0, 0]
    # two sequences: prompts of 20 and 3 tokens (causal), then single tokens, then trees
    for tok, parents in (((20, 3), None), ((1, 1), None), ((8, 5), True), ((1, 0), None)):
        n = sum(tok)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(tok)]), dtype=torch.int32).cuda()
        start = torch.tensor(lens, dtype=torch.int32).cuda()
        batch = w4.KVQBatch(cu, start, td)
        mask = None
        if parents:
            trees = [[int(rng.integers(-1, i)) if i else -1 for i in range(t)] for t in tok]
            mask = torch.cat([ex.tree_mask(t) for t in trees]).cuda()
            pos = torch.cat([ex.depths(t) + l for t, l in zip(trees, lens)]).to(torch.int32).cuda()
        else:
            pos = torch.cat([torch.arange(t, dtype=torch.int32) + l for t, l in zip(tok, lens)]).cuda()
        r = torch.from_numpy(rng.standard_normal((n, HIDDEN)).astype(np.float32)).cuda()
        trace = {}
        layer.step(r, None, cache, batch, pos, mask, trace)
        stages(ex, layer, trace, r, cache, table, lens, [t for t in tok], pos, mask, bits)
        lens = [l + t for l, t in zip(lens, tok)]
    assert w4.w4a8_device_error() == 0


def test_accepted_branch_is_what_decoding_would_have_cached(ex):
    """After verification the cache holds, slot by slot, the codes that the
    accepted tokens' own decoding writes: the layer's keys depend on the token and
    its position alone."""
    w4 = ex.w4
    layer = ex.DecoderLayer(HIDDEN, HEADS, KV, DIM, INNER)
    parents, accepted = [-1, 0, 0, 1, 2, 4, 4], [0, 2, 4, 6]
    table = torch.arange(3, dtype=torch.int32).view(1, 3).cuda()
    g = torch.Generator().manual_seed(3)
    first = torch.randn((9, HIDDEN), generator=g).cuda()
    drafted = torch.randn((len(parents), HIDDEN), generator=g).cuda()
    caches = [w4.kvq_cache(3, 16, KV, DIM) for _ in range(2)]
    for c in caches:
        batch = w4.KVQBatch(torch.tensor([0, 9], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda(), table)
        layer.step(first, None, c, batch, torch.arange(9, dtype=torch.int32).cuda())
    _, _, context = ex.verify_tree(layer, caches[0], table, 9, parents, accepted, drafted)
    assert context == 13
    for i, a in enumerate(accepted):  # the same tokens one by one
        batch = w4.KVQBatch(torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([9 + i], dtype=torch.int32).cuda(), table)
        layer.step(drafted[a:a + 1], None, caches[1], batch, torch.tensor([9 + i], dtype=torch.int32).cuda())
    for x, y in zip(*caches):
        assert torch.equal(x[:, :, :13], y[:, :, :13])  # 13 slots, all in the first page
    assert w4.w4a8_device_error() == 0
