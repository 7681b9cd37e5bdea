"""The serving loop of examples/decoder_layer.py where requests differ: prompts whose
positions are not their slots, and rows that have to wait between rows that go on."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_serving import DIM, HEADS, HIDDEN, INNER, KV, SIZES, VOCAB, ex, np_, prompts, server  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def recorded(layer):
    """The positions that each step turns its tokens at."""
    seen, step = [], layer.step

    def call(r, y, cache, batch, pos, *a, **k):
        seen.append(np_(pos))
        return step(r, y, cache, batch, pos, *a, **k)

    layer.step = call
    return seen


def test_steps_go_on_from_the_prompts_last_position(ex):  # noqa: F811
    """An image of 64 tokens takes 8 positions: what is said behind it goes on from the prompt's largest position,
    depth by depth in a drafted tree, until the request ends; a row that begins without a prompt counts from 0."""
    srv = server(ex)
    add, x, pos, axis = prompts(ex, srv)
    roots = srv.prompt(add, x, pos, axis).argmax(1).to(torch.int32)
    seen = recorded(srv.layer)
    base = np.array([n - 64 + 8 if n else 0 for n in SIZES])  # one past the largest position
    par = [-1, 0, 0, 1, 1, 2]
    depth = np.array([0, 1, 1, 2, 2, 2])
    g = torch.Generator(device="cuda").manual_seed(3)
    grown = np.zeros(4, np.int64)
    for it in range(4):
        adds = [6, 0, 6, 6]
        if it == 2:
            adds = [6, 0, -1, 6]  # the third request ends,
        if it == 3:
            adds = [6, 6, 6, 6]   # and its row and the second begin anew
            base[1:3] = grown[1:3] = 0
        live = [b for b in range(4) if adds[b] > 0]
        ids = torch.randint(0, VOCAB, (len(live), 6), generator=g, device="cuda", dtype=torch.int32)
        ids[:, 0] = roots[live]
        u = torch.full((ids.numel(),), 0.001, device="cuda")
        mask = ex.tree_mask(par).cuda().repeat(len(live))
        keep, out, count = srv.step(i32(*adds), ids.reshape(-1), mask, u, torch.full((4,), 30.0, device="cuda"))
        want = np.concatenate([base[b] + grown[b] + depth for b in live])
        assert np.array_equal(seen[-1], want), it
        grown += np_(count)
        for i, b in enumerate(live):
            roots[b] = out[6 * i + int(count[b]) - 1]
    assert ex.w4.w4a8_device_error() == 0


def test_rows_behind_one_that_waits_keep_their_own_tokens(ex):  # noqa: F811
    """The middle request has to wait for a page while the one behind it needs none, in a further part of a
    prompt and in a drafted step.  The others' results are those of the same calls in which the middle row asks for
    nothing: same shapes, hence the same bits."""
    pars = {0: [-1, 0, 0, 1, 3], 1: [-1, 0, 1, 2, 3, 4, 5, 6, 7], 2: [-1, 0, 1, 1, 0, 4, 2]}
    seen = []
    for asks in (True, False):
        layer = ex.DecoderLayer(HIDDEN, HEADS, KV, DIM, INNER, prompts=True)
        srv = ex.Server(layer, VOCAB, 3, 4, 3, page=64)
        g = torch.Generator(device="cuda").manual_seed(6)
        axis = ex.w4.rope_axes((8, 12, 12))

        def chunk(sizes, first):
            rows = [torch.randn((n, HIDDEN), generator=g, device="cuda") for n in sizes]
            pos = [torch.arange(f, f + n, dtype=torch.int32, device="cuda").expand(3, n) for n, f in zip(sizes, first)]
            if not asks and sizes[1] > 9:  # the same number of rows, of which the middle ones are behind the others
                rows, pos, sizes = [rows[0], rows[2], rows[1]], [pos[0], pos[2], pos[1]], [sizes[0], 0, sizes[2]]
            return srv.prompt(i32(*sizes), torch.cat(rows), torch.cat(pos, 1), axis)

        logits = [chunk([30, 9, 20], [0, 0, 0]), chunk([12, 90, 9], [30, 9, 20])[[0, 2]]]
        assert srv.grow.tolist() == [12, 0, 9]
        roots, took = [7, 8, 9], list(logits)
        order = (0, 1, 2) if asks else (0, 2, 1)
        srv.lens[1] += 50  # the middle row's page is nearly full
        for it in range(3):
            drafts = {b: torch.randint(0, VOCAB, (len(pars[b]),), generator=g, device="cuda", dtype=torch.int32) for b in pars}
            us = {b: torch.rand(len(pars[b]), generator=g, device="cuda") * 0.004 for b in pars}
            for b in (0, 2):
                drafts[b][0] = roots[b]
            mask = torch.cat([ex.tree_mask(pars[b]) for b in order]).cuda()
            keep, out, count = srv.step(i32(5, 9 if asks else 0, 7), torch.cat([drafts[b] for b in order]), mask,
                                        torch.cat([us[b] for b in order]), torch.full((3,), 5.0, device="cuda"))
            assert int(count[1]) == 0
            at = {0: 0, 2: 5 + 9 * asks}
            for b in (0, 2):
                own = slice(at[b], at[b] + len(pars[b]))
                roots[b] = int(out[own][int(count[b]) - 1])
                took += [keep[own], out[own]]
            if asks:
                assert bool((keep[5:14] == -1).all()) and bool((out[5:14] == -1).all())
            took += [count, srv.lens.clone()]
        batch = ex.w4.KVQBatch(i32(0, 42, 42, 71), i32(0, 0, 0), srv.pool.table)
        took += list(ex.w4.kvq_read(srv.cache, batch, 71))
        took.append(torch.tensor(roots))
        seen.append(took)
        assert ex.w4.w4a8_device_error() == 0
    for i, (a, b) in enumerate(zip(*seen)):
        assert torch.equal(a, b), i
