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
