"""One decoder layer on the quantized linears, from residual to residual:
decoding token by token, verifying a tree of drafted tokens whose accepted
branch stays in the cache, and serving several requests: prompts with images on
the linears for many rows, then drafted steps whose pages, positions and accepted tokens
never leave the GPU.

    python examples/decoder_layer.py [--hidden 3584 --heads 28 --kv-heads 4 --inner 18944]

Random weights; the drafts and what is accepted of them are random too.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bit_weight_quantized_w4a8_gb300 as w4  # noqa: E402


class DecoderLayer:
    """norm, q/k/v, rotary positions and cache, attention, o, norm, gated MLP."""

    def __init__(self, hidden, heads, kv_heads, dim, inner, base=1e6, seed=0, device="cuda", prompts=False):
        """prompts: keeps the weights as e4m3 blocks too, for calls of more than 64 rows."""
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.f8 = []  # q, k, v, o, gate, up, down

        def weight(n, k):
            w = torch.randn((n, k), generator=g, device=device) * k ** -0.5
            if prompts:
                self.f8.append(w4.f8_quantize_weights(w))
            return w4.w4_quantize_weights(w)

        self.qkv = [weight(n * dim, hidden) for n in (heads, kv_heads, kv_heads)]
        self.o = weight(hidden, heads * dim)
        self.gate_up = w4.w4_interleave_rows(*weight(inner, hidden), *weight(inner, hidden))
        self.down = weight(hidden, inner)
        self.norm1, self.norm2 = (1 + 0.1 * torch.randn(hidden, generator=g, device=device) for _ in range(2))
        self.freqs, self.mscale = w4.rope_frequencies(dim, base, device=device)

    def prompt(self, r, y, cache, batch, pos, axis=None, trace=None):
        """step for any number of rows, on the e4m3 weights; with axis, pos is [axes][M]."""
        M = r.shape[0]
        r1, x1 = w4.add_norm(r, self.norm1, y=y)
        q, k, v = (w4.f8_linear(x1, *w).view(M, -1, self.dim) for w in self.f8[:3])
        qr = w4.kvq_write(cache, batch, k, v, Q=q, pos=pos, freqs=self.freqs, mscale=self.mscale, axis=axis)
        a = w4.kvq_attention(qr, cache, batch)
        yo = w4.f8_linear(a.view(M, -1), *self.f8[3])
        r2, x2 = w4.add_norm(r1, self.norm2, y=yo)
        h = w4.w4a8_silu_mul(*(w4.f8_linear(x2, *w) for w in self.f8[4:6]))
        yd = w4.f8_linear(h, *self.f8[6])
        if trace is not None:
            trace.update(r1=r1, x1=x1, q=q, k=k, v=v, qr=qr, a=a, yo=yo, r2=r2, x2=x2, h=h, yd=yd)
        return r2, yd

    def step(self, r, y, cache, batch, pos, mask=None, trace=None):
        """r [M][hidden] fp32 residual, y the block before's output (or None), M <=
        64 rows; pos [M] int32.  Returns the residual after attention and the MLP's
        output, which the next layer's first norm adds.  trace: a dict that takes
        the values on the way."""
        M = r.shape[0]
        r1, x1 = w4.add_norm(r, self.norm1, y=y)
        q, k, v = w4.w4a8_linear_grouped(x1, [w for w, _ in self.qkv], [s for _, s in self.qkv])
        q, k, v = (t.view(M, n, self.dim) for t, n in ((q, self.heads), (k, self.kv_heads), (v, self.kv_heads)))
        qr = w4.kvq_write(cache, batch, k, v, Q=q, pos=pos, freqs=self.freqs, mscale=self.mscale)
        a = w4.kvq_attention(qr, cache, batch, mask=mask)
        yo = w4.w4a8_linear(a.view(M, -1), *self.o)
        r2, x2 = w4.add_norm(r1, self.norm2, y=yo)
        h, _ = w4.w4a8_gate_up_silu(x2, *self.gate_up)
        yd = w4.w4a8_linear(h, *self.down)
        if trace is not None:
            trace.update(r1=r1, x1=x1, q=q, k=k, v=v, qr=qr, a=a, yo=yo, r2=r2, x2=x2, h=h, yd=yd)
        return r2, yd


def tree_mask(parents):
    """Bit words of a tree given by parents (-1: child of the last cached token):
    each token sees its ancestors and itself."""
    words = []
    for i, p in enumerate(parents):
        words.append((words[p] if p >= 0 else 0) | 1 << i)
    return torch.tensor([w - (1 << 64) if w >= 1 << 63 else w for w in words], dtype=torch.int64)


def depths(parents):
    d = []
    for p in parents:
        d.append(d[p] + 1 if p >= 0 else 0)
    return torch.tensor(d, dtype=torch.int32)


def verify_tree(layer, cache, table, context, parents, accepted, r):
    """One pass over a drafted tree on top of `context` cached tokens, then the
    accepted branch (tree indices from the root on) moved together; returns the
    outputs and the new context length."""
    n = len(parents)
    dev = r.device
    batch = w4.KVQBatch(torch.tensor([0, n], dtype=torch.int32, device=dev),
                        torch.tensor([context], dtype=torch.int32, device=dev), table)
    r2, y = layer.step(r, None, cache, batch, depths(parents).to(dev) + context, tree_mask(parents).to(dev))
    keep = torch.full((n,), -1, dtype=torch.int32)
    keep[:len(accepted)] = torch.tensor(accepted, dtype=torch.int32)
    w4.kvq_keep(cache, batch, keep.to(dev))
    return r2, y, context + len(accepted)


class Server:
    """Requests decoded together: each call plans its step from the lengths, runs the layer
    and leaves on the device what the next call goes on from."""

    def __init__(self, layer, vocab, seqs, max_pages, pages, page=64, bits=8, seed=1, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        hidden = layer.norm1.shape[0]
        self.layer, self.page = layer, page
        self.embed = torch.randn((vocab, hidden), generator=g, device=device)
        self.head = w4.w4_quantize_weights(torch.randn((vocab, hidden), generator=g, device=device) * 3 * hidden ** -0.5)
        self.norm = torch.ones(hidden, device=device)
        self.cache = w4.kvq_cache(pages, page, layer.kv_heads, layer.dim, bits, device)
        self.pool = w4.kvq_pool(seqs, max_pages, pages, device)
        # shift: the next rotary position of each request less its cached tokens (an image's tokens share positions)
        self.lens, self.grow, self.shift = (torch.zeros(seqs, dtype=torch.int32, device=device) for _ in range(3))

    def logits(self, r, y):
        return w4.w4a8_linear(w4.add_norm(r, self.norm, y=y)[1], *self.head)

    def asked(self, add, batch, seq):
        """Of each token of the batch its number among those that `add` asks for: rows that wait
        leave theirs out.  (0 for those behind the last.)"""
        ask = add.clamp_min(0)
        at = ask.cumsum(0) - ask - batch.cu[:-1]
        n = seq.shape[0]
        number = at[seq.clamp_min(0).long()] + torch.arange(n, device=seq.device)
        return torch.where(seq < 0, 0, number).clamp_(0, n - 1)

    def prompt(self, add, x, pos, axis):
        """x [tokens][hidden]: the rows of add [seqs] new tokens each (0: none, -1: the
        request ended), pos [axes][tokens].  Returns the logits of each request's last token; a
        request that had to wait (grow 0) is to ask again and has none."""
        batch, _, _, seq = w4.kvq_plan(self.pool, self.page, self.lens, add, x.shape[0], grow=self.grow)
        number = self.asked(add, batch, seq)
        x, pos = x[number], pos[:, number]
        r, y = self.layer.prompt(x, None, self.cache, batch, pos, axis)
        self.grow = (batch.cu[1:] - batch.cu[:-1]).contiguous()  # a request that had to wait has grown by nothing
        top = torch.full((add.shape[0] + 1,), -1, dtype=torch.int32, device=pos.device)  # largest positions: of no row, of each
        top.scatter_reduce_(0, seq.long() + 1, pos.amax(0), "amax")
        ended = self.shift.masked_fill(add < 0, 0)
        self.shift.copy_(torch.where(self.grow > 0, top[1:] + 1 - self.lens - self.grow, ended))
        last = (batch.cu[1:] - 1).clamp_min(0).long()
        return self.logits(r[last], y[last])

    def step(self, add, ids, mask, u, temp, trace=None):
        """ids [tokens]: of each request its last token, then its drafts, a tree by mask, as
        add asks for them.  Returns what draft_verify does, in the same places: -1, and count 0, for a
        request that had to wait."""
        batch, pos, slot, seq = w4.kvq_plan(self.pool, self.page, self.lens, add, ids.shape[0], grow=self.grow, mask=mask)
        number = self.asked(add, batch, seq)
        ids, mask, u = ids[number], mask[number], u[number]
        self.shift.masked_fill_(add < 0, 0)
        at = pos + self.shift[seq.clamp_min(0).long()]  # slots count all tokens, positions go on from the prompt's
        r, y = self.layer.step(self.embed[ids.long()], None, self.cache, batch, at, mask)
        logits = self.logits(r, y)
        keep, out, count = w4.draft_verify(logits, batch.cu, ids, u, mask=mask, temp=temp)
        if trace is not None:
            trace.update(batch=batch, pos=pos, slot=slot, seq=seq, logits=logits, before=w4.kvq_read(self.cache, batch, ids.shape[0]))
        w4.kvq_keep(self.cache, batch, keep)
        self.grow = count
        places = torch.where(seq < 0, ids.shape[0], number)  # (one more for the tokens that no row holds)
        keep, out = (t.new_full((ids.shape[0] + 1,), -1).index_copy_(0, places, t)[:-1] for t in (keep, out))
        return keep, out, count


def image_positions(rows, cols, text):
    """Positions of an image's rows x cols tokens and `text` tokens behind it on three axes
    (time, height, width): the text goes on from the largest one on all of them."""
    h, w = (t.reshape(-1) for t in torch.meshgrid(torch.arange(rows), torch.arange(cols), indexing="ij"))
    image = torch.stack((torch.zeros_like(h), h, w))
    return torch.cat((image, (max(rows, cols) + torch.arange(text)).expand(3, text)), 1).to(torch.int32)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=3584)
    ap.add_argument("--heads", type=int, default=28)
    ap.add_argument("--kv-heads", type=int, default=4)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--inner", type=int, default=18944)
    ap.add_argument("--tokens", type=int, default=64, help="tokens decoded one by one")
    ap.add_argument("--bits", type=int, default=8, choices=(8, 4), help="of the cache")
    a = ap.parse_args()
    w4.build()
    layer = DecoderLayer(a.hidden, a.heads, a.kv_heads, a.dim, a.inner)
    pages = (a.tokens + 64) // 64 + 1
    cache = w4.kvq_cache(pages, 64, a.kv_heads, a.dim, a.bits)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    batch = w4.KVQBatch(cu, start, table)
    r = torch.randn((1, a.hidden), device="cuda")
    # one captured step serves every token: positions and lengths are on the device
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    layer.step(r, None, cache, batch, pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r2, y = layer.step(r, None, cache, batch, pos)
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    t0.record()
    for _ in range(a.tokens):
        graph.replay()
        pos += 1
        start += 1
    t1.record()
    torch.cuda.synchronize()
    print("%d tokens one by one: %.1f us a token" % (a.tokens, t0.elapsed_time(t1) * 1e3 / a.tokens))
    parents = [-1, -1, 0, 0, 1, 2, 3, 5]
    rt = torch.randn((len(parents), a.hidden), device="cuda")
    r2, y, context = verify_tree(layer, cache, table, a.tokens, parents, [0, 2, 5], rt)
    assert torch.isfinite(y).all() and w4.w4a8_device_error() == 0
    print("a tree of %d tokens verified, 3 accepted: %d tokens cached" % (len(parents), context))
    # three requests: prompts with an image, then steps of a tree of drafts each
    layer = DecoderLayer(a.hidden, a.heads, a.kv_heads, a.dim, a.inner, prompts=True)
    seqs, sizes = 3, (100, 164, 72)
    server = Server(layer, 1000, seqs, 16, 48, bits=a.bits)
    add = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    pos = torch.cat([image_positions(8, 8, n - 64) for n in sizes], 1).cuda()
    pairs = a.dim // 2
    axis = w4.rope_axes((pairs - 2 * (3 * pairs // 8), 3 * pairs // 8, 3 * pairs // 8))
    logits = server.prompt(add, torch.randn((sum(sizes), a.hidden), device="cuda"), pos, axis)
    roots = logits.argmax(1)
    parents = [-1, 0, 0, 1, 1, 2]
    mask = tree_mask(parents).cuda().repeat(seqs)
    add.fill_(len(parents))
    temp = torch.full((seqs,), 0.8, device="cuda")
    said = 0
    for _ in range(4):
        ids = torch.randint(0, 1000, (seqs, len(parents)), device="cuda", dtype=torch.int32)
        ids[:, 0] = roots
        keep, out, count = server.step(add, ids.reshape(-1), mask, torch.rand(ids.numel(), device="cuda"), temp)
        said_last = out.view(seqs, -1).gather(1, (count.long() - 1).clamp_min(0)[:, None])[:, 0]
        roots = torch.where(count > 0, said_last, roots)  # a request that had to wait asks again
        said += int(count.sum())
    assert w4.w4a8_device_error() == 0
    print("%d requests served: %d tokens of prompts, %d tokens said in 4 steps" % (seqs, sum(sizes), said))


if __name__ == "__main__":
    main()
