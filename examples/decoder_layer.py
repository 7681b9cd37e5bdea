"""One decoder layer on the quantized linears, from residual to residual:
decoding token by token, and verifying a tree of drafted tokens whose accepted
branch stays in the cache.

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

    def __init__(self, hidden, heads, kv_heads, dim, inner, base=1e6, seed=0, device="cuda"):
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(n, k):
            return w4.w4_quantize_weights(torch.randn((n, k), generator=g, device=device) * k ** -0.5)

        self.qkv = [weight(n * dim, hidden) for n in (heads, kv_heads, kv_heads)]
        self.o = weight(hidden, heads * dim)
        self.gate_up = w4.w4_interleave_rows(*weight(inner, hidden), *weight(inner, hidden))
        self.down = weight(hidden, inner)
        self.norm1, self.norm2 = (1 + 0.1 * torch.randn(hidden, generator=g, device=device) for _ in range(2))
        self.freqs, self.mscale = w4.rope_frequencies(dim, base, device=device)

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


if __name__ == "__main__":
    main()
