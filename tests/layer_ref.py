"""Plain references, in 64 bits, of the decoder layer's operators, and the
bounds of what the kernels' roundings may make of them.

U(t) is the largest relative error of one rounding to type t; every bound
counts roundings of the operations in the order that the C header gives them.
"""
import numpy as np

U32, U16 = 2.0 ** -24, 2.0 ** -11
TINY16 = 2.0 ** -25  # half the spacing of binary16's subnormals


def out_round(y, dtype):
    """Bound of the last rounding of values y."""
    return np.abs(y) * U16 + TINY16 if dtype == np.float16 else np.abs(y) * U32


# -- norms --------------------------------------------------------------------

def add_norm(r, w, y, post_w, gate, alpha, beta, eps):
    """(r', x, bound of r', bound of x before their last roundings).

    A sum of N squares, all positive, in any order of at most 48 additions on
    a path (32 in a thread, two trees of 5 and the fma's own), is within 48 U32
    of exact, its root within 24 U32; division by N, the added eps, root,
    reciprocal: 4 more; so rsqrt is within 28 U32."""
    f = lambda t: None if t is None else t.astype(np.float64)  # noqa: E731
    r, w, y, post_w, gate = map(f, (r, w, y, post_w, gate))
    inv_err = 28 * U32
    u, u_err = (0.0, 0.0) if y is None else (y, 0.0)
    if post_w is not None:
        u = y / np.sqrt((y * y).mean(1, keepdims=True) + eps) * post_w
        u_err = np.abs(u) * (inv_err + 2 * U32)
    g = beta if gate is None else beta * gate
    rn = alpha * r + g * u
    e_r = np.abs(alpha * r) * 2 * U32 + np.abs(g * u) * 3 * U32 + np.abs(g) * u_err
    if w is None:
        return rn, None, e_r, None
    inv = 1 / np.sqrt((rn * rn).mean(1, keepdims=True) + eps)
    x = rn * inv * w
    norm = np.sqrt((rn * rn).sum(1, keepdims=True))
    drift = np.sqrt((e_r * e_r).sum(1, keepdims=True)) / np.where(norm > 0, norm, 1)
    e_x = np.abs(w) * inv * e_r + np.abs(x) * (inv_err + drift + 2 * U32)
    return rn, x, e_r, e_x


# -- rotary positions -----------------------------------------------------------

def rotate(x, pos, freqs, inter, mscale=1.0):
    """(y, bound): the angle within 2^-23 + 2^-52 |pos| rad, cos and sin within 2
    units of 2^-24, mscale's product, two products' and one sum's roundings."""
    x = x.astype(np.float64)
    rot = 2 * len(freqs)
    a = pos.astype(np.float64)[:, None] * freqs[None, :]
    c, s = np.cos(a)[:, None, :] * mscale, np.sin(a)[:, None, :] * mscale
    y, mag = x.copy(), np.abs(x)
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    p, q = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = p * c - q * s, q * c + p * s
    mag[..., lo] = mag[..., hi] = (np.abs(p) + np.abs(q)) * abs(mscale)
    err = np.zeros_like(y)
    ang = 2.0 ** -23 + 2.0 ** -52 * np.abs(pos.astype(np.float64))[:, None, None]
    err[..., :rot] = mag[..., :rot] * (ang + (2 + 1 + 2) * U32)
    return y, err


# -- the cache ------------------------------------------------------------------

def quantize(x, bits):
    """Codes and scale of vectors (last axis), fp32 steps as the C header gives them: bit-exact."""
    top = np.float32(127 if bits == 8 else 7)
    x = x.astype(np.float32)
    s = np.abs(x).max(-1) * (np.float32(1) / top)
    q = np.divide(x, s[..., None], out=np.zeros_like(x), where=s[..., None] > 0)
    q = np.sign(q) * np.floor(np.abs(q).astype(np.float64) + 0.5)
    return np.clip(q, -top, top).astype(np.int8), s


def pack(codes, bits):
    if bits == 8:
        return codes
    c = codes.astype(np.int32)
    return ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).astype(np.uint8)


def unpack(raw, bits):
    if bits == 8:
        return raw.astype(np.int8)
    u = raw.astype(np.int32)
    n = np.stack((u & 15, u >> 4), -1).reshape(raw.shape[:-1] + (2 * raw.shape[-1],))
    return (n - ((n & 8) << 1)).astype(np.int8)


class Paged:
    """Ragged sequences over a shuffled pool: the page table and where every
    slot lies."""

    def __init__(self, rng, tok, ctx, page, spare=2, extra_cols=1):
        self.tok, self.ctx, self.page = list(tok), list(ctx), page
        need = [-(-(t + c) // page) for t, c in zip(tok, ctx)]
        self.width = max(need) + extra_cols
        self.pages = sum(need) + spare
        perm = rng.permutation(self.pages)
        self.table = np.full((len(tok), self.width), -1, np.int32)  # unused entries: no page
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(tok)]).astype(np.int32)
        self.start = np.array(ctx, np.int32)
        self.tokens = int(self.cu[-1])

    def where(self, b, slots):
        slots = np.asarray(slots)
        return self.table[b, slots // self.page], slots % self.page

    def own(self):
        """Pages and offsets of the call's own tokens."""
        at = [self.where(b, c + np.arange(t)) for b, (t, c) in enumerate(zip(self.tok, self.ctx))]
        return np.concatenate([p for p, _ in at]), np.concatenate([o for _, o in at])


def attention(q, kc, ks, vc, vs, seen, scale):
    """One sequence and one cache head: q [rows][dim], codes [slots][dim],
    scales [slots], seen [rows][slots].  (out, bound).

    t_j = scale ks_j (q . kc_j): dim products exact in fp32 and summed with at
    most dim roundings, three more factors (one of them log2 e); its error d
    moves every weight by at most 2 d (weight and sum), exp by 2^-21 and its
    scaling by 2^-22; a weight's rounding to binary16 by U16, or, below the
    subnormals, 2^-33 of the row's largest product; sums of L terms, merged in pieces, by
    (L + 64) U32.  NaN and infinities of unseen keys touch nothing."""
    q, kc, vc = q.astype(np.float64), kc.astype(np.float64), vc.astype(np.float64)
    ks, vs = ks.astype(np.float64), vs.astype(np.float64)
    out, err = np.zeros_like(q), np.zeros_like(q)
    for i in range(len(q)):
        j = np.nonzero(seen[i])[0]
        if not len(j):
            continue
        raw = kc[j] @ q[i]
        t = scale * ks[j] * raw
        d = (q.shape[1] + 4) * U32 * np.max(np.abs(scale * ks[j]) * (np.abs(kc[j]) @ np.abs(q[i])))
        p = np.exp(t - t.max())
        p /= p.sum()
        v = vc[j] * vs[j][:, None]
        out[i] = p @ v
        mag = p @ np.abs(v)
        err[i] = mag * (2 * d + U16 + 2.0 ** -21 + 2.0 ** -22 + (len(j) + 64) * U32) + \
            len(j) * 2.0 ** -33 * np.abs(v).max() + np.abs(out[i]) * U16 + TINY16
    return out, err


def tree_masks(rng, tok, empty=()):
    """Ancestor words of random trees; rows in `empty` see no drafted token."""
    words = []
    for t in tok:
        seen = []
        for i in range(t):
            p = int(rng.integers(-1, i)) if i else -1
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
        words += seen
    words = np.array(words, dtype=np.uint64)
    for i in empty:
        words[i] = 0
    return words


def seen_of(paged, b, mask):
    """[tokens of b][slots] of what each token sees."""
    t, c = paged.tok[b], paged.ctx[b]
    s = np.ones((t, c + t), bool)
    if mask is None:
        s[:, c:] = np.tril(np.ones((t, t), bool))
    else:
        w = mask[paged.cu[b]:paged.cu[b] + t]
        s[:, c:] = (w[:, None] >> np.arange(t, dtype=np.uint64)) & np.uint64(1)
    return s
