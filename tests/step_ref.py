"""Plain references, in 64 bits, of a serving step's operators: the linear with
e4m3 blocks, the verification of drafts, the plan of pages and positions, and
rotary positions with several axes; and the bounds of what the kernels'
roundings may make of them."""
import math

import numpy as np

import layer_ref as ref

U32 = ref.U32
BLOCK = 128


# -- e4m3 ------------------------------------------------------------------------

def _e4m3_table():
    t = []
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = math.nan if c & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        t.append(-v if c & 128 else v)
    return np.array(t)


E4M3 = _e4m3_table()


def e4m3_codes(q):
    """Codes of quotients q: the nearest number, ties to the even code, at most 448."""
    v = E4M3[:127]
    a = np.minimum(np.abs(q), 448.0)
    mid = (v[1:] + v[:-1]) / 2
    i = np.searchsorted(mid, a, side="left")  # midpoints below a
    at = np.minimum(i, 125)
    i = np.where((mid[at] == a) & (i % 2 == 1) & (i < 126), i + 1, i)
    return (i | np.where(np.signbit(q), 128, 0)).astype(np.uint8)


def f8_scale(amax):
    return (amax.astype(np.float32) * np.float32(np.float32(1) / np.float32(448))).astype(np.float32)


def f8_rows(x):
    """(codes, scales [blocks][rows]) as the C header gives them: bit-exact."""
    m, k = x.shape
    codes, scales = np.zeros((m, k), np.uint8), []
    for lo in range(0, k, BLOCK):
        p = x[:, lo:lo + BLOCK].astype(np.float64)
        s = f8_scale(np.abs(p).max(1))
        scales.append(s)
        with np.errstate(divide="ignore", invalid="ignore"):
            codes[:, lo:lo + BLOCK] = np.where(s[:, None] > 0, e4m3_codes(p / s.astype(np.float64)[:, None]), 0)
    return codes, np.array(scales)


def f8_weights(w):
    """(codes, scales [row blocks][blocks])"""
    n, k = w.shape
    codes = np.zeros((n, k), np.uint8)
    scales = np.zeros((-(-n // BLOCK), -(-k // BLOCK)), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            part = w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK].astype(np.float64)
            s = f8_scale(np.abs(part).max())
            scales[i, j] = s
            if s > 0:
                codes[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = e4m3_codes(part / np.float64(s))
    return codes, scales


def f8_product(xf, sa, wf, sw):
    """(Y, bound before the last rounding).

    A block's products are exact in fp32; of its sums each of at most 128 additions
    is within a unit of the last place (2^-23, should the tensor core cut
    instead of round) of the sum of magnitudes; the scales' product and the multiply-add of a
    block take two roundings of 2^-24, the sums of all blocks (and of at most 8 pieces) one each."""
    n = wf.shape[0]
    y = np.zeros((xf.shape[0], n))
    mag = np.zeros_like(y)
    blocks = sa.shape[0]
    for j in range(blocks):
        x = E4M3[xf[:, j * BLOCK:(j + 1) * BLOCK]] * sa[j].astype(np.float64)[:, None]
        w = E4M3[wf[:, j * BLOCK:(j + 1) * BLOCK]] * np.repeat(sw[:, j].astype(np.float64), BLOCK)[:n, None]
        y += x @ w.T
        mag += np.abs(x) @ np.abs(w).T
    return y, mag * (128 * 2 * U32 + (2 + blocks + 8) * U32)


# -- rotary positions with several axes -----------------------------------------------

def rotate_axes(x, pos, axis, freqs, inter, mscale=1.0):
    """(y, bound): pair i as layer_ref.rotate turns it at pos[axis[i]]."""
    y, err = x.astype(np.float64), np.zeros(x.shape)
    half = len(freqs)
    for a in sorted(set(axis)):
        ya, ea = ref.rotate(x, pos[a], freqs, inter, mscale)
        for i in range(half):
            if axis[i] == a:
                for c in ((2 * i, 2 * i + 1) if inter else (i, i + half)):
                    y[..., c], err[..., c] = ya[..., c], ea[..., c]
    return y, err


# -- verification of drafts --------------------------------------------------------

def parents(n, mask):
    """Parent of each token of a sequence, -1: none."""
    if mask is None:
        return [i - 1 for i in range(n)]
    return [int(m & ((1 << i) - 1)).bit_length() - 1 for i, m in enumerate(mask)]


def distribution(row, temp):
    """Target's distribution of a row; None where it has none."""
    x = row.astype(np.float64)
    if np.isnan(x).any() or x.max() == math.inf or x.max() == -math.inf:
        return None
    if not temp >= 2.0 ** -20:
        p = np.zeros_like(x)
        p[int(np.argmax(x))] = 1
        return p
    with np.errstate(under="ignore"):
        e = np.exp((x - x.max()) / temp)
    return e / e.sum()


def verify_seq(rows, ids, u, mask=None, q=None, temp=1.0):
    """(kept places, tokens said) of one sequence, from the formulas."""
    n = len(rows)
    par = parents(n, mask)
    greedy = not temp >= 2.0 ** -20
    kept, said, node, p = [0], [], 0, distribution(rows[0], temp)
    i = 1
    while i < n:
        if par[i] == node and p is not None:
            x = int(ids[i])
            inside = 0 <= x < rows.shape[1]
            px = p[x] if inside else 0.0
            if greedy:
                yes = px > 0
            else:
                lim = float(u[i]) * (1.0 if q is None else float(q[node, x]) if inside else 0.0)
                yes = inside and lim < px
            if yes:
                kept.append(i)
                said.append(x)
                node, p = i, distribution(rows[i], temp)
            elif not greedy:
                if q is None:
                    p = p.copy()
                    if inside:
                        p[x] = 0
                else:
                    p = np.maximum(p - q[node].astype(np.float64), 0)
                total = p.sum()
                p = p / total if total > 0 else distribution(rows[node], temp)
        i += 1
    if p is None:
        said.append(-1)
    else:
        c = np.cumsum(p)
        said.append(int(np.argmax(c > float(u[0]) * c[-1])))
    return kept, said


def verify(logits, cu, ids, u, mask=None, q=None, temp=None, fill=-7):
    """(keep, out, count) of a batch; places that no sequence holds keep `fill`."""
    n = len(logits)
    keep, out = np.full(n, fill, np.int32), np.full(n, fill, np.int32)
    count = []
    for b in range(len(cu) - 1):
        lo, hi = int(cu[b]), int(cu[b + 1])
        if hi == lo:
            count.append(0)
            continue
        sl = slice(lo, hi)
        keep[sl] = out[sl] = -1
        k, s = verify_seq(logits[sl], ids[sl], u[sl], None if mask is None else [int(m) for m in mask[sl].view(np.uint64)],
                          None if q is None else q[sl], 1.0 if temp is None else float(temp[b]))
        keep[lo:lo + len(k)], out[lo:lo + len(s)] = k, s
        count.append(len(k))
    return keep, out, np.array(count, np.int32)


# -- the plan of a step -----------------------------------------------------------

class Pool:
    """kvq_pool_t and lens on the host, request by request."""

    def __init__(self, table, held, stack, top, lens, page):
        self.table, self.held, self.stack = table.copy(), held.copy(), stack.copy()
        self.top, self.lens, self.page = int(top), lens.astype(np.int64), page

    def plan(self, add, tokens, grow=None, mask=None):
        """(cu, pos, slot, seq)"""
        seqs, width = self.table.shape
        if grow is not None:
            self.lens += grow
        back = []
        for b in range(seqs):
            if add[b] < 0:
                back += list(self.table[b, :self.held[b]])
                self.held[b] = self.lens[b] = 0
        for p in reversed(back):  # the first of all on top
            self.stack[self.top] = p
            self.top += 1
        free, asked_pages, asked_tokens = self.top, 0, 0
        cu, pos, slot, seq = [0], [], [], []
        for b in range(seqs):
            n = max(int(add[b]), 0)
            want = -(-(int(self.lens[b]) + n) // self.page)
            need = max(want - int(self.held[b]), 0) if n else 0
            ok = n > 0 and want <= width
            if ok:
                asked_pages += need
                asked_tokens += n
                ok = (need == 0 or asked_pages <= free) and asked_tokens <= tokens
            if ok:
                for _ in range(need):
                    self.top -= 1
                    self.table[b, self.held[b]] = self.stack[self.top]
                    self.held[b] += 1
                for i in range(n):
                    s = int(self.lens[b]) + i
                    pos.append(s if mask is None else int(self.lens[b]) + bin(int(mask[len(pos)]) & (1 << 64) - 1).count("1") - 1)
                    slot.append(int(self.table[b, s // self.page]) * self.page + s % self.page)
                    seq.append(b)
            cu.append(len(pos))
        rest = tokens - len(pos)
        return (np.array(cu, np.int32), np.array(pos + [0] * rest, np.int32), np.array(slot + [-1] * rest, np.int64),
                np.array(seq + [-1] * rest, np.int32))
