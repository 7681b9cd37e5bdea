"""The decoder layer's entry points without a GPU: refusals that return before
any CUDA call, the rotary frequencies, the fixed-point angle, and the cache's
look-ups with tables that hold anything."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bit_weight_quantized_w4a8_gb300 as w4  # noqa: E402
from bit_weight_quantized_w4a8_gb300 import _binding as B  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # a fake, aligned address: never dereferenced (checks fail first)


@pytest.fixture(scope="module")
def L():
    w4.build()
    return w4.lib()


def cache(**kw):
    d = dict(k=P, v=P, ks=P, vs=P, pages=4, page=64, heads=2, dim=128, bits=8)
    d.update(kw)
    return ctypes.byref(B._Cache(**d))


def batch(**kw):
    d = dict(cu=P, start=P, table=P, seqs=1, tokens=4, max_pages=2)
    d.update(kw)
    return ctypes.byref(B._Batch(**d))


NORM = dict(r=P, r_type=0, y=P, y_type=0, post_w=None, gate=None, ld_gate=0, w=P, M=1, N=64, alpha=1.0, beta=1.0,
            eps=1e-6, r_out=P, X=P, Xq=None, sa=None, flags=0)


@pytest.mark.parametrize("change,status", [
    (dict(r=None), B.ERR_NULL), (dict(w=None), B.ERR_NULL), (dict(Xq=P), B.ERR_NULL), (dict(sa=P), B.ERR_NULL),
    (dict(r_out=None, X=None), B.ERR_NULL), (dict(r_type=2), B.ERR_SHAPE), (dict(y_type=-1), B.ERR_SHAPE),
    (dict(M=0), B.ERR_SHAPE), (dict(M=1 << 31), B.ERR_SHAPE), (dict(N=0), B.ERR_SHAPE), (dict(N=32769), B.ERR_SHAPE),
    (dict(gate=P, ld_gate=63), B.ERR_SHAPE), (dict(alpha=math.inf), B.ERR_SHAPE), (dict(beta=math.nan), B.ERR_SHAPE),
    (dict(eps=-1e-6), B.ERR_SHAPE), (dict(N=63, Xq=P, sa=P), B.ERR_SHAPE), (dict(flags=2), B.ERR_SHAPE),
    (dict(r=P + 2), B.ERR_ALIGN), (dict(y=P + 1, y_type=1), B.ERR_ALIGN), (dict(w=P + 2), B.ERR_ALIGN),
    (dict(X=P + 1), B.ERR_ALIGN)])
def test_add_norm_refusals(L, change, status):
    a = dict(NORM)
    a.update(change)
    assert L.add_norm(*a.values(), None) == status
    assert L.w4a8_last_error().startswith(b"add_norm")


ROPE = dict(X=P, x_type=0, ld_x=256, tokens=4, heads=2, dim=128, pos=P, freqs=P, rot=64, interleaved=0, mscale=1.0, Y=P,
            y_type=0, ld_y=256, flags=0)


@pytest.mark.parametrize("change,status", [
    (dict(X=None), B.ERR_NULL), (dict(Y=None), B.ERR_NULL), (dict(pos=None), B.ERR_NULL), (dict(freqs=None), B.ERR_NULL),
    (dict(x_type=7), B.ERR_SHAPE), (dict(tokens=0), B.ERR_SHAPE), (dict(heads=0), B.ERR_SHAPE),
    (dict(dim=96), B.ERR_SHAPE), (dict(rot=12), B.ERR_SHAPE), (dict(rot=136), B.ERR_SHAPE), (dict(rot=0), B.ERR_SHAPE),
    (dict(ld_x=255), B.ERR_SHAPE), (dict(ld_x=258), B.ERR_SHAPE), (dict(y_type=1), B.ERR_SHAPE),  # in place, two types
    (dict(mscale=math.inf), B.ERR_SHAPE), (dict(flags=4), B.ERR_SHAPE), (dict(X=P + 8, Y=P + 8), B.ERR_ALIGN),
    (dict(pos=P + 2), B.ERR_ALIGN), (dict(freqs=P + 4), B.ERR_ALIGN)])
def test_rope_rotate_refusals(L, change, status):
    a = dict(ROPE)
    a.update(change)
    assert L.rope_rotate(*a.values(), None) == status
    assert L.w4a8_last_error().startswith(b"rope_rotate")


BAD_CACHE = [(dict(k=None), B.ERR_NULL), (dict(vs=None), B.ERR_NULL), (dict(pages=0), B.ERR_SHAPE),
             (dict(page=48), B.ERR_SHAPE), (dict(page=8), B.ERR_SHAPE), (dict(page=512), B.ERR_SHAPE),
             (dict(heads=0), B.ERR_SHAPE), (dict(dim=80), B.ERR_SHAPE), (dict(bits=5), B.ERR_SHAPE),
             (dict(k=P + 8), B.ERR_ALIGN), (dict(ks=P + 2), B.ERR_ALIGN)]
BAD_BATCH = [(dict(cu=None), B.ERR_NULL), (dict(table=None), B.ERR_NULL), (dict(seqs=0), B.ERR_SHAPE),
             (dict(seqs=65537), B.ERR_SHAPE), (dict(tokens=0), B.ERR_SHAPE), (dict(max_pages=0), B.ERR_SHAPE),
             (dict(start=P + 2), B.ERR_ALIGN)]


def calls(L, c, b):
    yield L.kvq_write(c, b, P, 256, P, 256, None, 0, 0, 0, None, None, 0, 0, 1.0, None, 0, None)
    yield L.kvq_read(c, b, P, P, 1, 0, None)
    yield L.kvq_keep(c, b, P, 0, None)
    yield L.kvq_attention(c, b, P, 4, None, 0.1, P, P, 1 << 40, 0, None)


@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_cache_refusals(L, change, status):
    assert all(st == status for st in calls(L, cache(**change), batch()))
    assert L.kvq_attention_workspace_bytes(cache(**change), batch(), 4) == 0


@pytest.mark.parametrize("change,status", BAD_BATCH)
def test_batch_refusals(L, change, status):
    assert all(st == status for st in calls(L, cache(), batch(**change)))
    assert L.kvq_attention_workspace_bytes(cache(), batch(**change), 4) == 0


def test_null_structs(L):
    assert all(st == B.ERR_NULL for st in calls(L, None, batch()))
    assert all(st == B.ERR_NULL for st in calls(L, cache(), None))


def test_kvq_write_refusals(L):
    def call(K=P, ld_k=256, V=P, ld_v=256, Q=P, ld_q=512, hq=4, t=0, pos=P, freqs=P, rot=128, out=P, flags=0):
        return L.kvq_write(cache(), batch(), K, ld_k, V, ld_v, Q, ld_q, hq, t, pos, freqs, rot, 0, 1.0, out, flags, None)
    assert call(K=None) == B.ERR_NULL and call(V=None) == B.ERR_NULL
    assert call(out=None) == B.ERR_NULL and call(Q=None) == B.ERR_NULL  # together or not at all
    assert call(pos=None) == B.ERR_NULL
    assert call(ld_k=252) == B.ERR_SHAPE and call(ld_v=257) == B.ERR_SHAPE and call(ld_q=256) == B.ERR_SHAPE
    assert call(hq=0) == B.ERR_SHAPE and call(t=3) == B.ERR_SHAPE and call(rot=130) == B.ERR_SHAPE
    assert call(flags=8) == B.ERR_SHAPE
    assert call(K=P + 8) == B.ERR_ALIGN and call(out=P + 4) == B.ERR_ALIGN


def test_kvq_read_and_keep_refusals(L):
    assert L.kvq_read(cache(), batch(), None, P, 1, 0, None) == B.ERR_NULL
    assert L.kvq_read(cache(), batch(), P, P, 2, 0, None) == B.ERR_SHAPE
    assert L.kvq_read(cache(), batch(), P, P + 8, 1, 0, None) == B.ERR_ALIGN
    assert L.kvq_keep(cache(), batch(), None, 0, None) == B.ERR_NULL
    assert L.kvq_keep(cache(), batch(), P + 2, 0, None) == B.ERR_ALIGN
    assert L.kvq_keep(cache(), batch(), P, 16, None) == B.ERR_SHAPE


def test_kvq_attention_refusals(L):
    def call(Q=P, hq=4, mask=None, scale=0.1, out=P, flags=0):
        return L.kvq_attention(cache(), batch(), Q, hq, mask, scale, out, P, 1 << 40, flags, None)
    assert call(Q=None) == B.ERR_NULL and call(out=None) == B.ERR_NULL
    assert call(hq=3) == B.ERR_SHAPE and call(hq=1) == B.ERR_SHAPE and call(hq=4096) == B.ERR_SHAPE
    assert call(scale=math.nan) == B.ERR_SHAPE and call(flags=32) == B.ERR_SHAPE
    assert call(Q=P + 8) == B.ERR_ALIGN and call(out=P + 8) == B.ERR_ALIGN and call(mask=P + 4) == B.ERR_ALIGN


def test_binding_refuses_cpu_tensors_and_wrong_types(L):
    f = torch.zeros
    with pytest.raises(ValueError):
        w4.add_norm(f(2, 8), f(8))
    with pytest.raises(TypeError):
        w4.add_norm(f(2, 8, dtype=torch.float64), f(8))
    with pytest.raises(ValueError):
        w4.rope_rotate(f(2, 2, 64), f(2, dtype=torch.int32), f(32, dtype=torch.float64))
    c = w4.kvq_cache(2, 16, 2, 64, device="cpu")
    b = w4.KVQBatch(f(2, dtype=torch.int32), f(1, dtype=torch.int32), f(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        w4.kvq_write(c, b, f(2, 2, 64), f(2, 2, 64))
    with pytest.raises(ValueError):
        w4.kvq_read(c, b, 2)
    with pytest.raises(ValueError):
        w4.kvq_attention(f(2, 2, 64, dtype=torch.float16), c, b)
    with pytest.raises(ValueError):
        w4.kvq_cache(2, 16, 2, 64, bits=6, device="cpu")


# -- rotary frequencies -----------------------------------------------------------

def test_frequencies_plain_linear_ntk(L):
    i = np.arange(32)
    f, m = w4.rope_frequencies(64, 10000.0)
    assert m == 1.0 and np.allclose(f.numpy(), 10000.0 ** (-i / 32), rtol=1e-14, atol=0)
    g, _ = w4.rope_frequencies(64, 10000.0, "linear", 8.0)
    assert np.allclose(g.numpy(), f.numpy() / 8, rtol=1e-14, atol=0)
    h, _ = w4.rope_frequencies(64, 10000.0, "ntk", 8.0)
    assert h[0] == 1.0 and np.isclose(float(h[-1]), float(f[-1]) / 8, rtol=1e-12)


def test_frequencies_by_parts(L):
    f = w4.rope_frequencies(128, 1e6)[0].numpy()
    y, m = w4.rope_frequencies(128, 1e6, "yarn", 4.0, old_ctx=32768, low=1.0, high=32.0)
    assert m == np.float32(0.1 * math.log(4.0) + 1.0)
    turns = 32768 * f / (2 * math.pi)
    ratio = f / y.numpy()
    assert np.all(ratio[turns > 40] == 1.0) and np.allclose(ratio[turns < 0.8], 4.0, rtol=1e-12)
    assert np.all(np.diff(ratio) >= -1e-12)  # between the two it only falls
    z = w4.rope_frequencies(128, 5e5, "bands", 8.0, old_ctx=8192, low=1.0, high=4.0)[0].numpy()
    f = w4.rope_frequencies(128, 5e5)[0].numpy()
    turns = 8192 * f / (2 * math.pi)
    keep = np.clip((turns - 1) / 3, 0, 1)
    assert np.allclose(z, f / 8 * (1 - keep) + f * keep, rtol=1e-13, atol=0)


def test_frequency_refusals(L):
    for kw in (dict(rot=12), dict(rot=0), dict(rot=264), dict(base=1.0), dict(base=math.nan), dict(factor=0.5),
               dict(scaling="yarn"), dict(scaling="bands", old_ctx=100, low=2.0, high=1.0),
               dict(scaling="yarn", old_ctx=100, low=0.0, high=1.0)):
        with pytest.raises(w4.W4A8Error):
            w4.rope_frequencies(**{**dict(rot=64), **kw})
    with pytest.raises(ValueError):
        w4.rope_frequencies(64, scaling="other")


def test_fixed_point_angle():
    """pos * F mod 2^64 with F = the 64-bit fraction of a turn, its top 32 bits
    as a signed number of 2^-32 turns: within 2^-23 + 2^-52 |pos| rad of pos *
    freq, far positions and negative ones included.  The exact angle is
    taken with integers of any size."""
    from fractions import Fraction
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    inv2pi = 0.15915494309189533577
    rng = np.random.default_rng(7)
    for freq in [1.0, 0.7, 1e-2, 1e-6] + list(rng.random(20)):
        t = freq * inv2pi
        F = int((t - math.floor(t)) * 18446744073709551616.0)
        for pos in [0, 1, -1, 4095, 131071, -131071, 10 ** 6, 2 ** 31 - 1, -2 ** 31]:
            top = ((F * pos) & (2 ** 64 - 1)) >> 32
            top = top - 2 ** 32 if top >= 2 ** 31 else top
            half_turns = Fraction(float(np.float32(top) * np.float32(2.0 ** -31)))
            exact = Fraction(freq) * pos / pi  # half turns
            d = (half_turns - exact) % 2
            d = min(d, 2 - d) * pi
            assert float(d) <= 2.0 ** -23 + 2.0 ** -52 * abs(pos), (freq, pos, float(d))


# -- the cache's look-ups ------------------------------------------------------------

@pytest.fixture(scope="module")
def index(tmp_path_factory):
    d = tmp_path_factory.mktemp("kvq")
    src = d / "index.cpp"
    src.write_text('#include "%s"\n' % os.path.join(ROOT, "bit_weight_quantized_w4a8_gb300", "csrc", "kvq_index.h") + """
extern "C" int find_seq(const int32_t* cu, int seqs, int i) { return w4a8::kvq_find_seq(cu, seqs, i); }
extern "C" int64_t slot_row(const int32_t* t, int64_t mp, int64_t pages, int shift, int b, int64_t s) {
    return w4a8::kvq_slot_row(t, mp, pages, shift, b, s); }
extern "C" int seq(const int32_t* cu, const int32_t* st, int b, int64_t tokens, int64_t mp, int shift) {
    const w4a8::KvqSeq q = w4a8::kvq_seq(cu, st, b, tokens, mp, shift);
    return q.ok ? q.count : -1 - q.count; }
""")
    so = d / "index.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-shared",
                    "-fPIC", "-o", str(so), str(src)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.slot_row.restype = ctypes.c_int64
    lib.slot_row.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int64]
    lib.find_seq.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int]
    lib.seq.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    return lib


def test_find_seq(index):
    rng = np.random.default_rng(1)
    for _ in range(50):
        tok = rng.integers(0, 5, rng.integers(1, 40))
        cu = np.concatenate([[0], np.cumsum(tok)]).astype(np.int32)
        want = np.repeat(np.arange(len(tok)), tok)
        got = [index.find_seq(cu.ctypes.data, len(tok), i) for i in range(cu[-1])]
        assert np.array_equal(got, want)
        assert index.find_seq(cu.ctypes.data, len(tok), int(cu[-1])) == -1
    for junk in ([5, 2, 9], [3, 3, 3], [-1, -7, 100], [0, 2 ** 31 - 1, -2 ** 31]):
        cu = np.array(junk, np.int32)
        for i in (0, 4, 2 ** 31 - 1):
            b = index.find_seq(cu.ctypes.data, 2, i)  # reads cu[0..2] only
            assert b == -1 or cu[b] <= i < cu[b + 1]


def test_slot_row_refuses_what_is_out_of_range(index):
    t = np.array([[3, -1, 7, 2 ** 31 - 1]], np.int32)
    row = lambda s, pages=8, mp=4: index.slot_row(t.ctypes.data, mp, pages, 4, 0, s)  # noqa: E731
    assert row(0) == 48 and row(15) == 63 and row(37) == 7 * 16 + 5
    assert row(16) == -1           # a negative page
    assert row(48) == -1           # a page past the pool
    assert row(48, pages=2 ** 31) == (2 ** 31 - 1) * 16  # 64-bit rows
    assert row(37, pages=7) == -1
    assert row(64) == -1 and row(-1) == -1 and row(2 ** 40) == -1  # past the table


def test_seq_checks_offsets_and_start(index):
    def seq(cu, st, tokens=100, mp=4):
        cu, st = np.array(cu, np.int32), np.array([st], np.int32)
        return index.seq(cu.ctypes.data, st.ctypes.data, 0, tokens, mp, 4)
    assert seq([2, 7], 10) == 5 and seq([2, 2], 0) == 0
    assert seq([7, 2], 0) == -1 and seq([-1, 3], 0) == -1 and seq([0, 101], 0) == -1 and seq([0, 3], -5) == -1
    assert seq([0, 5], 60) == -1 - 5  # runs past the table: flagged; its slots past the end have no row
    assert seq([0, 4], 60) == 4
