"""A serving step's entry points without a GPU: refusals that return before any
CUDA call, the binding's checks, and the references' own identities."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import bit_weight_quantized_w4a8_gb300 as w4  # noqa: E402
from bit_weight_quantized_w4a8_gb300 import _binding as B  # noqa: E402
import layer_ref as ref  # noqa: E402
import step_ref as sref  # noqa: E402

P = 0x10000  # a fake, aligned address: never dereferenced (checks fail first)
N, S, A = B.ERR_NULL, B.ERR_SHAPE, B.ERR_ALIGN


@pytest.fixture(scope="module")
def L():
    w4.build()
    return w4.lib()


def call(f, base, change, who, status):
    a = dict(base)
    a.update(change)
    assert f(*a.values(), None) == status
    assert w4.w4a8_last_error().startswith(who)


def axis_of(*a):
    return bytes(a) + bytes(64)


ROPE = dict(X=P, x_type=0, ld_x=256, tokens=4, heads=2, dim=128, pos=P, axes=3, axis=axis_of(0, 1, 2), freqs=P, rot=64,
            interleaved=0, mscale=1.0, Y=P, y_type=0, ld_y=256, flags=0)


@pytest.mark.parametrize("change,status", [
    (dict(axes=0), S), (dict(axes=5), S), (dict(axes=-1), S), (dict(axes=2), S), (dict(axis=None), N),
    (dict(axis=axis_of(0, 3)), S), (dict(axis=axis_of(255)), S), (dict(X=None), N), (dict(pos=None), N), (dict(rot=12), S),
    (dict(dim=96), S), (dict(flags=2), S), (dict(pos=P + 2), A)])
def test_rope_rotate_axes_refusals(L, change, status):
    call(L.rope_rotate_axes, ROPE, change, "rope_rotate_axes", status)


def test_kvq_write_axes_refusals(L):
    c = ctypes.byref(B._Cache(k=P, v=P, ks=P, vs=P, pages=4, page=64, heads=2, dim=128, bits=8))
    b = ctypes.byref(B._Batch(cu=P, start=P, table=P, seqs=1, tokens=4, max_pages=2))
    base = dict(c=c, b=b, K=P, ld_k=256, V=P, ld_v=256, Q=None, ld_q=0, heads_q=0, x_type=0, pos=P, axes=2,
                axis=axis_of(0, 1), freqs=P, rot=64, interleaved=0, mscale=1.0, Q_out=None, flags=0)
    for change, status in ((dict(axes=0), S), (dict(freqs=None), N), (dict(axis=None), N), (dict(axes=1), S),
                           (dict(Q=P), N), (dict(K=None), N), (dict(ld_v=255), S), (dict(pos=None), N)):
        call(L.kvq_write_axes, base, change, "kvq_write_axes", status)


POOL = dict(table=P, held=P, stack=P, top=P, seqs=4, max_pages=8, pages=32, page=64)
PLAN = dict(lens=P, grow=None, add=P, mask=None, tokens=16, cu=P, pos=P, slot=P, seq=P, ws=P, ws_bytes=1 << 20, flags=0)


def pool(**kw):
    d = dict(POOL)
    d.update(kw)
    return ctypes.byref(B._Pool(**d))


@pytest.mark.parametrize("change,status", [
    (dict(table=None), N), (dict(top=None), N), (dict(seqs=0), S), (dict(seqs=65537), S), (dict(max_pages=0), S),
    (dict(pages=0), S), (dict(pages=1 << 31), S), (dict(page=48), S), (dict(page=8), S), (dict(page=512), S),
    (dict(stack=P + 2), A)])
def test_kvq_pool_refusals(L, change, status):
    assert L.kvq_plan(pool(**change), *PLAN.values(), None) == status
    assert w4.w4a8_last_error().startswith("kvq_plan")
    assert L.kvq_plan_workspace_bytes(pool(**change)) == 0


@pytest.mark.parametrize("change,status", [
    (dict(lens=None), N), (dict(add=None), N), (dict(cu=None), N), (dict(tokens=0), S), (dict(tokens=1 << 31), S),
    (dict(lens=P + 1), A), (dict(grow=P + 2), A), (dict(mask=P + 4), A), (dict(slot=P + 4), A), (dict(flags=2), S),
    (dict(ws=None), B.ERR_WORKSPACE), (dict(ws_bytes=8), B.ERR_WORKSPACE), (dict(ws=P + 8), A)])
def test_kvq_plan_refusals(L, change, status):
    a = dict(PLAN)
    a.update(change)
    assert L.kvq_plan(pool(), *a.values(), None) == status
    assert w4.w4a8_last_error().startswith("kvq_plan")
    assert L.kvq_plan_workspace_bytes(pool()) > 0 and L.kvq_plan_workspace_bytes(None) == 0


VERIFY = dict(L=P, l_type=0, ld_l=100, vocab=100, cu=P, seqs=2, tokens=8, ids=P, mask=None, Q=None, q_type=0, ld_q=0,
              temp=None, u=P, keep=P, out=P, count=P, ws=P, ws_bytes=1 << 20, flags=0)


@pytest.mark.parametrize("change,status", [
    (dict(L=None), N), (dict(cu=None), N), (dict(ids=None), N), (dict(u=None), N), (dict(keep=None), N), (dict(out=None), N),
    (dict(count=None), N), (dict(l_type=2), S), (dict(Q=P, q_type=3, ld_q=100), S), (dict(vocab=0), S),
    (dict(vocab=(1 << 22) + 1, ld_l=1 << 23), S), (dict(tokens=0), S), (dict(seqs=0), S), (dict(seqs=65537), S),
    (dict(ld_l=99), S), (dict(Q=P, ld_q=99), S), (dict(flags=8), S), (dict(L=P + 2), A), (dict(L=P + 1, l_type=1), A),
    (dict(Q=P + 2, ld_q=100), A), (dict(mask=P + 4), A), (dict(u=P + 1), A), (dict(count=P + 2), A)])
def test_draft_verify_refusals(L, change, status):
    call(L.draft_verify, VERIFY, change, "draft_verify", status)


QW = dict(W=P, N=128, K=128, Wf=P, sw=P)
QR = dict(X=P, x_type=0, M=4, K=128, Xf=P, sa=P, flags=0)
GEMM = dict(Xf=P, sa=P, M=4, K=128, Wf=P, sw=P, N=128, Y=P, y_type=0, flags=0)
LIN = dict(X=P, x_type=1, M=4, K=128, Wf=P, sw=P, N=128, Y=P, y_type=1, ws=P, ws_bytes=1 << 20, flags=0)
SIZES = [(dict(K=0), S), (dict(K=24), S), (dict(K=131088), S)]


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(W=None), N), (dict(sw=None), N), (dict(N=0), S), (dict(N=1 << 31), S), (dict(W=P + 8), A), (dict(Wf=P + 4), A),
    (dict(sw=P + 2), A)])
def test_f8_quantize_weights_refusals(L, change, status):
    call(L.f8_quantize_weights, QW, change, "f8_quantize_weights", status)


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(X=None), N), (dict(Xf=None), N), (dict(M=0), S), (dict(M=(1 << 24) + 1), S), (dict(x_type=5), S),
    (dict(flags=2), S), (dict(X=P + 8), A), (dict(sa=P + 1), A)])
def test_f8_quantize_rows_refusals(L, change, status):
    call(L.f8_quantize_rows, QR, change, "f8_quantize_rows", status)


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(Xf=None), N), (dict(Y=None), N), (dict(M=0), S), (dict(N=0), S), (dict(M=1 << 24, N=1 << 20), S),
    (dict(y_type=2), S), (dict(flags=2), S), (dict(Xf=P + 8), A), (dict(Wf=P + 8), A), (dict(Y=P + 2), A),
    (dict(Y=P + 1, y_type=1), A)])
def test_f8_gemm_refusals(L, change, status):
    call(L.f8_gemm, GEMM, change, "f8_gemm", status)


@pytest.mark.parametrize("change,status", SIZES + [
    (dict(X=None), N), (dict(sw=None), N), (dict(x_type=2), S), (dict(y_type=-1), S), (dict(flags=2), S),
    (dict(X=P + 4), A), (dict(Y=P + 1), A)])
def test_f8_linear_refusals(L, change, status):
    call(L.f8_linear, LIN, change, "f8_linear", status)
    assert L.f8_linear_workspace_bytes(4, 128, 128) >= 4 * 128 + 4 * 4
    assert L.f8_linear_workspace_bytes(4, 24, 128) == 0


def test_binding_refuses_cpu_tensors_and_wrong_types(L):
    f, i32 = torch.zeros, torch.int32
    X, Wf, sw = f(2, 128), f(5, 128, dtype=torch.uint8), f(1, 1)
    for bad in (lambda: w4.f8_linear(X, Wf, sw), lambda: w4.f8_quantize_rows(X), lambda: w4.f8_quantize_weights(X),
                lambda: w4.f8_gemm(Wf, sw, Wf, sw), lambda: w4.draft_verify(X, f(2, dtype=i32), f(2, dtype=i32), f(2)),
                lambda: w4.kvq_plan(w4.kvq_pool(2, 2, 4, device="cpu"), 64, f(2, dtype=i32), f(2, dtype=i32), 8),
                lambda: w4.rope_rotate(f(2, 2, 64), f(3, 2, dtype=i32), f(32, dtype=torch.float64), axis=bytes(32)),
                lambda: w4.rope_rotate(f(2, 2, 64), f(3, 2, dtype=i32), f(32, dtype=torch.float64), axis=bytes(31))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        w4.f8_linear(X.double(), Wf, sw)
    with pytest.raises(TypeError):
        w4.draft_verify(None, None, None, None)


def test_rope_axes_layouts():
    assert w4.rope_axes((2, 3, 3)) == bytes([0, 0, 1, 1, 1, 2, 2, 2])
    assert w4.rope_axes((2, 3, 3), cycled=True) == bytes([0, 1, 2, 0, 1, 2, 1, 2])
    assert w4.rope_axes((4,)) == bytes(4)
    for bad in ((), (1,) * 5, (1, -1)):
        with pytest.raises(ValueError):
            w4.rope_axes(bad)


# -- the references ----------------------------------------------------------------

def test_e4m3_codes_are_the_nearest():
    v = sref.E4M3[:127]
    assert v[126] == 448 and v[1] == 2.0 ** -9 and math.isnan(sref.E4M3[127])
    assert np.array_equal(sref.e4m3_codes(v), np.arange(127)) and np.array_equal(sref.e4m3_codes(-v[1:]), np.arange(129, 255))
    mid = (v[1:] + v[:-1]) / 2  # ties to the even code
    assert np.all(sref.e4m3_codes(mid) % 2 == 0)
    assert np.array_equal(sref.e4m3_codes(np.nextafter(mid, 0)), np.arange(126))
    assert np.array_equal(sref.e4m3_codes(np.nextafter(mid, 1e9)), np.arange(1, 127))
    assert sref.e4m3_codes(np.array([449.0]))[0] == 126


@pytest.mark.parametrize("with_q", [False, True])
def test_verified_tokens_follow_the_target(with_q):
    """The reference itself: over a fine grid of random numbers, and over the drafts with
    their probabilities, the first token said has the target's distribution."""
    rng = np.random.default_rng(1)
    v, g = 4, 64
    rows = rng.standard_normal((2, v)).astype(np.float32)
    p = sref.distribution(rows[0], 1.0)
    q = np.array([[0.4, 0.1, 0.3, 0.2]] * 2)
    freq = np.zeros(v)
    grid = (np.arange(g) + 0.5) / g
    for x in range(v):
        for u1 in grid:
            for u0 in grid:
                _, said = sref.verify_seq(rows, [0, x], [u0, u1], None, q if with_q else None)
                freq[said[0]] += (q[0, x] if with_q else 1 / v) / g ** 2
    # each cell of the grid is off by at most one in each of the two numbers
    assert np.all(np.abs(freq - p) < 2.5 / g)


def test_several_axes_with_one_position_are_one_axis():
    rng = np.random.default_rng(2)
    x, pos = rng.standard_normal((5, 2, 64)), rng.integers(0, 1000, 5)
    f = 1e4 ** (-np.arange(16) / 16)
    one = ref.rotate(x, pos, f, True)
    many = sref.rotate_axes(x, np.stack([pos] * 3), [0, 1, 2, 1] * 4, f, True)
    assert np.array_equal(one[0], many[0]) and np.array_equal(one[1], many[1])


def test_pool_gives_back_what_it_handed_out():
    rng = np.random.default_rng(3)
    pool_ = sref.Pool(np.full((6, 9), -1, np.int32), np.zeros(6, np.int32), rng.permutation(40).astype(np.int32), 40,
                      np.zeros(6, np.int64), 16)
    before = pool_.stack.copy()
    cu, pos, slot, seq = pool_.plan([17, 0, 16, 1, 200, 33], 80)  # the fifth would need 13 pages of 9
    assert list(np.diff(cu)) == [17, 0, 16, 1, 0, 33] and len(set(slot[:67])) == 67
    pool_.plan([-1] * 6, 8)
    assert pool_.top == 40 and np.array_equal(pool_.stack, before) and not pool_.held.any()
