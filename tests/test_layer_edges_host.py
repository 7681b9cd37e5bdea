"""Offsets and starts that are out of range, in the cache's look-ups on the host."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    d = tmp_path_factory.mktemp("kvq_edges")
    (d / "index.cpp").write_text('#include "%s"\n' % os.path.join(ROOT, "bit_weight_quantized_w4a8_gb300", "csrc", "kvq_index.h") + """
// the slot of token i of a batch, as the write and the read find it
extern "C" int64_t slot(const int32_t* cu, const int32_t* st, int seqs, int i) {
    const int b = w4a8::kvq_find_seq(cu, seqs, i);
    return b < 0 ? -1 : w4a8::kvq_token_slot(cu, st, b, i); }
extern "C" int ctas(int tokens, int per) { return w4a8::kvq_ctas(tokens, per); }
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-shared", "-fPIC",
                    "-o", str(d / "index.so"), str(d / "index.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "index.so"))
    lib.slot.restype = ctypes.c_int64
    lib.slot.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int]
    return lib


def slot(index, cu, start, i):
    cu, start = np.array(cu, np.int32), np.array(start, np.int32)
    return index.slot(cu.ctypes.data, start.ctypes.data, len(start), i)


def test_token_slots(index):
    assert [slot(index, [0, 3, 3, 5], [7, 1, 20], i) for i in range(5)] == [7, 8, 9, 20, 21]
    assert slot(index, [0, 5], [2 ** 31 - 1], 4) == 2 ** 31 + 3  # past any table, not wrapped around


@pytest.mark.parametrize("cu,start", [([-3, 5], [4]), ([-2 ** 31, 5], [2 ** 31 - 1]), ([-2 ** 31, 5], [4]), ([0, 5], [-1]),
                                      ([0, 5], [-2 ** 31])])
def test_negative_offsets_and_starts_have_no_slot(index, cu, start):
    """A negative offset once moved tokens to slots further on, and far ones wrapped around."""
    assert all(slot(index, cu, start, i) == -1 for i in range(5))


def test_ctas_of_any_token_count(index):
    """Rounding up by adding first passed 2^31 at the largest counts that the entry points take."""
    for per in (1, 4, 8, 32):
        for tokens in (1, 3, 4, 5, 8191, 2 ** 31 - 4, 2 ** 31 - 2, 2 ** 31 - 1):
            assert index.ctas(tokens, per) == -(-tokens // per)


@pytest.mark.parametrize("rot,base,factor,old_ctx,low,high", [(128, 1e6, 4.0, 32768, 1.0, 32.0), (64, 1e4, 16.0, 4096, 1.0, 32.0),
                                                              (256, 5e5, 2.0, 8192, 2.0, 20.0)])
def test_yarn_between_its_ends(rot, base, factor, old_ctx, low, high):
    """The ramp over the pair index, from the pair that turns `high` times within old_ctx
    positions (rounded down) to the one that turns `low` times (rounded up)."""
    import math

    import bit_weight_quantized_w4a8_gb300 as w4
    w4.build()
    got, mscale = w4.rope_frequencies(rot, base, "yarn", factor, old_ctx=old_ctx, low=low, high=high)
    # freq(i) * old_ctx / (2 pi) = turns  <=>  i = rot / 2 * log_base(old_ctx / (2 pi turns))
    pair = lambda turns: rot / 2 * math.log(old_ctx / (2 * math.pi * turns)) / math.log(base)  # noqa: E731
    a, z = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    part = np.clip((i - a) / (z - a), 0, 1)
    assert np.allclose(got.numpy(), f * (1 - part) + f / factor * part, rtol=1e-13, atol=0)
    assert ((part > 0) & (part < 1)).sum() > 3 and mscale == np.float32(0.1 * math.log(factor) + 1)
