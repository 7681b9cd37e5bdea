"""Values at the ends of what the decoder layer's cache and attention hold, on
the GPU, against the 64-bit references and bounds of layer_ref.py: scales
that are tiny, huge, negative, zero or not finite."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import guards  # noqa: E402
import layer_ref as ref  # noqa: E402
from test_gpu_layer import (check_attention, dev, fill, make_batch, make_cache, w4,  # noqa: E402,F401
                            wide_cols)

pytestmark = pytest.mark.gpu

F32, F16 = np.float32, np.float16


@pytest.fixture(autouse=True)
def _no_error_left(w4):  # noqa: F811
    yield
    assert w4.w4a8_device_error() == 0


# -- the write's codes -------------------------------------------------------------

# Largest values of vectors: binary32's subnormals, the scales' (1.2e-38 times 127 or
# 7, and a quarter of that, where 1 / scale is no longer finite), ordinary ones.
TINY = [1e-45, 3e-45, 9e-44, 1e-42, 1e-40, 1.17e-38, 2e-38, 2.1e-38, 8e-38, 9e-38, 3.7e-37, 3.8e-37, 1.4e-36, 1.5e-36, 1e-35]


@pytest.mark.parametrize("dim,bits", [(64, 8), (128, 8), (128, 4), (256, 4)])
def test_write_of_tiny_vectors_is_exact(w4, dim, bits):  # noqa: F811
    rng = np.random.default_rng(dim + bits)
    n, heads = len(TINY), 3
    x = [rng.uniform(-1, 1, (n, heads, dim)) for _ in range(2)]
    for t in x:
        t[:, 0, 0], t[:, 1, -1] = 1, -1
        t[:, :, 5:9] = 0                # zeros inside
        t *= np.array(TINY)[:, None, None]
    k, v = (t.astype(F32) for t in x)
    pg = ref.Paged(rng, (n,), (3,), 16)
    c, gs = make_cache(w4, pg, heads, dim, bits)
    w4.kvq_write(c, make_batch(w4, pg), dev(k), dev(v))
    guards.check_all(*gs)
    p, o = pg.own()
    for t, codes, scales in ((k, c.k, c.ks), (v, c.v, c.vs)):
        q, s = ref.quantize(t, bits)
        assert np.array_equal(scales.cpu().numpy()[p, :, o], s)
        assert np.array_equal(codes.cpu().numpy()[p, :, o], ref.pack(q, bits))
