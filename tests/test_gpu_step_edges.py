"""A serving step's operators where one input makes another's error large: rows
without a distribution, sums that cancel, numbers at the ends of their types, idle
rows; and calls launched dependently behind what they read."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import guards  # noqa: E402
import step_ref as sref  # noqa: E402
from test_gpu_step import (_no_error_left, dev, drafts, make_pool, np_, run_verify, same, tree_words,  # noqa: E402,F401
                           w4)

pytestmark = pytest.mark.gpu

F32, F16, I32, I64 = np.float32, np.float16, np.int32, np.int64
NEG = F32(-np.inf)
ALMOST_ONE = F32(1 - 2.0 ** -24)


def words(*parents):
    """Masks of a tree by its tokens' parents."""
    w = []
    for i, p in enumerate(parents):
        w.append((w[p] if p >= 0 else 0) | 1 << i)
    return np.array(w, np.uint64).view(I64)


# -- verification of drafts ------------------------------------------------------------

def test_no_child_of_a_row_with_a_nan_is_taken(w4):  # noqa: F811
    """With draft probabilities and several children: a row with a NaN among ordinary logits has
    no distribution for the second and third child either."""
    rng = np.random.default_rng(31)
    seqs, v = 12, 3000
    logits = (2 * rng.standard_normal((5 * seqs, v))).astype(F32)
    q = np.exp(rng.standard_normal((5 * seqs, v)))
    q = (q / q.sum(1, keepdims=True)).astype(F32)
    ids = np.zeros(5 * seqs, I32)
    u = np.full(5 * seqs, 1e-6, F32)
    for b in range(seqs):
        # the tokens that have most left after a refusal; one child's own child behind them
        ids[5 * b + 1:5 * b + 5] = np.argsort(sref.distribution(logits[5 * b], 1.0) - q[5 * b])[-4:]
        if b % 3 < 2:
            logits[5 * b, rng.integers(0, v)] = np.nan
    mask = np.tile(words(-1, 0, 0, 0, 2), seqs)
    cu = np.arange(0, 5 * seqs + 1, 5, dtype=I32)
    got = run_verify(w4, logits, cu, ids, u, mask, q)
    same(got, sref.verify(logits, cu, ids, u, mask, q))
    bad = np.arange(seqs) % 3 < 2
    assert np.all(got[2][bad] == 1) and np.all(got[1][::5][bad] == -1) and np.all(got[2][~bad] > 1)
