"""Edges of the operators around the products, against plain implementations
in 64 bits, beside those of test_gpu_operators.py, whose helpers and derived
tolerances they share."""
import numpy as np
import pytest

from test_gpu_operators import check_log_probs, rng_of, up

pytestmark = pytest.mark.gpu


@pytest.fixture
def torch():
    return pytest.importorskip("torch")


# ---------------------------------------------------------------------------
# log probabilities

@pytest.mark.parametrize("m,n", [(1, 128256), (2, 40001), (16, 32768)])
@pytest.mark.parametrize("low", [0, 5])
def test_log_probs_join_of_many_alternatives(qmm, torch, m, n, low):
    """Eight CTAs a row, one of whose parts holds small words alone: the bound of the join is low, so
    nearly all of the eight times 32 alternatives are ranked.  Every repetition gives the same words."""
    g = rng_of(30, m, n, low)
    x = g.standard_normal((m, n)).astype(np.float32)
    part = n // 8
    x[:, low * part + 64: (low + 1) * part - 64] -= 30
    check_log_probs(qmm, x, 32)
    view = up(x)
    want = qmm.log_probs(view, top_k=32)
    for _ in range(200):
        got = qmm.log_probs(view, top_k=32)
        assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
