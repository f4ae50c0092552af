"""Verification of drafted tokens on the GPU at the ends of its random numbers' range, against the 64-bit oracle."""
import numpy as np
import pytest

from tests.test_gpu_verify import check, mnb  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [32 * 1024, 100 * 1024])
@pytest.mark.parametrize("refused", [False, True])
def test_a_pick_of_one_draws_the_last_weight(mnb, vocab, refused):  # noqa: F811
    """The last chunks' weights are far below an ulp of the sum, which sums of another order reach before them."""
    rng = np.random.default_rng(1)
    B = 200
    p = rng.random((B, vocab)).astype(np.float32)
    p[:, -4096:] *= np.float32(1e-18)
    pick, zeros = np.ones(B, np.float32), np.zeros(B, np.int32)
    if not refused:
        check(mnb, p, None, zeros, None, np.zeros(B, np.float32), pick)
        return
    # the first of two rows judges a draft that is refused: the draw is from what is left of it
    B //= 4
    q_start = np.arange(0, 2 * B + 1, 2, dtype=np.int32)
    draft = p[:2 * B] * np.float32(0.25)
    ids = np.full(2 * B, 5, np.int32)
    for q in (None, draft):
        assert not check(mnb, p[:2 * B], q, ids, q_start, np.full(2 * B, 1e9, np.float32), pick[:B]).any()
