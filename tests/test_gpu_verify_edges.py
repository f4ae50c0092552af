"""Verification of drafted tokens on the GPU at the ends of its random numbers' range, against the 64-bit oracle."""
import numpy as np
import pytest

from tests.test_gpu_verify import check, inputs, mnb  # noqa: F401 (fixture)

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


@pytest.mark.parametrize("vocab", [300, 70000])
def test_accept_outside_its_range(mnb, vocab):  # noqa: F811
    """Below 0 a certain draft is taken at a probability of 0 too, and one with q > 0; NaN and large ones refuse."""
    rng = np.random.default_rng(2)
    target, draft, ids, q_start, accept, pick = inputs(rng, [5] * 8, vocab, "f32")
    row = np.arange(len(ids) - 1)
    target[row, ids[1:]] = 0                            # no draft has a probability
    assert (draft[row, ids[1:]] > 0).all()
    for value, taken in ((-1.0, 4), (-2.0 ** -149, 4), (-np.inf, 4), (0.0, 0), (-0.0, 0), (1.0, 0), (np.inf, 0), (np.nan, 0)):
        accept[:] = value
        for q in (None, draft):
            counts = check(mnb, target, q, ids, q_start, accept, pick)
            assert (counts == taken).all(), (value, counts)
    accept[:] = -1.0
    ids[3], ids[7] = vocab, -1                          # still refused
    draft[row[10:15], ids[11:16]] = 0                   # -1 times 0 is not below 0
    assert check(mnb, target, None, ids, q_start, accept, pick)[:4].tolist() == [2, 1, 4, 4]
    assert check(mnb, target, draft, ids, q_start, accept, pick)[:4].tolist() == [2, 1, 0, 4]
