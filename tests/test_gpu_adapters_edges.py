"""Low-rank adapters with infinite weights and with scales at the ends of their range, against the 64-bit oracle."""
import numpy as np
import pytest

from oracle import requests as o
from tests import gpu_util as G
from tests.test_gpu_adapters import kind, mnb, run  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

# m, k, n, rank, count: one launch and two, every form of the second product
SIZES = [(20, 300, 90, 12, 2), (20, 300, 90, 25, 2), (70, 6000, 90, 12, 2), (70, 6000, 300, 25, 2), (90, 300, 90, 40, 1), (70, 300, 90, 100, 2),
         (130, 64, 32800, 40, 3), (300, 72, 8200, 128, 2)]
IDS = ["-".join(map(str, s)) for s in SIZES]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_infinite_weights(mnb, size, dt):  # noqa: F811
    """An infinite element of B makes its column's output infinite with the sign of its h, or NaN where h is 0 or two of
    them differ.  One h is 2^-40 and less of its row's largest."""
    m, k, n, rank, count = size
    rng = np.random.default_rng((961,) + size)
    x = rng.integers(-3, 4, (m, k)).astype(kind(dt))
    x[:, 0] = rng.integers(-2, 3, m)
    a = rng.integers(-2, 3, (count, rank, k)).astype(kind(dt))
    a[:, 0] *= 200
    a[:, 5], a[:, 5, 0] = 0, 2.0 ** -24
    b = rng.integers(-2, 3, (count, n, rank)).astype(kind(dt))
    for column, ranks in ((3, [0]), (4, [5]), (7, [1]), (8, [2]), (11, [5, 8]), (n - 2, [3, 7]), (n - 1, [9])):
        for r in ranks:
            b[:, column, r] = rng.choice([np.inf, -np.inf])
    b[:, 20, 4] = np.nan
    base = rng.normal(size=(m, n)).astype(kind(dt))
    scales = np.full(count, 2.0 ** -12, np.float32)
    adapter = rng.integers(0, count, m)
    got = G.host(run(mnb, a, b, scales, None, adapter, x, base))
    want, tol = o.adapters(a, b, scales, None, adapter, x, base)
    assert np.isinf(want[:, [3, 7, 8, n - 1]]).any(0).all() and np.isinf(want[:, 4]).any() and np.isnan(want[:, 20]).all()
    G.assert_within(got, want, None, "adapters", bound=np.where(np.isfinite(tol), tol, 0))


@pytest.mark.parametrize("size", SIZES[:1] + SIZES[4:6], ids=IDS[:1] + IDS[4:6])
@pytest.mark.parametrize("far", [60000.0, 2.0 ** -12])
def test_scales_at_the_ends_of_their_range(mnb, far, size):  # noqa: F811
    """h far above 1, or far below: a scale that leaves fp32's range together with h's power of two still leaves a
    column without weights as it is, and an infinite weight infinite."""
    m, k, n, rank, count = size
    rng = np.random.default_rng((962,) + size)
    x = (far * rng.uniform(0.5, 1, (m, k))).astype(np.float16)
    a = (far * rng.uniform(0.5, 1, (count, rank, k))).astype(np.float16)
    b = rng.integers(-2, 3, (count, n, rank)).astype(np.float16)
    b[:, 10:30] = 0
    b[:, 30, 1] = np.inf
    base = rng.normal(size=(m, n)).astype(np.float16)
    adapter = rng.integers(0, count, m)
    for scale in (3e38, -2.0 ** 120, 2.0 ** -126, -2.0 ** -149):
        got = G.host(run(mnb, a, b, np.full(count, scale, np.float32), None, adapter, x, base))
        assert (got[:, 10:30] == base[:, 10:30]).all() and (got[:, 30] == np.copysign(np.inf, scale)).all()
