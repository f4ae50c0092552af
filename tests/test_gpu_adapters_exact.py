"""Low-rank adapters on operands whose every sum is exact, so that the output has to match bit for bit; and the forms
that many rows take.

x, A and B are small whole numbers, scales powers of two: h and y are multiples of 2^-9 below 2^24 of them, in any
order of summation (checked), h has more than 11 bits, and base is -y rounded to fp16, so that what is left is the low
bits of the sums: a step of k that is left out or taken twice, h rounded to 16 bits or a wrong row changes them."""
import numpy as np
import pytest

from tests import gpu_util as G
from tests.test_gpu_adapters import kind, mnb, run  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

# m, n, k, rank, count; fields of the plan that the size is here for
SIZES = [
    ((6501, 2603, 1103, 12, 3), dict(one=0, down_tile=64, up_tile=64, down_ranks=1, up_blocks=1)),
    ((6501, 2603, 1103, 27, 3), dict(one=0, down_tile=64, up_tile=64, down_ranks=2, up_blocks=1)),
    ((6501, 2603, 1103, 50, 3), dict(one=0, down_tile=64, up_tile=64, down_ranks=4, up_blocks=2)),
    ((6501, 2603, 1103, 100, 3), dict(one=0, down_tile=64, up_tile=64, down_ranks=4, up_blocks=2)),
    ((3401, 70, 1100, 128, 2), dict(one=0, down_tile=64, down_ranks=4, up_blocks=1)),
    ((6500, 61, 1041, 32, 1), dict(one=0, down_tile=64, up_tile=16, down_ranks=2)),
    ((4101, 4099, 705, 40, 4), dict(one=0, down_tile=32, up_tile=64, up_blocks=2)),
    ((1501, 2603, 705, 128, 4), dict(one=0, down_tile=32, up_tile=32, up_blocks=2)),
    ((1001, 4096, 705, 64, 4), dict(one=0, down_tile=32, up_tile=32, up_blocks=1)),
    ((1001, 4096, 705, 65, 4), dict(one=0, down_tile=32, up_tile=32, up_blocks=1)),
    ((130, 700, 5000, 128, 3), dict(one=0, down_tile=16)),
    ((3, 200, 5000, 128, 3), dict(one=0, splits=8)),
    ((82, 4096, 11008, 64, 12), dict(one=0, splits=8)),
    ((1, 300, 2048, 16, 3), dict(one=1)),
    ((33, 515, 1100, 16, 2), dict(one=1)),
    ((50, 515, 1030, 31, 1), dict(one=1)),
]
IDS = ["-".join(map(str, s)) for s, _ in SIZES]


def whole(rng, size, mixed):
    m, n, k, rank, count = size
    x = rng.integers(-3, 13, (m, k)).astype(np.float32)
    a = rng.integers(0, 2, (count, rank, k)).astype(np.float32)
    b = rng.integers(-2, 3, (count, n, rank)).astype(np.float32)
    scales = (2.0 ** -rng.integers(6, 10, count)).astype(np.float32)
    ranks = rng.integers(0, rank + 2, count).astype(np.int32) if mixed else None
    adapter = rng.integers(-1, count, m)
    y, base = np.zeros((m, n)), rng.integers(-8, 9, (m, n)).astype(np.float16)
    for g in range(count):
        r = min(rank, int(ranks[g])) if mixed else rank
        rows = adapter == g
        h = x[rows] @ a[g, :r].T
        assert (np.abs(x[rows]) @ a[g, :r].T).max(initial=0) < 2 ** 22
        assert (np.abs(h) @ np.abs(b[g, :, :r]).T).max(initial=0) < 2 ** 24
        y[rows] = (h @ b[g, :, :r].T).astype(np.float64) * float(scales[g])
        if mixed:
            a[g, r:], b[g, :, r:] = np.nan, np.inf
    some = adapter >= 0
    base[some] = -y[some].astype(np.float16)
    assert np.isfinite(base).all()
    return a, b, scales, ranks, adapter, x, base, y + base.astype(np.float64)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("order", ["grouped", "any", "mixed"])
@pytest.mark.parametrize("size", [s for s, _ in SIZES], ids=IDS)
def test_exact_sums(mnb, size, order, dt):  # noqa: F811
    rng = np.random.default_rng((960,) + size)
    a, b, scales, ranks, adapter, x, base, y = whole(rng, size, order == "mixed")
    if order == "grouped":
        at = np.argsort(adapter, kind="stable")
        adapter, x, base, y = adapter[at], x[at], base[at], y[at]
    got = run(mnb, a.astype(kind(dt)), b.astype(kind(dt)), scales, ranks, adapter, x.astype(kind(dt)), base.astype(kind(dt)))
    got = G.host(got)
    want = y.astype(kind(dt)).astype(np.float64)
    wrong = got != want
    assert not wrong.any(), "%d of %d, the first at %s" % (wrong.sum(), wrong.size, np.argwhere(wrong)[:3].tolist())
