"""RMS norm at the ends of its range: rows of zeros without eps, infinities and NaN the weight hides, squares past
binary32, quotients that only the exact products place on their side of a tie."""
import numpy as np
import pytest

from oracle import decoder as o
from tests import gpu_util as G
from tests.test_gpu_norm import _dev, _inputs, _value_tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mnb():
    from block_wise_int4_amd import mnb as m
    return m


def codes_of(mnb, x, w, eps, kind, residual=None):
    t = G.torch()
    out, sc = t.full(x.shape, 99, dtype=kind, device="cuda"), t.full((x.shape[0],), -1.0, device="cuda")
    mnb.mnb_rms_norm(_dev(x), _dev(w), out, eps, residual=None if residual is None else _dev(residual), scales=sc)
    return G.host(out), G.host(sc)


def kinds():
    t = G.torch()
    return t.float16, t.int8


SIZES = [64, 67, 4099, 40003]       # within one vector a thread, past the vectors, several, past the registers


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("k", SIZES)
def test_a_row_of_zeros_without_eps_has_scale_zero(mnb, k, dt):
    x, _, w = _inputs(3, k, dt, 20)
    x[1] = 0
    for kind in kinds():
        q, s = codes_of(mnb, x, w, 0.0, kind)
        assert s[1] == 0 and (q[1] == 0).all()
        assert (s[[0, 2]] > 0).all() and np.isfinite(s).all()


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("k", SIZES)
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_a_bad_value_under_a_zero_weight_still_marks_its_row(mnb, value, k, dt):
    x, r, w = _inputs(4, k, dt, 21)
    for at in (3, k - 1):
        y, u = x.copy(), w.copy()
        y[2, at], u[at] = value, 0
        for kind in kinds():
            q, s = codes_of(mnb, y, u, 1e-5, kind, r)
            assert np.isnan(s[2]) and (q[2] == 0).all() and np.isfinite(s[[0, 1, 3]]).all(), (at, s)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("k", SIZES)
def test_a_bad_weight_marks_every_row(mnb, k, dt):
    x, r, w = _inputs(3, k, dt, 22)
    x[1], r[1] = 0, 0                                  # 0 times NaN is NaN too
    for at, value in ((5, np.nan), (k - 1, np.nan), (7, np.inf)):
        u = w.copy()
        u[at] = value
        for kind in kinds():
            _, s = codes_of(mnb, x, u, 1e-5, kind, r)
            assert np.isnan(s).all(), (at, value, s)


@pytest.mark.parametrize("k", SIZES)
@pytest.mark.parametrize("size,eps", [(1e19, 1e-5), (1e25, 1e-5), (1e36, 0.0), (1e-21, 0.0), (1e-30, 0.0), (1e-30, 1e-58),
                                      (1e-24, 1e-45)])
def test_squares_past_binary32(mnb, size, eps, k):
    """fp32 rows whose squares overflow or vanish, beside rows of usual size."""
    t = G.torch()
    x, _, w = _inputs(3, k, "f32", 23)
    x[1] = np.clip(x[1], -3, 3) * np.float32(size)
    eps = float(np.float32(eps))                       # as the call receives it
    _, y = o.rms_norm(x, None, w, eps)
    out = t.empty((3, k), device="cuda")
    mnb.mnb_rms_norm(_dev(x), _dev(w), out, eps)
    assert (np.abs(G.host(out) - y) <= _value_tolerance(y, k, "f32")).all()
    s, q = o.norm_codes(x, w, eps)
    for kind in kinds():
        c, got = codes_of(mnb, x, w, eps, kind)
        assert (np.abs(got - s) <= s * (0.5 * (k + 2) + 10) * o.EPS32).all()
        # the products h w are rounded to binary32, whose least normal value is 2^-126
        assert (np.abs(c - q) <= 0.5 + 2 * 127 * o.EPS32 + 1e-12).all()


@pytest.mark.parametrize("k", SIZES)
def test_quotients_beside_ties(mnb, k):
    """fp32 elements whose quotients lie within 4e-6 of a tie: the products in 64 bits decide."""
    rng = np.random.default_rng((24, k))
    x = rng.normal(size=(1, k)).astype(np.float32)
    x[0, 0] = np.float32(3.3)
    w = np.ones(k, np.float32)
    w[0] = np.float32(1.7)
    top = float(x[0, 0]) * float(w[0])                 # exact in 64 bits, not in 32
    want = rng.integers(-126, 126, k) + 0.5
    w[1:] = (want[1:] * top / 127.0 / x[0, 1:].astype(np.float64)).astype(np.float32)
    q = 127.0 * (x[0].astype(np.float64) * w.astype(np.float64)) / top
    near = np.abs(np.abs(q) % 1 - 0.5)
    assert 126.999 < np.abs(q).max() < 127.001 and np.median(near[1:]) < 4e-6
    sure = near > 1e-10
    want = np.trunc(q + np.copysign(0.5, q))
    for kind in kinds():
        c, s = codes_of(mnb, x, w, 1e-5, kind)
        assert (c[0, sure] == want[sure]).all(), int((c[0, sure] != want[sure]).sum())
