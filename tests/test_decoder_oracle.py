"""Pins of the plain oracle of the norm, the 4-bit cache and the attention:
hand-worked numbers, closed forms and the layout's own properties.  CPU only."""
import numpy as np
import pytest

from oracle import decoder as o


def test_norm_by_hand():
    x = np.array([[3.0, 4.0]], np.float32)
    h, y = o.rms_norm(x, None, np.array([1.0, 2.0], np.float32), 0.0)
    r = np.sqrt(12.5)
    assert (h == x).all() and np.allclose(y, [[3 / r, 8 / r]], rtol=1e-15)
    # the residual's sum is rounded to the type before it is normed: 1 + 2^-12 is 1 in fp16
    h, y = o.rms_norm(np.ones((1, 2), np.float16), np.full((1, 2), 2.0 ** -12, np.float16), np.ones(2, np.float16), 0.0)
    assert (h == 1).all() and (y == 1).all()
    s, q = o.norm_codes(np.array([[3.0, -4.0, 0.0]]), np.array([1.0, 0.5, 7.0]), 0.0)
    assert np.allclose(q, [[127.0, -127.0 * 2 / 3, 0.0]]) and np.allclose(s, 3.0 / np.sqrt(25 / 3) / 127)
    s, q = o.norm_codes(np.zeros((1, 4)), np.ones(4), 1e-5)
    assert s[0] == 0 and (q == 0).all()


def test_quantize_by_hand():
    x = np.zeros((1, 32), np.float32)
    x[0, :4] = [-7.5, 7.5, 0.4, 0.6]            # s = 1, z = rne(7.5) = 8
    c, s, z = o.quantize_rows(x, 32)
    assert s[0, 0] == 1 and z[0, 0] == 8
    assert c[0, :5].tolist() == [0, 15, 8, 9, 8]   # rne(-7.5) = -8, rne(7.5) + 8 clamped
    # one-sided groups keep zero in their range
    c, s, z = o.quantize_rows(np.full((1, 32), 3.0, np.float32), 32)
    assert z[0, 0] == 0 and (c == 15).all() and s[0, 0] == np.float16(0.2)
    c, s, z = o.quantize_rows(np.zeros((1, 32), np.float32), 32)
    assert s[0, 0] == 0 and (c == 0).all()
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones((1, 64), np.float32)
        x[0, 5] = bad
        c, s, z = o.quantize_rows(x, 32)
        assert not np.isfinite(s[0, 0]) and np.isfinite(s[0, 1])


def test_quantization_error_is_half_a_step():
    rng = np.random.default_rng(3)
    x = (rng.normal(size=(50, 128)) * np.exp(rng.normal(size=(50, 1)))).astype(np.float32)
    for group in (32, 64, 128):
        c, s, z = o.quantize_rows(x, group)
        s64 = np.repeat(s.astype(np.float64), group, -1)
        y = (c.astype(np.float64) - np.repeat(z.astype(np.float64), group, -1)) * s64
        # half a step, one more where the zero point's or the scale's rounding clamps an end
        assert (np.abs(y - x) <= 1.01 * s64).all()
        assert (np.abs(y - x) <= 0.502 * s64).mean() > 0.9


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(4)
    ang = rng.uniform(0, 6, (10, 32))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    x = rng.normal(size=(6, 2, 128)).astype(np.float32)
    pos = np.array([0, 3, 9, 12, 1, 2])
    for inter in (False, True):
        y = o.rotate(x, pos, cos, sin, 64, inter)
        assert (y[..., 64:] == x[..., 64:]).all()
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-5)
    y = o.rotate(x, pos, cos, sin, 64)
    assert np.allclose(y[1, 0, 5], x[1, 0, 5] * np.cos(ang[3, 5]) - x[1, 0, 37] * np.sin(ang[3, 5]), atol=1e-6)
    y = o.rotate(x, pos, cos, sin, 64, True)
    assert np.allclose(y[3, 1, 11], x[3, 1, 11] * np.cos(ang[9, 5]) + x[3, 1, 10] * np.sin(ang[9, 5]), atol=1e-6)


@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 128), (128, 32), (256, 64)])
def test_layout_holds_every_code_once(D, group):
    geo = o.Geometry(1, 1, D, group, 32, 1)
    seen = {}
    for t in range(32):
        for d in range(D):
            for at, what in ((o.key_at(geo, t, d), "k"), (o.value_at(geo, t, d), "v")):
                assert at not in seen
                seen[at] = (what, t, d)
    assert len(seen) == 2 * 32 * D and {a for a, _ in seen} == set(range(32 * D))
    # no byte of the codes holds two tokens
    for (a, s), (what, t, d) in seen.items():
        assert seen[(a, 4 - s)][1] == t


def test_store_and_load_give_the_quantized_values():
    rng = np.random.default_rng(5)
    geo = o.Geometry(4, 2, 128, 64, 64, 3)
    cache = rng.integers(0, 256, geo.bytes, dtype=np.uint8)
    k, v = (rng.normal(size=(70, 2, 128)).astype(np.float32) for _ in range(2))
    table = np.array([[2, 0, 7]], np.int32)
    o.append(geo, cache, table, [70], [0, 70], k, v)
    for h in range(2):
        K, V = o.gather(geo, cache, table[0], h, 70)
        for x, y in ((k, K), (v, V)):
            c, s, z = o.quantize_rows(x[:, h], 64)
            want = (c.astype(np.float64) - np.repeat(z.astype(np.float64), 64, -1)) * np.repeat(s.astype(np.float64), 64, -1)
            assert (y == want).all()


def test_attention_closed_forms():
    K = np.zeros((3, 64))
    V = np.arange(3.0)[:, None] * np.ones((3, 64))
    out, lse, _, _ = o.attention_row(np.ones(64), K, V, np.array([True, True, True]), 1.0)
    assert np.allclose(out, 1.0) and np.isclose(lse, np.log(3))
    out, lse, _, _ = o.attention_row(np.ones(64), K, V, np.array([False, False, True]), 1.0)
    assert np.allclose(out, 2.0) and np.isclose(lse, 0.0)
    out, lse, _, _ = o.attention_row(np.ones(64), K, V, np.zeros(3, bool), 1.0)
    assert (out == 0).all() and lse == -np.inf
