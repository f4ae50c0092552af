"""The oracle of the adapters and of the verification against their definitions by other routes.  No GPU."""
from fractions import Fraction

import numpy as np

from oracle import requests as o


def test_adapters_are_the_merged_weights():
    """base + s B A x is the product with W + s B A."""
    rng = np.random.default_rng(1)
    a, b = rng.normal(size=(3, 4, 20)).astype(np.float32), rng.normal(size=(3, 9, 4)).astype(np.float32)
    w, x = rng.normal(size=(9, 20)), rng.normal(size=(5, 20)).astype(np.float32)
    s, ranks = np.array([0.5, 2.0, -1.0], np.float32), np.array([4, 2, 9])
    which = np.array([0, 2, -1, 1, 3])
    y, tol = o.adapters(a, b, s, ranks, which, x, (x.astype(np.float64) @ w.T))
    for t, g in enumerate(which):
        merged = w.copy()
        if 0 <= g < 3:
            merged = w + float(s[g]) * b[g, :, :ranks[g]].astype(float) @ a[g, :min(4, ranks[g])].astype(float)
        assert np.allclose(y[t], merged @ x[t].astype(float), rtol=1e-12)
        assert (tol[t] > 0).all() if 0 <= g < 3 else (tol[t] == 0).all()


def _shares(p, q, steps):
    """How often each first token comes out over all (draft, accept, pick) on a grid, a draft weighted by q."""
    got = [Fraction(0)] * len(p)
    target, draft = np.array([p, p], np.float32), np.array([q, q], np.float32)
    for d in range(len(q)):
        for i in range(steps):
            for j in range(steps):
                u, r = (i + 0.5) / steps, (j + 0.5) / steps
                out, n = o.verify(target, draft, np.array([7, d], np.int32), [0, 2], np.array([u, 0], np.float32),
                                  np.array([r], np.float32), np.full(2, 99, np.int32))
                assert n[0] in (0, 1) and (out[0] == d or n[0] == 0) and (out[1] == -1) == (n[0] == 0)
                got[out[0]] += Fraction(q[d]) / (steps * steps)
    return got


def test_the_first_token_is_distributed_as_the_target():
    p, q = [1 / 16, 5 / 16, 8 / 16, 2 / 16], [4 / 16, 4 / 16, 4 / 16, 4 / 16]
    for have, want in zip(_shares(p, q, 24), p):
        assert abs(float(have) - want) <= 2 / 24


def test_draws_by_hand():
    w = np.array([0, 0.25, 0, 0.5, 0.25, 0])
    for pick, token in ((0.0, 1), (0.2499, 1), (0.25, 3), (0.74, 3), (0.75, 4), (0.999, 4), (1.0, 4), (7.0, 4),
                        (-1.0, 1), (float("nan"), 1)):
        assert o.draw(w, pick) == token, pick
    assert o.draw(np.zeros(3), 0.5) == -1


def test_certain_drafts_and_bad_values():
    t = np.array([[0.5, 0.5, np.nan], [np.inf, -1.0, 0.25]], np.float32)
    out, n = o.verify(t, None, np.array([0, 1], np.int32), [0, 2], np.array([0.6, 0.0], np.float32),
                      np.array([0.9], np.float32), np.zeros(2, np.int32))
    assert n[0] == 0 and list(out) == [0, -1]          # refused: drawn from p without token 1
    out, n = o.verify(t, None, np.array([0, 1], np.int32), [0, 2], np.array([0.4, 0.0], np.float32),
                      np.array([0.0], np.float32), np.zeros(2, np.int32))
    assert n[0] == 1 and list(out) == [1, 2]
