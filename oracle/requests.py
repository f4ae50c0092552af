"""Plain CPU oracle of the operators that serve many requests at once: low-rank
adapters beside a projection, and the verification of drafted tokens.  numpy, loops
and 64-bit arithmetic; shares no code with the GPU path.
"""
import numpy as np

EPS16, EPS32 = 2.0 ** -11, 2.0 ** -24


# ---- adapters ---------------------------------------------------------------

def adapters(a, b, scales, ranks, adapter, x, base):
    """y [m, n] in float64 and its bound |kernel - y|, for operands of fp16 or fp32.

    h is a sum of k products in fp32, a product rounded once in fp32 calls: off by at
    most (2 k + 32) 2^-24 sum |a x|.  In fp16 calls h enters the second product as two fp16
    parts of its sign, the row scaled to a largest in [2^15, 2^16): the first cut off to 11 bits, at most an ulp (2^-10
    relative) below, the second rounded to 11 bits: 2^-22 relative.  Neither is less than 2^-24, so the two of a
    smaller h are off by at most 2^-23, 2^-38 of the row's largest.  That
    product has rank terms (each twice in fp16 calls) and is scaled in two steps: (4 rank +
    32) 2^-24 of the sum of magnitudes.  The output is rounded once, to 2^-11 (2^-25
    absolute below fp16's normal range) or 2^-24, after its addition to base."""
    f16 = x.dtype == np.float16
    m, n = x.shape[0], b.shape[1]
    y = np.zeros((m, n)) if base is None else base.astype(np.float64)
    tol = np.zeros((m, n))
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(m):
            g = int(adapter[t])
            if not 0 <= g < a.shape[0]:
                continue
            r = a.shape[1] if ranks is None else min(int(ranks[g]), a.shape[1])
            if r <= 0:
                continue
            s = 1.0 if scales is None else float(scales[g])
            A, B, v = a[g, :r].astype(np.float64), b[g, :, :r].astype(np.float64), x[t].astype(np.float64)
            h = A @ v
            eh = (2 * x.shape[1] + 32) * EPS32 * (np.abs(A) @ np.abs(v))
            part = np.abs(h) * ((2.0 ** -22 if f16 else 0) + (4 * r + 32) * EPS32) + eh
            if f16:
                part = part + 2.0 ** -38 * np.abs(h).max()
            y[t] += s * (B @ h)
            tol[t] = abs(s) * (np.abs(B) @ part)
            tol[t] += (np.abs(y[t]) + tol[t]) * (EPS16 if f16 else EPS32) * 1.001 + (2.0 ** -25 if f16 else 2.0 ** -149)
            if not f16:
                tol[t] += EPS32 * abs(s) * (np.abs(B) @ np.abs(h))
    return y, tol


# ---- drafted tokens ---------------------------------------------------------

def _weights(row):
    w = row.astype(np.float64)
    return np.where(np.isfinite(w) & (w > 0), w, 0.0)


def draw(w, pick):
    """The lowest i with w[0] + .. + w[i] > pick * sum w; the last with a weight where none has; -1 without any."""
    if not (w > 0).any():
        return -1
    sums = np.cumsum(w)
    u = float(pick) if pick > 0 else 0.0
    over = np.nonzero((sums > u * sums[-1]) & (w > 0))[0]
    return int(over[0]) if len(over) and u < 1 else int(np.nonzero(w > 0)[0][-1])


def verify(target, draft, ids, q_start, accept, pick, out):
    """(out with the sequences' rows replaced, accepted [batch])."""
    out = out.copy()
    batch, tokens, vocab = len(pick), target.shape[0], target.shape[1]
    counts = np.zeros(batch, np.int32)
    for b in range(batch):
        first, end = (b, b + 1) if q_start is None else (max(0, int(q_start[b])), min(tokens, int(q_start[b + 1])))
        if end <= first:
            continue
        n = 0
        while first + n + 1 < end:
            row, d = first + n, int(ids[first + n + 1])
            if not 0 <= d < vocab:
                break
            p = _weights(target[row, d:d + 1])[0]
            q = 1.0 if draft is None else _weights(draft[row, d:d + 1])[0]
            if not float(accept[row]) * q < p:
                break
            n += 1
        row = first + n
        w = _weights(target[row])
        if row + 1 < end:
            if draft is None:
                rest = w.copy()
                if 0 <= ids[row + 1] < vocab:
                    rest[ids[row + 1]] = 0
            else:
                rest = np.maximum(w - _weights(draft[row]), 0)
            if (rest > 0).any():
                w = rest
        out[first:end] = -1
        out[first:row] = ids[first + 1:row + 1]
        out[row] = draw(w, pick[b])
        counts[b] = n
    return out, counts
