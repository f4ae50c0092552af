"""Plain CPU oracle of the operators between a decoder layer's products: the
RMS norm, the 4-bit key/value cache and the attention over it.  numpy, loops
and 64-bit arithmetic; shares no code with the GPU path.

The cache's quantization is defined in binary32 steps, each rounded once, so
`quantize_rows` and `rotate` follow those steps in numpy float32 and the
cache's bytes are comparable bit for bit; everything else is float64.
"""
import numpy as np

EPS16 = 2.0 ** -11       # half a unit in the last place of a normal fp16 value, relative
EPS32 = 2.0 ** -24


# ---- RMS norm ---------------------------------------------------------------

def rms_norm(x, residual, weight, eps):
    """(stream in x's dtype, y in float64)."""
    h = x if residual is None else (x.astype(np.float64) + residual.astype(np.float64)).astype(x.dtype)
    h64, w64 = h.astype(np.float64), weight.astype(np.float64)
    norm = np.sqrt((h64 * h64).mean(axis=1, keepdims=True) + eps)
    return h, h64 / norm * w64


def norm_codes(h, weight, eps):
    """(scales, exact quotients y / s) in float64; a zero row has quotients 0."""
    h64, w64 = h.astype(np.float64), weight.astype(np.float64)
    p = h64 * w64
    top = np.abs(p).max(axis=1)
    norm = np.sqrt((h64 * h64).mean(axis=1) + eps)
    q = np.divide(127.0 * p, top[:, None], out=np.zeros_like(p), where=top[:, None] > 0)
    return top / norm / 127.0, q


# ---- quantization and rotation ----------------------------------------------

def rotate(x, pos, cos, sin, rot, interleaved=False):
    """x [T, H, D] float32 rotated by row pos of cos and sin, in binary32 steps."""
    x = x.astype(np.float32).copy()
    if rot == 0:
        return x
    p = np.clip(pos, 0, cos.shape[0] - 1)
    c, s = cos[p][:, None, :], sin[p][:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2].copy(), x[..., 1:rot:2].copy()
        x[..., 0:rot:2] = a * c - b * s
        x[..., 1:rot:2] = b * c + a * s
    else:
        h = rot // 2
        a, b = x[..., :h].copy(), x[..., h:rot].copy()
        x[..., :h] = a * c - b * s
        x[..., h:rot] = b * c + a * s
    return x


def quantize_rows(x, group):
    """x [..., D] float32 to (codes u8 [..., D], scales fp16 [..., D/group], zero points u8)."""
    with np.errstate(all="ignore"):
        f32 = np.float32
        g = x.astype(f32).reshape(*x.shape[:-1], -1, group)
        bad = np.isnan(g).any(-1)
        lo = np.minimum(np.fmin.reduce(g, axis=-1), f32(0))
        hi = np.maximum(np.fmax.reduce(g, axis=-1), f32(0))
        lo, hi = np.where(np.isnan(lo), f32(0), lo), np.where(np.isnan(hi), f32(0), hi)
        s16 = ((hi - lo) * f32(1.0 / 15.0)).astype(np.float16)
        s16 = np.where(bad, np.float16(np.nan), s16)
        s = s16.astype(f32)
        fine = (s > 0) & np.isfinite(s)
        inv = np.where(fine, f32(1) / np.where(fine, s, f32(1)), f32(0)).astype(f32)
        z = np.where(fine, np.clip(np.rint(-lo * inv), 0, 15), f32(0)).astype(f32)
        t = np.rint(g * inv[..., None]) + z[..., None]
        c = np.fmin(np.fmax(t, f32(0)), f32(15))
    return c.astype(np.uint8).reshape(x.shape), s16, z.astype(np.uint8)


# ---- the cache's layout -----------------------------------------------------

class Geometry:
    def __init__(self, q_heads, kv_heads, D, group, page, num_pages):
        self.q_heads, self.kv_heads, self.D, self.group, self.page = q_heads, kv_heads, D, group, page
        self.G, self.num_pages = D // group, num_pages
        self.B = 32 * D + 256 * self.G
        self.bytes = num_pages * kv_heads * (page // 32) * self.B

    def base(self, page, head, in_page):
        return ((page * self.kv_heads + head) * (self.page // 32) + in_page // 32) * self.B


def key_at(geo, t, d):
    """(byte, shift) in a block of the key code of token t (0..31), dim d."""
    e, i = d // 8, d % 8
    w = (t // 16) * (geo.D // 32) + e // 4
    slot = (0, 4, 1, 5, 2, 6, 3, 7)[i]
    return 1024 * (w // 4) + 16 * (16 * (e % 4) + t % 16) + 4 * (w % 4) + slot // 2, 4 * (slot % 2)


def value_at(geo, t, d):
    at = (16 * geo.D + 1024 * (d // 64) + 16 * (16 * ((t % 16) // 4) + d % 16) + 8 * ((d // 32) % 2) +
          4 * (t // 16) + (0, 2, 1, 3)[t % 4])
    return at, 4 * ((d % 32) // 16)


def _index(geo):
    idx = getattr(geo, "_idx", None)
    if idx is None:
        k = np.array([[key_at(geo, t, d) for d in range(geo.D)] for t in range(32)])
        v = np.array([[value_at(geo, t, d) for d in range(geo.D)] for t in range(32)])
        idx = geo._idx = (k[..., 0], k[..., 1], v[..., 0], v[..., 1])
    return idx


def store(geo, cache, page, head, in_page, is_v, codes, scales, zeros):
    """One token's codes [D], scales [G] and zero points [G] into the bytes of `cache`."""
    ka, ks, va, vs = _index(geo)
    t = in_page % 32
    base = geo.base(page, head, in_page)
    at, sh = (va[t], vs[t]) if is_v else (ka[t], ks[t])
    for d in range(geo.D):
        a, s = base + at[d], int(sh[d])
        cache[a] = (int(cache[a]) & ~(15 << s)) & 255 | (int(codes[d]) << s)
    off = base + 32 * geo.D + (128 * geo.G if is_v else 0) + 4 * geo.G * t
    words = scales.view(np.uint16).astype(np.uint32) | (zeros.astype(np.uint32) << 16)
    cache[off:off + 4 * geo.G] = words.astype("<u4").view(np.uint8)


def load(geo, cache, page, head, in_page):
    """(K, V) [D] float64 of one stored token."""
    ka, ks, va, vs = _index(geo)
    t = in_page % 32
    base = geo.base(page, head, in_page)
    out = []
    for at, sh, off in ((ka[t], ks[t], 32 * geo.D), (va[t], vs[t], 32 * geo.D + 128 * geo.G)):
        c = (cache[base + at] >> sh.astype(np.uint8)) & 15
        w = cache[base + off + 4 * geo.G * t:base + off + 4 * geo.G * (t + 1)].copy().view("<u4")
        s = (w & 0xFFFF).astype(np.uint16).view(np.float16).astype(np.float64)
        z = ((w >> 16) & 15).astype(np.float64)
        with np.errstate(invalid="ignore"):
            out.append((c.astype(np.float64) - np.repeat(z, geo.group)) * np.repeat(s, geo.group))
    return out


def append(geo, cache, table, kv_len, q_start, k, v, cos=None, sin=None, rot=0, interleaved=False):
    """The new tokens' K and V into `cache`; returns the positions [T] (negative: none)."""
    T = k.shape[0]
    pos = positions(kv_len, q_start, T)
    kc = quantize_rows(rotate(k, pos, cos, sin, rot, interleaved), geo.group)
    vc = quantize_rows(v.astype(np.float32), geo.group)
    for b in range(len(kv_len)):
        for t in range(q_start[b], min(q_start[b + 1], T)):
            p = pos[t]
            if p < 0 or p // geo.page >= table.shape[1]:
                continue
            page = int(table[b, p // geo.page])
            if not 0 <= page < geo.num_pages:
                continue
            for h in range(geo.kv_heads):
                store(geo, cache, page, h, p % geo.page, False, kc[0][t, h], kc[1][t, h], kc[2][t, h])
                store(geo, cache, page, h, p % geo.page, True, vc[0][t, h], vc[1][t, h], vc[2][t, h])
    return pos


def positions(kv_len, q_start, T):
    pos = np.full(T, -1, np.int64)
    for b in range(len(kv_len)):
        for t in range(q_start[b], min(q_start[b + 1], T)):
            pos[t] = int(kv_len[b]) - (q_start[b + 1] - t)
    return pos


def gather(geo, cache, table_row, head, n):
    """Keys and values [n, D] of one sequence and head, float64."""
    rows = [load(geo, cache, int(table_row[p // geo.page]), head, p % geo.page) for p in range(n)]
    if not rows:
        return np.zeros((0, geo.D)), np.zeros((0, geo.D))
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


# ---- attention --------------------------------------------------------------

def attention_row(q, K, V, seen, scale):
    """(out [D], lse, sum_j p_j |V_j| [D], largest |logit| bound over seen keys) of one query, float64."""
    if not seen.any():
        return np.zeros(K.shape[1]), -np.inf, np.zeros(K.shape[1]), 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        x = scale * (K[seen] @ q)
        reach = abs(scale) * (np.abs(K[seen]) @ np.abs(q)).max()
        m = x.max()
        p = np.exp(x - m)
        total = p.sum()
        p /= total
        return p @ V[seen], m + np.log(total), p @ np.abs(V[seen]), reach


def attention(geo, cache, table, kv_len, q_start, q, scale, causal=True, window=0, max_kv=None, sinks=0):
    """out [T, H, D], lse [T, H], absolute bounds sum p|V| [T, H, D] and logit reach [T, H]; with a window the keys
    below `sinks` stay visible."""
    T, H, D = q.shape
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    size, reach = np.zeros((T, H, D)), np.zeros((T, H))
    per = geo.q_heads // geo.kv_heads
    for b in range(len(kv_len)):
        n, first, end = int(kv_len[b]), q_start[b], q_start[b + 1]
        n = max(0, min(n, table.shape[1] * geo.page, n if max_kv is None else max_kv))
        for h in range(geo.kv_heads):
            K, V = gather(geo, cache, table[b], h, n)
            j = np.arange(n)
            for t in range(first, end):
                p = n - (end - t)
                seen = j < n
                if causal:
                    seen = j <= p
                    if window > 0:
                        seen &= (j > p - window) | (j < sinks)
                for g in range(h * per, (h + 1) * per):
                    out[t, g], lse[t, g], size[t, g], reach[t, g] = attention_row(
                        q[t, g].astype(np.float64), K, V, seen, scale)
    return out, lse, size, reach


def attention_tolerance(size, reach, keys, D, f16, values_max):
    """Bound of |kernel - exact| per output.

    A logit is a sum of D products, exact operands, summed in fp32: its error is
    at most (D + 8) 2^-24 reach (D additions, the scales and the factor), and the
    exponential adds 2 ulp.  A weight p_j / sum is then off by a factor of at
    most 1 + 4 (D + 8) 2^-24 reach + 8 2^-24, and the sums over the keys by
    another (keys + 64) 2^-24.  The product p s' is rounded to fp16: below its
    normal range by 2^-25 absolute, with the running reference at least 2^10
    below the largest, so by 2^-35 of it a key, codes up to 15: together at
    most keys 2^-34 of the largest value; in fp16 calls also by 2^-11 relative, as
    is the output (2^-25 absolute below the normal range)."""
    rel = 4.0 * (D + 8) * EPS32 * reach + 8 * EPS32 + (keys + 64) * EPS32
    tol = size * rel[..., None] + keys * 2.0 ** -34 * values_max
    if f16:
        tol = tol + size * 2 * EPS16 * 1.001 + 2.0 ** -25
    return tol


def lse_tolerance(lse, reach, keys, D):
    """The largest logit's error, the sum's relative error, and the logarithm's and the result's roundings."""
    return 2.0 * (D + 8) * EPS32 * reach + (keys + 64) * EPS32 + 4 * EPS32 * (1 + np.abs(lse))
