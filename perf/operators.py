"""Cases and plain forms of the operators between a decoder's int4 products:
the RMS norm with the residual's addition, keys and values appended to a
paged 4-bit cache, and the attention that reads that cache.

`run` computes an operator in elementary torch operations, in 32 bits, or,
where `own` is true, by the library's own call.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # the norm before a projection, one token: latency
        dict(name="norm, one token", op="norm", m=1, k=4096, dtype="f16", codes=False),
        # speculative verify or a small batch: 8-bit codes for the products on int8 activations
        dict(name="norm to codes, 16 rows", op="norm", m=16, k=4096, dtype="f16", codes=True),
        # prompts of a whole batch
        dict(name="norm, 8192 rows", op="norm", m=8192, k=4096, dtype="f16", codes=False),
        # fp32 activations at the width of a feed-forward layer, an odd row count, to codes
        dict(name="norm to codes, fp32", op="norm", m=1023, k=11008, dtype="f32", codes=True),
        # one new token of each of 16 sequences
        dict(name="append, one token each", op="append", batch=16, new=1, past=2000, q_heads=32, kv_heads=8, dim=128,
             group=128, page=64, rotary=128, dtype="f16"),
        # three prompts of uneven length
        dict(name="append, prompts", op="append", batch=3, new=4096, past=0, q_heads=32, kv_heads=8, dim=128,
             group=64, page=64, rotary=128, dtype="f16"),
        # one sequence, one token: what a chat with one user waits for
        dict(name="attend, one sequence", op="attend", batch=1, new=1, kv=1000, q_heads=32, kv_heads=8, dim=128,
             group=128, page=64, window=0, dtype="f16"),
        # a serving batch of uneven lengths
        dict(name="attend, batch of 32", op="attend", batch=32, new=1, kv=8192, q_heads=32, kv_heads=8, dim=128,
             group=128, page=64, window=0, dtype="f16"),
        # a long document, one token
        dict(name="attend, long cache", op="attend", batch=1, new=1, kv=131072, q_heads=32, kv_heads=8, dim=128,
             group=64, page=256, window=0, dtype="f16"),
        # speculative verify in fp32, small heads, fine groups, a sliding window
        dict(name="attend, verify fp32", op="attend", batch=8, new=5, kv=4100, q_heads=24, kv_heads=8, dim=64,
             group=32, page=32, window=3000, dtype="f32"),
        # prompt chunks behind a cached prefix
        dict(name="attend, prompt chunks", op="attend", batch=2, new=2048, kv=4096, q_heads=32, kv_heads=8, dim=128,
             group=128, page=64, window=0, dtype="f16"),
        # one key head per query head (the 7B shape), a prompt without a prefix
        dict(name="attend, prompt, 32 kv heads", op="attend", batch=1, new=1000, kv=1000, q_heads=32, kv_heads=32,
             dim=128, group=128, page=64, window=0, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "append", "attend", "attend", "attend"])
    dtype = rng.choice(["f16", "f16", "f32"])
    if op == "norm":
        m = _log_int(rng, 1, 8192)
        k = _log_int(rng, 64, min(20000, 33_000_000 // m))
        if rng.random() < 0.7:
            k = max(16, k // 16 * 16)
        return dict(op=op, m=m, k=k, dtype=dtype, codes=rng.random() < 0.5)
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    heads = dict(q_heads=kv_heads * rng.choice([1, 2, 3, 4, 6, 8]), kv_heads=kv_heads, dim=dim,
                 group=rng.choice([g for g in (32, 64, 128) if g <= dim]), page=rng.choice([32, 64, 128, 256]))
    batch = _log_int(rng, 1, 32)
    if op == "append":
        new = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4096)
        while batch * new * heads["q_heads"] * dim > 3 * 4096 * 32 * 128:
            new = (new + 1) // 2
        return dict(op=op, batch=batch, new=new, past=rng.randint(0, 3000), **heads,
                    rotary=rng.choice([dim, dim, dim // 2, 0]), dtype=dtype)
    new = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, 2048)])
    kv = max(new, _log_int(rng, 64, 65536))
    while batch * kv * kv_heads * dim > 32 * 8192 * 8 * 128 or \
            batch * new * kv * heads["q_heads"] * dim > 2048 * 4096 * 32 * 128:
        batch, kv, new = max(1, batch // 2), max(1, kv * 3 // 4), max(1, new * 3 // 4)
        kv = max(kv, new)
    return dict(op=op, batch=batch, new=new, kv=kv, **heads, window=rng.choice([0, 0, 0, rng.randint(1, 4096)]),
                dtype=dtype)


def _spread(n, most, least):
    """n lengths in least..most, uneven, the first the longest."""
    return [max(least, most - int((most - least) * 0.75 * ((0.6180339887 * i) % 1.0))) for i in range(n)]


def _lengths(c):
    """(new tokens, cached tokens with them) of each sequence."""
    new = _spread(c["batch"], c["new"], 1)
    if c["op"] == "append":
        return new, [n + c["past"] + 7 * i for i, n in enumerate(new)]
    return new, [max(n, s) for n, s in zip(new, _spread(c["batch"], c["kv"], c["new"]))]


def _pairs(c):
    """(query, key) pairs that the masks leave, and keys that any query of its sequence sees."""
    pairs = keys = 0
    for n, s in zip(*_lengths(c)):
        first = s - n
        w = c["window"] if c["window"] > 0 else s
        pairs += sum(min(w, first + i + 1) for i in range(n))
        keys += s - max(0, first + 1 - w)
    return pairs, keys


def work(c):
    e = 2 if c["dtype"] == "f16" else 4
    if c["op"] == "norm":
        n = c["m"] * c["k"]
        out = 2 * n + 4 * c["m"] if c["codes"] else e * n
        return {"bytes": 3 * e * n + out + e * c["k"], "flops": 6 * n}
    D, H, Hkv = c["dim"], c["q_heads"], c["kv_heads"]
    token = Hkv * 2 * (D // 2 + 4 * (D // c["group"]))  # bytes of a cached token
    new = sum(_lengths(c)[0])
    if c["op"] == "append":  # q, k, v in, q out, the cache written and read, the values out
        return {"bytes": new * (2 * e * H * D + 4 * e * Hkv * D + 2 * token), "flops": new * (H + 2 * Hkv) * D * 6}
    pairs, keys = _pairs(c)
    return {"bytes": keys * token + 2 * e * new * H * D, "flops": 4 * pairs * H * D}


# ---- inputs -----------------------------------------------------------------

def _dtype(c):
    return torch.float16 if c["dtype"] == "f16" else torch.float32


def _block_bytes(c):
    return 32 * c["dim"] + 256 * (c["dim"] // c["group"])


def _cache(c, pages, gen):
    """A cache as it is after such keys and values were appended: codes about their zero points."""
    D, NG, H = c["dim"], c["dim"] // c["group"], c["kv_heads"]
    nb = pages * H * (c["page"] // 32)
    raw = torch.empty(nb, 2 * 32 * D, dtype=torch.float16, device=DEV).normal_(generator=gen)
    raw = (raw * 2.4 + 7.5).round().clamp_(0, 15).to(torch.uint8)
    codes = raw[:, 0::2] | (raw[:, 1::2] << 4)
    del raw
    s = torch.randn(nb, 2, 32 * NG, device=DEV, generator=gen).mul_(0.3).exp_()
    s[:, 0] *= 0.35
    s[:, 1] *= 0.15
    z = (torch.randn(nb, 2, 32 * NG, device=DEV, generator=gen) + 7.5).round().clamp(0, 15).to(torch.int32)
    meta = (s.half().view(torch.int16).to(torch.int32) & 0xFFFF) | (z << 16)
    return torch.cat([codes, meta.view(torch.uint8).reshape(nb, 256 * NG)], 1).reshape(-1)


def _tables(c, gen):
    """Page table, lengths and query offsets of the sequences, and the number of pages; pages in random order."""
    new, total = _lengths(c)
    need = [-(-s // c["page"]) for s in total]
    order = torch.randperm(sum(need), generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(c["batch"], max(need), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    q_start = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    return table, torch.tensor(total, dtype=torch.int32, device=DEV), q_start, sum(need)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device=DEV, generator=gen)

    t = _dtype(c)
    s = {"case": c}
    if c["op"] == "norm":
        m, k = c["m"], c["k"]
        # a residual stream has a few channels far larger than the rest
        gain = torch.ones(k, device=DEV)
        gain[torch.randint(0, k, (max(1, k // 500),), device=DEV, generator=gen)] = 12.0
        s.update(x=randn(m, k).to(t), residual=(randn(m, k) * gain).to(t), weight=(randn(k) * 0.1 + 1.0).to(t),
                 stream=torch.empty(m, k, dtype=t, device=DEV),
                 out=torch.empty(m, k, dtype=torch.float16 if c["codes"] else t, device=DEV),
                 scales=torch.empty(m, device=DEV) if c["codes"] else None)
        return s
    D, H, Hkv = c["dim"], c["q_heads"], c["kv_heads"]
    table, kv_len, q_start, pages = _tables(c, gen)
    new, total = _lengths(c)
    T = sum(new)
    s.update(table=table, kv_len=kv_len, q_start=q_start, pages=pages, tokens=T, max_new=max(new), max_kv=max(total))
    if c["op"] == "append":
        # slices of the output of one projection: their tokens are (H + 2 Hkv) D apart
        qkv = randn(T, H + 2 * Hkv, D).to(t)
        rows = max(total)
        ang = torch.arange(rows, device=DEV)[:, None] * \
            (10000.0 ** (-torch.arange(max(1, c["rotary"] // 2), device=DEV) * 2.0 / max(2, c["rotary"])))[None]
        s.update(q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:], cos=ang.cos().contiguous(),
                 sin=ang.sin().contiguous(),
                 cache=torch.zeros(pages * Hkv * (c["page"] // 32) * _block_bytes(c), dtype=torch.uint8, device=DEV),
                 q_out=torch.empty(T, H, D, dtype=t, device=DEV), k_out=torch.empty(T, Hkv, D, dtype=t, device=DEV),
                 v_out=torch.empty(T, Hkv, D, dtype=t, device=DEV))
        return s
    s.update(cache=_cache(c, pages, gen), q=(randn(T, H, D) * 1.5).to(t),
             out=torch.empty(T, H, D, dtype=t, device=DEV),
             workspace=torch.empty(192 << 20, dtype=torch.uint8, device=DEV))
    return s


# ---- the operators ----------------------------------------------------------

def _kv_desc(mnb, c, pages):
    return mnb.kv4_desc(c["q_heads"], c["kv_heads"], c["dim"], c["group"], c["page"], pages)


def _run_own(s):
    from block_wise_int4_amd import mnb
    c = s["case"]
    if c["op"] == "norm":
        mnb.mnb_rms_norm(s["x"], s["weight"], s["out"], EPS, residual=s["residual"], residual_out=s["stream"],
                         scales=s["scales"])
        if c["codes"]:
            return {"stream": s["stream"], "codes": s["out"], "scales": s["scales"]}
        return {"stream": s["stream"], "y": s["out"]}
    d = _kv_desc(mnb, c, s["pages"])
    if c["op"] == "append":
        rot = c["rotary"]
        mnb.mnb_kv4_append(d, s["cache"], s["k"], s["v"], s["table"], s["kv_len"], s["q_start"],
                           cos=s["cos"] if rot else None, sin=s["sin"] if rot else None, rotary_dim=rot, q=s["q"],
                           q_out=s["q_out"])
        mnb.mnb_kv4_read(d, s["cache"], s["table"], s["kv_len"], s["q_start"], s["k_out"], s["v_out"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    mnb.mnb_attention_kv4(d, s["cache"], s["q"], s["table"], s["kv_len"], s["q_start"], s["max_new"], s["max_kv"],
                          s["out"], _scale(c), causal=True, window=c["window"], workspace=s["workspace"])
    return s["out"]


def _scale(c):
    return 1.0 / math.sqrt(c["dim"])


def _plain_norm(s):
    c = s["case"]
    stream = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    h = stream.float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    if not c["codes"]:
        return {"stream": stream, "y": y.to(s["x"].dtype)}
    scales = y.abs().amax(1) / 127.0
    q = y / torch.where(scales == 0, torch.ones_like(scales), scales)[:, None]
    q = torch.sign(q) * torch.floor(q.abs() + 0.5)
    return {"stream": stream, "codes": q.half(), "scales": scales}


def _positions(s):
    """Position and sequence of each new token."""
    tok = torch.arange(s["tokens"], device=DEV)
    seq = (tok[:, None] >= s["q_start"][None, 1:]).sum(1)
    return tok - s["q_start"][seq + 1] + s["kv_len"][seq], seq


def _plain_rotate(x, cos, sin, rot):
    if rot == 0:
        return x
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)


def _plain_quantized(x, group):
    """x as the values that its 4-bit codes stand for."""
    g = x.reshape(*x.shape[:-1], -1, group)
    lo, hi = g.amin(-1, keepdim=True).clamp_max(0.0), g.amax(-1, keepdim=True).clamp_min(0.0)
    scale = ((hi - lo) * (1.0 / 15.0)).half().float()
    inv = torch.where(scale == 0, torch.zeros_like(scale), torch.ones_like(scale) / scale)
    zero = (-lo * inv).round().clamp(0.0, 15.0)
    code = ((g * inv).round() + zero).clamp(0.0, 15.0)
    return ((code - zero) * scale).reshape(x.shape)


def _plain_append(s):
    c, rot = s["case"], s["case"]["rotary"]
    pos, _ = _positions(s)
    cos, sin = s["cos"][pos][:, None, :], s["sin"][pos][:, None, :]
    t = s["q"].dtype
    q = _plain_rotate(s["q"].float(), cos, sin, rot).to(t)
    k = _plain_quantized(_plain_rotate(s["k"].float(), cos, sin, rot), c["group"]).to(t)
    return {"q": q, "k": k, "v": _plain_quantized(s["v"].float(), c["group"]).to(t)}


def _plain_cache(s):
    """Keys and values of every sequence, [batch, kv heads, table's tokens, dim], in 32 bits."""
    c = s["case"]
    D, NG, H, nblk = c["dim"], c["dim"] // c["group"], c["kv_heads"], c["page"] // 32
    blk = s["cache"].view(s["pages"], H, nblk, _block_bytes(c))[s["table"].long()]      # [B, P, H, nblk, bytes]
    B, P = blk.shape[:2]
    slot = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=DEV)
    byte = torch.tensor([0, 2, 1, 3], device=DEV)

    def values(codes, meta):  # codes and meta: [B, P, H, nblk, 32, D] and int32 [B, P, H, nblk, 32, NG]
        scale = (meta & 0xFFFF).to(torch.int16).view(torch.float16).float()
        zero = ((meta >> 16) & 15).float()
        x = codes.float().reshape(B, P, H, nblk, 32, NG, c["group"])
        x = (x - zero[..., None]) * scale[..., None]
        return x.reshape(B, P, H, nblk, 32, D).permute(0, 2, 1, 3, 4, 5).reshape(B, H, P * nblk * 32, D)

    kw = blk[..., :16 * D].contiguous().view(torch.int32).reshape(B, P, H, nblk, D // 64, 4, 16, 4)
    kc = ((kw[..., None] >> slot) & 15).to(torch.uint8)            # [.., quad, q, key, word, i]
    kc = kc.permute(0, 1, 2, 3, 4, 7, 5, 6, 8)                     # [.., quad, word, q, key, i]
    kc = kc.reshape(B, P, H, nblk, 2, D // 32, 4, 16, 8).permute(0, 1, 2, 3, 4, 7, 5, 6, 8)
    kc = kc.reshape(B, P, H, nblk, 32, D)                          # from [.., tile, key, j, q, i]
    km = blk[..., 32 * D:32 * D + 128 * NG].contiguous().view(torch.int32).reshape(B, P, H, nblk, 32, NG)
    keys = values(kc, km)
    del kw, kc
    vb = blk[..., 16 * D:32 * D].reshape(B, P, H, nblk, D // 64, 4, 16, 2, 2, 4)[..., byte]
    vc = torch.stack([vb & 15, vb >> 4], -1)                       # [.., quad, q, d, pair, half, i, nibble]
    vc = vc.permute(0, 1, 2, 3, 8, 5, 9, 4, 7, 10, 6)              # [.., half, q, i, quad, pair, nibble, d]
    vm = blk[..., 32 * D + 128 * NG:].contiguous().view(torch.int32).reshape(B, P, H, nblk, 32, NG)
    return keys, values(vc.reshape(B, P, H, nblk, 32, D), vm)


def _plain_attend(s):
    c = s["case"]
    D, H, Hkv, B, N = c["dim"], c["q_heads"], c["kv_heads"], c["batch"], s["max_new"]
    keys, vals = _plain_cache(s)
    S = keys.shape[2]
    pos, seq = _positions(s)
    at = torch.arange(s["tokens"], device=DEV) - s["q_start"][seq]
    q = torch.zeros(B, N, Hkv, H // Hkv, D, device=DEV)
    q[seq, at] = s["q"].float().reshape(-1, Hkv, H // Hkv, D)
    where = torch.full((B, N), -1, dtype=torch.long, device=DEV)
    where[seq, at] = pos.long()
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D), keys.transpose(2, 3)) * _scale(c)
    key = torch.arange(S, device=DEV)
    seen = key <= where[..., None]                                 # [B, N, S]; a key past the length is past every query
    if c["window"] > 0:
        seen &= key > where[..., None] - c["window"]
    x = x.reshape(B, Hkv, N, H // Hkv, S).masked_fill_(~seen[:, None, :, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp_min(-3e38)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    vals = vals.masked_fill(key[None, None, :, None] >= s["kv_len"][:, None, None, None], 0.0)
    o = torch.matmul(p.reshape(B, Hkv, -1, S), vals).reshape(B, Hkv, N, H // Hkv, D)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(0, 2, 1, 3, 4)[seq, at].reshape(-1, H, D).to(s["q"].dtype)


def run(s):
    if own:
        return _run_own(s)
    return {"norm": _plain_norm, "append": _plain_append, "attend": _plain_attend}[s["case"]["op"]](s)


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_norm(s):
    c, t = s["case"], s["x"].dtype
    stream = (s["x"].double() + s["residual"].double()).to(t)
    h, w = stream.double(), s["weight"].double()
    norm = (h.pow(2).sum(1) / c["k"] + EPS).sqrt()
    y = h * w / norm[:, None]
    if not c["codes"]:
        return {"stream": stream, "y": y}
    top = (h * w).abs().amax(1)
    q = torch.where(top[:, None] > 0, 127.0 * (h * w) / top[:, None].clamp_min(1e-300), torch.zeros_like(y))
    return {"stream": stream, "codes": torch.trunc(q + 0.5 * torch.sign(q)), "scales": top / norm / 127.0}


def _exact_append(s):
    c = s["case"]
    rot, G = c["rotary"], c["group"]
    total = [int(v) for v in s["kv_len"]]
    start = [int(v) for v in s["q_start"]]
    pos = torch.cat([torch.arange(n - (e - b), n) for n, b, e in zip(total, start[:-1], start[1:])]).to(DEV)

    def rotated(x):
        x = x.double()
        if not rot:
            return x
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous())
        z = z * torch.complex(s["cos"][pos].double(), s["sin"][pos].double())[:, None]
        return torch.cat([z.real, z.imag, x[..., rot:]], -1)

    def quantized(x):
        g = x.unflatten(-1, (-1, G))
        lo, hi = g.min(-1)[0].clamp(max=0), g.max(-1)[0].clamp(min=0)
        sc = ((hi - lo) / 15).to(torch.float16).double()
        safe = torch.where(sc > 0, sc, torch.ones_like(sc))
        z = torch.where(sc > 0, torch.round(-lo / safe), torch.zeros_like(sc)).clamp(0, 15)
        n = torch.where((sc > 0)[..., None], torch.round(g / safe[..., None]), torch.zeros_like(g))
        return (torch.minimum(torch.maximum(n, -z[..., None]), 15 - z[..., None]) * sc[..., None]).flatten(-2)

    return {"q": rotated(s["q"]), "k": quantized(rotated(s["k"])), "v": quantized(s["v"].double())}


def _exact_rows(s, b, h, n):
    """Keys and values [n, dim] of a sequence and head in 64 bits, each code fetched from its byte."""
    c = s["case"]
    D, G, nblk = c["dim"], c["group"], c["page"] // 32
    NG, size = D // G, _block_bytes(c)
    j = torch.arange(n, device=DEV)
    page = s["table"][b].long()[j // c["page"]]
    base = ((page * c["kv_heads"] + h) * nblk + j % c["page"] // 32) * size
    j, d = (j % 32)[:, None], torch.arange(D, device=DEV)[None]
    # keys: word (tile, d / 32) of lane (d / 8 % 4, key % 16), nibble slot of d % 8
    w = j // 16 * (D // 32) + d // 32
    at = base[:, None] + w // 4 * 1024 + (d // 8 % 4 * 16 + j % 16) * 16 + w % 4 * 4
    bit = (d % 8 // 2 + d % 2 * 4) * 4
    kc = (s["cache"][at + bit // 8].long() >> (bit % 8)) & 15
    # values: 32 dims a pair of 16-dim tiles, low and high nibble; lane (key % 16 / 4, d % 16), word key / 16, byte of key % 4
    u = d // 32
    byte = (j % 4 & 1) * 2 + (j % 4 >> 1)
    at = base[:, None] + 16 * D + u // 2 * 1024 + (j % 16 // 4 * 16 + d % 16) * 16 + u % 2 * 8 + j // 16 * 4 + byte
    vc = (s["cache"][at].long() >> (d // 16 % 2 * 4)) & 15

    def value(code, off):
        at = (base[:, None] + off + (j * NG + d // G) * 4)
        lo, hi, z = s["cache"][at].int(), s["cache"][at + 1].int(), s["cache"][at + 2].long() & 15
        sc = (lo | (hi << 8)).to(torch.int16).view(torch.float16).double()
        return (code - z) * sc

    return value(kc, 32 * D), value(vc, 32 * D + 128 * NG)


def _exact_attend(s):
    c = s["case"]
    H, Hkv = c["q_heads"], c["kv_heads"]
    out = torch.zeros(s["tokens"], H, c["dim"], dtype=torch.float64, device=DEV)
    start, total = s["q_start"].tolist(), s["kv_len"].tolist()
    for b in range(c["batch"]):
        n, N = total[b], start[b + 1] - start[b]
        i, key = torch.arange(n - N, n, device=DEV)[:, None], torch.arange(n, device=DEV)[None]
        hidden = key > i
        if c["window"] > 0:
            hidden = hidden | (i - key >= c["window"])
        for h in range(Hkv):
            k, v = _exact_rows(s, b, h, n)
            for g in range(h * H // Hkv, (h + 1) * H // Hkv):
                x = (s["q"][start[b]:start[b + 1], g].double() @ k.T) / math.sqrt(c["dim"])
                x = x.masked_fill(hidden, -math.inf)
                out[start[b]:start[b + 1], g] = torch.softmax(x, 1) @ v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)
