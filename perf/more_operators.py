"""Cases and plain forms of the operators that a step over many requests at
once needs beside the int4 products and the 4-bit cache: the requests' own
low-rank adapters, attention through a sliding window with a few first tokens
that stay visible, and the verification of drafted tokens.

`run` computes an operator in elementary torch operations, in 32 bits (the
verification in 64: a drawn token lies at the border of two sums), or, where
`own` is true, by the library's own call.
"""
import math

import torch

own = False

DEV = "cuda"


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # a chat with one user whose request has an adapter: latency
        dict(name="adapters: one token", op="adapters", batch=1, new=1, k=4096, n=4096, rank=16, count=8, mixed=False,
             wide=0, base=True, dtype="f16"),
        # one new token of each of 32 requests, most with an adapter of their own; q is a slice of the fused q, k, v
        dict(name="adapters: 32 requests", op="adapters", batch=32, new=1, k=4096, n=4096, rank=16, count=24,
             mixed=False, wide=2048, base=True, dtype="f16"),
        # drafts of 20 requests to verify, a feed-forward layer's way down, adapters of different ranks
        dict(name="adapters: 20 requests of 5 rows", op="adapters", batch=20, new=5, k=11008, n=4096, rank=64, count=12,
             mixed=True, wide=0, base=True, dtype="f16"),
        # prompts of five requests, of uneven length, in one call
        dict(name="adapters: prompts", op="adapters", batch=5, new=2500, k=4096, n=11008, rank=32, count=4, mixed=False,
             wide=0, base=True, dtype="f16"),
        # fp32 activations, odd sizes, the adapters' part by itself
        dict(name="adapters: fp32 and odd sizes", op="adapters", batch=7, new=150, k=2050, n=1001, rank=12, count=5,
             mixed=True, wide=3, base=False, dtype="f32"),
        # a long chat of one user, one token
        dict(name="sinks: one sequence", op="sinks", batch=1, new=1, kv=30000, window=4096, sinks=4, q_heads=32,
             kv_heads=8, dim=128, group=128, page=64, dtype="f16"),
        # a serving batch of long chats
        dict(name="sinks: batch of 32", op="sinks", batch=32, new=1, kv=16384, window=4096, sinks=4, q_heads=32,
             kv_heads=8, dim=128, group=128, page=64, dtype="f16"),
        # speculative verify in fp32, small heads, fine groups, a whole instruction kept visible
        dict(name="sinks: verify fp32", op="sinks", batch=8, new=5, kv=4100, window=1000, sinks=100, q_heads=24,
             kv_heads=8, dim=64, group=32, page=32, dtype="f32"),
        # chunks of a document behind what is cached of it
        dict(name="sinks: prompt chunks", op="sinks", batch=2, new=2048, kv=8192, window=2048, sinks=16, q_heads=32,
             kv_heads=8, dim=128, group=128, page=64, dtype="f16"),
        # four drafts of one request
        dict(name="verify: one sequence", op="verify", batch=1, new=5, vocab=32000, draft=True, top=0, dtype="f32"),
        # seven drafts of each of 32 requests, a large vocabulary
        dict(name="verify: 32 sequences", op="verify", batch=32, new=8, vocab=128000, draft=True, top=0, dtype="f32"),
        # drafts that were looked up, not drawn; 50 tokens are left to choose from; an odd vocabulary
        dict(name="verify: certain drafts", op="verify", batch=16, new=6, vocab=50257, draft=False, top=50, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_adapters(rng, dtype):
    k, n = _log_int(rng, 64, 16384), _log_int(rng, 64, 16384)
    if rng.random() < 0.75:
        k, n = k // 16 * 16, n // 16 * 16
    rank = rng.choice([4, 8, 16, 16, 32, 64, 128, rng.randint(1, 128)])
    batch = _log_int(rng, 1, 64)
    new = 1 if rng.random() < 0.5 else _log_int(rng, 2, 4096)
    count = _log_int(rng, 1, 64)
    while batch * new > 8192 or batch * new * (k + 2 * n) > 8000 * 26000 // (1 if dtype == "f16" else 2) or \
            batch * new * rank * (k + n) > 8000 * 32 * 15000 or min(batch, count) * rank * (k + n) > 32_000_000:
        batch, new = max(1, batch * 3 // 4), (new + 1) // 2
    return dict(op="adapters", batch=batch, new=new, k=k, n=n, rank=rank, count=count,
                mixed=rng.random() < 0.4, wide=rng.choice([0, 0, 8 * rng.randint(1, 500), rng.randint(1, 99)]),
                base=rng.random() < 0.8, dtype=dtype)


def _draw_sinks(rng, dtype):
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 6, 8])
    batch = _log_int(rng, 1, 32)
    new = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, 2048)])
    kv = max(new, _log_int(rng, 64, 65536))
    window = _log_int(rng, 1, 8192)
    while batch * kv * kv_heads * dim > 32 * 16384 * 8 * 128 or \
            batch * min(kv, window + new) * kv_heads * dim > 32 * 4096 * 8 * 128 or \
            batch * new * min(kv, window + new) * q_heads * dim > 2 * 2048 * 2048 * 32 * 128:
        batch, kv, new = max(1, batch // 2), max(1, kv * 3 // 4), max(1, new * 3 // 4)
        kv, window = max(kv, new), max(1, window * 3 // 4)
    return dict(op="sinks", batch=batch, new=new, kv=kv, window=window,
                sinks=rng.choice([1, 4, 4, 16, rng.randint(2, 300)]), q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                group=rng.choice([g for g in (32, 64, 128) if g <= dim]), page=rng.choice([32, 64, 128, 256]),
                dtype=dtype)


def draw(rng):
    op = rng.choice(["adapters", "adapters", "sinks", "sinks", "verify"])
    dtype = rng.choice(["f16", "f16", "f32"])
    if op == "adapters":
        return _draw_adapters(rng, dtype)
    if op == "sinks":
        return _draw_sinks(rng, dtype)
    vocab = _log_int(rng, 500, 260000)
    batch, new = _log_int(rng, 1, 64), rng.randint(1, 9)
    while batch * new * vocab > 32 * 8 * 128000:
        batch = max(1, batch // 2)
    return dict(op="verify", batch=batch, new=new, vocab=vocab, draft=rng.random() < 0.7,
                top=rng.choice([0, 0, 1, rng.randint(2, 200)]), dtype=dtype)


def _spread(n, most, least):
    """n lengths in least..most, uneven, the first the longest."""
    return [max(least, most - int((most - least) * 0.75 * ((0.6180339887 * i) % 1.0))) for i in range(n)]


def _lengths(c):
    """New tokens of each sequence, and cached tokens with them."""
    new = _spread(c["batch"], c["new"], 1)
    if c["op"] != "sinks":
        return new, None
    return new, [max(n, s) for n, s in zip(new, _spread(c["batch"], c["kv"], c["new"]))]


def _requests(c):
    """The adapter of each request (every eighth has none), and every adapter's rank."""
    ranks = [max(1, c["rank"] >> (a % 3)) if c["mixed"] else c["rank"] for a in range(c["count"])]
    return [-1 if i % 8 == 5 else (7 * i + 2) % c["count"] for i in range(c["batch"])], ranks


def work(c):
    e = 2 if c["dtype"] == "f16" else 4
    new, total = _lengths(c)
    if c["op"] == "adapters":
        which, ranks = _requests(c)
        rows = sum(m for m, a in zip(new, which) if a >= 0)
        held = sum(ranks[a] for a in set(which) if a >= 0) * (c["k"] + c["n"])
        flops = sum(2 * m * ranks[a] for m, a in zip(new, which) if a >= 0) * (c["k"] + c["n"])
        return {"bytes": e * (rows * c["k"] + held + sum(new) * c["n"] * (2 if c["base"] else 1)), "flops": flops}
    if c["op"] == "verify":  # of each sequence the row of the token that is drawn
        return {"bytes": e * c["batch"] * c["vocab"] * (2 if c["draft"] and c["new"] > 1 else 1),
                "flops": 3 * c["batch"] * c["vocab"]}
    D, H, Hkv = c["dim"], c["q_heads"], c["kv_heads"]
    token = Hkv * 2 * (D // 2 + 4 * (D // c["group"]))  # bytes of a cached token
    pairs = keys = 0
    for n, s in zip(new, total):
        lo = max(0, s - n + 1 - c["window"])
        keys += s - lo + min(c["sinks"], lo)
        for i in range(s - n, s):
            below = max(0, i + 1 - c["window"])
            pairs += i + 1 - below + min(c["sinks"], below)
    return {"bytes": keys * token + 2 * e * sum(new) * H * D, "flops": 4 * pairs * H * D}


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


def _prepare_adapters(c, s, gen):
    t, (new, _), (which, ranks) = _dtype(c), _lengths(c), _requests(c)
    k, n, r, m = c["k"], c["n"], c["rank"], sum(_lengths(c)[0])

    def randn(*shape):
        return torch.randn(*shape, device=DEV, generator=gen)

    ends = torch.tensor([0] + new).cumsum(0).tolist()
    s.update(a=(randn(c["count"], r, k) * k ** -0.5).to(t), b=(randn(c["count"], n, r) * 0.3 * r ** -0.5).to(t),
             scales=torch.rand(c["count"], device=DEV, generator=gen) * 1.5 + 0.5,
             ranks=torch.tensor(ranks, dtype=torch.int32, device=DEV) if c["mixed"] else None,
             adapter=torch.tensor([a for a, q in zip(which, new) for _ in range(q)], dtype=torch.int32, device=DEV),
             x=randn(m, k).to(t), base=randn(m, n + c["wide"]).to(t)[:, c["wide"]:] if c["base"] else None,
             y=torch.empty(m, n + c["wide"], dtype=t, device=DEV)[:, c["wide"]:], workspace=None, host_ranks=ranks,
             segments=[(i, j, a) for i, j, a in zip(ends[:-1], ends[1:], which)])


def _prepare_sinks(c, s, gen):
    t, D, H = _dtype(c), c["dim"], c["q_heads"]
    new, total = _lengths(c)
    need = [-(-v // c["page"]) for v in total]
    order = torch.randperm(sum(need), generator=gen, device=DEV).to(torch.int32)   # pages in random order
    table = torch.zeros(c["batch"], max(need), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s.update(table=table, kv_len=torch.tensor(total, dtype=torch.int32, device=DEV), pages=sum(need),
             tokens=sum(new), max_new=max(new), max_kv=max(total), cache=_cache(c, sum(need), gen),
             q=(torch.randn(sum(new), H, D, device=DEV, generator=gen) * 1.5).to(t),
             out=torch.empty(sum(new), H, D, dtype=t, device=DEV), workspace=None)


def _prepare_verify(c, s, gen):
    t, V = _dtype(c), c["vocab"]
    new, _ = _lengths(c)
    m = sum(new)

    def chosen(x):
        if c["top"]:
            x = x.masked_fill(x < x.topk(min(c["top"], V), 1)[0][:, -1:], float("-inf"))
        return torch.softmax(x, 1)

    logits = torch.randn(m, V, device=DEV, generator=gen) * 2.5
    target = chosen(logits)
    logits += 0.5 * torch.randn(m, V, device=DEV, generator=gen)   # the draft model comes close
    draft = chosen(logits)
    ids = torch.randint(0, V, (m,), device=DEV, generator=gen)
    if c["draft"]:
        ids[1:] = torch.multinomial(draft, 1, generator=gen)[:-1, 0]   # row i draws the token of row i + 1
    else:
        ids[1:] = logits.argmax(1)[:-1]
    s.update(target=target.to(t), draft=draft.to(t) if c["draft"] else None, ids=ids.to(torch.int32),
             accept=torch.rand(m, device=DEV, generator=gen), pick=torch.rand(c["batch"], device=DEV, generator=gen),
             out=torch.empty(m, dtype=torch.int32, device=DEV), tokens=m, max_new=max(new),
             accepted=torch.empty(c["batch"], dtype=torch.int32, device=DEV), workspace=None)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": c, "q_start": torch.tensor([0] + _lengths(c)[0], device=DEV).cumsum(0).to(torch.int32)}
    {"adapters": _prepare_adapters, "sinks": _prepare_sinks, "verify": _prepare_verify}[c["op"]](c, s, gen)
    if own:
        _prepare_own(s)
    return s


# ---- the operators ----------------------------------------------------------

def _prepare_own(s):
    """Descriptor and workspace, as a program holds them."""
    from block_wise_int4_amd import mnb
    c = s["case"]
    if c["op"] == "adapters":
        s["desc"] = mnb.adapter_desc(c["n"], c["k"], c["rank"], c["count"], s["x"].dtype)
        size = mnb.mnb_adapters_workspace_bytes(s["desc"], s["x"].shape[0])
    elif c["op"] == "sinks":
        s["desc"] = mnb.kv4_desc(c["q_heads"], c["kv_heads"], c["dim"], c["group"], c["page"], s["pages"])
        size = mnb.mnb_attention_kv4_sinks_workspace_bytes(s["desc"], c["batch"], s["tokens"], s["max_new"],
                                                           s["max_kv"], c["window"], c["sinks"])
    else:
        size = mnb.mnb_verify_workspace_bytes(c["batch"], c["vocab"])
    s["workspace"] = torch.empty(max(256, size), dtype=torch.uint8, device=DEV)


def _run_own(s):
    from block_wise_int4_amd import mnb
    c = s["case"]
    if "desc" not in s and s["workspace"] is None:
        _prepare_own(s)
    if c["op"] == "adapters":
        mnb.mnb_adapters_add(s["desc"], s["a"], s["b"], s["scales"], s["adapter"], s["x"], s["y"], base=s["base"],
                             ranks=s["ranks"], workspace=s["workspace"])
        return s["y"]
    if c["op"] == "sinks":
        mnb.mnb_attention_kv4_sinks(s["desc"], s["cache"], s["q"], s["table"], s["kv_len"], s["q_start"], s["max_new"],
                                    s["max_kv"], s["out"], 1.0 / math.sqrt(c["dim"]), c["window"], c["sinks"],
                                    workspace=s["workspace"])
        return s["out"]
    mnb.mnb_verify_drafts(s["target"], s["ids"], s["accept"], s["pick"], s["out"], s["accepted"], q_start=s["q_start"],
                          draft=s["draft"], workspace=s["workspace"])
    return {"ids": s["out"], "accepted": s["accepted"]}


def _plain_adapters(s):
    c = s["case"]
    x = s["x"].float()
    out = torch.zeros(x.shape[0], c["n"], device=DEV) if s["base"] is None else s["base"].float()
    if c["new"] == 1:  # a row a request: every row's adapter side by side
        which = s["adapter"].long().clamp(min=0)
        a, b = s["a"][which].float(), s["b"][which].float()
        h = torch.matmul(a, x[:, :, None])
        if c["mixed"]:
            h = h * (torch.arange(c["rank"], device=DEV)[None] < s["ranks"][which][:, None])[:, :, None]
        d = torch.matmul(b, h)[:, :, 0] * s["scales"][which][:, None]
        return (out + d * (s["adapter"] >= 0)[:, None]).to(s["x"].dtype)
    for i, j, a in s["segments"]:
        if a >= 0:
            r = s["host_ranks"][a]
            h = torch.matmul(x[i:j], s["a"][a, :r].float().t())
            out[i:j] += torch.matmul(h, s["b"][a, :, :r].float().t()) * s["scales"][a]
    return out.to(s["x"].dtype)


def _positions(s):
    """Position and sequence of each new token."""
    tok = torch.arange(s["tokens"], device=DEV)
    seq = (tok[:, None] >= s["q_start"][None, 1:]).sum(1)
    return tok - s["q_start"][seq + 1] + s["kv_len"][seq], seq


def _plain_values(c, blk):
    """Keys and values [batch, kv heads, tokens, dim] of the blocks of chosen pages, in 32 bits."""
    D, NG, H, nblk = c["dim"], c["dim"] // c["group"], c["kv_heads"], c["page"] // 32
    B, P = blk.shape[:2]
    slot = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], dtype=torch.int32, device=DEV)
    byte = torch.tensor([0, 2, 1, 3], device=DEV)

    def values(codes, meta):
        scale = (meta & 0xFFFF).to(torch.int16).view(torch.float16).float()
        zero = ((meta >> 16) & 15).float()
        x = (codes.float().reshape(B, P, H, nblk, 32, NG, c["group"]) - zero[..., None]) * scale[..., None]
        return x.reshape(B, P, H, nblk, 32, D).permute(0, 2, 1, 3, 4, 5).reshape(B, H, P * nblk * 32, D)

    kw = blk[..., :16 * D].contiguous().view(torch.int32).reshape(B, P, H, nblk, D // 64, 4, 16, 4)
    kc = ((kw[..., None] >> slot) & 15).to(torch.uint8).permute(0, 1, 2, 3, 4, 7, 5, 6, 8)
    kc = kc.reshape(B, P, H, nblk, 2, D // 32, 4, 16, 8).permute(0, 1, 2, 3, 4, 7, 5, 6, 8)
    km = blk[..., 32 * D:32 * D + 128 * NG].contiguous().view(torch.int32).reshape(B, P, H, nblk, 32, NG)
    keys = values(kc.reshape(B, P, H, nblk, 32, D), km)
    vb = blk[..., 16 * D:32 * D].reshape(B, P, H, nblk, D // 64, 4, 16, 2, 2, 4)[..., byte]
    vc = torch.stack([vb & 15, vb >> 4], -1).permute(0, 1, 2, 3, 8, 5, 9, 4, 7, 10, 6)
    vm = blk[..., 32 * D + 128 * NG:].contiguous().view(torch.int32).reshape(B, P, H, nblk, 32, NG)
    return keys, values(vc.reshape(B, P, H, nblk, 32, D), vm)


def _plain_sinks(s):
    c = s["case"]
    D, H, Hkv, B, N, page = c["dim"], c["q_heads"], c["kv_heads"], c["batch"], s["max_new"], c["page"]
    # the pages that a row may see: of the first tokens, and from the first row's window on
    width = s["table"].shape[1]
    low = (s["kv_len"] - (s["q_start"][1:] - s["q_start"][:-1]) + 1 - c["window"]).clamp(min=0) // page
    lead = min(width, -(-c["sinks"] // page))
    tail = min(width, (c["window"] + N) // page + 2)
    col = torch.cat([torch.arange(lead, device=DEV)[None].expand(B, -1), low[:, None] + torch.arange(tail, device=DEV)], 1)
    there = torch.cat([col[:, :lead] < low[:, None], col[:, lead:] < width], 1)
    pages = torch.gather(s["table"].long(), 1, col.clamp(max=width - 1).long())
    nblk = page // 32
    keys, vals = _plain_values(c, s["cache"].view(s["pages"], Hkv, nblk, _block_bytes(c))[pages])
    key = (col[:, :, None] * page + torch.arange(page, device=DEV)).reshape(B, -1)
    there = there.repeat_interleave(page, 1) & (key < s["kv_len"][:, None])
    vals = vals.masked_fill(~there[:, None, :, None], 0.0)
    pos, seq = _positions(s)
    at = torch.arange(s["tokens"], device=DEV) - s["q_start"][seq]
    q = torch.zeros(B, N, Hkv, H // Hkv, D, device=DEV)
    q[seq, at] = s["q"].float().reshape(-1, Hkv, H // Hkv, D)
    where = torch.full((B, N), -1, dtype=torch.long, device=DEV)
    where[seq, at] = pos.long()
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D), keys.transpose(2, 3)) * (1.0 / math.sqrt(D))
    key, where = key[:, None], where[..., None]
    seen = there[:, None] & (key <= where) & ((key > where - c["window"]) | (key < c["sinks"]))
    S = key.shape[2]
    x = x.reshape(B, Hkv, N, H // Hkv, S).masked_fill_(~seen[:, None, :, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp_min(-3e38)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hkv, -1, S), vals).reshape(B, Hkv, N, H // Hkv, D)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    return o.permute(0, 2, 1, 3, 4)[seq, at].reshape(-1, H, D).to(s["q"].dtype)


def _plain_verify(s):
    c, first = s["case"], s["q_start"][:-1].long()
    n = s["q_start"][1:].long() - first - 1                            # drafts of each sequence
    i = torch.arange(max(1, s["max_new"] - 1), device=DEV)
    drafted = i < n[:, None]
    row = torch.where(drafted, first[:, None] + i, torch.zeros_like(i))
    token = s["ids"].long()[(row + 1).clamp(max=s["tokens"] - 1)]
    p = s["target"][row, token].double()
    q = 1.0 if s["draft"] is None else s["draft"][row, token].double()
    good = drafted & (s["accept"][row].double() * q < p)
    accepted = good.long().cumprod(1).sum(1)
    at, refused = first + accepted, accepted < n
    p = s["target"][at].double()
    if s["draft"] is None:
        bad = s["ids"].long()[(at + 1).clamp(max=s["tokens"] - 1)]
        gone = torch.arange(c["vocab"], device=DEV) == bad[:, None]
        left = p.masked_fill(gone, 0.0)
    else:
        left = (p - s["draft"][at].double()).clamp(min=0.0)
    w = torch.where((refused & (left.sum(1) > 0))[:, None], left, p)
    sums = w.cumsum(1)
    drawn = (sums <= s["pick"].double()[:, None] * sums[:, -1:]).sum(1)
    tok = torch.arange(s["tokens"], device=DEV)
    seq = (tok[:, None] >= s["q_start"][None, 1:]).sum(1)
    i = tok - first[seq]
    out = torch.where(i < accepted[seq], s["ids"].long()[(tok + 1).clamp(max=s["tokens"] - 1)],
                      torch.where(i == accepted[seq], drawn[seq], torch.full_like(tok, -1)))
    return {"ids": out.to(torch.int32), "accepted": accepted.to(torch.int32)}


def run(s):
    if own:
        return _run_own(s)
    return {"adapters": _plain_adapters, "sinks": _plain_sinks, "verify": _plain_verify}[s["case"]["op"]](s)


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_adapters(s):
    n, which = s["case"]["n"], s["adapter"].tolist()
    y = torch.zeros(len(which), n, dtype=torch.float64, device=DEV)
    for a in sorted(set(which) - {-1}):
        rows = (s["adapter"] == a).nonzero()[:, 0]
        r = s["case"]["rank"] if s["ranks"] is None else int(s["ranks"][a])
        h = s["x"][rows].double() @ s["a"][a, :r].double().mT
        y[rows] = float(s["scales"][a]) * (h @ s["b"][a, :, :r].double().mT)
    return y if s["base"] is None else y + s["base"].double()


def _exact_rows(s, b, h, j):
    """Keys and values [len(j), dim] of the tokens j of a sequence and head in 64 bits, each code fetched from its byte."""
    c = s["case"]
    D, G, nblk = c["dim"], c["group"], c["page"] // 32
    NG, size = D // G, _block_bytes(c)
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
        return (code - z) * (lo | (hi << 8)).to(torch.int16).view(torch.float16).double()

    return value(kc, 32 * D), value(vc, 32 * D + 128 * NG)


def _exact_sinks(s):
    c = s["case"]
    H, Hkv = c["q_heads"], c["kv_heads"]
    out = torch.zeros(s["tokens"], H, c["dim"], dtype=torch.float64, device=DEV)
    start, total = s["q_start"].tolist(), s["kv_len"].tolist()
    for b in range(c["batch"]):
        n, first = total[b], total[b] - (start[b + 1] - start[b])
        i, key = torch.arange(first, n, device=DEV)[:, None], torch.arange(n, device=DEV)
        key = key[(key < c["sinks"]) | (key > first - c["window"])]
        hidden = (key > i) | ((i - key >= c["window"]) & (key >= c["sinks"]))
        for h in range(Hkv):
            k, v = _exact_rows(s, b, h, key)
            for g in range(h * H // Hkv, (h + 1) * H // Hkv):
                x = (s["q"][start[b]:start[b + 1], g].double() @ k.T) / math.sqrt(c["dim"])
                out[start[b]:start[b + 1], g] = torch.softmax(x.masked_fill(hidden, -math.inf), 1) @ v
    return out


def _exact_verify(s):
    start, ids = s["q_start"].tolist(), s["ids"].tolist()
    out, counts = [], []
    for b, (i, end) in enumerate(zip(start[:-1], start[1:])):
        taken = 0
        while i + taken + 1 < end:
            row, token = i + taken, ids[i + taken + 1]
            q = 1.0 if s["draft"] is None else float(s["draft"][row, token])
            if float(s["accept"][row]) * q >= float(s["target"][row, token]):
                break
            taken += 1
        row = i + taken
        w = s["target"][row].cpu().double()
        if row + 1 < end:
            q = torch.zeros_like(w)
            if s["draft"] is None:
                q[ids[row + 1]] = math.inf
            else:
                q = s["draft"][row].cpu().double()
            rest = torch.relu(w - q)
            w = rest if float(rest.max()) > 0 else w
        sums = torch.cumsum(w, 0)
        border = torch.tensor(float(s["pick"][b]) * float(sums[-1]), dtype=torch.float64)
        out += ids[i + 1:row + 1] + [int(torch.searchsorted(sums, border, right=True))] + [-1] * (end - row - 1)
        counts.append(taken)
    return {"ids": torch.tensor(out, dtype=torch.int32, device=DEV),
            "accepted": torch.tensor(counts, dtype=torch.int32, device=DEV)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"adapters": _exact_adapters, "sinks": _exact_sinks, "verify": _exact_verify}[case["op"]](s)
