"""A batch of requests served together over int4 weights: each with its own
low-rank adapter, a sliding window beside which its first tokens stay visible, and
drafted tokens that are verified.

    python examples/serve_batch.py [--requests 5] [--steps 4] [--drafts 3]

    q, k, v = qkv(norm(stream)) + adapter(norm(stream))
    stream += o(attention(rotate(q), cache))
    tokens = verify(softmax(head(norm(stream))), drafts)

The first call takes all prompts, every later one a sure token and the drafts of each
request.  A refused draft's place in the cache is written again by the next step.  Each
call is compared with the same step in plain torch, request by request, on dequantized
weights and the keys and values that the cache holds; prints the largest differences, and how
many drafts were accepted.
"""
import argparse
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
for p in (os.path.dirname(HERE), HERE):
    if p not in sys.path:
        sys.path.insert(0, p)

import torch

from block_wise_int4_amd import mnb
from decoder_layer import EPS, Linear


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, requests, hidden=512, q_heads=8, kv_heads=2, dim=64, vocab=1000, rank=12, adapters=4, window=48,
                 sinks=4, most=400, page=32, seed=0):
        gen = self.gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.H, self.Hkv, self.D, self.vocab, self.window, self.sinks = q_heads, kv_heads, dim, vocab, window, sinks
        n = (q_heads + 2 * kv_heads) * dim
        self.embed = torch.randn(vocab, hidden, generator=gen, device="cuda").half()
        self.qkv, self.o, self.head = Linear(n, hidden, gen), Linear(hidden, q_heads * dim, gen), Linear(vocab, hidden, gen)
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")).half()
        # the adapters' weights lie side by side, each of its own rank; one request in four has none
        self.set = mnb.adapter_desc(n, hidden, rank, adapters, torch.float16)
        self.a = (torch.randn(adapters, rank, hidden, generator=gen, device="cuda") * hidden ** -0.5).half()
        self.b = (torch.randn(adapters, n, rank, generator=gen, device="cuda") * 0.5 * rank ** -0.5).half()
        self.scales = torch.rand(adapters, generator=gen, device="cuda") + 0.5
        self.ranks = [max(1, rank - 3 * i) for i in range(adapters)]
        self.adapter = [-1 if i % 4 == 3 else i % adapters for i in range(requests)]
        pages = -(-most // page)
        self.kv = mnb.kv4_desc(q_heads, kv_heads, dim, dim, page, requests * pages)
        self.cache = torch.empty(mnb.mnb_kv4_cache_bytes(self.kv), dtype=torch.uint8, device="cuda")
        self.table = torch.randperm(requests * pages, generator=gen, device="cuda").to(torch.int32).view(requests, pages)
        ang = torch.arange(most, device="cuda")[:, None] * 10000.0 ** (-torch.arange(dim // 2, device="cuda") * 2.0 / dim)[None]
        self.cos, self.sin = ang.cos().contiguous(), ang.sin().contiguous()

    def __call__(self, ids, rows, past, draft, accept, pick):
        """ids of all rows, rows and cached tokens of each request, the drafts' distributions and random numbers."""
        H, Hkv, D, T = self.H, self.Hkv, self.D, len(ids)
        start = i32([0] + rows).cumsum(0).to(torch.int32)
        kv_len = i32([p + n for p, n in zip(past, rows)])
        which = i32([a for a, n in zip(self.adapter, rows) for _ in range(n)])
        longest = max(p + n for p, n in zip(past, rows))
        x = self.embed[ids.long()]
        h = torch.empty_like(x)
        mnb.mnb_rms_norm(x, self.norm, h, EPS)
        qkv = self.qkv(h)
        ws = torch.empty(max(16, mnb.mnb_adapters_workspace_bytes(self.set, T)), dtype=torch.uint8, device="cuda")
        mnb.mnb_adapters_add(self.set, self.a, self.b, self.scales, which, h, qkv, base=qkv, ranks=i32(self.ranks), workspace=ws)
        qkv = qkv.view(T, H + 2 * Hkv, D)
        q = torch.empty((T, H, D), dtype=torch.float16, device="cuda")
        mnb.mnb_kv4_append(self.kv, self.cache, qkv[:, H:H + Hkv], qkv[:, H + Hkv:], self.table, kv_len, start,
                           cos=self.cos, sin=self.sin, rotary_dim=D, q=qkv[:, :H], q_out=q)
        att = torch.empty_like(q)
        size = mnb.mnb_attention_kv4_sinks_workspace_bytes(self.kv, len(rows), T, max(rows), longest, self.window, self.sinks)
        ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
        mnb.mnb_attention_kv4_sinks(self.kv, self.cache, q, self.table, kv_len, start, max(rows), longest, att, D ** -0.5,
                                    self.window, self.sinks, workspace=ws)
        stream, last = torch.empty_like(x), torch.empty_like(x)
        mnb.mnb_rms_norm(self.o(att.view(T, H * D)), self.norm, last, EPS, residual=x, residual_out=stream)
        probs = torch.softmax(self.head(last).float(), 1)
        out, accepted = torch.empty_like(ids), torch.empty(len(rows), dtype=torch.int32, device="cuda")
        ws = torch.empty(mnb.mnb_verify_workspace_bytes(len(rows), self.vocab), dtype=torch.uint8, device="cuda")
        mnb.mnb_verify_drafts(probs, ids, accept, pick, out, accepted, q_start=start, draft=draft, workspace=ws)
        return out, accepted, probs, (h, qkv, q, att, stream)

    def plain(self, ids, rows, past, inner):
        """Largest differences of (qkv, attention, stream) from plain torch, request by request."""
        h, qkv, q, att, stream = inner
        H, Hkv, D = self.H, self.Hkv, self.D
        worst, first = [0.0] * 3, 0
        for r, (n, p) in enumerate(zip(rows, past)):
            at, total, g = slice(first, first + n), p + n, self.adapter[r]
            first += n
            w = self.qkv.values
            if g >= 0:
                k = self.ranks[g]
                w = w + self.scales[g] * (self.b[g, :, :k].float() @ self.a[g, :k].float())
            worst[0] = max(worst[0], float((h[at].float() @ w.T - qkv[at].view(n, -1).float()).abs().max()))
            k, v = (torch.empty((total, Hkv, D), dtype=torch.float32, device="cuda") for _ in range(2))
            mnb.mnb_kv4_read(self.kv, self.cache, self.table[r:r + 1], i32([total]), i32([0, total]), k, v)
            k, v = (t.repeat_interleave(H // Hkv, 1).transpose(0, 1) for t in (k, v))
            x = torch.stack([q[at, i].float() @ k[i].T for i in range(H)]) * D ** -0.5
            i, j = torch.arange(p, total, device="cuda")[:, None], torch.arange(total, device="cuda")[None]
            seen = (j <= i) & ((j > i - self.window) | (j < self.sinks))
            y = torch.softmax(x.masked_fill(~seen, float("-inf")), -1)
            y = torch.stack([y[i] @ v[i].contiguous() for i in range(H)], 1)
            worst[1] = max(worst[1], float((y - att[at].float()).abs().max()))
            s = self.embed[ids[at].long()].float() + (att[at].reshape(n, -1).float() @ self.o.values.T).half().float()
            worst[2] = max(worst[2], float((s - stream[at].float()).abs().max()))
        return worst


def run(requests=5, steps=4, drafts=3, prompt=90, seed=0, **kw):
    """Largest differences (qkv, attention, stream), drafts accepted and offered, and every call's tokens with what they came
    from: (target, draft, ids, offsets, accept, pick, out, accepted)."""
    server = Server(requests, most=prompt + requests + (steps + 1) * (drafts + 1), seed=seed, **kw)
    gen, V = server.gen, server.vocab

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    past, rows = [0] * requests, [max(1, prompt - 17 * i) for i in range(requests)]
    ids = torch.randint(0, V, (sum(rows),), generator=gen, device="cuda").to(torch.int32)
    worst, taken, calls = [0.0] * 3, 0, []
    for step in range(steps + 1):
        # the prompt's tokens are sure: an accept below 0 takes a certain draft whatever its probability
        T = len(ids)
        draft = torch.softmax(1.5 * torch.randn(T, V, generator=gen, device="cuda"), 1) if step else None
        accept = rand(T) if step else torch.full((T,), -1.0, device="cuda")
        if step:                       # each request's rows but the first are drawn from the draft's rows before them
            drawn = torch.multinomial(draft, 1, generator=gen)[:, 0].to(torch.int32)
            for r in range(requests):
                ids[r * (drafts + 1) + 1:(r + 1) * (drafts + 1)] = drawn[r * (drafts + 1):(r + 1) * (drafts + 1) - 1]
        pick = rand(requests)
        out, accepted, probs, inner = server(ids, rows, past, draft, accept, pick)
        worst = [max(a, b) for a, b in zip(worst, server.plain(ids, rows, past, inner))]
        offsets = [0]
        for n in rows:
            offsets.append(offsets[-1] + n)
        calls.append((probs, draft, ids.clone(), offsets, accept, pick, out, accepted))
        n = accepted.tolist()
        taken += sum(n) if step else 0
        sure = out[[offsets[r] + n[r] for r in range(requests)]]
        past = [p + k + 1 for p, k in zip(past, n)]
        rows = [drafts + 1] * requests
        ids = torch.zeros(requests * (drafts + 1), dtype=torch.int32, device="cuda")
        ids[::drafts + 1] = sure
    return worst, taken, steps * drafts * requests, calls


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=5)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--drafts", type=int, default=3)
    a = ap.parse_args()
    worst, taken, offered, _ = run(a.requests, a.steps, a.drafts)
    print("largest differences from plain torch: " + ", ".join("%s %.2g" % v for v in zip(("qkv", "attention", "stream"), worst)))
    print("%d of %d drafts accepted" % (taken, offered))
