"""One decoder layer over int4 weights: a prompt, then tokens one by one.

    python examples/decoder_layer.py [--hidden 512] [--prompt 100] [--steps 8]

    stream += o(attention(rotate(q), cache)),  q, k, v = qkv(norm(stream))
    stream += down(silu(gate(norm(stream))) * up(norm(stream)))

Every step runs in the library: the RMS norm with the residual's addition, the
int4 products, the append of rotated keys and values to the paged 4-bit cache and
the attention over it.  The feed-forward's up and gate products take the
norm's 8-bit codes (accuracy_level 4).  Each call's output is compared with the
same layer in plain torch, on dequantized weights and the keys and values
that the cache holds; prints the largest difference.
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

from block_wise_int4_amd import mnb

GROUP = 64
EPS = 1e-5


class Linear:
    """An int4 weight [n, k] and its dequantized values."""

    def __init__(self, n, k, gen):
        codes = torch.randint(0, 16, (n, k), generator=gen, device="cuda", dtype=torch.uint8)
        scales = (torch.rand(n, k // GROUP, generator=gen, device="cuda") * 0.2 + 0.1) * (k ** -0.5)
        scales = scales.half()
        packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()
        self.q = mnb.repack(packed.view(-1), scales.reshape(-1), None, n, k, GROUP)
        self.n = n
        self.values = (codes.float() - 8.0) * scales.float().repeat_interleave(GROUP, 1)

    def __call__(self, a, out_bias=None):
        """fp16 product, with a residual added in fp32 before the one rounding."""
        m = a.shape[0]
        y = torch.empty((m, self.n), dtype=torch.float16, device="cuda")
        ws = torch.empty(max(16, mnb.mnb_gemm_workspace_bytes(self.q.desc, m)), dtype=torch.uint8, device="cuda")
        if out_bias is None:
            mnb.mnb_gemm(self.q.desc, self.q.repacked, a, m, y, ws)
        else:
            mnb.mnb_gemm_bias(self.q.desc, self.q.repacked, a, m, out_bias, self.n, mnb.MNB_BIAS_FUSED, y, ws)
        return y

    def from_codes(self, codes, scales):
        """fp32 product of 8-bit activations."""
        y = torch.empty((codes.shape[0], self.n), device="cuda")
        mnb.mnb_gemm_accuracy4_codes(self.q.desc, self.q.repacked, codes, scales, codes.shape[0], None, y)
        return y


class Layer:
    def __init__(self, hidden, q_heads, kv_heads, dim, ffn, max_tokens, page=64, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.hidden, self.q_heads, self.kv_heads, self.dim, self.gen = hidden, q_heads, kv_heads, dim, gen
        self.qkv = Linear((q_heads + 2 * kv_heads) * dim, hidden, gen)
        self.o = Linear(hidden, q_heads * dim, gen)
        self.gate, self.up = Linear(ffn, hidden, gen), Linear(ffn, hidden, gen)
        self.down = Linear(hidden, ffn, gen)
        self.norm1, self.norm2 = ((1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")).half() for _ in range(2))
        pages = -(-max_tokens // page)
        self.kv = mnb.kv4_desc(q_heads, kv_heads, dim, min(dim, 128), page, pages)
        self.cache = torch.empty(mnb.mnb_kv4_cache_bytes(self.kv), dtype=torch.uint8, device="cuda")
        self.table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)[None]
        ang = torch.arange(max_tokens, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(dim // 2, device="cuda") * 2.0 / dim)[None]
        self.cos, self.sin = ang.cos().contiguous(), ang.sin().contiguous()

    def __call__(self, x, past):
        """The layer on the rows x of one sequence's new tokens, `past` tokens being cached; appends theirs."""
        n, H, Hkv, D = x.shape[0], self.q_heads, self.kv_heads, self.dim
        kv_len = torch.tensor([past + n], dtype=torch.int32, device="cuda")
        q_start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        a = torch.empty_like(x)
        mnb.mnb_rms_norm(x, self.norm1, a, EPS)
        qkv = self.qkv(a).view(n, H + 2 * Hkv, D)
        q = torch.empty((n, H, D), dtype=torch.float16, device="cuda")
        mnb.mnb_kv4_append(self.kv, self.cache, qkv[:, H:H + Hkv], qkv[:, H + Hkv:], self.table, kv_len, q_start,
                           cos=self.cos, sin=self.sin, rotary_dim=D, q=qkv[:, :H], q_out=q)
        att = torch.empty_like(q)
        ws = torch.empty(max(16, mnb.mnb_attention_kv4_workspace_bytes(self.kv, 1, n, n, past + n)), dtype=torch.uint8,
                         device="cuda")
        mnb.mnb_attention_kv4(self.kv, self.cache, q, self.table, kv_len, q_start, n, past + n, att, D ** -0.5,
                              workspace=ws)
        mid = self.o(att.view(n, H * D))
        stream = torch.empty_like(x)
        codes, scales = torch.empty_like(x), torch.empty(n, device="cuda")
        mnb.mnb_rms_norm(mid, self.norm2, codes, EPS, residual=x, residual_out=stream, scales=scales)
        g, u = self.gate.from_codes(codes, scales), self.up.from_codes(codes, scales)
        return self.down((g * torch.sigmoid(g) * u).half(), out_bias=stream), (qkv, q, att, stream, kv_len, q_start)

    def plain(self, x, past, inner):
        """The same in plain torch, from the library's own qkv product on (its rounding decides codes)."""
        qkv, q, _, _, kv_len, _ = inner
        n, H, Hkv, D = x.shape[0], self.q_heads, self.kv_heads, self.dim
        f = x.float()
        a = f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * self.norm1.float()
        worst = [(a.half().float() @ self.qkv.values.T - qkv.view(n, -1).float()).abs().max()]
        pos = torch.arange(past, past + n, device="cuda")
        c, s = self.cos[pos][:, None], self.sin[pos][:, None]
        x1, x2 = qkv[:, :H, :D // 2].float(), qkv[:, :H, D // 2:].float()
        qr = torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)
        worst.append((qr - q.float()).abs().max())
        total = past + n
        k, v = (torch.empty((total, Hkv, D), dtype=torch.float32, device="cuda") for _ in range(2))
        every = torch.tensor([0, total], dtype=torch.int32, device="cuda")
        mnb.mnb_kv4_read(self.kv, self.cache, self.table, kv_len, every, k, v)
        per = H // Hkv
        k, v = k.repeat_interleave(per, 1), v.repeat_interleave(per, 1)
        logits = torch.stack([q[:, h].float() @ k[:, h].T for h in range(H)], 1) * D ** -0.5
        logits = logits.masked_fill((torch.arange(total, device="cuda")[None] > pos[:, None])[:, None], float("-inf"))
        p = torch.softmax(logits, -1)
        att = torch.stack([p[:, h] @ v[:, h] for h in range(H)], 1)
        stream = (x.float() + (att.half().reshape(n, -1).float() @ self.o.values.T).half().float()).half().float()
        b = stream * torch.rsqrt(stream.square().mean(1, keepdim=True) + EPS) * self.norm2.float()
        sc = b.abs().amax(1, keepdim=True) / 127
        b = (b / sc).round() * sc
        g, u = b @ self.gate.values.T, b @ self.up.values.T
        y = stream + (g * torch.sigmoid(g) * u).half().float() @ self.down.values.T
        return y, worst + [(att - inner[2].float()).abs().max(), (stream - inner[3].float()).abs().max()]


def run(hidden=512, q_heads=8, kv_heads=2, dim=64, ffn=1024, prompt=100, steps=8, seed=0):
    """Largest differences over a prompt and `steps` tokens: (qkv, rotated q, attention, stream, output)."""
    layer = Layer(hidden, q_heads, kv_heads, dim, ffn, prompt + steps, seed=seed)
    worst = [0.0] * 5
    past = 0
    for n in [prompt] + [1] * steps:
        x = torch.randn(n, hidden, generator=layer.gen, device="cuda").half()
        y, inner = layer(x, past)
        want, diffs = layer.plain(x, past, inner)
        for i, d in enumerate(diffs + [(want - y.float()).abs().max()]):
            worst[i] = max(worst[i], float(d))
        past += n
    return worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    names = ("qkv", "rotated q", "attention", "stream", "output")
    print("largest differences from plain torch: " +
          ", ".join("%s %.2g" % nv for nv in zip(names, run(hidden=a.hidden, prompt=a.prompt, steps=a.steps))))
