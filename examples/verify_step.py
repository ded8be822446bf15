"""Speculative-decode steps of a small decoder on one GPU, everything between the projections in the
library's kernels: K and V in the 4-bit paged cache, tree attention over it, grouped routing and the
NVFP4 experts, then the accepted tokens kept and a branch forked.  Random weights; the projections
are plain matrix products, or with --fp8 the library's: norms that write rows in 8 bits, projections and a
vocabulary in 8 bits with a scale for 128 x 128, and draft tokens accepted by their log probabilities.

    python examples/verify_step.py [--fp8]

No call waits for the GPU: lengths, page tables and acceptance stay on the device, so a step can be
captured in a CUDA graph.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Decoder:
    """`layers` layers of attention and routed experts over one cache of `seqs` sequences."""

    def __init__(self, layers=2, d=256, heads=8, kv_heads=2, head_dim=64, experts=32, ffn=256, k=4, groups=4, seqs=4,
                 pages=64, page_size=32, max_rows=8, seed=0, fp8=False, vocab=1000):
        import routed_moe_decode_gb300 as moe
        self.moe, self.layers, self.d, self.heads, self.max_rows = moe, layers, d, heads, max_rows
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=None):
            return (torch.randn(*shape, generator=gen, device="cuda") * (std or shape[-1] ** -0.5)).to(torch.bfloat16)

        def codes(*shape):
            return torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)

        def scales(*shape):  # E4M3 values from 1/8 to 1/4
            return torch.randint(0x20, 0x28, shape, generator=gen, device="cuda", dtype=torch.uint8)

        self.cache = moe.Kv4Cache(layers=layers, pages=pages, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size,
                                  seqs=seqs, max_pages=pages)
        self.routing = moe.Routing(experts, k, score="sigmoid", groups=groups, keep_groups=(groups + 1) // 2,
                                   group_score="top2", scale=1.0)
        self.weights = [dict(
            qkv=normal((heads + 2 * kv_heads) * head_dim, d), out=normal(d, heads * head_dim), router=normal(experts, d),
            bias=0.1 * torch.randn(experts, generator=gen, device="cuda"),
            experts=dict(w13_codes=codes(experts, 2 * ffn, d // 2), w13_scales=scales(experts, 2 * ffn, d // 16), w13_ts=0.1,
                         w2_codes=codes(experts, d, ffn // 2), w2_scales=scales(experts, d, ffn // 16), w2_ts=0.1))
            for _ in range(layers)]
        self.ffn, self.experts, self.k, self.vocab = ffn, experts, k, vocab
        self._layers = {}
        self.fp8 = fp8
        if fp8:
            def norm():
                return moe.RmsNorm(0.1 * torch.randn(d, generator=gen, device="cuda"), one_plus=True)

            for w in self.weights:
                w["attn_norm"], w["moe_norm"] = norm(), norm()
                w["qkv"], w["out"] = (moe.Fp8Linear(*quantized_weight(w[n])) for n in ("qkv", "out"))
            self.final_norm, self.head = norm(), moe.Fp8Linear(*quantized_weight(normal(vocab, d)))

    def _moe(self, rows):
        """The routed layer for `rows` rows (one workspace per number of rows)."""
        if rows not in self._layers:
            self._layers[rows] = self.moe.MoeLayer(rows, self.d, self.ffn, self.experts, self.k, routing=self.routing)
        return self._layers[rows]

    def forward(self, x, cu_rows, new_tokens, tree=None):
        """One step of x [rows, d] (cu_rows, new_tokens: on the device): the rows' outputs."""
        c = self.cache
        c.reserve(new_tokens)
        hq, hk, hd = self.heads, c.kv_heads, c.head_dim
        layer = self._moe(x.shape[0])
        logits = torch.empty((x.shape[0], self.experts), dtype=torch.float32, device="cuda")
        if self.fp8:
            return self._layers_fp8(x, cu_rows, tree, layer, logits)
        for i, w in enumerate(self.weights):
            qkv = (rms_norm(x) @ w["qkv"].t()).view(x.shape[0], hq + 2 * hk, hd)
            c.append(i, qkv[:, hq:hq + hk], qkv[:, hq + hk:], cu_rows)
            heads = c.attend(i, qkv[:, :hq], cu_rows, max_rows=self.max_rows, tree=tree)
            x = x + heads.flatten(1) @ w["out"].t()
            normed = rms_norm(x)
            self.moe.router_logits(layer.shape, normed, w["router"], logits)
            x = layer(logits, normed, w["experts"], residual=x, router_bias=w["bias"])
        return x

    def _layers_fp8(self, x, cu_rows, tree, layer, logits):
        """The layers with the dense path in 8 bits; x is the residual stream."""
        moe, c = self.moe, self.cache
        hq, hk, hd = self.heads, c.kv_heads, c.head_dim
        for i, w in enumerate(self.weights):
            _, _, rows = w["attn_norm"](x, normed=False, quantize=True)
            qkv = w["qkv"](rows).view(x.shape[0], hq + 2 * hk, hd)
            c.append(i, qkv[:, hq:hq + hk], qkv[:, hq + hk:], cu_rows)
            heads = c.attend(i, qkv[:, :hq], cu_rows, max_rows=self.max_rows, tree=tree)
            delta = w["out"](moe.quantize_rows(heads.flatten(1)))
            normed, x, _ = w["moe_norm"](delta, residual=x)
            moe.router_logits(layer.shape, normed, w["router"], logits)
            x = layer(logits, normed, w["experts"], residual=x, router_bias=w["bias"])
        return x

    def scores(self, x, tokens, top=0):
        """Log probabilities of each row's tokens [rows, n] int32 after the final norm and the vocabulary (fp8)."""
        _, _, rows = self.final_norm(x, normed=False, quantize=True)
        return self.moe.token_logprobs(self.head(rows, dtype=torch.float32), tokens, top=top)


def quantized_weight(w):
    """A weight [n, k] as E4M3 codes and one FP32 scale for 128 x 128 of it."""
    n, k = w.shape
    padded = torch.nn.functional.pad(w.float(), (0, -k % 128, 0, -n % 128))
    blocks = padded.view(padded.shape[0] // 128, 128, padded.shape[1] // 128, 128)
    scales = blocks.abs().amax((1, 3)).clamp(min=1e-30) / 448.0
    codes = (blocks / scales[:, None, :, None]).view_as(padded)[:n, :k]
    return codes.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).contiguous(), scales


def rms_norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def chain_tree(rows):
    """Tree bits of a step without branches: row i sees the step's rows 0 .. i."""
    return [(1 << (i + 1)) - 1 for i in range(rows)]


def main(prompts=(37, 64, 5), steps=3, seed=0, fp8=False):
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    seqs = len(prompts) + 1  # the last one starts as a fork
    m = Decoder(seqs=seqs, seed=seed, fp8=fp8)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def rows_of(counts):
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        return ints(cu), ints(counts), cu[-1]

    def states(n):
        return torch.randn(n, m.d, generator=gen, device="cuda").to(torch.bfloat16)

    counts = list(prompts) + [0]
    cu, new, total = rows_of(counts)
    m.forward(states(total), cu, new)                           # the prompts
    m.cache.fork(ints([0]), ints([seqs - 1]))                   # a second answer to the first prompt
    # a draft of 7 tokens a sequence: two branches after the first token
    parents = [-1, 0, 0, 1, 2, 3, 4]
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
    kept = torch.zeros(seqs, dtype=torch.int64, device="cuda")
    for _ in range(steps):
        cu, new, total = rows_of([len(parents)] * seqs)
        tree = torch.tensor(bits * seqs, dtype=torch.int64, device="cuda")
        out = m.forward(states(total), cu, new, tree=tree)
        # accept one branch as far as a (made-up) check of its rows agrees, on the device: with fp8, a row's next token
        # in the draft is likelier than an even choice
        if fp8:
            drafted = torch.randint(0, m.vocab, (out.shape[0],), generator=gen, device="cuda").to(torch.int32)
            ok = (m.scores(out, drafted).logprobs > -math.log(m.vocab)).view(seqs, -1)
        else:
            ok = (out.float().mean(-1) > -0.05).view(seqs, -1)
        take = torch.zeros_like(ok)
        take[:, 0] = True
        for i, p in enumerate(parents[1:], 1):
            if i % 2 == 1:
                take[:, i] = ok[:, i] & take[:, p]
        m.cache.compact(take.flatten().to(torch.uint8), cu, max_rows=len(parents))
        kept += take.sum(-1)
    return m, kept


if __name__ == "__main__":
    decoder, kept = main(fp8="--fp8" in sys.argv[1:])
    torch.cuda.synchronize()
    print("tokens of each sequence:", decoder.cache.lens.tolist(), "accepted:", kept.tolist(),
          "pages in use:", int((decoder.cache.refs > 0).sum()), "status:", decoder.cache.status())
