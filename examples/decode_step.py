"""One decoder layer and the vocabulary's projection, from a prompt to generated
tokens, through the library's calls: what a serving program does between the
products on GGUF weights.

    python examples/decode_step.py [--tokens 8]

Weights are random Q8_0 blocks, so the text is noise; the point is the
order of the calls and who owns what.  Per step

    gguf_mm_gemm        hidden -> q, k, v in one projection
    gguf_kv_append      q and k turned to their positions, k and v into the pages
    gguf_paged_attn     the new tokens over every key so far
    gguf_mm_gemm        attention -> hidden, the residual added in its store
    gguf_mm_gemm        hidden -> logits of each sequence's last token
    gguf_logits_adjust  penalties for what was generated, a bias, a mask

The prompt is one call of several tokens a sequence, each later step one token a
sequence; only the arrays of the batch change.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gguf_quant_weight_gb300 as g  # noqa: E402
import gguf_synth as syn  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, VOCAB, PAGE = 1024, 16, 4, 64, 4096, 32
DEV = "cuda"


class Layer:
    """The weights, as their GGUF blocks on the device, and the pages of the cache."""

    def __init__(self, n_pages, seed=0):
        rs = syn.rng(seed)
        blocks = lambda qt, n, k: (torch.from_numpy(syn.weight_blocks(rs, qt, n, k)).to(DEV), qt, n, k)  # noqa: E731
        self.qkv = blocks(syn.Q8_0, (HEADS + 2 * KV_HEADS) * DIM, HIDDEN)
        self.out = blocks(syn.Q8_0, HIDDEN, HEADS * DIM)
        self.vocab = blocks(syn.Q8_0, VOCAB, HIDDEN)
        self.embed = torch.randn((VOCAB, HIDDEN), generator=torch.Generator().manual_seed(seed)).to(DEV, torch.bfloat16)
        shape = (n_pages, KV_HEADS, PAGE, DIM)
        self.k, self.v = (torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.cache = g.gguf_kv_cache(self.k, self.v)
        i = torch.arange(DIM // 2, dtype=torch.float64)
        self.rope = g.gguf_rope((10000.0 ** (-2 * i / DIM)).float().to(DEV), DIM, g.GGUF_ROPE_NEOX)


def product(x, weight, residual=None, dtype=torch.bfloat16):
    w, qt, n, k = weight
    dt = {torch.bfloat16: g.GGUF_DT_BF16, torch.float32: g.GGUF_DT_F32}[dtype]
    y = torch.empty((x.shape[0], n), dtype=dtype, device=DEV)
    size = g.gguf_mm_workspace_size(g.GGUF_OP_GEMM, qt, n, k, x.shape[0])
    ws = torch.empty(max(16, size), dtype=torch.uint8, device=DEV)
    g.gguf_mm_gemm(w, qt, 0, n, k, x, g.GGUF_DT_BF16, x.shape[0], residual, y, dt, ws, size)
    return y


def norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-5)).to(torch.bfloat16)


def step(layer, tokens, counts, kv_len, pages, max_kv, rules):
    """tokens: the new tokens of all sequences one after the other, counts[b] of sequence b.  Returns
    the adjusted logits of each sequence's last token."""
    start = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device=DEV)
    batch = g.gguf_kv_batch(start, kv_len, pages, len(tokens), max(counts), max_kv)
    x = layer.embed[tokens]
    qkv = product(norm(x), layer.qkv)
    ld = qkv.stride(0)
    q, k, v = qkv.split((HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM), dim=1)
    turned, heads = (torch.empty((len(tokens), HEADS * DIM), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g.gguf_kv_append(q, ld, k, ld, v, ld, g.GGUF_DT_BF16, HEADS, layer.rope, batch, layer.cache, turned, HEADS * DIM)
    size = g.gguf_paged_attn_workspace_size(batch, layer.cache, HEADS)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device=DEV)
    g.gguf_paged_attn(turned, HEADS * DIM, HEADS, batch, layer.cache, DIM ** -0.5, 1, 0, heads, HEADS * DIM, None, ws, size)
    x = product(heads, layer.out, residual=x)
    logits = product(norm(x[(start[1:] - 1).long()]), layer.vocab, dtype=torch.float32)
    g.gguf_logits_adjust(logits, g.GGUF_DT_F32, VOCAB, len(counts), VOCAB, rules, logits, g.GGUF_DT_F32, VOCAB)
    return logits


def generate(n_tokens=8, prompts=(5, 40, 1), seed=0):
    """The generated tokens [sequence][n_tokens], greedily."""
    room = [-(-(p + n_tokens) // PAGE) for p in prompts]
    layer = Layer(sum(room), seed)
    pages = torch.full((len(prompts), max(room)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, r in enumerate(room):
        pages[b, :r] = torch.arange(at, at + r, dtype=torch.int32)
        at += r
    max_kv = max(room) * PAGE
    rs = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, VOCAB, (sum(prompts),), generator=rs).to(DEV)
    counts, kv_len = list(prompts), torch.tensor(prompts, dtype=torch.int32, device=DEV)
    B = len(prompts)
    made = torch.empty((B, 0), dtype=torch.int32, device=DEV)
    one = lambda v: torch.full((B,), v, device=DEV)  # noqa: E731
    allow = torch.full((B, VOCAB // 32), 0x55555555, dtype=torch.int32, device=DEV)      # even tokens only
    for _ in range(n_tokens):
        rules = g.gguf_logit_rules(hist=made.reshape(-1), hist_start=torch.arange(B + 1, dtype=torch.int32, device=DEV) * made.shape[1],
                                   repeat=one(1.3), frequency=one(0.1), presence=one(0.4),
                                   bias_ids=torch.zeros(B, dtype=torch.int32, device=DEV), bias=one(-100.0),
                                   bias_start=torch.arange(B + 1, dtype=torch.int32, device=DEV), allow=allow)
        tokens = step(layer, tokens, counts, kv_len, pages, max_kv, rules).argmax(-1)
        made = torch.cat((made, tokens[:, None].to(torch.int32)), dim=1).contiguous()
        counts, kv_len = [1] * B, kv_len + 1
    torch.cuda.synchronize()
    status = g.gguf_mm_check_errors()
    if status != 0:
        raise RuntimeError(g.status_string(status))
    return made


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=8)
    for row in generate(ap.parse_args().tokens).tolist():
        print(row)
