"""One decoder layer with a mixture of experts, from a prompt to drawn tokens: the
calls of decode_step.py with normed query and key heads, experts in the
place of a dense feed-forward, and sampling instead of the largest logit.

    python examples/moe_decode_step.py [--tokens 8] [--eager]

Weights are random blocks, so the text is noise; the point is the order of the
calls and who owns what.  Per step

    gguf_mm_gemm          hidden -> q, k, v in one projection
    gguf_kv_append_norm   q and k normed head by head and turned, k and v into the pages
    gguf_paged_attn       the new tokens over every key so far
    gguf_mm_gemm          attention -> hidden, the residual added in its store
    gguf_moe_router       each token's experts and their weights
    gguf_moe_ffn          the tokens through those experts, the residual added in its store
    gguf_mm_gemm          hidden -> logits of each sequence's last token
    gguf_logits_adjust    a mask, penalties
    gguf_sample           temperature, top-k, top-p, min-p and the draw

The prompt is one call of several tokens a sequence.  The steps after it work in
fixed buffers and are captured into a CUDA graph once: a step is then one launch.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gguf_quant_weight_gb300 as g  # noqa: E402
import gguf_synth as syn  # noqa: E402
from examples.decode_step import DEV, DIM, HEADS, HIDDEN, KV_HEADS, PAGE, VOCAB, Layer, norm, product  # noqa: E402

EXPERTS, TOP_K, INNER = 16, 4, 512
BF16 = g.GGUF_DT_BF16


class MoeLayer(Layer):
    """Layer's weights and cache, the heads' norms, the router and the experts."""

    def __init__(self, n_pages, seed=0):
        super().__init__(n_pages, seed)
        rs, gen = syn.rng(seed + 1), torch.Generator().manual_seed(seed + 1)
        draw = lambda *s: torch.randn(s, generator=gen).to(DEV)  # noqa: E731
        self.head_norm = g.gguf_head_norm(1 + 0.1 * draw(DIM), 1 + 0.1 * draw(DIM))
        self.router = g.gguf_router(draw(EXPERTS, HIDDEN) * HIDDEN ** -0.5, TOP_K)
        self.types = syn.Q4_K, syn.Q4_K, syn.Q6_K
        shapes = (INNER, HIDDEN), (INNER, HIDDEN), (HIDDEN, INNER)
        self.blocks = [torch.from_numpy(syn.weight_blocks(rs, qt, EXPERTS * n, k)).to(DEV) for qt, (n, k) in zip(self.types, shapes)]
        self.experts = g.gguf_moe_weights(*self.blocks, *self.types, HIDDEN, INNER, EXPERTS)


def feed_forward(layer, x):
    """x + the experts' share of it.  Prompts go in pieces that one call takes."""
    h, y = norm(x), torch.empty_like(x)
    ids = torch.empty((len(x), TOP_K), dtype=torch.int32, device=DEV)
    weights = torch.empty((len(x), TOP_K), dtype=torch.float32, device=DEV)
    g.gguf_moe_router(h, BF16, len(x), HIDDEN, layer.router, ids, weights)
    most = 512 // TOP_K
    for a in range(0, len(x), most):
        b = min(len(x), a + most)
        size = g.gguf_moe_ffn_workspace_size(INNER, b - a, TOP_K)
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        g.gguf_moe_ffn(layer.experts, h[a:b], BF16, b - a, ids[a:b], weights[a:b], TOP_K, x[a:b], y[a:b], BF16, ws, size)
    return y, (h, ids, weights)


def step(layer, tokens, start, kv_len, pages, max_q, max_kv, rules, sampler, u, seen=None):
    """Draws each sequence's next token: int32 [sequence].  `seen`, a dict, receives what the operators had and gave."""
    T, B = len(tokens), len(kv_len)
    batch = g.gguf_kv_batch(start, kv_len, pages, T, max_q, max_kv)
    x = layer.embed[tokens.long()]
    qkv = product(norm(x), layer.qkv)
    ld = qkv.stride(0)
    q, k, v = qkv.split((HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM), dim=1)
    turned, heads = (torch.empty((T, HEADS * DIM), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g.gguf_kv_append_norm(q, ld, k, ld, v, ld, BF16, HEADS, layer.head_norm, layer.rope, batch, layer.cache, turned, HEADS * DIM)
    size = g.gguf_paged_attn_workspace_size(batch, layer.cache, HEADS)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device=DEV)
    g.gguf_paged_attn(turned, HEADS * DIM, HEADS, batch, layer.cache, DIM ** -0.5, 1, 0, heads, HEADS * DIM, None, ws, size)
    x = product(heads, layer.out, residual=x)
    y, routed = feed_forward(layer, x)
    logits = product(norm(y[(start[1:] - 1).long()]), layer.vocab, dtype=torch.float32)
    g.gguf_logits_adjust(logits, g.GGUF_DT_F32, VOCAB, B, VOCAB, rules, logits, g.GGUF_DT_F32, VOCAB)
    token = torch.empty(B, dtype=torch.int32, device=DEV)
    logprob = torch.empty(B, dtype=torch.float32, device=DEV)
    g.gguf_sample(logits, g.GGUF_DT_F32, VOCAB, B, VOCAB, sampler, u, token, logprob)
    if seen is not None:
        seen.update(q=q, k=k, v=v, turned=turned, x=x, y=y, routed=routed, logits=logits, token=token, logprob=logprob)
    return token


def generate(n_tokens=8, prompts=(5, 40, 1), seed=0, graph=True, watch=None):
    """The drawn tokens [sequence][n_tokens]; watch(layer, seen, start, kv_len, pages) is called after each eager step."""
    room = [-(-(p + n_tokens) // PAGE) for p in prompts]
    layer, B = MoeLayer(sum(room), seed), len(prompts)
    pages = torch.full((B, max(room)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, r in enumerate(room):
        pages[b, :r] = torch.arange(at, at + r, dtype=torch.int32)
        at += r
    max_kv = max(room) * PAGE
    gen = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, VOCAB, (sum(prompts),), generator=gen).to(DEV)
    draws = torch.rand((n_tokens, B), generator=gen).to(DEV)
    allow = torch.full((B, VOCAB // 32), 0x55555555, dtype=torch.int32, device=DEV)      # even tokens only
    rules = g.gguf_logit_rules(allow=allow)
    one = lambda v, dt=torch.float32: torch.full((B,), v, dtype=dt, device=DEV)  # noqa: E731
    sampler = g.gguf_sampler(one(0.8), one(50, torch.int32), one(0.95), one(0.02))
    start = torch.tensor([0] + list(torch.tensor(prompts).cumsum(0)), dtype=torch.int32, device=DEV)
    ones = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    kv_len = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    u = draws[0].clone()

    def run(tokens, start, max_q):
        seen = None if watch is None else {}
        token = step(layer, tokens, start, kv_len, pages, max_q, max_kv, rules, sampler, u, seen)
        if watch is not None:
            watch(layer, seen, start, kv_len, pages)
        return token

    last = run(tokens, start, max(prompts)).clone()
    made = [last.clone()]

    def one_step():
        kv_len.add_(1)
        last.copy_(run(last, ones, 1))

    replay = one_step
    if graph and n_tokens > 1:
        # a step ahead of the capture, as libraries set themselves up in their first calls; what it changed is put back
        kept = last.clone(), kv_len.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            one_step()
            last.copy_(kept[0]), kv_len.copy_(kept[1])
        torch.cuda.current_stream().wait_stream(side)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            one_step()
        replay = captured.replay
    for i in range(1, n_tokens):
        u.copy_(draws[i])
        replay()
        made.append(last.clone())
    torch.cuda.synchronize()
    status = g.gguf_mm_check_errors()
    if status != 0:
        raise RuntimeError(g.status_string(status))
    return torch.stack(made, 1)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--eager", action="store_true")
    args = ap.parse_args()
    for row in generate(args.tokens, graph=not args.eager).tolist():
        print(row)
