"""The serving operators next to the quantized matmuls, as they are measured.

Three operators carry a decode step between the projections and the sampled token:

  append   gguf_kv_append      rotates the new queries and keys to their positions and writes keys and values into a paged cache
  attn     gguf_paged_attn     attention of each sequence's new tokens (a prompt, a chunk or one token) over that cache
  logits   gguf_logits_adjust  penalties for repeated tokens, biases and a grammar's mask on the logits

`own` chooses between the library's calls (True) and their plain form in elementary torch operations (False).

A batch of sequences is ragged: sequence b's new tokens are rows q_start[b] .. q_start[b+1] of the packed inputs, and
kv_len[b] counts its keys with the new ones, so that its j-th new token stands at position kv_len[b] - n_b + j.  Its keys
live in the pages that row b of the page table names.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one user's next token: a handful of microseconds between two matrix-vector products
        dict(name="append_token", op="append", xdt="bf16", dt="bf16", seqs=1, q=1, q_hi=1, past=1000, past_hi=1000, heads=32,
             kv_heads=8, dim=128, rot=128, style=0, page=16, layout="hnd", fused=True, lens=1),
        # a serving batch: most sequences add one token, some a chunk of a prompt; rotation of part of the head in halves
        dict(name="append_mixed", op="append", xdt="f16", dt="f16", seqs=48, q=1, q_hi=90, past=0, past_hi=700, heads=24,
             kv_heads=8, dim=96, rot=48, style=1, page=32, layout="nhd", fused=False, lens=2),
        # whole prompts, f32 rows of a fused projection into a bf16 cache
        dict(name="append_prompts", op="append", xdt="f32", dt="bf16", seqs=5, q=900, q_hi=2500, past=0, past_hi=64, heads=32,
             kv_heads=8, dim=128, rot=128, style=1, page=64, layout="hnd", fused=True, lens=3),
        # one user, one token, a short conversation: latency alone
        dict(name="attn_token", op="attn", dt="bf16", seqs=1, q=1, q_hi=1, past=1020, past_hi=1020, heads=32, kv_heads=8,
             dim=128, page=16, layout="hnd", causal=True, window=0, lens=4),
        # a decode batch with histories of every length: the cache's bytes
        dict(name="attn_token_batch", op="attn", dt="bf16", seqs=64, q=1, q_hi=1, past=100, past_hi=8000, heads=32, kv_heads=8,
             dim=128, page=16, layout="hnd", causal=True, window=0, lens=5),
        # one token after a very long document, f16, no shared heads' luxury of a batch
        dict(name="attn_token_long", op="attn", dt="f16", seqs=1, q=1, q_hi=1, past=131070, past_hi=131070, heads=16, kv_heads=4,
             dim=128, page=64, layout="nhd", causal=True, window=0, lens=6),
        # chunks of prompts together with single tokens, every head its own keys
        dict(name="attn_chunks", op="attn", dt="f16", seqs=24, q=1, q_hi=500, past=0, past_hi=3000, heads=16, kv_heads=16, dim=64,
             page=32, layout="hnd", causal=True, window=0, lens=7),
        # long chunks under a sliding window, three heads to a key head, an odd head size
        dict(name="attn_window", op="attn", dt="bf16", seqs=3, q=1500, q_hi=2100, past=0, past_hi=2500, heads=24, kv_heads=8,
             dim=96, page=16, layout="nhd", causal=True, window=1000, lens=8),
        # a long prompt: the tensor cores' work
        dict(name="attn_prompt", op="attn", dt="bf16", seqs=1, q=8111, q_hi=8111, past=0, past_hi=0, heads=32, kv_heads=8, dim=128,
             page=64, layout="hnd", causal=True, window=0, lens=9),
        # one user's logits, every rule on
        dict(name="logits_token", op="logits", dt="f32", odt="f32", rows=1, vocab=32003, hist=300, hist_hi=300, bias=20,
             grammar=True, lens=10),
        # a batch whose rows have histories of every length, none among them
        dict(name="logits_batch", op="logits", dt="bf16", odt="f32", rows=37, vocab=128259, hist=0, hist_hi=4096, bias=64,
             grammar=True, lens=11),
        # a large batch without a grammar
        dict(name="logits_large", op="logits", dt="f32", odt="f32", rows=256, vocab=131072, hist=1, hist_hi=2048, bias=0,
             grammar=False, lens=12),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    while True:
        c = _draw(rng)
        if c["op"] == "logits":
            if c["rows"] * c["vocab"] <= 256 * 131072:
                return c
            continue
        n, past = _lens(c)
        tokens, keys = sum(n), sum(a + b for a, b in zip(n, past))
        if c["op"] == "append":
            if tokens * (c["heads"] + 2 * c["kv_heads"]) * c["dim"] <= 8000 * 48 * 128 and keys <= 60000:
                return c
            continue
        padded = c["seqs"] * max(a + b for a, b in zip(n, past))     # what the plain form gathers
        if (work(c)["flops"] <= 5e11 and padded * c["heads"] * max(n) <= 32 * 8111 ** 2 and
                padded * c["kv_heads"] * c["dim"] <= 64 * 8100 * 8 * 128):
            return c


def _draw(rng):
    op = rng.choice(("append", "attn", "attn", "logits"))
    if op == "logits":
        hist = rng.choice((0, 1, _log(rng, 1, 4000)))
        return dict(op=op, dt=rng.choice(("f32", "f16", "bf16")), odt="f32", rows=_log(rng, 1, 256), vocab=_log(rng, 1000, 160000),
                    hist=hist, hist_hi=hist + _log(rng, 1, 4000), bias=rng.choice((0, 1, _log(rng, 1, 300))),
                    grammar=rng.random() < 0.6, lens=rng.randrange(1 << 20))
    kv_heads = rng.choice((1, 2, 4, 8, 16))
    group = rng.choice((1, 2, 3, 4, 5, 7, 8))
    dim = rng.choice((64, 64, 80, 96, 128, 128, 128))
    both = dict(dt=rng.choice(("f16", "bf16")), heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=rng.choice((16, 32, 64, 128)),
                layout=rng.choice(("hnd", "nhd")), lens=rng.randrange(1 << 20))
    form = rng.choice(("token", "chunk", "prompt"))
    seqs = _log(rng, 1, 96) if form == "token" else _log(rng, 1, 24) if form == "chunk" else _log(rng, 1, 4)
    q_hi = 1 if form == "token" else _log(rng, 2, 500) if form == "chunk" else _log(rng, 300, 8000)
    q = rng.choice((1, max(1, q_hi // 2), q_hi))
    past_hi = _log(rng, 1, 30000 if form == "token" else 5000) if rng.random() < 0.8 else 0
    past = rng.choice((0, past_hi // 2, past_hi))
    more = dict(seqs=seqs, q=q, q_hi=q_hi, past=past, past_hi=past_hi)
    if op == "append":
        return dict(op=op, xdt=rng.choice(("f32", "f16", "bf16")), rot=rng.choice((dim, dim, dim // 2)), style=rng.randrange(2),
                    fused=rng.random() < 0.5, **more, **both)
    return dict(op=op, causal=rng.random() < 0.85, window=rng.choice((0, 0, 0, _log(rng, 16, 4000))), **more, **both)


def _lens(c):
    """New tokens and earlier keys of each sequence: the case's own, the same for every seed."""
    r = random.Random(c["lens"])
    n = [_log(r, c["q"], c["q_hi"]) for _ in range(c["seqs"])]
    past = [min(c["past_hi"], max(c["past"], _log(r, c["past"] + 1, c["past_hi"] + 1) - 1)) for _ in range(c["seqs"])]
    return n, past


def _hist_lens(c):
    r = random.Random(c["lens"])
    return [r.randint(c["hist"], c["hist_hi"]) for _ in range(c["rows"])]


def _seen(a, b, causal, window):
    """Keys that `a` new tokens after `b` earlier ones attend to, added up over the tokens."""
    total = 0
    for p in range(b, b + a):
        total += (p + 1 if causal else a + b) - (max(0, p + 1 - window) if window else 0)
    return total


def work(case):
    c = case
    if c["op"] == "logits":
        n = c["rows"] * c["vocab"]
        size = {"f32": 4, "f16": 2, "bf16": 2}
        b = n * (size[c["dt"]] + size[c["odt"]]) + 4 * sum(_hist_lens(c)) + 8 * c["bias"] * c["rows"]
        return {"bytes": b + (n // 8 if c["grammar"] else 0), "flops": 4 * n}
    n, past = _lens(c)
    tokens, D, H, KV = sum(n), c["dim"], c["heads"], c["kv_heads"]
    if c["op"] == "append":
        x = 4 if c["xdt"] == "f32" else 2
        return {"bytes": tokens * (H + 2 * KV) * D * (x + 2), "flops": tokens * (H + KV) * c["rot"] * 3}
    pairs = sum(_seen(a, b, c["causal"], c["window"]) for a, b in zip(n, past))
    keys = sum(a + (min(b, c["window"] - 1) if c["window"] else b) for a, b in zip(n, past))
    return {"bytes": 2 * tokens * H * D * 2 + 4 * tokens * H + 2 * keys * KV * D * 2, "flops": 4 * pairs * H * D}


# ---------------------------------------------------------------- the inputs

def _batch(c, g):
    """The ragged batch's arrays and a page table with the pages in no order; entries past a sequence's end hold -1."""
    n, past = _lens(c)
    total = [a + b for a, b in zip(n, past)]
    page = c["page"]
    need = [-(-t // page) for t in total]
    wide = max(need)
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(wide, device=DEV)
    need_t = torch.tensor(need, device=DEV)
    first = torch.cumsum(need_t, 0) - need_t
    at = (first[:, None] + col).clamp(max=n_pages - 1)
    pages = torch.where(col < need_t[:, None], order[at], torch.full_like(at, -1, dtype=torch.int32))
    start = torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=DEV)
    return dict(q_start=start, kv_len=torch.tensor(total, dtype=torch.int32, device=DEV), pages=pages.contiguous(), n_pages=n_pages,
                tokens=sum(n), max_q=max(n), max_kv=max(total))


def _cache(c, n_pages, g, dt):
    """Keys or values as [page, head, token, dim], whatever the order in memory."""
    shape = (n_pages, c["kv_heads"], c["page"], c["dim"])
    if c["layout"] == "nhd":
        shape = (shape[0], shape[2], shape[1], shape[3])
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    x += 0.4 * torch.randn(shape[-1], generator=g, device=DEV)       # the channels' own offsets
    x = x.to(dt)
    return x if c["layout"] == "hnd" else x.transpose(1, 2)


def _inputs(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    if c["op"] == "logits":
        return _logits_inputs(c, g)
    s = _batch(c, g)
    dt, D, H, KV, T = DT[c["dt"]], c["dim"], c["heads"], c["kv_heads"], s["tokens"]
    s["k_cache"], s["v_cache"] = _cache(c, s["n_pages"], g, dt), _cache(c, s["n_pages"], g, dt)
    if c["op"] == "append":
        x = DT[c["xdt"]]
        if c["fused"]:      # the rows of one fused projection
            qkv = torch.randn((T, (H + 2 * KV) * D), generator=g, device=DEV).to(x)
            s["q"], s["k"], s["v"] = (t.view(T, -1, D) for t in qkv.split((H * D, KV * D, KV * D), dim=1))
        else:
            s["q"], s["k"], s["v"] = (torch.randn((T, h, D), generator=g, device=DEV).to(x) for h in (H, KV, KV))
        i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
        s["freqs"] = (10000.0 ** (-2.0 * i / c["rot"])).to(torch.float32)
        s["q_out"] = torch.zeros((T, H, D), device=DEV, dtype=dt)
        return s
    s["q"] = (1.5 * torch.randn((T, H, D), generator=g, device=DEV)).to(dt)
    # what the slots after a sequence's last key held before is anything at all
    last = (s["kv_len"] - 1).to(torch.int64)
    page = s["pages"].gather(1, (last // c["page"])[:, None])[:, 0].to(torch.int64)
    after = torch.arange(c["page"], device=DEV) > (last % c["page"])[:, None]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[page] = torch.where(after[:, None, :, None], torch.full_like(cache[page], math.nan), cache[page])
    s["out"] = torch.empty((T, H, D), device=DEV, dtype=dt)
    s["lse"] = torch.empty((T, H), device=DEV, dtype=torch.float32)
    return s


def _logits_inputs(c, g):
    rows, V = c["rows"], c["vocab"]
    lens = _hist_lens(c)
    start = torch.tensor([sum(lens[:i]) for i in range(rows + 1)], dtype=torch.int32, device=DEV)
    s = dict(logits=(3.0 * torch.randn((rows, V), generator=g, device=DEV)).to(DT[c["dt"]]), hist_start=start)
    # text repeats itself: most of a history is a few hundred tokens
    u = torch.rand((sum(lens) + 1,), generator=g, device=DEV)
    s["hist"] = (u ** 4 * (V - 1)).to(torch.int32)[:sum(lens)]
    s["repeat"] = 1.0 + 0.3 * torch.rand((rows,), generator=g, device=DEV)
    s["frequency"] = 0.2 * torch.rand((rows,), generator=g, device=DEV)
    s["presence"] = 0.5 * torch.rand((rows,), generator=g, device=DEV)
    b = c["bias"]
    s["bias_start"] = torch.arange(rows + 1, device=DEV, dtype=torch.int32) * b
    s["bias_ids"] = torch.randint(0, V, (rows * b,), generator=g, device=DEV, dtype=torch.int32)
    s["bias"] = torch.randn((rows * b,), generator=g, device=DEV)
    words = -(-V // 32)
    if c["grammar"]:        # a grammar allows about one token in sixteen
        m = torch.randint(-2 ** 31, 2 ** 31, (4, rows, words), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
        s["allow"] = m[0] & m[1] & m[2] & m[3]
    s["out"] = torch.empty((rows, V), device=DEV, dtype=DT[c["odt"]])
    return s


def prepare(case, seed):
    c = dict(case)
    s = _inputs(c, seed)
    s["case"] = c
    if own:     # what a serving program keeps from call to call: the descriptions of its cache and batch, a workspace
        import gguf_quant_weight_gb300 as g
        dts = {"f32": g.GGUF_DT_F32, "f16": g.GGUF_DT_F16, "bf16": g.GGUF_DT_BF16}
        s["stream"] = torch.cuda.current_stream().cuda_stream
        if c["op"] == "logits":
            s["rules"] = g.gguf_logit_rules(hist=s["hist"], hist_start=s["hist_start"], repeat=s["repeat"], frequency=s["frequency"],
                                            presence=s["presence"], bias_ids=s["bias_ids"], bias=s["bias"],
                                            bias_start=s["bias_start"], allow=s.get("allow"))
            s["dts"] = dts[c["dt"]], dts[c["odt"]]
            return s
        s["cache"] = g.gguf_kv_cache(s["k_cache"], s["v_cache"])
        s["batch"] = g.gguf_kv_batch(s["q_start"], s["kv_len"], s["pages"], s["tokens"], s["max_q"], s["max_kv"])
        if c["op"] == "append":
            s["rope"] = g.gguf_rope(s["freqs"], c["rot"], c["style"])
            s["xdt"] = dts[c["xdt"]]
        else:
            s["ws_bytes"] = g.gguf_paged_attn_workspace_size(s["batch"], s["cache"], c["heads"])
            s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- the plain forms

def _tokens(s):
    """Sequence, place among its new tokens, and position of every packed row."""
    start, kv_len = s["q_start"].to(torch.int64), s["kv_len"].to(torch.int64)
    t = torch.arange(s["tokens"], device=start.device)
    b = torch.searchsorted(start, t, right=True) - 1
    j = t - start[b]
    return b, j, kv_len[b] - (start[b + 1] - start[b]) + j


def _rotate(x, cos, sin, rot, style):
    """The first `rot` values of each head in pairs: neighbours (style 0) or halves (style 1)."""
    y = x.float().clone()
    if style == 0:
        a, b = x[..., 0:rot:2].float(), x[..., 1:rot:2].float()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :rot // 2].float(), x[..., rot // 2:rot].float()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_append(s, c):
    b, j, pos = _tokens(s)
    angle = pos.float()[:, None] * s["freqs"]
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    dt = s["k_cache"].dtype
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["rot"], c["style"]))
    page, slot = s["pages"][b, pos // c["page"]].to(torch.int64), pos % c["page"]
    s["k_cache"][page, :, slot] = _rotate(s["k"], cos, sin, c["rot"], c["style"]).to(dt)
    s["v_cache"][page, :, slot] = s["v"].to(dt)
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _plain_attn(s, c):
    H, KV, D, L, Q = c["heads"], c["kv_heads"], c["dim"], s["max_kv"], s["max_q"]
    G, B = H // KV, c["seqs"]
    b, j, _ = _tokens(s)
    kv_len = s["kv_len"].to(torch.int64)
    n = (s["q_start"][1:] - s["q_start"][:-1]).to(torch.int64)
    # every sequence's keys and values, padded to the longest; what is past its end counts as nothing
    t = torch.arange(L, device=kv_len.device)
    held = t < kv_len[:, None]
    page = s["pages"][:, t // c["page"]].clamp(min=0).to(torch.int64)
    slot = (t % c["page"]).expand(B, L)
    keys = torch.where(held[:, :, None, None], s["k_cache"][page, :, slot], 0).float().permute(0, 2, 3, 1)      # [B, KV, D, L]
    vals = torch.where(held[:, :, None, None], s["v_cache"][page, :, slot], 0).float().permute(0, 2, 1, 3)      # [B, KV, L, D]
    q = torch.zeros((B, Q, H, D), device=kv_len.device)
    q[b, j] = s["q"].float()
    q = q.view(B, Q, KV, G, D).permute(0, 2, 3, 1, 4).reshape(B, KV, G * Q, D)
    p = (kv_len - n)[:, None] + torch.arange(Q, device=kv_len.device)       # positions [B, Q]
    see = held[:, None, :].expand(B, Q, L)
    if c["causal"]:
        see = see & (t <= p[:, :, None])
    if c["window"]:
        see = see & (t > p[:, :, None] - c["window"])
    x = torch.matmul(q, keys).view(B, KV, G, Q, L)
    x *= D ** -0.5
    x.masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    safe = torch.where(top == -math.inf, 0.0, top)
    x.sub_(safe).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, KV, G * Q, L), vals).view(B, KV, G, Q, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (safe + torch.log(total))[..., 0]                                 # a row that sees nothing: log 0
    out = o.permute(0, 3, 1, 2, 4).reshape(B, Q, H, D)[b, j]
    return {"out": out.to(s["out"].dtype), "lse": lse.permute(0, 3, 1, 2).reshape(B, Q, H)[b, j]}


def _plain_logits(s, c):
    rows, V = c["rows"], c["vocab"]
    x = s["logits"].float()

    def row_of(start, n):
        return torch.searchsorted(start.to(torch.int64), torch.arange(n, device=x.device), right=True) - 1

    count = torch.zeros((rows * V,), device=x.device)
    hist = s["hist"].to(torch.int64)
    count.scatter_add_(0, row_of(s["hist_start"], hist.numel()) * V + hist, torch.ones(hist.shape, device=x.device))
    count = count.view(rows, V)
    r, f, p = (s[k][:, None] for k in ("repeat", "frequency", "presence"))
    y = torch.where(x > 0, x / r, x * r) - (count * f + p)
    y = torch.where(count > 0, y, x)
    if c["bias"]:
        ids = s["bias_ids"].to(torch.int64)
        y.view(-1).scatter_add_(0, row_of(s["bias_start"], ids.numel()) * V + ids, s["bias"])
    if c["grammar"]:
        v = torch.arange(V, device=x.device)
        ok = (s["allow"][:, v // 32] >> (v % 32).to(torch.int32)) & 1
        y = torch.where(ok == 1, y, -math.inf)
    return {"out": y.to(s["out"].dtype)}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"append": _plain_append, "attn": _plain_attn, "logits": _plain_logits}[c["op"]](s, c)
    import gguf_quant_weight_gb300 as g
    if c["op"] == "append":
        q, k, v = s["q"], s["k"], s["v"]
        g.gguf_kv_append(q, q.stride(0), k, k.stride(0), v, v.stride(0), s["xdt"], c["heads"], s["rope"], s["batch"], s["cache"],
                         s["q_out"], c["heads"] * c["dim"], s["stream"])
        return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
    if c["op"] == "attn":
        ld = c["heads"] * c["dim"]
        g.gguf_paged_attn(s["q"], ld, c["heads"], s["batch"], s["cache"], c["dim"] ** -0.5, c["causal"], c["window"], s["out"], ld,
                          s["lse"], s["ws"], s["ws_bytes"], s["stream"])
        return {"out": s["out"], "lse": s["lse"]}
    V = c["vocab"]
    g.gguf_logits_adjust(s["logits"], s["dts"][0], V, c["rows"], V, s["rules"], s["out"], s["dts"][1], V, s["stream"])
    return {"out": s["out"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    c = dict(case)
    s = _inputs(c, seed)
    if c["op"] == "logits":
        return _exact_logits(s, c)
    n, past = _lens(c)
    start = [sum(n[:i]) for i in range(len(n))]
    f64 = torch.float64
    if c["op"] == "append":
        out = {"q": torch.zeros(s["q_out"].shape, dtype=f64, device=DEV), "k": s["k_cache"].to(f64), "v": s["v_cache"].to(f64)}
        for i in range(c["seqs"]):
            rows = slice(start[i], start[i] + n[i])
            pos = torch.arange(past[i], past[i] + n[i], device=DEV)
            z = torch.polar(torch.ones((n[i], c["rot"] // 2), dtype=f64, device=DEV), pos.to(f64)[:, None] * s["freqs"].to(f64))

            def turned(x):
                x = x[rows].to(f64).clone()
                h = c["rot"] // 2
                head = x[..., :c["rot"]]
                pairs = head.unflatten(-1, (h, 2)) if c["style"] == 0 else head.unflatten(-1, (2, h)).transpose(-1, -2)
                w = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z[:, None])
                x[..., :c["rot"]] = w.flatten(-2) if c["style"] == 0 else w.transpose(-1, -2).flatten(-2)
                return x

            out["q"][rows] = turned(s["q"])
            page = s["pages"][i].to(torch.int64)[pos // c["page"]]
            out["k"][page, :, pos % c["page"]] = turned(s["k"])
            out["v"][page, :, pos % c["page"]] = s["v"][rows].to(f64)
        return out
    H, KV, D = c["heads"], c["kv_heads"], c["dim"]
    out = torch.zeros((s["tokens"], H, D), dtype=f64, device=DEV)
    lse = torch.full((s["tokens"], H), -math.inf, dtype=f64, device=DEV)
    for i in range(c["seqs"]):
        t = torch.arange(past[i] + n[i], device=DEV)
        page = s["pages"][i].to(torch.int64)[t // c["page"]]
        K, W = (x[page, :, t % c["page"]].to(f64) for x in (s["k_cache"], s["v_cache"]))
        for lo in range(0, n[i], 1024):
            hi = min(n[i], lo + 1024)
            pos = torch.arange(past[i] + lo, past[i] + hi, device=DEV)[:, None]
            hide = torch.zeros((hi - lo, len(t)), dtype=torch.bool, device=DEV)
            if c["causal"]:
                hide |= t > pos
            if c["window"]:
                hide |= t <= pos - c["window"]
            rows = slice(start[i] + lo, start[i] + hi)
            for h in range(H):
                a = s["q"][rows, h].to(f64) @ K[:, h * KV // H].T / math.sqrt(D)
                a[hide] = -math.inf
                lse[rows, h] = torch.logsumexp(a, -1)
                out[rows, h] = torch.nan_to_num(torch.softmax(a, -1), nan=0.0) @ W[:, h * KV // H]
    return {"out": out, "lse": lse}


def _exact_logits(s, c):
    x = s["logits"].to(torch.float64)
    start, first = s["hist_start"].tolist(), s["bias_start"].tolist()
    bits = torch.arange(32, device=DEV, dtype=torch.int32)
    for i in range(c["rows"]):
        ids, times = torch.unique(s["hist"][start[i]:start[i + 1]].to(torch.int64), return_counts=True)
        r, f, p = (float(s[k][i]) for k in ("repeat", "frequency", "presence"))
        y = x[i, ids]
        x[i, ids] = torch.where(y > 0, y / r, y * r) - f * times - p
        which = s["bias_ids"][first[i]:first[i + 1]].to(torch.int64)
        x[i].index_add_(0, which, s["bias"][first[i]:first[i + 1]].to(torch.float64))
        if c["grammar"]:
            ok = ((s["allow"][i][:, None] >> bits) & 1).flatten()[:c["vocab"]]
            x[i, ok == 0] = -math.inf
    return {"out": x}
