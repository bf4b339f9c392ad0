"""More operators of a decode step, as they are measured.

What a model with normed heads and experts needs between the products besides the cache's append, attention and the rules on
the logits:

  append  gguf_kv_append_norm  norms each head of the new queries and keys, rotates them to their positions and appends keys and values
  router  gguf_moe_router      scores the experts for each token and picks the best, with their weights
  ffn     gguf_moe_ffn         a few tokens through their experts' gated feed-forward, on the GGUF blocks, weighted and added up
  sample  gguf_sample          draws each row's next token from given random numbers, after temperature, top-k, top-p and min-p

`own` chooses between the library's calls (True) and their plain form in elementary torch operations (False).
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# type id, values and bytes of a block, where its f16 scale (and min) lie, and for random codes: 1 / the weights' spread at
# a scale of one, the min that centres them
FORMATS = {
    "Q4_0": (2, 32, 18, 0, None, 4.6, 0.0), "Q4_1": (3, 32, 20, 0, 2, 4.6, -7.5), "Q5_0": (6, 32, 22, 0, None, 9.2, 0.0),
    "Q5_1": (7, 32, 24, 0, 2, 9.2, -15.5), "Q8_0": (8, 32, 34, 0, None, 74.0, 0.0), "Q2_K": (10, 256, 84, 80, 82, 13.0, 1.5),
    "Q3_K": (11, 256, 110, 108, None, 43.0, 0.0), "Q4_K": (12, 256, 144, 0, 2, 300.0, 7.5), "Q5_K": (13, 256, 176, 0, 2, 600.0, 15.5),
    "Q6_K": (14, 256, 210, 208, None, 1370.0, 0.0)}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one user's next token: normed heads, 4 key heads for 32 query heads
        dict(name="append_norm_token", op="append", xdt="bf16", dt="bf16", seqs=1, q=1, q_hi=1, past=1000, past_hi=1000, heads=32,
             kv_heads=4, dim=128, rot=128, style=1, page=16, layout="hnd", fused=True, lens=21),
        # a serving batch of single tokens and chunks; heads of an odd size, rotated in part and in neighbours
        dict(name="append_norm_mixed", op="append", xdt="f16", dt="f16", seqs=48, q=1, q_hi=90, past=0, past_hi=700, heads=24,
             kv_heads=8, dim=80, rot=40, style=0, page=32, layout="nhd", fused=False, lens=22),
        # whole prompts, f32 rows of a fused projection into a bf16 cache
        dict(name="append_norm_prompts", op="append", xdt="f32", dt="bf16", seqs=5, q=900, q_hi=2500, past=0, past_hi=64, heads=32,
             kv_heads=4, dim=128, rot=128, style=1, page=64, layout="hnd", fused=True, lens=23),
        # one token's eight of 128 experts
        dict(name="router_token", op="router", xdt="bf16", wdt="f32", T=1, K=2048, experts=128, top_k=8, score="softmax", bias=False,
             renorm=True, scale=1.0),
        # chunks of prompts: sigmoid scores, a balancing bias that chooses and does not weigh
        dict(name="router_chunk", op="router", xdt="bf16", wdt="f32", T=509, K=2048, experts=128, top_k=8, score="sigmoid", bias=True,
             renorm=True, scale=2.5),
        # one token through its experts, the mix of types of a medium file
        dict(name="ffn_token", op="ffn", types="Q4_K/Q4_K/Q6_K", xdt="bf16", ydt="bf16", T=1, K=2048, F=768, experts=128,
             top_k=8, act="silu", residual=True, route=31),
        # seven tokens of a draft through small experts of the 32-value types, f32 all along
        dict(name="ffn_small_blocks", op="ffn", types="Q8_0/Q5_1/Q4_0", xdt="f32", ydt="f32", T=7, K=2080, F=1440, experts=60,
             top_k=4, act="gelu", residual=False, route=32),
        # a decode batch: nearly every expert is some token's
        dict(name="ffn_batch", op="ffn", types="Q4_K/Q4_K/Q4_K", xdt="bf16", ydt="bf16", T=64, K=2048, F=768, experts=128,
             top_k=8, act="silu", residual=True, route=33),
        # three tokens through few wide experts
        dict(name="ffn_wide", op="ffn", types="Q5_K/Q5_K/Q6_K", xdt="f16", ydt="f16", T=3, K=4096, F=14336, experts=8, top_k=2,
             act="silu", residual=True, route=34),
        # one user's next token, every filter on
        dict(name="sample_token", op="sample", dt="f32", rows=1, vocab=128259, temp=0.8, temp_hi=0.8, top_k=40, top_k_hi=40,
             top_p=0.95, top_p_hi=0.95, min_p=0.05, min_p_hi=0.05, grammar=False),
        # a batch in which every row has its own settings, greedy rows and grammars among them
        dict(name="sample_mixed", op="sample", dt="bf16", rows=37, vocab=32003, temp=0.0, temp_hi=1.5, top_k=0, top_k_hi=200,
             top_p=0.5, top_p_hi=1.05, min_p=-0.02, min_p_hi=0.1, grammar=True),
        # a large batch that keeps a share of the whole distribution
        dict(name="sample_large", op="sample", dt="f32", rows=256, vocab=131072, temp=0.6, temp_hi=1.2, top_k=0, top_k_hi=0,
             top_p=0.8, top_p_hi=1.05, min_p=0.0, min_p_hi=0.0, grammar=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    while True:
        c = _draw(rng)
        if c["op"] == "append":
            n, past = _lens(c)
            if sum(n) * (c["heads"] + 2 * c["kv_heads"]) * c["dim"] <= 8000 * 40 * 128 and sum(n) + sum(past) <= 60000:
                return c
        elif c["op"] == "router":
            if c["T"] * c["K"] * c["experts"] <= 509 * 2048 * 128:
                return c
        elif c["op"] == "ffn":
            if c["T"] * c["top_k"] <= 512 and c["T"] * c["top_k"] * c["K"] * c["F"] <= 512 * 768 * 2048 and \
                    c["experts"] * c["K"] * c["F"] <= 8 * 4096 * 14336:
                return c
        elif c["rows"] * c["vocab"] <= 256 * 131072:
            return c


def _draw(rng):
    op = rng.choice(("append", "router", "ffn", "ffn", "sample", "sample"))
    if op == "sample":
        k = rng.choice((0, 0, 1, _log(rng, 2, 500), _log(rng, 100, 5000)))
        c = dict(op=op, dt=rng.choice(("f32", "f16", "bf16")), rows=_log(rng, 1, 256), vocab=_log(rng, 1000, 160000))
        c["temp"], c["temp_hi"] = rng.choice(((1.0, 1.0), (0.0, 1.2), (0.3, 2.0)))
        c["top_k"], c["top_k_hi"] = rng.choice(((0, 0), (k, k), (0, k)))
        c["top_p"], c["top_p_hi"] = rng.choice(((1.0, 1.0), (0.9, 0.9), (0.3, 1.05)))
        c["min_p"], c["min_p_hi"] = rng.choice(((0.0, 0.0), (0.05, 0.05), (-0.1, 0.2)))
        return dict(c, grammar=rng.random() < 0.3)
    if op == "router":
        e = rng.choice((8, 16, 60, 64, 128, 160, 256, _log(rng, 2, 384)))
        return dict(op=op, xdt=rng.choice(("f32", "f16", "bf16")), wdt=rng.choice(("f32", "f32", "f16", "bf16")), T=_log(rng, 1, 509),
                    K=32 * _log(rng, 8, 224), experts=e, top_k=min(e, rng.choice((1, 2, 4, 6, 8, 10))),
                    score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.4, renorm=rng.random() < 0.7,
                    scale=rng.choice((1.0, 2.5)))
    if op == "ffn":
        big = rng.random() < 0.6
        kinds = [t for t, f in FORMATS.items() if f[1] == (256 if big else 32)]
        e = rng.choice((4, 8, 32, 60, 64, 128))
        return dict(op=op, types="/".join(rng.choice(kinds) for _ in range(3)), xdt=rng.choice(("f32", "f16", "bf16", "bf16")),
                    ydt=rng.choice(("f32", "f16", "bf16", "bf16")), T=_log(rng, 1, 64),
                    K=256 * _log(rng, 2, 20) if big else 32 * _log(rng, 16, 160),
                    F=256 * _log(rng, 2, 40) if big else 32 * _log(rng, 16, 300), experts=e, top_k=min(e, rng.choice((1, 2, 4, 6, 8))),
                    act=rng.choice(("silu", "silu", "gelu")), residual=rng.random() < 0.6, route=rng.randrange(1 << 20))
    kv_heads = rng.choice((1, 2, 4, 8, 16))
    dim = rng.choice((64, 80, 96, 128, 128, 128))
    form = rng.choice(("token", "chunk", "prompt"))
    q_hi = 1 if form == "token" else _log(rng, 2, 500) if form == "chunk" else _log(rng, 300, 8000)
    past_hi = _log(rng, 1, 30000 if form == "token" else 5000) if rng.random() < 0.8 else 0
    return dict(op=op, xdt=rng.choice(("f32", "f16", "bf16")), dt=rng.choice(("f16", "bf16")),
                seqs=_log(rng, 1, 96) if form == "token" else _log(rng, 1, 24) if form == "chunk" else _log(rng, 1, 4),
                q=rng.choice((1, max(1, q_hi // 2), q_hi)), q_hi=q_hi, past=rng.choice((0, past_hi // 2, past_hi)), past_hi=past_hi,
                heads=kv_heads * rng.choice((1, 2, 3, 4, 5, 7, 8)), kv_heads=kv_heads, dim=dim, rot=rng.choice((dim, dim, dim // 2)),
                style=rng.randrange(2), page=rng.choice((16, 32, 64, 128)), layout=rng.choice(("hnd", "nhd")), fused=rng.random() < 0.5,
                lens=rng.randrange(1 << 20))


def _lens(c):
    """New tokens and earlier keys of each sequence: the case's own, the same for every seed."""
    r = random.Random(c["lens"])
    n = [_log(r, c["q"], c["q_hi"]) for _ in range(c["seqs"])]
    past = [min(c["past_hi"], max(c["past"], _log(r, c["past"] + 1, c["past_hi"] + 1) - 1)) for _ in range(c["seqs"])]
    return n, past


def _route(c):
    """Each token's experts before they are renamed by the seed: some are more popular than others, as routers have it."""
    r = np.random.default_rng(c["route"])
    popular = 1.0 / (np.arange(c["experts"]) + 4.0)
    score = np.log(popular)[None] + r.gumbel(size=(c["T"], c["experts"]))
    return np.argsort(-score, axis=1)[:, :c["top_k"]].astype(np.int64)


def _row_bytes(t, k):
    return k // FORMATS[t][1] * FORMATS[t][2]


def work(case):
    c = case
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if c["op"] == "append":
        tokens = sum(_lens(c)[0])
        H, KV, D = c["heads"], c["kv_heads"], c["dim"]
        return {"bytes": tokens * (H + 2 * KV) * D * (size[c["xdt"]] + 2), "flops": tokens * (H + KV) * (3 * c["rot"] + 4 * D)}
    if c["op"] == "router":
        b = c["T"] * c["K"] * size[c["xdt"]] + c["experts"] * c["K"] * size[c["wdt"]] + 8 * c["T"] * c["top_k"]
        return {"bytes": b, "flops": 2 * c["T"] * c["K"] * c["experts"]}
    if c["op"] == "ffn":
        touched = len(np.unique(_route(c)))
        g, u, d = c["types"].split("/")
        per = c["F"] * (_row_bytes(g, c["K"]) + _row_bytes(u, c["K"])) + c["K"] * _row_bytes(d, c["F"])
        rows = c["T"] * c["top_k"]
        b = touched * per + c["T"] * c["K"] * (size[c["xdt"]] + size[c["ydt"]] * (2 if c["residual"] else 1)) + 8 * rows
        return {"bytes": b, "flops": 6 * rows * c["K"] * c["F"]}
    n = c["rows"] * c["vocab"]
    return {"bytes": n * size[c["dt"]] + 28 * c["rows"], "flops": 8 * n}


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
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dt)
    return x if c["layout"] == "hnd" else x.transpose(1, 2)


def _blocks(t, experts, n, k, g):
    """Random weights of a type as a file holds them: [experts, n, bytes of a row]."""
    _, values, size, d_at, m_at, spread, centre = FORMATS[t]
    b = torch.randint(0, 256, (experts, n, k // values, size), generator=g, device=DEV, dtype=torch.uint8)
    d = (0.5 + torch.rand(b.shape[:-1], generator=g, device=DEV)) / (spread * math.sqrt(k))
    b[..., d_at:d_at + 2] = d.to(torch.float16)[..., None].view(torch.uint8)
    if m_at is not None:
        b[..., m_at:m_at + 2] = (d * centre).to(torch.float16)[..., None].view(torch.uint8)
    return b.view(experts, n, -1)


def _between(c, what, rows, g):
    lo, hi = c[what], c[what + "_hi"]
    return lo + (hi - lo) * torch.rand((rows,), generator=g, device=DEV)


def _inputs(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    if c["op"] == "append":
        s = _batch(c, g)
        dt, x, D, H, KV, T = DT[c["dt"]], DT[c["xdt"]], c["dim"], c["heads"], c["kv_heads"], s["tokens"]
        s["k_cache"], s["v_cache"] = _cache(c, s["n_pages"], g, dt), _cache(c, s["n_pages"], g, dt)
        if c["fused"]:      # the rows of one fused projection
            qkv = (2.0 * torch.randn((T, (H + 2 * KV) * D), generator=g, device=DEV)).to(x)
            s["q"], s["k"], s["v"] = (t.view(T, -1, D) for t in qkv.split((H * D, KV * D, KV * D), dim=1))
        else:
            s["q"], s["k"], s["v"] = ((2.0 * torch.randn((T, h, D), generator=g, device=DEV)).to(x) for h in (H, KV, KV))
        i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
        s["freqs"] = (10000.0 ** (-2.0 * i / c["rot"])).to(torch.float32)
        s["q_norm"], s["k_norm"] = (1.0 + 0.3 * torch.randn((D,), generator=g, device=DEV) for _ in range(2))
        s["eps"] = 1e-6
        s["q_out"] = torch.zeros((T, H, D), device=DEV, dtype=dt)
        return s
    if c["op"] == "router":
        T, K, E = c["T"], c["K"], c["experts"]
        s = dict(x=torch.randn((T, K), generator=g, device=DEV).to(DT[c["xdt"]]),
                 w=(torch.randn((E, K), generator=g, device=DEV) / math.sqrt(K)).to(DT[c["wdt"]]))
        s["bias"] = 0.2 * torch.randn((E,), generator=g, device=DEV) if c["bias"] else None
        s["ids"] = torch.empty((T, c["top_k"]), dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty((T, c["top_k"]), dtype=torch.float32, device=DEV)
        return s
    if c["op"] == "ffn":
        T, K, F, E, kinds = c["T"], c["K"], c["F"], c["experts"], c["types"].split("/")
        names = torch.randperm(E, generator=g, device=DEV)
        s = dict(ids=names[torch.from_numpy(_route(c)).to(DEV)].to(torch.int32).contiguous())
        w = torch.softmax(torch.randn((T, c["top_k"]), generator=g, device=DEV), -1)
        s["weights"] = w.contiguous()
        s["x"] = torch.randn((T, K), generator=g, device=DEV).to(DT[c["xdt"]])
        s["residual"] = torch.randn((T, K), generator=g, device=DEV).to(DT[c["ydt"]]) if c["residual"] else None
        s["gate"], s["up"] = (_blocks(t, E, F, K, g) for t in kinds[:2])
        s["down"] = _blocks(kinds[2], E, K, F, g)
        s["y"] = torch.empty((T, K), dtype=DT[c["ydt"]], device=DEV)
        return s
    rows, V = c["rows"], c["vocab"]
    x = 3.0 * torch.randn((rows, V), generator=g, device=DEV)
    if c["grammar"]:        # in half of the rows a grammar allows one token in sixteen
        hide = (torch.rand((rows, V), generator=g, device=DEV) > 1 / 16) & (torch.rand((rows, 1), generator=g, device=DEV) < 0.5)
        x.masked_fill_(hide, -math.inf)
    temp = _between(c, "temp", rows, g)
    s = dict(logits=x.to(DT[c["dt"]]), temp=torch.where(temp < 0.1, 0.0, temp), u=torch.rand((rows,), generator=g, device=DEV))
    s["top_k"] = _between(c, "top_k", rows, g).round().to(torch.int32)
    s["top_p"], s["min_p"] = _between(c, "top_p", rows, g), _between(c, "min_p", rows, g)
    s["token"] = torch.empty((rows,), dtype=torch.int32, device=DEV)
    s["logprob"] = torch.empty((rows,), dtype=torch.float32, device=DEV)
    return s


def prepare(case, seed):
    c = dict(case)
    s = _inputs(c, seed)
    s["case"] = c
    if own:     # what a serving program keeps from call to call: the descriptions of its cache, weights and rules, a workspace
        import gguf_quant_weight_gb300 as g
        dts = {"f32": g.GGUF_DT_F32, "f16": g.GGUF_DT_F16, "bf16": g.GGUF_DT_BF16}
        s["stream"] = torch.cuda.current_stream().cuda_stream
        s["dts"] = {k: dts[c[k]] for k in ("dt", "xdt", "ydt", "wdt") if k in c}
        if c["op"] == "append":
            s["cache"] = g.gguf_kv_cache(s["k_cache"], s["v_cache"])
            s["batch"] = g.gguf_kv_batch(s["q_start"], s["kv_len"], s["pages"], s["tokens"], s["max_q"], s["max_kv"])
            s["rope"] = g.gguf_rope(s["freqs"], c["rot"], c["style"])
            s["norm"] = g.gguf_head_norm(s["q_norm"], s["k_norm"], s["eps"])
        elif c["op"] == "router":
            score = {"softmax": g.GGUF_SCORE_SOFTMAX, "sigmoid": g.GGUF_SCORE_SIGMOID}[c["score"]]
            s["router"] = g.gguf_router(s["w"], c["top_k"], score, s["bias"], c["renorm"], c["scale"])
        elif c["op"] == "ffn":
            act = {"silu": g.GGUF_ACT_SILU, "gelu": g.GGUF_ACT_GELU}[c["act"]]
            kinds = (FORMATS[t][0] for t in c["types"].split("/"))
            s["experts"] = g.gguf_moe_weights(s["gate"], s["up"], s["down"], *kinds, c["K"], c["F"], c["experts"], act)
            s["ws_bytes"] = g.gguf_moe_ffn_workspace_size(c["F"], c["T"], c["top_k"])
            s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)
        else:
            s["sampler"] = g.gguf_sampler(s["temp"], s["top_k"], s["top_p"], s["min_p"])
    return s


# ---------------------------------------------------------------- the plain forms

def _rotate(x, cos, sin, rot, style):
    """The first `rot` values of each head in pairs: neighbours (style 0) or halves (style 1)."""
    y = x.clone()
    if style == 0:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_append(s, c):
    start, kv_len = s["q_start"].to(torch.int64), s["kv_len"].to(torch.int64)
    t = torch.arange(s["tokens"], device=start.device)
    b = torch.searchsorted(start, t, right=True) - 1
    pos = kv_len[b] - start[b + 1] + t
    angle = pos.double()[:, None] * s["freqs"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def normed(x, w):
        x = x.float()
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w

    s["q_out"].copy_(_rotate(normed(s["q"], s["q_norm"]), cos, sin, c["rot"], c["style"]))
    dt = s["k_cache"].dtype
    page, slot = s["pages"][b, pos // c["page"]].to(torch.int64), pos % c["page"]
    s["k_cache"][page, :, slot] = _rotate(normed(s["k"], s["k_norm"]), cos, sin, c["rot"], c["style"]).to(dt)
    s["v_cache"][page, :, slot] = s["v"].to(dt)
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _plain_router(s, c):
    z = torch.matmul(s["x"].double(), s["w"].double().T)        # 64 bits: experts whose scores are next to each other keep their order
    p = torch.softmax(z, -1) if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-z))
    rank = p if s["bias"] is None else p + s["bias"].double()
    ids = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    s["ids"].copy_(ids)
    s["weights"].copy_(w * c["scale"])
    return {"ids": s["ids"], "weights": s["weights"]}


def _f16(b, at):
    return b[..., at:at + 2].contiguous().view(torch.float16).float()


def _six_bits(s):
    """The eight scales and eight mins of six bits in the twelve bytes of Q4_K and Q5_K."""
    a, b, c = s[..., 0:4], s[..., 4:8], s[..., 8:12]
    return (torch.cat((a & 63, (c & 15) | (a >> 6 << 4)), -1), torch.cat((b & 63, (c >> 4) | (b >> 6 << 4)), -1))


def _weights(b, t):
    """Blocks [..., blocks, bytes] as f32 values [..., blocks * values]."""
    out = b.shape[:-2] + (-1,)
    d = _f16(b, FORMATS[t][3])
    m = _f16(b, FORMATS[t][4]) if FORMATS[t][4] is not None else None
    lead = b.shape[:-1]
    if t == "Q8_0":
        return (b[..., 2:].contiguous().view(torch.int8) * d).view(out)
    if t in ("Q4_0", "Q4_1", "Q5_0", "Q5_1"):
        qs = b[..., -16:]
        q = torch.cat((qs & 15, qs >> 4), -1)
        if t[1] == "5":
            at = 2 if t == "Q5_0" else 4
            bit = torch.arange(8, dtype=torch.uint8, device=b.device)
            q = q | (((b[..., at:at + 4, None] >> bit) & 1) << 4).view(lead + (32,))
        return ((q * d + m) if m is not None else (q.float() - (8 if t == "Q4_0" else 16)) * d).view(out)
    two = torch.arange(0, 8, 2, dtype=torch.uint8, device=b.device)
    if t in ("Q4_K", "Q5_K"):
        sc, mn = _six_bits(b[..., 4:16])
        qs = b[..., -128:].view(lead + (4, 32))
        q = torch.stack((qs & 15, qs >> 4), -2).view(lead + (8, 32))
        if t == "Q5_K":
            bit = torch.arange(8, dtype=torch.uint8, device=b.device)[:, None]
            q = q | (((b[..., None, 16:48] >> bit) & 1) << 4)
        return ((d * sc)[..., None] * q - (m * mn)[..., None]).view(out)
    if t == "Q6_K":
        ql, qh = b[..., :128].view(lead + (2, 64)), b[..., 128:192].view(lead + (2, 1, 32))
        low = torch.stack((ql & 15, ql >> 4), -2).view(lead + (2, 4, 32))
        q = (low | (((qh >> two[:, None]) & 3) << 4)).view(lead + (16, 16)).float() - 32.0
        return ((b[..., 192:208].contiguous().view(torch.int8) * d)[..., None] * q).view(out)
    qs = b[..., 16:80] if t == "Q2_K" else b[..., 32:96]
    q = ((qs.view(lead + (2, 1, 32)) >> two[:, None]) & 3).view(lead + (16, 16))
    if t == "Q2_K":
        s = b[..., :16]
        return ((d * (s & 15))[..., None] * q - (m * (s >> 4))[..., None]).view(out)
    bit = torch.arange(8, dtype=torch.uint8, device=b.device)[:, None]
    high = ((b[..., None, :32] >> bit) & 1).view(lead + (16, 16))
    low, top = b[..., 96:104], b[..., None, 104:108]
    six = torch.cat((low & 15, low >> 4), -1) | (((top >> two[:, None]) & 3) << 4).view(lead + (16,))
    return ((d * (six.float() - 32.0))[..., None] * (q.float() - 4.0 * (1 - high.float()))).view(out)


def _plain_ffn(s, c):
    T, k, (g, u, d) = c["T"], c["top_k"], c["types"].split("/")
    e = s["ids"].reshape(-1).to(torch.int64)
    of = lambda w, t: _weights(w.view(w.shape[0], w.shape[1], -1, FORMATS[t][2])[e], t)      # noqa: E731
    x = s["x"].float().repeat_interleave(k, 0)[:, :, None]
    a, b = torch.bmm(of(s["gate"], g), x), torch.bmm(of(s["up"], u), x)
    if c["act"] == "silu":
        h = a / (1.0 + torch.exp(-a)) * b
    else:
        h = 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3))) * b
    y = torch.bmm(of(s["down"], d), h).view(T, k, -1)
    y = (y * s["weights"][:, :, None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    s["y"].copy_(y)
    return {"y": s["y"]}


def _plain_sample(s, c):
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    temp = s["temp"].double()[:, None]
    w = torch.where(temp > 0, torch.exp((x - top) / temp.clamp(min=1e-30)), (x == top).double())
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    sorted_w = w.gather(1, order)
    rank = torch.arange(c["vocab"], device=x.device)
    k = s["top_k"][:, None]
    k = torch.where(k > 0, k, c["vocab"])
    k = torch.where(temp > 0, k, 1)
    sorted_w = torch.where(rank < k, sorted_w, 0.0)
    upto = sorted_w.cumsum(-1)
    p = s["top_p"].double()[:, None]
    in_p = (upto - sorted_w < p.clamp(min=0.0) * upto[:, -1:]) | (p >= 1) | (rank == 0)
    in_m = sorted_w >= s["min_p"].double()[:, None].clamp(max=1.0)
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(in_p & in_m, sorted_w, 0.0))
    upto = kept.cumsum(-1)
    total = upto[:, -1:]
    token = (upto <= s["u"].double()[:, None] * total).sum(-1, keepdim=True)
    s["token"].copy_(token[:, 0])
    s["logprob"].copy_(torch.log(kept.gather(1, token) / total)[:, 0])
    return {"token": s["token"], "logprob": s["logprob"]}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"append": _plain_append, "router": _plain_router, "ffn": _plain_ffn, "sample": _plain_sample}[c["op"]](s, c)
    import gguf_quant_weight_gb300 as g
    if c["op"] == "append":
        q, k, v = s["q"], s["k"], s["v"]
        g.gguf_kv_append_norm(q, q.stride(0), k, k.stride(0), v, v.stride(0), s["dts"]["xdt"], c["heads"], s["norm"], s["rope"],
                              s["batch"], s["cache"], s["q_out"], c["heads"] * c["dim"], s["stream"])
        return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
    if c["op"] == "router":
        g.gguf_moe_router(s["x"], s["dts"]["xdt"], c["T"], c["K"], s["router"], s["ids"], s["weights"], s["stream"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if c["op"] == "ffn":
        g.gguf_moe_ffn(s["experts"], s["x"], s["dts"]["xdt"], c["T"], s["ids"], s["weights"], c["top_k"], s["residual"], s["y"],
                       s["dts"]["ydt"], s["ws"], s["ws_bytes"], s["stream"])
        return {"y": s["y"]}
    g.gguf_sample(s["logits"], s["dts"]["dt"], c["vocab"], c["rows"], c["vocab"], s["sampler"], s["u"], s["token"], s["logprob"],
                  s["stream"])
    return {"token": s["token"], "logprob": s["logprob"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_append(s, c):
    n, past = _lens(c)
    f64 = torch.float64
    out = {"q": torch.zeros(s["q_out"].shape, dtype=f64, device=DEV), "k": s["k_cache"].to(f64), "v": s["v_cache"].to(f64)}
    at = 0
    for i in range(c["seqs"]):
        rows = slice(at, at + n[i])
        at += n[i]
        pos = torch.arange(past[i], past[i] + n[i], device=DEV)
        z = torch.polar(torch.ones((n[i], c["rot"] // 2), dtype=f64, device=DEV), pos.to(f64)[:, None] * s["freqs"].to(f64))

        def turned(x, w):
            x = x[rows].to(f64)
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["dim"] + s["eps"]) * w.to(f64)
            h = c["rot"] // 2
            head = x[..., :c["rot"]]
            pairs = head.unflatten(-1, (h, 2)) if c["style"] == 0 else head.unflatten(-1, (2, h)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z[:, None])
            x[..., :c["rot"]] = y.flatten(-2) if c["style"] == 0 else y.transpose(-1, -2).flatten(-2)
            return x

        out["q"][rows] = turned(s["q"], s["q_norm"])
        page = s["pages"][i].to(torch.int64)[pos // c["page"]]
        out["k"][page, :, pos % c["page"]] = turned(s["k"], s["k_norm"])
        out["v"][page, :, pos % c["page"]] = s["v"][rows].to(f64)
    return out


def _exact_router(s, c):
    x, w = s["x"].cpu().double().numpy(), s["w"].cpu().double().numpy()
    z = x @ w.T
    if c["score"] == "softmax":
        p = np.exp(z - z.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
    else:
        p = 1.0 / (1.0 + np.exp(-z))
    rank = p + (s["bias"].cpu().double().numpy() if c["bias"] else 0.0)
    ids = np.argsort(-rank, axis=1, kind="stable")[:, :c["top_k"]]
    v = np.take_along_axis(p, ids, 1)
    if c["renorm"]:
        v = v / v.sum(-1, keepdims=True)
    return {"ids": ids.astype(np.int32), "weights": v * c["scale"]}


# Of each type, element e of a block as pieces of its code: (byte, shift, bits, place); then its scale and min by element.
def _pieces(t):
    e = np.arange(FORMATS[t][1])
    half, in_half = e // 128, e % 128
    if t == "Q8_0":
        return [(2 + e, 0 * e, 8, 0)]
    if t in ("Q4_0", "Q4_1", "Q5_0", "Q5_1"):
        first = FORMATS[t][2] - 16
        low = [(first + e % 16, 4 * (e // 16), 4, 0)]
        return low + ([(first - 4 + e // 8, e % 8, 1, 4)] if t[1] == "5" else [])
    if t in ("Q4_K", "Q5_K"):
        low = [((16 if t == "Q4_K" else 48) + 32 * (e // 64) + e % 32, 4 * (e // 32 % 2), 4, 0)]
        return low + ([(16 + e % 32, e // 32, 1, 4)] if t == "Q5_K" else [])
    if t == "Q6_K":
        return [(64 * half + in_half % 64, 4 * (in_half // 64), 4, 0), (128 + 32 * half + e % 32, 2 * (in_half // 32), 2, 4)]
    low = [((16 if t == "Q2_K" else 32) + 32 * half + e % 32, 2 * (in_half // 32), 2, 0)]
    return low + ([(e % 32, e // 32, 1, 2)] if t == "Q3_K" else [])


def _exact_weights(b, t):
    """Blocks [..., blocks, bytes] in 64 bits, element by element."""
    at = lambda i: b[..., torch.as_tensor(i, device=b.device)].to(torch.int64)      # noqa: E731
    f = lambda i: b[..., i:i + 2].contiguous().view(torch.float16).double()         # noqa: E731
    q = 0
    for byte, shift, bits, place in _pieces(t):
        q = q + (((at(byte) >> torch.as_tensor(shift, device=b.device)) & ((1 << bits) - 1)) << place)
    e = np.arange(FORMATS[t][1])
    scale, less = f(FORMATS[t][3]), 0.0
    if t == "Q8_0":
        q = (q + 128) % 256 - 128
    elif t in ("Q4_0", "Q5_0"):
        q = q - (8 if t == "Q4_0" else 16)
    elif t in ("Q4_1", "Q5_1"):
        less = -f(2)
    elif t in ("Q4_K", "Q5_K"):
        j = e // 32
        r, far = j % 4, torch.as_tensor(j >= 4, device=b.device)
        sc = torch.where(far, at(12 + r) % 16 + 16 * (at(4 + r) // 64), at(4 + r) % 64)
        mn = torch.where(far, at(12 + r) // 16 + 16 * (at(8 + r) // 64), at(8 + r) % 64)
        scale, less = scale * sc, f(2) * mn
    elif t == "Q6_K":
        scale, q = scale * ((at(192 + e // 16) + 128) % 256 - 128), q - 32
    elif t == "Q2_K":
        scale, less = scale * (at(e // 16) % 16), f(82) * (at(e // 16) // 16)
    else:
        j = e // 16
        six = (at(96 + j % 8) >> torch.as_tensor(4 * (j // 8), device=b.device)) % 16
        six = six + 16 * ((at(104 + j % 4) >> torch.as_tensor(2 * (j // 4), device=b.device)) % 4)
        scale, q = scale * (six - 32), q - 4
    return (scale * q - less).flatten(-2)


def _exact_ffn(s, c):
    y = torch.zeros((c["T"], c["K"]), dtype=torch.float64, device=DEV)
    if s["residual"] is not None:
        y += s["residual"].double()
    ids, w, kinds = s["ids"].to(torch.int64), s["weights"].double(), c["types"].split("/")
    for e in torch.unique(ids).tolist():
        of = lambda name, t: _exact_weights(s[name][e].unflatten(-1, (-1, FORMATS[t][2])), t)      # noqa: E731
        rows, slots = torch.nonzero(ids == e, as_tuple=True)
        x = s["x"][rows].double()
        a, b = x @ of("gate", kinds[0]).T, x @ of("up", kinds[1]).T
        if c["act"] == "silu":
            a = a * torch.sigmoid(a)
        else:
            a = torch.nn.functional.gelu(a, approximate="tanh")
        y.index_add_(0, rows, w[rows, slots][:, None] * ((a * b) @ of("down", kinds[2]).T))
    return {"y": y}


def _exact_sample(s, c):
    x = s["logits"].cpu().double().numpy()
    get = lambda k: s[k].cpu().double().numpy()      # noqa: E731
    temp, top_k, top_p, min_p, u = (get(k) for k in ("temp", "top_k", "top_p", "min_p", "u"))
    token, logprob = np.zeros(c["rows"], np.int32), np.zeros(c["rows"])
    for r in range(c["rows"]):
        if temp[r] == 0:
            token[r] = int(np.argmax(x[r]))
            continue
        order = np.argsort(-x[r], kind="stable")
        if top_k[r] > 0:
            order = order[:int(top_k[r])]
        w = np.exp((x[r][order] - x[r][order[0]]) / temp[r])
        n = len(order)
        if top_p[r] < 1:
            n = 1 + int(np.searchsorted(np.cumsum(w), top_p[r] * w.sum()))
        if min_p[r] > 0:
            n = min(n, int((w >= min(1.0, min_p[r])).sum()))
        kept = np.sort(order[:n])
        w = np.exp((x[r][kept] - x[r][order[0]]) / temp[r])
        upto = np.cumsum(w)
        at = min(len(kept) - 1, int(np.searchsorted(upto, u[r] * upto[-1], side="right")))
        token[r], logprob[r] = kept[at], np.log(w[at] / upto[-1])
    return {"token": token, "logprob": logprob}


def exact(case, seed):
    c = dict(case)
    return {"append": _exact_append, "router": _exact_router, "ffn": _exact_ffn, "sample": _exact_sample}[c["op"]](_inputs(c, seed), c)
