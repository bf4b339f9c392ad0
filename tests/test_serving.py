"""The serving operators on the GPU (cache append, paged attention, rules on
logits) against the 64-bit definitions in oracle/serving_oracle.py, at the
sizes and masks where they can go wrong.

Tolerances.  A 16-bit output must be the type's rounding of a value close to
the reference (gpu_util._rounding_interval); how close:
  * append: the turn of a pair is two products and a sum in f32, and cos and
    sin are within 2 units of 2**-23 of theirs: 8 * 2**-24 * (|a| + |b|) covers
    them; values that are only converted are exact.
  * attention: the weights are rounded to the cache's type, which moves a row
    by at most u * max |V| (u = 2**-8 for bf16, 2**-11 for f16), and a score's
    f32 error e moves it by at most 2 e max |V|, where e is at most
    2**-23 * D/4 * scale * sum |q K| (a sum of D products in f32, in any
    order of partial sums of four) plus 2**-20 for the exponential and the
    sums.  lse is off by at most e + 2**-20.
  * logits: three f32 operations and a sum for each bias, each half a unit of
    what it holds: (4 + biases) * 2**-23 * (|x| max + penalties + biases).
"""
import math

import numpy as np
import pytest
import torch

import gguf_quant_weight_gb300 as g
from oracle import serving_oracle as S
from tests import gpu_util as U

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    U.require_gpu()


def near(got, ref, dt, bound, what=""):
    """Every element of got rounds from a value within `bound` (an array) of ref."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bound = np.broadcast_to(bound, ref.shape)
    assert got.shape == ref.shape
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{what}: infinities differ"
    assert np.all(np.isfinite(got[~inf])), f"{what}: not finite"
    got, ref, bound = got[~inf], ref[~inf], bound[~inf]
    if not got.size:
        return
    if dt == "f32":
        off = np.abs(got - ref) - 2.0 ** -24 * np.abs(ref)
    else:
        lo, hi = U._rounding_interval(got, dt)
        off = np.maximum(lo - ref, ref - hi)
    worst = int(np.argmax(off - bound))
    assert np.all(off <= bound), f"{what}: off by {off[worst]:.3e}, bound {bound[worst]:.3e}"


# ------------------------------------------------------------------ batches

class Case:
    """A ragged batch with its cache: sequences of (new tokens, keys)."""

    def __init__(self, seqs, kv_heads, dim, dt, page=16, layout="hnd", extra_rows=0, seed=0, wide=None, first_page=None):
        rs = np.random.default_rng(seed)
        self.rs, self.dt, self.dim, self.kv_heads, self.page = rs, dt, dim, kv_heads, page
        n, self.kv_len = [a for a, _ in seqs], [b for _, b in seqs]
        self.q_start = [0] + list(np.cumsum(n))
        self.rows = int(self.q_start[-1])
        self.n_tokens = max(1, self.rows + extra_rows)
        need = [-(-b // page) for b in self.kv_len]
        wide = wide or max(max(need), 1)
        self.n_pages = sum(need) + 2
        order = rs.permutation(self.n_pages)
        self.pages = np.full((len(seqs), wide), -7, np.int32)
        at = 0
        for i, m in enumerate(need):
            self.pages[i, :m] = order[at:at + m]
            at += m
        for i, f in enumerate(first_page or ()):      # pages before a window are gone
            self.pages[i, :f] = -1
        shape = (self.n_pages, kv_heads, page, dim)
        self.k, self.v = self.cache(shape, layout), self.cache(shape, layout)
        self.start_d, self.len_d, self.pages_d = (torch.tensor(np.asarray(a, np.int32), device=DEV)
                                                  for a in (self.q_start, self.kv_len, self.pages))
        self.max_q, self.max_kv = max(max(n), 1), max(self.kv_len)

    def cache(self, shape, layout):
        if layout == "nhd":
            return self.values((shape[0], shape[2], shape[1], shape[3])).transpose(1, 2)
        if layout == "padded":       # rows further apart than they are long
            return self.values((shape[0], shape[1], shape[2], shape[3] + 24))[..., :shape[3]]
        return self.values(shape)

    def values(self, shape, dt=None, spread=1.0):
        x = torch.tensor(self.rs.standard_normal(shape) * spread, dtype=torch.float32, device=DEV)
        return x.to(U.TORCH_DT[dt or self.dt])

    def batch(self, **kw):
        a = dict(n_tokens=self.n_tokens, max_q_len=self.max_q, max_kv_len=self.max_kv)
        a.update(kw)
        return g.gguf_kv_batch(self.start_d, self.len_d, self.pages_d, a["n_tokens"], a["max_q_len"], a["max_kv_len"])

    def poison(self):
        """NaN and infinities in every slot that holds no key."""
        held = torch.zeros((self.n_pages, self.page), dtype=torch.bool, device=DEV)
        for b, length in enumerate(self.kv_len):
            for t in range(length):
                if self.pages[b, t // self.page] >= 0:
                    held[int(self.pages[b, t // self.page]), t % self.page] = True
        junk = torch.tensor([math.nan, math.inf, -math.inf, 6e4] * (self.dim // 4), device=DEV)
        for c in (self.k, self.v):
            c.copy_(torch.where(held[:, None, :, None], c.float(), junk).to(c.dtype))


# ------------------------------------------------------------------ append

def freqs_of(rot, base=10000.0):
    return torch.tensor(base ** (-2.0 * np.arange(rot // 2) / rot), dtype=torch.float32, device=DEV)


def check_append(c, xdt, heads, rot, style, scale=1.0, positions=None, fused=False, with_q=True, in_place=False,
                 ld_pad=0):
    T, D, KV = c.n_tokens, c.dim, c.kv_heads
    if fused:
        row = (heads + 2 * KV) * D + ld_pad
        qkv = c.values((T, row), xdt)
        q, k, v = (qkv[:, a:b].unflatten(1, (-1, D)) for a, b in
                   ((0, heads * D), (heads * D, (heads + KV) * D), ((heads + KV) * D, (heads + 2 * KV) * D)))
        ld = (row, row, row)
    else:
        q, k, v = c.values((T, heads, D), xdt), c.values((T, KV, D), xdt), c.values((T, KV, D), xdt)
        ld = (heads * D, KV * D, KV * D)
    q64, k64, v64 = (U.host64(x) for x in (q, k, v))
    kc0, vc0 = U.host64(c.k), U.host64(c.v)
    freqs = freqs_of(rot) if rot else None
    rope = g.gguf_rope(freqs, rot, style, scale, positions) if rot else None
    out = None
    if with_q:
        out = q if in_place else U.guarded((T, heads, D), U.TORCH_DT[c.dt], fill=3.0)
    out_t = out if in_place or out is None else out.t
    ldqo = ld[0] if in_place else heads * D
    g.gguf_kv_append(q if with_q else None, ld[0], k, ld[1], v, ld[2], U.DT[xdt], heads, rope, c.batch(),
                     g.gguf_kv_cache(c.k, c.v), out_t, ldqo)
    torch.cuda.synchronize()
    assert g.gguf_mm_check_errors() == 0
    fr = freqs.cpu().numpy() if rot else []
    qr, kr, vr = S.append(q64[:c.rows], k64, v64, fr, rot, style, scale, c.q_start, c.kv_len, c.pages, kc0, vc0,
                          None if positions is None else positions.cpu().numpy())
    bound = 8 * 2.0 ** -24 * 2 * max(abs(scale), 1.0) * max(np.abs(q64).max(), np.abs(k64).max()) if rot else 0.0
    if with_q:
        got = U.host64(out_t)
        near(got[:c.rows], qr, c.dt, bound, "q")
        if not in_place:
            out.check("q_out")
            assert np.all(got[c.rows:] == 3.0), "rows of no sequence were written"
        else:
            assert np.array_equal(got[c.rows:], q64[c.rows:])
    near(U.host64(c.k), kr, c.dt, bound, "k")
    near(U.host64(c.v), vr, c.dt, 0.0, "v")


@pytest.mark.parametrize("xdt,dt", [("f32", "bf16"), ("f32", "f16"), ("f16", "bf16"), ("bf16", "bf16"), ("f16", "f16"),
                                    ("bf16", "f16")])
@pytest.mark.parametrize("style", [S.NORM, S.NEOX])
def test_append_types(xdt, dt, style):
    c = Case([(1, 1), (7, 40), (0, 5), (3, 3), (1, 17)], 2, 64, dt, seed=1)
    check_append(c, xdt, 6, 64, style)


@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (96, 48), (80, 40), (80, 20), (112, 36), (16, 2), (48, 6),
                                     (64, 22), (32, 0)])
@pytest.mark.parametrize("style", [S.NORM, S.NEOX])
def test_append_rotated_part(dim, rot, style):
    c = Case([(5, 21), (1, 33)], 3, dim, "bf16", page=16, seed=dim + rot)
    check_append(c, "f16", 3, rot, style)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "padded"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_append_layouts(layout, page):
    c = Case([(3, 300), (2, 2), (40, 130)], 4, 128, "f16", page=page, layout=layout, extra_rows=5, seed=page)
    check_append(c, "f32", 8, 128, S.NEOX, fused=True, ld_pad=12)


def test_append_more_tokens_than_keys_and_none_at_all():
    # positions below zero are not stored; their queries are turned all the same
    c = Case([(4, 2), (3, 0), (2, 2)], 1, 64, "bf16", seed=5)
    check_append(c, "bf16", 2, 64, S.NORM)


def test_append_forms():
    for kw in (dict(with_q=False), dict(in_place=True), dict(scale=1.35), dict(in_place=True, fused=True)):
        c = Case([(9, 50), (1, 1)], 2, 128, "bf16", extra_rows=2, seed=6)
        check_append(c, "bf16", 8, 128, S.NEOX, **kw)


def test_append_far_and_given_positions():
    # angles of hundreds of thousands of turns keep their digits
    c = Case([(6, 9)], 2, 64, "f16", seed=7)
    pos = torch.tensor([0, 1, 131071, 1 << 20, (1 << 30) + 3, -5], dtype=torch.int32, device=DEV)
    check_append(c, "f32", 4, 64, S.NORM, positions=pos)


def test_append_page_out_of_range_is_reported_and_not_followed():
    c = Case([(4, 4), (3, 20)], 2, 64, "bf16", seed=8)
    c.pages_d[0, 0] = c.n_pages
    c.pages_d[1, 1] = -1
    k, v, q = c.values((7, 2, 64)), c.values((7, 2, 64)), c.values((7, 2, 64))
    before = c.k.clone(), c.v.clone()
    g.gguf_kv_append(q, 128, k, 128, v, 128, U.DT["bf16"], 2, None, c.batch(), g.gguf_kv_cache(c.k, c.v),
                     torch.empty_like(q), 128)
    assert g.gguf_mm_check_errors() == g.GGUF_ERR_INVALID_ARG
    assert g.gguf_mm_check_errors() == 0
    assert torch.equal(before[0], c.k) and torch.equal(before[1], c.v)


# ------------------------------------------------------------------ attention

def run_attn(c, q, causal=1, window=0, scale=None, lse=True, ldq=None, stream=None, **bounds):
    T, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    batch, cache = c.batch(**bounds), g.gguf_kv_cache(c.k, c.v)
    n = g.gguf_paged_attn_workspace_size(batch, cache, H)
    ws = U.workspace(n, 0xFF)
    out = U.guarded((c.n_tokens, H, D), U.TORCH_DT[c.dt], fill=3.0)
    ls = U.guarded((c.n_tokens, H), torch.float32, fill=3.0) if lse else None
    torch.cuda.synchronize()
    g.gguf_paged_attn(q, ldq or q.stride(0), H, batch, cache, scale, causal, window, out.t, H * D, ls.t if lse else None,
                      ws.t, n, stream)
    torch.cuda.synchronize()
    for b in (out, ws) + ((ls,) if lse else ()):
        b.check("attention")
    assert g.gguf_mm_check_errors() == 0
    return out.t, ls.t if lse else None


def check_attn(c, group, causal=1, window=0, scale=None, spread=1.0, ref_cache=None, poison=True, q=None, **kw):
    H, D = group * c.kv_heads, c.dim
    q = c.values((c.n_tokens, H, D), spread=spread) if q is None else q
    if poison:
        c.poison()
    out, lse = run_attn(c, q, causal, window, scale, **kw)
    kc, vc = ref_cache or (U.host64(c.k), U.host64(c.v))
    s = D ** -0.5 if scale is None else scale
    ref, rlse, vmax, smax = S.attention(U.host64(q)[:c.rows], kc, vc, c.q_start, c.kv_len, c.pages, s, causal, window)
    u = 2.0 ** -8 if c.dt == "bf16" else 2.0 ** -11
    e = 2.0 ** -23 * max(1, D / 4) * smax + 2.0 ** -20
    got = U.host64(out)
    near(got[:c.rows], ref, c.dt, ((u + 2 * e) * vmax)[..., None], "out")
    assert np.all(got[c.rows:] == 3.0), "rows of no sequence were written"
    if lse is not None:
        near(lse.cpu().numpy()[:c.rows], rlse, "f32", e, "lse")
    return out, lse


# bounds that make a call a large one: its keys are dealt out to all warps
LARGE = dict(max_kv_len=16 * 6000)
LARGE_WIDE = 6000          # pages of 16


# (new tokens, keys) of each sequence: single tokens, chunks, more tokens than
# keys, no keys, no tokens, lengths on both sides of pages and tiles
RAGGED = [(1, 1), (1, 16), (1, 17), (5, 5), (0, 9), (3, 200), (1, 129), (2, 0), (4, 2), (33, 64), (1, 255)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128])
@pytest.mark.parametrize("causal", [0, 1])
def test_attn_ragged(dt, dim, causal):
    check_attn(Case(RAGGED, 2, dim, dt, page=16, extra_rows=3, seed=dim), 4, causal)


@pytest.mark.parametrize("dt,dim", [("bf16", 128), ("f16", 64), ("bf16", 80), ("f16", 16)])
@pytest.mark.parametrize("causal,window", [(1, 0), (0, 0), (1, 21), (0, 130)])
@pytest.mark.parametrize("seqs,group", [(RAGGED[:6] + RAGGED[6:9], 1), ([(1, 2000)], 4), ([(3, 700), (16, 900)], 3),
                                        ([(1, 0), (1, 0)], 2), ([(1, 1 + 37 * i % 90) for i in range(300)], 1)])
def test_attn_keys_dealt_out(dt, dim, causal, window, seqs, group):
    check_attn(Case(seqs, 2, dim, dt, page=16, seed=dim + window, wide=LARGE_WIDE), group, causal, window, **LARGE)


@pytest.mark.parametrize("dt,dim", [("bf16", 128), ("f16", 64), ("bf16", 96)])
@pytest.mark.parametrize("seqs,group,window", [([(1, 9000)], 4, 0), ([(2, 3000)], 8, 0), ([(1, 5000)], 1, 700),
                                               ([(1, 3)], 16, 0), ([(3, 2500), (0, 10), (1, 1)], 5, 0)])
def test_attn_few_items_in_many_shares(dt, dim, seqs, group, window):
    # hundreds of shares of one item are joined, and as many warps have nothing where keys are few
    check_attn(Case(seqs, 2, dim, dt, page=16, seed=dim + group, wide=20000), group, 1, window, max_kv_len=16 * 20000)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 16, 20])
@pytest.mark.parametrize("seqs", [[(1, 300), (1, 77)], [(6, 70), (1, 1)], [(150, 200)]])
def test_attn_groups(group, seqs):
    check_attn(Case(seqs, 2, 64, "bf16", page=32, seed=group), group)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "padded"])
def test_attn_layouts(page, layout):
    check_attn(Case([(1, 400), (140, 300), (2, 3)], 2, 128, "f16", page=page, layout=layout, seed=page), 2)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 128, 1 << 40])
@pytest.mark.parametrize("causal", [0, 1])
def test_attn_window(window, causal):
    check_attn(Case([(1, 300), (130, 260), (20, 20), (3, 1)], 2, 64, "bf16", page=16, seed=3), 3, causal, min(window, 1 << 40))


def test_attn_pages_before_the_window_are_gone():
    # keys that no row sees any more: their pages may be anyone's
    c = Case([(1, 500), (70, 400), (1, 40)], 2, 64, "bf16", page=16, seed=4, first_page=[25, 14, 0])
    check_attn(c, 4, 1, 100)


def test_attn_long_single_tokens():
    check_attn(Case([(1, 3001), (1, 1), (1, 40), (1, 2048)], 1, 128, "bf16", page=64, seed=9), 8)
    check_attn(Case([(1, 9000)], 2, 64, "f16", page=16, seed=10), 1)


def test_attn_prompt_longer_than_tiles():
    check_attn(Case([(300, 300), (129, 600)], 2, 128, "bf16", page=32, seed=11), 2)


@pytest.mark.parametrize("spread,scale", [(30.0, None), (1.0, 1e-4), (200.0, 1.0), (0.0, None)])
def test_attn_scores_of_any_size(spread, scale):
    # one key takes all the weight; all keys the same; scores of many thousands
    check_attn(Case([(1, 700), (40, 90), (140, 140)], 2, 64, "f16", page=16, seed=12), 2, scale=scale, spread=spread)


def test_attn_extreme_keys():
    # keys whose scores overflow to -inf beside ordinary ones: they weigh nothing
    c = Case([(1, 50), (130, 130)], 1, 64, "bf16", page=16, seed=13)
    q = c.values((c.n_tokens, 2, 64)).abs() + 0.5
    c.k[int(c.pages[0, 1]), 0, 3] = -3.0e38
    c.k[int(c.pages[1, 0]), 0, 5] = -3.0e38
    out, lse = run_attn(c, q)
    kc = U.host64(c.k)
    ref, rlse, vmax, _ = S.attention(U.host64(q), kc, U.host64(c.v), c.q_start, c.kv_len, c.pages, 64 ** -0.5, 1, 0)
    near(U.host64(out), ref, "bf16", (2.0 ** -8 + 1e-3) * vmax[..., None])
    near(lse.cpu().numpy(), rlse, "f32", 1e-4)


@pytest.mark.parametrize("n", [1, 130])
@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("where", range(12, 20))
def test_attn_nan_in_a_seen_key_reaches_its_rows_alone(n, what, where):
    # a value: one column of the rows that see it; a key: all of them, wherever it stands
    c = Case([(n, n + 20), (n, n + 20)], 1, 64, "bf16", page=16, seed=14)
    at = int(c.pages[0, where // 16]), 0, where % 16
    q = c.values((2 * n, 1, 64)).abs() + 0.5
    keep = c.v[at][7].clone()
    c.v[at][7] = what
    out, _ = run_attn(c, q)
    assert not torch.isfinite(out[:n, 0, 7]).any() and torch.isfinite(out[n:]).all()
    assert torch.isfinite(out[:n, 0, :7]).all() and torch.isfinite(out[:n, 0, 8:]).all()
    c.v[at][7] = keep
    c.k[at][:] = what
    out, lse = run_attn(c, q)
    assert torch.isnan(out[:n]).all() and torch.isfinite(out[n:]).all() and torch.isfinite(lse[n:]).all()


def test_attn_strided_queries():
    c = Case([(1, 90), (20, 41), (130, 130)], 2, 64, "bf16", seed=15)
    wide = c.values((c.n_tokens, 4 * 64 + 2 * 2 * 64))
    q = wide[:, :256].unflatten(1, (4, 64))
    check_attn(c, 2, q=q, ldq=wide.stride(0))


def test_attn_without_lse_and_with_loose_bounds():
    c = Case([(1, 90), (20, 41)], 2, 64, "bf16", seed=16, wide=40)
    q = c.values((c.n_tokens, 4, 64))
    a, _ = run_attn(c, q, lse=False)
    b, _ = run_attn(c, q, max_q_len=21, max_kv_len=640)
    ref, _, vmax, _ = S.attention(U.host64(q), U.host64(c.k), U.host64(c.v), c.q_start, c.kv_len, c.pages, 0.125, 1, 0)
    for x in (a, b):
        near(U.host64(x), ref, "bf16", (2.0 ** -8 + 1e-4) * vmax[..., None])


def test_attn_cache_beyond_32_bit_offsets():
    # pages 3 GB apart: element offsets pass 2**31
    D, KV, page = 64, 2, 16
    far = torch.empty(((1 << 31) + (1 << 30)) * 2, dtype=torch.bfloat16, device=DEV)
    c = Case([(1, 40), (130, 140)], KV, D, "bf16", page=page, seed=17)
    n, step = c.n_pages, (far.numel() // c.n_pages) // 64 * 64
    views = [torch.as_strided(far, (n, KV, page, D), (step, 2 * page * D, D, 1), off) for off in (0, page * D)]
    for view, x in zip(views, (c.k, c.v)):
        view.copy_(x)
    near_k, near_v = c.k, c.v
    q = c.values((c.n_tokens, 4, D))
    a, _ = run_attn(c, q)
    c.k, c.v = views
    b, _ = run_attn(c, q)
    assert torch.equal(a, b)
    # and the append writes there
    k, v = c.values((c.n_tokens, KV, D)), c.values((c.n_tokens, KV, D))
    for kk, vv in ((near_k, near_v), views):
        g.gguf_kv_append(None, 0, k, KV * D, v, KV * D, U.DT["bf16"], 0, None, c.batch(), g.gguf_kv_cache(kk, vv), None, 0)
    torch.cuda.synchronize()
    assert torch.equal(views[0], near_k) and torch.equal(views[1], near_v)


def test_attn_repeats_bit_for_bit_and_on_another_stream():
    c = Case([(1, 4000), (1, 1000), (90, 130)], 2, 128, "bf16", page=16, seed=18)
    q = c.values((c.n_tokens, 16, 128))
    first, lse = run_attn(c, q)
    side = torch.cuda.Stream()
    for _ in range(5):
        again, l2 = run_attn(c, q, stream=side)
        assert torch.equal(first, again) and torch.equal(lse, l2)


def test_attn_page_out_of_range_is_reported_and_not_followed():
    for seqs in ([(1, 40), (1, 40)], [(150, 150), (1, 40)]):
        c = Case(seqs, 1, 64, "bf16", page=16, seed=19)
        c.pages_d[0, 1] = 1 << 28
        q = c.values((c.n_tokens, 2, 64))
        out = torch.zeros_like(q)
        n = g.gguf_paged_attn_workspace_size(c.batch(), g.gguf_kv_cache(c.k, c.v), 2)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        g.gguf_paged_attn(q, 128, 2, c.batch(), g.gguf_kv_cache(c.k, c.v), 0.125, 1, 0, out, 128, None, ws, n)
        assert g.gguf_mm_check_errors() == g.GGUF_ERR_INVALID_ARG
        assert g.gguf_mm_check_errors() == 0
        # the other sequence has its result
        ref, _, vmax, _ = S.attention(U.host64(q)[-1:], U.host64(c.k), U.host64(c.v), [0, 1], [40], c.pages[1:], 0.125, 1, 0)
        near(U.host64(out)[-1:], ref, "bf16", (2.0 ** -8 + 1e-4) * vmax[..., None])


def test_append_then_attend_in_a_captured_graph():
    # the arrays may change between replays: the graph reads them when it runs
    c = Case([(1, 30), (1, 64)], 2, 64, "bf16", seed=20)
    KV, D, H = 2, 64, 8
    qkv = c.values((2, (H + 2 * KV) * D))
    q, k, v = (qkv[:, a:b].unflatten(1, (-1, D)) for a, b in ((0, H * D), (H * D, (H + KV) * D), ((H + KV) * D, (H + 2 * KV) * D)))
    ld = qkv.stride(0)
    qo, out = torch.empty((2, H, D), dtype=torch.bfloat16, device=DEV), torch.empty((2, H, D), dtype=torch.bfloat16, device=DEV)
    batch, cache, rope = c.batch(), g.gguf_kv_cache(c.k, c.v), g.gguf_rope(freqs_of(64), 64, S.NEOX)
    n = g.gguf_paged_attn_workspace_size(batch, cache, H)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        g.gguf_kv_append(q, ld, k, ld, v, ld, U.DT["bf16"], H, rope, batch, cache, qo, H * D, stream)
        g.gguf_paged_attn(qo, H * D, H, batch, cache, D ** -0.5, 1, 0, out, H * D, None, ws, n, stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for length in ([30, 64], [25, 50], [1, 17]):
        c.len_d.copy_(torch.tensor(length, dtype=torch.int32))
        qkv.copy_(c.values(qkv.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        ref, _, vmax, _ = S.attention(U.host64(qo), U.host64(c.k), U.host64(c.v), c.q_start, length, c.pages, 0.125, 1, 0)
        near(U.host64(got), ref, "bf16", (2.0 ** -8 + 1e-4) * vmax[..., None])


# ------------------------------------------------------------------ logits

def check_logits(rows, vocab, dt="f32", odt="f32", hist=None, biases=None, grammar=None, pens=(True, True, True), pad=0,
                 in_place=False, seed=0, x=None):
    rs = np.random.default_rng(seed)
    ld = vocab + pad
    base = torch.tensor(rs.standard_normal((rows, ld)) * 4, dtype=torch.float32, device=DEV).to(U.TORCH_DT[dt])
    if x is not None:
        base[:, :vocab] = torch.as_tensor(x, device=DEV).to(base.dtype)
    x64 = U.host64(base)
    if in_place:
        out, ldo = base, ld
    else:
        out_g, ldo = U.guarded((rows, vocab + 3), U.TORCH_DT[odt], fill=7.0), vocab + 3
        out = out_g.t
    t = lambda a, d: torch.tensor(np.asarray(a, d), device=DEV)  # noqa: E731
    kw, pen = {}, [None, None, None]
    if hist is not None:
        kw["hist"] = t([i for h in hist for i in h] or [0], np.int32)
        kw["hist_start"] = t(np.cumsum([0] + [len(h) for h in hist]), np.int32)
        for k, (name, on, lo, hi) in enumerate(zip(("repeat", "frequency", "presence"), pens, (1.0, -0.3, -0.5), (1.5, 0.5, 1.0))):
            if on:
                pen[k] = rs.uniform(lo, hi, rows).astype(np.float32)
                kw[name] = t(pen[k], np.float32)
    if biases is not None:
        kw["bias_ids"] = t([i for b in biases for i, _ in b] or [0], np.int32)
        kw["bias"] = t([v for b in biases for _, v in b] or [0], np.float32)
        kw["bias_start"] = t(np.cumsum([0] + [len(b) for b in biases]), np.int32)
    allow = None
    if grammar is not None:
        allow = rs.random((rows, vocab)) < np.reshape(grammar, (-1, 1))
        words = -(-vocab // 32)
        full = np.ones((rows, words * 32), bool)       # bits past the vocabulary mean nothing
        full[:, :vocab] = allow
        bits = (full.reshape(rows, words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
        kw["allow"] = t(bits.view(np.int32), np.int32)
    g.gguf_logits_adjust(base, U.DT[dt], ld, rows, vocab, g.gguf_logit_rules(**kw), out, U.DT[odt], ldo)
    torch.cuda.synchronize()
    assert g.gguf_mm_check_errors() == 0
    f32b = None if biases is None else [[(i, np.float32(v)) for i, v in b] for b in biases]
    ref = S.logits(x64[:, :vocab], hist, *pen, f32b, allow)
    got = U.host64(out)
    most = max([len(h) for h in hist or [[]]] + [1])
    nb = max([len(b) for b in biases or [[]]] + [0])
    finite = np.abs(x64[:, :vocab][np.isfinite(x64[:, :vocab])]).max()
    bound = (4 + nb) * 2.0 ** -23 * (1.5 * finite + 0.5 * most + 1 + sum(abs(v) for b in biases or [] for _, v in b))
    nan = np.isnan(ref)
    assert np.array_equal(nan, np.isnan(got[:, :vocab]))
    near(np.where(nan, 0, got[:, :vocab]), np.where(nan, 0, ref), odt, bound, "logits")
    if in_place:
        assert np.array_equal(got[:, vocab:], x64[:, vocab:]), "wrote past the rows"
    else:
        assert np.all(got[:, vocab:] == 7.0), "wrote past the rows"
        out_g.check("logits")


def some_hist(rs, vocab, lens):
    return [list(rs.integers(0, min(vocab, 50), n)) for n in lens]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("odt", ["f32", "f16", "bf16"])
def test_logits_types(dt, odt):
    rs = np.random.default_rng(1)
    check_logits(3, 5003, dt, odt, some_hist(rs, 5003, [0, 400, 31]), [[(7, 1.5)], [], [(0, -2.0), (5002, 3.0)]], [0.5])


@pytest.mark.parametrize("vocab", [1, 2, 3, 5, 31, 33, 4095, 4096, 4097, 8195, 70001])
@pytest.mark.parametrize("pad", [0, 1, 2, 7])
def test_logits_sizes(vocab, pad):
    rs = np.random.default_rng(vocab)
    hist = some_hist(rs, vocab, [5, 0, 900, 1, 64])
    hist[1] = [vocab - 1, 0, vocab - 1]
    biases = [[], [(vocab - 1, 2.0)], [(0, 1.0), (0, 0.25), (vocab - 1, -1.0)], [], [(vocab // 2, 0.5)]]
    check_logits(5, vocab, hist=hist, biases=biases, grammar=[0.3], pad=pad, seed=vocab)


@pytest.mark.parametrize("pens", [(True, False, False), (False, True, False), (False, False, True), (False, False, False)])
def test_logits_each_rule_alone(pens):
    rs = np.random.default_rng(2)
    check_logits(2, 999, hist=some_hist(rs, 999, [40, 3]), pens=pens)


def test_logits_only_a_mask_or_only_biases_or_nothing():
    check_logits(4, 3001, grammar=[0.0, 1.0, 0.5, 0.01])          # one row leaves no token, one leaves all
    check_logits(2, 3001, biases=[[(i, 0.1) for i in range(300)], [(5, 1.0)] * 40])
    check_logits(2, 3001, "f16", "f16", in_place=True, pad=5)


def test_logits_in_place():
    rs = np.random.default_rng(3)
    for dt in ("f32", "bf16"):
        check_logits(3, 4501, dt, dt, some_hist(rs, 4501, [10, 100, 0]), [[(1, 1.0)], [], []], [0.5], pad=3, in_place=True)


def test_logits_of_no_finite_value():
    x = np.random.default_rng(4).standard_normal((3, 600))
    x[0, :40] = -np.inf
    x[1, 10:50] = np.inf
    x[2, 5:30] = np.nan
    x[0, 100] = np.finfo(np.float32).min / 2
    check_logits(3, 600, hist=[list(range(0, 60)), list(range(0, 30)), list(range(0, 10))], x=x, pens=(True, False, False),
                 biases=[[(3, 1.0)], [(12, -1.0)], [(6, 1.0)]], grammar=[0.8])


def test_logits_ids_outside_the_vocabulary_count_nowhere():
    check_logits(2, 100, hist=[[-1, 100, 5, 2 ** 31 - 1, -2 ** 31], [99, 99]], biases=[[(-3, 9.0), (100, 9.0), (4, 1.0)], []])


def test_logits_long_history_of_one_token():
    check_logits(1, 64, hist=[[9] * 70000], pens=(False, True, False))


# ------------------------------------------------------------------ refusals that need a device's pointers

def test_refusals():
    c = Case([(1, 5)], 2, 64, "bf16")
    q, out = c.values((1, 4, 64)), c.values((1, 4, 64))
    cache = g.gguf_kv_cache(c.k, c.v)

    def attn(q=q, ldq=256, heads=4, batch=None, cache=cache, scale=0.125, causal=1, window=0, out=out, ldo=256):
        n = 1 << 20
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
        g.gguf_paged_attn(q, ldq, heads, batch or c.batch(), cache, scale, causal, window, out, ldo, None, ws, n)

    attn()
    for want, kw in ((g.GGUF_ERR_INVALID_ARG, dict(heads=3)), (g.GGUF_ERR_INVALID_ARG, dict(scale=0.0)),
                     (g.GGUF_ERR_INVALID_ARG, dict(scale=math.inf)), (g.GGUF_ERR_INVALID_ARG, dict(window=-1)),
                     (g.GGUF_ERR_INVALID_ARG, dict(ldq=255)), (g.GGUF_ERR_MISALIGNED, dict(ldq=260)),
                     (g.GGUF_ERR_MISALIGNED, dict(q=q.data_ptr() + 2)), (g.GGUF_ERR_INVALID_ARG, dict(q=None)),
                     (g.GGUF_ERR_INVALID_ARG, dict(batch=c.batch(max_kv_len=17))),
                     (g.GGUF_ERR_UNSUPPORTED, dict(heads=2 * 129, ldq=2 * 129 * 64, ldo=2 * 129 * 64))):
        with pytest.raises(g.GGUFError) as e:
            attn(**kw)
        assert e.value.status == want, kw
    torch.cuda.synchronize()
    assert g.gguf_mm_check_errors() == 0
