"""The normed append, the router, the experts' feed-forward and sampling on the
GPU against the 64-bit definitions in oracle/serving_oracle.py.

Tolerances.
  * normed append: as the append's (8 * 2**-24 * (|a| + |b|) of the normed pair),
    and the norm's own: a sum of D squares is off by at most D * 2**-24 of
    itself, its root by half of that, the division, the root and the two
    products by half a unit each: (D / 2 + 4) * 2**-24 more.  Values v are exact.
  * router: ids are equal.  A score's f32 error is at most (K + 8) * 2**-24 * |x| . |w|
    (K products summed in any order); a weight moves by twice the largest of
    those, relative to itself, before the renormalisation and by as much through
    it, and by 2**-20 for the exponentials and the quotient.
  * feed-forward: see ffn_bound().
  * sampling: tokens are equal.  log(w / W) has an f32 quotient, its
    logarithm and W's rounding: 2**-21 absolutely and relatively.
"""
import math

import numpy as np
import pytest
import torch

import gguf_quant_weight_gb300 as g
import gguf_synth as syn
from oracle import gguf_oracle as O
from oracle import serving_oracle as S
from tests import gpu_util as U
from tests.test_serving import Case, freqs_of, near

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    U.require_gpu()


def h64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ normed append

def run_append(c, xdt, heads, rot, style, fused, q_norm=True, k_norm=True, eps=1e-6, has_q=True, scale=1.0, in_place=False, spread=2.0):
    T, D, KV = c.n_tokens, c.dim, c.kv_heads
    if fused:
        qkv = c.values((T, (heads + 2 * KV) * D), xdt, spread)
        q, k, v = (t.view(T, -1, D) for t in qkv.split((heads * D, KV * D, KV * D), dim=1))
    else:
        q, k, v = (c.values((T, h, D), xdt, spread) for h in (heads, KV, KV))
    if in_place:
        q = q.contiguous()
    wq, wk = (torch.tensor(1 + 0.3 * c.rs.standard_normal(D), dtype=torch.float32, device=DEV) for _ in range(2))
    wq, wk = (wq if q_norm else None), (wk if k_norm else None)
    norm = g.gguf_head_norm(wq, wk, eps)
    out = U.guarded((T, heads, D), U.TORCH_DT[c.dt], 3.0)
    before = c.k.clone(), c.v.clone(), q.clone()
    freqs = freqs_of(rot) if rot else None
    rope = g.gguf_rope(freqs, rot, style, scale) if rot else None
    target = q if in_place else out.t
    g.gguf_kv_append_norm(q if has_q else None, q.stride(0), k, k.stride(0), v, v.stride(0), U.DT[xdt], heads, norm, rope, c.batch(),
                          g.gguf_kv_cache(c.k, c.v), target if has_q else None, heads * D)
    assert g.gguf_mm_check_errors() == 0
    out.check()
    cpu = lambda t: None if t is None else h64(t)      # noqa: E731
    nq, nk = S.head_norm(h64(before[2]), cpu(wq), eps), S.head_norm(h64(k), cpu(wk), eps)
    f = freqs.cpu().numpy() if rot else np.zeros(0)
    qo, kc, vc = S.append(nq, nk, h64(v), f, rot, style, scale, c.q_start, c.kv_len, c.pages, h64(before[0]), h64(before[1]))
    rows = c.rows
    u = (8 + D / 2 + 4) * 2.0 ** -24 * 2 * abs(scale)
    if has_q and rows:
        near(h64(target)[:rows], qo[:rows], c.dt, u * np.abs(nq[:rows]).max(-1, keepdims=True), "q")
    if not in_place:
        assert torch.equal(out.t[rows if has_q else 0:], torch.full_like(out.t[rows if has_q else 0:], 3.0))
    near(h64(c.k), kc, c.dt, u * max(1.0, np.abs(nk).max()), "k")
    near(h64(c.v), vc, c.dt, 0.0, "v")


@pytest.mark.parametrize("dim,rot,style", [(128, 128, 1), (128, 128, 0), (64, 64, 1), (80, 40, 0), (96, 48, 1), (128, 2, 1), (128, 6, 1),
                                           (112, 10, 0), (128, 8, 1), (128, 4, 0), (16, 16, 1), (128, 0, 0), (128, 126, 1), (48, 24, 1)])
@pytest.mark.parametrize("xdt,dt", [("bf16", "bf16"), ("f32", "f16")])
def test_append_norm_head_layouts(dim, rot, style, xdt, dt):
    run_append(Case([(1, 9), (5, 17), (0, 3), (2, 2)], 2, dim, dt, extra_rows=2, seed=dim + rot), xdt, 6, rot, style, fused=True)


@pytest.mark.parametrize("kw", [dict(q_norm=False), dict(k_norm=False), dict(q_norm=False, k_norm=False), dict(has_q=False),
                                dict(scale=0.5), dict(in_place=True, fused=False), dict(eps=0.0), dict(spread=1e-3), dict(eps=1.0)])
def test_append_norm_forms(kw):
    a = dict(fused=True)
    a.update(kw)
    run_append(Case([(3, 20), (1, 1), (7, 7)], 3, 128, "bf16", page=32, layout="nhd", seed=5), "bf16", 9, 128, 1, **a)


@pytest.mark.parametrize("seqs,heads,kv", [([(1, 1)], 1, 1), ([(1, 1001)], 32, 4), ([(700, 800)], 5, 1), ([(1, 50 + i) for i in range(200)], 16, 16)])
def test_append_norm_batches(seqs, heads, kv):
    run_append(Case(seqs, kv, 128, "bf16", page=64, layout="padded", seed=7), "bf16", heads, 128, 1, fused=False)


def test_append_norm_without_norms_is_the_append():
    outs = []
    for normed in (False, True):
        c = Case([(4, 30), (1, 5)], 2, 96, "bf16", seed=11)
        q, k, v = (c.values((c.n_tokens, h, 96)) for h in (4, 2, 2))
        out = torch.zeros((c.n_tokens, 4, 96), dtype=torch.bfloat16, device=DEV)
        rope, cache = g.gguf_rope(freqs_of(48), 48, 1), g.gguf_kv_cache(c.k, c.v)
        if normed:
            g.gguf_kv_append_norm(q, 384, k, 192, v, 192, 2, 4, g.gguf_head_norm(None, None), rope, c.batch(), cache, out, 384)
        else:
            g.gguf_kv_append(q, 384, k, 192, v, 192, 2, 4, rope, c.batch(), cache, out, 384)
        outs.append((out, c.k, c.v))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_append_norm_reports_arrays_out_of_range():
    c = Case([(2, 9), (3, 9)], 2, 64, "bf16", seed=3)
    q, k, v = (c.values((5, h, 64)) for h in (2, 2, 2))
    was = c.k.clone()
    out = torch.full((5, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    c.start_d.copy_(torch.tensor([0, 4, 2], dtype=torch.int32))
    g.gguf_kv_append_norm(q, 128, k, 128, v, 128, 2, 2, g.gguf_head_norm(torch.ones(64, device=DEV), None), None, c.batch(max_q_len=5),
                          g.gguf_kv_cache(c.k, c.v), out, 128)
    assert g.gguf_mm_check_errors() == g.GGUF_ERR_INVALID_ARG
    assert torch.equal(c.k, was) and bool((out == 3.0).all())


# ------------------------------------------------------------------ router

def run_router(x, w, top_k, sigmoid=False, bias=None, renorm=True, scale=1.0, stream=None):
    T, K = x.shape
    ids, weights = U.guarded((T, top_k), torch.int32, -9), U.guarded((T, top_k), torch.float32, -9.0)
    xdt = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[x.dtype]
    router = g.gguf_router(w, top_k, int(sigmoid), bias, renorm, scale)
    g.gguf_moe_router(x, xdt, T, K, router, ids.t, weights.t, stream)
    assert g.gguf_mm_check_errors() == 0
    ids.check(), weights.check()
    return ids.t.cpu().numpy(), h64(weights.t)


def check_router(x, w, top_k, **kw):
    ids, weights = run_router(x, w, top_k, **kw)
    b = kw.get("bias")
    ri, rw = S.router(h64(x), h64(w), None if b is None else h64(b), top_k, kw.get("sigmoid", False), kw.get("renorm", True),
                      kw.get("scale", 1.0))
    assert np.array_equal(ids, ri), (np.argwhere(ids != ri)[:5], ids[ids != ri][:5], ri[ids != ri][:5])
    e = (x.shape[1] + 8) * 2.0 ** -24 * (np.abs(h64(x)) @ np.abs(h64(w)).T).max(-1, keepdims=True)
    assert np.all(np.abs(weights - rw) <= (4 * e + 2.0 ** -20) * np.abs(rw))


def router_inputs(T, K, E, xdt="bf16", wdt="f32", seed=0):
    rs = np.random.default_rng(seed)
    f = lambda a, dt: torch.tensor(a, dtype=torch.float32, device=DEV).to(U.TORCH_DT[dt])      # noqa: E731
    return f(rs.standard_normal((T, K)), xdt), f(rs.standard_normal((E, K)) / math.sqrt(K), wdt), f(0.2 * rs.standard_normal(E), "f32")


@pytest.mark.parametrize("T,K,E,k", [(1, 2048, 128, 8), (1, 8, 1, 1), (2, 40, 3, 3), (5, 7168, 256, 8), (7, 64, 1024, 64), (19, 2080, 60, 4),
                                     (33, 512, 17, 2), (64, 1024, 160, 6), (150, 264, 128, 8), (509, 256, 128, 8), (600, 128, 8, 2), (1300, 72, 33, 5)])
@pytest.mark.parametrize("kw", [dict(), dict(sigmoid=True, biased=True, scale=2.5), dict(biased=True, renorm=False)])
def test_router_sizes(T, K, E, k, kw):
    x, w, b = router_inputs(T, K, E, seed=T + K)
    kw = dict(kw)
    if kw.pop("biased", False):
        kw["bias"] = b
    check_router(x, w, k, **kw)


@pytest.mark.parametrize("xdt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("wdt", ["f32", "f16", "bf16"])
def test_router_types(xdt, wdt):
    x, w, b = router_inputs(9, 1032, 40, xdt, wdt, 3)
    check_router(x, w, 7, sigmoid=True, bias=b, renorm=False)


@pytest.mark.parametrize("T", [1, 40, 200])
@pytest.mark.parametrize("kw", [dict(), dict(sigmoid=True, biased=True), dict(biased=True), dict(sigmoid=True)])
def test_router_orders_scores_that_f32_cannot_tell(T, kw):
    """Experts in families of copies whose rows differ in one value by a last bit, or not at all."""
    rs = np.random.default_rng(4)
    x, w, b = router_inputs(T, 2048, 64, "f32", "f32", 5)
    w = w.cpu().numpy()
    for e in range(64):
        w[e] = w[e % 16]
        if e >= 32:     # the others are equal and go by their index
            w[e, rs.integers(2048)] *= 1 + 2.0 ** -rs.integers(20, 24)
    kw = dict(kw)
    if kw.pop("biased", False):
        b = b.cpu().numpy()
        kw["bias"] = torch.tensor(b[np.arange(64) % 16], device=DEV)
    check_router(x, torch.tensor(w, device=DEV), 12, **kw)


def test_router_all_scores_equal():
    x, w, _ = router_inputs(3, 64, 100)
    ids, weights = run_router(torch.zeros_like(x), w, 10)
    assert np.array_equal(ids, np.tile(np.arange(10), (3, 1))) and np.allclose(weights, 0.1, rtol=1e-6)


def test_router_scores_that_are_not_finite():
    x, w, b = router_inputs(4, 64, 20)
    x[1, 3] = math.nan
    x[2, 5] = math.inf
    for kw in (dict(), dict(sigmoid=True, bias=b)):
        ids, weights = run_router(x, w, 6, **kw)
        assert all(len(set(r)) == 6 and r.min() >= 0 and r.max() < 20 for r in ids)
        for t in (0, 3):
            ri, rw = S.router(h64(x[t:t + 1]), h64(w), None if "bias" not in kw else h64(b), 6, "bias" in kw, True, 1.0)
            assert np.array_equal(ids[t], ri[0]) and np.allclose(weights[t], rw[0], rtol=1e-5)


@pytest.mark.parametrize("top_k", [1, 5, 12, 20])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_router_experts_masked_by_their_bias(top_k, sigmoid):
    """Biases of -inf shut experts out: they come last, by index; +inf ones come first."""
    x, w, b = router_inputs(6, 256, 20, seed=8)
    b[[0, 3, 7, 8, 19]] = -math.inf
    b[11] = math.inf
    w[5] = w[4]
    b[5] = b[4]
    check_router(x, w, top_k, sigmoid=sigmoid, bias=b)


@pytest.mark.parametrize("kw", [dict(), dict(sigmoid=True), dict(biased=True), dict(sigmoid=True, biased=True)])
@pytest.mark.parametrize("top_k", [2, 15, 20])
def test_router_ids_differ_whatever_the_scores_are(kw, top_k):
    x, w, b = router_inputs(8, 64, 20, "f32", seed=9)
    w[6] = w[5]                        # a tie, so that the scores are computed again
    x[0, 3], x[1, 5], x[2], x[3, 0], x[3, 1] = math.nan, math.inf, math.nan, math.inf, -math.inf
    x[4] = 3e38
    w[9, 2] = math.nan
    b[3], b[5], b[6] = math.nan, 0.1, 0.1
    kw = dict(kw)
    if kw.pop("biased", False):
        kw["bias"] = b
    ids, _ = run_router(x, w, top_k, **kw)
    assert all(len(set(r)) == top_k and r.min() >= 0 and r.max() < 20 for r in ids)


# ------------------------------------------------------------------ the experts' feed-forward

FORMATS = {"Q4_0": syn.Q4_0, "Q4_1": syn.Q4_1, "Q5_0": syn.Q5_0, "Q5_1": syn.Q5_1, "Q8_0": syn.Q8_0, "Q2_K": syn.Q2_K, "Q3_K": syn.Q3_K,
           "Q4_K": syn.Q4_K, "Q5_K": syn.Q5_K, "Q6_K": syn.Q6_K}
MIN_AT = {"Q4_1": 2, "Q5_1": 2, "Q2_K": 82, "Q4_K": 2, "Q5_K": 2}


class Experts:
    """Random experts as blocks on the device, their values, and the magnitudes that their products are made of: where a
    weight is a scaled code less a min, those of the two parts."""

    def __init__(self, types, K, F, E, seed=0):
        rs = syn.rng(seed)
        self.K, self.F, self.E = K, F, E
        self.types = [FORMATS[t] for t in types]
        self.dev, self.val, self.mag = [], [], []
        for t, n, k in zip(types, (F, F, K), (K, K, F)):
            qt, scale = FORMATS[t], 20.0 / math.sqrt(k)
            blocks = [self.scaled(syn.weight_blocks(rs, qt, n, k), t, scale) for _ in range(E)]
            val = np.stack([O.dequant(b, qt, n, k) for b in blocks])
            mag = np.abs(val)
            if t in MIN_AT:
                rest = []
                for b in blocks:
                    b = b.copy().reshape(-1, g.BLOCK_BYTES[qt])
                    b[:, MIN_AT[t]:MIN_AT[t] + 2] = 0
                    rest.append(O.dequant(b.reshape(n, -1), qt, n, k))
                rest = np.stack(rest)
                mag = np.abs(rest) + np.abs(val - rest)
            self.dev.append(torch.from_numpy(np.stack(blocks)).to(DEV))
            self.val.append(val)
            self.mag.append(mag)

    @staticmethod
    def scaled(blocks, t, scale):
        """The f16 fields brought to the size of a layer's weights."""
        qt = FORMATS[t]
        b = blocks.copy().reshape(-1, g.BLOCK_BYTES[qt])
        at = {"Q2_K": (80, 82), "Q3_K": (108,), "Q6_K": (208,)}.get(t, (0,) + ((MIN_AT[t],) if t in MIN_AT else ()))
        spread = float(np.std(O.dequant(blocks, qt, blocks.shape[0], b.shape[0] // blocks.shape[0] * g.BLOCK_VALUES[qt])))
        for a in at:
            v = b[:, a:a + 2].copy().view(np.float16).astype(np.float64) * (0.05 * scale / spread)
            b[:, a:a + 2] = v.astype(np.float16).view(np.uint8).reshape(-1, 2)
        return b.reshape(blocks.shape)

    def struct(self, gelu=False):
        return g.gguf_moe_weights(*self.dev, *self.types, self.K, self.F, self.E, int(gelu))


def ffn_bound(ex, x, ids, weights, gelu, ydt, residual):
    """The largest error of y that the arithmetic allows.

    Products: an f32 activation is two f16 numbers, within 2**-21 of it (16-bit ones are exact) and 2**-33 of the row's largest;
    a sum of K products in f32 is off by (K / 16 + 40) * 2**-23 of the sum of magnitudes (an addition per 16 products in the
    tensor core, then the chunks', parts' and warps').
    Activation: its slope is below 1.13, expf and tanhf with the arithmetic around them are off by 2**-20 of the value and, where
    1 + tanh cancels, of 2**-22 |a|.  The hidden value is rounded to 2**-11 (bf16 outputs) or 2**-21 of itself and 2**-33
    (2**-24) of its chunk's largest.
    Then the second product and the weighted sum: top_k + 2 additions and products of half a unit each."""
    T, K = x.shape
    out = np.zeros((T, K))
    sums = lambda k: (k / 16 + 40) * 2.0 ** -23 + 2.0 ** -21      # noqa: E731
    for t in range(T):
        big = np.abs(x[t]).max()
        for s, e in enumerate(ids[t]):
            if not 0 <= e < ex.E:
                continue
            ax = np.abs(x[t]) + 2.0 ** -10 * big
            a, b = ex.val[0][e] @ x[t], ex.val[1][e] @ x[t]
            ea, eb = sums(K) * (ex.mag[0][e] @ ax), sums(K) * (ex.mag[1][e] @ ax)
            act = S.activate(a, gelu)
            h = act * b
            eh = 1.13 * ea * (np.abs(b) + eb) + np.abs(act) * eb + 2.0 ** -20 * np.abs(h) + 2.0 ** -22 * np.abs(a * b)
            eh += (2.0 ** -11 if ydt == "bf16" else 2.0 ** -21) * np.abs(h) + (2.0 ** -24 if ydt == "bf16" else 2.0 ** -33) * np.abs(h).max()
            row = ex.mag[2][e] @ (np.abs(h) + eh)
            out[t] += abs(weights[t, s]) * (np.abs(ex.val[2][e]) @ eh + (sums(ex.F) + (len(ids[t]) + 2) * 2.0 ** -23) * row)
        if residual is not None:
            out[t] += 2.0 ** -23 * (len(ids[t]) + 2) * np.abs(residual[t])
    return out


def run_ffn(ex, T, top_k, xdt="bf16", ydt="bf16", gelu=False, residual=True, ids=None, seed=0, alias=False, x=None, weights=None, stream=None):
    rs = np.random.default_rng(seed)
    x = torch.tensor(rs.standard_normal((T, ex.K)) if x is None else x, dtype=torch.float32, device=DEV).to(U.TORCH_DT[xdt])
    if ids is None:
        ids = np.stack([rs.permutation(ex.E)[:top_k] for _ in range(T)])
    ids = np.asarray(ids, np.int32)
    weights = rs.dirichlet(np.ones(top_k), T).astype(np.float32) if weights is None else np.asarray(weights, np.float32)
    res = torch.tensor(rs.standard_normal((T, ex.K)), dtype=torch.float32, device=DEV).to(U.TORCH_DT[ydt]) if residual else None
    y = U.guarded((T, ex.K), U.TORCH_DT[ydt], 7.0)
    ref_res = None if res is None else h64(res)
    if alias:
        y.t.copy_(res)
        res = y.t
    size = g.gguf_moe_ffn_workspace_size(ex.F, T, top_k)
    ws = U.workspace(size, 0xff)
    idt, wt = torch.tensor(ids, device=DEV), torch.tensor(weights, device=DEV)
    torch.cuda.synchronize()
    g.gguf_moe_ffn(ex.struct(gelu), x, U.DT[xdt], T, idt, wt, top_k, res, y.t, U.DT[ydt], ws.t, size, stream)
    assert g.gguf_mm_check_errors(stream) == 0
    y.check(), ws.check()
    return h64(x), ids, weights.astype(np.float64), ref_res, h64(y.t)


def check_ffn(ex, T, top_k, **kw):
    x, ids, weights, res, y = run_ffn(ex, T, top_k, **kw)
    gelu, ydt = kw.get("gelu", False), kw.get("ydt", "bf16")
    ref = S.moe_ffn(x, *ex.val, ids, weights, gelu, res)
    near(y, ref, ydt, ffn_bound(ex, x, ids, weights, gelu, ydt, res))


@pytest.mark.parametrize("t", list(FORMATS))
@pytest.mark.parametrize("xdt,ydt", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f16")])
def test_ffn_formats(t, xdt, ydt):
    K, F = (512, 768) if FORMATS[t] in (syn.Q2_K, syn.Q3_K, syn.Q4_K, syn.Q5_K, syn.Q6_K) else (416, 288)
    ex = Experts((t, t, t), K, F, 5, seed=1)
    check_ffn(ex, 3, 2, xdt=xdt, ydt=ydt, gelu=xdt == "f16", seed=2)
    check_ffn(ex, 1, 4, xdt=xdt, ydt=ydt, residual=False, seed=3)


@pytest.mark.parametrize("t", list(FORMATS))
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
def test_ffn_error_by_norm(t, xdt):
    """f32 outputs lie within 2**-20 of themselves by norm.  Some six stages round by at most 2**-22 of what they add up (an
    activation and a hidden value to two f16 parts, the products' alignment, the sums that mins meet, the two sums), which
    for codes centred by a min is about twice the values; apart from each other: 2**-22 * (6 * 2) ** 0.5 < 2**-20."""
    ex = Experts((t, t, t), 512, 512, 4, seed=20)
    x, ids, weights, _, y = run_ffn(ex, 4, 2, xdt=xdt, ydt="f32", residual=False, seed=21)
    ref = S.moe_ffn(x, *ex.val, ids, weights, False, None)
    assert np.linalg.norm(y - ref) <= 2.0 ** -20 * np.linalg.norm(ref)


@pytest.mark.parametrize("types", [("Q4_K", "Q4_K", "Q6_K"), ("Q8_0", "Q5_1", "Q4_0"), ("Q2_K", "Q6_K", "Q3_K"), ("Q5_K", "Q8_0", "Q5_0"),
                                   ("Q4_1", "Q3_K", "Q4_K"), ("Q4_0", "Q2_K", "Q4_1")])
def test_ffn_mixed_types(types):
    check_ffn(Experts(types, 512, 512, 6, seed=4), 5, 3, xdt="f32", ydt="f32", seed=5)


@pytest.mark.parametrize("K,F", [(32, 32), (64, 2080), (1056, 32), (288, 544)])
def test_ffn_sizes_of_32_value_blocks(K, F):
    ex = Experts(("Q8_0", "Q8_0", "Q5_1"), K, F, 3, seed=6)
    check_ffn(ex, 1, 1, xdt="f32", ydt="f32")
    check_ffn(ex, 9, 2, ydt="f32")


@pytest.mark.parametrize("T,top_k", [(1, 1), (1, 12), (2, 6), (8, 2), (9, 4), (33, 3), (64, 8), (512, 1), (128, 4)])
@pytest.mark.parametrize("xdt,ydt", [("bf16", "bf16"), ("f32", "f32")])
def test_ffn_rows(T, top_k, xdt, ydt):
    check_ffn(Experts(("Q4_K", "Q4_K", "Q4_K"), 256, 256, 12, seed=7), T, top_k, xdt=xdt, ydt=ydt, seed=T)


def test_ffn_every_row_at_one_expert():
    ex = Experts(("Q5_K", "Q5_K", "Q6_K"), 256, 512, 4, seed=8)
    check_ffn(ex, 50, 1, xdt="f32", ydt="f32", ids=np.full((50, 1), 2))
    check_ffn(ex, 50, 2, ids=np.tile([3, 3], (50, 1)))        # the same index twice: added twice


def test_ffn_many_experts_and_ids_of_none():
    ex = Experts(("Q8_0", "Q8_0", "Q8_0"), 64, 64, 300, seed=9)
    ids = np.random.default_rng(1).integers(0, 300, (40, 6))
    ids[3] = -1                 # a token without experts
    ids[7, 2], ids[8, 0], ids[9, 5] = 300, -2 ** 31, 2 ** 31 - 1
    check_ffn(ex, 40, 6, ydt="f32", ids=ids)
    check_ffn(ex, 40, 6, ydt="f32", ids=ids, residual=False)
    check_ffn(ex, 2, 3, ids=np.full((2, 3), 999))


@pytest.mark.parametrize("scale", [1e-15, 1e-6, 3e4, 1e15])
def test_ffn_activations_of_any_size(scale):
    ex = Experts(("Q4_K", "Q4_K", "Q4_K"), 512, 256, 3, seed=10)
    x = np.random.default_rng(2).standard_normal((3, 512)) * scale
    x[1, :256] *= 1e-12                                       # one chunk far below the other
    x[2, 5] = 100 * scale
    check_ffn(ex, 3, 2, xdt="f32", ydt="f32", x=x, residual=False, weights=np.full((3, 2), 1.0))


def test_ffn_values_that_are_not_finite_stay_in_their_rows():
    ex = Experts(("Q4_K", "Q4_K", "Q6_K"), 256, 256, 4, seed=11)
    x = np.random.default_rng(3).standard_normal((6, 256))
    clean = x.copy()
    x[1, 7], x[4, 200] = np.nan, np.inf
    ids = np.array([[0, 1], [0, 1], [1, 2], [0, 3], [0, 1], [2, 0]])
    w = np.full((6, 2), 0.5)
    got = run_ffn(ex, 6, 2, x=x, ids=ids, weights=w, residual=False)[4]
    want = run_ffn(ex, 6, 2, x=clean, ids=ids, weights=w, residual=False)[4]
    assert np.isnan(got[1]).all() and not np.isfinite(got[4]).any()
    keep = [0, 2, 3, 5]
    assert np.array_equal(got[keep], want[keep])


@pytest.mark.parametrize("types", [(t, t, t) for t in FORMATS] + [("Q4_K", "Q6_K", "Q5_0"), ("Q5_1", "Q8_0", "Q2_K")])
@pytest.mark.parametrize("xdt,ydt", [("bf16", "f32"), ("f32", "bf16")])
def test_ffn_many_rows_of_each_expert(types, xdt, ydt):
    """Two tiles of columns at a time, and what an expert's last group has left of them."""
    ex = Experts(types, 256, 256, 3, seed=17)
    for rows in ((93, 51, 6), (49, 48, 80)):
        ids = np.random.default_rng(18).permutation(np.repeat(np.arange(3), rows)).reshape(-1, 1)
        check_ffn(ex, len(ids), 1, xdt=xdt, ydt=ydt, ids=ids, seed=19)


@pytest.mark.parametrize("types,K,F,E,T,top_k", [
    (("Q4_K", "Q4_K", "Q4_K"), 16384, 256, 2, 3, 2),        # columns of all of K's chunks have no room
    (("Q6_K", "Q6_K", "Q6_K"), 16384, 256, 2, 20, 1),
    (("Q8_0", "Q8_0", "Q8_0"), 12832, 64, 2, 2, 1),
    (("Q5_K", "Q2_K", "Q3_K"), 13312, 256, 2, 9, 1),
    (("Q4_K", "Q4_K", "Q6_K"), 256, 16384, 2, 3, 1),        # many chunks of F
    (("Q8_0", "Q8_0", "Q8_0"), 64, 12832, 2, 17, 2),
    (("Q8_0", "Q4_0", "Q8_0"), 64, 64, 1024, 64, 8),        # as many experts and rows as there may be
    (("Q6_K", "Q6_K", "Q6_K"), 256, 256, 7, 256, 2),
    (("Q3_K", "Q3_K", "Q5_K"), 256, 512, 3, 1, 512),        # one token, experts many times over
    (("Q5_0", "Q5_0", "Q4_1"), 32, 32, 1, 512, 1),
])
@pytest.mark.parametrize("xdt,ydt", [("bf16", "bf16"), ("f32", "f32")])
def test_ffn_ends_of_the_ranges(types, K, F, E, T, top_k, xdt, ydt):
    ids = np.random.default_rng(E).integers(0, E, (T, top_k))
    check_ffn(Experts(types, K, F, E, seed=13), T, top_k, xdt=xdt, ydt=ydt, ids=ids, seed=14)


def test_ffn_weights_at_the_end_of_their_allocation():
    """Nothing past the last expert's bytes is read: what stands there does not matter, and they may end anywhere."""
    for t, K, F in (("Q6_K", 256, 256), ("Q5_0", 32, 96), ("Q3_K", 256, 512), ("Q8_0", 96, 32), ("Q4_0", 64, 32)):
        ex = Experts((t, t, t), K, F, 3, seed=15)
        for i in range(3):
            flat = ex.dev[i].reshape(-1)
            room = torch.full((flat.numel() + 64,), 0xff, dtype=torch.uint8, device=DEV)
            room[:flat.numel()] = flat
            ex.dev[i] = room[:flat.numel()]
        check_ffn(ex, 2, 2, xdt="f32", ydt="f32", seed=16)


def test_ffn_in_place_and_again():
    ex = Experts(("Q4_K", "Q4_K", "Q4_K"), 512, 512, 6, seed=12)
    a = run_ffn(ex, 17, 3, seed=1)[4]
    assert np.array_equal(a, run_ffn(ex, 17, 3, seed=1, alias=True)[4])
    assert np.array_equal(a, run_ffn(ex, 17, 3, seed=1)[4])


# ------------------------------------------------------------------ sampling

def run_sample(logits, sampler, u, vocab=None, logprob=True, stream=None):
    rows = logits.shape[0]
    token, lp = U.guarded((rows,), torch.int32, -7), U.guarded((rows,), torch.float32, -7.0)
    dt = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[logits.dtype]
    g.gguf_sample(logits, dt, logits.stride(0), rows, vocab or logits.shape[1], sampler, u, token.t, lp.t if logprob else None, stream)
    assert g.gguf_mm_check_errors(stream) == 0
    token.check(), lp.check()
    return token.t.cpu().numpy(), h64(lp.t)


def check_sample(logits, temp=None, top_k=None, top_p=None, min_p=None, u=None, vocab=None):
    rows, V = logits.shape[0], vocab or logits.shape[1]
    f32 = lambda a: None if a is None else torch.tensor(np.broadcast_to(a, (rows,)).copy(), dtype=torch.float32, device=DEV)      # noqa: E731
    t, p, m, uu = f32(temp), f32(top_p), f32(min_p), f32(u)
    k = None if top_k is None else torch.tensor(np.broadcast_to(top_k, (rows,)).copy(), dtype=torch.int32, device=DEV)
    token, lp = run_sample(logits, g.gguf_sampler(t, k, p, m), uu, V)
    x = h64(logits[:, :V])
    at = lambda a, r, none: none if a is None else float(a[r])      # noqa: E731
    for r in range(rows):
        want, wlp, n = S.sample(x[r], at(t, r, 1.0), 0 if k is None else int(k[r]), at(p, r, 1.0), at(m, r, 0.0), float(uu[r]))
        assert token[r] == want, (r, token[r], want, n, at(t, r, 1.0), k is not None and int(k[r]), at(p, r, 1.0), at(m, r, 0.0), float(uu[r]))
        if want < 0:
            assert np.isnan(lp[r])
        else:
            assert abs(lp[r] - wlp) <= 2.0 ** -21 * (1 + abs(wlp)), (r, lp[r], wlp)


def logits_of(rows, V, dt="f32", seed=0, spread=3.0, pad=0):
    rs = np.random.default_rng(seed)
    x = torch.tensor(rs.standard_normal((rows, V + pad)) * spread, dtype=torch.float32, device=DEV).to(U.TORCH_DT[dt])
    if pad:
        x[:, V:] = math.nan        # between the rows is anything
        x = x[:, :V]
    return x, rs


FILTERS = [dict(), dict(top_k=40), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=50, top_p=0.8, min_p=0.02), dict(top_k=2000, top_p=0.95),
           dict(temp=2.0, top_p=0.97), dict(temp=0.0), dict(temp=0.3, top_k=1), dict(top_p=0.0), dict(temp=5.0, top_k=300),
           dict(temp=3.0, top_p=0.5, min_p=0.001), dict(min_p=1.0), dict(top_k=10 ** 9, top_p=1.5, min_p=-1.0)]


@pytest.mark.parametrize("kw", FILTERS)
@pytest.mark.parametrize("V,dt,pad", [(1000, "f32", 0), (32003, "bf16", 5), (5001, "f16", 3), (40000, "f32", 1)])
def test_sample_filters(V, dt, pad, kw):
    x, rs = logits_of(6, V, dt, seed=V, pad=pad)
    check_sample(x, u=rs.random(6), **kw)


@pytest.mark.parametrize("V", [1, 2, 3, 4, 5, 127, 128, 129, 2045, 2046, 2047, 4096, 16381, 16384, 16385, 131072, 150001])
def test_sample_vocabularies(V):
    x, rs = logits_of(3, V, seed=V)
    check_sample(x, u=rs.random(3), temp=0.9, top_p=[0.95, 1.0, 0.5], top_k=[0, 20, 0])


@pytest.mark.parametrize("rows", [1, 2, 40, 200, 700])
def test_sample_rows_of_different_settings(rows):
    x, rs = logits_of(rows, 3001, "bf16", seed=rows)
    pick = lambda *a: rs.choice(a, rows)      # noqa: E731
    check_sample(x, temp=pick(0.0, 0.7, 1.0, 2.5), top_k=pick(0, 1, 10, 500), top_p=pick(0.3, 0.9, 1.0), min_p=pick(0.0, 0.01, 0.3), u=rs.random(rows))


@pytest.mark.parametrize("kw", [dict(), dict(top_k=700), dict(top_p=0.37), dict(top_k=900, top_p=0.61), dict(top_k=3), dict(top_p=0.01, top_k=600),
                                dict(min_p=0.5), dict(temp=0.0)])
@pytest.mark.parametrize("V", [1000, 20011])
def test_sample_ties_go_by_index(V, kw):
    rs = np.random.default_rng(6)
    u = rs.random(8)
    check_sample(torch.full((8, V), 2.5, device=DEV), u=u, **kw)                             # all equal
    few = torch.tensor(rs.integers(0, 4, (8, V)), dtype=torch.float32, device=DEV)          # thousands of each of four
    check_sample(few, u=u, **kw)
    check_sample(-few * 0.0, u=u, **kw)                                                      # zeros of both signs


def test_sample_given_numbers_at_their_ends():
    x, rs = logits_of(8, 700, seed=1)
    u = [0.0, 1 - 2.0 ** -24, 1.0, 7.0, -3.0, math.nan, 2.0 ** -149, 0.5]
    check_sample(x, u=u)
    check_sample(x, u=u, top_k=5)
    check_sample(x, u=u, top_p=0.99, temp=4.0)
    x[:, 650:] = -math.inf
    x[:, :3] = -math.inf
    check_sample(x, u=u)


def test_sample_settings_at_their_ends():
    x, rs = logits_of(10, 5000, seed=2)
    inf, nan = math.inf, math.nan
    check_sample(x, u=rs.random(10), temp=[inf, nan, -1.0, 1e-30, 1e-3, 1e30, 1e-45, 1.0, 1.0, -0.0])
    check_sample(x, u=rs.random(10), temp=[inf, inf, 1e-30, 1e-30, 1e-3, 1e30, 1e-45, 1.0, 1.0, 1e4], top_k=700, top_p=0.6)
    check_sample(x, u=rs.random(10), top_p=[nan, -1.0, 0.0, 1.0, 1 - 2.0 ** -24, 2.0 ** -149, inf, -inf, 0.5, 1e-10])
    check_sample(x, u=rs.random(10), min_p=[nan, -1.0, 0.0, 1.0, 2.0, 2.0 ** -149, inf, -inf, 1 - 2.0 ** -24, 1e-10])
    check_sample(x, u=rs.random(10), top_k=[-5, 0, 1, 2, 4999, 5000, 5001, 2 ** 31 - 1, -2 ** 31, 256])


def test_sample_masked_rows_and_rows_without_a_distribution():
    x, rs = logits_of(9, 3000, seed=3)
    x[0] = -math.inf
    x[1, 5] = math.nan
    x[2, 2999] = math.inf
    x[3] = -math.inf
    x[3, 1234] = -1e30                # one token left
    x[4, 100:] = -math.inf
    x[5] = torch.finfo(torch.float32).min        # masks of the type's lowest value, and nothing but
    x[6, ::2] = torch.finfo(torch.float32).min
    x[7, 1] = torch.finfo(torch.float32).max
    for kw in (dict(), dict(top_k=300), dict(top_p=0.9), dict(temp=0.0), dict(top_k=40, top_p=0.9, min_p=0.1), dict(temp=math.inf)):
        check_sample(x, u=rs.random(9), **kw)


def test_sample_does_not_depend_on_the_cut():
    """A row alone is spread over eight blocks, in a large batch over fewer: the tokens are the same."""
    x, rs = logits_of(300, 9000, seed=4)
    u = torch.tensor(rs.random(300), dtype=torch.float32, device=DEV)
    t = torch.full((300,), 1.7, device=DEV)
    p = torch.full((300,), 0.98, device=DEV)
    many, lp = run_sample(x, g.gguf_sampler(t, None, p), u)
    for r in (0, 7, 299):
        one, l1 = run_sample(x[r:r + 1], g.gguf_sampler(t, None, p), u[r:r + 1])
        assert one[0] == many[r] and l1[0] == lp[r]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_sample_top_p_of_masked_rows_at_any_temperature(dt):
    """What lies below top-p's bound is summed without being listed: masked tokens add nothing to it."""
    x, rs = logits_of(12, 6000, dt, seed=7)
    x[:, 1::3] = -math.inf
    x[6:, 2::3] = torch.finfo(x.dtype).min
    t = [math.inf, 1e30, 1e4, 1.0, 1e-3, 1e-30] * 2
    for p in (0.3, 0.9, 0.999):
        check_sample(x, u=rs.random(12), temp=t, top_p=p)
        check_sample(x, u=rs.random(12), temp=t, top_p=p, min_p=0.2)


def test_sample_top_p_does_not_depend_on_the_cut():
    rs = np.random.default_rng(8)
    x = torch.tensor(rs.standard_normal((400, 20000)) * 1.5, dtype=torch.float32, device=DEV)
    u = torch.tensor(rs.random(400), dtype=torch.float32, device=DEV)
    p = torch.tensor(rs.uniform(0.05, 0.95, 400), dtype=torch.float32, device=DEV)
    many, lp = run_sample(x, g.gguf_sampler(None, None, p), u)
    for r in range(0, 400, 7):
        one, l1 = run_sample(x[r:r + 1], g.gguf_sampler(None, None, p[r:r + 1]), u[r:r + 1])
        assert one[0] == many[r] and l1[0] == lp[r]


@pytest.mark.parametrize("kw", [dict(), dict(top_k=50), dict(top_k=100000, top_p=0.8), dict(top_p=0.9), dict(min_p=0.1)])
def test_sample_largest_vocabulary(kw):
    x, rs = logits_of(2, 1 << 22, "bf16", seed=9, spread=2.0)
    check_sample(x, u=rs.random(2), **kw)


def test_sample_draws_with_the_frequencies_asked_for():
    """The same row many times with numbers evenly spaced: each token comes as often as its share, to one."""
    V, n = 50, 4000
    x, _ = logits_of(1, V, seed=5, spread=1.0)
    u = torch.arange(n, dtype=torch.float32, device=DEV) / n
    token, lp = run_sample(x.expand(n, V).contiguous(), None, u)
    share = torch.softmax(x[0].double(), 0).cpu().numpy()
    assert np.abs(np.bincount(token, minlength=V) - n * share).max() <= 1.01
    assert np.allclose(np.exp(lp), share[token], rtol=1e-6)


def test_sample_without_logprob():
    x, rs = logits_of(2, 100, seed=6)
    token, lp = run_sample(x, None, torch.tensor([0.3, 0.6], device=DEV), logprob=False)
    assert (lp == -7.0).all() and (token >= 0).all()


# ------------------------------------------------------------------ streams, graphs, calls next to each other

class Work:
    """One call of each operator on fixed buffers."""

    def __init__(self, seed, T=5, ws=None):
        rs = np.random.default_rng(seed)
        f = lambda *s: torch.tensor(rs.standard_normal(s), dtype=torch.float32, device=DEV)      # noqa: E731
        self.case = Case([(T, 20)], 2, 64, "bf16", seed=seed)
        self.qkv = f(T, 8 * 64).bfloat16()
        self.turned = torch.empty((T, 4, 64), dtype=torch.bfloat16, device=DEV)
        self.norm, self.rope = g.gguf_head_norm(1 + f(64) / 8, 1 + f(64) / 8), g.gguf_rope(freqs_of(64), 64, 1)
        self.batch, self.cache = self.case.batch(), g.gguf_kv_cache(self.case.k, self.case.v)
        self.x, self.router = f(T, 512), g.gguf_router(f(9, 512) / 22, 3)
        self.ids, self.w = torch.empty((T, 3), dtype=torch.int32, device=DEV), torch.empty((T, 3), device=DEV)
        self.experts = Experts(("Q4_K", "Q4_K", "Q6_K"), 512, 256, 9, seed=seed)
        self.T, self.y = T, torch.empty((T, 512), device=DEV)
        self.size = g.gguf_moe_ffn_workspace_size(256, T, 3)
        self.ws = torch.empty(self.size, dtype=torch.uint8, device=DEV) if ws is None else ws
        self.logits, self.u = f(T, 9001) * 3, torch.tensor(rs.random(T), dtype=torch.float32, device=DEV)
        self.sampler = g.gguf_sampler(None, None, torch.full((T,), 0.9, device=DEV))
        self.token, self.lp = torch.empty(T, dtype=torch.int32, device=DEV), torch.empty(T, device=DEV)

    def run(self, stream=None):
        q, k, v = self.qkv.split((256, 128, 128), dim=1)
        g.gguf_kv_append_norm(q, 512, k, 512, v, 512, 2, 4, self.norm, self.rope, self.batch, self.cache, self.turned, 256, stream)
        g.gguf_moe_router(self.x, 0, self.T, 512, self.router, self.ids, self.w, stream)
        g.gguf_moe_ffn(self.experts.struct(), self.x, 0, self.T, self.ids, self.w, 3, None, self.y, 0, self.ws, self.size, stream)
        g.gguf_sample(self.logits, 0, 9001, self.T, 9001, self.sampler, self.u, self.token, self.lp, stream)

    def outputs(self):
        return [t.clone() for t in (self.turned, self.case.k, self.case.v, self.ids, self.w, self.y, self.token, self.lp)]

    def clear(self):
        for t in (self.turned, self.case.k, self.case.v, self.ids, self.w, self.y, self.token, self.lp, self.ws):
            t.fill_(1)


def expect(works):
    out = []
    for w in works:
        w.clear()
        w.run()
        out.append(w.outputs())
    torch.cuda.synchronize()
    assert g.gguf_mm_check_errors() == 0
    for w in works:
        w.clear()
    torch.cuda.synchronize()
    return out


def same(works, want):
    torch.cuda.synchronize()
    assert g.gguf_mm_check_errors() == 0
    assert all(torch.equal(a, b) for w, o in zip(works, want) for a, b in zip(w.outputs(), o))


def test_two_streams_at_once():
    works = [Work(1), Work(2, T=40)]
    want = expect(works)
    streams = [torch.cuda.Stream() for _ in works]
    for _ in range(20):
        for w, s in zip(works, streams):
            w.run(s)
    same(works, want)


def test_graphs_that_share_a_workspace():
    """Replayed one after the other on one stream, without anything in between."""
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    works = [Work(3, T=40, ws=ws), Work(4, T=1, ws=ws), Work(5, T=2, ws=ws)]
    want = expect(works)
    graphs = []
    for w in works:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w.run()
        graphs.append(graph)
    for _ in range(5):
        for graph in graphs:
            graph.replay()
    same(works, want)
    # new inputs in the captured buffers
    for w in works:
        w.x.mul_(-0.5), w.logits.neg_(), w.qkv.mul_(2)
    want = expect(works)
    for graph in graphs:
        graph.replay()
    same(works, want)


def test_calls_back_to_back_on_one_workspace():
    """A call's kernels may begin before the call ahead has ended: what they write and read of the workspace does not."""
    ws = torch.empty(1 << 21, dtype=torch.uint8, device=DEV)
    works = [Work(6 + i, T=t, ws=ws) for i, t in enumerate((1, 64, 3, 17, 1, 30))]
    want = expect(works)
    for _ in range(10):
        for w in works:
            w.run()
    same(works, want)
    for _ in range(10):                      # the experts' calls alone, next to each other
        for w in works:
            g.gguf_moe_ffn(w.experts.struct(), w.x, 0, w.T, w.ids, w.w, 3, None, w.y, 0, ws, w.size)
    same(works, want)
