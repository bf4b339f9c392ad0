"""The sampler, the router and the normed append where their arithmetic is at its ends, against the 64-bit definitions in
oracle/serving_oracle.py.

Which tokens top-p keeps shows in what u just below 1 draws where the likely tokens come first in the vocabulary and in
falling order: the last one kept.  top_p is put next to a border between two sets, `gap` of the whole sum away from it, and
rounded to f32, by 2**-25 of the sum at most; the expected token is that of the rounded number.
"""
import math

import numpy as np
import pytest
import torch

import gguf_quant_weight_gb300 as g
from oracle import serving_oracle as S
from tests import gpu_util as U
from tests.test_decode_operators import check_sample, h64, run_sample
from tests.test_serving import Case, near

pytestmark = pytest.mark.gpu
DEV = "cuda"
LAST = 1 - 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    U.require_gpu()


# ------------------------------------------------------------------ top-p: what lies far below the border

def next_to_a_border(x, temp, j, gap):
    """The top_p, as f32, `gap` of the sum beyond the weight of the first j tokens of the falling row x."""
    w = np.exp((x.astype(np.float64) - float(x.max())) / temp)
    return np.float32((np.sort(w)[::-1][:j].sum() + gap * w.sum()) / w.sum())


@pytest.mark.parametrize("V", [131072, 262144, 1 << 20, 1 << 22])
def test_sample_top_p_counts_a_flat_rest(V):
    """Ten equal tokens over a flat rest of some percent, which no single token of shows."""
    x = np.full(V, -15.388, np.float32)
    at = np.sort(np.random.default_rng(V).permutation(V)[:10])
    x[at] = 0
    rest = (V - 10) * math.exp(-15.388)
    x = torch.tensor(x, device=DEV).expand(3, V).contiguous()
    check_sample(x, top_p=5.01 / (10 + rest), u=[0.07, 0.5, 0.9])       # six are kept, and five without the rest


def test_sample_top_p_counts_a_flat_rest_of_two_tokens():
    x = np.full(131072, -15.3, np.float32)
    x[:2] = 0, -0.034
    u = (np.arange(16) + 0.5) / 16
    check_sample(torch.tensor(x, device=DEV).expand(16, -1).contiguous(), top_p=0.505, u=u)


@pytest.mark.parametrize("V,rows,dt", [(131072, 40, "f32"), (131071, 12, "bf16"), (262144, 12, "f32"), (1 << 20, 5, "f16"), (1 << 22, 3, "f32")])
def test_sample_top_p_over_a_bulk_far_below(V, rows, dt):
    """A few dozen likely tokens over a bulk 15 to 20 nats lower.  The rest's weights are f32 numbers of arguments z (in bits)
    with two roundings, up to 2**-23 z ln 2 + 2**-22 of themselves, below 4e-6 for z <= 45; the rest is a tenth of the sum at
    most, so a gap of 1e-6 of the sum is further than what it may be off by."""
    rs = np.random.default_rng(V)
    x = np.empty((rows, V), np.float32)
    temp, p = rs.choice([0.5, 1.0, 2.0], rows), np.empty(rows, np.float32)
    for r in range(rows):
        n = int(rs.integers(20, 60))
        x[r] = (rs.standard_normal(V) * rs.uniform(0.2, 0.8) - rs.uniform(15, 20)) * temp[r]
        x[r, :n] = np.sort(rs.standard_normal(n) * 0.8)[::-1] * temp[r]
    x = torch.tensor(x, device=DEV).to(U.TORCH_DT[dt])
    host = x.float().cpu().numpy()
    for r in range(rows):
        w = np.exp((host[r].astype(np.float64) - host[r].max()) / temp[r])
        assert 1e-7 < np.sort(w)[:-60].sum() / w.sum() < 0.1
        p[r] = next_to_a_border(host[r], temp[r], int(rs.integers(3, 18)), float(rs.choice([-1e-6, 1e-6])))
    check_sample(x, temp=temp, top_p=p, u=np.full(rows, LAST))


@pytest.mark.parametrize("depth", [15.0, 15.4])
def test_sample_top_p_where_one_cut_overflows_its_lists(depth):
    """A thousand neighbours near the top: more than a warp lists where few blocks share a row, and not where many do."""
    rs = np.random.default_rng(5)
    V, rows = 32003, 200
    x = np.full((rows, V), -depth, np.float32)
    x[:, :1000] = np.linspace(0, -0.02, 1000)
    p = np.array([next_to_a_border(x[r], 1.0, int(rs.integers(100, 900)), float(rs.choice([-1e-6, 1e-6]))) for r in range(rows)])
    x = torch.tensor(x, device=DEV)
    f = lambda a: torch.tensor(a, dtype=torch.float32, device=DEV)      # noqa: E731
    u = np.full(rows, LAST)
    many, lp = run_sample(x, g.gguf_sampler(None, None, f(p)), f(u))
    for r in range(0, rows, 9):
        one, l1 = run_sample(x[r:r + 1].clone(), g.gguf_sampler(None, None, f(p[r:r + 1])), f(u[r:r + 1]))
        assert one[0] == many[r] and l1[0] == lp[r]
    keep = slice(0, 30)
    check_sample(x[keep].contiguous(), top_p=p[keep], u=u[keep])
    want = [S.sample(x[r].double().cpu().numpy(), 1.0, 0, float(np.float32(p[r])), 0.0, float(u[r]))[0] for r in range(0, rows, 10)]
    assert np.array_equal(many[::10], want)


# ------------------------------------------------------------------ top-p: weights at the edges of a bin

@pytest.mark.parametrize("share", [0.0099, 0.05, 0.1, 0.2, 0.3, 0.5, 0.8])
@pytest.mark.parametrize("n", [100, 299, 1500])
def test_sample_top_p_between_the_edges_of_two_bins(share, n):
    """The likely tokens at the far edge of the first sixteenth of a bit, the others at the near edge of the next: counted by
    sixteenths, the first look heavier than they are and the others lighter.  One of the others is kept."""
    others = int(n / share)
    x = np.empty(1 + n + others, np.float32)
    x[0], x[1:n + 1], x[n + 1:] = 0, -0.99995 / 16 * math.log(2), -1.00005 / 16 * math.log(2)
    p = next_to_a_border(x, 1.0, 1 + n, 1e-6)
    check_sample(torch.tensor(x, device=DEV)[None].contiguous(), top_p=p, u=[LAST])


def test_sample_top_p_at_the_edge_of_a_bin_in_a_long_row():
    x = np.empty(101002, np.float32)
    x[0], x[1:1001], x[1001:] = 0, -0.99995 / 16 * math.log(2), -1.00005 / 16 * math.log(2)
    check_sample(torch.tensor(x, device=DEV)[None].contiguous(), top_p=0.009914, u=[LAST])


# ------------------------------------------------------------------ weights at the end of their integers

@pytest.mark.parametrize("V", [1 << 20, 1 << 22])
@pytest.mark.parametrize("kw", [dict(), dict(top_p=0.9999), dict(top_k=1000), dict(min_p=1e-13)])
def test_sample_tokens_at_the_last_bits(V, kw):
    """Tokens 40 to 47 bits below the largest, where integers of so large a vocabulary end."""
    x = -torch.linspace(40, 47, V, device=DEV) * math.log(2)
    x[V // 3] = 0
    check_sample(x.expand(2, V).contiguous(), u=[0.0, 0.99999], **kw)


# ------------------------------------------------------------------ router: weights of small scores

def router_of(z):
    """A router and a token whose scores are z, exactly (multiples of 1/64 below 2**10, each from one product)."""
    z = np.asarray(z, np.float64)
    assert np.array_equal(z, np.round(z * 64) / 64) and np.abs(z).max() < 1024
    w = np.zeros((len(z), 8), np.float32)
    w[np.arange(len(z)), 0] = z
    x = torch.zeros((1, 8), device=DEV)
    x[0, 0] = 1
    return x, torch.tensor(w, device=DEV)


def check_exact_scores(z, top_k, sigmoid, bias, renorm, scale=1.0):
    """Scores are exact here, so weights are off by two exponentials (2 units of 2**-23 each), a sum of top_k (or of all
    experts) positive terms, a quotient and two products: 2**-19 of themselves; 8 of
    the smallest f32 where exponentials (2 of them, times scale) and quotients are subnormal."""
    x, w = router_of(z)
    b = None if bias is None else torch.tensor(np.asarray(bias), dtype=torch.float32, device=DEV)
    ids, weights = torch.empty((1, top_k), dtype=torch.int32, device=DEV), torch.empty((1, top_k), device=DEV)
    g.gguf_moe_router(x, 0, 1, 8, g.gguf_router(w, top_k, int(sigmoid), b, renorm, scale), ids, weights)
    assert g.gguf_mm_check_errors() == 0
    ri, rw = S.router(x.double().cpu().numpy(), w.double().cpu().numpy(), None if b is None else b.double().cpu().numpy(), top_k,
                      sigmoid, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), ri)
    got = weights.double().cpu().numpy()
    assert np.all(np.abs(got - rw) <= 2.0 ** -19 * np.abs(rw) + 2.0 ** -146), (got, rw)


def scores(n, at, spread, seed):
    return at + np.round(np.random.default_rng(seed).uniform(-spread, spread, n) * 64) / 64


@pytest.mark.parametrize("at", [-60, -87, -88, -95, -103, -200, -690])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_sigmoids_of_very_negative_scores(at, biased, renorm):
    z = scores(40, at, 5, 1)
    check_exact_scores(z, 6, True, np.random.default_rng(2).standard_normal(40) if biased else None, renorm, 2.5)


@pytest.mark.parametrize("above", [20, 87, 95, 104, 150, 600])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_softmax_beside_an_expert_that_is_shut_out(above, renorm):
    """The softmax goes over all experts, the weights' sum over the chosen: a shut-out expert far above leaves them their digits."""
    z, b = scores(30, 0, 3, 3), np.zeros(30)
    z[7], b[7] = above, -math.inf
    check_exact_scores(z, 5, False, b, renorm)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_router_weights_of_scores_far_apart(sigmoid):
    for at in (-150, -40, 0, 40):
        z = scores(24, at, 3, 4)
        z[::5] -= 30
        b = np.random.default_rng(6).standard_normal(24)
        for bias in (None, b):
            check_exact_scores(z, 24, sigmoid, bias, True)


# ------------------------------------------------------------------ router: the order of small scores

@pytest.mark.parametrize("power", [-60, -80, -90])
@pytest.mark.parametrize("side", ["x", "w"])
def test_router_orders_small_scores_that_f32_cannot_tell(power, side):
    """Families of copies whose values differ in their last bits, of activations or weights whose squares f32 does not hold."""
    rs = np.random.default_rng(7)
    x, w = rs.standard_normal((20, 2048)).astype(np.float32), (rs.standard_normal((64, 2048)) / 45).astype(np.float32)
    for e in range(16, 64):
        w[e] = w[e % 16] * (1 + rs.integers(-2, 3, 2048) * 2.0 ** -23)
    x, w = (x * np.float32(2.0 ** power), w) if side == "x" else (x, w * np.float32(2.0 ** power))
    ids, weights = torch.empty((20, 12), dtype=torch.int32, device=DEV), torch.empty((20, 12), device=DEV)
    g.gguf_moe_router(torch.tensor(x, device=DEV), 0, 20, 2048, g.gguf_router(torch.tensor(w, device=DEV), 12), ids, weights)
    ri, _ = S.router(x.astype(np.float64), w.astype(np.float64), None, 12, False, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), ri)


# ------------------------------------------------------------------ normed append: angles

@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("freqs", ["rope", "near 1", "large"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_append_norm_far_and_given_positions(style, freqs, dt):
    """Angles are good to 2**-24 of a turn, 2 pi 2**-24, twice where f64 takes over, cos and sin to 2 units of 2**-23 and the turn
    to 3 roundings; the norm of 16 values to (16 / 2 + 4) * 2**-24: below 32 * 2**-24 of |a| + |b| <= 2 max |x|."""
    rs = np.random.default_rng(8)
    D, heads, KV = 16, 24, 8
    f = {"rope": 10000.0 ** (-np.arange(8) / 8), "near 1": 1 - np.arange(8) / 77, "large": np.geomspace(3, 100, 8)}[freqs].astype(np.float32)
    lowest = -2 ** 31
    at = np.array([0, 1, -1, 2 ** 24 - 1, 2 ** 24, 2 ** 24 + 1, 1 - 2 ** 24, -2 ** 24, -2 ** 24 - 1, lowest, lowest + 1, 2 ** 31 - 1,
                   9999999, -9999999, 123456789, 4095, 131071, 1048575, -7, 16000001], np.int32)
    if freqs == "large":        # of farther ones f64 keeps too few digits
        at = np.clip(at, -2 ** 24 - 1, 2 ** 24 + 1)
    T = len(at)
    c = Case([(T, T)], KV, D, dt, seed=1)
    q, k, v = (c.values((T, h, D), "f32") for h in (heads, KV, KV))
    wq, wk = (torch.tensor(1 + 0.3 * rs.standard_normal(D), dtype=torch.float32, device=DEV) for _ in range(2))
    out = torch.empty((T, heads, D), dtype=U.TORCH_DT[dt], device=DEV)
    kc, vc = h64(c.k), h64(c.v)
    rope = g.gguf_rope(torch.tensor(f, device=DEV), D, style, 1.0, torch.tensor(at, device=DEV))
    g.gguf_kv_append_norm(q, heads * D, k, KV * D, v, KV * D, 0, heads, g.gguf_head_norm(wq, wk), rope, c.batch(),
                          g.gguf_kv_cache(c.k, c.v), out, heads * D)
    assert g.gguf_mm_check_errors() == 0
    nq, nk = S.head_norm(h64(q), h64(wq), 1e-6), S.head_norm(h64(k), h64(wk), 1e-6)
    qo, kc, vc = S.append(nq, nk, h64(v), f, D, style, 1.0, c.q_start, c.kv_len, c.pages, kc, vc, at)
    u = 32 * 2.0 ** -24 * 2
    near(h64(out), qo, dt, u * np.abs(nq).max(-1, keepdims=True), "q")
    near(h64(c.k), kc, dt, u * np.abs(nk).max(), "k")
    near(h64(c.v), vc, dt, 0.0, "v")
