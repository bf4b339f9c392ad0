"""Paged attention on the GPU where its kernels have most to get right: maxima
that rise with every tile, values that are not finite, weights of every size,
and calls cut into many shares.  Tolerances are those derived in
tests/test_serving.py unless a test derives its own."""
import math

import numpy as np
import pytest
import torch

import gguf_quant_weight_gb300 as g
from oracle import serving_oracle as S
from tests import gpu_util as U
from tests.test_serving import Case, check_attn, near, run_attn

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    U.require_gpu()


def poison(c):
    """NaN and infinities in every slot that holds no key (as Case.poison, at once)."""
    held = np.zeros((c.n_pages, c.page), bool)
    for b, length in enumerate(c.kv_len):
        t = np.arange(length)
        page = c.pages[b, t // c.page]
        held[page[page >= 0], (t % c.page)[page >= 0]] = True
    junk = torch.tensor([math.nan, math.inf, -math.inf, 6e4] * (c.dim // 4), device=DEV)
    keep = torch.tensor(held, device=DEV)[:, None, :, None]
    for x in (c.k, c.v):
        x.copy_(torch.where(keep, x.float(), junk).to(x.dtype))


@pytest.mark.parametrize("dt,dim", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 48)])
@pytest.mark.parametrize("seqs,group", [([(700, 700)], 2), ([(130, 900), (300, 301)], 5), ([(40, 1500)], 1)])
def test_maximum_rises_with_every_tile(dt, dim, seqs, group):
    # scores grow by more than 2^8 from one tile of keys to the next, so the sums are rescaled at each
    c = Case(seqs, 2, dim, dt, page=32, seed=dim + group)
    q = c.values((c.n_tokens, 2 * group, dim)).abs() + 0.5
    for b, length in enumerate(c.kv_len):
        for t in range(length):
            at = int(c.pages[b, t // c.page]), slice(None), t % c.page
            c.k[at] = (c.k[at].float() * 0.05 + 8.0 * t / 128 / dim ** 0.5).to(c.k.dtype)
    first, lse = check_attn(c, group, q=q)
    for _ in range(20):
        again, l2 = run_attn(c, q)
        assert torch.equal(first, again) and torch.equal(lse, l2)


# ------------------------------------------------------------------ values that are not finite

# Bounds that make calls of these few sequences large ones, whose keys are dealt out
# to all warps (a page table of LARGE pages of 16).
LARGE = 20000


def run_in(c, form, group, causal=1, window=0, q=None):
    """Runs c in the form that its bounds give: "cluster", "dealt" (the keys dealt out to all warps) or "many" rows, and
    checks that it was that one: only dealt-out keys leave their places in the line in the workspace."""
    rows = c.max_q * group
    assert (rows > 16) == (form == "many")
    kw = dict(max_kv_len=16 * LARGE) if form == "dealt" else {}
    batch = c.batch(**kw)
    H = group * c.kv_heads
    n = g.gguf_paged_attn_workspace_size(batch, g.gguf_kv_cache(c.k, c.v), H)
    if form != "many":
        assert (n > 0) == (form == "dealt"), "another form than the test means to run"
    return run_attn(c, c.values((c.n_tokens, H, c.dim)) if q is None else q, causal, window, **kw)


# One sequence is short enough for one worker; of the other every worker has a part.
@pytest.mark.parametrize("dt,dim", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("form,group,seqs", [
    ("cluster", 4, [(1, 1), (1, 700), (1, 16)]), ("cluster", 8, [(2, 33), (1, 1)]), ("cluster", 1, [(3, 3), (9, 40)]),
    ("dealt", 4, [(1, 1), (1, 900), (1, 16)]), ("dealt", 8, [(2, 500), (1, 1)]), ("dealt", 1, [(3, 3), (9, 3000)]),
    ("many", 8, [(3, 3), (5, 600)]), ("many", 8, [(1, 1), (9, 2000)])])
def test_nan_query_makes_its_rows_nan(dt, dim, form, group, seqs):
    c = Case(seqs, 2, dim, dt, page=16, seed=dim + group, wide=LARGE if form == "dealt" else None)
    c.poison()
    q = c.values((c.n_tokens, 2 * group, dim))
    clean, clean_lse = run_in(c, form, group, q=q)
    assert torch.isfinite(clean).all() and torch.isfinite(clean_lse).all()
    for t in range(c.n_tokens):
        bad = q.clone()
        bad[t, 1, 3] = math.nan
        out, lse = run_in(c, form, group, q=bad)
        assert torch.isnan(out[t, 1]).all() and torch.isnan(lse[t, 1]), t
        out[t, 1], lse[t, 1] = clean[t, 1], clean_lse[t, 1]
        assert torch.equal(out, clean) and torch.equal(lse, clean_lse), "another row changed"


@pytest.mark.parametrize("dt,dim", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("form,group,n", [("cluster", 4, 1), ("cluster", 8, 2), ("dealt", 4, 1), ("dealt", 8, 2), ("many", 8, 4)])
@pytest.mark.parametrize("length,where", [(1, 0), (17, 16), (33, 32), (1601, 1600), (1601, 0), (1601, 800), (129, 128), (300, 256)])
def test_nan_key_makes_the_rows_that_see_it_nan(dt, dim, form, group, n, length, where):
    # the only seen key of a worker's share among them: position 16 k as the last key
    c = Case([(n, length), (n, length)], 2, dim, dt, page=16, seed=where, wide=LARGE if form == "dealt" else None)
    c.poison()
    q = c.values((2 * n, 2 * group, dim))
    clean, clean_lse = run_in(c, form, group, q=q)
    c.k[int(c.pages[0, where // 16]), 0, where % 16] = math.nan
    out, lse = run_in(c, form, group, q=q)
    for j in range(n):
        if length - n + j >= where:
            assert torch.isnan(out[j, :group]).all() and torch.isnan(lse[j, :group]).all()
            out[j, :group], lse[j, :group] = clean[j, :group], clean_lse[j, :group]
    assert torch.equal(out.nan_to_num(7.0), clean.nan_to_num(7.0)) and torch.equal(lse, clean_lse), "another row changed"


@pytest.mark.parametrize("dt,dim", [("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("group,n,length", [(16, 62, 1908), (3, 100, 6000), (1, 300, 7000), (7, 90, 2700)])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_bad_key_before_keys_that_a_row_does_not_see(dt, dim, group, n, length, what):
    # Split keys: a share whose first tile of keys makes a row NaN and whose next holds keys of later tokens alone.
    KV = 8
    c = Case([(n, length)], KV, dim, dt, page=64, seed=group)
    poison(c)
    q = c.values((n, KV * group, dim)).abs() + 0.5          # so that a key of infinities scores infinity
    clean, clean_lse = run_in(c, "many", group, q=q)
    splits = g.gguf_paged_attn_workspace_size(c.batch(), g.gguf_kv_cache(c.k, c.v), KV * group) / (n * KV * group * (4 * dim + 8))
    assert 2 <= splits <= length / 128 / 1.9, "shares of at least two tiles are meant"
    for at in list(range(length - n - 3, length, 9)) + [length // 128 * 128 - 1, length - 1, 0]:
        where = int(c.pages[0, at // 64]), slice(None), at % 64
        keep = c.k[where].clone()
        c.k[where] = what
        out, lse = run_in(c, "many", group, q=q)
        c.k[where] = keep
        sees = torch.arange(length - n, length, device=DEV) >= at
        assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all(), at
        assert torch.equal(out[~sees], clean[~sees]) and torch.equal(lse[~sees], clean_lse[~sees]), at


# ------------------------------------------------------------------ weights of every size

@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("form,group,n", [("cluster", 4, 1), ("cluster", 8, 2), ("dealt", 2, 1), ("dealt", 16, 1), ("many", 20, 1),
                                          ("many", 1, 40)])
@pytest.mark.parametrize("first", [True, False])
def test_many_small_weights_beside_one_dominant_key(dt, form, group, n, first):
    # One key at weight 1 (the first, or the last before the new tokens) and 131072 at 2^-23 .. 2^-28, which are
    # together a few thousandths of the row: all of the output is theirs, and all of it of one sign.  Bounds:
    #   * a weight is rounded to within u of itself, which moves the output by u times itself; an f16 below what
    #     the lifted type holds whole, by 2^-25 of the lift instead: 2^-40 a key (2^-32 with many rows);
    #   * a weight's own error is e as in tests/test_serving.py, so the output's is 2 e of it;
    #   * a lane adds the weights of at most 512 keys to its sum, one after the other, each to within 2^-24 of it.
    N = 131073 + n
    c = Case([(n, N)], 1, 64, dt, page=64, seed=group, wide=16 * LARGE // 64 if form == "dealt" else None)
    q = c.values((n, group, 64))
    q[..., 0] = 8.0
    low = torch.tensor(c.rs.uniform(-19.4, -16.0, N), dtype=torch.float32)
    low[0 if first else N - n - 1] = 0.0
    pages = torch.tensor(c.pages[0, :-(-N // 64)].astype(np.int64), device=DEV)
    flat = torch.zeros((len(pages) * 64, 64), device=DEV)
    flat[:N, 0] = low.to(DEV)
    values = torch.ones_like(flat) + 0.5 * torch.rand(flat.shape, device=DEV)
    values[0 if first else N - n - 1] = 0.0
    for cache, x in ((c.k, flat), (c.v, values)):
        cache[pages, 0] = x.reshape(len(pages), 64, 64).to(cache.dtype)
    out, lse = run_in(c, form, group, q=q)
    ref, rlse, vmax, smax = S.attention(U.host64(q), U.host64(c.k), U.host64(c.v), c.q_start, c.kv_len, c.pages, 0.125, 1, 0)
    u = 2.0 ** -8 if dt == "bf16" else 2.0 ** -11
    e = 2.0 ** -23 * 16 * smax + 2.0 ** -20
    assert 1e-3 < np.abs(ref).max() < 1e-1
    sums = 512 * 2.0 ** -24
    small = 0.0 if dt == "bf16" else N * (2.0 ** -32 if form == "many" else 2.0 ** -40)
    near(U.host64(out), ref, dt, (u + 2 * e + sums)[..., None] * np.abs(ref) + small * vmax[..., None], "out")
    near(lse.cpu().numpy(), rlse, "f32", e + sums, "lse")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_small_weights_in_rows_of_one_share(dt):
    # the same in the many-rows form with its keys in one piece, as so many heads leave them: fewer keys, larger values
    N, n, KV = 2001, 40, 160
    c = Case([(n, N)], KV, 64, dt, page=32, seed=30)
    q = c.values((n, KV, 64))
    q[..., 0] = 8.0
    c.k.zero_()
    low = torch.tensor(c.rs.uniform(-19.4, -16.0, N), dtype=torch.float32)
    low[0] = 0.0
    c.v.copy_(100.0 + 50.0 * torch.rand(c.v.shape, device=DEV))
    t = np.arange(N)
    pages, slots = (torch.tensor(x.astype(np.int64), device=DEV) for x in (c.pages[0, t // 32], t % 32))
    c.k[pages, :, slots, 0] = low.to(DEV, c.k.dtype)[:, None]
    c.v[int(c.pages[0, 0]), :, 0] = 0.0
    out, lse = run_in(c, "many", 1, q=q)
    assert g.gguf_paged_attn_workspace_size(c.batch(), g.gguf_kv_cache(c.k, c.v), KV) == 0, "the keys were split"
    ref, rlse, vmax, smax = S.attention(U.host64(q), U.host64(c.k), U.host64(c.v), c.q_start, c.kv_len, c.pages, 0.125, 1, 0)
    u = 2.0 ** -8 if dt == "bf16" else 2.0 ** -11
    e = 2.0 ** -23 * 16 * smax + 2.0 ** -20
    sums = 32 * 2.0 ** -24         # two chains of 32 weights to a tile, and a tile at a time
    small = 0.0 if dt == "bf16" else N * 2.0 ** -32
    near(U.host64(out), ref, dt, (u + 2 * e + sums)[..., None] * np.abs(ref) + small * vmax[..., None], "out")
    near(lse.cpu().numpy(), rlse, "f32", e + sums, "lse")


# ------------------------------------------------------------------ each form at the shapes that it has most to do with

def check_form(c, form, group, causal=1, window=0, q=None):
    """check_attn on bounds as they are, in the form that is meant: "cluster", "dealt", "many", "split" (many rows with
    split keys) or "mixed" (sequences of few rows beside others).  Dealt-out keys leave the line's beginnings in the
    workspace, and split ones their partial rows; the other forms ask for none.  (A window can make a call a small one
    whatever its workspace, so what was written is looked at.)"""
    H, D = group * c.kv_heads, c.dim
    batch, cache = c.batch(), g.gguf_kv_cache(c.k, c.v)
    rows = c.max_q * group
    assert (rows > 16) == (form in ("many", "split", "mixed"))
    if form == "mixed":
        n = np.diff(c.q_start)
        assert group <= 16 and len(n) > 1 and ((n > 0) & (n * group <= 16)).any()
    q = c.values((c.n_tokens, H, D)) if q is None else q
    poison(c)
    n = g.gguf_paged_attn_workspace_size(batch, cache, H)
    ws, out, lse = U.workspace(n, 0xFF), U.guarded((c.n_tokens, H, D), U.TORCH_DT[c.dt], 3.0), U.guarded((c.n_tokens, H), torch.float32, 3.0)
    g.gguf_paged_attn(q, q.stride(0), H, batch, cache, D ** -0.5, causal, window, out.t, H * D, lse.t, ws.t, n)
    torch.cuda.synchronize()
    for b in (out, lse, ws):
        b.check("attention")
    assert g.gguf_mm_check_errors() == 0
    assert bool((ws.t != 0xFF).any()) == (form in ("dealt", "split")), "another form than the test means to run"
    ref, rlse, vmax, smax = S.attention(U.host64(q)[:c.rows], U.host64(c.k), U.host64(c.v), c.q_start, c.kv_len, c.pages, D ** -0.5,
                                        causal, window)
    u = 2.0 ** -8 if c.dt == "bf16" else 2.0 ** -11
    e = 2.0 ** -23 * max(1, D / 4) * smax + 2.0 ** -20
    got = U.host64(out.t)
    near(got[:c.rows], ref, c.dt, ((u + 2 * e) * vmax)[..., None], "out")
    assert np.all(got[c.rows:] == 3.0), "rows of no sequence were written"
    near(lse.t.cpu().numpy()[:c.rows], rlse, "f32", e, "lse")


def window_batch(n, window):
    """Sequences shorter and longer than the window, `n` new tokens in most; the pages before some windows are gone."""
    seqs = [(n if i % 7 else 1, 1 + 211 * i % 1900) for i in range(300)]
    seqs[5], seqs[8] = (0, 40), (n, 0)
    gone = [max(0, (b - a - window + 1) // 16) if i % 3 else 0 for i, (a, b) in enumerate(seqs)]
    return seqs, gone


@pytest.mark.parametrize("dt,dim", [("bf16", 64), ("f16", 128), ("bf16", 48)])
@pytest.mark.parametrize("group,n,window", [(1, 1, 700), (4, 1, 501), (3, 5, 640), (16, 1, 700), (2, 8, 513)])
def test_keys_dealt_out_under_a_causal_window(dt, dim, group, n, window):
    # 300 sequences of two key heads whose windows hold 32 to 44 chunks of 16 keys: over 19000 chunks, where every
    # item begins at its own first key
    seqs, gone = window_batch(n, window)
    check_form(Case(seqs, 2, dim, dt, page=16, seed=window + n, first_page=gone, extra_rows=2), "dealt", group, 1, window)


@pytest.mark.parametrize("window", [1, 16, 100])
def test_a_small_window_takes_clusters_whatever_the_lengths(window):
    seqs, gone = window_batch(2, window)
    check_form(Case(seqs, 2, 64, "bf16", page=16, seed=window, first_page=gone), "cluster", 4, 1, window)


@pytest.mark.parametrize("dt,dim", [("bf16", 32), ("f16", 48), ("bf16", 112), ("f16", 128)])
@pytest.mark.parametrize("form,group,seqs,window", [
    ("dealt", 4, [(1, 3000 + 97 * i) for i in range(48)], 0), ("dealt", 8, [(2, 2900 + 61 * i) for i in range(50)], 0),
    ("dealt", 4, [(1, 3000 + 97 * i) for i in range(60)], 2400), ("cluster", 5, [(3, 17 * i) for i in range(20)], 0),
    ("many", 3, [(90, 100 + i) for i in range(80)], 0), ("mixed", 3, [(90 if i % 2 else 4, 100 + i) for i in range(80)], 50)])
def test_head_sizes(dt, dim, form, group, seqs, window):
    check_form(Case(seqs, 2, dim, dt, page=32, seed=dim), form, group, 1, window)


@pytest.mark.parametrize("dt,dim", [("bf16", 128), ("f16", 64), ("bf16", 80)])
@pytest.mark.parametrize("group,seqs,window", [
    (20, [(1, 9000)], 0), (32, [(1, 5000), (1, 70)], 0), (128, [(1, 3333)], 0), (64, [(2, 2000), (0, 3), (1, 0)], 1111),
    (24, [(1, 4000), (3, 4001)], 600), (9, [(2, 6000)], 0)])
def test_many_heads_to_a_key_head_over_long_histories(dt, dim, group, seqs, window):
    check_form(Case(seqs, 1, dim, dt, page=64, seed=group), "split", group, 1, window)


@pytest.mark.parametrize("dt,dim", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("window", [0, 4500])
def test_single_tokens_with_long_histories_beside_chunks(dt, dim, window):
    # the few-rows sequences' keys are split over clusters of several blocks; 160 pieces of the chunks leave none of
    # their keys to be split
    seqs = [(200, 6000), (1, 9000), (1, 5000), (2, 100), (1, 1), (8, 7001), (9, 4100)]
    check_form(Case(seqs, 8, dim, dt, page=64, seed=dim + window), "mixed", 2, 1, window)


# ------------------------------------------------------------------ counts that pass 32 bits

def test_a_sequence_of_more_chunks_than_31_bits():
    # 2^26 + 16 keys (a table that names three pages over and over) of 512 key heads: 2^31 + 512 chunks of 16 keys.
    # All scores are 0 and the values 0 or 1, so that the sums are whole numbers: a worker's stay below 2^24, and
    # what joins rounds a few of them to f32.
    KV, D, page, N = 512, 16, 256, (1 << 26) + 16
    rs = np.random.default_rng(31)
    k = torch.tensor(rs.standard_normal((3, KV, page, D)), dtype=torch.bfloat16, device=DEV)
    v = torch.tensor(rs.integers(0, 2, (3, KV, page, D)), dtype=torch.bfloat16, device=DEV)
    table = rs.integers(0, 3, -(-N // page)).astype(np.int32)
    i32 = lambda a: torch.tensor(np.asarray(a, np.int32), device=DEV)  # noqa: E731
    batch, cache = g.gguf_kv_batch(i32([0, 1]), i32([N]), i32(table[None]), 1, 1, N), g.gguf_kv_cache(k, v)
    n = g.gguf_paged_attn_workspace_size(batch, cache, KV)
    q, ws = torch.zeros((1, KV, D), dtype=torch.bfloat16, device=DEV), U.workspace(n, 0xFF)
    out, lse = U.guarded((1, KV, D), torch.bfloat16, 3.0), U.guarded((1, KV), torch.float32, 3.0)
    g.gguf_paged_attn(q, KV * D, KV, batch, cache, 0.25, 1, 0, out.t, KV * D, lse.t, ws.t, n)
    torch.cuda.synchronize()
    for b in (out, lse, ws):
        b.check("attention")
    assert g.gguf_mm_check_errors() == 0
    times = np.bincount(table[:-1], minlength=3).astype(np.float64)
    v64 = U.host64(v)
    ref = (times[:, None, None] * v64.sum(2)).sum(0) + v64[table[-1], :, :N % page].sum(1)
    near(U.host64(out.t)[0], ref / N, "bf16", 2.0 ** -20, "out")
    near(lse.t.cpu().numpy()[0], np.full(KV, math.log(N)), "f32", 2.0 ** -19, "lse")


# ------------------------------------------------------------------ values of keys that only some rows see

@pytest.mark.parametrize("dt,dim", [("bf16", 128), ("f16", 64), ("bf16", 80)])
@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("form,group,n,length,window", [
    ("cluster", 4, 3, 40, 0), ("cluster", 1, 7, 300, 0), ("cluster", 1, 16, 16, 5), ("cluster", 2, 8, 70, 20),
    ("dealt", 4, 4, 900, 0), ("dealt", 1, 8, 500, 0), ("many", 1, 40, 40, 0), ("many", 3, 300, 300, 0),
    ("many", 2, 200, 2000, 0), ("many", 5, 150, 700, 100), ("many", 40, 30, 1000, 7)])
def test_a_value_that_is_not_finite_reaches_only_rows_that_see_its_key(dt, dim, what, form, group, n, length, window):
    # Rows share their tiles of keys: a row's weight of 0 for a key that only others see must not meet what stands there.
    c = Case([(n, length), (1, 20)], 2, dim, dt, page=16, seed=n + dim, wide=LARGE if form == "dealt" else None)
    c.poison()
    q = c.values((c.n_tokens, 2 * group, dim))
    clean, clean_lse = run_in(c, form, group, 1, window, q)
    ref, _, vmax, smax = S.attention(U.host64(q), U.host64(c.k), U.host64(c.v), c.q_start, c.kv_len, c.pages, dim ** -0.5, 1, window)
    u = 2.0 ** -8 if dt == "bf16" else 2.0 ** -11
    e = 2.0 ** -23 * max(1, dim / 4) * smax + 2.0 ** -20
    p = np.arange(length - n, length)
    for at, d in ((length - 1, 5), (length - 1 - n // 2, dim - 1), (length - n + 1, slice(None)), (length - n - 3, 17)):
        if at < 0:
            continue
        where = int(c.pages[0, at // 16]), 1, at % 16, d
        keep = c.v[where].clone()
        c.v[where] = what
        out, lse = run_in(c, form, group, 1, window, q)
        c.v[where] = keep
        assert torch.equal(lse, clean_lse)
        assert torch.equal(out[n:], clean[n:]) and torch.equal(out[:n, :group], clean[:n, :group]), "another head or sequence"
        sees = (p >= at) & (not window or at > p - window)
        got = U.host64(out)[:n, group:]
        assert not np.isfinite(got[sees][..., d]).any(), at
        near(got[~sees], ref[:n, group:][~sees], dt, ((u + 2 * e) * vmax)[:n, group:][~sees][..., None], "rows that do not see it")
        others = np.ones(dim, bool)
        others[d] = False
        near(got[sees][..., others], ref[:n, group:][sees][..., others], dt, ((u + 2 * e) * vmax)[:n, group:][sees][..., None], "others")
