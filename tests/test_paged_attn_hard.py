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
