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
