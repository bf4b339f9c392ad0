"""The operators of a decode step together, as the example calls them: normed
append, attention, router, experts, sampling.  Each step's values are held to
the 64-bit definitions on what that step had, and a captured step draws what an
eager one does."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

from oracle import gguf_oracle as O
from oracle import serving_oracle as S
from tests import gpu_util as U
from tests.test_decode_operators import ffn_bound
from tests.test_serving import near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    U.require_gpu()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("moe_decode_step", os.path.join(root, "examples", "moe_decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = m
    spec.loader.exec_module(m)
    return m


def h64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Values:
    """The experts' values, and the magnitudes their products are made of (Q4_K: the scaled code's and the min's)."""

    def __init__(self, ex, layer):
        self.E, self.K, self.F = ex.EXPERTS, ex.HIDDEN, ex.INNER
        self.val, self.mag = [], []
        for b, qt, (n, k) in zip(layer.blocks, layer.types, ((self.F, self.K), (self.F, self.K), (self.K, self.F))):
            b = b.cpu().numpy().reshape(self.E * n, -1)
            val = O.dequant(b, qt, self.E * n, k)
            mag = np.abs(val)
            if qt == layer.types[0]:
                rest = b.copy().reshape(-1, 144)
                rest[:, 2:4] = 0
                rest = O.dequant(rest.reshape(b.shape), qt, self.E * n, k)
                mag = np.abs(rest) + np.abs(val - rest)
            self.val.append(val.reshape(self.E, n, k))
            self.mag.append(mag.reshape(self.E, n, k))


def test_captured_steps_draw_what_eager_ones_do(ex):
    eager = ex.generate(7, graph=False)
    assert eager.shape == (3, 7) and bool((eager % 2 == 0).all()) and bool((eager >= 0).all()) and bool((eager < ex.VOCAB).all())
    assert len(set(eager.flatten().tolist())) > 7
    assert torch.equal(eager, ex.generate(7, graph=True))


def test_prompts_of_many_pieces(ex):
    made = ex.generate(3, prompts=(300, 1, 170))
    assert bool((made >= 0).all()) and bool((made % 2 == 0).all())


def test_each_operator_of_each_step(ex):
    steps = []
    values = {}

    def watch(layer, seen, start, kv_len, pages):
        T = len(seen["x"])
        rows = lambda t, h: h64(t).reshape(T, h, ex.DIM)      # noqa: E731
        # append: this step's keys as the cache now has them
        norm = layer.head_norm
        wq, wk = (h64(w) for w in norm._keep)
        nq, nk = S.head_norm(rows(seen["q"], ex.HEADS), wq, norm.eps), S.head_norm(rows(seen["k"], ex.KV_HEADS), wk, norm.eps)
        kc, vc = h64(layer.k), h64(layer.v)
        f = (10000.0 ** (-2 * torch.arange(ex.DIM // 2, dtype=torch.float64) / ex.DIM)).float().numpy()
        want = S.append(nq, nk, rows(seen["v"], ex.KV_HEADS), f, ex.DIM, 1, 1.0, start.cpu().numpy(), kv_len.cpu().numpy(), pages.cpu().numpy(),
                        kc, vc)
        # a head's sum of 64 squares, root, products and turn: (64 / 2 + 12) half units of up to twice the largest
        u = (ex.DIM / 2 + 12) * 2.0 ** -24 * 2
        near(rows(seen["turned"], ex.HEADS), want[0], "bf16", u * np.abs(nq).max(), "q")
        near(kc, want[1], "bf16", u * np.abs(nk).max(), "k")
        near(vc, want[2], "bf16", 0.0, "v")
        # router: ids are those of 64 bits
        h, ids, weights = seen["routed"]
        w = h64(layer.router._keep[0])
        ri, rw = S.router(h64(h), w, None, ex.TOP_K, False, True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), ri)
        e = (ex.HIDDEN + 8) * 2.0 ** -24 * (np.abs(h64(h)) @ np.abs(w).T).max(-1, keepdims=True)
        assert np.all(np.abs(h64(weights) - rw) <= (4 * e + 2.0 ** -20) * rw)
        # experts, on the ids and weights that the router gave
        if not values:
            values["ex"] = Values(ex, layer)
        ref = S.moe_ffn(h64(h), *values["ex"].val, ri, h64(weights), False, h64(seen["x"]))
        near(h64(seen["y"]), ref, "bf16", ffn_bound(values["ex"], h64(h), ri, h64(weights), False, "bf16", h64(seen["x"])))
        # sampling
        for r in range(len(kv_len)):
            t, lp, _ = S.sample(h64(seen["logits"])[r], np.float32(0.8), 50, np.float32(0.95), np.float32(0.02), float(steps_u[len(steps)][r]))
            assert int(seen["token"][r]) == t and abs(float(seen["logprob"][r]) - lp) <= 2.0 ** -21 * (1 + abs(lp))
        steps.append(1)

    n, prompts = 4, (5, 40, 1)
    gen = torch.Generator().manual_seed(0)
    torch.randint(0, ex.VOCAB, (sum(prompts),), generator=gen)
    steps_u = torch.rand((n, 3), generator=gen).numpy()
    ex.generate(n, prompts, graph=False, watch=watch)
    assert len(steps) == n
