"""The decode example: its calls run together, its rules hold, and a prompt fills
the cache alike whether it comes at once or in chunks."""
import pytest
import torch

from tests import gpu_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    U.require_gpu()
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_generates_allowed_tokens_without_errors(ex):
    made = ex.generate(6)
    assert made.shape == (3, 6) and bool((made % 2 == 0).all()) and bool((made >= 0).all()) and bool((made < ex.VOCAB).all())
    assert not bool((made == 0).any())          # token 0 carries a bias of -100
    assert len({tuple(r) for r in made.tolist()}) == 3 and len(set(made.flatten().tolist())) > 6    # not one token all over
    assert torch.equal(made, ex.generate(6))


def test_chunks_of_a_prompt_fill_the_cache_alike(ex):
    import gguf_quant_weight_gb300 as g
    n = 40
    tokens = torch.randint(0, ex.VOCAB, (n,), generator=torch.Generator().manual_seed(3)).to("cuda")
    rules = g.gguf_logit_rules()
    pages = torch.arange(2, dtype=torch.int32, device="cuda").reshape(1, 2)
    last = []
    caches = []
    for parts in ([40], [17, 22, 1], [8] * 5):
        layer = ex.Layer(2)
        at = 0
        for m in parts:
            at += m
            kv_len = torch.tensor([at], dtype=torch.int32, device="cuda")
            logits = ex.step(layer, tokens[at - m:at], [m], kv_len, pages, 64, rules)
        last.append(logits)
        caches.append((layer.k.float(), layer.v.float()))
    # the projections take other paths for few rows (int8 activations), so the keys agree to that rounding
    for k, v in caches[1:]:
        for a, b in ((k, caches[0][0]), (v, caches[0][1])):
            assert (a - b).norm() < 0.02 * b.norm()
    for x in last[1:]:
        assert (x - last[0]).norm() < 0.05 * last[0].norm()
