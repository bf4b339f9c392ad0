"""CPU checks of the normed append's, the router's, the experts' and the sampler's
C ABI: the host structs' layout, and the refusals that come before any device
is asked for."""
import ctypes
import math

import pytest

import gguf_quant_weight_gb300 as g
from tests.test_serving_abi import batch, cache, lib, make, rope  # noqa: F401

INV, UNS, MIS, WS = -1, -2, -3, -4
r = ctypes.byref


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(g.gguf_head_norm) == 24
    assert ctypes.sizeof(g.gguf_router) == 40
    assert ctypes.sizeof(g.gguf_moe_weights) == 64
    assert ctypes.sizeof(g.gguf_sampler) == 32


def norm(**kw):
    return make(g.gguf_head_norm, **dict(dict(q=16, k=16, eps=1e-6), **kw))


def test_append_norm_refusals(lib):  # noqa: F811
    c, b = cache(), batch()

    def call(n=None, q=16, ldq=256, k=16, ldk=128, xdt=2, heads=4, ro=None, out=16, ldo=256):
        n = norm() if n is None else n
        return lib.gguf_kv_append_norm(q, ldq, k, ldk, 16, 128, xdt, heads, r(n) if n else None, r(ro) if ro else None, r(b), r(c),
                                       out, ldo, None)

    assert call(n=0) == INV
    for eps in (-1e-9, math.inf, math.nan, -math.inf):
        assert call(n=norm(eps=eps)) == INV
    assert call(n=norm(q=18)) == MIS and call(n=norm(k=17)) == MIS
    # and what the append without norms refuses
    assert call(k=None) == INV and call(q=None) == INV and call(heads=3) == INV and call(ldq=255) == INV
    assert call(xdt=9) == UNS and call(q=24) == MIS and call(ro=rope(rot_dim=66)) == INV
    assert call(q=4096, out=4096, xdt=1) == INV and call(q=4096, out=4096, ldo=264) == INV


def router(**kw):
    return make(g.gguf_router, **dict(dict(w=16, bias=None, wdt=0, n_expert=8, top_k=2, score=0, renormalize=1, scale=1.0), **kw))


def test_router_refusals(lib):  # noqa: F811
    def call(ro=None, x=16, xdt=2, T=1, K=64, ids=16, weights=16):
        return lib.gguf_moe_router(x, xdt, T, K, r(ro or router()), ids, weights, None)

    assert call(x=None) == INV and call(ids=None) == INV and call(weights=None) == INV and call(T=0) == INV and call(K=0) == INV
    assert lib.gguf_moe_router(16, 2, 1, 64, None, 16, 16, None) == INV
    for kw in (dict(w=None), dict(n_expert=0), dict(top_k=0), dict(top_k=9), dict(score=2), dict(renormalize=2), dict(scale=math.nan),
               dict(scale=math.inf)):
        assert call(router(**kw)) == INV, kw
    for kw in (dict(wdt=3), dict(n_expert=1025), dict(n_expert=128, top_k=65)):
        assert call(router(**kw)) == UNS, kw
    assert call(xdt=7) == UNS and call(K=60) == UNS and call(K=1 << 21) == UNS and call(T=1 << 25) == UNS
    assert call(x=24) == MIS and call(router(w=8)) == MIS and call(router(bias=18)) == MIS and call(ids=18) == MIS and call(weights=17) == MIS


def experts(**kw):
    a = dict(gate=16, up=16, down=16, gate_type=12, up_type=12, down_type=14, act=0, n_expert=4, K=256, F=512)
    return make(g.gguf_moe_weights, **dict(a, **kw))


def test_ffn_refusals(lib):  # noqa: F811
    def call(m=None, x=16, xdt=2, T=2, ids=16, weights=16, top_k=2, res=None, y=1 << 40, ydt=2, ws=16, size=1 << 20):
        return lib.gguf_moe_ffn(r(m or experts()), x, xdt, T, ids, weights, top_k, res, y, ydt, ws, size, None)

    assert lib.gguf_moe_ffn(None, 16, 2, 1, 16, 16, 1, None, 16, 2, 16, 1 << 20, None) == INV
    for kw in (dict(x=None), dict(ids=None), dict(weights=None), dict(y=None), dict(T=0), dict(top_k=0)):
        assert call(**kw) == INV, kw
    for kw in (dict(gate=None), dict(up=None), dict(down=None), dict(n_expert=0), dict(K=0), dict(F=0), dict(act=2), dict(K=128), dict(F=100),
               dict(K=264), dict(F=544)):
        assert call(experts(**kw)) == INV, kw
    for kw in (dict(gate_type=0), dict(up_type=9), dict(down_type=15), dict(n_expert=1025), dict(K=1 << 21), dict(F=1 << 21)):
        assert call(experts(**kw), size=1 << 40) == UNS, kw
    assert call(xdt=5) == UNS and call(ydt=5) == UNS and call(T=513, top_k=1) == UNS and call(T=257) == UNS and call(T=1, top_k=513) == UNS
    assert call(T=2 ** 62, top_k=4) == UNS
    for kw in (dict(x=24), dict(res=8), dict(y=4), dict(ws=8), dict(ids=18), dict(weights=17)):
        assert call(**kw) == MIS, kw
    for name in ("gate", "up", "down"):
        assert call(experts(**{name: 24})) == MIS
    # y may be the residual itself, and overlaps neither it in part nor x (2 rows of 256 bf16 values: 1024 bytes)
    assert call(y=16) == INV and call(y=16 + 1008) == INV and call(x=2048, y=16, ydt=0) == INV
    assert call(res=(1 << 40) - 1008) == INV and call(res=(1 << 40) + 16) == INV
    assert call(y=16 + 1024, ws=None) == WS and call(res=1 << 40, ws=None) == WS and call(res=(1 << 40) + 1024, ws=None) == WS
    assert call(ws=None) == WS and call(size=g.gguf_moe_ffn_workspace_size(512, 2, 2) - 1) == WS


def test_ffn_workspace_size(lib):  # noqa: F811
    size = g.gguf_moe_ffn_workspace_size
    # at least the hidden values in f32 and, as two f16 parts, as columns; and little else
    for F, T, k in ((512, 2, 2), (32, 512, 1), (1 << 20, 1, 512), (4096, 64, 8)):
        assert 8 * F * T * k <= size(F, T, k) <= 8 * 1.2 * max(F, 256) * T * k + 20 * T * k + 512
    assert [size(*a) for a in ((0, 1, 1), (512, 0, 1), (512, 1, 0), (512, 513, 1), (512, 2 ** 62, 4), (1 << 21, 1, 1), (-5, 1, 1))] == [0] * 7


def test_sample_refusals(lib):  # noqa: F811
    def call(x=16, dt=0, ld=100, rows=2, vocab=100, u=16, token=16, lp=None, **kw):
        return lib.gguf_sample(x, dt, ld, rows, vocab, r(make(g.gguf_sampler, **kw)), u, token, lp, None)

    assert call(x=None) == INV and call(u=None) == INV and call(token=None) == INV and call(rows=0) == INV and call(vocab=0) == INV
    assert call(ld=99) == INV
    assert call(dt=3) == UNS and call(rows=1 << 16) == UNS and call(vocab=(1 << 22) + 1, ld=1 << 23) == UNS and call(ld=1 << 39) == UNS
    assert call(x=24) == MIS and call(u=18) == MIS and call(token=18) == MIS and call(lp=17) == MIS
    for name in ("temperature", "top_k", "top_p", "min_p"):
        assert call(**{name: 18}) == MIS
    assert lib.gguf_sample(16, 3, 100, 2, 100, None, 16, 16, None, None) == UNS


def test_python_structs_refuse_other_types_and_gaps():
    torch = pytest.importorskip("torch")
    f, i = torch.ones(8), torch.zeros(8, dtype=torch.int32)
    for bad in (f.double(), f.half(), torch.ones(16)[::2], i):
        for make_it in (lambda: g.gguf_head_norm(bad, None), lambda: g.gguf_head_norm(None, bad), lambda: g.gguf_sampler(temperature=bad),
                        lambda: g.gguf_sampler(top_p=bad), lambda: g.gguf_sampler(min_p=bad), lambda: g.gguf_router(torch.ones((8, 16)), 2, bias=bad)):
            with pytest.raises(ValueError):
                make_it()
    for bad in (i.long(), torch.zeros(16, dtype=torch.int32)[::2], f):
        with pytest.raises(ValueError):
            g.gguf_sampler(top_k=bad)
    w = torch.ones((8, 16))
    assert g.gguf_router(w.bfloat16(), 2, bias=f).wdt == g.GGUF_DT_BF16
    for bad in (w.double(), w.T, w[:, ::2], w[0]):
        with pytest.raises(ValueError):
            g.gguf_router(bad, 2)
    with pytest.raises(ValueError):
        g.gguf_router(w, 2, bias=f[:7])
    b = torch.zeros(4 * 512 * 144, dtype=torch.uint8)
    kinds = (g.GGUF_Q4_K,) * 3
    assert g.gguf_moe_weights(b, b, b.clone(), *kinds, 256, 512, 4).n_expert == 4
    for a in ((b[:-1], b, b), (b, b[::2], b), (b, b, b.to(torch.int8)), (b, b, b[: 4 * 144])):
        with pytest.raises(ValueError):
            g.gguf_moe_weights(*a, *kinds, 256, 512, 4)
