"""What the serving operators refuse, report and leave alone: the C entries'
refusals and the binding's own checks (CPU), and the device's reports (GPU)."""
import ctypes

import numpy as np
import pytest

import gguf_quant_weight_gb300 as g
from tests.test_serving_abi import batch, cache, lib  # noqa: F401

INV = g.GGUF_ERR_INVALID_ARG


# ------------------------------------------------------------------ in place

def test_append_in_place_wants_the_same_type_and_rows(lib):  # noqa: F811
    r = ctypes.byref
    c = cache()

    def call(ldo=256, ldq=256, xdt=2):
        return lib.gguf_kv_append(1024, ldq, 4096, 128, 8192, 128, xdt, 4, None, r(batch()), r(c), 1024, ldo, None)

    assert call(xdt=0) == INV and call(xdt=1) == INV          # f32 or f16 rows under bf16 ones
    assert call(ldo=264) == INV and call(ldq=264) == INV      # rows that overlap their neighbours


@pytest.mark.gpu
def test_one_row_in_place_may_name_any_stride():
    torch = pytest.importorskip("torch")
    from tests import gpu_util as U
    U.require_gpu()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn((1, 2, 64), device="cuda").bfloat16()
    keep, cache16 = x.clone(), torch.zeros((1, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    b = g.gguf_kv_batch(i32([0, 1]), i32([1]), i32([[0]]), 1, 1, 1)
    g.gguf_kv_append(x, 128, keep, 128, keep, 128, g.GGUF_DT_BF16, 2, None, b, g.gguf_kv_cache(cache16, torch.zeros_like(cache16)), x, 256)
    y = torch.randn((1, 100), device="cuda")
    was = y.clone()
    g.gguf_logits_adjust(y, g.GGUF_DT_F32, 104, 1, 100, g.gguf_logit_rules(), y, g.GGUF_DT_F32, 100)
    assert g.gguf_mm_check_errors() == 0
    assert torch.equal(x, keep) and torch.equal(cache16[0, :, 0], keep[0]) and torch.equal(y, was)


# ------------------------------------------------------------------ indexes on the device

@pytest.mark.gpu
@pytest.mark.parametrize("what,start,length,kw,good", [
    ("falling q_start", [0, 5, 3, 8], [9, 9, 9], {}, []),
    ("a falling pair of other sequences", [0, 2, 7, 6], [9, 9, 9], {}, []),
    ("negative q_start", [-2, 3, 4, 8], [9, 9, 9], {}, [1, 2]),
    ("q_start past the tokens", [0, 3, 4, 9], [9, 9, 9], {}, [0, 1]),
    ("more new tokens than stated", [0, 2, 3, 8], [9, 9, 9], dict(max_q_len=4), [0, 1]),
    ("more keys than stated", [0, 3, 4, 8], [9, 31, 9], dict(max_kv_len=30), [0, 2]),
    ("more keys than pages", [0, 3, 4, 8], [9, 33, 9], {}, [0, 2])])
def test_append_reports_arrays_out_of_range(what, start, length, kw, good):
    torch = pytest.importorskip("torch")
    from tests import gpu_util as U
    U.require_gpu()
    T, H, KV, D, page = 8, 2, 2, 64, 16
    rs = np.random.default_rng(1)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kc, vc = (U.guarded((6, KV, page, D), torch.bfloat16, 3.0) for _ in range(2))
    q, k, v = (torch.tensor(rs.standard_normal((T, h, D)), dtype=torch.bfloat16, device="cuda") for h in (H, KV, KV))
    out = U.guarded((T, H, D), torch.bfloat16, 3.0)
    pages = i32([[0, 1], [2, 3], [4, 5]])
    b = g.gguf_kv_batch(i32(start), i32(length), pages, T, kw.get("max_q_len", T), kw.get("max_kv_len", 32))
    g.gguf_kv_append(q, H * D, k, KV * D, v, KV * D, g.GGUF_DT_BF16, H, None, b, g.gguf_kv_cache(kc.t, vc.t), out.t, H * D)
    assert g.gguf_mm_check_errors() == INV, what
    assert g.gguf_mm_check_errors() == 0
    ko, vo, qo = (torch.full_like(x.t, 3.0) for x in (kc, vc, out))
    for s in good:
        for t in range(start[s], start[s + 1]):
            p = length[s] - start[s + 1] + t
            ko[int(pages[s, p // page]), :, p % page], vo[int(pages[s, p // page]), :, p % page], qo[t] = k[t], v[t], q[t]
    for got, want in ((kc, ko), (vc, vo), (out, qo)):
        got.check(what)
        assert torch.equal(got.t, want), what


# ------------------------------------------------------------------ the binding's structs

def test_batch_refuses_arrays_with_gaps():
    torch = pytest.importorskip("torch")
    i, pages = torch.zeros(6, dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int32)
    g.gguf_kv_batch(i[:3], i[:2], pages, 3, 1, 1)
    for a in ((i[::2], i[:2], pages), (i[:3], i[:4:2], pages), (i[:3].long(), i[:2], pages), (i[:3], i[:2].to(torch.uint8), pages),
              (i[:3], i[:2], pages.to(torch.int16)), (i[:3], i[:2], pages.T[:2])):
        with pytest.raises(ValueError):
            g.gguf_kv_batch(*a, 3, 1, 1)
    column = torch.zeros((1, 2), dtype=torch.int32).T        # one page a sequence: its stride says nothing
    assert g.gguf_kv_batch(i[:3], i[:2], column, 3, 1, 1).pages_stride == 1


def test_rope_refuses_other_types_and_gaps():
    torch = pytest.importorskip("torch")
    f = torch.zeros(64)
    p = torch.zeros(8, dtype=torch.int32)
    g.gguf_rope(f[:32], 64, positions=p)
    g.gguf_rope(f, 64)
    assert g.gguf_rope(16, 64).freqs == 16                    # a device address
    for a, kw in (((f.double(), 64), {}), ((f.half(), 64), {}), ((f[::2], 64), {}), ((f[:31], 64), {}),
                  ((f, 64), dict(positions=p.long())), ((f, 64), dict(positions=p[::2]))):
        with pytest.raises(ValueError):
            g.gguf_rope(*a, **kw)


def test_rules_refuse_other_types_and_gaps():
    torch = pytest.importorskip("torch")
    i, f, words = torch.zeros(8, dtype=torch.int32), torch.ones(8), torch.zeros((2, 8), dtype=torch.int32)
    good = dict(hist=i, hist_start=i[:3], repeat=f[:2], frequency=f[:2], presence=f[:2], bias_ids=i, bias=f, bias_start=i[:3],
                allow=words)
    assert g.gguf_logit_rules(**good).allow_stride == 8
    assert g.gguf_logit_rules(allow=words[:, :5]).allow_stride == 8
    g.gguf_logit_rules()
    for name in ("hist", "hist_start", "bias_ids", "bias_start"):
        for bad in (i.long(), torch.zeros(16, dtype=torch.int32)[::2], f):
            with pytest.raises(ValueError, match=name):
                g.gguf_logit_rules(**dict(good, **{name: bad}))
    for name in ("repeat", "frequency", "presence", "bias"):
        for bad in (f.double(), torch.ones(4)[::2], torch.ones(1).expand(2), f.bfloat16(), i):
            with pytest.raises(ValueError, match=name):
                g.gguf_logit_rules(**dict(good, **{name: bad}))
    for bad in (words.long(), words.T, words[0], words.bool()):
        with pytest.raises(ValueError, match="allow"):
            g.gguf_logit_rules(**dict(good, allow=bad))


def test_an_address_may_be_any_integer(lib):  # noqa: F811
    class Address(int):
        pass

    x = Address(4096)
    for call in (lambda: g.gguf_mm_gemv(x, 99, 0, 32, 32, x, 2, 1, None, x, 2, stream=Address(0)),
                 lambda: g.gguf_logits_adjust(x, 9, 8, 1, 8, g.gguf_logit_rules(repeat=x), x, 0, 8, Address(0))):
        with pytest.raises(g.GGUFError):
            call()


def test_logits_in_place_want_the_same_type_and_rows(lib):  # noqa: F811
    rules = g.gguf_logit_rules()

    def call(dt=0, odt=0, ld=104, ldo=104):
        return lib.gguf_logits_adjust(4096, dt, ld, 2, 100, ctypes.byref(rules), 4096, odt, ldo, None)

    assert call(dt=2) == INV and call(odt=1) == INV and call(ldo=100) == INV and call(ld=112) == INV
