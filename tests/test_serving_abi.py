"""CPU checks of the serving operators' C ABI: the host structs' layout and the
refusals that come before any device is asked for."""
import ctypes
import math

import pytest

import gguf_quant_weight_gb300 as g


@pytest.fixture(scope="module")
def lib():
    from gguf_quant_weight_gb300 import _build
    _build.build()
    return g.load_library()


def make(cls, **kw):
    s = cls.__new__(cls)
    ctypes.Structure.__init__(s)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def cache(**kw):
    a = dict(k=16, v=32, dtype=2, page_size=16, kv_heads=2, head_dim=64, n_pages=8, page_stride=2048, head_stride=1024,
             token_stride=64)
    a.update(kw)
    return make(g.gguf_kv_cache, **a)


def batch(**kw):
    a = dict(q_start=16, kv_len=16, pages=16, n_seq=2, n_tokens=4, pages_stride=4, max_q_len=2, max_kv_len=64)
    a.update(kw)
    return make(g.gguf_kv_batch, **a)


def rope(**kw):
    a = dict(freqs=16, positions=None, rot_dim=64, style=0, scale=1.0)
    a.update(kw)
    return make(g.gguf_rope, **a)


def test_struct_sizes_match_the_header():
    # five 4-byte and pointer-sized members laid out as the header's structs on a 64-bit machine
    assert ctypes.sizeof(g.gguf_kv_cache) == 64
    assert ctypes.sizeof(g.gguf_kv_batch) == 64
    assert ctypes.sizeof(g.gguf_rope) == 32
    assert ctypes.sizeof(g.gguf_logit_rules) == 80


INV, UNS, MIS, WS = -1, -2, -3, -4


@pytest.mark.parametrize("want,kw", [
    (INV, dict(k=None)), (INV, dict(n_pages=0)), (INV, dict(kv_heads=0)), (INV, dict(token_stride=-64)),
    (UNS, dict(dtype=0)), (UNS, dict(head_dim=136)), (UNS, dict(head_dim=72)), (UNS, dict(page_size=24)),
    (UNS, dict(page_size=8)), (UNS, dict(page_size=512)), (MIS, dict(v=40)), (MIS, dict(token_stride=68))])
def test_cache_refusals(lib, want, kw):
    c, b = cache(**kw), batch()
    r = ctypes.byref
    assert lib.gguf_kv_append(None, 0, 16, 128, 16, 128, 2, 0, None, r(b), r(c), None, 0, None) == want
    assert lib.gguf_paged_attn(16, 256, 4, r(b), r(c), 1.0, 1, 0, 16, 256, None, None, 0, None) == want
    assert lib.gguf_paged_attn_workspace_size(r(b), r(c), 4) == 0


@pytest.mark.parametrize("want,kw", [
    (INV, dict(q_start=None)), (INV, dict(n_seq=0)), (INV, dict(n_tokens=0)), (INV, dict(max_q_len=0)),
    (INV, dict(max_kv_len=65)), (INV, dict(max_kv_len=-1)), (UNS, dict(n_seq=1 << 16)), (UNS, dict(n_tokens=1 << 25)),
    (MIS, dict(pages=18))])
def test_batch_refusals(lib, want, kw):
    c, b = cache(), batch(**kw)
    r = ctypes.byref
    assert lib.gguf_kv_append(None, 0, 16, 128, 16, 128, 2, 0, None, r(b), r(c), None, 0, None) == want
    assert lib.gguf_paged_attn(16, 256, 4, r(b), r(c), 1.0, 1, 0, 16, 256, None, None, 0, None) == want


def test_append_refusals(lib):
    r = ctypes.byref
    c, b = cache(), batch()

    def call(q=16, ldq=256, k=16, ldk=128, v=16, ldv=128, xdt=2, heads=4, ro=None, out=16, ldo=256):
        return lib.gguf_kv_append(q, ldq, k, ldk, v, ldv, xdt, heads, r(ro) if ro else None, r(b), r(c), out, ldo, None)

    assert call(k=None) == INV and call(q=None) == INV and call(out=None) == INV
    assert call(heads=3) == INV and call(heads=0) == INV and call(ldq=255) == INV and call(ldk=127) == INV
    assert call(ldo=248) == INV
    assert call(xdt=9) == UNS
    assert call(q=24) == MIS and call(ldk=132) == MIS and call(ldo=260) == MIS
    assert call(xdt=0, ldq=258) == MIS
    for ro, want in ((rope(freqs=None), INV), (rope(rot_dim=0), INV), (rope(rot_dim=66), INV), (rope(rot_dim=33), INV),
                     (rope(style=2), INV), (rope(freqs=18), MIS), (rope(positions=17), MIS)):
        assert call(ro=ro) == want
    assert lib.gguf_kv_append(16, 256, 16, 128, 16, 128, 2, 4, None, None, r(c), 16, 256, None) == INV
    assert lib.gguf_kv_append(16, 256, 16, 128, 16, 128, 2, 4, None, r(b), None, 16, 256, None) == INV


def test_attention_refusals(lib):
    r = ctypes.byref
    c, b = cache(), batch()

    def call(q=16, ldq=256, heads=4, scale=0.125, causal=1, window=0, out=16, ldo=256, lse=None):
        return lib.gguf_paged_attn(q, ldq, heads, r(b), r(c), scale, causal, window, out, ldo, lse, None, 0, None)

    assert call(q=None) == INV and call(out=None) == INV and call(heads=5) == INV and call(heads=0) == INV
    assert call(heads=2 * 129, ldq=2 * 129 * 64, ldo=2 * 129 * 64) == UNS
    for s in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=s) == INV
    assert call(window=-1) == INV and call(causal=2) == INV and call(ldq=248) == INV
    assert call(ldq=260) == MIS and call(out=20) == MIS and call(lse=18) == MIS


def test_logits_refusals(lib):
    r = ctypes.byref

    def call(x=16, dt=0, ld=100, rows=2, vocab=100, out=16, odt=0, ldo=100, **kw):
        rules = make(g.gguf_logit_rules, **kw)
        return lib.gguf_logits_adjust(x, dt, ld, rows, vocab, r(rules), out, odt, ldo, None)

    assert call(x=None) == INV and call(out=None) == INV and call(rows=0) == INV and call(vocab=0) == INV
    assert call(ld=99) == INV and call(ldo=99) == INV and call(hist=16) == INV and call(bias_ids=16, bias=16) == INV
    assert call(allow=16, allow_stride=3) == INV
    assert call(dt=5) == UNS and call(odt=5) == UNS and call(rows=1 << 16) == UNS
    assert call(x=20) == MIS and call(out=4) == MIS and call(hist=16, hist_start=18) == MIS
    assert lib.gguf_logits_adjust(16, 0, 100, 2, 100, None, 16, 0, 100, None) == INV


def test_python_structs_refuse_what_they_cannot_describe():
    torch = pytest.importorskip("torch")
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        g.gguf_kv_cache(k, torch.zeros((4, 2, 16, 32), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        g.gguf_kv_cache(k.transpose(2, 3), k.transpose(2, 3))
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        g.gguf_kv_batch(i, i, torch.zeros((3, 2), dtype=torch.int32), 3, 1, 1)
    with pytest.raises(ValueError):
        g.gguf_kv_batch(i, i[:2], torch.zeros((2, 2), dtype=torch.int64), 3, 1, 1)
    nhd = torch.zeros((4, 16, 2, 64), dtype=torch.float16).transpose(1, 2)
    c = g.gguf_kv_cache(nhd, nhd)
    assert (c.page_size, c.kv_heads, c.head_dim, c.n_pages, c.dtype) == (16, 2, 64, 4, g.GGUF_DT_F16)
    assert (c.page_stride, c.head_stride, c.token_stride) == (2048, 64, 128)
