"""Python binding of libgguf_mm.so (matmul on GGUF block-quantized weights, GB300).

Argument marshalling only: every function has the name and the arguments of
the C entry point in include/gguf_mm.h.  Tensor arguments may be torch tensors
(their data_ptr() is passed) or raw integer device addresses; `stream` defaults
to torch's current CUDA stream.  A non-zero status raises GGUFError.  There is
no fallback: if the library is missing the import of a function fails loudly.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgguf_mm.so")

# enums (same values as include/gguf_mm.h)
GGUF_Q4_0, GGUF_Q4_1, GGUF_Q5_0, GGUF_Q5_1 = 2, 3, 6, 7
GGUF_Q8_0, GGUF_Q4_K, GGUF_Q5_K, GGUF_Q6_K = 8, 12, 13, 14
GGUF_Q2_K, GGUF_Q3_K = 10, 11
GGUF_LAYOUT_BLOCKS, GGUF_LAYOUT_Q6K_PLANES = 0, 1
GGUF_DT_F32, GGUF_DT_F16, GGUF_DT_BF16 = 0, 1, 2
GGUF_PATH_AUTO, GGUF_PATH_GEMV, GGUF_PATH_FUSED = 0, 1, 2
GGUF_OP_GEMV, GGUF_OP_GEMM, GGUF_OP_ID, GGUF_OP_DENSE = 0, 1, 2, 3
GGUF_OK = 0
GGUF_ERR_INVALID_ARG, GGUF_ERR_UNSUPPORTED, GGUF_ERR_MISALIGNED = -1, -2, -3
GGUF_ERR_WORKSPACE, GGUF_ERR_CUDA, GGUF_ERR_TIMEOUT, GGUF_ERR_NO_DEVICE = -4, -5, -6, -7
GGUF_ERR_IO, GGUF_ERR_FORMAT, GGUF_ERR_NOT_FOUND = -8, -9, -10

BLOCK_VALUES = {GGUF_Q4_0: 32, GGUF_Q4_1: 32, GGUF_Q5_0: 32, GGUF_Q5_1: 32, GGUF_Q8_0: 32, GGUF_Q2_K: 256,
                GGUF_Q3_K: 256, GGUF_Q4_K: 256, GGUF_Q5_K: 256, GGUF_Q6_K: 256}
BLOCK_BYTES = {GGUF_Q4_0: 18, GGUF_Q4_1: 20, GGUF_Q5_0: 22, GGUF_Q5_1: 24, GGUF_Q8_0: 34, GGUF_Q2_K: 84,
               GGUF_Q3_K: 110, GGUF_Q4_K: 144, GGUF_Q5_K: 176, GGUF_Q6_K: 210}

_c_i64, _c_int, _c_sz, _c_vp = ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p

# name -> (restype, argtypes); mirrors include/gguf_mm.h
_SIGS = {
    "gguf_mm_workspace_size": (_c_sz, [_c_int, _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64]),
    "gguf_mm_gemv": (_c_int, [_c_vp, _c_int, _c_int, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_vp, _c_vp,
                              _c_int, _c_vp, _c_sz, _c_vp]),
    "gguf_mm_gemv_host": (_c_int, [_c_vp, _c_int, _c_int, _c_i64, _c_i64, _c_vp, _c_vp, _c_int, _c_i64, _c_vp,
                                   _c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_sz, _c_vp]),
    "gguf_mm_gemm": (_c_int, [_c_vp, _c_int, _c_int, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_vp, _c_vp,
                              _c_int, _c_vp, _c_sz, _c_int, _c_vp]),
    "gguf_mm_id": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_vp, _c_i64,
                            _c_vp, _c_vp, _c_int, _c_vp, _c_sz, _c_vp]),
    "gguf_mm_id_slots": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_vp, _c_i64,
                                  _c_vp, _c_vp, _c_int, _c_vp, _c_sz, _c_vp]),
    "gguf_mm_id_form": (_c_int, [_c_int, _c_i64, _c_i64]),
    "gguf_mm_id_path": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_vp, _c_i64,
                                 _c_int, _c_vp, _c_vp, _c_int, _c_vp, _c_sz, _c_int, _c_vp]),
    "gguf_repack_q6k_planes": (_c_int, [_c_vp, _c_vp, _c_i64, _c_int, _c_vp]),
    "gguf_dequant_padded": (_c_int, [_c_vp, _c_int, _c_int, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_vp]),
    "gguf_dense_gemm": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_vp, _c_vp,
                                 _c_int, _c_vp, _c_sz, _c_vp]),
    "gguf_dense_gemm_noalloc": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_vp,
                                         _c_vp, _c_int, _c_vp]),
    "gguf_mm_check_errors": (_c_int, [_c_vp]),
    "gguf_mm_status_string": (ctypes.c_char_p, [_c_int]),
    "gguf_mm_version": (_c_int, []),
    "gguf_mm_debug_gemv_terms": (_c_int, [_c_vp, _c_int, _c_int, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_vp,
                                          _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_int,
                                          ctypes.POINTER(_c_int), _c_vp]),
    "gguf_mm_gemv_kernel": (_c_int, [_c_int, _c_int, _c_i64, _c_i64, _c_i64, _c_int]),
    "gguf_mm_auto_path": (_c_int, [_c_int, _c_int, _c_i64, _c_i64, _c_i64, _c_int]),
    "gguf_mm_debug_moe_route": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp]),
    "gguf_mm_debug_timeout": (_c_int, [_c_i64, _c_vp]),
    "gguf_mm_debug_moe_mv_terms": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_int, _c_i64, _c_vp,
                                            _c_i64, _c_int, _c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                                            _c_sz, _c_vp]),
    "gguf_file_open": (_c_int, [ctypes.c_char_p, ctypes.POINTER(_c_vp)]),
    "gguf_file_close": (None, [_c_vp]),
    "gguf_file_version": (_c_int, [_c_vp]),
    "gguf_file_alignment": (_c_i64, [_c_vp]),
    "gguf_file_tensor_count": (_c_i64, [_c_vp]),
    "gguf_file_tensor_info": (_c_int, [_c_vp, _c_i64, ctypes.c_char_p, _c_sz, ctypes.POINTER(_c_int),
                                       ctypes.POINTER(_c_int), ctypes.POINTER(_c_i64),
                                       ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64)]),
    "gguf_file_find_tensor": (_c_i64, [_c_vp, ctypes.c_char_p]),
    "gguf_file_read_tensor": (_c_int, [_c_vp, _c_i64, _c_vp, _c_sz]),
    "gguf_file_tensor_as_weight": (_c_int, [_c_vp, _c_i64, ctypes.POINTER(_c_int), ctypes.POINTER(_c_i64),
                                            ctypes.POINTER(_c_i64)]),
    "gguf_file_kv_count": (_c_i64, [_c_vp]),
    "gguf_file_kv_key": (_c_int, [_c_vp, _c_i64, ctypes.c_char_p, _c_sz, ctypes.POINTER(_c_int)]),
    "gguf_file_get_int": (_c_int, [_c_vp, ctypes.c_char_p, ctypes.POINTER(_c_i64)]),
    "gguf_file_get_float": (_c_int, [_c_vp, ctypes.c_char_p, ctypes.POINTER(ctypes.c_double)]),
    "gguf_file_get_string": (_c_int, [_c_vp, ctypes.c_char_p, ctypes.c_char_p, _c_sz, ctypes.POINTER(_c_sz)]),
    "gguf_file_get_array": (_c_int, [_c_vp, ctypes.c_char_p, ctypes.POINTER(_c_int), ctypes.POINTER(_c_i64),
                                     _c_vp, _c_sz]),
}



# --- host structs of the serving operators (same members as include/gguf_mm.h) ---

GGUF_ROPE_NORM, GGUF_ROPE_NEOX = 0, 1


def _array(name, t, *dtypes):
    """t as an array that the kernels read element after element: of one of the types, without gaps (None and a device
    address pass)."""
    if t is None or isinstance(t, int):
        return t
    if str(t.dtype).rsplit(".", 1)[-1] not in dtypes or not t.is_contiguous():
        raise ValueError(f"{name} is a contiguous array of {' or '.join(dtypes)}, not {t.dtype} of strides {tuple(t.stride())}")
    return t


def _dt_of(t):
    import torch
    return {torch.float32: GGUF_DT_F32, torch.float16: GGUF_DT_F16, torch.bfloat16: GGUF_DT_BF16}[t.dtype]


class gguf_kv_cache(ctypes.Structure):
    """A layer's paged cache from two tensors [page, head, slot, dim] of any strides whose last is 1."""
    _fields_ = [("k", _c_vp), ("v", _c_vp), ("dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("n_pages", _c_i64),
                ("page_stride", _c_i64), ("head_stride", _c_i64), ("token_stride", _c_i64)]

    def __init__(self, k, v):
        if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.dim() != 4 or k.stride(3) != 1:
            raise ValueError("k and v are [page, head, slot, dim] tensors of one type and the same strides, the last 1")
        n, h, p, d = k.shape
        super().__init__(k.data_ptr(), v.data_ptr(), _dt_of(k), p, h, d, n, k.stride(0), k.stride(1), k.stride(2))
        self._keep = (k, v)
        self._ref = ctypes.addressof(self)


class gguf_kv_batch(ctypes.Structure):
    """A ragged batch: q_start [n_seq + 1], kv_len [n_seq], pages [n_seq, width] (int32 tensors on the device)."""
    _fields_ = [("q_start", _c_vp), ("kv_len", _c_vp), ("pages", _c_vp), ("n_seq", _c_i64), ("n_tokens", _c_i64),
                ("pages_stride", _c_i64), ("max_q_len", _c_i64), ("max_kv_len", _c_i64)]

    def __init__(self, q_start, kv_len, pages, n_tokens, max_q_len, max_kv_len):
        if q_start.numel() != kv_len.numel() + 1 or pages.shape[0] != kv_len.numel() or \
                (pages.shape[1] > 1 and pages.stride(1) != 1):
            raise ValueError("q_start has one entry more than kv_len, and pages a row of stride 1 for each sequence")
        if str(pages.dtype) not in ("torch.int32", "torch.uint32"):
            raise ValueError("q_start, kv_len and pages are int32")
        _array("q_start", q_start, "int32", "uint32"), _array("kv_len", kv_len, "int32", "uint32")
        stride = pages.stride(0) if pages.shape[0] > 1 else pages.shape[1]
        super().__init__(_p(q_start), _p(kv_len), _p(pages), kv_len.numel(), n_tokens, stride, max_q_len, max_kv_len)
        self._keep = (q_start, kv_len, pages)
        self._ref = ctypes.addressof(self)


class gguf_rope(ctypes.Structure):
    """Rotary positions: freqs f32 [rot_dim / 2] in radians a position, positions int32 [n_tokens] or None."""
    _fields_ = [("freqs", _c_vp), ("positions", _c_vp), ("rot_dim", ctypes.c_int32), ("style", ctypes.c_int32),
                ("scale", ctypes.c_float)]

    def __init__(self, freqs, rot_dim, style=GGUF_ROPE_NORM, scale=1.0, positions=None):
        _array("freqs", freqs, "float32"), _array("positions", positions, "int32", "uint32")
        if not (freqs is None or isinstance(freqs, int)) and 2 * freqs.numel() < rot_dim:
            raise ValueError(f"freqs has {freqs.numel()} entries for {rot_dim // 2} pairs")
        super().__init__(_p(freqs), _p(positions), rot_dim, style, scale)
        self._keep = (freqs, positions)
        self._ref = ctypes.addressof(self)


class gguf_logit_rules(ctypes.Structure):
    """Rules on a batch of logits; what is None is not used."""
    _fields_ = [("hist", _c_vp), ("hist_start", _c_vp), ("repeat", _c_vp), ("frequency", _c_vp), ("presence", _c_vp),
                ("bias_ids", _c_vp), ("bias", _c_vp), ("bias_start", _c_vp), ("allow", _c_vp), ("allow_stride", _c_i64)]

    def __init__(self, hist=None, hist_start=None, repeat=None, frequency=None, presence=None, bias_ids=None, bias=None,
                 bias_start=None, allow=None):
        for name, t in (("hist", hist), ("hist_start", hist_start), ("bias_ids", bias_ids), ("bias_start", bias_start)):
            _array(name, t, "int32", "uint32")
        for name, t in (("repeat", repeat), ("frequency", frequency), ("presence", presence), ("bias", bias)):
            _array(name, t, "float32")
        if allow is not None and (str(allow.dtype) not in ("torch.int32", "torch.uint32") or allow.dim() != 2 or
                                  (allow.shape[1] > 1 and allow.stride(1) != 1)):
            raise ValueError("allow is a matrix of 32-bit words whose rows are dense")
        stride = 0 if allow is None else allow.stride(0) if allow.shape[0] > 1 else allow.shape[1]
        super().__init__(*(_p(t) for t in (hist, hist_start, repeat, frequency, presence, bias_ids, bias, bias_start,
                                           allow)), stride)
        self._keep = (hist, hist_start, repeat, frequency, presence, bias_ids, bias, bias_start, allow)
        self._ref = ctypes.addressof(self)


class gguf_head_norm(ctypes.Structure):
    """Norms of the query and key heads: weights f32 [head_dim] (None: those heads are not normed) and eps."""
    _fields_ = [("q", _c_vp), ("k", _c_vp), ("eps", ctypes.c_float)]

    def __init__(self, q, k, eps=1e-6):
        _array("q", q, "float32"), _array("k", k, "float32")
        super().__init__(_p(q), _p(k), eps)
        self._keep = (q, k)
        self._ref = ctypes.addressof(self)


GGUF_SCORE_SOFTMAX, GGUF_SCORE_SIGMOID = 0, 1
GGUF_ACT_SILU, GGUF_ACT_GELU = 0, 1


class gguf_router(ctypes.Structure):
    """A router: w [n_expert, K] of f32, f16 or bf16 without gaps, bias f32 [n_expert] or None."""
    _fields_ = [("w", _c_vp), ("bias", _c_vp), ("wdt", ctypes.c_int32), ("n_expert", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]

    def __init__(self, w, top_k, score=GGUF_SCORE_SOFTMAX, bias=None, renormalize=True, scale=1.0):
        _array("w", w, "float32", "float16", "bfloat16"), _array("bias", bias, "float32")
        if w.dim() != 2 or not (bias is None or isinstance(bias, int)) and bias.numel() != w.shape[0]:
            raise ValueError("w is [n_expert, K], and bias has one entry for each expert")
        super().__init__(_p(w), _p(bias), _dt_of(w), w.shape[0], top_k, score, int(renormalize), scale)
        self._keep = (w, bias)
        self._ref = ctypes.addressof(self)


class gguf_moe_weights(ctypes.Structure):
    """Experts' gate and up [n_expert][F, K] and down [n_expert][K, F] as GGUF blocks back to back (uint8 tensors without
    gaps, or device addresses)."""
    _fields_ = [("gate", _c_vp), ("up", _c_vp), ("down", _c_vp), ("gate_type", ctypes.c_int32), ("up_type", ctypes.c_int32),
                ("down_type", ctypes.c_int32), ("act", ctypes.c_int32), ("n_expert", _c_i64), ("K", _c_i64), ("F", _c_i64)]

    def __init__(self, gate, up, down, gate_type, up_type, down_type, K, F, n_expert, act=GGUF_ACT_SILU):
        for name, t, qt, n, k in (("gate", gate, gate_type, F, K), ("up", up, up_type, F, K), ("down", down, down_type, K, F)):
            _array(name, t, "uint8")
            if qt in BLOCK_VALUES and not (t is None or isinstance(t, int)) and \
                    t.numel() != n_expert * n * (k // BLOCK_VALUES[qt]) * BLOCK_BYTES[qt]:
                raise ValueError(f"{name} has {t.numel()} bytes, not those of {n_expert} tensors [{n}, {k}]")
        super().__init__(_p(gate), _p(up), _p(down), gate_type, up_type, down_type, act, n_expert, K, F)
        self._keep = (gate, up, down)
        self._ref = ctypes.addressof(self)


class gguf_sampler(ctypes.Structure):
    """What each row is drawn by: temperature, top_p, min_p f32 [rows], top_k int32 [rows]; what is None is not used."""
    _fields_ = [("temperature", _c_vp), ("top_k", _c_vp), ("top_p", _c_vp), ("min_p", _c_vp)]

    def __init__(self, temperature=None, top_k=None, top_p=None, min_p=None):
        _array("top_k", top_k, "int32")
        for name, t in (("temperature", temperature), ("top_p", top_p), ("min_p", min_p)):
            _array(name, t, "float32")
        super().__init__(_p(temperature), _p(top_k), _p(top_p), _p(min_p))
        self._keep = (temperature, top_k, top_p, min_p)
        self._ref = ctypes.addressof(self)


_SIGS.update({
    "gguf_kv_append_norm": (_c_int, [_c_vp, _c_i64, _c_vp, _c_i64, _c_vp, _c_i64, _c_int, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp,
                                     _c_vp, _c_i64, _c_vp]),
    "gguf_moe_router": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp]),
    "gguf_moe_ffn": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_int, _c_vp, _c_sz, _c_vp]),
    "gguf_moe_ffn_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "gguf_sample": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "gguf_kv_append": (_c_int, [_c_vp, _c_i64, _c_vp, _c_i64, _c_vp, _c_i64, _c_int, _c_i64, _c_vp, _c_vp, _c_vp,
                                _c_vp, _c_i64, _c_vp]),
    "gguf_paged_attn": (_c_int, [_c_vp, _c_i64, _c_i64, _c_vp, _c_vp, ctypes.c_float, _c_int, _c_i64, _c_vp, _c_i64,
                                 _c_vp, _c_vp, _c_sz, _c_vp]),
    "gguf_paged_attn_workspace_size": (_c_sz, [_c_vp, _c_vp, _c_i64]),
    "gguf_logits_adjust": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_vp, _c_int, _c_i64, _c_vp]),
})

_lib = None


class GGUFError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: status {status} ({status_string(status)})")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load (once) and return the shared library; raises if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with __graft_entry__.build() "
                              "(or python gguf_quant_weight_gb300/_build.py)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def exported_symbols():
    return list(_SIGS)


def _p(t):
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


def _s(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, st):
    if st != 0:
        raise GGUFError(fn, st)
    return st


def status_string(status: int) -> str:
    return load_library().gguf_mm_status_string(status).decode()


def gguf_mm_version() -> int:
    return load_library().gguf_mm_version()


def gguf_mm_workspace_size(op, qtype, N, K, M, n_expert=0, top_k=0) -> int:
    return load_library().gguf_mm_workspace_size(op, qtype, N, K, M, n_expert, top_k)


def gguf_mm_gemv(w, qtype, layout, N, K, x, xdt, M, residual, y, ydt, workspace=None, ws_bytes=0, stream=None):
    return _check("gguf_mm_gemv", load_library().gguf_mm_gemv(
        _p(w), qtype, layout, N, K, _p(x), xdt, M, _p(residual), _p(y), ydt, _p(workspace), ws_bytes, _s(stream)))


def gguf_mm_gemv_host(w, qtype, layout, N, K, x_host, x_dev, xdt, M, residual_host, residual_dev, y_host, y_dev,
                      ydt, workspace=None, ws_bytes=0, stream=None):
    return _check("gguf_mm_gemv_host", load_library().gguf_mm_gemv_host(
        _p(w), qtype, layout, N, K, _p(x_host), _p(x_dev), xdt, M, _p(residual_host), _p(residual_dev),
        _p(y_host), _p(y_dev), ydt, _p(workspace), ws_bytes, _s(stream)))


def gguf_mm_gemm(w, qtype, layout, N, K, x, xdt, M, residual, y, ydt, workspace=None, ws_bytes=0,
                 path=GGUF_PATH_AUTO, stream=None):
    return _check("gguf_mm_gemm", load_library().gguf_mm_gemm(
        _p(w), qtype, layout, N, K, _p(x), xdt, M, _p(residual), _p(y), ydt, _p(workspace), ws_bytes, path,
        _s(stream)))


def gguf_mm_id(w_experts, qtype, n_expert, N, K, x, xdt, T, ids, top_k, residual, y, ydt, workspace=None,
               ws_bytes=0, stream=None):
    return _check("gguf_mm_id", load_library().gguf_mm_id(
        _p(w_experts), qtype, n_expert, N, K, _p(x), xdt, T, _p(ids), top_k, _p(residual), _p(y), ydt,
        _p(workspace), ws_bytes, _s(stream)))


def gguf_mm_id_slots(w_experts, qtype, n_expert, N, K, x, xdt, T, ids, top_k, residual, y, ydt, workspace=None,
                     ws_bytes=0, stream=None):
    return _check("gguf_mm_id_slots", load_library().gguf_mm_id_slots(
        _p(w_experts), qtype, n_expert, N, K, _p(x), xdt, T, _p(ids), top_k, _p(residual), _p(y), ydt,
        _p(workspace), ws_bytes, _s(stream)))


def gguf_mm_id_form(qtype, T, top_k) -> int:
    return load_library().gguf_mm_id_form(qtype, T, top_k)


def gguf_mm_id_path(w_experts, qtype, n_expert, N, K, x, xdt, T, ids, top_k, per_slot, residual, y, ydt,
                    workspace=None, ws_bytes=0, path=GGUF_PATH_AUTO, stream=None):
    return _check("gguf_mm_id_path", load_library().gguf_mm_id_path(
        _p(w_experts), qtype, n_expert, N, K, _p(x), xdt, T, _p(ids), top_k, per_slot, _p(residual), _p(y), ydt,
        _p(workspace), ws_bytes, path, _s(stream)))


def gguf_repack_q6k_planes(src, dst, nblk, inverse=0, stream=None):
    return _check("gguf_repack_q6k_planes", load_library().gguf_repack_q6k_planes(
        _p(src), _p(dst), nblk, inverse, _s(stream)))


def gguf_dequant_padded(w, qtype, layout, N, K, out, odt, ld, stream=None):
    return _check("gguf_dequant_padded", load_library().gguf_dequant_padded(
        _p(w), qtype, layout, N, K, _p(out), odt, ld, _s(stream)))


def gguf_dense_gemm(wdense, wdt, ld, N, K, x, xdt, M, residual, y, ydt, workspace=None, ws_bytes=0, stream=None):
    return _check("gguf_dense_gemm", load_library().gguf_dense_gemm(
        _p(wdense), wdt, ld, N, K, _p(x), xdt, M, _p(residual), _p(y), ydt, _p(workspace), ws_bytes, _s(stream)))


def gguf_dense_gemm_noalloc(wdense, wdt, ld, N, K, x, xdt, M, residual, y, ydt, stream=None):
    return _check("gguf_dense_gemm_noalloc", load_library().gguf_dense_gemm_noalloc(
        _p(wdense), wdt, ld, N, K, _p(x), xdt, M, _p(residual), _p(y), ydt, _s(stream)))


def gguf_mm_check_errors(stream=None) -> int:
    """Returns the device status (0 or a negative code) without raising."""
    return load_library().gguf_mm_check_errors(_s(stream))


GEMV_KERNELS = {0: "staged", 1: "direct", 2: "tile", 3: "pair", 4: "rowlane"}


def gguf_mm_debug_gemv_terms(w, qtype, layout, N, K, x, xdt, M, residual, y, ydt, qa=None, d_a=None, s=None,
                             D=None, workspace=None, ws_bytes=0, kernel=-1, stream=None) -> int:
    """Runs the GEMV with its integer intermediates dumped; returns the id of the kernel that ran."""
    out = _c_int(-1)
    _check("gguf_mm_debug_gemv_terms", load_library().gguf_mm_debug_gemv_terms(
        _p(w), qtype, layout, N, K, _p(x), xdt, M, _p(residual), _p(y), ydt, _p(qa), _p(d_a), _p(s), _p(D),
        _p(workspace), ws_bytes, kernel, ctypes.byref(out), _s(stream)))
    return out.value


def gguf_mm_auto_path(qtype, layout, N, K, M, xdt=GGUF_DT_BF16) -> int:
    """The path GGUF_PATH_AUTO takes for this shape (GGUF_PATH_GEMV or GGUF_PATH_FUSED)."""
    return load_library().gguf_mm_auto_path(qtype, layout, N, K, M, xdt)


def gguf_mm_gemv_kernel(qtype, layout, N, K, M, xdt=GGUF_DT_BF16) -> int:
    """The id of the GEMV kernel gguf_mm_gemv picks for this shape (negative status on error)."""
    return load_library().gguf_mm_gemv_kernel(qtype, layout, N, K, M, xdt)


def gguf_mm_debug_moe_route(ids, entries, n_expert, offsets, ntiles, tiles, max_tiles, rows, stream=None):
    return _check("gguf_mm_debug_moe_route", load_library().gguf_mm_debug_moe_route(
        _p(ids), entries, n_expert, _p(offsets), _p(ntiles), _p(tiles), max_tiles, _p(rows), _s(stream)))


def gguf_mm_debug_moe_mv_terms(w_experts, qtype, n_expert, N, K, x, xdt, T, ids, top_k, per_slot, residual, y, ydt,
                               qa=None, d_a=None, s=None, D=None, workspace=None, ws_bytes=0, stream=None):
    return _check("gguf_mm_debug_moe_mv_terms", load_library().gguf_mm_debug_moe_mv_terms(
        _p(w_experts), qtype, n_expert, N, K, _p(x), xdt, T, _p(ids), top_k, per_slot, _p(residual), _p(y), ydt,
        _p(qa), _p(d_a), _p(s), _p(D), _p(workspace), ws_bytes, _s(stream)))


def gguf_mm_debug_timeout(spin_limit, stream=None):
    return _check("gguf_mm_debug_timeout", load_library().gguf_mm_debug_timeout(spin_limit, _s(stream)))


# --- serving operators --------------------------------------------------------

# These run between products that take a few microseconds each, so the
# marshalling is kept short: a call of one token is bound by the host.

def gguf_kv_append(q, ldq, k, ldk, v, ldv, xdt, heads, rope, batch, cache, q_out, ldqo, stream=None):
    st = (_lib or load_library()).gguf_kv_append(
        _p(q), ldq, _p(k), ldk, _p(v), ldv, xdt, heads, rope and rope._ref, batch and batch._ref, cache and cache._ref,
        _p(q_out), ldqo, stream if stream.__class__ is int else _s(stream))
    return _check("gguf_kv_append", st) if st else st


def gguf_paged_attn(q, ldq, heads, batch, cache, scale, causal, window, out, ldo, lse=None, workspace=None, ws_bytes=0,
                    stream=None):
    st = (_lib or load_library()).gguf_paged_attn(
        _p(q), ldq, heads, batch and batch._ref, cache and cache._ref, scale, causal, window, _p(out), ldo, _p(lse),
        _p(workspace), ws_bytes, stream if stream.__class__ is int else _s(stream))
    return _check("gguf_paged_attn", st) if st else st


def gguf_paged_attn_workspace_size(batch, cache, heads) -> int:
    return load_library().gguf_paged_attn_workspace_size(batch and batch._ref, cache and cache._ref, heads)


def gguf_logits_adjust(logits, dt, ld, rows, vocab, rules, out, odt, ldo, stream=None):
    st = (_lib or load_library()).gguf_logits_adjust(
        _p(logits), dt, ld, rows, vocab, rules and rules._ref, _p(out), odt, ldo,
        stream if stream.__class__ is int else _s(stream))
    return _check("gguf_logits_adjust", st) if st else st


def gguf_kv_append_norm(q, ldq, k, ldk, v, ldv, xdt, heads, norm, rope, batch, cache, q_out, ldqo, stream=None):
    st = (_lib or load_library()).gguf_kv_append_norm(
        _p(q), ldq, _p(k), ldk, _p(v), ldv, xdt, heads, norm and norm._ref, rope and rope._ref, batch and batch._ref,
        cache and cache._ref, _p(q_out), ldqo, stream if stream.__class__ is int else _s(stream))
    return _check("gguf_kv_append_norm", st) if st else st


def gguf_moe_router(x, xdt, T, K, router, ids, weights, stream=None):
    st = (_lib or load_library()).gguf_moe_router(
        _p(x), xdt, T, K, router and router._ref, _p(ids), _p(weights), stream if stream.__class__ is int else _s(stream))
    return _check("gguf_moe_router", st) if st else st


def gguf_moe_ffn(experts, x, xdt, T, ids, weights, top_k, residual, y, ydt, workspace=None, ws_bytes=0, stream=None):
    st = (_lib or load_library()).gguf_moe_ffn(
        experts and experts._ref, _p(x), xdt, T, _p(ids), _p(weights), top_k, _p(residual), _p(y), ydt, _p(workspace), ws_bytes,
        stream if stream.__class__ is int else _s(stream))
    return _check("gguf_moe_ffn", st) if st else st


def gguf_moe_ffn_workspace_size(F, T, top_k) -> int:
    return load_library().gguf_moe_ffn_workspace_size(F, T, top_k)


def gguf_sample(logits, dt, ld, rows, vocab, sampler, u, token, logprob=None, stream=None):
    st = (_lib or load_library()).gguf_sample(
        _p(logits), dt, ld, rows, vocab, sampler and sampler._ref, _p(u), _p(token), _p(logprob),
        stream if stream.__class__ is int else _s(stream))
    return _check("gguf_sample", st) if st else st


# --- GGUF container reader (host only) ---------------------------------------

def _enc(s):
    return s.encode("utf-8", "surrogateescape")


def _dec(b):
    return b.decode("utf-8", "surrogateescape")


class GGUFFile:
    """A .gguf file opened through gguf_file_open: metadata values and tensor bytes.

    Thin marshalling over the gguf_file_* entry points; the parsing and every
    bounds check are in the library.  `tensors()` lists (name, type, dims);
    `tensor_bytes(name)` returns the tensor's bytes as a numpy u8 array, which
    for a block-quantized weight W[N, K] is the [N, K/blk*bb] block array the
    matmul entry points take."""

    def __init__(self, path):
        self._h = None
        lib = load_library()
        h = _c_vp()
        _check("gguf_file_open", lib.gguf_file_open(os.fsencode(path), ctypes.byref(h)))
        self._h = h.value
        self._lib = lib

    def close(self):
        if getattr(self, "_h", None):
            self._lib.gguf_file_close(self._h)
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        self.close()

    @property
    def version(self) -> int:
        return self._lib.gguf_file_version(self._h)

    @property
    def alignment(self) -> int:
        return self._lib.gguf_file_alignment(self._h)

    def tensor_info(self, index):
        """(name, type, dims (contiguous first), absolute data offset, nbytes)."""
        n = 1024
        while True:
            name = ctypes.create_string_buffer(n)
            t, nd = _c_int(), _c_int()
            dims = (_c_i64 * 4)()
            off, nb = ctypes.c_uint64(), ctypes.c_uint64()
            st = self._lib.gguf_file_tensor_info(self._h, index, name, n, ctypes.byref(t), ctypes.byref(nd), dims,
                                                 ctypes.byref(off), ctypes.byref(nb))
            if st == GGUF_ERR_WORKSPACE:
                n *= 16
                continue
            _check("gguf_file_tensor_info", st)
            return _dec(name.value), t.value, tuple(dims[:nd.value]), off.value, nb.value

    def tensors(self):
        return [self.tensor_info(i)[:3] for i in range(self._lib.gguf_file_tensor_count(self._h))]

    def find_tensor(self, name) -> int:
        i = self._lib.gguf_file_find_tensor(self._h, _enc(name))
        if i < 0:
            raise GGUFError("gguf_file_find_tensor", int(i))
        return int(i)

    def tensor_bytes(self, name_or_index):
        import numpy as np
        i = self.find_tensor(name_or_index) if isinstance(name_or_index, str) else name_or_index
        nb = self.tensor_info(i)[4]
        out = np.empty(nb, np.uint8)
        _check("gguf_file_read_tensor", self._lib.gguf_file_read_tensor(self._h, i, out.ctypes.data, nb))
        return out

    def weight(self, name):
        """(blocks as a [N, row_bytes] u8 array, qtype, N, K) of a 2-D block-quantized tensor."""
        i = self.find_tensor(name)
        qt, n, k = _c_int(), _c_i64(), _c_i64()
        _check("gguf_file_tensor_as_weight", self._lib.gguf_file_tensor_as_weight(
            self._h, i, ctypes.byref(qt), ctypes.byref(n), ctypes.byref(k)))
        return self.tensor_bytes(i).reshape(n.value, -1), qt.value, n.value, k.value

    def keys(self):
        out = []
        for i in range(self._lib.gguf_file_kv_count(self._h)):
            n = 256
            while True:
                buf, vt = ctypes.create_string_buffer(n), _c_int()
                st = self._lib.gguf_file_kv_key(self._h, i, buf, n, ctypes.byref(vt))
                if st == GGUF_ERR_WORKSPACE:
                    n *= 16
                    continue
                _check("gguf_file_kv_key", st)
                out.append((_dec(buf.value), vt.value))
                break
        return out

    def get_int(self, key) -> int:
        v = _c_i64()
        _check("gguf_file_get_int", self._lib.gguf_file_get_int(self._h, _enc(key), ctypes.byref(v)))
        return v.value

    def get_float(self, key) -> float:
        v = ctypes.c_double()
        _check("gguf_file_get_float", self._lib.gguf_file_get_float(self._h, _enc(key), ctypes.byref(v)))
        return v.value

    def get_string(self, key) -> str:
        n = _c_sz()
        _check("gguf_file_get_string", self._lib.gguf_file_get_string(self._h, _enc(key), None, 0,
                                                                      ctypes.byref(n)))
        buf = ctypes.create_string_buffer(n.value + 1)
        _check("gguf_file_get_string", self._lib.gguf_file_get_string(self._h, _enc(key), buf, n.value + 1,
                                                                      None))
        return _dec(buf.raw[:n.value])

    _ARRAY_NP = {0: "u1", 1: "i1", 2: "<u2", 3: "<i2", 4: "<u4", 5: "<i4", 6: "<f4", 7: "u1", 10: "<u8",
                 11: "<i8", 12: "<f8"}

    def get_array(self, key):
        """A scalar array as numpy; a string array as (8, count)."""
        import numpy as np
        et, cnt = _c_int(), _c_i64()
        _check("gguf_file_get_array", self._lib.gguf_file_get_array(self._h, _enc(key), ctypes.byref(et),
                                                                    ctypes.byref(cnt), None, 0))
        if et.value not in self._ARRAY_NP:
            return et.value, cnt.value
        out = np.empty(cnt.value, self._ARRAY_NP[et.value])
        _check("gguf_file_get_array", self._lib.gguf_file_get_array(self._h, _enc(key), None, None,
                                                                    out.ctypes.data, out.nbytes))
        return out


def raw_status(fn_name: str, *args) -> int:
    """Call a C entry point with raw arguments and return its status (tests of argument checks)."""
    return getattr(load_library(), fn_name)(*args)
