"""Exact softmax attention for GB300 (sm_103a): Python binding of the C ABI in ``include/attn.h``.

The functions here only marshal arguments (tensor data pointers, sizes, the CUDA
stream) and call the native library; every step of the computation runs in its
CUDA kernels. There is no fallback: if the library is missing, importing this
package raises.

Tensors may be ``torch.Tensor`` objects (their ``data_ptr()`` is passed) or raw
integer device addresses. ``stream`` may be a ``torch.cuda.Stream``, an integer
``cudaStream_t`` handle, or ``None`` for the current PyTorch stream (the legacy
default stream when PyTorch is not in use).
"""
from __future__ import annotations

import ctypes
import os
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libattn_gb300.so")

ATTN_OK = 0
ATTN_ERR_NULL_PTR = -1
ATTN_ERR_BAD_SHAPE = -2
ATTN_ERR_ALIGN = -3
ATTN_ERR_UNSUPPORTED_ARCH = -4
ATTN_ERR_CUDA = -5
ATTN_ERR_DEVICE_TIMEOUT = -6
ATTN_ERR_DEVICE_BAD_INDEX = -7
ATTN_ERR_BAD_ARG = -8
ATTN_ERR_SCRATCH_TOO_SMALL = -9

ATTN_FP8_E4M3 = 0
ATTN_FP8_E5M2 = 1
ATTN_KV_BF16 = 2
FP8_FORMATS = {"e4m3": ATTN_FP8_E4M3, "e5m2": ATTN_FP8_E5M2}
KV_FORMATS = {**FP8_FORMATS, "bf16": ATTN_KV_BF16}

ATTN_TYPE_BF16 = 0
ATTN_TYPE_F32 = 1
ELEM_TYPES = {"bf16": ATTN_TYPE_BF16, "f32": ATTN_TYPE_F32}
ATTN_ROPE_PLAIN = 0
ATTN_ROPE_LINEAR = 1
ATTN_ROPE_NTK = 2
ATTN_ROPE_YARN = 3
ROPE_SCALINGS = {"plain": ATTN_ROPE_PLAIN, "linear": ATTN_ROPE_LINEAR, "ntk": ATTN_ROPE_NTK, "yarn": ATTN_ROPE_YARN}

#: every symbol the header declares
EXPORTS = ("attn_fwd", "attn_fwd_hd", "attn_fwd_fp8", "attn_decode_paged", "attn_decode_paged_fp8", "attn_decode_paged_noalloc",
           "attn_rope", "attn_rope_freqs", "attn_kv_write_paged", "attn_kv_read_paged", "attn_decode_paged_tree", "attn_qk_norm_rope",
           "attn_qk_norm_rope_bwd", "attn_kv_score_paged", "attn_kv_select_paged", "attn_kv_compact_paged", "attn_decode_plan",
           "attn_decode_workspace_bytes", "attn_status_string", "attn_get_device_status",
           "attn_set_option", "attn_get_option", "attn_read_counters", "attn_debug_exp2", "attn_debug_watchdog",
           "attn_version")


class AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {status_string(code)} (status {code})")
        self.code = code


if not os.path.exists(LIB_PATH):
    raise ImportError(f"CUDA attention library not built: {LIB_PATH} is missing "
                      "(run __graft_entry__.build() or python exact_softmax_attention_gb300/build.py)")

lib = ctypes.CDLL(LIB_PATH)
_vp, _i, _f, _d = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_double
_ll = ctypes.c_longlong
lib.attn_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp]
lib.attn_fwd.restype = _i
lib.attn_fwd_hd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp]
lib.attn_fwd_hd.restype = _i
lib.attn_fwd_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp, _i, _f, _f, _f]
lib.attn_fwd_fp8.restype = _i
lib.attn_decode_paged.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i]
lib.attn_decode_paged.restype = _i
lib.attn_decode_paged_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _i, _f,
                                       _f]
lib.attn_decode_paged_fp8.restype = _i
lib.attn_decode_paged_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i]
lib.attn_decode_paged_noalloc.restype = _i
lib.attn_rope.argtypes = [_vp] * 6 + [_i] * 6 + [_ll] * 4 + [_i] * 3 + [_f, _vp]
lib.attn_rope.restype = _i
lib.attn_rope_freqs.argtypes = [ctypes.POINTER(_d), ctypes.POINTER(_d), _i, _d, _i, _d, _d, _d, _d]
lib.attn_rope_freqs.restype = _i
lib.attn_kv_write_paged.argtypes = [_vp, _vp, _ll, _ll] + [_vp] * 5 + [_i] * 8 + [_f, _f, _vp, _vp, _i, _i, _i, _f, _vp]
lib.attn_kv_write_paged.restype = _i
lib.attn_kv_read_paged.argtypes = [_vp] * 4 + [_ll, _ll] + [_vp] * 3 + [_i] * 8 + [_f, _f, _vp]
lib.attn_kv_read_paged.restype = _i
lib.attn_decode_paged_tree.argtypes = [_vp] * 7 + [_i, _i] + [_vp] * 3 + [_i] * 8 + [_f, _i, _i, _f, _f]
lib.attn_decode_paged_tree.restype = _i
lib.attn_qk_norm_rope.argtypes = [_vp] * 6 + [_f] + [_vp] * 2 + [_i] * 6 + [_ll] * 4 + [_i] * 2 + [_f, _vp]
lib.attn_qk_norm_rope.restype = _i
lib.attn_qk_norm_rope_bwd.argtypes = [_vp] * 6 + [_f] + [_vp] * 6 + [_i] * 6 + [_ll] * 6 + [_i] * 2 + [_f, _vp]
lib.attn_qk_norm_rope_bwd.restype = _i
lib.attn_kv_score_paged.argtypes = [_vp] * 7 + [_i] * 9 + [_f, _f, _i, _f, _vp]
lib.attn_kv_score_paged.restype = _i
lib.attn_kv_select_paged.argtypes = [_vp] * 5 + [_i] * 8 + [_vp]
lib.attn_kv_select_paged.restype = _i
lib.attn_kv_compact_paged.argtypes = [_vp] * 6 + [_i] * 8 + [_vp]
lib.attn_kv_compact_paged.restype = _i
lib.attn_decode_plan.argtypes = [_i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_i), ctypes.POINTER(_i)]
lib.attn_decode_plan.restype = _i
lib.attn_decode_workspace_bytes.argtypes = [_i, _i, _i, _i]
lib.attn_decode_workspace_bytes.restype = ctypes.c_size_t
lib.attn_status_string.argtypes = [_i]
lib.attn_status_string.restype = ctypes.c_char_p
lib.attn_get_device_status.argtypes = [_vp]
lib.attn_get_device_status.restype = _i
lib.attn_set_option.argtypes = [ctypes.c_char_p, _d]
lib.attn_set_option.restype = _i
lib.attn_get_option.argtypes = [ctypes.c_char_p, ctypes.POINTER(_d)]
lib.attn_get_option.restype = _i
lib.attn_read_counters.argtypes = [ctypes.POINTER(ctypes.c_ulonglong), _i]
lib.attn_read_counters.restype = _i
lib.attn_debug_exp2.argtypes = [_vp, _vp, ctypes.c_longlong, _i, _vp]
lib.attn_debug_exp2.restype = _i
lib.attn_debug_watchdog.argtypes = [ctypes.c_ulonglong, _vp]
lib.attn_debug_watchdog.restype = _i
lib.attn_version.argtypes = []
lib.attn_version.restype = ctypes.c_char_p


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        torch = sys.modules.get("torch")  # not imported: the caller does not use its streams
        if torch is not None and torch.cuda.is_initialized():
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without making a Stream object
            return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(code: int, where: str, raise_on_error: bool):
    if raise_on_error and code != ATTN_OK:
        raise AttnError(code, where)
    return code


def _code(names, x):
    return names[x] if isinstance(x, str) else int(x)


def status_string(code: int) -> str:
    return lib.attn_status_string(code).decode()


def attn_fwd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, cu_seqlens=None, stream=None,
             raise_on_error=True):
    """Exact attention forward; see ``attn_fwd`` in include/attn.h."""
    rc = lib.attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq), int(Hkv), int(Nq), int(Nk),
                      int(d), float(scale), int(causal), _ptr(cu_seqlens), _stream(stream))
    return _check(rc, "attn_fwd", raise_on_error)


def attn_fwd_hd(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, dv, scale, causal, cu_seqlens=None, stream=None,
                raise_on_error=True):
    """Forward with values narrower than queries and keys, (d, dv) = (192, 128); see
    ``attn_fwd_hd`` in include/attn.h."""
    rc = lib.attn_fwd_hd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq), int(Hkv), int(Nq), int(Nk),
                         int(d), int(dv), float(scale), int(causal), _ptr(cu_seqlens), _stream(stream))
    return _check(rc, "attn_fwd_hd", raise_on_error)


def attn_fwd_fp8(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, scale, causal, cu_seqlens=None, stream=None,
                 fp8_format="e4m3", q_descale=1.0, k_descale=1.0, v_descale=1.0, raise_on_error=True):
    """Forward on 8-bit floating-point Q/K/V; see ``attn_fwd_fp8`` in include/attn.h."""
    fmt = FP8_FORMATS[fp8_format] if isinstance(fp8_format, str) else int(fp8_format)
    rc = lib.attn_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq), int(Hkv), int(Nq), int(Nk),
                          int(d), float(scale), int(causal), _ptr(cu_seqlens), _stream(stream), fmt, float(q_descale),
                          float(k_descale), float(v_descale))
    return _check(rc, "attn_fwd_fp8", raise_on_error)


def attn_decode_paged(q, k_cache, v_cache, page_table, seqlens, page_size, o, lse, stream, B, Hq, Hkv, d,
                      max_pages_per_seq, num_pages, scale, num_splits=0, raise_on_error=True):
    """Paged-KV split decode; see ``attn_decode_paged`` in include/attn.h."""
    rc = lib.attn_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seqlens),
                               int(page_size), _ptr(o), _ptr(lse), _stream(stream), int(B), int(Hq), int(Hkv), int(d),
                               int(max_pages_per_seq), int(num_pages), float(scale), int(num_splits))
    return _check(rc, "attn_decode_paged", raise_on_error)


def attn_decode_paged_fp8(q, k_cache, v_cache, page_table, seqlens, page_size, o, lse, stream, B, Hq, Hkv, d,
                          max_pages_per_seq, num_pages, scale, num_splits=0, kv_format="e4m3", k_descale=1.0,
                          v_descale=1.0, raise_on_error=True):
    """Paged decode over FP8 key/value caches; see ``attn_decode_paged_fp8`` in include/attn.h.
    ``kv_format`` is "e4m3" or "e5m2" (or the ATTN_FP8_* code)."""
    fmt = FP8_FORMATS[kv_format] if isinstance(kv_format, str) else int(kv_format)
    rc = lib.attn_decode_paged_fp8(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seqlens),
                                   int(page_size), _ptr(o), _ptr(lse), _stream(stream), int(B), int(Hq), int(Hkv),
                                   int(d), int(max_pages_per_seq), int(num_pages), float(scale), int(num_splits), fmt,
                                   float(k_descale), float(v_descale))
    return _check(rc, "attn_decode_paged_fp8", raise_on_error)


def attn_decode_paged_noalloc(q, k_cache, v_cache, page_table, seqlens, page_size, o, lse, stream, B, Hq, Hkv, d,
                              max_pages_per_seq, num_pages, scale, num_splits=0, raise_on_error=True):
    """attn_decode_paged without allocating: split partials use the library's fixed 32 MiB
    device array (see include/attn.h for the size limit and the sharing rules)."""
    rc = lib.attn_decode_paged_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seqlens),
                                       int(page_size), _ptr(o), _ptr(lse), _stream(stream), int(B), int(Hq), int(Hkv),
                                       int(d), int(max_pages_per_seq), int(num_pages), float(scale), int(num_splits))
    return _check(rc, "attn_decode_paged_noalloc", raise_on_error)


def attn_rope(q, k, q_out, k_out, positions, inv_freq, T, Hq, Hk, d, rot_begin, rot_dim, q_stride, k_stride, q_out_stride,
              k_out_stride, elem_type="bf16", interleaved=0, transpose=0, amplitude=1.0, stream=None, raise_on_error=True):
    """Rotary positions of q and k (``transpose=1``: the gradient); see ``attn_rope`` in include/attn.h.
    ``elem_type`` is "bf16" or "f32" (or the ATTN_TYPE_* code)."""
    rc = lib.attn_rope(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _ptr(positions), _ptr(inv_freq), int(T), int(Hq), int(Hk),
                       int(d), int(rot_begin), int(rot_dim), int(q_stride), int(k_stride), int(q_out_stride),
                       int(k_out_stride), _code(ELEM_TYPES, elem_type), int(interleaved), int(transpose), float(amplitude),
                       _stream(stream))
    return _check(rc, "attn_rope", raise_on_error)


def attn_rope_freqs(rot_dim, theta=10000.0, scaling="plain", factor=1.0, trained_len=0.0, beta_fast=32.0, beta_slow=1.0):
    """(frequencies, amplitude) of ``attn_rope``: a list of rot_dim / 2 floats (put it on the device
    as float64) and the factor that belongs to it; see ``attn_rope_freqs`` in include/attn.h.
    ``scaling`` is "plain", "linear", "ntk" or "yarn" (or the ATTN_ROPE_* code)."""
    out, amp = (_d * max(1, int(rot_dim) // 2))(), _d()
    rc = lib.attn_rope_freqs(out, ctypes.byref(amp), int(rot_dim), float(theta), _code(ROPE_SCALINGS, scaling), float(factor),
                             float(trained_len), float(beta_fast), float(beta_slow))
    _check(rc, "attn_rope_freqs", True)
    return list(out), amp.value


def attn_kv_write_paged(k, v, k_stride, v_stride, k_cache, v_cache, page_table, seqlens, cu_seqlens, page_size, T, B, Hkv, d,
                        max_pages_per_seq, num_pages, kv_format="bf16", k_descale=1.0, v_descale=1.0, positions=None,
                        inv_freq=None, rot_begin=0, rot_dim=0, interleaved=0, amplitude=1.0, stream=None,
                        raise_on_error=True):
    """New keys (optionally rotated) and values into a paged cache; see ``attn_kv_write_paged`` in
    include/attn.h. ``kv_format`` is "bf16", "e4m3" or "e5m2" (or the code)."""
    rc = lib.attn_kv_write_paged(_ptr(k), _ptr(v), int(k_stride), int(v_stride), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(page_table), _ptr(seqlens), _ptr(cu_seqlens), int(page_size), int(T), int(B), int(Hkv),
                                 int(d), int(max_pages_per_seq), int(num_pages), _code(KV_FORMATS, kv_format),
                                 float(k_descale), float(v_descale), _ptr(positions), _ptr(inv_freq), int(rot_begin),
                                 int(rot_dim), int(interleaved), float(amplitude), _stream(stream))
    return _check(rc, "attn_kv_write_paged", raise_on_error)


def attn_kv_read_paged(k_cache, v_cache, k, v, k_stride, v_stride, page_table, seqlens, cu_seqlens, page_size, T, B, Hkv, d,
                       max_pages_per_seq, num_pages, kv_format="bf16", k_descale=1.0, v_descale=1.0, stream=None,
                       raise_on_error=True):
    """Cached tokens back as bf16 rows; see ``attn_kv_read_paged`` in include/attn.h."""
    rc = lib.attn_kv_read_paged(_ptr(k_cache), _ptr(v_cache), _ptr(k), _ptr(v), int(k_stride), int(v_stride),
                                _ptr(page_table), _ptr(seqlens), _ptr(cu_seqlens), int(page_size), int(T), int(B), int(Hkv),
                                int(d), int(max_pages_per_seq), int(num_pages), _code(KV_FORMATS, kv_format),
                                float(k_descale), float(v_descale), _stream(stream))
    return _check(rc, "attn_kv_read_paged", raise_on_error)


def attn_decode_paged_tree(q, k_cache, v_cache, page_table, seqlens, cu_seqlens, tree_mask, mask_words, page_size, o, lse,
                           stream, T, B, max_q, Hq, Hkv, d, max_pages_per_seq, num_pages, scale, num_splits=0,
                           kv_format="bf16", k_descale=1.0, v_descale=1.0, raise_on_error=True):
    """Decode of a tree (or, without a mask, a chain) of drafted tokens per sequence; see
    ``attn_decode_paged_tree`` in include/attn.h."""
    rc = lib.attn_decode_paged_tree(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seqlens), _ptr(cu_seqlens),
                                    _ptr(tree_mask), int(mask_words), int(page_size), _ptr(o), _ptr(lse), _stream(stream),
                                    int(T), int(B), int(max_q), int(Hq), int(Hkv), int(d), int(max_pages_per_seq),
                                    int(num_pages), float(scale), int(num_splits), _code(KV_FORMATS, kv_format),
                                    float(k_descale), float(v_descale))
    return _check(rc, "attn_decode_paged_tree", raise_on_error)


def attn_qk_norm_rope(q, k, q_out, k_out, q_weight, k_weight, eps, positions, inv_freq, T, Hq, Hk, d, rot_begin, rot_dim, q_stride,
                      k_stride, q_out_stride, k_out_stride, elem_type="bf16", interleaved=0, amplitude=1.0, stream=None,
                      raise_on_error=True):
    """Norms of the heads of q and k and their rotary positions in one pass; see ``attn_qk_norm_rope`` in
    include/attn.h. ``elem_type`` is "bf16" or "f32" (or the ATTN_TYPE_* code)."""
    rc = lib.attn_qk_norm_rope(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _ptr(q_weight), _ptr(k_weight), float(eps),
                               _ptr(positions), _ptr(inv_freq), int(T), int(Hq), int(Hk), int(d), int(rot_begin), int(rot_dim),
                               int(q_stride), int(k_stride), int(q_out_stride), int(k_out_stride), _code(ELEM_TYPES, elem_type),
                               int(interleaved), float(amplitude), _stream(stream))
    return _check(rc, "attn_qk_norm_rope", raise_on_error)


def attn_qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight, k_weight, eps, positions, inv_freq, dq, dk, dq_weight, dk_weight, T, Hq, Hk, d,
                          rot_begin, rot_dim, q_stride, k_stride, dq_out_stride, dk_out_stride, dq_stride, dk_stride, elem_type="bf16",
                          interleaved=0, amplitude=1.0, stream=None, raise_on_error=True):
    """Gradient of ``attn_qk_norm_rope``; see ``attn_qk_norm_rope_bwd`` in include/attn.h."""
    rc = lib.attn_qk_norm_rope_bwd(_ptr(q), _ptr(k), _ptr(dq_out), _ptr(dk_out), _ptr(q_weight), _ptr(k_weight), float(eps),
                                   _ptr(positions), _ptr(inv_freq), _ptr(dq), _ptr(dk), _ptr(dq_weight), _ptr(dk_weight), int(T),
                                   int(Hq), int(Hk), int(d), int(rot_begin), int(rot_dim), int(q_stride), int(k_stride),
                                   int(dq_out_stride), int(dk_out_stride), int(dq_stride), int(dk_stride),
                                   _code(ELEM_TYPES, elem_type), int(interleaved), float(amplitude), _stream(stream))
    return _check(rc, "attn_qk_norm_rope_bwd", raise_on_error)


def attn_kv_score_paged(q, lse, k_cache, score, page_table, seqlens, cu_seqlens, page_size, T, B, max_q, Hq, Hkv, d, max_pages_per_seq,
                        num_pages, scale, decay=1.0, kv_format="bf16", k_descale=1.0, stream=None, raise_on_error=True):
    """Attention weight per cached token, added to its sums; see ``attn_kv_score_paged`` in include/attn.h."""
    rc = lib.attn_kv_score_paged(_ptr(q), _ptr(lse), _ptr(k_cache), _ptr(score), _ptr(page_table), _ptr(seqlens), _ptr(cu_seqlens),
                                 int(page_size), int(T), int(B), int(max_q), int(Hq), int(Hkv), int(d), int(max_pages_per_seq),
                                 int(num_pages), float(scale), float(decay), _code(KV_FORMATS, kv_format), float(k_descale),
                                 _stream(stream))
    return _check(rc, "attn_kv_score_paged", raise_on_error)


def attn_kv_select_paged(score, page_table, seqlens, kept, new_seqlens, page_size, B, Hkv, max_pages_per_seq, num_pages, budget,
                         sinks=0, recent=0, stream=None, raise_on_error=True):
    """The cached tokens that stay within ``budget``; see ``attn_kv_select_paged`` in include/attn.h."""
    rc = lib.attn_kv_select_paged(_ptr(score), _ptr(page_table), _ptr(seqlens), _ptr(kept), _ptr(new_seqlens), int(page_size), int(B),
                                  int(Hkv), int(max_pages_per_seq), int(num_pages), int(budget), int(sinks), int(recent),
                                  _stream(stream))
    return _check(rc, "attn_kv_select_paged", raise_on_error)


def attn_kv_compact_paged(k_cache, v_cache, score, kept, new_seqlens, page_table, page_size, B, Hkv, d, max_pages_per_seq, num_pages,
                          budget, kv_format="bf16", stream=None, raise_on_error=True):
    """The kept tokens to their slots, in place; see ``attn_kv_compact_paged`` in include/attn.h."""
    rc = lib.attn_kv_compact_paged(_ptr(k_cache), _ptr(v_cache), _ptr(score), _ptr(kept), _ptr(new_seqlens), _ptr(page_table),
                                   int(page_size), int(B), int(Hkv), int(d), int(max_pages_per_seq), int(num_pages), int(budget),
                                   _code(KV_FORMATS, kv_format), _stream(stream))
    return _check(rc, "attn_kv_compact_paged", raise_on_error)


def attn_decode_plan(B, Hq, Hkv, max_pages_per_seq, page_size, num_splits=0, num_sms=0):
    """(chunk tokens per split, splits per sequence) chosen by the library."""
    c, s = _i(), _i()
    rc = lib.attn_decode_plan(int(B), int(Hq), int(Hkv), int(max_pages_per_seq), int(page_size), int(num_splits),
                              int(num_sms), ctypes.byref(c), ctypes.byref(s))
    _check(rc, "attn_decode_plan", True)
    return c.value, s.value


def attn_decode_workspace_bytes(B, Hq, d, max_splits) -> int:
    """Bytes of split-KV workspace attn_decode_paged takes for these sizes."""
    return int(lib.attn_decode_workspace_bytes(int(B), int(Hq), int(d), int(max_splits)))


def attn_get_device_status(stream=None) -> int:
    """Synchronise the stream, read and clear the device status word (returns the status code)."""
    return lib.attn_get_device_status(_stream(stream))


def attn_set_option(name: str, value: float):
    _check(lib.attn_set_option(name.encode(), float(value)), f"attn_set_option({name})", True)


def attn_get_option(name: str) -> float:
    v = _d()
    _check(lib.attn_get_option(name.encode(), ctypes.byref(v)), f"attn_get_option({name})", True)
    return v.value


def attn_read_counters():
    out = (ctypes.c_ulonglong * 6)()
    _check(lib.attn_read_counters(out, 6), "attn_read_counters", True)
    return list(out)


def attn_debug_exp2(x, y, n, mode, stream=None):
    return _check(lib.attn_debug_exp2(_ptr(x), _ptr(y), int(n), int(mode), _stream(stream)), "attn_debug_exp2", True)


def attn_debug_watchdog(limit_ns, stream=None):
    return _check(lib.attn_debug_watchdog(int(limit_ns), _stream(stream)), "attn_debug_watchdog", True)


def attn_version() -> str:
    return lib.attn_version().decode()
