"""Python binding of libvqattn.so, the sm_103a VQ KV-cache decode-attention library.

Two layers, both argument marshalling only (every step of the computation runs
in the library's CUDA kernels):

* ``vq_*`` functions mirror the C ABI of include/vqattn.h one to one: they take
  device pointers as Python ints and raise :class:`VQError` on a non-OK status.
* ``encode_kv`` / ``decode_attention`` / ``append_slots`` / ``rotary`` / ``append_kv`` /
  ``tree_attention`` / ``keep_tokens`` /
  ``alloc_pools`` / ``alloc_workspace`` and their like accept torch tensors (PyTorch supplies device memory and streams), check
  dtypes, shapes and devices, and pass their pointers to the ``vq_*`` calls.

There is no fallback: if libvqattn.so has not been built the first call raises.
Build it with ``python -m bit_vector_quantized_gb300.build``.
"""
from __future__ import annotations

import array
import ctypes
import os
from typing import NamedTuple, Optional, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvqattn.so")

VQ_OK = 0
VQ_ERR_INVALID_ARG = -1
VQ_ERR_UNSUPPORTED = -2
VQ_ERR_WORKSPACE = -3
VQ_ERR_CUDA = -4
STATUS_NAMES = {0: "VQ_OK", -1: "VQ_ERR_INVALID_ARG", -2: "VQ_ERR_UNSUPPORTED",
                -3: "VQ_ERR_WORKSPACE", -4: "VQ_ERR_CUDA"}
VQ_DEV_OK, VQ_DEV_BAD_PAGE, VQ_DEV_BAD_SLOT, VQ_DEV_TIMEOUT, VQ_DEV_BAD_CONFIG = 0, 1, 2, 3, 4
VQ_DEV_BAD_LENGTH, VQ_DEV_NO_PAGES = 5, 6
VQ_FP16, VQ_BF16 = 0, 1
VQ_ROTARY_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3, "wavelength": 4}

# every symbol include/vqattn.h declares
EXPORTED = ("vq_code_row_bytes", "vq_check_layout", "vq_encode_kv", "vq_decode_workspace_bytes",
            "vq_default_num_splits", "vq_decode_units_balanced", "vq_decode_attention",
            "vq_decode_partial",
            "vq_decode_partial_method", "vq_decode_combine", "vq_decode_step", "vq_dequantize_kv",
            "vq_decode_residual_workspace_bytes", "vq_decode_attention_residual",
            "vq_decode_attention_static", "vq_static_scratch_bytes", "vq_chunk_attention",
            "vq_chunk_workspace_bytes", "vq_append_slots", "vq_rotary", "vq_tree_attention",
            "vq_tree_workspace_bytes", "vq_append_kv", "vq_keep_tokens", "vq_last_error", "vq_version")


class VQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class vq_layout(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("k_sub", ctypes.c_int32),
                ("k_bits", ctypes.c_int32), ("v_sub", ctypes.c_int32),
                ("v_bits", ctypes.c_int32), ("page_size", ctypes.c_int32)]

    def __repr__(self):
        return "vq_layout(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


def make_layout(head_dim=128, num_q_heads=32, num_kv_heads=8, k_sub=4, k_bits=8, v_sub=4,
                v_bits=8, page_size=256) -> vq_layout:
    return vq_layout(head_dim, num_q_heads, num_kv_heads, k_sub, k_bits, v_sub, v_bits, page_size)


class vq_rotary_config(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_double), ("low_turns", ctypes.c_double),
                ("high_turns", ctypes.c_double), ("attention_factor", ctypes.c_double)]


def make_rotary(head_dim=128, rotary_dim=128, interleaved=False, base=10000.0, scaling="none",
                factor=1.0, original_len=8192, low_turns=1.0, high_turns=32.0,
                attention_factor=1.0) -> vq_rotary_config:
    """Rotary positions (see vq_rotary_config in the header); scaling is "none", "linear",
    "base", "parts" or "wavelength"."""
    if scaling not in VQ_ROTARY_SCALINGS:
        raise ValueError(f"scaling {scaling!r} is not one of {sorted(VQ_ROTARY_SCALINGS)}")
    return vq_rotary_config(head_dim, rotary_dim, int(bool(interleaved)),
                            VQ_ROTARY_SCALINGS[scaling], base, factor, original_len, low_turns,
                            high_turns, attention_factor)


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m bit_vector_quantized_gb300.build` (no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        LP = ctypes.POINTER(vq_layout)
        sig = {
            "vq_code_row_bytes": (SZ, [I32, I32, I32]),
            "vq_check_layout": (I32, [LP, I32]),
            "vq_encode_kv": (I32, [LP, I32, P, P, P, P, P, P, P, P, I64, P, P]),
            "vq_dequantize_kv": (I32, [LP, I32, P, P, P, P, P, P, I64, P, P, P, P]),
            "vq_decode_residual_workspace_bytes": (SZ, [LP, I32, I32, I32, I32]),
            "vq_decode_attention_residual": (I32, [LP, I32, P, P, P, P, P, P, I64, P, I32, P, I32,
                                                   P, P, P, I32, ctypes.c_float, I32, P, P, SZ,
                                                   P, P]),
            "vq_decode_workspace_bytes": (SZ, [LP, I32, I32, I32, I32]),
            "vq_default_num_splits": (I32, [LP, I32, I32, I32]),
            "vq_decode_units_balanced": (I32, [LP, I32, I32, I32, I32]),
            "vq_decode_attention": (I32, [LP, I32, P, P, P, P, P, P, I64, P, I32, P, I32,
                                          ctypes.c_float, I32, P, P, SZ, P, P]),
            "vq_decode_partial": (I32, [LP, I32, P, P, P, P, P, P, I64, P, I32, P, I32,
                                        ctypes.c_float, I32, P, SZ, P, P]),
            "vq_decode_partial_method": (I32, [LP, I32, P, P, P, P, P, P, I64, P, I32, P, I32,
                                               ctypes.c_float, I32, I32, P, SZ, P, P]),
            "vq_decode_combine": (I32, [LP, I32, I32, I32, P, SZ, P, P]),
            "vq_decode_step": (I32, [LP, I32, P, P, P, P, P, P, P, P, I64, P, I32, P, I32,
                                     ctypes.c_float, I32, P, P, SZ, P, P]),
            "vq_decode_attention_static": (I32, [LP, I32, P, P, P, P, P, P, I64, P, I32, P, I32,
                                                 ctypes.c_float, I32, P, P, P]),
            "vq_static_scratch_bytes": (SZ, []),
            "vq_chunk_attention": (I32, [LP, I32, I32, P, P, P, P, P, P, I64, P, I32, P, I32, P, I32,
                                         I32, I32, ctypes.c_float, P, P, SZ, P, P]),
            "vq_chunk_workspace_bytes": (SZ, [LP, I32, I32, I32, I32, I32]),
            "vq_append_slots": (I32, [I32, P, P, P, I32, P, I32, P, I32, I64, I32, P, P, P, P, P,
                                      P, P]),
            "vq_rotary": (I32, [ctypes.POINTER(vq_rotary_config), I32, P, I32, P, I64, I32, P, P,
                                I64, P, I64, I32, P, P, P]),
            "vq_tree_attention": (I32, [LP, I32, I32, P, P, P, P, P, P, I64, P, I32, P, I32, P, I32, P, I32, P,
                                        I32, I32, ctypes.c_float, P, P, SZ, P, P]),
            "vq_tree_workspace_bytes": (SZ, [LP, I32, I32, I32, I32, I32]),
            "vq_append_kv": (I32, [LP, ctypes.POINTER(vq_rotary_config), I32, P, P, I32, P, I64, P, I64, P, I64,
                                   P, P, P, P, P, P, I64, P, P]),
            "vq_keep_tokens": (I32, [LP, I32, P, P, P, I32, P, P, I32, I64, I32, P, P, P, I32, P, P, P, P, P]),
            "vq_last_error": (ctypes.c_char_p, []),
            "vq_version": (ctypes.c_char_p, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(st: int) -> None:
    if st != VQ_OK:
        raise VQError(st, lib().vq_last_error().decode())


def _ptr(x) -> Optional[int]:
    return None if x is None or x == 0 else int(x)


# ------------------------------------------------------------- C ABI layer ---

def vq_code_row_bytes(head_dim: int, sub: int, bits: int) -> int:
    return int(lib().vq_code_row_bytes(head_dim, sub, bits))


def vq_check_layout(layout: vq_layout, for_decode: bool = False) -> None:
    _check(lib().vq_check_layout(ctypes.byref(layout), int(for_decode)))


def vq_encode_kv(layout, num_tokens, k, v, slot_mapping, lambda_, codebook_k, codebook_v,
                 k_pool, v_pool, num_pages, status=None, stream=None) -> None:
    _check(lib().vq_encode_kv(ctypes.byref(layout), num_tokens, _ptr(k), _ptr(v),
                              _ptr(slot_mapping), _ptr(lambda_), _ptr(codebook_k),
                              _ptr(codebook_v), _ptr(k_pool), _ptr(v_pool), num_pages,
                              _ptr(status), _ptr(stream)))


def vq_dequantize_kv(layout, num_tokens, slot_mapping, lambda_, codebook_k, codebook_v, k_pool,
                     v_pool, num_pages, k_out, v_out, status=None, stream=None) -> None:
    _check(lib().vq_dequantize_kv(ctypes.byref(layout), num_tokens, _ptr(slot_mapping),
                                  _ptr(lambda_), _ptr(codebook_k), _ptr(codebook_v), _ptr(k_pool),
                                  _ptr(v_pool), num_pages, _ptr(k_out), _ptr(v_out), _ptr(status),
                                  _ptr(stream)))


def vq_decode_residual_workspace_bytes(layout, batch, max_seq_len, num_splits=0, num_sms=0) -> int:
    return int(lib().vq_decode_residual_workspace_bytes(ctypes.byref(layout), batch, max_seq_len,
                                                        num_splits, num_sms))


def vq_decode_attention_residual(layout, batch, q, lambda_, codebook_k, codebook_v, k_pool,
                                 v_pool, num_pages, page_table, max_pages_per_seq, seq_lens,
                                 max_seq_len, k_res, v_res, res_lens, res_capacity, softmax_scale,
                                 num_splits, out, workspace, workspace_bytes, status=None,
                                 stream=None) -> None:
    _check(lib().vq_decode_attention_residual(
        ctypes.byref(layout), batch, _ptr(q), _ptr(lambda_), _ptr(codebook_k), _ptr(codebook_v),
        _ptr(k_pool), _ptr(v_pool), num_pages, _ptr(page_table), max_pages_per_seq,
        _ptr(seq_lens), max_seq_len, _ptr(k_res), _ptr(v_res), _ptr(res_lens), res_capacity,
        float(softmax_scale), num_splits, _ptr(out), _ptr(workspace), workspace_bytes,
        _ptr(status), _ptr(stream)))


def vq_decode_workspace_bytes(layout, batch, max_seq_len, num_splits=0, num_sms=0) -> int:
    return int(lib().vq_decode_workspace_bytes(ctypes.byref(layout), batch, max_seq_len,
                                               num_splits, num_sms))


def vq_default_num_splits(layout, batch, max_seq_len, num_sms=0) -> int:
    return int(lib().vq_default_num_splits(ctypes.byref(layout), batch, max_seq_len, num_sms))


def vq_decode_units_balanced(layout, batch, max_seq_len, num_splits=0, num_sms=0) -> int:
    return int(lib().vq_decode_units_balanced(ctypes.byref(layout), batch, max_seq_len,
                                              num_splits, num_sms))


def vq_decode_attention(layout, batch, q, lambda_, codebook_k, codebook_v, k_pool, v_pool,
                        num_pages, page_table, max_pages_per_seq, seq_lens, max_seq_len,
                        softmax_scale, num_splits, out, workspace, workspace_bytes,
                        status=None, stream=None) -> None:
    _check(lib().vq_decode_attention(ctypes.byref(layout), batch, _ptr(q), _ptr(lambda_),
                                     _ptr(codebook_k), _ptr(codebook_v), _ptr(k_pool),
                                     _ptr(v_pool), num_pages, _ptr(page_table), max_pages_per_seq,
                                     _ptr(seq_lens), max_seq_len, float(softmax_scale),
                                     num_splits, _ptr(out), _ptr(workspace), workspace_bytes,
                                     _ptr(status), _ptr(stream)))


def vq_decode_partial(layout, batch, q, lambda_, codebook_k, codebook_v, k_pool, v_pool,
                      num_pages, page_table, max_pages_per_seq, seq_lens, max_seq_len,
                      softmax_scale, num_splits, workspace, workspace_bytes, status=None,
                      stream=None) -> None:
    _check(lib().vq_decode_partial(ctypes.byref(layout), batch, _ptr(q), _ptr(lambda_),
                                   _ptr(codebook_k), _ptr(codebook_v), _ptr(k_pool), _ptr(v_pool),
                                   num_pages, _ptr(page_table), max_pages_per_seq, _ptr(seq_lens),
                                   max_seq_len, float(softmax_scale), num_splits, _ptr(workspace),
                                   workspace_bytes, _ptr(status), _ptr(stream)))


VQ_METHOD_GATHER, VQ_METHOD_LUT, VQ_METHOD_BINS = 0, 1, 2


def vq_decode_partial_method(layout, batch, q, lambda_, codebook_k, codebook_v, k_pool, v_pool,
                             num_pages, page_table, max_pages_per_seq, seq_lens, max_seq_len,
                             softmax_scale, num_splits, method, workspace, workspace_bytes,
                             status=None, stream=None) -> None:
    _check(lib().vq_decode_partial_method(
        ctypes.byref(layout), batch, _ptr(q), _ptr(lambda_), _ptr(codebook_k), _ptr(codebook_v),
        _ptr(k_pool), _ptr(v_pool), num_pages, _ptr(page_table), max_pages_per_seq, _ptr(seq_lens),
        max_seq_len, float(softmax_scale), num_splits, method, _ptr(workspace), workspace_bytes,
        _ptr(status), _ptr(stream)))


def vq_decode_combine(layout, batch, max_seq_len, num_splits, workspace, workspace_bytes, out,
                      stream=None) -> None:
    _check(lib().vq_decode_combine(ctypes.byref(layout), batch, max_seq_len, num_splits,
                                   _ptr(workspace), workspace_bytes, _ptr(out), _ptr(stream)))


def vq_decode_step(layout, batch, q, k_new, v_new, lambda_, codebook_k, codebook_v, k_pool,
                   v_pool, num_pages, page_table, max_pages_per_seq, seq_lens, max_seq_len,
                   softmax_scale, num_splits, out, workspace, workspace_bytes, status=None,
                   stream=None) -> None:
    """Append the new token of every sequence (position seq_lens - 1), then decode attention."""
    _check(lib().vq_decode_step(ctypes.byref(layout), batch, _ptr(q), _ptr(k_new), _ptr(v_new),
                                _ptr(lambda_), _ptr(codebook_k), _ptr(codebook_v), _ptr(k_pool),
                                _ptr(v_pool), num_pages, _ptr(page_table), max_pages_per_seq,
                                _ptr(seq_lens), max_seq_len, float(softmax_scale), num_splits,
                                _ptr(out), _ptr(workspace), workspace_bytes, _ptr(status),
                                _ptr(stream)))


def vq_decode_attention_static(layout, batch, q, lambda_, codebook_k, codebook_v, k_pool, v_pool,
                               num_pages, page_table, max_pages_per_seq, seq_lens, max_seq_len,
                               softmax_scale, num_splits, out, status=None, stream=None) -> None:
    """vq_decode_attention for callers that cannot allocate: no workspace argument;
    the split partials live in the library's fixed device array (see the header)."""
    _check(lib().vq_decode_attention_static(ctypes.byref(layout), batch, _ptr(q), _ptr(lambda_),
                                            _ptr(codebook_k), _ptr(codebook_v), _ptr(k_pool),
                                            _ptr(v_pool), num_pages, _ptr(page_table),
                                            max_pages_per_seq, _ptr(seq_lens), max_seq_len,
                                            float(softmax_scale), num_splits, _ptr(out),
                                            _ptr(status), _ptr(stream)))


def vq_static_scratch_bytes() -> int:
    return int(lib().vq_static_scratch_bytes())


def vq_chunk_attention(layout, batch, num_tokens, q, lambda_, codebook_k, codebook_v, k_pool,
                       v_pool, num_pages, page_table, max_pages_per_seq, seq_lens, max_seq_len,
                       cu_new_lens, max_new_len, window, num_sinks, softmax_scale, out, workspace,
                       workspace_bytes, status=None, stream=None) -> None:
    _check(lib().vq_chunk_attention(
        ctypes.byref(layout), batch, num_tokens, _ptr(q), _ptr(lambda_), _ptr(codebook_k),
        _ptr(codebook_v), _ptr(k_pool), _ptr(v_pool), num_pages, _ptr(page_table),
        max_pages_per_seq, _ptr(seq_lens), max_seq_len, _ptr(cu_new_lens), max_new_len, window,
        num_sinks, float(softmax_scale), _ptr(out), _ptr(workspace), workspace_bytes,
        _ptr(status), _ptr(stream)))


def vq_chunk_workspace_bytes(layout, batch, num_tokens, max_seq_len, max_new_len,
                             num_sms=0) -> int:
    return int(lib().vq_chunk_workspace_bytes(ctypes.byref(layout), batch, num_tokens,
                                              max_seq_len, max_new_len, num_sms))


def vq_append_slots(batch, seq_lens, new_lens, page_table, max_pages_per_seq, free_pages,
                    free_capacity, num_free, page_size, num_pages, max_tokens, seq_lens_out,
                    num_free_out, cu_new_lens, slot_mapping, positions, status=None,
                    stream=None) -> None:
    _check(lib().vq_append_slots(batch, _ptr(seq_lens), _ptr(new_lens), _ptr(page_table),
                                 max_pages_per_seq, _ptr(free_pages), free_capacity,
                                 _ptr(num_free), page_size, num_pages, max_tokens,
                                 _ptr(seq_lens_out), _ptr(num_free_out), _ptr(cu_new_lens),
                                 _ptr(slot_mapping), _ptr(positions), _ptr(status), _ptr(stream)))


def vq_rotary(config, num_tokens, positions, dtype, q, q_stride, num_q_heads, q_out, k, k_stride,
              v, v_stride, num_kv_heads, k_out, v_out, stream=None) -> None:
    _check(lib().vq_rotary(ctypes.byref(config), num_tokens, _ptr(positions), dtype, _ptr(q),
                           q_stride, num_q_heads, _ptr(q_out), _ptr(k), k_stride, _ptr(v),
                           v_stride, num_kv_heads, _ptr(k_out), _ptr(v_out), _ptr(stream)))


def vq_tree_attention(layout, batch, num_tokens, q, lambda_, codebook_k, codebook_v, k_pool, v_pool, num_pages, page_table,
                      max_pages_per_seq, seq_lens, max_seq_len, cu_new_lens, max_new_len, tree_masks, mask_words, positions,
                      window, num_sinks, softmax_scale, out, workspace, workspace_bytes, status=None, stream=None) -> None:
    _check(lib().vq_tree_attention(
        ctypes.byref(layout), batch, num_tokens, _ptr(q), _ptr(lambda_), _ptr(codebook_k),
        _ptr(codebook_v), _ptr(k_pool), _ptr(v_pool), num_pages, _ptr(page_table),
        max_pages_per_seq, _ptr(seq_lens), max_seq_len, _ptr(cu_new_lens), max_new_len,
        _ptr(tree_masks), mask_words, _ptr(positions), window, num_sinks, float(softmax_scale),
        _ptr(out), _ptr(workspace), workspace_bytes, _ptr(status), _ptr(stream)))


def vq_tree_workspace_bytes(layout, batch, num_tokens, max_seq_len, max_new_len, num_sms=0) -> int:
    return int(lib().vq_tree_workspace_bytes(ctypes.byref(layout), batch, num_tokens, max_seq_len,
                                             max_new_len, num_sms))


def vq_append_kv(layout, config, num_tokens, positions, slot_mapping, dtype, q, q_stride, k, k_stride,
                 v, v_stride, lambda_, codebook_k, codebook_v, q_out, k_pool, v_pool, num_pages,
                 status=None, stream=None) -> None:
    _check(lib().vq_append_kv(ctypes.byref(layout), ctypes.byref(config), num_tokens, _ptr(positions),
                              _ptr(slot_mapping), dtype, _ptr(q), q_stride, _ptr(k), k_stride, _ptr(v),
                              v_stride, _ptr(lambda_), _ptr(codebook_k), _ptr(codebook_v), _ptr(q_out),
                              _ptr(k_pool), _ptr(v_pool), num_pages, _ptr(status), _ptr(stream)))


def vq_keep_tokens(layout, batch, seq_lens, cu_new_lens, keep, max_keep, keep_lens, page_table,
                   max_pages_per_seq, num_pages, k_pools, v_pools, free_pages, free_capacity, num_free,
                   seq_lens_out, num_free_out, status=None, stream=None) -> None:
    """k_pools, v_pools: device pointers of the layers' pools, as many of the one as of the other."""
    if len(k_pools) != len(v_pools):
        raise ValueError("k_pools and v_pools have different numbers of layers")
    kp, vp = ((ctypes.c_void_p * len(x))(*map(_ptr, x)) for x in (k_pools, v_pools))
    _check(lib().vq_keep_tokens(ctypes.byref(layout), batch, _ptr(seq_lens), _ptr(cu_new_lens), _ptr(keep),
                                max_keep, _ptr(keep_lens), _ptr(page_table), max_pages_per_seq, num_pages,
                                len(k_pools), kp, vp, _ptr(free_pages), free_capacity, _ptr(num_free),
                                _ptr(seq_lens_out), _ptr(num_free_out), _ptr(status), _ptr(stream)))


def vq_last_error() -> str:
    return lib().vq_last_error().decode()


def vq_version() -> str:
    return lib().vq_version().decode()


# ------------------------------------------------------------ torch layer ---

def _torch():
    import torch
    return torch


def _dev_ptr(t, dtype, name, shape=None):
    torch = _torch()
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _stream(stream) -> int:
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def row_bytes(layout: vq_layout) -> Tuple[int, int]:
    return (vq_code_row_bytes(layout.head_dim, layout.k_sub, layout.k_bits),
            vq_code_row_bytes(layout.head_dim, layout.v_sub, layout.v_bits))


def alloc_pools(layout: vq_layout, num_pages: int, device="cuda", zero: bool = False):
    """(k_pool, v_pool) uint8 tensors [num_pages][Hkv][P][row_bytes]."""
    torch = _torch()
    kr, vr = row_bytes(layout)
    mk = torch.zeros if zero else torch.empty
    shape = (num_pages, layout.num_kv_heads, layout.page_size)
    return (mk(shape + (kr,), dtype=torch.uint8, device=device),
            mk(shape + (vr,), dtype=torch.uint8, device=device))


def alloc_workspace(layout: vq_layout, batch: int, max_seq_len: int, num_splits: int = 0,
                    device="cuda"):
    torch = _torch()
    n = vq_decode_workspace_bytes(layout, batch, max_seq_len, num_splits)
    if n == 0 and batch > 0:
        raise VQError(VQ_ERR_INVALID_ARG, "cannot size the workspace")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def encode_kv(layout: vq_layout, k, v, slot_mapping, lambda_, codebook_k, codebook_v,
              k_pool, v_pool, status=None, stream=None) -> None:
    """Encode fp16 keys/values [T][Hkv][D] into the pools at slot_mapping (int64 [T])."""
    torch = _torch()
    ref = k if k is not None else v
    T = ref.shape[0]
    D, H = layout.head_dim, layout.num_kv_heads
    vq_encode_kv(layout, T,
                 _dev_ptr(k, torch.float16, "k", (T, H, D)),
                 _dev_ptr(v, torch.float16, "v", (T, H, D)),
                 _dev_ptr(slot_mapping, torch.int64, "slot_mapping", (T,)),
                 _dev_ptr(lambda_, torch.float32, "lambda", (H, D)) if k is not None else None,
                 _dev_ptr(codebook_k, torch.float16, "codebook_k",
                          (1 << layout.k_bits, layout.k_sub)) if k is not None else None,
                 _dev_ptr(codebook_v, torch.float16, "codebook_v",
                          (1 << layout.v_bits, layout.v_sub)) if v is not None else None,
                 _dev_ptr(k_pool, torch.uint8, "k_pool") if k is not None else None,
                 _dev_ptr(v_pool, torch.uint8, "v_pool") if v is not None else None,
                 (k_pool if k is not None else v_pool).shape[0],
                 _dev_ptr(status, torch.int32, "status", (1,)), _stream(stream))


def dequantize_kv(layout: vq_layout, slot_mapping, lambda_, codebook_k, codebook_v, k_pool,
                  v_pool, keys: bool = True, values: bool = True, k_out=None, v_out=None,
                  status=None, stream=None):
    """(K^, V^) fp16 [T][Hkv][D] read back from the pools at slot_mapping (int64 [T]);
    keys in the original space.  A half not asked for is returned as None."""
    torch = _torch()
    T = slot_mapping.shape[0]
    D, H = layout.head_dim, layout.num_kv_heads
    dev = slot_mapping.device
    if keys and k_out is None:
        k_out = torch.empty((T, H, D), dtype=torch.float16, device=dev)
    if values and v_out is None:
        v_out = torch.empty((T, H, D), dtype=torch.float16, device=dev)
    k_out, v_out = (k_out if keys else None), (v_out if values else None)
    vq_dequantize_kv(layout, T, _dev_ptr(slot_mapping, torch.int64, "slot_mapping", (T,)),
                     _dev_ptr(lambda_, torch.float32, "lambda", (H, D)) if keys else None,
                     _dev_ptr(codebook_k, torch.float16, "codebook_k",
                              (1 << layout.k_bits, layout.k_sub)) if keys else None,
                     _dev_ptr(codebook_v, torch.float16, "codebook_v",
                              (1 << layout.v_bits, layout.v_sub)) if values else None,
                     _dev_ptr(k_pool, torch.uint8, "k_pool") if keys else None,
                     _dev_ptr(v_pool, torch.uint8, "v_pool") if values else None,
                     (k_pool if keys else v_pool).shape[0],
                     _dev_ptr(k_out, torch.float16, "k_out", (T, H, D)) if keys else None,
                     _dev_ptr(v_out, torch.float16, "v_out", (T, H, D)) if values else None,
                     _dev_ptr(status, torch.int32, "status", (1,)), _stream(stream))
    return k_out, v_out


def decode_attention(layout: vq_layout, q, lambda_, codebook_k, codebook_v, k_pool, v_pool,
                     page_table, seq_lens, max_seq_len: int, out=None, workspace=None,
                     softmax_scale: float = 0.0, num_splits: int = 0, status=None,
                     stream=None):
    """fp16 [B][Hq][D] attention of queries q [B][Hq][D] over the quantized pools."""
    torch = _torch()
    B = q.shape[0]
    D = layout.head_dim
    if out is None:
        out = torch.empty((B, layout.num_q_heads, D), dtype=torch.float16, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(layout, B, max_seq_len, num_splits, q.device)
    vq_decode_attention(layout, B,
                        _dev_ptr(q, torch.float16, "q", (B, layout.num_q_heads, D)),
                        _dev_ptr(lambda_, torch.float32, "lambda", (layout.num_kv_heads, D)),
                        _dev_ptr(codebook_k, torch.float16, "codebook_k",
                                 (1 << layout.k_bits, layout.k_sub)),
                        _dev_ptr(codebook_v, torch.float16, "codebook_v",
                                 (1 << layout.v_bits, layout.v_sub)),
                        _dev_ptr(k_pool, torch.uint8, "k_pool"),
                        _dev_ptr(v_pool, torch.uint8, "v_pool"), k_pool.shape[0],
                        _dev_ptr(page_table, torch.int32, "page_table"), page_table.shape[1],
                        _dev_ptr(seq_lens, torch.int32, "seq_lens", (B,)), max_seq_len,
                        softmax_scale, num_splits,
                        _dev_ptr(out, torch.float16, "out", (B, layout.num_q_heads, D)),
                        _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                        _dev_ptr(status, torch.int32, "status", (1,)), _stream(stream))
    return out


def decode_attention_method(layout: vq_layout, q, lambda_, codebook_k, codebook_v, k_pool,
                            v_pool, page_table, seq_lens, max_seq_len: int, method: int,
                            out=None, workspace=None, softmax_scale: float = 0.0,
                            num_splits: int = 0, status=None, stream=None):
    """decode_attention with an explicit score / P.V method (vq_decode_partial_method,
    then vq_decode_combine)."""
    torch = _torch()
    B = q.shape[0]
    D = layout.head_dim
    if out is None:
        out = torch.empty((B, layout.num_q_heads, D), dtype=torch.float16, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(layout, B, max_seq_len, num_splits, q.device)
    st = _stream(stream)
    vq_decode_partial_method(layout, B,
                             _dev_ptr(q, torch.float16, "q", (B, layout.num_q_heads, D)),
                             _dev_ptr(lambda_, torch.float32, "lambda", (layout.num_kv_heads, D)),
                             _dev_ptr(codebook_k, torch.float16, "codebook_k",
                                      (1 << layout.k_bits, layout.k_sub)),
                             _dev_ptr(codebook_v, torch.float16, "codebook_v",
                                      (1 << layout.v_bits, layout.v_sub)),
                             _dev_ptr(k_pool, torch.uint8, "k_pool"),
                             _dev_ptr(v_pool, torch.uint8, "v_pool"), k_pool.shape[0],
                             _dev_ptr(page_table, torch.int32, "page_table"), page_table.shape[1],
                             _dev_ptr(seq_lens, torch.int32, "seq_lens", (B,)), max_seq_len,
                             softmax_scale, num_splits, method,
                             _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                             _dev_ptr(status, torch.int32, "status", (1,)), st)
    vq_decode_combine(layout, B, max_seq_len, num_splits,
                      _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                      _dev_ptr(out, torch.float16, "out", (B, layout.num_q_heads, D)), st)
    return out


def decode_attention_residual(layout: vq_layout, q, lambda_, codebook_k, codebook_v, k_pool,
                              v_pool, page_table, seq_lens, max_seq_len: int, k_res, v_res,
                              res_lens, out=None, workspace=None, softmax_scale: float = 0.0,
                              num_splits: int = 0, status=None, stream=None):
    """fp16 [B][Hq][D] attention of q over the quantized pools (seq_lens tokens)
    plus the full-precision residual k_res / v_res [B][Hkv][capacity][D]
    (res_lens tokens), one softmax."""
    torch = _torch()
    B = q.shape[0]
    D, H = layout.head_dim, layout.num_kv_heads
    cap = k_res.shape[2]
    if out is None:
        out = torch.empty((B, layout.num_q_heads, D), dtype=torch.float16, device=q.device)
    if workspace is None:
        n = vq_decode_residual_workspace_bytes(layout, B, max_seq_len, num_splits)
        if n == 0 and B > 0:
            raise VQError(VQ_ERR_INVALID_ARG, "cannot size the workspace")
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    vq_decode_attention_residual(
        layout, B, _dev_ptr(q, torch.float16, "q", (B, layout.num_q_heads, D)),
        _dev_ptr(lambda_, torch.float32, "lambda", (H, D)),
        _dev_ptr(codebook_k, torch.float16, "codebook_k", (1 << layout.k_bits, layout.k_sub)),
        _dev_ptr(codebook_v, torch.float16, "codebook_v", (1 << layout.v_bits, layout.v_sub)),
        _dev_ptr(k_pool, torch.uint8, "k_pool"), _dev_ptr(v_pool, torch.uint8, "v_pool"),
        k_pool.shape[0], _dev_ptr(page_table, torch.int32, "page_table"), page_table.shape[1],
        _dev_ptr(seq_lens, torch.int32, "seq_lens", (B,)), max_seq_len,
        _dev_ptr(k_res, torch.float16, "k_res", (B, H, cap, D)),
        _dev_ptr(v_res, torch.float16, "v_res", (B, H, cap, D)),
        _dev_ptr(res_lens, torch.int32, "res_lens", (B,)), cap, softmax_scale, num_splits,
        _dev_ptr(out, torch.float16, "out", (B, layout.num_q_heads, D)),
        _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        _dev_ptr(status, torch.int32, "status", (1,)), _stream(stream))
    return out


def decode_step(layout: vq_layout, q, k_new, v_new, lambda_, codebook_k, codebook_v, k_pool,
                v_pool, page_table, seq_lens, max_seq_len: int, out=None, workspace=None,
                softmax_scale: float = 0.0, num_splits: int = 0, status=None, stream=None):
    """One decode step: append k_new / v_new [B][Hkv][D] as token seq_lens - 1 of each
    sequence, then fp16 [B][Hq][D] attention of q [B][Hq][D] over seq_lens tokens."""
    torch = _torch()
    B = q.shape[0]
    D, H = layout.head_dim, layout.num_kv_heads
    if out is None:
        out = torch.empty((B, layout.num_q_heads, D), dtype=torch.float16, device=q.device)
    if workspace is None:
        n = vq_decode_workspace_bytes(layout, B, max_seq_len, num_splits)
        if n == 0 and B > 0:
            raise VQError(VQ_ERR_INVALID_ARG, "cannot size the workspace")
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    vq_decode_step(layout, B,
                   _dev_ptr(q, torch.float16, "q", (B, layout.num_q_heads, D)),
                   _dev_ptr(k_new, torch.float16, "k_new", (B, H, D)),
                   _dev_ptr(v_new, torch.float16, "v_new", (B, H, D)),
                   _dev_ptr(lambda_, torch.float32, "lambda", (H, D)),
                   _dev_ptr(codebook_k, torch.float16, "codebook_k", (1 << layout.k_bits, layout.k_sub)),
                   _dev_ptr(codebook_v, torch.float16, "codebook_v", (1 << layout.v_bits, layout.v_sub)),
                   _dev_ptr(k_pool, torch.uint8, "k_pool"),
                   _dev_ptr(v_pool, torch.uint8, "v_pool"), k_pool.shape[0],
                   _dev_ptr(page_table, torch.int32, "page_table"), page_table.shape[1],
                   _dev_ptr(seq_lens, torch.int32, "seq_lens", (B,)), max_seq_len,
                   softmax_scale, num_splits,
                   _dev_ptr(out, torch.float16, "out", (B, layout.num_q_heads, D)),
                   _dev_ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                   _dev_ptr(status, torch.int32, "status", (1,)), _stream(stream))
    return out


# ------------------------------------------------- torch layer: serving step ---
# These calls run on the device of their tensors whatever the current one is, and
# make the outputs and workspaces that they are not given on the stream they run on.
# A decode step's calls take a few microseconds on the GPU, so the checks keep a
# short path: one comparison per property, and errors are told apart only on failure.

def _launch(device, stream, call):
    """call(raw stream) on `device` and `stream` (None: the device's current one); where either
    is not the current one it is entered first, so that what `call` allocates belongs to it."""
    torch = _torch()
    index = device.index
    if stream is None and index == torch.cuda.current_device():
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # torch's own short form
        return call(raw(index) if raw else torch.cuda.current_stream().cuda_stream)
    with torch.cuda.device(device):
        if stream is None:
            return call(torch.cuda.current_stream().cuda_stream)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _arg(t, dtype, name, device, shape=None):
    """data_ptr of a tensor argument (contiguous, of this type and shape, on this device)."""
    if t is None:
        return None
    if not (hasattr(t, "data_ptr") and t.dtype is dtype and t.device == device and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        _dev_ptr(t, dtype, name, shape)  # raises for all but the device
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.data_ptr()


def _need(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.device


def alloc_chunk_workspace(layout: vq_layout, batch: int, num_tokens: int, max_seq_len: int,
                          max_new_len: int, device="cuda"):
    torch = _torch()
    with torch.cuda.device(device):
        n = vq_chunk_workspace_bytes(layout, batch, num_tokens, max_seq_len, max_new_len)
        if n == 0:
            raise VQError(VQ_ERR_INVALID_ARG, "cannot size the workspace")
        return torch.empty(n, dtype=torch.uint8, device="cuda")


def chunk_attention(layout: vq_layout, q, lambda_, codebook_k, codebook_v, k_pool, v_pool,
                    page_table, seq_lens, max_seq_len: int, cu_new_lens=None,
                    max_new_len: Optional[int] = None, window: int = 0, num_sinks: int = 0, out=None,
                    workspace=None, softmax_scale: float = 0.0, status=None, stream=None):
    """fp16 [T][Hq][D] attention of the newest tokens' queries q [T][Hq][D] over the quantized
    pools, causal; row offsets cu_new_lens int32 [B + 1] (None: one row per sequence).
    max_new_len bounds the rows of every sequence and is needed with row offsets: a sequence
    with more is left out, which only `status` tells.  Rows that are left out, and rows behind
    the last sequence, stay as they are in `out` (undefined where it is made here).  With
    `window` a row sees that many last tokens and the first `num_sinks` (see vq_chunk_attention)."""
    if max_new_len is None:
        if cu_new_lens is not None:
            raise ValueError("max_new_len is needed with cu_new_lens")
        max_new_len = 1
    torch = _torch()
    dev = _need(q, "q")
    f16, i32, u8 = torch.float16, torch.int32, torch.uint8
    T, B, pages = q.shape[0], seq_lens.shape[0], k_pool.shape[0]
    L = layout
    D, H, P = L.head_dim, L.num_kv_heads, L.page_size
    rows = (T, L.num_q_heads, D)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B][max_pages]")
    width = page_table.shape[1]
    args = (_arg(q, f16, "q", dev, rows), _arg(lambda_, torch.float32, "lambda", dev, (H, D)),
            _arg(codebook_k, f16, "codebook_k", dev, (1 << L.k_bits, L.k_sub)),
            _arg(codebook_v, f16, "codebook_v", dev, (1 << L.v_bits, L.v_sub)),
            _arg(k_pool, u8, "k_pool", dev, (pages, H, P, (D // L.k_sub * L.k_bits + 31) // 32 * 4)),
            _arg(v_pool, u8, "v_pool", dev, (pages, H, P, (D // L.v_sub * L.v_bits + 31) // 32 * 4)),
            pages, _arg(page_table, i32, "page_table", dev, (B, width)), width,
            _arg(seq_lens, i32, "seq_lens", dev, (B,)), max_seq_len,
            _arg(cu_new_lens, i32, "cu_new_lens", dev, (B + 1,)), max_new_len, window, num_sinks,
            softmax_scale)

    def call(st):
        o = torch.empty(rows, dtype=f16, device=dev) if out is None else out
        w = workspace
        if w is None:
            w = alloc_chunk_workspace(layout, B, T, max_seq_len, max_new_len, dev)
        _check(lib().vq_chunk_attention(ctypes.byref(layout), B, T, *args, _arg(o, f16, "out", dev, rows),
                                        _arg(w, u8, "workspace", dev), w.numel(),
                                        _arg(status, i32, "status", dev, (1,)), st))
        return o

    return _launch(dev, stream, call)


class AppendedSlots(NamedTuple):
    seq_lens: object      # int32 [B]
    num_free: object      # int32 [1]
    cu_new_lens: object   # int32 [B + 1]
    slot_mapping: object  # int64 [max_tokens]
    positions: object     # int32 [max_tokens]


def append_slots(seq_lens, new_lens, page_table, free_pages, num_free, page_size: int,
                 num_pages: int, max_tokens: int, seq_lens_out=None, num_free_out=None,
                 cu_new_lens=None, slot_mapping=None, positions=None, status=None,
                 stream=None) -> AppendedSlots:
    """Page tables, slots, positions and row offsets of one step (see vq_append_slots):
    page_table [B][max_pages] is extended in place with pages off the free stack."""
    torch = _torch()
    dev, i32, i64 = _need(seq_lens, "seq_lens"), torch.int32, torch.int64
    B = seq_lens.shape[0]
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B][max_pages]")
    width, free = page_table.shape[1], free_pages.numel()
    args = (_arg(seq_lens, i32, "seq_lens", dev, (B,)), _arg(new_lens, i32, "new_lens", dev, (B,)),
            _arg(page_table, i32, "page_table", dev, (B, width)), width,
            _arg(free_pages, i32, "free_pages", dev, (free,)), free,
            _arg(num_free, i32, "num_free", dev, (1,)), page_size, num_pages, max_tokens)

    def call(st):
        empty = torch.empty
        r = AppendedSlots(empty(B, dtype=i32, device=dev) if seq_lens_out is None else seq_lens_out,
                          empty(1, dtype=i32, device=dev) if num_free_out is None else num_free_out,
                          empty(B + 1, dtype=i32, device=dev) if cu_new_lens is None else cu_new_lens,
                          empty(max_tokens, dtype=i64, device=dev) if slot_mapping is None else slot_mapping,
                          empty(max_tokens, dtype=i32, device=dev) if positions is None else positions)
        _check(lib().vq_append_slots(B, *args, _arg(r[0], i32, "seq_lens_out", dev, (B,)),
                                     _arg(r[1], i32, "num_free_out", dev, (1,)),
                                     _arg(r[2], i32, "cu_new_lens", dev, (B + 1,)),
                                     _arg(r[3], i64, "slot_mapping", dev, (max_tokens,)),
                                     _arg(r[4], i32, "positions", dev, (max_tokens,)),
                                     _arg(status, i32, "status", dev, (1,)), st))
        return r

    return _launch(dev, stream, call)


def _rows_arg(t, dtype, name, device, tokens, head_dim):
    """(data_ptr, token stride, heads) of [T][heads][D] rows whose heads are contiguous."""
    if t is None:
        return None, 0, 0
    if _need(t, name) != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != head_dim:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({tokens}, heads, {head_dim})")
    heads = t.shape[1]
    s0, s1, s2 = t.stride()
    if tokens and heads and (s2 != 1 or (heads > 1 and s1 != head_dim)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), s0 if tokens > 1 else heads * head_dim, heads


def rotary(config: vq_rotary_config, positions, q=None, k=None, v=None, q_out=None, k_out=None,
           v_out=None, stream=None):
    """(q, k, v) fp16 [T][heads][D]: q and k turned by positions (int32 [T]), v carried along.
    Inputs are fp16 or bf16, all of one type, and may be slices of one fused projection; one
    not given comes back as None.  An output may be its own (fp16, contiguous) input."""
    torch = _torch()
    some = q if q is not None else k if k is not None else v
    if some is None:
        raise ValueError("q, k and v are all None")
    dt, f16, dev = some.dtype, torch.float16, _need(some, "q, k or v")
    if dt is not f16 and dt is not torch.bfloat16:
        raise TypeError(f"q, k and v must be float16 or bfloat16, got {dt}")
    T, D = positions.shape[0], config.head_dim
    qp, qs, qh = _rows_arg(q, dt, "q", dev, T, D)
    kp, ks, kh = _rows_arg(k, dt, "k", dev, T, D)
    vp, vs, vh = _rows_arg(v, dt, "v", dev, T, D)
    if k is not None and v is not None and kh != vh:
        raise ValueError("k and v have different numbers of heads")
    for x, o, name in ((q, q_out, "q"), (k, k_out, "k"), (v, v_out, "v")):
        if x is None and o is not None:
            raise ValueError(f"{name}_out is given without {name}")
    pos = _arg(positions, torch.int32, "positions", dev, (T,))

    def call(st):
        def make(x, o, heads, name):
            if x is None:
                return None, None
            shape = (T, heads, D)
            if o is None:
                o = torch.empty(shape, dtype=f16, device=dev)
                return o, o.data_ptr()
            return o, _arg(o, f16, name, dev, shape)
        qo, qop = make(q, q_out, qh, "q_out")
        ko, kop = make(k, k_out, kh, "k_out")
        vo, vop = make(v, v_out, vh, "v_out")
        _check(lib().vq_rotary(ctypes.byref(config), T, pos, VQ_FP16 if dt is f16 else VQ_BF16, qp, qs, qh,
                               qop, kp, ks, vp, vs, kh or vh, kop, vop, st))
        return qo, ko, vo

    return _launch(dev, stream, call)


# ------------------------------------- torch layer: trees of drafted tokens ---

def alloc_tree_workspace(layout: vq_layout, batch: int, num_tokens: int, max_seq_len: int,
                         max_new_len: int, device="cuda"):
    torch = _torch()
    with torch.cuda.device(device):
        n = vq_tree_workspace_bytes(layout, batch, num_tokens, max_seq_len, max_new_len)
        if n == 0:
            raise VQError(VQ_ERR_INVALID_ARG, "cannot size the workspace")
        return torch.empty(n, dtype=torch.uint8, device="cuda")


def tree_attention(layout: vq_layout, q, lambda_, codebook_k, codebook_v, k_pool, v_pool,
                   page_table, seq_lens, max_seq_len: int, cu_new_lens, max_new_len: int, tree_masks,
                   positions=None, window: int = 0, num_sinks: int = 0, out=None, workspace=None,
                   softmax_scale: float = 0.0, status=None, stream=None):
    """fp16 [T][Hq][D] attention of trees of drafted tokens, queries q [T][Hq][D], over the quantized
    pools, which hold their codes already: each row sees the tokens before the drafted ones and of
    these the ones that its bits name.  tree_masks int64 [T][words], bit j of a row (bit j % 64 of
    word j // 64) for the sequence's j-th drafted token; up to max_new_len <= 256 per sequence.
    With `window` positions (int32 [T]) are needed (see vq_tree_attention).  Rows that are left
    out, and rows behind the last sequence, stay as they are in `out` (undefined where it is made
    here)."""
    torch = _torch()
    dev = _need(q, "q")
    f16, i32, u8 = torch.float16, torch.int32, torch.uint8
    T, B, pages = q.shape[0], seq_lens.shape[0], k_pool.shape[0]
    L = layout
    D, H, P = L.head_dim, L.num_kv_heads, L.page_size
    rows = (T, L.num_q_heads, D)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B][max_pages]")
    if tree_masks.dim() != 2:
        raise ValueError("tree_masks must be [T][words]")
    width, words = page_table.shape[1], tree_masks.shape[1]
    args = (_arg(q, f16, "q", dev, rows), _arg(lambda_, torch.float32, "lambda", dev, (H, D)),
            _arg(codebook_k, f16, "codebook_k", dev, (1 << L.k_bits, L.k_sub)),
            _arg(codebook_v, f16, "codebook_v", dev, (1 << L.v_bits, L.v_sub)),
            _arg(k_pool, u8, "k_pool", dev, (pages, H, P, (D // L.k_sub * L.k_bits + 31) // 32 * 4)),
            _arg(v_pool, u8, "v_pool", dev, (pages, H, P, (D // L.v_sub * L.v_bits + 31) // 32 * 4)),
            pages, _arg(page_table, i32, "page_table", dev, (B, width)), width,
            _arg(seq_lens, i32, "seq_lens", dev, (B,)), max_seq_len,
            _arg(cu_new_lens, i32, "cu_new_lens", dev, (B + 1,)), max_new_len,
            _arg(tree_masks, torch.int64, "tree_masks", dev, (T, words)), words,
            _arg(positions, i32, "positions", dev, (T,)), window, num_sinks, softmax_scale)

    def call(st):
        o = torch.empty(rows, dtype=f16, device=dev) if out is None else out
        w = workspace
        if w is None:
            w = alloc_tree_workspace(layout, B, T, max_seq_len, max_new_len, dev)
        _check(lib().vq_tree_attention(ctypes.byref(layout), B, T, *args, _arg(o, f16, "out", dev, rows),
                                       _arg(w, u8, "workspace", dev), w.numel(),
                                       _arg(status, i32, "status", dev, (1,)), st))
        return o

    return _launch(dev, stream, call)


def append_kv(layout: vq_layout, config: vq_rotary_config, positions, slot_mapping, k, v, lambda_, codebook_k,
              codebook_v, k_pool, v_pool, q=None, q_out=None, status=None, stream=None):
    """Append k and v [T][Hkv][D] to the pools at slot_mapping (int64 [T]), keys turned by positions
    (int32 [T]) on the way, and return q [T][Hq][D] turned (fp16; None without q): what rotary and
    encode_kv do, in one launch and without rounding the turned keys.  Inputs are fp16 or bf16,
    all of one type, and may be slices of one fused projection; q_out may be its own (fp16,
    contiguous) q."""
    torch = _torch()
    dev, dt, f16, u8 = _need(k, "k"), k.dtype, torch.float16, torch.uint8
    if dt is not f16 and dt is not torch.bfloat16:
        raise TypeError(f"q, k and v must be float16 or bfloat16, got {dt}")
    L = layout
    T, D, H, P, pages = positions.shape[0], L.head_dim, L.num_kv_heads, L.page_size, k_pool.shape[0]
    qp, qs, qh = _rows_arg(q, dt, "q", dev, T, D)
    kp, ks, kh = _rows_arg(k, dt, "k", dev, T, D)
    vp, vs, vh = _rows_arg(v, dt, "v", dev, T, D)
    if kh != H or vh != H or (q is not None and qh != L.num_q_heads):
        raise ValueError(f"q, k and v have {qh}, {kh} and {vh} heads, the layout has {L.num_q_heads} and {H}")
    if q is None and q_out is not None:
        raise ValueError("q_out is given without q")
    head = (ctypes.byref(config), T, _arg(positions, torch.int32, "positions", dev, (T,)),
            _arg(slot_mapping, torch.int64, "slot_mapping", dev, (T,)), VQ_FP16 if dt is f16 else VQ_BF16,
            qp, qs, kp, ks, vp, vs, _arg(lambda_, torch.float32, "lambda", dev, (H, D)),
            _arg(codebook_k, f16, "codebook_k", dev, (1 << L.k_bits, L.k_sub)),
            _arg(codebook_v, f16, "codebook_v", dev, (1 << L.v_bits, L.v_sub)))
    tail = (_arg(k_pool, u8, "k_pool", dev, (pages, H, P, (D // L.k_sub * L.k_bits + 31) // 32 * 4)),
            _arg(v_pool, u8, "v_pool", dev, (pages, H, P, (D // L.v_sub * L.v_bits + 31) // 32 * 4)), pages,
            _arg(status, torch.int32, "status", dev, (1,)))

    def call(st):
        o = q_out
        if q is not None and o is None:
            o = torch.empty((T, qh, D), dtype=f16, device=dev)
        _check(lib().vq_append_kv(ctypes.byref(layout), *head,
                                  None if q is None else _arg(o, f16, "q_out", dev, (T, qh, D)), *tail, st))
        return o

    return _launch(dev, stream, call)


class KeptTokens(NamedTuple):
    seq_lens: object  # int32 [B]
    num_free: object  # int32 [1]


def _layers_arg(pools, name, device, shape):
    """Device pointers of the layers' pools: one tensor [layers][..], or one tensor per layer.
    (Filled as an array of the standard library's: 1 us for 32 layers, as one of ctypes 3.)"""
    torch = _torch()
    if isinstance(pools, torch.Tensor):
        first = _arg(pools, torch.uint8, name, device, (pools.shape[0],) + shape)
        step, n = pools.stride(0), pools.shape[0]
        at = range(first, first + n * step, step) if n * step else [first] * n
    else:
        at = [_arg(x, torch.uint8, f"{name}[{i}]", device, shape) or 0 for i, x in enumerate(pools)]
    return (ctypes.c_uint64 * len(at)).from_buffer(array.array("Q", at))


def keep_tokens(layout: vq_layout, seq_lens, cu_new_lens, keep, keep_lens, page_table, k_pools, v_pools, free_pages,
                num_free, seq_lens_out=None, num_free_out=None, status=None, stream=None) -> KeptTokens:
    """Keep the accepted ones of a step's drafted tokens: those with indices keep[b][:keep_lens[b]]
    (int32 [B][max_keep], ascending) move together behind the context in the pools of all
    layers, and emptied pages go back on the free stack (see vq_keep_tokens).  k_pools and
    v_pools: one tensor [layers][pages][Hkv][P][row bytes], or a sequence of the layers' pools."""
    torch = _torch()
    dev, i32 = _need(seq_lens, "seq_lens"), torch.int32
    L = layout
    D, H, P, B = L.head_dim, L.num_kv_heads, L.page_size, seq_lens.shape[0]
    if page_table.dim() != 2 or keep.dim() != 2:
        raise ValueError("page_table and keep must be [B][max_pages] and [B][max_keep]")
    layers = len(k_pools)
    if layers != len(v_pools):
        raise ValueError("k_pools and v_pools have different numbers of layers")
    if layers == 0:
        raise ValueError("there are no pools")
    pages = k_pools.shape[1] if isinstance(k_pools, torch.Tensor) else k_pools[0].shape[0]
    width, most, free = page_table.shape[1], keep.shape[1], free_pages.numel()
    kp = _layers_arg(k_pools, "k_pools", dev, (pages, H, P, (D // L.k_sub * L.k_bits + 31) // 32 * 4))
    vp = _layers_arg(v_pools, "v_pools", dev, (pages, H, P, (D // L.v_sub * L.v_bits + 31) // 32 * 4))
    args = (_arg(seq_lens, i32, "seq_lens", dev, (B,)), _arg(cu_new_lens, i32, "cu_new_lens", dev, (B + 1,)),
            _arg(keep, i32, "keep", dev, (B, most)), most, _arg(keep_lens, i32, "keep_lens", dev, (B,)),
            _arg(page_table, i32, "page_table", dev, (B, width)), width, pages, layers,
            kp, vp, _arg(free_pages, i32, "free_pages", dev, (free,)), free, _arg(num_free, i32, "num_free", dev, (1,)))

    def call(st):
        r = KeptTokens(torch.empty(B, dtype=i32, device=dev) if seq_lens_out is None else seq_lens_out,
                       torch.empty(1, dtype=i32, device=dev) if num_free_out is None else num_free_out)
        _check(lib().vq_keep_tokens(ctypes.byref(layout), B, *args, _arg(r[0], i32, "seq_lens_out", dev, (B,)),
                                    _arg(r[1], i32, "num_free_out", dev, (1,)),
                                    _arg(status, i32, "status", dev, (1,)), st))
        if B == 0 and r.num_free is not num_free:  # (the call writes nothing then)
            r.num_free.copy_(num_free)
        return r

    return _launch(dev, stream, call)
