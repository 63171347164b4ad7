"""Thin binding of the serving operators (include/tfserve.h): the 8-bit KV
cache, attention over shared prefixes, and logit rows' log probabilities.

As in ``binding``: each function has the C name and marshals arguments only
(in _serve.so, compiled from csrc/serve_ext.cpp: at a decode step's sizes the
checks of a dozen tensors from Python would take longer than the call), raises
``TfError`` when the library returns a status other than TF_OK, and has no
fallback: without the built libraries every call raises.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import TF_OK, TfError, _stream

TF_KV_E4M3, TF_KV_INT8 = 1, 2
TF_DEV_BAD_TOKEN = 32

SERVE_EXPORTS = ("tf_kv_append_q8", "tf_kv_read_q8", "tf_paged_attn_q8", "tf_paged_attn_q8_workspace_bytes",
                 "tf_paged_attn_shared", "tf_paged_attn_shared_workspace_bytes", "tf_logprob_rows")

_lib = None
_ext = None


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("kv_type", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def load() -> ctypes.CDLL:
    """Load the library once and declare the signatures of tfserve.h."""
    global _lib
    if _lib is not None:
        return _lib
    lib = binding.load()
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.tf_kv_append_q8.argtypes = [P, P, i32, P, P, i32, P, i32, P, P, P, P]
    lib.tf_kv_read_q8.argtypes = [P, P, i32, P, i32, P, P, P, P, i32, P, P, P, P]
    lib.tf_paged_attn_q8.argtypes = [P, i32, i32, P, P, i32, P, i32, P, P, f32, i32, i32, i32, P, sz, P, i32, P, P, P]
    lib.tf_paged_attn_q8_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.tf_paged_attn_shared.argtypes = [P, i32, i32, P, P, i32, i32, i32, i32, P, i32, P, i32, P, P, i32, P, P, f32,
                                         i32, i32, i32, P, sz, P, i32, P, P, P]
    lib.tf_paged_attn_shared_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.tf_logprob_rows.argtypes = [P, i32, i32, i32, i64, f32, P, i32, P, P, P, i32, P, P, P, P, P]
    for name in SERVE_EXPORTS:
        getattr(lib, name).restype = sz if name.endswith("_bytes") else ctypes.c_int
    _lib = lib
    return lib


def _serve():
    """The compiled marshalling module, loaded once."""
    global _ext
    if _ext is None:
        load()
        try:
            from . import _serve as m
        except ImportError as e:
            raise RuntimeError("_serve.so is missing: build it with `python -m paged_kv_cache_segment_b200.build`") from e
        _ext = m
    return _ext


def _raw(stream):
    return None if stream is None else _stream(stream)


def _done(fn: str, rc: int):
    if rc != TF_OK:
        raise TfError(fn, rc)


def _dev(t: torch.Tensor, name: str, dtypes) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


class Q8Cache:
    """An 8-bit KV cache (tf_q8_cache): codes [n_pages][Hkv][P][D] (float8_e4m3fn or int8, which set the type) and
    scale bytes uint8 [n_pages][Hkv][P].  Holds the tensors it is made of; checked once, here."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale):
        if k_codes.dtype not in (torch.float8_e4m3fn, torch.int8):
            raise TypeError(f"codes have dtype {k_codes.dtype}, expected float8_e4m3fn or int8")
        if k_codes.dim() != 4 or v_codes.shape != k_codes.shape or v_codes.dtype != k_codes.dtype:
            raise ValueError("k_codes and v_codes must be [n_pages][Hkv][P][D] of one type")
        if tuple(k_scale.shape) != tuple(k_codes.shape[:3]) or k_scale.shape != v_scale.shape:
            raise ValueError("scales must be [n_pages][Hkv][P]")
        n_pages, hkv, psz, d = k_codes.shape
        self.tensors = (k_codes, v_codes, k_scale, v_scale)
        if len({t.device for t in self.tensors}) != 1:
            raise ValueError("the cache's tensors must be on one device")
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = n_pages, hkv, psz, d
        self.kv_type = TF_KV_E4M3 if k_codes.dtype == torch.float8_e4m3fn else TF_KV_INT8
        codes, u8 = (k_codes.dtype,), (torch.uint8,)
        self.struct = _CacheStruct(_dev(k_codes, "k_codes", codes), _dev(v_codes, "v_codes", codes),
                                   _dev(k_scale, "k_scale", u8), _dev(v_scale, "v_scale", u8), self.kv_type, n_pages,
                                   psz, hkv, d)
        self.address = ctypes.addressof(self.struct)
        self.device = k_codes.get_device()

    def here(self) -> int:
        """The struct's address, for a call on the cache's device (the calls check the other tensors')."""
        if self.device != torch._C._cuda_getDevice():
            raise ValueError("the cache must be on the current CUDA device")
        return self.address


def tf_kv_append_q8(k_rows, v_rows, cache, page_table, segs, *, status, segs_host=None, page_table_host=None,
                    stream=None):
    """Each stream's new rows [rows][Hkv][D], quantised into their pages (tf_kv_append_q8)."""
    _done("tf_kv_append_q8", _serve().kv_append_q8(k_rows, v_rows, cache.here(), page_table, segs, status, segs_host,
                                                   page_table_host, _raw(stream)))


def tf_kv_read_q8(cache, page_table, segs, k_pool, v_pool, dst_page_table, *, status, segs_host=None,
                  page_table_host=None, dst_page_table_host=None, stream=None):
    """The last n_rows keys of every stream from an 8-bit cache into bf16 pages (tf_kv_read_q8)."""
    _done("tf_kv_read_q8", _serve().kv_read_q8(cache.here(), page_table, segs, k_pool, v_pool, dst_page_table, status,
                                               segs_host, page_table_host, dst_page_table_host, _raw(stream)))


def tf_paged_attn_q8_workspace_bytes(n_rows_total: int, n_q_heads: int, head_dim: int, n_splits_max: int) -> int:
    return int(load().tf_paged_attn_q8_workspace_bytes(n_rows_total, n_q_heads, head_dim, n_splits_max))


def tf_paged_attn_q8(q, cache, page_table, segs, *, scale, n_splits_max, workspace, out, flags, status, split_keys=0,
                     full=False, segs_host=None, page_table_host=None, stream=None):
    """Attention over an 8-bit cache, partials and merge (tf_paged_attn_q8).  out dtype picks the output type:
    torch.bfloat16 or torch.float32."""
    _done("tf_paged_attn_q8", _serve().paged_attn_q8(q, cache.here(), page_table, segs, scale, full, split_keys,
                                                     n_splits_max, workspace, out, flags, status, segs_host,
                                                     page_table_host, _raw(stream)))


def tf_paged_attn_shared_workspace_bytes(n_rows_total: int, n_q_heads: int, head_dim: int, n_prefix_splits: int,
                                         n_splits_max: int) -> int:
    return int(load().tf_paged_attn_shared_workspace_bytes(n_rows_total, n_q_heads, head_dim, n_prefix_splits,
                                                           n_splits_max))


def tf_paged_attn_shared(q, k_pool, v_pool, page_table, prefixes, segs, *, scale, n_prefix_splits, n_splits_max,
                         workspace, out, flags, status, split_keys=0, prefixes_host=None, segs_host=None,
                         page_table_host=None, stream=None):
    """Attention of streams over shared prefixes and their own keys (tf_paged_attn_shared).  out dtype picks the
    output type: torch.bfloat16 or torch.float32."""
    _done("tf_paged_attn_shared", _serve().paged_attn_shared(
        q, k_pool, v_pool, page_table, prefixes, segs, scale, split_keys, n_prefix_splits, n_splits_max, workspace,
        out, flags, status, prefixes_host, segs_host, page_table_host, _raw(stream)))


def tf_logprob_rows(logits, tokens, *, token_logprobs, flags, status, entropy=None, lse=None, top_ids=None,
                    top_logprobs=None, scale=1.0, n_cols=None, stream=None):
    """Log probabilities of tokens [rows][n_tokens], entropy, log-sum-exp and the top alternatives (as many as
    top_ids has columns) of logit rows [rows][ld] over their first n_cols columns (tf_logprob_rows).  The logits are
    bf16 or f32 with unit column stride; rows may be strided."""
    _done("tf_logprob_rows", _serve().logprob_rows(logits, tokens, scale, n_cols, token_logprobs, entropy, lse,
                                                   top_ids, top_logprobs, flags, status, _raw(stream)))
