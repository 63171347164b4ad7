"""Thin ctypes binding of the serving operators (include/tfserve.h): the 8-bit
KV cache, attention over shared prefixes, and logit rows' log probabilities.

As in ``binding``: each function has the C name and marshals arguments only,
raises ``TfError`` when the library returns a status other than TF_OK, and has
no fallback.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import binding
from .binding import BF16, TF_OUT_BF16, TF_OUT_F32, _check, _stream

TF_KV_E4M3, TF_KV_INT8 = 1, 2
TF_DEV_BAD_TOKEN = 32

SERVE_EXPORTS = ("tf_kv_append_q8", "tf_kv_read_q8", "tf_paged_attn_q8", "tf_paged_attn_q8_workspace_bytes",
                 "tf_paged_attn_shared", "tf_paged_attn_shared_workspace_bytes", "tf_logprob_rows")

I32 = (torch.int32,)
STATUS = (torch.int32, torch.uint32)
OUT = (torch.float32, torch.bfloat16)

_lib = None


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


def _dev(t: torch.Tensor, name: str, dtypes) -> int:
    """The address of a contiguous tensor of the current CUDA device (kernels launch there)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _table(a):
    """A host table as contiguous int32 (kept alive by the caller) and its address; (None, None) for None."""
    if a is None:
        return None, None
    a = np.ascontiguousarray(a, np.int32)
    return a, a.__array_interface__["data"][0]


def _host_tables(segs, segs_host, page_table, page_table_host):
    """Host copies of a segment and a page table, as long as the device tables they copy."""
    sh, sp = _table(segs_host)
    ph, pp = _table(page_table_host)
    if sh is not None and sh.size != segs.numel():
        raise ValueError("segs_host and segs differ in length")
    if ph is not None and ph.size != page_table.numel():
        raise ValueError("page_table_host and page_table differ in length")
    return sh, sp, ph, pp


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
        """The struct's address, for a call on the cache's device."""
        if self.device != torch.cuda.current_device():
            raise ValueError("the cache must be on the current CUDA device")
        return self.address


def tf_kv_append_q8(k_rows, v_rows, cache, page_table, segs, *, status, segs_host=None, page_table_host=None,
                    stream=None):
    """Each stream's new rows [rows][Hkv][D], quantised into their pages (tf_kv_append_q8)."""
    lib = load()
    rows, hkv, d = k_rows.shape
    if (hkv, d) != (cache.n_kv_heads, cache.head_dim) or v_rows.shape != k_rows.shape:
        raise ValueError("rows / cache shapes disagree")
    sh, sp, ph, pp = _host_tables(segs, segs_host, page_table, page_table_host)
    _check("tf_kv_append_q8", lib.tf_kv_append_q8(
        _dev(k_rows, "k_rows", BF16), _dev(v_rows, "v_rows", BF16), rows, cache.here(),
        _dev(page_table, "page_table", I32), page_table.numel(), _dev(segs, "segs", I32), segs.numel() // 5, sp, pp,
        _dev(status, "status", STATUS), _stream(stream)))


def tf_kv_read_q8(cache, page_table, segs, k_pool, v_pool, dst_page_table, *, status, segs_host=None,
                  page_table_host=None, dst_page_table_host=None, stream=None):
    """The last n_rows keys of every stream from an 8-bit cache into bf16 pages (tf_kv_read_q8)."""
    lib = load()
    if tuple(k_pool.shape[1:]) != (cache.n_kv_heads, cache.page_size, cache.head_dim) or v_pool.shape != k_pool.shape:
        raise ValueError("pool / cache shapes disagree")
    if dst_page_table.numel() != page_table.numel():
        raise ValueError("page_table and dst_page_table differ in length")
    sh, sp, ph, pp = _host_tables(segs, segs_host, page_table, page_table_host)
    dh, dp = _table(dst_page_table_host)
    if dh is not None and dh.size != page_table.numel():
        raise ValueError("dst_page_table_host and dst_page_table differ in length")
    _check("tf_kv_read_q8", lib.tf_kv_read_q8(
        cache.here(), _dev(page_table, "page_table", I32), page_table.numel(), _dev(segs, "segs", I32),
        segs.numel() // 5, sp, pp, _dev(k_pool, "k_pool", BF16), _dev(v_pool, "v_pool", BF16), k_pool.shape[0],
        _dev(dst_page_table, "dst_page_table", I32), dp, _dev(status, "status", STATUS), _stream(stream)))


def tf_paged_attn_q8_workspace_bytes(n_rows_total: int, n_q_heads: int, head_dim: int, n_splits_max: int) -> int:
    return int(load().tf_paged_attn_q8_workspace_bytes(n_rows_total, n_q_heads, head_dim, n_splits_max))


def tf_paged_attn_q8(q, cache, page_table, segs, *, scale, n_splits_max, workspace, out, flags, status, split_keys=0,
                     full=False, segs_host=None, page_table_host=None, stream=None):
    """Attention over an 8-bit cache, partials and merge (tf_paged_attn_q8).  out dtype picks the output type:
    torch.bfloat16 or torch.float32."""
    lib = load()
    rows, hq, d = q.shape
    if d != cache.head_dim or out.shape != q.shape or tuple(flags.shape) != (rows, hq):
        raise ValueError("q / cache / out / flags shapes disagree")
    sh, sp, ph, pp = _host_tables(segs, segs_host, page_table, page_table_host)
    _check("tf_paged_attn_q8", lib.tf_paged_attn_q8(
        _dev(q, "q", BF16), rows, hq, cache.here(), _dev(page_table, "page_table", I32), page_table.numel(),
        _dev(segs, "segs", I32), segs.numel() // 5, sp, pp, scale, 1 if full else 0, split_keys, n_splits_max,
        _dev(workspace, "workspace", (torch.uint8,)), workspace.numel(), _dev(out, "out", OUT),
        TF_OUT_BF16 if out.dtype == torch.bfloat16 else TF_OUT_F32, _dev(flags, "flags", (torch.uint8,)),
        _dev(status, "status", STATUS), _stream(stream)))


def tf_paged_attn_shared_workspace_bytes(n_rows_total: int, n_q_heads: int, head_dim: int, n_prefix_splits: int,
                                         n_splits_max: int) -> int:
    return int(load().tf_paged_attn_shared_workspace_bytes(n_rows_total, n_q_heads, head_dim, n_prefix_splits,
                                                           n_splits_max))


def tf_paged_attn_shared(q, k_pool, v_pool, page_table, prefixes, segs, *, scale, n_prefix_splits, n_splits_max,
                         workspace, out, flags, status, split_keys=0, prefixes_host=None, segs_host=None,
                         page_table_host=None, stream=None):
    """Attention of streams over shared prefixes and their own keys (tf_paged_attn_shared).  out dtype picks the
    output type: torch.bfloat16 or torch.float32."""
    lib = load()
    rows, hq, d = q.shape
    n_pages, hkv, psz, d2 = k_pool.shape
    if d2 != d or v_pool.shape != k_pool.shape or out.shape != q.shape or tuple(flags.shape) != (rows, hq):
        raise ValueError("q / pool / out / flags shapes disagree")
    sh, sp, ph, pp = _host_tables(segs, segs_host, page_table, page_table_host)
    xh, xp = _table(prefixes_host)
    if xh is not None and xh.size != prefixes.numel():
        raise ValueError("prefixes_host and prefixes differ in length")
    _check("tf_paged_attn_shared", lib.tf_paged_attn_shared(
        _dev(q, "q", BF16), rows, hq, _dev(k_pool, "k_pool", BF16), _dev(v_pool, "v_pool", BF16), n_pages, psz, hkv, d,
        _dev(page_table, "page_table", I32), page_table.numel(), _dev(prefixes, "prefixes", I32),
        prefixes.numel() // 5, xp, _dev(segs, "segs", I32), segs.numel() // 5, sp, pp, scale, split_keys,
        n_prefix_splits, n_splits_max, _dev(workspace, "workspace", (torch.uint8,)), workspace.numel(),
        _dev(out, "out", OUT), TF_OUT_BF16 if out.dtype == torch.bfloat16 else TF_OUT_F32,
        _dev(flags, "flags", (torch.uint8,)), _dev(status, "status", STATUS), _stream(stream)))


def tf_logprob_rows(logits, tokens, *, token_logprobs, flags, status, entropy=None, lse=None, top_ids=None,
                    top_logprobs=None, scale=1.0, n_cols=None, stream=None):
    """Log probabilities of tokens [rows][n_tokens], entropy, log-sum-exp and the top alternatives (as many as
    top_ids has columns) of logit rows [rows][ld] over their first n_cols columns (tf_logprob_rows).  The logits are
    bf16 or f32 with unit column stride; rows may be strided."""
    lib = load()
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be 2-D with unit column stride")
    _dev(logits[:0], "logits", (logits.dtype,))
    if logits.dtype not in BF16 and logits.dtype != torch.float32:
        raise TypeError(f"logits have dtype {logits.dtype}, expected bfloat16 or float32")
    rows = logits.shape[0]
    ld = logits.stride(0) if rows > 1 else logits.shape[1]
    nc = logits.shape[1] if n_cols is None else int(n_cols)
    if nc > logits.shape[1]:
        raise ValueError("n_cols is past the logits' columns")
    if tokens.dim() != 2 or tokens.shape[0] != rows or token_logprobs.shape != tokens.shape:
        raise ValueError("tokens and token_logprobs must be [rows][n_tokens]")
    k = 0
    if top_ids is not None:
        k = top_ids.shape[1]
        if top_ids.shape[0] != rows or top_logprobs is None or top_logprobs.shape != top_ids.shape:
            raise ValueError("top_ids and top_logprobs must be [rows][top_k]")
    if any(x is not None and x.numel() != rows for x in (entropy, lse, flags)):
        raise ValueError("entropy, lse and flags must have a value a row")
    f32 = (torch.float32,)
    _check("tf_logprob_rows", lib.tf_logprob_rows(
        logits.data_ptr(), TF_OUT_F32 if logits.dtype == torch.float32 else TF_OUT_BF16, rows, nc, ld, scale,
        _dev(tokens, "tokens", I32), tokens.shape[1], _dev(token_logprobs, "token_logprobs", f32),
        None if entropy is None else _dev(entropy, "entropy", f32), None if lse is None else _dev(lse, "lse", f32), k,
        None if k == 0 else _dev(top_ids, "top_ids", I32), None if k == 0 else _dev(top_logprobs, "top_logprobs", f32),
        _dev(flags, "flags", (torch.uint8,)), _dev(status, "status", STATUS), _stream(stream)))
